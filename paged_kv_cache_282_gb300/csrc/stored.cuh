// stored.cuh -- values of a pool's rows as fp32, for code on the CUDA cores.
#pragma once

#include <cuda_fp8.h>
#include <stdint.h>

namespace pkv {
namespace {

// N neighbouring stored values from element i on (i a multiple of N), as one load.
template <int KV, int N>
__device__ __forceinline__ void load_values(const void* pool, size_t i, float* x) {
  if constexpr (KV == 0) {
    const float* at = static_cast<const float*>(pool) + i;
    if constexpr (N == 4) {
      const float4 v = __ldg(reinterpret_cast<const float4*>(at));
      x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
    } else {
      const float2 v = __ldg(reinterpret_cast<const float2*>(at));
      x[0] = v.x, x[1] = v.y;
    }
  } else if constexpr (KV == 1) {
    uint32_t w[N / 2];
    const uint16_t* at = static_cast<const uint16_t*>(pool) + i;
    if constexpr (N == 4) {
      const uint2 v = __ldg(reinterpret_cast<const uint2*>(at));
      w[0] = v.x, w[1] = v.y;
    } else {
      w[0] = __ldg(reinterpret_cast<const uint32_t*>(at));
    }
#pragma unroll
    for (int e = 0; e < N; ++e) x[e] = __uint_as_float(e & 1 ? w[e / 2] & 0xffff0000u : w[e / 2] << 16);
  } else {
    const uint8_t* at = static_cast<const uint8_t*>(pool) + i;
    uint32_t w;
    if constexpr (N == 4)
      w = __ldg(reinterpret_cast<const uint32_t*>(at));
    else
      w = __ldg(reinterpret_cast<const uint16_t*>(at));
#pragma unroll
    for (int e = 0; e < N; ++e) {
      const uint8_t c = (uint8_t)(w >> (8 * e));
      x[e] = KV == 2 ? __half2float(__half(__nv_cvt_fp8_to_halfraw(c, __NV_E4M3))) : (float)(int8_t)c;
    }
  }
}

// The values of 16 stored bytes.
template <int KV>
__device__ __forceinline__ void unpack16(uint4 u, float* x) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (KV == 0) {
      x[i] = __uint_as_float(w[i]);
    } else if constexpr (KV == 1) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint8_t c = (uint8_t)(w[i] >> (8 * e));
        x[4 * i + e] = KV == 2 ? __half2float(__half(__nv_cvt_fp8_to_halfraw(c, __NV_E4M3))) : (float)(int8_t)c;
      }
    }
  }
}

}  // namespace
}  // namespace pkv
