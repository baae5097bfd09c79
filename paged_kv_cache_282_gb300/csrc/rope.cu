// rope.cu -- per-head norms and the position rotation of new queries and
// keys, in one pass with storing the keys and values in the paged pool
// (sm_103a).
//
// For a row x of one head (D values) of a token at position p:
//   y = x rsqrt(mean(x^2) + eps) w                       (w given; else y = x)
//   half pairing         (a, b) = (y_i, y_{i + r/2}),  i < r/2
//   interleaved pairing  (a, b) = (y_2i, y_2i+1),      i < r/2
//   (a, b) -> (a cos - b sin, b cos + a sin) with the table's angle p f_i
// over the first r = rot_dim values, the rest unchanged.  Everything is fp32
// and rounded once: to the output's type, or (FP8 / INT8 pools) straight to
// the codes of the row's own scale, as in the plain append.
//
// Each value is read once and written once, and the fp32 cos / sin rows (4 r
// bytes a token) are shared by all heads of a token: 16001 tokens of 32 + 8
// heads of 128 take 67 us, 4.9 TB/s or 0.72 of the copy rate, with the issue
// slots 72 % busy; neither is full.  A row is held by D es / 16 lanes with two
// 8-byte pieces each.  With half pairing the pieces are the two sides of the
// lane's pairs (past rot_dim, where nothing turns, two halves of the rest),
// with interleaved pairing neighbours: either way a pair lies in one lane, and
// only the sums and row maxima are shuffles.  (Rows of one 16-byte piece a
// lane, with the other side of a pair shuffled in, took 98.6 us there.)
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include <algorithm>

#include "pkv_internal.h"

namespace pkv {
namespace {

constexpr unsigned kFull = 0xffffffffu;

// Rows of 8-byte pieces: kPer values each.
template <int KV>
struct Elem {
  using T = __nv_bfloat16;
  static constexpr int kPer = 4;
};
template <>
struct Elem<0> {
  using T = float;
  static constexpr int kPer = 2;
};

template <int KV>
__device__ __forceinline__ void unpack(const uint2& r, float* x) {
  if constexpr (KV == 0) {
    x[0] = __uint_as_float(r.x), x[1] = __uint_as_float(r.y);
  } else {
    x[0] = __uint_as_float(r.x << 16), x[1] = __uint_as_float(r.x & 0xffff0000u);
    x[2] = __uint_as_float(r.y << 16), x[3] = __uint_as_float(r.y & 0xffff0000u);
  }
}

template <int KV>
__device__ __forceinline__ uint2 pack(const float* x) {
  if constexpr (KV == 0) {
    return make_uint2(__float_as_uint(x[0]), __float_as_uint(x[1]));
  } else {
    const __nv_bfloat162 lo = __floats2bfloat162_rn(x[0], x[1]), hi = __floats2bfloat162_rn(x[2], x[3]);
    return make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
  }
}

template <int N>
__device__ __forceinline__ void load_floats(const float* p, float* x) {  // 4 or 2, 4 N-byte aligned
  if constexpr (N == 4) {
    const float4 v = __ldg(reinterpret_cast<const float4*>(p));
    x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
  } else {
    const float2 v = __ldg(reinterpret_cast<const float2*>(p));
    x[0] = v.x, x[1] = v.y;
  }
}

// The code of x / sc.
template <int KV>
__device__ __forceinline__ uint32_t code_of(float x, float sc) {
  if constexpr (KV == 3) {
    const int n = __float2int_rn(__fdiv_rn(x, sc));
    return (uint32_t)(uint8_t)(int8_t)max(-127, min(127, n));
  } else {
    return __nv_cvt_float_to_fp8(__fdiv_rn(x, sc), __NV_SATFINITE, __NV_E4M3);
  }
}

// A block takes one token's rows (H query, Hk key, then Hv value rows), slot
// after slot, or several tokens' when its slots hold more than one: the
// position, the cos / sin and everything else of the token is then the same
// for all of a thread's rows.  B: rows whose loads a thread has in flight.
template <int KV, int D, int kThreads, int B>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeArgs a) {
  using T = typename Elem<KV>::T;
  constexpr int P = Elem<KV>::kPer, LPR = D / (2 * P);  // values per piece, lanes per row
  constexpr int kSlots = kThreads / LPR;
  for (int i = blockIdx.x * kThreads + threadIdx.x; i < a.n_patches; i += gridDim.x * kThreads) {
    const TablePatch* p = a.patches ? a.patches : a.inline_patches;
    a.tables[p[i].index] = p[i].value;
  }
  if (a.n_tokens == 0) return;
  const int R = a.H + a.Hk + a.Hv, lane = threadIdx.x % LPR, slot = threadIdx.x / LPR;
  const int per_block = R >= kSlots ? 1 : kSlots / R, sub = R >= kSlots ? 0 : slot / R;
  const int first = slot - sub * R;
  int t = blockIdx.x * per_block + sub;
  const bool live = sub < per_block && t < a.n_tokens;  // every lane stays for the shuffles
  if (!live) t = a.n_tokens - 1;
  // this lane's pairs q0 .. q0 + P - 1 and its pieces' first values
  const int rot = a.rot, half = rot >> 1, q0 = lane * P;
  const bool inside = q0 < half;
  const int pa = a.interleaved ? 2 * q0 : inside ? q0 : q0 + half;
  const int pb = a.interleaved ? pa + P : inside ? pa + half : pa + ((D - rot) >> 1);

  const TokenAt* toks = a.tokens ? a.tokens : a.inline_tokens;
  int64_t at = 0;
  int pos = 0;
  if (a.append) {
    const TokenAt ta = toks[t];
    at = ta.slot;
    pos = ta.pos;
  }
  if (a.positions) pos = a.positions[t];
  bool ok = live;
  if (rot > 0 && (pos < 0 || pos >= a.n_positions)) {
    if (live && lane == 0) {
      atomicOr(a.status, kStatusBadBlock);
      a.status[1] = t;
      a.status[2] = pos;
    }
    ok = false;  // no row of this token is written
    pos = 0;
  }
  float c[P], s[P];  // of this lane's pairs
#pragma unroll
  for (int e = 0; e < P; ++e) c[e] = 1.0f, s[e] = 0.0f;
  if (inside) {
    const float* row = a.cos_sin + (int64_t)pos * rot + q0;
    load_floats<P>(row, c);
    load_floats<P>(row + half, s);
  }
  // the lanes of this lane's row, for shuffles that other rows of the warp may skip
  const unsigned row_mask = LPR == 32 ? kFull : ((1u << (LPR % 32)) - 1u) << (threadIdx.x % 32 / LPR * LPR);
  const bool norms = a.q_weight != nullptr || a.k_weight != nullptr;

  const int64_t tok = ((at >> 4) * a.Hk) * kBlock + (at & 15);  // pool row of kv head 0
  const int rounds = R >= kSlots ? (R + kSlots - 1) / kSlots : 1;
  for (int i0 = 0; i0 < rounds; i0 += B) {
    uint2 raw[B][2];
#pragma unroll
    for (int i = 0; i < B; ++i) {
      const int r = min(first + (i0 + i) * kSlots, R - 1);
      const T* src = r < a.H          ? static_cast<const T*>(a.q) + (int64_t)t * a.q_stride + r * D
                     : r < a.H + a.Hk ? static_cast<const T*>(a.k) + (int64_t)t * a.k_stride + (r - a.H) * D
                                      : static_cast<const T*>(a.v) + (int64_t)t * a.v_stride + (r - a.H - a.Hk) * D;
      raw[i][0] = *reinterpret_cast<const uint2*>(src + pa);
      raw[i][1] = *reinterpret_cast<const uint2*>(src + pb);
    }
#pragma unroll
    for (int i = 0; i < B; ++i) {
      const int r1 = first + (i0 + i) * kSlots, r = min(r1, R - 1);
      const bool store = ok && r1 < R && (R >= kSlots || i0 + i == 0);
      const bool is_q = r < a.H, is_v = r >= a.H + a.Hk;
      float x[2 * P];
      unpack<KV>(raw[i][0], x);
      unpack<KV>(raw[i][1], x + P);
      bool copied = is_v || rot == 0;  // keeps its bits (NaNs' as well)
      if (norms) {
        float ss = 0.0f;
#pragma unroll
        for (int e = 0; e < 2 * P; ++e) ss += x[e] * x[e];
#pragma unroll
        for (int o = LPR / 2; o; o >>= 1) ss += __shfl_xor_sync(kFull, ss, o);
        const T* w = is_v ? nullptr : static_cast<const T*>(is_q ? a.q_weight : a.k_weight);
        if (w != nullptr) {
          float wv[2 * P];
          unpack<KV>(__ldg(reinterpret_cast<const uint2*>(w + pa)), wv);
          unpack<KV>(__ldg(reinterpret_cast<const uint2*>(w + pb)), wv + P);
          const float f = rsqrtf(ss * (1.0f / D) + a.eps);
#pragma unroll
          for (int e = 0; e < 2 * P; ++e) x[e] = x[e] * f * wv[e];
          copied = false;
        }
      }
      if (inside && !is_v) {
        if (a.interleaved) {
#pragma unroll
          for (int e = 0; e < P; ++e) {
            const float y0 = x[2 * e], y1 = x[2 * e + 1];
            x[2 * e] = y0 * c[e] - y1 * s[e];
            x[2 * e + 1] = y1 * c[e] + y0 * s[e];
          }
        } else {
#pragma unroll
          for (int e = 0; e < P; ++e) {
            const float y0 = x[e], y1 = x[P + e];
            x[e] = y0 * c[e] - y1 * s[e];
            x[P + e] = y1 * c[e] + y0 * s[e];
          }
        }
      }
      const int g = is_q ? 0 : r - a.H - (is_v ? a.Hk : 0);
      const int64_t srow = tok + g * kBlock;
      T* to_q = static_cast<T*>(a.q_out) + (int64_t)t * a.q_out_stride + r * D;
      auto put = [&](T* dst) {
        if (!store) return;
        *reinterpret_cast<uint2*>(dst + pa) = copied ? raw[i][0] : pack<KV>(x);
        *reinterpret_cast<uint2*>(dst + pb) = copied ? raw[i][1] : pack<KV>(x + P);
      };
      if constexpr (KV < 2) {
        put(is_q       ? to_q
            : a.append ? static_cast<T*>(is_v ? a.v_pool : a.k_pool) + srow * D
                       : static_cast<T*>(a.k_out) + (int64_t)t * a.k_out_stride + g * D);
      } else {  // appending only; every lane shares in the row maximum
        constexpr float kMaxCode = KV == 3 ? 127.0f : 448.0f;
        if (is_q) put(to_q);
        if (a.k_channel != nullptr && !is_q) {  // per-channel scales: x / c first
          const float* ch = (is_v ? a.v_channel : a.k_channel) + g * D;
#pragma unroll
          for (int e = 0; e < P; ++e) {
            x[e] = __fdiv_rn(x[e], ch[pa + e]);
            x[P + e] = __fdiv_rn(x[P + e], ch[pb + e]);
          }
        }
        if (r >= a.H) {
          float amax = 0.0f;
#pragma unroll
          for (int e = 0; e < 2 * P; ++e) amax = fmaxf(amax, fabsf(x[e]));
#pragma unroll
          for (int o = LPR / 2; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(row_mask, amax, o));
          if (!is_q && store) {
            const float sc = amax == 0.0f ? 1.0f : __fdiv_rn(amax, kMaxCode);
            uint32_t w[2] = {0, 0};
#pragma unroll
            for (int e = 0; e < 2 * P; ++e) w[e / P] |= code_of<KV>(x[e], sc) << (8 * (e % P));
            uint8_t* dst = static_cast<uint8_t*>(is_v ? a.v_pool : a.k_pool) + srow * D;
            *reinterpret_cast<uint32_t*>(dst + pa) = w[0];
            *reinterpret_cast<uint32_t*>(dst + pb) = w[1];
            if (lane == 0) (is_v ? a.v_scale : a.k_scale)[srow] = sc;
          }
        }
      }
    }
  }
}

template <int KV, int D, int kThreads>
void start(const RopeArgs& a, cudaStream_t st) {
  constexpr int kSlots = kThreads * 2 * Elem<KV>::kPer / D;
  const int R = a.H + a.Hk + a.Hv, per_block = R >= kSlots ? 1 : kSlots / R;
  const int grid = std::max((a.n_tokens + per_block - 1) / per_block, a.n_patches > 0 ? 1 : 0);
  if (grid <= 0) return;
  // Rows in flight a thread: up to 6, as many as waste the fewest loads in the
  // last round, the most of those.
  const int rounds = (R + kSlots - 1) / kSlots;
  int best = 1;
  for (int b = 2, least = rounds; b <= 6; ++b)
    if (const int used = (rounds + b - 1) / b * b; used <= least) best = b, least = used;
  switch (best) {
    case 1: rope_kernel<KV, D, kThreads, 1><<<grid, kThreads, 0, st>>>(a); break;
    case 2: rope_kernel<KV, D, kThreads, 2><<<grid, kThreads, 0, st>>>(a); break;
    case 3: rope_kernel<KV, D, kThreads, 3><<<grid, kThreads, 0, st>>>(a); break;
    case 4: rope_kernel<KV, D, kThreads, 4><<<grid, kThreads, 0, st>>>(a); break;
    case 5: rope_kernel<KV, D, kThreads, 5><<<grid, kThreads, 0, st>>>(a); break;
    default: rope_kernel<KV, D, kThreads, 6><<<grid, kThreads, 0, st>>>(a); break;
  }
}

// Blocks of 128 threads stream best (more tokens at different stages on an
// SM: 16001 tokens of 40 rows 69 us, with 256 threads 97 us); while all rows fit on the
// GPU at once, 512 threads give a token's rows the most lanes (128 tokens of 80 rows: 10 us
// against 15 us).
template <int KV, int D>
void start_d(const RopeArgs& a, cudaStream_t st) {
  const int64_t lanes = (int64_t)a.n_tokens * (a.H + a.Hk + a.Hv) * (D / (2 * Elem<KV>::kPer));
  if (lanes < (1 << 18))
    start<KV, D, 512>(a, st);
  else
    start<KV, D, 128>(a, st);
}

template <int KV>
void start_kv(const RopeArgs& a, cudaStream_t st) {
  if (a.D == 64)
    start_d<KV, 64>(a, st);
  else
    start_d<KV, 128>(a, st);
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, cudaStream_t st) {
  if (a.D != 64 && a.D != 128) return cudaErrorInvalidValue;
  switch (a.kv_dtype) {
    case 0: start_kv<0>(a, st); break;
    case 1: start_kv<1>(a, st); break;
    case 2: start_kv<2>(a, st); break;
    case 3: start_kv<3>(a, st); break;
    default: return cudaErrorInvalidValue;
  }
  return cudaGetLastError();
}

}  // namespace pkv
