// prefill_simple.cu -- attention of several query tokens per sequence over
// the paged cache on the CUDA cores, for every kv dtype (sm_103a).
//
// For query token t of a sequence of L tokens, T of them queries, at position
// i = L - T + t, and query head h:
//   s_j = scale q K_j,   out = sum_j softmax(s)_j V_j,   lse = ln sum_j exp(s_j)
// over the kept keys j <= i, j < sinks or j > i - window.  fp32 throughout,
// with the running maximum and sum of an online softmax.
//
// fp32 pools, which have no tensor-core path, run on it, and calls of few rows
// over few keys in every pool.  One warp per (token, query head), 32 keys at a
// time: for the logits a lane takes a key, so that one exponential serves 32
// keys; for the values it takes D / 32 neighbouring columns, with kAt rows'
// loads in flight.  The group's warps keep the same keys and bring their rows
// to shared memory together.  Bound by instruction issue: fp32, 32 / 8 / 128, a
// prompt of 2048 takes 3.7 ms (9.3 with each lane reading its key's row from
// the pool, 6.8 with a key at a time and a 5-step shuffle for its logit), 16 x
// 4 tokens behind 4092 0.88 ms (1.75, 3.1); 8 rows over 64 keys 12 us.
#include <cuda_bf16.h>

#include "pkv_internal.h"
#include "stored.cuh"

namespace pkv {
namespace {

constexpr unsigned kFull = 0xffffffffu;

constexpr int kAt = 8;

template <int KV, int D>
__global__ void prefill_simple_kernel(const PrefillSimpleParams p) {
  constexpr int E = D / 32, kSize = KV == 0 ? 4 : KV == 1 ? 2 : 1, N = 16 / kSize, kLoads = D / N;
  constexpr int kRow = D * kSize / 16 + 1;  // a staged row in 16-byte pieces, padded: lanes in neighbouring rows meet no bank twice
  extern __shared__ float4 query[];  // [head of the group][D / 4], times K's channel scales; then 32 rows of K
  const int lane = threadIdx.x & 31, t = blockIdx.x, g = blockIdx.y;
  const int Hk = p.n_kv_heads, G = p.n_heads / Hk, h = g * G + (threadIdx.x >> 5);
  int b = 0;  // the sequence whose queries hold token t: the last with q_start <= t
  for (int hi = p.n_seqs; b + 1 < hi;) {
    const int mid = (b + hi) >> 1;
    if (p.seqs[mid].q_start <= t)
      b = mid;
    else
      hi = mid;
  }
  const PrefillSeq sq = p.seqs[b];
  const int i = sq.ctx_len - sq.q_len + (t - sq.q_start);  // query position
  const size_t qrow = ((size_t)t * p.n_heads + h) * D + lane * E;
  uint4* rows = reinterpret_cast<uint4*>(query + G * (D / 4));
  const float4* mine = query + (threadIdx.x >> 5) * (D / 4);
  float q[E], o[E];
  load_values<KV == 0 ? 0 : 1, E>(p.q, qrow, q);
#pragma unroll
  for (int e = 0; e < E; ++e) {
    o[e] = 0.0f;
    if (KV >= 2 && p.k_channel != nullptr) q[e] *= p.k_channel[g * D + lane * E + e];
    reinterpret_cast<float*>(query)[(threadIdx.x >> 5) * D + lane * E + e] = q[e];
  }
  float m = -INFINITY, l = 0.0f;  // l: the sum over this lane's keys
  bool bad = false;
  // The row's kept keys: [0, sinks) and [win, i].
  const int sinks = min(p.sinks, i + 1), win = max(sinks, i - p.window + 1), kept = sinks + max(0, i + 1 - win);
  for (int n0 = 0; n0 < kept; n0 += 32) {
    // Past the last key it is read again, and a bad block's rows are block
    // 0's, so that no load waits on a branch; neither counts.
    const int n = min(n0 + lane, kept - 1), j = n < sinks ? n : win + (n - sinks);
    const int blk = p.tables[(size_t)sq.seq_slot * p.max_blocks + j / kBlock];
    const bool good = blk >= 0 && blk < p.num_blocks, have = good && n0 + lane < kept;
    bad |= !good;
    const size_t row = ((size_t)(good ? blk : 0) * Hk + g) * kBlock + (j & 15);
    const float ks = KV >= 2 ? __ldg(p.k_scale + row) : 1.0f, vs = KV >= 2 ? __ldg(p.v_scale + row) : 1.0f;
    __syncthreads();  // the tile before is read
    constexpr int kBatch = kLoads < 8 ? kLoads : 8;
#pragma unroll 1
    for (int c0 = threadIdx.x; c0 < 32 * kLoads; c0 += kBatch * blockDim.x) {
      uint4 w[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int c = c0 + u * blockDim.x;  // 32 neighbours a warp: all of them in or out
        if (c >= 32 * kLoads) break;
        const size_t from = (size_t)__shfl_sync(kFull, (unsigned long long)row, c / kLoads) * kLoads + c % kLoads;
        w[u] = __ldg(static_cast<const uint4*>(p.k_pool) + from);
      }
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int c = c0 + u * blockDim.x;
        if (c < 32 * kLoads) rows[(c / kLoads) * kRow + c % kLoads] = w[u];
      }
    }
    __syncthreads();
    const uint4* kr = rows + lane * kRow;
    float part[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 1
    for (int c = 0; c < kLoads; c += kBatch) {
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        float x[N];
        unpack16<KV>(kr[c + u], x);
#pragma unroll
        for (int e = 0; e < N; e += 4) {
          const float4 y = mine[((c + u) * N + e) / 4];
          part[0] += y.x * x[e];
          part[1] += y.y * x[e + 1];
          part[2] += y.z * x[e + 2];
          part[3] += y.w * x[e + 3];
        }
      }
    }
    const float dot = (part[0] + part[1]) + (part[2] + part[3]);
    const float s = have ? dot * (ks * p.scale) : -INFINITY;
    float mn = fmaxf(m, s);
#pragma unroll
    for (int off = 16; off; off >>= 1) mn = fmaxf(mn, __shfl_xor_sync(kFull, mn, off));
    const float alpha = m == -INFINITY ? 0.0f : expf(m - mn);
    const float w = s == -INFINITY ? 0.0f : expf(s - mn), wv = w * vs;
    l = l * alpha + w;
    m = mn;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] *= alpha;
    const unsigned counts = __ballot_sync(kFull, have);
    const int keys = min(32, kept - n0);
#pragma unroll 1
    for (int u0 = 0; u0 < keys; u0 += kAt) {
      float v[kAt][E];
#pragma unroll
      for (int u = 0; u < kAt; ++u)
        load_values<KV, E>(p.v_pool, (size_t)__shfl_sync(kFull, (unsigned long long)row, u0 + u) * D + lane * E, v[u]);
#pragma unroll
      for (int u = 0; u < kAt; ++u) {
        const float wu = __shfl_sync(kFull, wv, u0 + u);
        if ((counts >> (u0 + u)) & 1) {
#pragma unroll
          for (int e = 0; e < E; ++e) o[e] += wu * v[u][e];
        }
      }
    }
  }
#pragma unroll
  for (int off = 16; off; off >>= 1) l += __shfl_xor_sync(kFull, l, off);
  if (bad) atomicOr(p.status, kStatusBadBlock);
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    o[e] = l == 0.0f ? 0.0f : o[e] * inv;  // (weights of zero: o may be NaN)
    if (KV >= 2 && p.v_channel != nullptr) o[e] *= p.v_channel[g * D + lane * E + e];
  }
  if constexpr (KV == 0) {
    float* out = static_cast<float*>(p.out) + qrow;
#pragma unroll
    for (int e = 0; e < E; e += 2) *reinterpret_cast<float2*>(out + e) = make_float2(o[e], o[e + 1]);
  } else {
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out) + qrow;
#pragma unroll
    for (int e = 0; e < E; e += 2)
      *reinterpret_cast<__nv_bfloat162*>(out + e) = __floats2bfloat162_rn(o[e], o[e + 1]);
  }
  if (p.lse != nullptr && lane == 0) p.lse[(size_t)t * p.n_heads + h] = l == 0.0f ? -INFINITY : m + logf(l);
}

template <int KV>
void start(const PrefillSimpleParams& p, cudaStream_t st) {
  const dim3 grid((unsigned)p.n_tokens, (unsigned)p.n_kv_heads);
  const int threads = 32 * (p.n_heads / p.n_kv_heads);
  const size_t row = (size_t)p.head_dim * (KV == 0 ? 4 : KV == 1 ? 2 : 1) + 16;
  const size_t smem = (size_t)threads / 32 * p.head_dim * sizeof(float) + 32 * row;
  if (p.head_dim == 64)
    prefill_simple_kernel<KV, 64><<<grid, threads, smem, st>>>(p);
  else
    prefill_simple_kernel<KV, 128><<<grid, threads, smem, st>>>(p);
}

}  // namespace

cudaError_t launch_prefill_simple(const PrefillSimpleParams& p, cudaStream_t st) {
  if (p.n_tokens <= 0) return cudaSuccess;
  switch (p.kv_dtype) {
    case 0: start<0>(p, st); break;
    case 1: start<1>(p, st); break;
    case 2: start<2>(p, st); break;
    case 3: start<3>(p, st); break;
    default: return cudaErrorInvalidValue;
  }
  return cudaGetLastError();
}

}  // namespace pkv
