// prefill_tc.cuh -- attention of several query tokens per sequence over the
// paged cache on the tensor cores: BF16, FP8-E4M3 and INT8 KV, head_dim D in
// {64, 128}, group G in {1, 2, 4, 8}; sm_103a.  Included by one translation
// unit per head_dim.
//
// For a query row q at position i:  s_j = scale q K_j over the kept keys
// j <= i;  out = sum_j 2^(c s_j - m) V_j / sum_j 2^(c s_j - m), c = log2 e.
//
// One CTA per SM walks its pieces.  A piece takes two tiles of 128 query rows
// (the G heads of a kv head are rows, so its K / V are read once for all of
// them) through a run of 128-key tiles:
//   S_i = Q_i K^T              tcgen05, operands in shared memory, S in TMEM
//   P_i = 2^(c scale S_i - m)  a thread per row, P (bf16) over S in TMEM
//   O_i += P_i V               tcgen05, P from TMEM, V from shared memory
// While the tensor core works for one tile, the other tile's threads take
// exponentials.  Roles: 4 softmax warps for each tile, then one warp that
// issues the products and two that load Q and K, and V; for one-byte pools
// these load Q and the scales, and 8 more warps widen the codes to bf16
// (exact: 8 significant bits hold both kinds).
//
// What bounds it: in bf16 the chain of a query tile, S -> P (about 1300 clocks
// with the other tile's threads beside it) -> O and the next S (1024 clocks of
// products, 2048 with the other tile's): an 8192-token prompt of 32 / 8 heads of
// 128 takes 364 us, 1510 TFLOP/s at 2070 MHz.  In one-byte pools no unit is full
// either (FP8: issue slots 55 % busy, tensor pipe 41 %; INT8 at D = 64: 47 % and
// 18 %): a key tile takes 4900 clocks, 2048 of products (D = 64: 4600, 1024), in
// the same chain, with widening beside the exponentials and on fewer registers.
// Which wait of it is the longest has not been told apart.  2048 tokens at
// 30719 in an FP8 pool take 988 us, 1077 TFLOP/s.
//
// The order of issue, PV_i(k) then QK_i(k + 1), makes the arrival of S_i(k + 1)
// also say that O_i holds tile k.  A row's reference m is known before the
// tile, so the exponentials need no pass over S first (a row's first tile has
// one, for its maximum).  When a tile's weights sum to more than 1024, m moves
// by the sum's logarithm and the row's O and sum are rescaled before the next
// tile: rare after the first tiles.  Logits that rise by more than about 87
// from one tile to the next leave fp32's range: the tile's sum is infinite, or
// the factor for what came before no normal number.  The factor is then NaN,
// which stays in the row's O and sum.
//
// One-byte pools: logits are scaled by the token's K scale in fp32, weights
// by its V scale before their rounding to bf16; per-channel scales (powers of
// two) go into the widened codes.
//
// Keys a row does not keep get weight 0, but 0 times a NaN or infinity of V
// would still reach the row.  Slots past the sequence's end (never written)
// are zeroed in shared memory; for written ones, a row whose O or sum is not
// finite is computed again key by key on the CUDA cores.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "pkv_internal.h"
#include "stored.cuh"
#include "tensor_core.cuh"

namespace pkv {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr int kTile = kPreBlocks * kBlock;  // keys of a key tile
constexpr int kChunk = 32;                  // logits a softmax thread takes at a time
constexpr uint64_t kDrainNs = 50000000ull;

// K and V stages hold groups of 8 keys, each [64-value column][8 rows][128
// bytes] with the 128-byte swizzle: a block's 16 keys arrive in one box, and
// both products step from group to group evenly.
template <int KV, int D>
struct PC {
  static constexpr bool kOneByte = KV != 1;
  static constexpr int kSoft = 256;                  // softmax threads, one per query row
  static constexpr int kWiden = kOneByte ? 256 : 0;  // threads that widen codes
  static constexpr int kThreads = kSoft + 128 + kWiden;
  static constexpr int kHalf = kTile * 128;          // bytes of 128 rows x 64 values
  static constexpr int kOperand = kHalf * (D / 64);  // a Q tile, a K or V stage
  static constexpr int kGroup = 1024 * (D / 64);     // bytes of 8 keys
  static constexpr int kStages = D == 128 ? (kOneByte ? 3 : 4) : 8;
  static constexpr int kRaw = kOneByte ? kTile * D : 0;  // bytes of an operand's codes
  static constexpr int kScaleStages = kOneByte ? 4 : 0;
  static constexpr int kScale = kTile * 4 * 2;  // bytes of a tile's K and V scales
  static constexpr int kOut = 32 * 32;          // bytes of a softmax warp's output staging
  // offsets from a 1024-byte boundary
  static constexpr int kQ = 0;
  static constexpr int kStage = kQ + kPreTiles * kOperand;
  static constexpr int kRawAt = kStage + kStages * kOperand;
  static constexpr int kScaleAt = kRawAt + 2 * kRaw;
  static constexpr int kOutAt = kScaleAt + kScaleStages * kScale;
  static constexpr int kBars = kOutAt + kSoft / 32 * kOut;
  static constexpr int kNumBars = 2 + 3 * kStages + 2 * kScaleStages + 11;
  static constexpr int kBytes = 1024 + kBars + kNumBars * 8;
  static_assert(kBytes + 64 <= 232448, "shared memory of a CTA");
  // registers per thread: softmax (more than the launch gives), then products
  // and loads, and widening (fewer).  In one-byte pools they do not quite hold
  // the softmax: 100 bytes are spilled at D = 128, 36 at D = 64.
  static constexpr int kSoftRegs = kOneByte ? 144 : 208, kIssueRegs = kOneByte ? 64 : 88, kWidenRegs = 64;
  static constexpr int kLaunchRegs = 65536 / kThreads / 8 * 8;
  static_assert(kSoftRegs > kLaunchRegs && kIssueRegs < kLaunchRegs && kWidenRegs < kLaunchRegs, "");
  static_assert(kSoft * kSoftRegs + 128 * kIssueRegs + kWiden * kWidenRegs <= kLaunchRegs * kThreads, "");
};

// Shared-memory addresses and limits every role uses.
template <int KV, int D>
struct Ctx {
  using C = PC<KV, D>;
  uint32_t base;  // of shared memory, on a 1024-byte boundary
  volatile int* abort;  // [0]: a wait ran out; [1]: key tiles that rows were computed over key by key
  uint64_t limit_ns;
  __device__ uint32_t q(int tile) const { return base + C::kQ + tile * C::kOperand; }
  __device__ uint32_t stage(int s) const { return base + C::kStage + s * C::kOperand; }
  __device__ uint32_t raw(int s) const { return base + C::kRawAt + s * C::kRaw; }
  __device__ uint32_t scales(int s) const { return base + C::kScaleAt + s * C::kScale; }
  __device__ uint32_t out(int warp) const { return base + C::kOutAt + warp * C::kOut; }
  __device__ uint32_t bar(int i) const { return base + C::kBars + i * 8; }
  __device__ uint32_t q_full() const { return bar(0); }
  __device__ uint32_t q_empty() const { return bar(1); }
  __device__ uint32_t full(int s) const { return bar(2 + s); }
  __device__ uint32_t empty(int s) const { return bar(2 + C::kStages + s); }
  __device__ uint32_t tail(int s) const { return bar(2 + 2 * C::kStages + s); }  // its unread V rows are zero
  __device__ uint32_t sc_full(int s) const { return bar(2 + 3 * C::kStages + s); }
  __device__ uint32_t sc_empty(int s) const { return bar(2 + 3 * C::kStages + C::kScaleStages + s); }
  __device__ uint32_t s_full(int i) const { return bar(C::kNumBars - 11 + i); }
  __device__ uint32_t p_full(int i, int half) const { return bar(C::kNumBars - 9 + 2 * i + half); }
  __device__ uint32_t o_full(int i) const { return bar(C::kNumBars - 5 + i); }
  __device__ uint32_t written() const { return bar(C::kNumBars - 3); }  // a piece's partial record
  __device__ uint32_t counted() const { return bar(C::kNumBars - 2); }  // and its merge item's counter
  __device__ uint32_t idle() const { return bar(C::kNumBars - 1); }     // every product is done

  // Waits for phase `parity`; false when the limit ran out here or elsewhere
  // in the CTA (every role then leaves).  Rows computed key by key can take
  // longer than the limit: as long as they go on, the time starts anew.
  __device__ bool wait_one(uint32_t bar, uint32_t parity, int32_t* status) const {
    if (mbar_try_wait(bar, parity)) return true;
    uint64_t t0 = global_timer();
    int steps = abort[1];
    for (uint32_t it = 1;; ++it) {
      if (mbar_try_wait(bar, parity)) return true;
      if ((it & 63) == 0) {
        if (abort[0]) return false;
        if (global_timer() - t0 > limit_ns) {
          if (abort[1] != steps) {
            steps = abort[1];
            t0 = global_timer();
            continue;
          }
          abort[0] = 1;
          atomicOr(status, kStatusTimeout);
          return false;
        }
      }
    }
  }
  // The same for a whole warp: all its lanes get the same answer.
  __device__ bool wait(uint32_t bar, uint32_t parity, int32_t* status) const {
    return __all_sync(kFull, wait_one(bar, parity, status));
  }
};

// A ring position: stage and the parity of its current round.
struct Ring {
  int stage = 0;
  uint32_t round = 0;
  __device__ void next(int n, int steps = 1) {
    stage += steps;
    if (stage >= n) {
      stage -= n;
      round ^= 1;
    }
  }
};

// A piece, with the next one on its way to L1.
__device__ __forceinline__ PrefillPiece piece_at(const PrefillTCParams& p, int ip, int last) {
  if (ip + 1 < last) asm volatile("prefetch.global.L1 [%0];" ::"l"(p.pieces + ip + 1));
  return p.pieces[ip];
}

__device__ __forceinline__ int tiles_a(const PrefillPiece& pc) { return (pc.a1 - pc.a0 + kPreBlocks - 1) / kPreBlocks; }
// First logical block of key tile k, and its number of blocks.
__device__ __forceinline__ int tile_block(const PrefillPiece& pc, int na, int k, int& n) {
  const int lo = k < na ? pc.a0 + kPreBlocks * k : pc.b0 + kPreBlocks * (k - na);
  n = min(kPreBlocks, (k < na ? pc.a1 : pc.b1) - lo);
  return lo;
}
// Positions of tile i's first and last query; none: last < first.
struct Span {
  int lo, hi;
};
__device__ __forceinline__ Span tile_span(const PrefillPiece& pc, int i, int g_log2) {
  const int per = kPreRows >> g_log2;
  return {pc.pos0 + i * per, pc.pos0 + min(pc.n_tok, (i + 1) * per) - 1};
}
// Key tiles that a query tile takes part in: k < a_end, and b_lo <= k < b_hi.
// They hold every key that one of its rows keeps (and, where the sinks' range
// runs into the window's, tiles between the two).
struct Part {
  int a_end, b_lo, b_hi;
  __device__ bool has(int k) const { return k < a_end || (k >= b_lo && k < b_hi); }
  // The last of them in [k0, k1), or -1.
  __device__ int last(int k0, int k1) const {
    if (min(b_hi, k1) > max(b_lo, k0)) return min(b_hi, k1) - 1;
    return min(a_end, k1) > k0 ? min(a_end, k1) - 1 : -1;
  }
};
__device__ __forceinline__ Part part_of(const PrefillPiece& pc, int na, const Span& s, int sinks, int window) {
  if (s.hi < s.lo) return {0, 0, 0};
  const int end = s.hi / kBlock, start = max(0, s.lo - window + 1) / kBlock;  // last and first block of the window
  const int nb = (pc.b1 - pc.b0 + kPreBlocks - 1) / kPreBlocks;
  const int hi = end < pc.b0 ? 0 : min(nb, (end - pc.b0) / kPreBlocks + 1);
  const int lo = na == 0 && sinks > 0 ? 0 : max(0, start - pc.b0) / kPreBlocks;
  return {min(na, (end - pc.a0) / kPreBlocks + 1), na + lo, na + hi};
}
__device__ __forceinline__ bool keeps(int j, int i, int sinks, int window) {
  return j <= i && (j < sinks || j > i - window);
}

__device__ __forceinline__ int block_of(const PrefillTCParams& p, const PrefillPiece& pc, int lb) {
  const int blk = p.tables[(size_t)pc.seq_slot * p.max_blocks + lb];
  if (blk >= 0 && blk < p.num_blocks) return blk;
  atomicOr(p.status, kStatusBadBlock);
  p.status[1] = pc.seq_slot;
  p.status[2] = lb;
  return 0;  // keeps the copy in bounds; the status word reports the fault
}

// ---- loads -------------------------------------------------------------------

// Waits for the copies this warp has in flight, before it leaves: a wait that
// fails elsewhere can end the CTA at any time after that, and shared memory
// must not be written then.
template <int KV, int D>
__device__ void drain(const PrefillTCParams& p, const Ctx<KV, D>& x, int first, int issued, int q_issued, int lane,
                      bool starved = false) {
  using C = PC<KV, D>;
  bool drained = true;
  for (int v = max(first, issued - C::kStages); v < issued; ++v)
    if ((v - first) % 2 == 0 && !(starved && v == first)) drained &= mbar_wait(x.full(v % C::kStages), (v / C::kStages) & 1, kDrainNs);
  if (q_issued > 0) drained &= mbar_wait(x.q_full(), (q_issued - 1) & 1, kDrainNs);
  if (!drained && lane == 0) atomicOr(p.status, kStatusUndrained);
}

// The queries of a piece.
template <int KV, int D>
__device__ __forceinline__ void load_q(const PrefillTCParams& p, const Ctx<KV, D>& x, const PrefillPiece& pc, int lane) {
  using C = PC<KV, D>;
  const int per = kPreRows >> p.g_log2, tiles = pc.n_tok > per ? 2 : 1;
  if (lane == 0) {
    mbar_expect_tx(x.q_full(), tiles * C::kOperand);
    for (int i = 0; i < tiles; ++i)
#pragma unroll
      for (int h = 0; h < D / 64; ++h)
        tma_load_3d(x.q(i) + h * C::kHalf, &p.tmap_q, h * 64, pc.kv_head << p.g_log2, pc.q_row + i * per, x.q_full());
  }
  __syncwarp();
}

// bf16 pools: one warp (IS_V false) loads the key tiles into the ring's even
// positions and the queries, another the value tiles into the odd ones.  Lane
// l takes block l of a tile, in one box.
template <int D, bool IS_V>
__device__ void load_role(const PrefillTCParams& p, const Ctx<1, D>& x, int first, int last, int lane) {
  using C = PC<1, D>;
  Ring ring;
  ring.stage = IS_V ? 1 : 0;
  int pieces = 0, issued = IS_V ? 1 : 0;  // ring positions passed, for the drain
  const bool starve = IS_V && p.starve && blockIdx.x == 0;
  bool ok = true;
  // A tile past whose `valid` keys V is to read as zeros once it landed
  // (slots never written, blocks past the run: their weight is 0, which needs
  // a finite value): done behind the next load, so that this one overlaps it.
  int tail_valid = kTile;
  Ring tail;
  auto zero_tail = [&]() {
    if (tail_valid == kTile) return true;
    if (!x.wait(x.full(tail.stage), tail.round, p.status)) return false;
    for (int c = lane; c < (kTile - tail_valid) * (D / 8); c += 32) {
      const int row = tail_valid + c / (D / 8), part = c % (D / 8);
      asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(x.stage(tail.stage) + (row / 8) * C::kGroup +
                                                                    (part / 8) * 1024 + (row % 8) * 128 + (part % 8) * 16),
                   "r"(0)
                   : "memory");
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
    if (lane == 0) mbar_arrive(x.tail(tail.stage));
    tail_valid = kTile;
    return true;
  };
  for (int ip = first; ip < last && ok; ++ip) {
    const PrefillPiece pc = piece_at(p, ip, last);
    if (pc.k0 >= pc.k1) continue;
    const int na = tiles_a(pc);
    int n, nn = 0;
    int lb = tile_block(pc, na, pc.k0, n), lb1 = lb;
    int blk = lane < n ? block_of(p, pc, lb + lane) : 0;
    for (int k = pc.k0; k < pc.k1; ++k) {
      ok = x.wait(x.empty(ring.stage), ring.round ^ 1, p.status);
      if (!ok) break;
      if (lane == 0) mbar_expect_tx(x.full(ring.stage), n * kBlock * D * 2);
      __syncwarp();
      if (lane < n && !(starve && issued == 1)) {
        const int group = (blk * p.n_kv_heads + pc.kv_head) * (kBlock / 8);
        tma_load_4d(x.stage(ring.stage) + lane * 2 * C::kGroup, IS_V ? &p.tmap_v : &p.tmap_k, 0, 0, 0, group,
                    x.full(ring.stage));
      }
      issued += 2;
      if constexpr (IS_V) {
        ok = zero_tail();
        if (!ok) break;
        const int valid = min(n * kBlock, pc.ctx_len - lb * kBlock);
        if (valid < kTile) {
          tail_valid = valid;
          tail = ring;
        }
      }
      ring.next(C::kStages, 2);
      if (k + 1 < pc.k1) {  // the next tile's table entries
        lb1 = tile_block(pc, na, k + 1, nn);
        blk = lane < nn ? block_of(p, pc, lb1 + lane) : 0;
      }
      if (!IS_V && k == pc.k0) {  // the piece's queries, behind its first keys
        if (pieces > 0) {
          ok = x.wait(x.q_empty(), (pieces - 1) & 1, p.status);
          if (!ok) break;
        }
        load_q(p, x, pc, lane);
        ++pieces;
      }
      n = nn;
      lb = lb1;
    }
  }
  if (IS_V && ok) ok = zero_tail();
  drain(p, x, IS_V ? 1 : 0, issued, pieces, lane, starve);
}

// One-byte pools: one warp loads the queries only.
template <int KV, int D>
__device__ void query_role(const PrefillTCParams& p, const Ctx<KV, D>& x, int first, int last, int lane) {
  int pieces = 0;
  bool ok = true;
  for (int ip = first; ip < last && ok; ++ip) {
    const PrefillPiece pc = piece_at(p, ip, last);
    if (pc.k0 >= pc.k1) continue;
    if (pieces > 0) ok = x.wait(x.q_empty(), (pieces - 1) & 1, p.status);
    if (!ok) break;
    load_q(p, x, pc, lane);
    ++pieces;
  }
  drain(p, x, 0, 0, pieces, lane);
}

// One-byte pools: one warp brings the tiles' scales, the keys' times the
// logits' factor.  Lane l takes 4 keys of block l / 4.
template <int KV, int D>
__device__ void scale_role(const PrefillTCParams& p, const Ctx<KV, D>& x, int first, int last, int lane) {
  using C = PC<KV, D>;
  const float c = p.scale * kLog2e;
  Ring ring;
  for (int ip = first; ip < last; ++ip) {
    const PrefillPiece pc = piece_at(p, ip, last);
    const int na = tiles_a(pc);
    for (int k = pc.k0; k < pc.k1; ++k) {
      int n;
      const int lb = tile_block(pc, na, k, n), b = lane / 4;
      float4 ks = make_float4(0.f, 0.f, 0.f, 0.f), vs = ks;
      if (b < n) {
        const size_t row = ((size_t)block_of(p, pc, lb + b) * p.n_kv_heads + pc.kv_head) * kBlock + (lane % 4) * 4;
        ks = __ldg(reinterpret_cast<const float4*>(p.k_scale + row));
        vs = __ldg(reinterpret_cast<const float4*>(p.v_scale + row));
      }
      if (!x.wait(x.sc_empty(ring.stage), ring.round ^ 1, p.status)) return;
      const uint32_t at = x.scales(ring.stage) + lane * 16;
      asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(at), "f"(ks.x * c), "f"(ks.y * c), "f"(ks.z * c),
                   "f"(ks.w * c)
                   : "memory");
      asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(at + kTile * 4), "f"(vs.x), "f"(vs.y), "f"(vs.z),
                   "f"(vs.w)
                   : "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive(x.sc_full(ring.stage));
      ring.next(C::kScaleStages);
    }
  }
}

// ---- products ----------------------------------------------------------------

// One thread issues everything.
template <int KV, int D>
__device__ void product_role(const PrefillTCParams& p, const Ctx<KV, D>& x, uint32_t tmem, int first, int last) {
  using C = PC<KV, D>;
  constexpr uint32_t kQK = mma_desc(kPreRows, kTile, false), kPV = mma_desc(kPreRows, D, true);
  Ring ring;  // the next stage to wait for
  uint32_t p_round[2] = {0, 0};
  uint32_t q_round = 0, tail_rounds = 0;  // tail_rounds: one bit per stage
  bool ok = true;

  // S_i = Q_i K^T from stage s
  auto qk = [&](int i, int s) {
    const uint32_t a = desc_low(x.q(i), 16), b = desc_low(x.stage(s), 16);
#pragma unroll
    for (int d = 0; d < D / 16; ++d)
      mma_smem(tmem + i * kTile, a + (((d / 4) * C::kHalf + (d % 4) * 32) >> 4), desc_high(1024),
               b + (((d / 4) * 1024 + (d % 4) * 32) >> 4), desc_high(C::kGroup), kQK, d > 0);
    mma_commit(x.s_full(i));
  };
  // O_i (+)= P_i V over half of the keys, from stage s
  auto pv = [&](int i, int s, int half, bool add) {
    const uint32_t b = desc_low(x.stage(s), 1024) + half * (kTile / 32) * (2 * C::kGroup >> 4);
#pragma unroll
    for (int u = 0; u < kTile / 32; ++u)
      mma_tmem(tmem + 2 * kTile + i * 128, tmem + i * kTile + half * (kTile / 4) + u * 8, b + u * (2 * C::kGroup >> 4),
               desc_high(C::kGroup), kPV, add || u > 0);
  };

  for (int ip = first; ip < last && ok; ++ip) {
    const PrefillPiece pc = piece_at(p, ip, last);
    if (pc.k0 >= pc.k1) continue;
    const int na = tiles_a(pc);
    Part part[2];
    int end[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      part[i] = part_of(pc, na, tile_span(pc, i, p.g_log2), p.sinks, p.window);
      end[i] = part[i].last(pc.k0, pc.k1);
    }
    // key tiles whose V is zeroed past the last key (bf16): the last of a range that does not fill it
    const int a_keys = min(pc.a1 * kBlock, pc.ctx_len) - pc.a0 * kBlock, b_keys = min(pc.b1 * kBlock, pc.ctx_len) - pc.b0 * kBlock;
    const int tail_a = na > 0 && a_keys % kTile ? na - 1 : -1, tail_b = b_keys > 0 && b_keys % kTile ? na + b_keys / kTile : -1;
    bool now[2] = {part[0].has(pc.k0), part[1].has(pc.k0)}, started[2] = {false, false};
    ok = x.wait_one(x.q_full(), q_round, p.status) && x.wait_one(x.full(ring.stage), ring.round, p.status);
    if (!ok) break;
    q_round ^= 1;
    tc_fence_after();
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (now[i]) qk(i, ring.stage);
    mma_commit(x.empty(ring.stage));
    if (pc.k0 + 1 == pc.k1) mma_commit(x.q_empty());
    ring.next(C::kStages);
    for (int k = pc.k0; k < pc.k1; ++k) {
      // V of tile k, and K of tile k + 1
      const int v_stage = ring.stage;
      const bool more = k + 1 < pc.k1, then[2] = {more && part[0].has(k + 1), more && part[1].has(k + 1)};
      ok = x.wait_one(x.full(v_stage), ring.round, p.status);
      if (!ok) break;
      if constexpr (!C::kOneByte) {
        if (k == tail_a || k == tail_b) {
          ok = x.wait_one(x.tail(v_stage), (tail_rounds >> v_stage) & 1, p.status);
          if (!ok) break;
          tail_rounds ^= 1u << v_stage;
        }
      }
      ring.next(C::kStages);
      const int k_stage = ring.stage;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (now[i]) {
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            ok = ok && x.wait_one(x.p_full(i, half), p_round[i], p.status);
            if (!ok) break;
            tc_fence_after();
            pv(i, v_stage, half, started[i]);
            started[i] = true;
          }
          if (!ok) break;
          p_round[i] ^= 1;
          if (k == end[i]) mma_commit(x.o_full(i));
        }
        if (i == 0 && more) {
          ok = x.wait_one(x.full(k_stage), ring.round, p.status);
          if (!ok) break;
          tc_fence_after();
        }
        if (then[i]) qk(i, k_stage);
      }
      if (!ok) break;
      mma_commit(x.empty(v_stage));
      if (more) {
        mma_commit(x.empty(k_stage));
        if (k + 2 == pc.k1) mma_commit(x.q_empty());
        ring.next(C::kStages);
      }
      now[0] = then[0];
      now[1] = then[1];
    }
  }
  // tensor memory is freed only when nothing uses it any more (the softmax may
  // have left after a failed wait)
  mma_commit(x.idle());
  if (!mbar_wait(x.idle(), 0, kDrainNs)) atomicOr(p.status, kStatusUndrained);
}

// ---- widening one-byte codes ---------------------------------------------------

// Four codes -> four bf16 values, exactly.
template <int KV>
__device__ __forceinline__ void widen4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if constexpr (KV == 2) {
    uint32_t a, b;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(a), "=r"(b)
        : "r"(w));
    const float2 fa = __half22float2(*reinterpret_cast<const __half2*>(&a));
    const float2 fb = __half22float2(*reinterpret_cast<const __half2*>(&b));
    lo = bf16_pair(fa.x, fa.y);
    hi = bf16_pair(fb.x, fb.y);
  } else {
    // u = code + 128 in a byte; bf16 0x4300 | (u & 127) is 128 + (u & 127), and
    // subtracting 256 (u < 128) or 128 (u >= 128) leaves u - 128
    w ^= 0x80808080u;
    const uint32_t t0 = __byte_perm(w, 0, 0x4140), t1 = __byte_perm(w, 0, 0x4342);
    const uint32_t m0 = (t0 & 0x007f007fu) | 0x43004300u, m1 = (t1 & 0x007f007fu) | 0x43004300u;
    const uint32_t s0 = (t0 & 0x00800080u) ^ 0x43804380u, s1 = (t1 & 0x00800080u) ^ 0x43804380u;
    const __nv_bfloat162 r0 = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&m0),
                                      *reinterpret_cast<const __nv_bfloat162*>(&s0));
    const __nv_bfloat162 r1 = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&m1),
                                      *reinterpret_cast<const __nv_bfloat162*>(&s1));
    lo = *reinterpret_cast<const uint32_t*>(&r0);
    hi = *reinterpret_cast<const uint32_t*>(&r1);
  }
}

__device__ __forceinline__ uint32_t scale_pair(uint32_t v, float a, float b) {
  return bf16_pair(__uint_as_float(v << 16) * a, __uint_as_float(v & 0xffff0000u) * b);
}

// 8 warps: 16-byte pieces of codes from the pool, widened into a stage.
// Thread t takes one of the D / 16 pieces of every 256 / (D / 16)-th row.  It copies
// them to shared memory two operands ahead and reads back its own, so the
// copies need no barrier; the loops stay short, as the softmax's code and
// this share the instruction cache.
template <int KV, int D>
__device__ void widen_role(const PrefillTCParams& p, const Ctx<KV, D>& x, int first, int last, int t) {
  using C = PC<KV, D>;
  constexpr int kParts = D / 16, kStep = C::kWiden / kParts, kIt = kTile / kStep;
  // 8 lanes in a row write 4 pieces of each of two rows: different banks
  const int lane = t & 31, part = D == 128 ? (t & 3) | ((t >> 1) & 4) : t & 3;
  const int row0 = D == 128 ? ((t >> 2) & 1) | ((t >> 4) << 1) : t >> 2;
  // the operand to copy next
  PrefillPiece ahead;
  int a_ip = first - 1, a_k = 0, a_kv = 0, a_ids = 0, a_n = 0, a_slot = 0;
  ahead.k0 = ahead.k1 = 0;
  auto copy_next = [&]() {
    if (a_kv == 0) {
      if (++a_k >= ahead.k1) {  // on to the next piece that has key tiles
        do {
          if (++a_ip >= last) break;
          ahead = piece_at(p, a_ip, last);
        } while (ahead.k0 >= ahead.k1);
        a_k = ahead.k0;
      }
      if (a_ip < last) {
        const int lb = tile_block(ahead, tiles_a(ahead), a_k, a_n);
        a_ids = lane < a_n ? block_of(p, ahead, lb + lane) : 0;
      }
    }
    if (a_ip < last) {
      const char* pool = static_cast<const char*>(a_kv ? p.v_pool : p.k_pool);
#pragma unroll
      for (int it = 0; it < kIt; ++it) {
        const int row = row0 + it * kStep;
        const int blk = __shfl_sync(kFull, a_ids, row / kBlock);
        const size_t at = (((size_t)blk * p.n_kv_heads + ahead.kv_head) * kBlock + row % kBlock) * D + part * 16;
        if (row < a_n * kBlock)
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(x.raw(a_slot) + (it * C::kWiden + t) * 16),
                       "l"(pool + at)
                       : "memory");
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    a_kv ^= 1;
    a_slot ^= 1;
  };
  copy_next();
  copy_next();
  Ring ring;
  int slot = 0;
  bool starve = p.starve && blockIdx.x == 0;
  for (int ip = first; ip < last; ++ip) {
    const PrefillPiece pc = piece_at(p, ip, last);
    const int na = tiles_a(pc);
    for (int k = pc.k0; k < pc.k1; ++k) {
      int n;
      const int lo = tile_block(pc, na, k, n) * kBlock;
      const int valid = min(n * kBlock, pc.ctx_len - lo);
#pragma unroll 1
      for (int kv = 0; kv < 2; ++kv) {
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        if (!x.wait(x.empty(ring.stage), ring.round ^ 1, p.status)) {
          asm volatile("cp.async.wait_group 0;" ::: "memory");
          return;
        }
        const float* ch = kv ? p.v_channel : p.k_channel;
        if (ch != nullptr) ch += (size_t)pc.kv_head * D + part * 16;
        const uint32_t src = x.raw(slot) + t * 16;
        const uint32_t dst = x.stage(ring.stage) + (part / 4) * 1024;
        const int c0 = (part % 4) * 2;
#pragma unroll 1
        for (int it = 0; it < kIt; ++it) {
          const int row = row0 + it * kStep;
          uint32_t w[4], r[8];
          asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                       : "r"(src + it * C::kWiden * 16));
#pragma unroll
          for (int e = 0; e < 4; ++e) widen4<KV>(w[e], r[2 * e], r[2 * e + 1]);
          if (ch != nullptr) {
#pragma unroll
            for (int e = 0; e < 8; ++e) r[e] = scale_pair(r[e], __ldg(ch + 2 * e), __ldg(ch + 2 * e + 1));
          }
          const uint32_t at = dst + (row / 8) * C::kGroup + (row % 8) * 128 + ((c0 ^ (row & 6)) << 4);
          const uint32_t odd = (row & 1) << 4;
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at + odd), "r"(r[0]), "r"(r[1]), "r"(r[2]),
                       "r"(r[3])
                       : "memory");
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at + (odd ^ 16)), "r"(r[4]), "r"(r[5]),
                       "r"(r[6]), "r"(r[7])
                       : "memory");
        }
        if (valid < kTile) {  // never written, or past the run: weight 0 needs a finite value
#pragma unroll 1
          for (int row = row0; row < kTile; row += kStep) {
            if (row < valid) continue;
            const uint32_t at = dst + (row / 8) * C::kGroup + (row % 8) * 128;
#pragma unroll
            for (int h = 0; h < 2; ++h)
              asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(at + (((c0 + h) ^ (row & 7)) << 4)), "r"(0)
                           : "memory");
          }
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0 && !(starve && kv == 1)) mbar_arrive(x.full(ring.stage));
        starve = starve && kv == 0;
        ring.next(C::kStages);
        slot ^= 1;
        copy_next();
      }
    }
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// ---- softmax, output -----------------------------------------------------------

__device__ __forceinline__ float row_lse(float m, float l) { return l == 0.0f ? -INFINITY : (m + log2f(l)) * kLn2; }

// Rows `todo` (a bit each) of a softmax warp over the piece's key tiles on the
// CUDA cores, one after the other, 32 keys at a time with the row's true
// maximum, written in place of what the warp has written.  For the logits kLK
// lanes take a row of K, 16 bytes each; their sums, kLK of them a lane, are
// added up and spread out at once (half as many with each exchange), so that
// lane t of the group g ends with key t * 32 / kLK + g.  For the values a lane
// takes the D / 32 columns from lane * (D / 32) on, with kAt rows' loads in
// flight.  Bound by the latency of its loads: 32768 rows over 8192 keys of 128
// take 31 ms in bf16, 26 in FP8 (264 and 272 with a key at a time and a 5-step
// shuffle for its logit), where the tensor cores take 0.11 and 0.16.  (Not
// inlined, with few registers: they are not to weigh on the main loop.)
template <int KV, int D>
__device__ __noinline__ void exact_rows(const PrefillTCParams& p, const PrefillPiece& pc, int warp, int lane, unsigned todo,
                                        int* steps) {
  constexpr int E = D / 32, N = KV == 1 ? 8 : 16, kLK = D / N, kAt = 4;
  const int t = lane % kLK, mine = t * (32 / kLK) + lane / kLK;
#pragma unroll 1
  for (; todo; todo &= todo - 1) {
    const int r = warp * 32 + __ffs(todo) - 1, tok = r >> p.g_log2;
    const size_t row_out = (size_t)(pc.q_row + tok) * p.n_heads + (pc.kv_head << p.g_log2) + (r & ((1 << p.g_log2) - 1));
    float q[N], o[E], m, l;
#pragma unroll
    for (int e = 0; e < N; e += 4) load_values<1, 4>(p.q, row_out * D + t * N + e, q + e);
    if (KV != 1 && p.k_channel != nullptr) {
#pragma unroll
      for (int e = 0; e < N; ++e) q[e] *= p.k_channel[pc.kv_head * D + t * N + e];
    }
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = 0.0f;
    m = -INFINITY;
    l = 0.0f;  // this lane's keys', until the end
    const int i = pc.pos0 + tok, na = tiles_a(pc);
#pragma unroll 1
    for (int k = pc.k0; k < pc.k1; ++k) {
      if (lane == 0) atomicAdd(steps, 1);  // waits elsewhere see that this goes on
      int n;
      const int lb = tile_block(pc, na, k, n);
      const int hi = min(min((lb + n) * kBlock, pc.ctx_len), i + 1);
#pragma unroll 1
      for (int j0 = lb * kBlock; j0 < hi; j0 += 32) {
        const bool have = j0 + mine < hi && keeps(j0 + mine, i, p.sinks, p.window);
        const unsigned counts = __ballot_sync(kFull, have);
        if (counts == 0) continue;
        const int j = min(j0 + mine, hi - 1);  // past the last key it is read again, and does not count
        const unsigned row = ((unsigned)block_of(p, pc, j / kBlock) * p.n_kv_heads + pc.kv_head) * kBlock + (j & 15);
        const float ks = KV != 1 ? __ldg(p.k_scale + row) : 1.0f, vs = KV != 1 ? __ldg(p.v_scale + row) : 1.0f;
        float part[kLK];
#pragma unroll
        for (int u0 = 0; u0 < kLK; u0 += 4) {
          uint4 w[4];
#pragma unroll
          for (int u = 0; u < 4; ++u)
            w[u] = __ldg(static_cast<const uint4*>(p.k_pool) + (size_t)__shfl_sync(kFull, row, u0 + u, kLK) * kLK + t);
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            float x[N];
            unpack16<KV>(w[u], x);
            part[u0 + u] = 0.0f;
#pragma unroll
            for (int e = 0; e < N; ++e) part[u0 + u] += q[e] * x[e];
          }
          __syncwarp();
        }
#pragma unroll
        for (int half = kLK / 2; half; half /= 2) {
          const bool high = t & half;
#pragma unroll
          for (int u = 0; u < half; ++u)
            part[u] = (high ? part[u + half] : part[u]) + __shfl_xor_sync(kFull, high ? part[u] : part[u + half], half);
        }
        const float s = have ? part[0] * (ks * p.scale) * kLog2e : -INFINITY;
        float mn = fmaxf(m, s);
#pragma unroll
        for (int off = 16; off; off >>= 1) mn = fmaxf(mn, __shfl_xor_sync(kFull, mn, off));
        const float wk = s == -INFINITY ? 0.0f : exp2f(s - mn), alpha = m == -INFINITY ? 0.0f : exp2f(m - mn);
        const float wv = wk * vs;
        l = l * alpha + wk;
        m = mn;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] *= alpha;
#pragma unroll 1
        for (int u0 = 0; u0 < 32; u0 += kAt) {
          float v[kAt][E];
#pragma unroll
          for (int u = 0; u < kAt; ++u)
            load_values<KV, E>(p.v_pool, (size_t)__shfl_sync(kFull, row, u0 + u) * D + lane * E, v[u]);
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
    }
#pragma unroll
    for (int off = 16; off; off >>= 1) l += __shfl_xor_sync(kFull, l, off);
    if (KV != 1 && p.v_channel != nullptr) {
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] *= p.v_channel[pc.kv_head * D + lane * E + e];
    }
    if (pc.record >= 0) {
      float* rec = p.records + (size_t)pc.record * prefill_record_floats(D);
#pragma unroll
      for (int e = 0; e < E; ++e) rec[(size_t)r * D + lane * E + e] = o[e];
      if (lane == 0) {
        rec[2 * kPreRows * D + r] = m;
        rec[2 * kPreRows * (D + 1) + r] = l;
      }
    } else {
      const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
      for (int e = 0; e < E; ++e)
        static_cast<__nv_bfloat16*>(p.out)[row_out * D + lane * E + e] = __float2bfloat16_rn(l == 0.0f ? 0.0f : o[e] * inv);
      if (lane == 0 && p.lse != nullptr) p.lse[row_out] = row_lse(m, l);
    }
  }
}

// The item's output rows from its partial records, by the softmax warps of the
// CTA that wrote the last one: w_c = 2^(m_c - M), out = sum_c w_c O_c /
// sum_c w_c l_c, records taken in order.  A warp takes its rows' weights a
// lane each, then kAt rows' O at a time, whose loads are all in flight.  (Not
// inlined, like exact_rows.)
template <int D, int kWarps, int kAt>
__device__ __noinline__ void merge_records(const PrefillTCParams& p, const PrefillPiece& pc, int warp, int lane) {
  constexpr int NV = D / 32;
  const PrefillMerge mg = p.merges[pc.merge];
  const size_t rf = prefill_record_floats(D);
  const float* base = p.records + (size_t)mg.first * rf;
  constexpr int kRows = kPreTiles * kPreRows / kWarps;
  const int r0 = warp * kRows, left = min(kRows, (pc.n_tok << p.g_log2) - r0);  // this warp's rows
  if (left <= 0) return;
  const int mine = r0 + min(lane, left - 1);
  const float *ms = base + 2 * kPreRows * D + mine, *ls = base + 2 * kPreRows * (D + 1) + mine;
  float M = -INFINITY, l = 0.0f;
  for (int c = 0; c < mg.count; ++c) {  // online, so that each record is read once
    const float mc = __ldcg(ms + c * rf), lc = __ldcg(ls + c * rf);
    if (lc == 0.0f) continue;
    const float top = fmaxf(M, mc);
    l = l * (M == -INFINITY ? 0.0f : exp2f(M - top)) + lc * exp2f(mc - top);
    M = top;
  }
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  auto out_row = [&](int r) {
    return (size_t)(pc.q_row + (r >> p.g_log2)) * p.n_heads + (pc.kv_head << p.g_log2) + (r & ((1 << p.g_log2) - 1));
  };
  if (lane < left && p.lse != nullptr) p.lse[out_row(mine)] = row_lse(M, l);
#pragma unroll 1
  for (int g = 0; g < left; g += kAt) {
    float o[kAt][NV];
#pragma unroll
    for (int u = 0; u < kAt; ++u)
#pragma unroll
      for (int e = 0; e < NV; ++e) o[u][e] = 0.0f;
#pragma unroll 1
    for (int c = 0; c < mg.count; ++c) {
      const float lc = __ldcg(ls + c * rf);
      const float wc = lc == 0.0f ? 0.0f : exp2f(__ldcg(ms + c * rf) - M) * inv;
      const float* rec = base + c * rf + (size_t)(r0 + g) * D + lane * NV;
      float v[kAt][NV];
#pragma unroll
      for (int u = 0; u < kAt; ++u) {
        if (g + u >= left) continue;
        if constexpr (NV == 4) {
          const float4 x = __ldcg(reinterpret_cast<const float4*>(rec + u * D));
          v[u][0] = x.x, v[u][1] = x.y, v[u][2] = x.z, v[u][3] = x.w;
        } else {
          const float2 x = __ldcg(reinterpret_cast<const float2*>(rec + u * D));
          v[u][0] = x.x, v[u][1] = x.y;
        }
      }
#pragma unroll
      for (int u = 0; u < kAt; ++u) {
        const float w = __shfl_sync(kFull, wc, g + u);
        if (g + u < left && w != 0.0f)
#pragma unroll
          for (int e = 0; e < NV; ++e) o[u][e] += w * v[u][e];
      }
    }
#pragma unroll
    for (int u = 0; u < kAt; ++u) {
      if (g + u >= left) continue;
      uint32_t* dst =
          reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(p.out) + out_row(r0 + g + u) * D + lane * NV);
#pragma unroll
      for (int e = 0; e < NV; e += 2) dst[e / 2] = bf16_pair(o[u][e], o[u][e + 1]);
    }
  }
}

// A warp's 32 rows, of which lane l holds 32 bytes of row l in w: through
// shared memory to row[e] + at for rows 16 e + lane / 2, so that 2 lanes write
// one row's 32 bytes.  Rows that are null are not written.
__device__ __forceinline__ void store_rows(uint32_t stage, const uint32_t* w, char* const* row, int at, int lane) {
#pragma unroll
  for (int e = 0; e < 2; ++e)
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(stage + lane * 32 + ((e ^ ((lane >> 2) & 1)) << 4)),
                 "r"(w[4 * e]), "r"(w[4 * e + 1]), "r"(w[4 * e + 2]), "r"(w[4 * e + 3])
                 : "memory");
  __syncwarp();
  const int c = lane & 1;
  uint4 v[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int r = 16 * e + lane / 2;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v[e].x), "=r"(v[e].y), "=r"(v[e].z), "=r"(v[e].w)
                 : "r"(stage + r * 32 + ((c ^ ((r >> 2) & 1)) << 4)));
  }
#pragma unroll
  for (int e = 0; e < 2; ++e)
    if (row[e] != nullptr) *reinterpret_cast<uint4*>(row[e] + at + c * 16) = v[e];
  __syncwarp();
}

// Bits j of 32 keys from key `from` on that a row keeps; past, win, sink: the
// first key it does not keep any more, its window's first, and the first
// behind the sinks.
__device__ __forceinline__ uint32_t kept_bits(int from, int past, int win, int sink) {
  auto below = [](int n) { return n <= 0 ? 0u : n >= 32 ? kFull : (1u << n) - 1u; };
  return below(past - from) & (~below(win - from) | below(sink - from));
}

// Four floats of shared memory, as two pairs.  Not volatile, so that it can be
// scheduled: its address holds its place.
__device__ __forceinline__ void load_pairs(uint32_t at, uint64_t& a, uint64_t& b) {
  asm("ld.shared.v2.b64 {%0, %1}, [%2];" : "=l"(a), "=l"(b) : "r"(at));
}
// log2 x on the hardware approximation: only moves the reference, whose step
// the row's factor follows, so that its error cancels.
__device__ __forceinline__ float hw_log2(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The softmax warps, 4 for each query tile: a thread per row.
template <int KV, int D>
__device__ void softmax_role(const PrefillTCParams& p, const Ctx<KV, D>& x, uint32_t tmem, int first, int last,
                             volatile int* last_flag) {
  using C = PC<KV, D>;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, i = warp >> 2;
  const int r = threadIdx.x & (kPreRows - 1);  // row of the tile
  const uint32_t quarter = (uint32_t)(warp & 3) << 21;  // lane field of this warp's rows
  const uint32_t ts = tmem + quarter + i * kTile, to = tmem + quarter + 2 * kTile + i * 128;
  const float c = p.scale * kLog2e;
  uint32_t s_round = 0, o_round = 0, m_round = 0;
  Ring sc;

  for (int ip = first; ip < last; ++ip) {
    const PrefillPiece& pc = *(p.pieces + ip);
    if (ip + 1 < last) asm volatile("prefetch.global.L1 [%0];" ::"l"(p.pieces + ip + 1));
    const int na = tiles_a(pc), k1 = pc.k1;
    const Span span = tile_span(pc, i, p.g_log2);
    const Part part = part_of(pc, na, span, p.sinks, p.window);
    // Key tiles [whole_lo, whole_hi): every row keeps every key.
    const int past0 = min((span.lo + 1) / kBlock, pc.b1) - pc.b0, win0 = max(0, span.hi - p.window + 1);
    const int whole_hi = na + (past0 < 0 ? 0 : past0 / kPreBlocks);
    const int whole_lo = na + (max(0, (win0 + kBlock - 1) / kBlock - pc.b0) + kPreBlocks - 1) / kPreBlocks;
    const int pos = span.lo + (r >> p.g_log2);
    const bool valid_row = pos <= span.hi;
    float m = valid_row ? -INFINITY : 0.0f;  // the row's reference (log2 units)
    float l = 0.0f;                          // its sum, up to the tile before
    float tile = 0.0f;                       // the last tile's
    bool any = false;
    // Takes the last tile's sum into l.  When it is large, so are weights of
    // it: the reference moves by its logarithm, over > 0.
    auto settle = [&]() {
      l += tile;
      return tile > 1024.0f ? hw_log2(tile) : 0.0f;
    };
    // Moves the reference by over > 0; the factor of what the row holds, from
    // the step that m really took.  NaN where it would flush to 0: weights of
    // the tile may have left fp32's range, so the row is computed again.
    auto move = [&](float over) {
      const float from = m;
      m += over;
      const float f = hw_exp2(from - m);
      return f == 0.0f ? __int_as_float(0x7fffffff) : f;
    };
    for (int k = pc.k0; k < k1; ++k) {
      if (!part.has(k)) {
        if constexpr (C::kOneByte) {  // in step with the ring, so that no arrival counts for a later round
          if (!x.wait(x.sc_full(sc.stage), sc.round, p.status)) return;
          if (lane == 0) mbar_arrive(x.sc_empty(sc.stage));
          sc.next(C::kScaleStages);
        }
        continue;
      }
      const bool whole = k >= whole_lo && k < whole_hi;
      uint32_t fac = x.scales(sc.stage);
      if constexpr (C::kOneByte) {
        if (!x.wait(x.sc_full(sc.stage), sc.round, p.status)) return;
        asm volatile("" : "+r"(fac)::"memory");  // the loads depend on it: none moves ahead of the wait
      }
      const float over = any ? settle() : 0.0f;
      int past = 0, win = 0, sink = 0;  // what this row keeps of its keys, where that differs from row to row
      if (!whole) {
        int n;
        const int lo = tile_block(pc, na, k, n) * kBlock;
        past = min(pos + 1 - lo, n * kBlock);
        win = pos - p.window + 1 - lo;
        sink = p.sinks - lo;
      }
      // 4 logits, from key j on, times their factors, plus ref
      auto scaled = [&](const uint32_t* v, int j, uint64_t ref, float* a) {
        uint64_t f01 = pack2(c, c), f23 = f01;
        if constexpr (C::kOneByte) {
          load_pairs(fac + j * 4, f01, f23);
        }
        unpack2(fma2(pack2(__uint_as_float(v[0]), __uint_as_float(v[1])), f01, ref), a[0], a[1]);
        unpack2(fma2(pack2(__uint_as_float(v[2]), __uint_as_float(v[3])), f23, ref), a[2], a[3]);
      };
      const bool rare = __any_sync(kFull, over > 0.0f || m == -INFINITY);
      if (!x.wait(x.s_full(i), s_round, p.status)) return;
      s_round ^= 1;
      tc_fence_after();
      uint32_t s[kChunk];
      tmem_load32(ts, s);
      if (rare) {
        if (__any_sync(kFull, over > 0.0f)) {
          const float f = over > 0.0f ? move(over) : 1.0f;
          l *= f;
#pragma unroll 1
          for (int b = 0; b < D; b += 16) {  // O, which holds the tiles before this one
            uint32_t o[16];
            tmem_load16(to + b, o);
            tmem_wait_load<16>(o);
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
            tmem_store16(to + b, o);
          }
        }
        if (__any_sync(kFull, m == -INFINITY)) {  // a row's first tile: its own maximum
          float top = -INFINITY;
#pragma unroll 1
          for (int b = 0; b < kTile; b += 16) {
            uint32_t u[16];
            tmem_load16(ts + b, u);
            tmem_wait_load<16>(u);
            const uint32_t bits = whole ? kFull : kept_bits(b, past, win, sink);
#pragma unroll
            for (int j = 0; j < 16; j += 4) {
              float a[4];
              scaled(u + j, b + j, 0, a);
#pragma unroll
              for (int e = 0; e < 4; ++e) top = fmaxf(top, (bits >> (j + e)) & 1 ? a[e] : -INFINITY);
            }
          }
          if (m == -INFINITY) m = top;
        }
      }
      const float ref = m == -INFINITY ? 0.0f : -m;
      const uint64_t ref2 = pack2(ref, ref);
      uint64_t la = 0, lb = 0;  // this tile's sum, in four parts
      // kChunk keys from b on: weights into P's columns
      auto weigh = [&](const uint32_t* v, int b) {
        constexpr int N = kChunk;
        float a[N];
#pragma unroll
        for (int j = 0; j < N; j += 4) scaled(v + j, b + j, ref2, a + j);
        uint32_t bits = kFull;
        if (!whole) {
          bits = kept_bits(b, past, win, sink);
#pragma unroll
          for (int j = 0; j < N; ++j)
            if (!((bits >> j) & 1)) a[j] = -INFINITY;
        }
        uint32_t w[N / 2];
#pragma unroll
        for (int j = 0; j < N; j += 4) {
#pragma unroll
          for (int e = 0; e < 4; ++e) a[j + e] = hw_exp2(a[j + e]);
          la = add2(la, pack2(a[j], a[j + 1]));
          lb = add2(lb, pack2(a[j + 2], a[j + 3]));
          if constexpr (C::kOneByte) {
            uint64_t g01, g23;
            load_pairs(fac + (kTile + b + j) * 4, g01, g23);
            unpack2(mul2(pack2(a[j], a[j + 1]), g01), a[j], a[j + 1]);
            unpack2(mul2(pack2(a[j + 2], a[j + 3]), g23), a[j + 2], a[j + 3]);
          }
          // Rounded to bf16 (by 2^-8 at most), as both operands of a product have
          // one type and V is bf16 or codes widened to it: the result's error
          // against 64 bits grows from 0.0017 (its own rounding) to 0.0023.  fp16,
          // which codes would fit, holds no weight above 65504, and here they grow
          // with the logits until the reference moves; a second product with what
          // the rounding drops would make three products of two.
          w[j / 2] = bf16_pair(a[j], a[j + 1]);
          w[j / 2 + 1] = bf16_pair(a[j + 2], a[j + 3]);
        }
        if constexpr (C::kOneByte) {
          if (!whole) {  // a key that is not kept has weight 0 whatever its scale
#pragma unroll
            for (int j = 0; j < N / 2; ++j) {
              const uint32_t two = bits >> (2 * j);
              w[j] &= (two & 1 ? 0x0000ffffu : 0u) | (two & 2 ? 0xffff0000u : 0u);
            }
          }
        }
        tmem_store16(ts + b / 2, w);
      };
#pragma unroll 1
      for (int b = 0; b < kTile; b += kTile / 2) {
#pragma unroll
        for (int u = 0; u < kTile / 2; u += kChunk) {
          if (b + u > 0) tmem_load32(ts + b + u, s);
          tmem_wait_load<kChunk>(s);
          weigh(s, b + u);
        }
        // half of the tile's keys: their product with V may start
        tmem_wait_store();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(x.p_full(i, b > 0));
      }
      any = true;
      float l0, l1;
      unpack2(add2(la, lb), l0, l1);
      tile = l0 + l1;
      if constexpr (C::kOneByte) {
        if (lane == 0) mbar_arrive(x.sc_empty(sc.stage));
        sc.next(C::kScaleStages);
      }
    }

    const float over = any ? settle() : 0.0f, f = over > 0.0f ? move(over) : 1.0f;
    l *= f;
    // output row (or partial record's row) of this warp's row r32
    const int per = kPreRows >> p.g_log2, base = (warp & 3) * 32;
    float* rec = pc.record >= 0 ? p.records + (size_t)pc.record * prefill_record_floats(D) : nullptr;
    auto out_row = [&](int r32) {
      const int rt = base + r32;
      return (size_t)((pc.q_row + i * per + (rt >> p.g_log2)) * p.n_heads + (pc.kv_head << p.g_log2) +
                      (rt & ((1 << p.g_log2) - 1)));
    };
    auto dst = [&](int r32) -> char* {
      const int rt = base + r32;
      if (span.lo + (rt >> p.g_log2) > span.hi) return nullptr;
      if (rec != nullptr) return reinterpret_cast<char*>(rec + (i * kPreRows + rt) * D);
      return static_cast<char*>(p.out) + out_row(r32) * (D * 2);
    };
    const float inv = rec != nullptr ? f : l == 0.0f ? 0.0f : f / l;
    auto row_stats = [&](int r32, float mr, float lr) {
      if (rec != nullptr) {
        rec[2 * kPreRows * D + i * kPreRows + base + r32] = mr;
        rec[2 * kPreRows * (D + 1) + i * kPreRows + base + r32] = lr;
      } else if (p.lse != nullptr) {
        p.lse[out_row(r32)] = row_lse(mr, lr);
      }
    };
    if (valid_row) row_stats(lane, m, l);
    float bad = l * 0.0f;  // NaN once the sum or some O is not finite
    if (any) {
      if (!x.wait(x.o_full(i), o_round, p.status)) return;
      o_round ^= 1;
      tc_fence_after();
    }
    if (__any_sync(kFull, valid_row)) {
      char* rows[2];  // the rows this lane writes a part of
#pragma unroll
      for (int e = 0; e < 2; ++e) rows[e] = dst(16 * e + lane / 2);
      uint32_t o[16];
      if (any) {
        tmem_load16(to, o);
      } else {
#pragma unroll
        for (int e = 0; e < 16; ++e) o[e] = 0;
      }
#pragma unroll 1
      for (int b = 0; b < D; b += 16) {
        if (any) tmem_wait_load<16>(o);
        float nan[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        uint32_t w[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) nan[e & 3] = fmaf(__uint_as_float(o[e]), 0.0f, nan[e & 3]);
        bad += (nan[0] + nan[1]) + (nan[2] + nan[3]);
#pragma unroll
        for (int e = 0; e < 16; ++e) w[e] = __float_as_uint(__uint_as_float(o[e]) * inv);
        if (any && b + 16 < D) tmem_load16(to + b + 16, o);
        if (rec != nullptr) {
          store_rows(x.out(warp), w, rows, b * 4, lane);
          store_rows(x.out(warp), w + 8, rows, b * 4 + 32, lane);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) w[e] = bf16_pair(__uint_as_float(w[2 * e]), __uint_as_float(w[2 * e + 1]));
          store_rows(x.out(warp), w, rows, b * 2, lane);
        }
      }
    }
    const unsigned todo = __ballot_sync(kFull, valid_row && bad != 0.0f);
    if (todo != 0) exact_rows<KV, D>(p, pc, warp, lane, todo, const_cast<int*>(x.abort + 1));
    if (rec != nullptr) {
      __threadfence();
      __syncwarp();
      if (lane == 0) mbar_arrive(x.written());
      if (warp == 0) {
        if (!x.wait(x.written(), m_round, p.status)) return;
        if (lane == 0) {
          __threadfence();
          *last_flag = atomicAdd(p.counters + pc.merge, 1) == p.merges[pc.merge].count - 1;
          mbar_arrive(x.counted());
        }
        __syncwarp();
      }
      if (!x.wait(x.counted(), m_round, p.status)) return;
      m_round ^= 1;
      if (*last_flag) {
        __threadfence();
        merge_records<D, C::kSoft / 32, C::kOneByte ? 8 : 16>(p, pc, warp, lane);
      }
    }
  }
}

// ---- the kernel ------------------------------------------------------------------

template <int KV, int D>
__global__ void __launch_bounds__(PC<KV, D>::kThreads, 1)
    prefill_tc_kernel(const __grid_constant__ PrefillTCParams p) {
  using C = PC<KV, D>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint32_t tmem_at;
  __shared__ int aborted[2], last_flag;
  Ctx<KV, D> x;
  x.base = (smem_addr(smem_raw) + 1023u) & ~1023u;
  x.abort = aborted;
  x.limit_ns = p.wait_limit_ns;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    aborted[0] = aborted[1] = 0;
    mbar_init(x.q_full(), 1);
    mbar_init(x.q_empty(), 1);
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(x.full(s), C::kOneByte ? C::kWiden / 32 : 1);
      mbar_init(x.empty(s), 1);
      mbar_init(x.tail(s), 1);
    }
    for (int s = 0; s < C::kScaleStages; ++s) {
      mbar_init(x.sc_full(s), 1);
      mbar_init(x.sc_empty(s), C::kSoft / 32);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(x.s_full(i), 1);
      mbar_init(x.p_full(i, 0), 4);
      mbar_init(x.p_full(i, 1), 4);
      mbar_init(x.o_full(i), 1);
    }
    mbar_init(x.written(), C::kSoft / 32);
    mbar_init(x.counted(), 1);
    mbar_init(x.idle(), 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  constexpr int kIssue = C::kSoft / 32;  // the first warp behind the softmax's
  if (warp == kIssue) tmem_alloc(smem_addr(&tmem_at), 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_at;
  const int first = p.cta_begin[blockIdx.x], last = p.cta_begin[blockIdx.x + 1];
  if (warp < kIssue) {
    more_registers<C::kSoftRegs>();
    softmax_role<KV, D>(p, x, tmem, first, last, &last_flag);
  } else if (warp < kIssue + 4) {
    fewer_registers<C::kIssueRegs>();
    if (warp == kIssue && elect_one()) product_role<KV, D>(p, x, tmem, first, last);
    __syncwarp();
    if constexpr (C::kOneByte) {
      if (warp == kIssue + 1) query_role<KV, D>(p, x, first, last, lane);
      if (warp == kIssue + 2) scale_role<KV, D>(p, x, first, last, lane);
    } else {
      if (warp == kIssue + 1) load_role<D, false>(p, x, first, last, lane);
      if (warp == kIssue + 2) load_role<D, true>(p, x, first, last, lane);
    }
  } else {
    if constexpr (C::kOneByte) {
      fewer_registers<C::kWidenRegs>();
      widen_role<KV, D>(p, x, first, last, threadIdx.x - C::kSoft - 128);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kIssue) tmem_free(tmem, 512);
}

// The roles' register shares are made for kLaunchRegs: with fewer, a warpgroup
// would wait for registers that never come free.  Such a build is refused.
template <int KV, int D>
cudaError_t prefill_prepare_one() {
  using C = PC<KV, D>;
  cudaFuncAttributes at;
  if (cudaError_t e = cudaFuncGetAttributes(&at, prefill_tc_kernel<KV, D>)) return e;
  if (at.numRegs != C::kLaunchRegs) return cudaErrorLaunchOutOfResources;
  return cudaFuncSetAttribute(prefill_tc_kernel<KV, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kBytes);
}

template <int D>
cudaError_t prefill_prepare(int kv) {
  switch (kv) {
    case 1: return prefill_prepare_one<1, D>();
    case 2: return prefill_prepare_one<2, D>();
    case 3: return prefill_prepare_one<3, D>();
  }
  return cudaErrorInvalidValue;
}

template <int D>
cudaError_t prefill_launch(int kv, const PrefillTCParams& p, int ctas, cudaStream_t st) {
  if (ctas <= 0) return cudaSuccess;
  switch (kv) {
    case 1: prefill_tc_kernel<1, D><<<ctas, PC<1, D>::kThreads, PC<1, D>::kBytes, st>>>(p); break;
    case 2: prefill_tc_kernel<2, D><<<ctas, PC<2, D>::kThreads, PC<2, D>::kBytes, st>>>(p); break;
    case 3: prefill_tc_kernel<3, D><<<ctas, PC<3, D>::kThreads, PC<3, D>::kBytes, st>>>(p); break;
    default: return cudaErrorInvalidValue;
  }
  return cudaGetLastError();
}

}  // namespace
}  // namespace pkv
