// pa_prompt.cuh -- causal attention over whole prompts, packed one after another
// ([T, H, D] query rows, [T, Hk, D] key and value rows, sequence s the tokens
// seq_starts[s] .. seq_starts[s + 1] - 1), on the sm_100a tensor cores:
//   z_ij = scale q_i . k_j,   lse_i = log sum_{j <= i} exp(z_ij),
//   out_i = sum_{j <= i} exp(z_ij - lse_i) v_j.
//
// Work item: (sequence, KV head, pair of query tiles).  A tile is 128 / G
// consecutive tokens x the G query heads of the KV head, token-major: 128 rows,
// the M of one MMA.  Both tiles walk the same keys in blocks of 128, one TMA
// box per 64-column slab of K and V, each block loaded once for 256 rows.  Per
// tile t and block j:
//   S_t  = Q_t K_j^T    128 x 128 fp32 in tensor memory
//   P_t  = 2^(S_t scale log2 e - m)   by the tile's softmax warpgroup (thread
//                       r = row r), written over S_t in the inputs' type
//   O_t += P_t V_j      128 x D fp32 in tensor memory
// One pass over the keys: m is a running reference maximum (O and l are rescaled
// only when a row outgrows it by 2^8), l the fp32 sum of the fp32 p.  P is
// rounded to the inputs' type because the product takes both operands in one
// type: at most 2^-8 (bf16) or 2^-11 (fp16) of each term, as much as the
// output's own rounding, with random signs over the keys.  An fp16 P is held 2^7
// up (2^15 at most, with the slack of m; O and l scale alike): so it is normal down
// to 2^-21 of m's term and what it loses below is at most 2^-32 of it a key, where
// thousands of keys at 2^-25 of a large one would have come to nothing.
//
// The grid is persistent, one CTA per SM, items longest first, every ring and
// phase running on from item to item.  Warps: 0-3 and 4-7 the softmax of tiles
// A and B, 8 issues the MMAs, 9 the loads, 10-11 look through V.
//
// With few tiles (kHalves) an item is one tile, and A and B are its even and its
// odd key blocks, each with its own m, l and O; the epilogue joins them, each
// warpgroup half of the columns.  Twice the items, half as long.
//
// A key that a row does not see has p = 0, but 0 times a NaN or an infinite
// value is NaN.  Only a block that holds such a key for some row (the diagonal,
// the sequence's end) can carry one over, so warps 10-11 look through those
// blocks of V, set what is not finite to 0 there and mark the CTA; from then on
// its epilogues add such values to the rows that do see them.
//
// Measured (head_dim 128, bf16, 32 heads over 8): one prompt of 16384 tokens 1.71
// to 1.77 ms, 1242 to 1284 TFLOP/s of the 1648 that cuBLAS reaches in short runs
// (2.0 ms when repeated under the power cap, 1100 of 1374); eight prompts of
// 77 to 4001 tokens 281 us, 1033 TFLOP/s.  Neither the tensor pipe (51 %) nor the
// special-function unit (47 %) is full: a tile's chain S -> softmax -> P V takes
// longer than the four products of both tiles, and two tiles in turn cover it in part.
// Three tiles do not fit the 512 columns.  Figures of single choices are at them.
#pragma once

#include <limits.h>

#include "pa_prefill.cuh"

namespace pa {

constexpr int kPromptThreads = 12 * 32;
constexpr int kWarpGuard = 10;
constexpr int kGuardWarps = 2;
// 384 threads launched at 168 registers: 504 x 128; two warpgroups at 208 and one at 88
constexpr uint32_t kPromptRegsSoftmax = 208, kPromptRegsOther = 88;
// log2 of what P is held up by (and with it O and l), and the way back
template <bool BF16>
constexpr float kPromptLift = BF16 ? 0.f : 7.f;
template <bool BF16>
constexpr float kPromptDrop = BF16 ? 1.f : 0x1p-7f;
constexpr int kPromptRankSeqs = 256;    // batches ranked longest-first: sequences,
constexpr int kPromptRankUnits = 2048;  // units (sequence, tile pair),
constexpr int kPromptRankWork = 65536;  // and units x sequences counted

struct PromptArgs {
  uint16_t* out;               // [T, H, D]
  float* lse;                  // [T, H] or null
  const uint16_t* value;       // rows value_stride elements apart
  long long value_stride;
  const int32_t* seq_starts;   // [S + 1]
  float scale_log2;
  int num_seqs;
  int num_tokens;              // T
  int num_heads;
  int num_kv_heads;
  int group;
  int tile_tokens;             // 128 / group, rounded down
};

template <int D>
struct PromptSmem {
  static constexpr int NST = D == 64 ? 4 : 2;       // K (and V) blocks in flight
  static constexpr int kSlabs = D / 64;
  static constexpr int kSlab = 128 * 128;           // 128 rows x 128 B
  static constexpr int kQTile = kSlabs * kSlab;
  static constexpr int kStage = kSlabs * kSlab;
  static constexpr int kQ = 0;
  static constexpr int kK = kQ + 2 * kQTile;
  static constexpr int kV = kK + NST * kStage;
  static constexpr int kBarQ = kV + NST * kStage;
  static constexpr int kBarKFull = kBarQ + 8;
  static constexpr int kBarKEmpty = kBarKFull + 8 * NST;
  static constexpr int kBarVFull = kBarKEmpty + 8 * NST;
  static constexpr int kBarVEmpty = kBarVFull + 8 * NST;
  static constexpr int kBarVOk = kBarVEmpty + 8 * NST;   // looked through by the guard warps
  static constexpr int kBarS = kBarVOk + 8 * NST;        // per tile: S_t(j) (and P_t(j-1) V) done
  static constexpr int kBarP = kBarS + 16;               // per tile: P_t(j) written
  static constexpr int kBarEnd = kBarP + 16;             // every MMA done
  static constexpr int kBarQFree = kBarEnd + 8;          // an item's S products done
  static constexpr int kBarOFull = kBarQFree + 8;        // per tile: an item's last P V done
  static constexpr int kBarOFree = kBarOFull + 16;       // per tile: O read by the epilogue
  // one tile in two halves: the halves' m and l are in, and where they are (the
  // second tile's Q has no use then)
  static constexpr int kBarHalves = kBarOFree + 8;
  static constexpr int kHalfStats = kQ + kQTile;
  static constexpr int kTmemSlot = kBarOFree + 16;
  static constexpr int kAbort = kTmemSlot + 4;
  static constexpr int kMark = kAbort + 4;               // a V value that is not finite was met
  static constexpr int kSched = kMark + 4;               // unit count and per-warp sums
  static constexpr int kSeqs = (kSched + 128 + 15) & ~15;      // int4 per ranked sequence
  static constexpr int kList = kSeqs + 16 * kPromptRankSeqs;   // unit of each rank
  // per softmax warp: 32 output rows x 32 columns on their way out
  static constexpr int kStore = (kList + 4 * kPromptRankUnits + 15) & ~15;
  static constexpr int kBytes = kStore + 8 * 2048;
  static constexpr int kAlloc = kBytes + 1024;
};

template <uint32_t R>
__device__ __forceinline__ void regs_grow() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R));
}
template <uint32_t R>
__device__ __forceinline__ void regs_shrink() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R));
}

// One lane of the (converged) warp, always the same.
__device__ __forceinline__ bool elect_lane() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}

// x of lane 0: a value that the whole warp shares, known to the compiler as one.
// The MMA's operands sit in uniform registers; one computed from a value that
// the compiler takes for a lane's own is moved there for every MMA.
__device__ __forceinline__ int warp_uniform(int x) { return __shfl_sync(0xffffffffu, x, 0); }

// 2^x of two values as p * s on the FMA pipe, for part of the elements where the
// special-function unit (16 results a cycle and SM) would bound: with n the
// nearest integer of x, s = 2^n and p a polynomial of degree 5 for 2^(x - n),
// the minimax fit of the relative error on [-1/2, 1/2] (7.5e-8, 2.1e-7 in fp32).
// The smallest exponents give an s of 0 (no exponent field), so a masked key's p is; a
// NaN stays one, +inf gives NaN.  kUp: a factor 2^kUp is in p, not in s, so that s
// has a field up to n = 127 + kUp; the smallest are then those below kUp - 126.5.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
template <int kUp = 0>
__device__ __forceinline__ void exp2_fma(float2 x, float2& p, float2& s) {
  constexpr float kTimes = static_cast<float>(1 << kUp);
  auto both = [](float v) { return make_float2(v, v); };
  x = make_float2(max_nan(x.x, kUp - 127.f), max_nan(x.y, kUp - 127.f));
  const float2 t = ffma2(x, both(1.f), both(12582912.f));          // 1.5 * 2^23 + n
  const float2 f = ffma2(ffma2(t, both(1.f), both(-12582912.f)), both(-1.f), x);
  p = ffma2(f, both(kTimes * 0.0013276472454890609f), both(kTimes * 0.009675540961325169f));
  p = ffma2(p, f, both(kTimes * 0.05550713092088699f));
  p = ffma2(p, f, both(kTimes * 0.24022120237350464f));
  p = ffma2(p, f, both(kTimes * 0.6931469440460205f));
  p = ffma2(p, f, both(kTimes * 1.0000001192092896f));
  constexpr uint32_t kBias = static_cast<uint32_t>(127 - kUp) << 23;
  s = make_float2(__uint_as_float((__float_as_uint(t.x) << 23) + kBias),
                  __uint_as_float((__float_as_uint(t.y) << 23) + kBias));
}

// Store 32 32-bit columns of this thread's lane (complete after tmem_wait_st).
__device__ __forceinline__ void tmem_st32u_async(uint32_t taddr, const uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
      "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]),
      "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]), "r"(v[19]), "r"(v[20]), "r"(v[21]),
      "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]), "r"(v[28]),
      "r"(v[29]), "r"(v[30]), "r"(v[31])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// ---------------------------------------------------------------------------
// Units and their order.  A unit is (sequence, tile pair p); item i is unit
// i / Hk, KV head i % Hk.  CTA b of g takes items k g + b (k even) and
// k g + g - 1 - b (k odd) of the list.  Up to kPromptRankSeqs sequences and
// small unit counts every CTA ranks the units by the keys their last token
// sees, min(span (p + 1), len), longest first (ties by sequence); other
// batches take them sequence-major.
// ---------------------------------------------------------------------------

// Length of sequence s, or -1 if its bounds are not 0 <= start <= end <= T.
__device__ __forceinline__ int prompt_len(const int32_t* starts, int s, int num_tokens) {
  const int b = starts[s], e = starts[s + 1];
  return b < 0 || e < b || e > num_tokens ? -1 : e - b;
}

struct PromptOrder {
  int total;       // units
  bool ranked;
};

// Every thread of the CTA calls it; the same order in every CTA.  A sequence
// with bad bounds has no units and is reported by one CTA.
template <class Args>
__device__ __forceinline__ PromptOrder prompt_order(const Args& a, int span, int* sched,
                                                    int4* seqs, int* list, int warp, int lane) {
  const int t = threadIdx.x, n = static_cast<int>(blockDim.x);
  const bool table = a.num_seqs <= kPromptRankSeqs;
  const int chunk = (a.num_seqs + n - 1) / n;     // 1 for a table
  int mine = 0, len0 = 0;                        // a table entry: length, first unit, first row
  for (int s = t * chunk; s < min(a.num_seqs, (t + 1) * chunk); ++s) {
    const int len = prompt_len(a.seq_starts, s, a.num_tokens);
    if (len < 0) {
      if (s % gridDim.x == blockIdx.x) record_error(kErrQuery, s);
      continue;
    }
    len0 = len;
    mine += (len + span - 1) / span;
  }
  int first = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, first, d);
    if (lane >= d) first += v;
  }
  if (lane == 31) sched[4 + warp] = first;
  __syncthreads();
  for (int w = 0; w < warp; ++w) first += sched[4 + w];
  if (t == n - 1) sched[0] = first;
  first -= mine;
  if (table && t < a.num_seqs) seqs[t] = make_int4(len0, first, a.seq_starts[t], 0);
  if (!table) list[t] = first;
  __syncthreads();
  PromptOrder o;
  o.total = sched[0];
  o.ranked = table && o.total <= kPromptRankUnits &&
             static_cast<long long>(o.total) * a.num_seqs <= kPromptRankWork;
  if (o.ranked) {
    const float inv = 1.f / static_cast<float>(span);
    for (int u = t; u < o.total; u += n) {
      int lo = 0, hi = a.num_seqs;     // the last sequence whose first unit is <= u
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (seqs[mid].y <= u) lo = mid;
        else hi = mid;
      }
      const int p = u - seqs[lo].y;
      const int keys = min(span * (p + 1), seqs[lo].x);
      int rank = 0;
      for (int i = 0; i < a.num_seqs; ++i) {
        const int len = seqs[i].x;
        // pairs of sequence i that see more keys than this unit; its own earlier
        // sequences' pairs that see as many come first too
        const int bound = i < lo ? keys - 1 : keys;
        if (len > bound) rank += (len + span - 1) / span - div_floor(bound, span, inv);
      }
      list[rank] = lo | (p << 16);
    }
    __syncthreads();
  }
  return o;
}

struct PromptUnit {
  int s, pair, q0, len;    // sequence, its pair, first row and length
};

template <class Args>
__device__ __forceinline__ PromptUnit prompt_unit(const Args& a, const PromptOrder& o,
                                                  const int4* seqs, const int* list, int u,
                                                  int span) {
  if (o.ranked) {
    const int e = list[u], s = e & 0xffff;
    return {s, e >> 16, seqs[s].z, seqs[s].x};
  }
  if (a.num_seqs <= kPromptRankSeqs) {
    int lo = 0, hi = a.num_seqs;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (seqs[mid].y <= u) lo = mid;
      else hi = mid;
    }
    return {lo, u - seqs[lo].y, seqs[lo].z, seqs[lo].x};
  }
  const int n = static_cast<int>(blockDim.x), chunk = (a.num_seqs + n - 1) / n;
  int lo = 0, hi = n;                  // the last chunk whose first unit is <= u
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (list[mid] <= u) lo = mid;
    else hi = mid;
  }
  int first = list[lo], s = lo * chunk;
  for (;; ++s) {                       // u is below the unit count: found before the chunk ends
    const int units = (max(prompt_len(a.seq_starts, s, a.num_tokens), 0) + span - 1) / span;
    if (u < first + units || s + 1 >= a.num_seqs) break;
    first += units;
  }
  const int q0 = a.seq_starts[s];
  return {s, u - first, q0, a.seq_starts[s + 1] - q0};
}

struct PromptItem {
  int s, kvh, q0, len, tile_a, blocks;   // key blocks of the item
  int lim[2], nkb[2];                    // keys each tile's last token sees, its blocks
};

template <bool kHalves>
__device__ __forceinline__ void prompt_item(const PromptArgs& a, const PromptOrder& o,
                                            const int4* seqs, const int* list, int i, int span,
                                            PromptItem& it) {
  const int u = i / a.num_kv_heads;
  it.kvh = i - u * a.num_kv_heads;
  const PromptUnit unit = prompt_unit(a, o, seqs, list, u, span);
  it.s = unit.s;
  it.q0 = unit.q0;
  it.len = unit.len;
  it.tile_a = unit.pair * span;
  if constexpr (kHalves) {   // one tile, its even and its odd blocks
    it.lim[0] = it.lim[1] = min(it.tile_a + span, it.len);
    it.blocks = (it.lim[0] + kPrefillKeys - 1) / kPrefillKeys;
    it.nkb[0] = (it.blocks + 1) / 2;
    it.nkb[1] = it.blocks / 2;
    return;
  }
  const int half = span / 2;
  it.lim[0] = min(it.tile_a + half, it.len);
  it.lim[1] = it.tile_a + half < it.len ? min(it.tile_a + span, it.len) : 0;
  it.nkb[0] = (it.lim[0] + kPrefillKeys - 1) / kPrefillKeys;
  it.nkb[1] = (it.lim[1] + kPrefillKeys - 1) / kPrefillKeys;
  it.blocks = max(it.nkb[0], it.nkb[1]);
}

// One 128-key block of a tile's online softmax, thread = row: S (fp32, in p)
// -> P over S in tensor memory in the inputs' type; l and the reference
// maximum m updated, O rescaled in tensor memory when m moves.  lim = keys of
// this row within the block and after it (<= 0: none).
template <bool BF16, int D>
__device__ __forceinline__ void prompt_softmax_block(float (&p)[kPrefillKeys], bool first, int lim,
                                                     float sl2, float& m, float& l,
                                                     uint32_t s_addr, uint32_t o_addr) {
  if (lim < kPrefillKeys) {
#pragma unroll
    for (int c = 0; c < kPrefillKeys; ++c) p[c] = c < lim ? p[c] : -INFINITY;
  }
  float mul = sl2;
  if (!(sl2 > 0.f)) {   // the maximum of the scaled logits is not that of the raw ones
#pragma unroll
    for (int c = 0; c < kPrefillKeys; ++c) p[c] = c < lim ? p[c] * sl2 : -INFINITY;
    mul = 1.f;
  }
  float mx[8];
#pragma unroll
  for (int q = 0; q < 8; ++q) mx[q] = p[q];
#pragma unroll
  for (int c = 8; c + 16 <= kPrefillKeys; c += 16) {
#pragma unroll
    for (int q = 0; q < 8; ++q) mx[q] = fmax3(mx[q], p[c + q], p[c + 8 + q]);
  }
#pragma unroll
  for (int q = 0; q < 8; ++q) mx[q] = fmaxf(mx[q], p[kPrefillKeys - 8 + q]);
  const float top = fmax3(fmax3(mx[0], mx[1], mx[2]), fmax3(mx[3], mx[4], mx[5]),
                          fmaxf(mx[6], mx[7])) * mul;
  const bool need = top > m + kRescaleSlack;
  float alpha = 1.f;
  if (need) {
    alpha = ex2(m - top);
    m = top;
  }
  l *= alpha;
  const float ref = m == -INFINITY ? 0.f : m;
  const float up = kPromptLift<BF16> - ref;
  const float2 neg = make_float2(up, up), mul2 = make_float2(mul, mul);
  const float2 one = make_float2(1.f, 1.f);
  float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    uint32_t h[32];
#pragma unroll
    for (int q = 0; q < 32; ++q) {
      const int c = 64 * half + 2 * q;
      const float2 x = ffma2(make_float2(p[c], p[c + 1]), mul2, neg);
      float2 e;
      if (q % 8 == 7) {   // one pair in eight on the FMA pipe (packed batch 306.5 -> 300.6 us)
        float2 u, s;
        exp2_fma(x, u, s);
        e = fmul2(u, s);
      } else {
        e = make_float2(ex2(x.x), ex2(x.y));
      }
      h[q] = pack2<BF16>(e.x, e.y);
      sum[q & 1] = ffma2(e, one, sum[q & 1]);
    }
    tmem_st32u_async(s_addr + 32 * half, h);
  }
  l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
  if (!first && __any_sync(0xffffffffu, need)) {
#pragma unroll 1
    for (int c = 0; c < D / 32; ++c) {
      float o[32];
      tmem_ld32(o_addr + 32 * c, o);
#pragma unroll
      for (int q = 0; q < 32; ++q) o[q] *= alpha;
      tmem_st32(o_addr + 32 * c, o);
    }
  }
  tmem_wait_st();
}

template <int D, bool BF16, bool kHalves>
__global__ void __launch_bounds__(kPromptThreads, 1)
    prompt_attention_kernel(const __grid_constant__ CUtensorMap qmap,
                            const __grid_constant__ CUtensorMap kmap,
                            const __grid_constant__ CUtensorMap vmap, const PromptArgs a) {
  using L = PromptSmem<D>;
  constexpr int NST = L::NST;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sb = smem_addr(smem);
  const int warp = warp_uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (warp == kWarpTma && lane == 0) {
    prefetch_tensormap(&qmap);
    prefetch_tensormap(&kmap);
    prefetch_tensormap(&vmap);
  }
  pdl_launch_dependents();
  pdl_wait();

  const int G = a.group, span = kHalves ? a.tile_tokens : 2 * a.tile_tokens;
  int4* seqs = reinterpret_cast<int4*>(smem + L::kSeqs);
  int* list = reinterpret_cast<int*>(smem + L::kList);
  const PromptOrder order = prompt_order(a, span, reinterpret_cast<int*>(smem + L::kSched), seqs,
                                         list, warp, lane);
  const int total = order.total * a.num_kv_heads;
  if (prefill_item_index(0, total, blockIdx.x, gridDim.x) < 0) return;
  const int q_rows = a.tile_tokens * G;

  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kAbort);
  volatile int* mark = reinterpret_cast<volatile int*>(smem + L::kMark);
  if (threadIdx.x == 0) {
    mbar_init(sb + L::kBarQ, 1);
    mbar_init(sb + L::kBarQFree, 1);
    for (int i = 0; i < NST; ++i) {
      mbar_init(sb + L::kBarKFull + 8 * i, 1);
      mbar_init(sb + L::kBarKEmpty + 8 * i, 1);
      mbar_init(sb + L::kBarVFull + 8 * i, 1);
      mbar_init(sb + L::kBarVEmpty + 8 * i, 1);
      mbar_init(sb + L::kBarVOk + 8 * i, kGuardWarps * 32);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(sb + L::kBarS + 8 * t, 1);
      mbar_init(sb + L::kBarP + 8 * t, 128);
      mbar_init(sb + L::kBarOFull + 8 * t, 1);
      mbar_init(sb + L::kBarOFree + 8 * t, kHalves ? 256 : 128);
    }
    mbar_init(sb + L::kBarEnd, 1);
    *abort_flag = 0;
    *mark = 0;
    fence_barrier_init();
  }
  if (warp == kWarpMma) tmem_alloc(sb + L::kTmemSlot, kTmemCols);
  if (warp < 8 && q_rows < kPrefillRows) {
    // rows no Q box covers: zero, so that they are finite (they are masked)
    const int t = warp >> 2, chunks = (kPrefillRows - q_rows) * 8;
    for (int i = threadIdx.x & 127; i < chunks * L::kSlabs; i += 128) {
      const int b = i / chunks, c = i % chunks;
      sts128(sb + L::kQ + t * L::kQTile + b * L::kSlab + q_rows * 128 + c * 16, 0u, 0u, 0u, 0u);
    }
    fence_proxy_async_smem();
  }
  tmem_fence_before_sync();
  __syncthreads();
  tmem_fence_after_sync();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + L::kTmemSlot);
  const int wgroup = warp >> 2;

  if (wgroup == 2) {
    regs_shrink<kPromptRegsOther>();
    if (warp == kWarpTma) {
      // ================= loads =================
      int n_q = 0, issued = 0, k_issued = 0, v_issued = 0;
      bool ok = true;
      for (int k = 0; ok; ++k) {
        const int i = prefill_item_index(k, total, blockIdx.x, gridDim.x);
        if (i < 0) break;
        PromptItem it;
        prompt_item<kHalves>(a, order, seqs, list, i, span, it);
        // the first K block goes ahead of Q, which has to wait for the last
        // item's S products
        const int nkb = it.blocks;
        for (int j = 0; j < nkb; ++j, ++issued) {
          const int st = issued % NST;
          const uint32_t par = ((issued / NST) & 1) ^ 1;
          const int row = it.q0 + j * kPrefillKeys;
          if (issued >= NST && !(ok = __all_sync(0xffffffffu, wait_or_abort(
                                     sb + L::kBarKEmpty + 8 * st, par, abort_flag))))
            break;
          if (lane == 0) {
            mbar_arrive_expect_tx(sb + L::kBarKFull + 8 * st, L::kStage);
#pragma unroll
            for (int b = 0; b < L::kSlabs; ++b)
              tma_load_4d(sb + L::kK + st * L::kStage + b * L::kSlab, &kmap,
                          sb + L::kBarKFull + 8 * st, 0, b, it.kvh, row);
          }
          __syncwarp();
          k_issued = issued + 1;
          if (j == 0) {
            if (n_q > 0 && !(ok = __all_sync(0xffffffffu, wait_or_abort(
                                 sb + L::kBarQFree, (n_q - 1) & 1, abort_flag))))
              break;
            if (lane == 0) {
              const int tiles = !kHalves && it.lim[1] > 0 ? 2 : 1;
              mbar_arrive_expect_tx(sb + L::kBarQ, tiles * L::kSlabs * q_rows * 128);
              for (int t = 0; t < tiles; ++t) {
#pragma unroll
                for (int b = 0; b < L::kSlabs; ++b)
                  tma_load_4d(sb + L::kQ + t * L::kQTile + b * L::kSlab, &qmap, sb + L::kBarQ, 0,
                              b, it.kvh * G, it.q0 + it.tile_a + t * a.tile_tokens);
              }
            }
            __syncwarp();
            ++n_q;
          }
          if (issued >= NST && !(ok = __all_sync(0xffffffffu, wait_or_abort(
                                     sb + L::kBarVEmpty + 8 * st, par, abort_flag))))
            break;
          if (lane == 0) {
            mbar_arrive_expect_tx(sb + L::kBarVFull + 8 * st, L::kStage);
#pragma unroll
            for (int b = 0; b < L::kSlabs; ++b)
              tma_load_4d(sb + L::kV + st * L::kStage + b * L::kSlab, &vmap,
                          sb + L::kBarVFull + 8 * st, 0, b, it.kvh, row);
          }
          __syncwarp();
          v_issued = issued + 1;
        }
      }
      // every load issued lands before the CTA can exit
      if (n_q > 0 && !mbar_wait_bounded(sb + L::kBarQ, (n_q - 1) & 1) && lane == 0)
        record_error(kErrWaitTimeout, blockIdx.x);
      for (int g = max(0, k_issued - NST); g < k_issued; ++g)
        mbar_wait_bounded(sb + L::kBarKFull + 8 * (g % NST), (g / NST) & 1);
      for (int g = max(0, v_issued - NST); g < v_issued; ++g)
        mbar_wait_bounded(sb + L::kBarVFull + 8 * (g % NST), (g / NST) & 1);
    } else if (warp == kWarpMma) {
      // ================= MMA issuer =================
      constexpr uint32_t kIdS = umma_idesc_f16(BF16, kPrefillRows, kPrefillKeys, false);
      constexpr uint32_t kIdO = umma_idesc_f16(BF16, kPrefillRows, D, true);
      constexpr uint32_t kStage16 = L::kStage / 16;
      const uint32_t tm = warp_uniform(tmem);
      const uint64_t qdesc = umma_desc_sw128(sb + L::kQ, 16, 1024);
      const uint64_t kdesc = umma_desc_sw128(sb + L::kK, 16, 1024);
      const uint64_t vdesc = umma_desc_sw128(sb + L::kV, L::kSlab, 1024);
      const bool leader = elect_lane();
      auto issue_s = [&](int t, int st) {
        const uint64_t q = qdesc + (kHalves ? 0 : t * (L::kQTile / 16)), kd = kdesc + st * kStage16;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = ((kk >> 2) * L::kSlab + (kk & 3) * 32) / 16;
          umma_f16_ss(tm + kTmemS + 128 * t, q + off, kd + off, kIdS, kk > 0 ? 1u : 0u);
        }
        umma_commit(sb + L::kBarS + 8 * t);
      };
      // O_t (+)= P_t V over the 16-key steps below the tile's last key (`keys` of the block)
      auto issue_pv = [&](int t, int st, bool first, int keys) {
        const uint64_t vd = vdesc + st * kStage16;
        const uint32_t o = tm + kTmemO + 128 * t, p = tm + kTmemS + 128 * t;
        if (keys > kPrefillKeys - 16) {
#pragma unroll
          for (int k = 0; k < kPrefillKeys / 16; ++k)
            umma_f16_ts(o, p + 8 * k, vd + k * 128, kIdO, k > 0 || !first ? 1u : 0u);
        } else {
          for (int k = 0; k * 16 < keys; ++k)
            umma_f16_ts(o, p + 8 * k, vd + k * 128, kIdO, k > 0 || !first ? 1u : 0u);
        }
      };
      auto wait = [&](uint32_t bar, uint32_t parity) {
        const bool r = __all_sync(0xffffffffu, wait_or_abort(bar, parity, abort_flag));
        tmem_fence_after_sync();
        return r;
      };
      // The issue order is S_A(j), P_B(j-1) V, S_B(j), P_A(j) V, so that each
      // tile's softmax overlaps the other tile's products.  g: blocks so far
      // (st their stage, par its phase); done[t], items[t]: S/P rounds and items
      // of tile t.
      int n_q = 0, st = 0, par = 0, done[2] = {0, 0}, items[2] = {0, 0};
      bool ok = true;
      for (int k = 0; ok; ++k) {
        const int i = prefill_item_index(k, total, blockIdx.x, gridDim.x);
        if (i < 0) break;
        PromptItem it;
        prompt_item<kHalves>(a, order, seqs, list, i, span, it);
        const int nkb[2] = {warp_uniform(it.nkb[0]), warp_uniform(it.nkb[1])};
        const int lim[2] = {warp_uniform(it.lim[0]), warp_uniform(it.lim[1])};
        const int blocks = warp_uniform(it.blocks);
        // P_t of block j (stage vs) is in: its product, after the epilogue has
        // read the last item's O_t
        auto pv = [&](int t, int j, int vs) {
          if (j == 0 && items[t] > 0 && !wait(sb + L::kBarOFree + 8 * t, (items[t] - 1) & 1))
            return false;
          if (!wait(sb + L::kBarP + 8 * t, (done[t] + j) & 1)) return false;
          if (leader) {
            issue_pv(t, vs, j == 0, lim[t] - j * kPrefillKeys);
            if (j == nkb[t] - 1) umma_commit(sb + L::kBarOFull + 8 * t);
          }
          __syncwarp();
          return true;
        };
        if (!(ok = wait(sb + L::kBarQ, n_q & 1))) break;
        ++n_q;
        if constexpr (kHalves) {
          // S(j) by the half j & 1, then P(j - 1) V by the other
          int last = 0, last_par = 0;
          for (int j = 0; j <= blocks; ++j) {
            if (j < blocks) {
              if (!(ok = wait(sb + L::kBarKFull + 8 * st, par))) break;
              if (leader) {
                if (j & 1) issue_s(1, st);
                else issue_s(0, st);
                umma_commit(sb + L::kBarKEmpty + 8 * st);
                if (j == blocks - 1) umma_commit(sb + L::kBarQFree);
              }
              __syncwarp();
            }
            if (j > 0) {
              const int t = (j - 1) & 1, r = (j - 1) >> 1;
              if (!(ok = wait(sb + L::kBarVOk + 8 * last, last_par))) break;
              // (both epilogue halves free both accumulators at once)
              if (r == 0 && items[0] > 0 &&
                  !(ok = wait(sb + L::kBarOFree, (items[0] - 1) & 1)))
                break;
              if (!(ok = wait(sb + L::kBarP + 8 * t, (done[t] + r) & 1))) break;
              if (leader) {
                const int keys = lim[0] - (j - 1) * kPrefillKeys;
                if (t) issue_pv(1, last, r == 0, keys);
                else issue_pv(0, last, r == 0, keys);
                umma_commit(sb + L::kBarVEmpty + 8 * last);
                if (r == nkb[t] - 1) umma_commit(sb + L::kBarOFull + 8 * t);
              }
              __syncwarp();
            }
            last = st;
            last_par = par;
            if (j < blocks && ++st == NST) {
              st = 0;
              par ^= 1;
            }
          }
          if (!ok) break;
          done[0] += nkb[0];
          done[1] += nkb[1];
          ++items[0];
          continue;
        }
        if (!(ok = wait(sb + L::kBarKFull + 8 * st, par))) break;
        int last = 0;                      // the stage of the block before
        for (int j = 0; j <= blocks && ok; ++j) {
          if (j < nkb[0]) {
            if (leader) issue_s(0, st);
            __syncwarp();
          }
          if (j > 0 && j - 1 < nkb[1] && !(ok = pv(1, j - 1, last))) break;
          if (leader) {
            if (j > 0) umma_commit(sb + L::kBarVEmpty + 8 * last);
            if (j < nkb[1]) issue_s(1, st);
            if (j < blocks) umma_commit(sb + L::kBarKEmpty + 8 * st);
            if (j == blocks - 1) umma_commit(sb + L::kBarQFree);
          }
          __syncwarp();
          if (j < blocks) {
            // V of this block and K of the next one, while P_A is on its way
            if (!(ok = wait(sb + L::kBarVOk + 8 * st, par))) break;
            last = st;
            if (++st == NST) {
              st = 0;
              par ^= 1;
            }
            if (j + 1 < blocks && !(ok = wait(sb + L::kBarKFull + 8 * st, par))) break;
            if (j < nkb[0] && !(ok = pv(0, j, last))) break;
          }
        }
        if (!ok) break;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          done[t] += nkb[t];
          items[t] += nkb[t] > 0;
        }
      }
      if (leader) umma_commit(sb + L::kBarEnd);
      __syncwarp();
      if (!mbar_wait_bounded(sb + L::kBarEnd, 0) && lane == 0)
        record_error(kErrWaitTimeout, blockIdx.x);
    } else {
      // ================= guard: V blocks with keys some row does not see =================
      const int ct = threadIdx.x - kWarpGuard * 32;
      constexpr uint32_t kExp = BF16 ? 0x7f807f80u : 0x7c007c00u;
      int g0 = 0;
      bool ok = true;
      for (int k = 0; ok; ++k) {
        const int i = prefill_item_index(k, total, blockIdx.x, gridDim.x);
        if (i < 0) break;
        PromptItem it;
        prompt_item<kHalves>(a, order, seqs, list, i, span, it);
        const int nkb = it.blocks;
        for (int j = 0; j < nkb; ++j) {
          const int g = g0 + j, st = g % NST;
          if (!(ok = __all_sync(0xffffffffu, wait_or_abort(sb + L::kBarVFull + 8 * st,
                                                           (g / NST) & 1, abort_flag))))
            break;
          if ((j + 1) * kPrefillKeys > it.tile_a + 1) {   // past the keys of the item's first row
            const uint32_t vst = sb + L::kV + st * L::kStage;
            bool found = false;
            for (int c = ct; c < L::kStage / 16; c += kGuardWarps * 32) {
              uint32_t w[4];
              asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                           : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(vst + c * 16));
              uint32_t hit[4], any = 0;
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                hit[q] = __vcmpeq2(w[q] & kExp, kExp);
                any |= hit[q];
              }
              if (any) {
                found = true;
                sts128(vst + c * 16, w[0] & ~hit[0], w[1] & ~hit[1], w[2] & ~hit[2],
                       w[3] & ~hit[3]);
              }
            }
            if (found) *mark = 1;
            fence_proxy_async_smem();
          }
          mbar_arrive(sb + L::kBarVOk + 8 * st);
        }
        g0 += nkb;
      }
    }
  } else {
    // ================= softmax: tile t = warp / 4, row = tensor-memory lane =================
    regs_grow<kPromptRegsSoftmax>();
    const int t = wgroup;
    const int row = threadIdx.x & 127;
    const uint32_t t_lane = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const uint32_t s_addr = t_lane + kTmemS + 128 * t, o_addr = t_lane + kTmemO + 128 * t;
    const float sl2 = a.scale_log2;
    int done = 0, items = 0, twos = 0;   // twos: items with blocks for both halves
    bool ok = true;
    for (int k = 0; ok; ++k) {
      const int i = prefill_item_index(k, total, blockIdx.x, gridDim.x);
      if (i < 0) break;
      PromptItem it;
      prompt_item<kHalves>(a, order, seqs, list, i, span, it);
      if (it.lim[t] == 0) continue;
      const int tok0 = it.tile_a + (kHalves ? 0 : t * a.tile_tokens);
      const int tok = tok0 + row / G;                             // this row's token
      const bool live = row < q_rows && tok < it.len;
      const int lim = live ? tok + 1 : it.blocks * kPrefillKeys;   // (what a row of no token holds is not written)
      float m = -INFINITY, l = 0.f;
      const int nkb = it.nkb[t];
      for (int j = 0; j < nkb; ++j) {
        // S_t(j) is in, and with it every earlier P_t V: O_t is current
        ok = __all_sync(0xffffffffu, wait_or_abort(sb + L::kBarS + 8 * t, (done + j) & 1,
                                                   abort_flag));
        if (!ok) break;
        tmem_fence_after_sync();
        float p[kPrefillKeys];
        tmem_ld128_x32(s_addr, p);
        prompt_softmax_block<BF16, D>(p, j == 0,
                                      lim - (kHalves ? 2 * j + t : j) * kPrefillKeys, sl2, m, l, s_addr,
                                      o_addr);
        tmem_fence_before_sync();
        mbar_arrive(sb + L::kBarP + 8 * t);
      }
      if (!ok) break;
      done += nkb;
      const int of = kHalves ? 0 : t;
      ok = __all_sync(0xffffffffu, wait_or_abort(sb + L::kBarOFull + 8 * of, items & 1,
                                                 abort_flag));
      if (!ok) break;
      // Both halves are in: each takes half of the columns of
      // O = 2^(m_a - m) O_a + 2^(m_b - m) O_b, from the same lanes of tensor memory
      float fa = 1.f, fb = 0.f;
      const bool two = kHalves && it.nkb[1] > 0;
      if constexpr (kHalves) {
        if (two && !(ok = __all_sync(0xffffffffu, wait_or_abort(sb + L::kBarOFull + 8, twos & 1,
                                                                abort_flag))))
          break;
        // (the exchange's last readers arrived at OFree before this item's products began)
        float2* ml = reinterpret_cast<float2*>(smem + L::kHalfStats);
        ml[128 * t + row] = make_float2(m, l);
        mbar_arrive(sb + L::kBarHalves);
        ok = __all_sync(0xffffffffu, wait_or_abort(sb + L::kBarHalves, items & 1, abort_flag));
        if (!ok) break;
        const float2 ha = ml[row], hb = ml[128 + row];
        m = fmaxf(ha.x, hb.x);
        const float ref = m == -INFINITY ? 0.f : m;
        fa = ex2(ha.x - ref);
        fb = ex2(hb.x - ref);
        l = fa * ha.y + fb * hb.y;
      }
      // ---- O / l, and the log-sum-exp ----
      tmem_fence_after_sync();
      const bool marked = *mark != 0;
      const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);   // a NaN stays one
      const size_t hrow = static_cast<size_t>(it.q0 + tok) * a.num_heads + it.kvh * G + row % G;
      if (live && a.lse && (!kHalves || t == 0))
        a.lse[hrow] = m * kLn2 + logf(l * kPromptDrop<BF16>);
      // 32 columns at a time through shared memory (16-byte chunk c of row r at
      // c ^ (r / 2 % 4), free of bank conflicts), so that four lanes store a row's
      // 64 bytes: a lane a row touched 32 lines a store, and the epilogue took
      // 3700 to 6000 cycles an item
      const uint32_t stage = sb + L::kStore + warp * 2048;
      const int r0 = warp & 3;                         // this warp's rows: 32 r0 ..
      const int c_end = kHalves ? (t + 1) * (D / 64) : D / 32;
#pragma unroll 1
      for (int c = kHalves ? t * (D / 64) : 0; c < c_end; ++c) {
        float o[32];
        tmem_ld32((kHalves ? t_lane + kTmemO : o_addr) + 32 * c, o);
        if constexpr (kHalves) {
          if (two) {
            float b[32];
            tmem_ld32(t_lane + kTmemO + 128 + 32 * c, b);
#pragma unroll
            for (int q = 0; q < 32; ++q) o[q] = fa * o[q] + fb * b[q];
          }
        }
        if (c == c_end - 1) {                          // O_t is in registers
          tmem_fence_before_sync();
          mbar_arrive(sb + L::kBarOFree + 8 * of);
        }
        if (marked && live) {
          // what the guard took out, for the keys this row sees
          for (int j = (it.tile_a + 1) / kPrefillKeys * kPrefillKeys; j < lim; ++j) {
            const uint16_t* v = a.value + (it.q0 + j) * a.value_stride + it.kvh * D + 32 * c;
#pragma unroll
            for (int q = 0; q < 32; ++q) {
              const float2 x = unpack2<BF16>(v[q]);
              if (!isfinite(x.x)) o[q] += x.x;
            }
          }
        }
        __syncwarp();                                  // the rows before have been read
#pragma unroll
        for (int q = 0; q < 4; ++q)
          sts128(stage + lane * 64 + ((q ^ (lane >> 1 & 3)) << 4),
                 pack2<BF16>(o[8 * q + 0] * inv, o[8 * q + 1] * inv),
                 pack2<BF16>(o[8 * q + 2] * inv, o[8 * q + 3] * inv),
                 pack2<BF16>(o[8 * q + 4] * inv, o[8 * q + 5] * inv),
                 pack2<BF16>(o[8 * q + 6] * inv, o[8 * q + 7] * inv));
        __syncwarp();
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int r = 8 * q + (lane >> 2), ch = lane & 3, tr = 32 * r0 + r;
          uint4 v;
          asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                       : "r"(stage + r * 64 + ((ch ^ (r >> 1 & 3)) << 4)));
          const int rt = tok0 + tr / G;
          if (tr < q_rows && rt < it.len)
            *reinterpret_cast<uint4*>(a.out +
                (static_cast<size_t>(it.q0 + rt) * a.num_heads + it.kvh * G + tr % G) * D +
                32 * c + 8 * ch) = v;
        }
      }
      ++items;
      twos += two;
    }
  }

  tmem_fence_before_sync();
  __syncthreads();
  if (warp == kWarpMma) {
    tmem_fence_after_sync();
    tmem_dealloc(tmem, kTmemCols);
  }
}

}  // namespace pa
