// pa_prompt_weights.cuh -- the attention weight each token of a packed prompt
// receives from the last `window` tokens of its sequence:
//   weights_j = sum over those query tokens i >= j and the G heads g of
//               exp(scale q_gi . k_j - lse_gi),
// given the attention's own log-sum-exp.  No softmax is redone: one product, one
// 2^x and one addition an element.
//
// The products run transposed on the tensor cores, S^T = K Q^T: 128 keys as the
// MMA's rows, the query rows of a tile (128 / G tokens x G heads, token-major)
// as its columns.  A thread then owns a key (its tensor-memory lane) and sums
// over its columns in registers; nothing is shuffled, no sum leaves the thread
// before it is written, and the order of the additions is fixed.
//
// Work item: (sequence, KV head, two blocks of 128 keys).  The item's K stays in
// shared memory (two items' in flight) while the query tiles stream through a
// ring, each loaded once for both key blocks.  Four consumer warpgroups: key block
// b of the even tiles and of the odd ones, each with an S^T buffer of its own, so
// that the next tile's product runs during this one's 2^x and the four warps of a
// scheduler are at different places.  At the end of an item the two partial sums
// of a key meet in shared memory.  Where there are few items, a cluster of up to
// eight CTAs takes one: CTA r the query tiles r, r + C, ..., and the first CTA adds
// the others' sums up, in their order, as they arrive in its shared memory.  Warps: 0-15 the
// sums, 16 issues the MMAs, 17 the loads, 18 brings each tile's lse into shared
// memory (negated, in log2 units).
//
// Measured: prompts of 4096 and 1333 tokens, 32 heads of 128, whole: 107 us, 2.3
// times what the products alone take at cuBLAS's rate (46; the 13 of 16 2^x that are
// left to the special-function unit take 54); that unit is 60 % used, issue slots 50 %,
// the tensor pipe 35 %.  Instead of the even/odd split, four key blocks an item with a
// warpgroup each took 124 us where it took 115, one block's columns over four warpgroups
// 130.  One prompt of 4096 tokens, 32 heads over 8 (128 items): 104 us with clusters of
// four, 175 without; of 1000 tokens 24 and 48.
#pragma once

#include "pa_prompt.cuh"

namespace pa {

constexpr int kPwBlocks = 2;                    // key blocks of an item
constexpr int kPwSpan = 128 * kPwBlocks;        // keys of an item
constexpr int kPwThreads = 19 * 32;
constexpr int kPwWarpMma = 16, kPwWarpTma = 17, kPwWarpLse = 18;

struct PromptWeightsArgs {
  float* weights;              // [S, Hk, max_tokens]
  const float* lse;            // [T, H]
  const int32_t* seq_starts;   // [S + 1]
  float scale_log2;
  int num_seqs;
  int num_tokens;
  int num_heads;
  int num_kv_heads;
  int group;
  int tile_tokens;
  int cluster;                 // CTAs of an item
  int max_tokens;
  int window;
};

template <int D>
struct PwSmem {
  static constexpr int kSlabs = D / 64;
  static constexpr int kSlab = 128 * 128;
  static constexpr int kTile = kSlabs * kSlab;        // one key block, or one query tile
  static constexpr int NK = 2;                        // items' K in flight
  static constexpr int NQ = D == 64 ? 4 : 2;          // query tiles in flight
  static constexpr int NL = 4;                        // tiles' lse in flight
  static constexpr int kK = 0;
  static constexpr int kQ = kK + NK * kPwBlocks * kTile;
  static constexpr int kLse = kQ + NQ * kTile;        // NL x 128 floats
  static constexpr int kBarKFull = kLse + NL * 512;
  static constexpr int kBarKEmpty = kBarKFull + 8 * NK;
  static constexpr int kBarSFull = kBarKEmpty + 8 * NK;    // [block][tile parity]
  static constexpr int kBarSEmpty = kBarSFull + 8 * 4;
  static constexpr int kBarQFull = kBarSEmpty + 8 * 4;
  static constexpr int kBarQEmpty = kBarQFull + 8 * NQ;
  static constexpr int kBarLFull = kBarQEmpty + 8 * NQ;
  static constexpr int kBarLEmpty = kBarLFull + 8 * NL;
  static constexpr int kBarSums = kBarLEmpty + 8 * NL;     // an item's partial sums are in
  static constexpr int kBarCFull = kBarSums + 8;           // the other CTAs' sums, two items,
  static constexpr int kBarCFree = kBarCFull + 16;         // and that they have been added up
  static constexpr int kBarEnd = kBarCFree + 16;
  static constexpr int kTmemSlot = kBarEnd + 8;
  static constexpr int kAbort = kTmemSlot + 4;
  static constexpr int kSched = kAbort + 4;
  static constexpr int kSeqs = (kSched + 128 + 15) & ~15;
  static constexpr int kList = kSeqs + 16 * kPromptRankSeqs;
  static constexpr int kSums = kList + 4 * kPromptRankUnits;   // of two items: one float a key
  static constexpr int kOthers = kSums + 2 * kPwSpan * 4;   // two items, 7 CTAs, a float a key
  static constexpr int kBytes = kOthers + 2 * 7 * kPwSpan * 4;
  static constexpr int kAlloc = kBytes + 1024;        // one CTA per SM: both sizes pass 114 KB
  static_assert(kBytes > 114 * 1024, "one CTA holds all of an SM's tensor memory");
};

struct PwItem {
  int s, kvh, q0, len;   // sequence, KV head, its first row and its length
  int k0;                // first key
  int blocks;            // key blocks
  int t0, step, tiles;   // first token of this CTA's first query tile, tokens from one of its
                         // tiles to the next, and their number
};

// The pairs of a sequence are ranked as the attention's are (more keys, more
// work); here the first keys are seen by most tokens.
__device__ __forceinline__ void pw_item(const PromptWeightsArgs& a, const PromptOrder& o,
                                        const int4* seqs, const int* list, int i, int rank,
                                        PwItem& it) {
  const int u = i / a.num_kv_heads;
  it.kvh = i - u * a.num_kv_heads;
  const PromptUnit unit = prompt_unit(a, o, seqs, list, u, kPwSpan);
  it.s = unit.s;
  it.q0 = unit.q0;
  it.len = unit.len;
  it.k0 = ((it.len + kPwSpan - 1) / kPwSpan - 1 - unit.pair) * kPwSpan;
  it.t0 = max(it.k0, it.len - a.window) + rank * a.tile_tokens;
  it.step = a.cluster * a.tile_tokens;
  it.tiles = max(0, it.len - it.t0 + it.step - 1) / it.step;
  it.blocks = min(kPwBlocks, (it.len - it.k0 + 127) / 128);
}

// The first of its query tiles that sees a key of block b.
__device__ __forceinline__ int pw_first(const PwItem& it, int tile_tokens, int b) {
  const int before = it.k0 + 128 * b - it.t0 - (tile_tokens - 1);   // its last token reaches the key
  return before > 0 ? (before + it.step - 1) / it.step : 0;
}

// Barriers of another CTA of the cluster, and waits for what other CTAs wrote.
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar)
               : "memory");
}
__device__ __forceinline__ bool mbar_wait_cluster(uint32_t bar, uint32_t parity,
                                                  volatile int* abort_flag) {
  const unsigned long long t0 = global_timer_ns();
  for (;;) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done) : "r"(bar), "r"(parity) : "memory");
    if (done) return true;
    if (*abort_flag) return false;
    if (global_timer_ns() - t0 > kWaitLimitNs) {
      *abort_flag = 1;
      record_error(kErrWaitTimeout, blockIdx.x);
      return false;
    }
  }
}

// sum += 2^(s scale + neg) over 32 columns, three pairs of sixteen on the FMA
// pipe and the others on the special-function unit (4096 + 1333 tokens, 32 heads,
// whole: none 113.7 us, two 110.6, three 107.1, four 108.5, six 113.3).  `most` is the largest exponent on the FMA pipe: from 129 on
// exp2_fma's results wrap around.
__device__ __forceinline__ void add_columns(const float (&s)[32], const float4* neg4, float2 scale,
                                            float2 (&sum)[2], float& most) {
  const float2 one = make_float2(1.f, 1.f);
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    const float4 neg = neg4[q];
    const float2 x = ffma2(make_float2(s[4 * q], s[4 * q + 1]), scale, make_float2(neg.x, neg.y));
    const float2 y = ffma2(make_float2(s[4 * q + 2], s[4 * q + 3]), scale, make_float2(neg.z, neg.w));
    if (q == 1 || q == 3 || q == 5) {
      float2 p, e;
      exp2_fma<1>(x, p, e);
      most = fmax3(most, x.x, x.y);
      sum[0] = ffma2(p, e, sum[0]);
    } else {
      sum[0] = ffma2(make_float2(ex2(x.x), ex2(x.y)), one, sum[0]);
    }
    sum[1] = ffma2(make_float2(ex2(y.x), ex2(y.y)), one, sum[1]);
  }
}

template <int D, bool BF16>
__global__ void __launch_bounds__(kPwThreads, 1)
    prompt_weights_kernel(const __grid_constant__ CUtensorMap qmap,
                          const __grid_constant__ CUtensorMap kmap, const PromptWeightsArgs a) {
  using L = PwSmem<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sb = smem_addr(smem);
  const int warp = warp_uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (warp == kPwWarpTma && lane == 0) {
    prefetch_tensormap(&qmap);
    prefetch_tensormap(&kmap);
  }
  pdl_launch_dependents();
  pdl_wait();

  const int G = a.group;
  int4* seqs = reinterpret_cast<int4*>(smem + L::kSeqs);
  int* list = reinterpret_cast<int*>(smem + L::kList);
  const PromptOrder order = prompt_order(a, kPwSpan, reinterpret_cast<int*>(smem + L::kSched),
                                         seqs, list, warp, lane);
  const int total = order.total * a.num_kv_heads;
  const int C = a.cluster, rank = blockIdx.x % C;
  const int cid = blockIdx.x / C, clusters = gridDim.x / C;
  if (prefill_item_index(0, total, cid, clusters) < 0) return;
  const int q_rows = a.tile_tokens * G;
  float* lse_sh = reinterpret_cast<float*>(smem + L::kLse);

  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kAbort);
  if (threadIdx.x == 0) {
    for (int i = 0; i < L::NK; ++i) {
      mbar_init(sb + L::kBarKFull + 8 * i, 1);
      mbar_init(sb + L::kBarKEmpty + 8 * i, 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(sb + L::kBarSFull + 8 * i, 1);
      mbar_init(sb + L::kBarSEmpty + 8 * i, 128);
    }
    mbar_init(sb + L::kBarSums, 512);
    for (int i = 0; i < 2; ++i) {
      mbar_init(sb + L::kBarCFull + 8 * i, max(1, C - 1) * kPwSpan);
      mbar_init(sb + L::kBarCFree + 8 * i, kPwSpan);
    }
    for (int i = 0; i < L::NQ; ++i) {
      mbar_init(sb + L::kBarQFull + 8 * i, 1);
      mbar_init(sb + L::kBarQEmpty + 8 * i, 1);
    }
    for (int i = 0; i < L::NL; ++i) {
      mbar_init(sb + L::kBarLFull + 8 * i, 32);
      mbar_init(sb + L::kBarLEmpty + 8 * i, 256);
    }
    mbar_init(sb + L::kBarEnd, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == kPwWarpMma) tmem_alloc(sb + L::kTmemSlot, kTmemCols);
  if (warp < kPwWarpMma && q_rows < 128) {   // rows no query box covers: finite (their lse is +inf)
    const int chunks = (128 - q_rows) * 8;
    for (int i = threadIdx.x; i < chunks * L::kSlabs * L::NQ; i += 512) {
      const int b = i / chunks, c = i % chunks;
      sts128(sb + L::kQ + b * L::kSlab + q_rows * 128 + c * 16, 0u, 0u, 0u, 0u);
    }
    fence_proxy_async_smem();
  }
  tmem_fence_before_sync();
  if (C > 1) {
    __syncwarp();
    cluster_sync();            // every CTA's barriers are ready
  } else {
    __syncthreads();
  }
  tmem_fence_after_sync();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + L::kTmemSlot);
  auto wait = [&](uint32_t bar, uint32_t parity) {
    return __all_sync(0xffffffffu, wait_or_abort(bar, parity, abort_flag)) != 0;
  };

  if (warp == kPwWarpTma) {
    // ================= loads =================
    int nk = 0, nq = 0;
    bool ok = true;
    for (int k = 0; ok; ++k) {
      const int i = prefill_item_index(k, total, cid, clusters);
      if (i < 0) break;
      PwItem it;
      pw_item(a, order, seqs, list, i, rank, it);
      if (it.tiles == 0) continue;
      const int ks = nk % L::NK;
      if (nk >= L::NK && !(ok = wait(sb + L::kBarKEmpty + 8 * ks, ((nk / L::NK) & 1) ^ 1))) break;
      if (lane == 0) {
        mbar_arrive_expect_tx(sb + L::kBarKFull + 8 * ks, it.blocks * L::kTile);
        for (int b = 0; b < it.blocks; ++b) {
#pragma unroll
          for (int c = 0; c < L::kSlabs; ++c)
            tma_load_4d(sb + L::kK + (ks * kPwBlocks + b) * L::kTile + c * L::kSlab, &kmap,
                        sb + L::kBarKFull + 8 * ks, 0, c, it.kvh, it.q0 + it.k0 + 128 * b);
        }
      }
      __syncwarp();
      ++nk;
      for (int j = 0; j < it.tiles && ok; ++j) {
        const int qs = nq % L::NQ;
        if (nq >= L::NQ && !(ok = wait(sb + L::kBarQEmpty + 8 * qs, ((nq / L::NQ) & 1) ^ 1))) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(sb + L::kBarQFull + 8 * qs, L::kSlabs * q_rows * 128);
#pragma unroll
          for (int c = 0; c < L::kSlabs; ++c)
            tma_load_4d(sb + L::kQ + qs * L::kTile + c * L::kSlab, &qmap,
                        sb + L::kBarQFull + 8 * qs, 0, c, it.kvh * G,
                        it.q0 + it.t0 + j * it.step);
        }
        __syncwarp();
        ++nq;
      }
    }
    // every load issued lands before the CTA can exit
    for (int g = max(0, nk - L::NK); g < nk; ++g)
      mbar_wait_bounded(sb + L::kBarKFull + 8 * (g % L::NK), (g / L::NK) & 1);
    for (int g = max(0, nq - L::NQ); g < nq; ++g)
      mbar_wait_bounded(sb + L::kBarQFull + 8 * (g % L::NQ), (g / L::NQ) & 1);
  } else if (warp == kPwWarpMma) {
    // ================= MMA issuer =================
    constexpr uint32_t kId = umma_idesc_f16(BF16, 128, 128, false);
    const uint32_t tm = warp_uniform(tmem);
    const uint64_t kdesc = umma_desc_sw128(sb + L::kK, 16, 1024);
    const uint64_t qdesc = umma_desc_sw128(sb + L::kQ, 16, 1024);
    const bool leader = elect_lane();
    int nk = 0, nq = 0, ns = 0;          // ns: bit 2 b + h the phase of that S buffer
    bool ok = true;
    for (int k = 0; ok; ++k) {
      const int i = prefill_item_index(k, total, cid, clusters);
      if (i < 0) break;
      PwItem it;
      pw_item(a, order, seqs, list, i, rank, it);
      const int tiles = warp_uniform(it.tiles);
      if (tiles == 0) continue;
      const int first1 = warp_uniform(it.blocks > 1 ? pw_first(it, a.tile_tokens, 1) : it.tiles);
      const int ks = nk % L::NK;
      if (!(ok = wait(sb + L::kBarKFull + 8 * ks, (nk / L::NK) & 1))) break;
      for (int j = 0; j < tiles && ok; ++j, ++nq) {
        const int qs = nq % L::NQ, h = nq & 1;
        if (!(ok = wait(sb + L::kBarQFull + 8 * qs, (nq / L::NQ) & 1))) break;
#pragma unroll
        for (int b = 0; b < kPwBlocks; ++b) {
          if ((b == 1 && j < first1) || !ok) continue;
          const int buf = 2 * b + h;
          // (the phase before the first completes at once: a fresh barrier's)
          if (!(ok = wait(sb + L::kBarSEmpty + 8 * buf, ((ns >> buf) & 1) ^ 1))) continue;
          tmem_fence_after_sync();
          if (leader) {
            const uint64_t kd = kdesc + (ks * kPwBlocks + b) * (L::kTile / 16);
            const uint64_t qd = qdesc + qs * (L::kTile / 16);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint32_t off = ((kk >> 2) * L::kSlab + (kk & 3) * 32) / 16;
              umma_f16_ss(tm + 128 * buf, kd + off, qd + off, kId, kk > 0 ? 1u : 0u);
            }
            umma_commit(sb + L::kBarSFull + 8 * buf);
          }
          __syncwarp();
          ns ^= 1 << buf;
        }
        if (!ok) break;
        if (leader) {
          umma_commit(sb + L::kBarQEmpty + 8 * qs);
          if (j == tiles - 1) umma_commit(sb + L::kBarKEmpty + 8 * ks);
        }
        __syncwarp();
      }
      ++nk;
    }
    if (leader) umma_commit(sb + L::kBarEnd);
    __syncwarp();
    if (!mbar_wait_bounded(sb + L::kBarEnd, 0) && lane == 0)
      record_error(kErrWaitTimeout, blockIdx.x);
  } else if (warp == kPwWarpLse) {
    // ================= the tiles' lse =================
    int n = 0;
    bool ok = true;
    for (int k = 0; ok; ++k) {
      const int i = prefill_item_index(k, total, cid, clusters);
      if (i < 0) break;
      PwItem it;
      pw_item(a, order, seqs, list, i, rank, it);
      for (int j = 0; j < it.tiles; ++j, ++n) {
        const int sl = n % L::NL;
        const int tok0 = it.t0 + j * it.step;
        const int rows = min(a.tile_tokens, it.len - tok0) * G;
        float v[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int r = lane + 32 * u;
          v[u] = r < rows ? a.lse[static_cast<size_t>(it.q0 + tok0 + r / G) * a.num_heads +
                                  it.kvh * G + r % G]
                          : INFINITY;
        }
        if (n >= L::NL && !(ok = wait(sb + L::kBarLEmpty + 8 * sl, ((n / L::NL) & 1) ^ 1))) break;
#pragma unroll
        for (int u = 0; u < 4; ++u)   // a row without a finite logit gives nothing
          lse_sh[sl * 128 + lane + 32 * u] = v[u] == -INFINITY ? -INFINITY : -v[u] * kLog2e;
        mbar_arrive(sb + L::kBarLFull + 8 * sl);
      }
    }
  } else {
    // ================= key block b, tiles of parity h, key = tensor-memory lane ==========
    const int b = (warp >> 2) & 1, h = warp >> 3, key = threadIdx.x & 127;
    const uint32_t s_addr = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) +
                            128 * (2 * b + h);
    const uint32_t full = sb + L::kBarSFull + 8 * (2 * b + h);
    const uint32_t empty = sb + L::kBarSEmpty + 8 * (2 * b + h);
    const float2 scale = make_float2(a.scale_log2, a.scale_log2);
    float* sums = reinterpret_cast<float*>(smem + L::kSums);
    int n = 0, ns = 0, items = 0;
    bool ok = true;
    for (int k = 0; ok; ++k) {
      const int i = prefill_item_index(k, total, cid, clusters);
      if (i < 0) break;
      PwItem it;
      pw_item(a, order, seqs, list, i, rank, it);
      const int kb = it.k0 + 128 * b, kj = kb + key;
      const int first = b < it.blocks ? pw_first(it, a.tile_tokens, b) : it.tiles;
      float acc = 0.f;
      for (int j = (n & 1) ^ h; j < it.tiles; j += 2) {    // tile n + j has parity h
        const int sl = (n + j) % L::NL;
        if (!(ok = wait(sb + L::kBarLFull + 8 * sl, ((n + j) / L::NL) & 1))) break;
        if (j >= first) {
          if (!(ok = wait(full, ns & 1))) break;
          tmem_fence_after_sync();
          const int tok0 = it.t0 + j * it.step;
          const int rows = min(a.tile_tokens, it.len - tok0) * G;
          const float4* lse4 = reinterpret_cast<const float4*>(lse_sh + sl * 128);
          float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
          if (rows == q_rows && tok0 >= kb + 127) {
            float most = -INFINITY;
            // every column counts (those past q_rows are 0 and have an lse of +inf)
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
              float u[32];
              tmem_ld32(s_addr + 32 * c, u);
              if (c == 3) {
                tmem_fence_before_sync();
                mbar_arrive(empty);                    // S is in registers
                if (q_rows < 128) {
                  // (a zero query row times an infinite key is NaN; at least 117 rows are live)
#pragma unroll
                  for (int e = 117 - 96; e < 32; ++e) u[e] = 96 + e < q_rows ? u[e] : 0.f;
                }
              }
              add_columns(u, lse4 + 8 * c, scale, sum, most);
            }
            if (most >= 128.f) sum[0].x = sum[0].y = INFINITY;   // a term past the largest number
          } else {
            // columns of tokens before this key, or past the tile's rows, do not count
            const int c0 = max(0, kj - tok0) * G;
#pragma unroll 1
            for (int g = 0; g < 4; ++g) {
              float s[32];
              tmem_ld32(s_addr + 32 * g, s);
#pragma unroll
              for (int q = 0; q < 8; ++q) {
                const float4 neg = lse4[8 * g + q];
                const float n4[4] = {neg.x, neg.y, neg.z, neg.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const int c = 32 * g + 4 * q + e;
                  const float v = ex2(s[4 * q + e] * a.scale_log2 + n4[e]);
                  sum[e & 1].x += c >= c0 && c < rows ? v : 0.f;
                }
              }
            }
            tmem_fence_before_sync();
            mbar_arrive(empty);
          }
          acc += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
          ++ns;
        }
        mbar_arrive(sb + L::kBarLEmpty + 8 * sl);
      }
      if (!ok) break;
      n += it.tiles;
      // the odd tiles' sums go to the even tiles' warpgroup, and their own goes on to
      // the next item.  Two items' sums alternate: whoever writes those of the item
      // after next has waited for the next one's barrier, which the readers of this
      // one's reach later.
      float* part = sums + (items & 1) * kPwSpan;
      if (h == 1) {
        if (items > 0 && !(ok = wait(sb + L::kBarSums, (items - 1) & 1))) break;
        part[128 * b + key] = acc;
        mbar_arrive(sb + L::kBarSums);
        ++items;
        continue;
      }
      mbar_arrive(sb + L::kBarSums);
      if (!(ok = wait(sb + L::kBarSums, items & 1))) break;
      ++items;
      float sum = acc + part[128 * b + key];
      if (C > 1) {
        // slot: of two items; use: how often it has been used before
        const int slot = (items - 1) & 1, use = (items - 1) >> 1;
        const uint32_t cfull = sb + L::kBarCFull + 8 * slot, cfree = sb + L::kBarCFree + 8 * slot;
        const uint32_t others = sb + L::kOthers + slot * 7 * kPwSpan * 4 + (128 * b + key) * 4;
        if (rank > 0) {
          if (use > 0 && !(ok = __all_sync(0xffffffffu, mbar_wait_cluster(cfree, (use - 1) & 1,
                                                                          abort_flag)) != 0))
            break;
          asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(
                           map_cluster(others + (rank - 1) * kPwSpan * 4, 0)), "f"(sum)
                       : "memory");
          mbar_arrive_cluster(map_cluster(cfull, 0));
          continue;
        }
        if (!(ok = __all_sync(0xffffffffu, mbar_wait_cluster(cfull, use & 1, abort_flag)) != 0))
          break;
        for (int r = 0; r < C - 1; ++r) {
          float v;
          asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(others + r * kPwSpan * 4) : "memory");
          sum += v;
        }
        for (int r = 1; r < C; ++r) mbar_arrive_cluster(map_cluster(cfree, r));
      }
      if (it.len > a.max_tokens) {
        if (key == 0 && b == 0 && it.k0 == 0 && it.kvh == 0) record_error(kErrContextLen, it.s);
      } else if (kj < it.len && b < it.blocks) {
        a.weights[(static_cast<size_t>(it.s) * a.num_kv_heads + it.kvh) * a.max_tokens + kj] = sum;
      }
    }
  }

  tmem_fence_before_sync();
  if (C > 1) {
    __syncwarp();
    cluster_sync();            // no CTA leaves while another writes to it
  } else {
    __syncthreads();
  }
  if (warp == kPwWarpMma) {
    tmem_fence_after_sync();
    tmem_dealloc(tmem, kTmemCols);
  }
}

}  // namespace pa
