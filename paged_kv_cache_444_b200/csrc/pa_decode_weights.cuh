// pa_decode_weights.cuh -- paged decode attention that also adds up the weight
// each cached token receives.
//
// For one query token per sequence and the G query heads of a KV head,
//   z_gj = scale q_g . k_j,   p_gj = exp(z_gj - lse_g),   lse_g = log sum_j exp(z_gj),
//   out_g = sum_j p_gj v_j,   weights_j += sum_g p_gj.
// The weights need lse_g, which is known only after the last token, and the
// K rows are far larger than the logits (2 D bytes a token against 4 G): so
// the pass over K and V leaves its logits in scratch memory, and a second,
// small pass turns them into weights.
//
//   weights_split_kernel  one CTA per (sequence, KV head, partition of
//     up to kWeightsPart tokens): the page pipeline and the transposed page step of
//     the split decode (tokens and head dims as the mma's rows, heads as its
//     columns, one or two column tiles of 8), with the logits written out.
//   weights_merge_kernel  a CTA per (sequence, KV head, run of tokens) finds the
//     heads' lse from the partitions' maxima and sums, adds the weights of its
//     run up, and merges a share of the heads' output columns.
//
// The first pass is bound by HBM (128 sequences of 512 to 4096 tokens, 32/8 heads:
// 193 us for 1.26 GB, 6.5 TB/s).  K and V are loaded evict-first, so that the
// logits, small enough for L2 (16 bytes a token at G = 4), are still there when
// the second pass reads them: it reads 4 MB of its 58 from DRAM, and costs the
// call another 15 us, most of it latency at the first pass's end.  8 sequences of
// 32768 to 131072 tokens: 460 us, the second pass 35 of them.
// Few rows take smaller partitions and runs: 64 contexts of 1368 to 4104 tokens,
// 16 heads over one, 29 us instead of 51; 28 of 1899 18 instead of 26; 11 of 390 to
// 3125, 4 heads of 64, 11 instead of 17.
//
//   weights_single_kernel  both in one, a CTA per (sequence, KV head), where there
//     are enough of those: the CTA knows its heads' lse at the end of its own
//     pages.  The 128 sequences above: 198 to 203 us.
#pragma once

#include "pa_decode.cuh"

namespace pa {

constexpr int kWeightsPart = 512;          // tokens per partition, at most
constexpr int kWeightsPartMin = 128;       // and at least
constexpr int kWeightsRun = 4096;          // tokens per CTA of the second pass, at most
constexpr int kWeightsThreads = 256;
constexpr int kWeightsBatch = 4;           // tokens (or partitions of O) loaded before any is used

struct WeightsArgs {
  const uint16_t* query;         // [S, H, D]
  uint16_t* out;                 // [S, H, D]
  float* weights;                // [S, Hk, max_tokens]
  float* tmp_out;                // [S, H, P, D] partition sums of p v, p against the partition's max
  float* part_m;                 // [S, H, P] partition max, log2 units
  float* part_l;                 // [S, H, P] partition sum of p
  float* logits;                 // [S, Hk, MB * 16, G] z in log2 units
  const int32_t* block_tables;   // [S, MB]
  const int32_t* context_lens;   // [S]
  float scale_log2;
  int num_seqs;
  int num_heads;
  int num_kv_heads;
  int group;
  int max_blocks_per_seq;
  int num_blocks;
  int max_tokens;
  int new_tokens;
  int part;                      // tokens of a partition
  int run;                       // tokens of a second-pass CTA
  int parts;                     // P
  int runs;                      // CTAs per (sequence, KV head) that add weights up
};

// tma_load_4d for data read once: first to leave L2.
__device__ __forceinline__ uint64_t evict_first_policy() {
  uint64_t p;
  asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
  return p;
}
__device__ __forceinline__ void tma_load_4d_once(uint32_t dst, const CUtensorMap* map, uint32_t bar,
                                                 int c0, int c1, int c2, int c3, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".L2::cache_hint [%0], [%1, {%2, %3, %4, %5}], [%6], %7;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(bar), "l"(policy)
      : "memory");
}

// ---------------------------------------------------------------------------
// Per-warp state and page step: S^T = K Q^T, O^T = V^T P^T for NT tiles of 8
// query heads, the logits of the page's tokens written to z.  bf16 P goes in
// as a hi + lo pair; the reference max may trail the true one by 2^kSlack.
// fp16 P is one operand, as in pa_decode (at most 2^-11 of each term, the
// output's own rounding; a pair's lo of 0 would make NaN of an infinite value),
// held 2^kLift up until publish: 2^15 at most, normal down to 2^-21 of the
// reference, off by at most 2^-32 of it a token below.
// ---------------------------------------------------------------------------
template <int D, bool BF16, int NT>
struct WeightsWarp {
  static constexpr int KSTEPS = D / 16;
  static constexpr int MTILES = D / 16;
  static constexpr float kSlack = 8.f;
  static constexpr float kLift = BF16 ? 0.f : 7.f, kDrop = BF16 ? 1.f : 0x1p-7f;
  uint32_t qb[KSTEPS][NT][2];   // Q^T B fragments of query row 8 n + lane / 4
  float acc[MTILES][NT][4];     // O^T: (dim 16c + g, rows 8n + 2t, + 1), (dim 16c + 8 + g, ...)
  float m[NT][2], l[NT][2], mt[NT][2];

  __device__ __forceinline__ void init(const uint16_t* q_group, int group, int lane) {
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int row = 8 * n + g;
      const uint32_t* q = reinterpret_cast<const uint32_t*>(q_group + row * D);
#pragma unroll
      for (int kk = 0; kk < KSTEPS; ++kk) {
        qb[kk][n][0] = row < group ? q[(kk * 16 + 2 * t) >> 1] : 0u;
        qb[kk][n][1] = row < group ? q[(kk * 16 + 8 + 2 * t) >> 1] : 0u;
      }
#pragma unroll
      for (int i = 0; i < MTILES; ++i)
        acc[i][n][0] = acc[i][n][1] = acc[i][n][2] = acc[i][n][3] = 0.f;
      m[n][0] = m[n][1] = mt[n][0] = mt[n][1] = -INFINITY;
      l[n][0] = l[n][1] = 0.f;
    }
  }

  // z: the logits of the page's first token, `group` a token.
  __device__ __forceinline__ void page(uint32_t kbase, uint32_t vbase, int lim, float scale_log2,
                                       int lane, float* z, int group) {
    const int g = lane >> 2, t = lane & 3;
    const int ktok = (lane & 7) + ((lane >> 3) & 1) * 8;
    const int kchk = lane >> 4;
    float s[NT][2][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) s[n][0][i] = s[n][1][i] = 0.f;
#pragma unroll
    for (int kk = 0; kk < KSTEPS; ++kk) {
      uint32_t a[4];
      ldsm_x4(page_chunk<D>(kbase, ktok, 2 * kk + kchk), a[0], a[1], a[2], a[3]);
#pragma unroll
      for (int n = 0; n < NT; ++n) mma_16816<BF16>(s[n][kk & 1], a, qb[kk][n][0], qb[kk][n][1]);
    }
    const bool lo_live = g < lim, hi_live = g + 8 < lim;
    const bool odd = g & 1;
    float x[NT][4];
    bool grow = false;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      x[n][0] = lo_live ? (s[n][0][0] + s[n][1][0]) * scale_log2 : -INFINITY;
      x[n][1] = lo_live ? (s[n][0][1] + s[n][1][1]) * scale_log2 : -INFINITY;
      x[n][2] = hi_live ? (s[n][0][2] + s[n][1][2]) * scale_log2 : -INFINITY;
      x[n][3] = hi_live ? (s[n][0][3] + s[n][1][3]) * scale_log2 : -INFINITY;
      const int row = 8 * n + 2 * t;
      if (row + 1 < group && !(group & 1)) {
        if (lo_live) *reinterpret_cast<float2*>(z + g * group + row) = make_float2(x[n][0], x[n][1]);
        if (hi_live)
          *reinterpret_cast<float2*>(z + (g + 8) * group + row) = make_float2(x[n][2], x[n][3]);
      } else {
        if (row < group) {
          if (lo_live) z[g * group + row] = x[n][0];
          if (hi_live) z[(g + 8) * group + row] = x[n][2];
        }
        if (row + 1 < group) {
          if (lo_live) z[g * group + row + 1] = x[n][1];
          if (hi_live) z[(g + 8) * group + row + 1] = x[n][3];
        }
      }
      // row maxima over the page: each lane reduces one of its two rows over
      // the 8 lanes of equal t, the other comes from the neighbour
      float keep = odd ? fmaxf(x[n][1], x[n][3]) : fmaxf(x[n][0], x[n][2]);
      const float send = odd ? fmaxf(x[n][0], x[n][2]) : fmaxf(x[n][1], x[n][3]);
      keep = fmaxf(keep, __shfl_xor_sync(0xffffffffu, send, 4));
      keep = fmaxf(keep, __shfl_xor_sync(0xffffffffu, keep, 8));
      keep = fmaxf(keep, __shfl_xor_sync(0xffffffffu, keep, 16));
      const float other = __shfl_xor_sync(0xffffffffu, keep, 4);
      mt[n][0] = fmaxf(mt[n][0], odd ? other : keep);
      mt[n][1] = fmaxf(mt[n][1], odd ? keep : other);
      grow |= (mt[n][0] > m[n][0] + kSlack) | (mt[n][1] > m[n][1] + kSlack);
    }
    if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          // (a row of logits that are all -inf so far keeps a reference of -inf)
          const float al = mt[n][h] > -INFINITY ? ex2(m[n][h] - mt[n][h]) : 1.f;
          m[n][h] = mt[n][h];
          l[n][h] *= al;
#pragma unroll
          for (int i = 0; i < MTILES; ++i) {
            acc[i][n][h] *= al;
            acc[i][n][2 + h] *= al;
          }
        }
      }
    }
    uint32_t pb[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const float r0 = (m[n][0] == -INFINITY ? 0.f : m[n][0]) - kLift;
      const float r1 = (m[n][1] == -INFINITY ? 0.f : m[n][1]) - kLift;
      const float p0 = ex2(x[n][0] - r0), p1 = ex2(x[n][1] - r1);
      const float p2 = ex2(x[n][2] - r0), p3 = ex2(x[n][3] - r1);
      const uint32_t h_lo = pack2<BF16>(p0, p1), h_hi = pack2<BF16>(p2, p3);
      pb[n][0] = movmatrix_trans(h_lo);
      pb[n][1] = movmatrix_trans(h_hi);
      if constexpr (BF16) {
        const float2 u = unpack2<true>(h_lo), w = unpack2<true>(h_hi);
        pb[n][2] = movmatrix_trans(pack2<true>(p0 - u.x, p1 - u.y));
        pb[n][3] = movmatrix_trans(pack2<true>(p2 - w.x, p3 - w.y));
      }
      // l sums the fp32 p: the weights are exp(z - lse) of the same p
      l[n][0] += p0 + p2;
      l[n][1] += p1 + p3;
    }
    const int vtok = (lane & 7) + (lane >> 4) * 8;
    const int vchk = (lane >> 3) & 1;
#pragma unroll
    for (int c = 0; c < MTILES; ++c) {
      uint32_t a[4];
      ldsm_x4_trans(page_chunk<D>(vbase, vtok, 2 * c + vchk), a[0], a[1], a[2], a[3]);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        mma_16816<BF16>(acc[c][n], a, pb[n][0], pb[n][1]);
        if constexpr (BF16) mma_16816<BF16>(acc[c][n], a, pb[n][2], pb[n][3]);
      }
    }
  }

  // Rows < group into the merge buffers, restated against the true max.
  __device__ __forceinline__ void publish(float* red_acc, float* red_m, float* red_l, int group,
                                          int lane) {
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float f = kDrop * (mt[n][h] > -INFINITY ? ex2(m[n][h] - mt[n][h]) : 1.f);
        float lh = l[n][h] * f;
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) lh += __shfl_xor_sync(0xffffffffu, lh, o);
        const int row = 8 * n + 2 * t + h;
        if (row < group) {
#pragma unroll
          for (int c = 0; c < MTILES; ++c) {
            red_acc[row * D + 16 * c + g] = acc[c][n][h] * f;
            red_acc[row * D + 16 * c + 8 + g] = acc[c][n][2 + h] * f;
          }
          if (g == 0) {
            red_m[row] = mt[n][h];
            red_l[row] = lh;
          }
        }
      }
    }
  }
};

template <int D, int NST, bool BF16, int NT>
__global__ void __launch_bounds__(kThreads)
    weights_split_kernel(const __grid_constant__ CUtensorMap kmap,
                         const __grid_constant__ CUtensorMap vmap, const WeightsArgs a) {
  using L = DecodeSmem<D, NST>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  prefetch_tensormap(&kmap);
  prefetch_tensormap(&vmap);
  pdl_launch_dependents();
  pdl_wait();

  int item = blockIdx.x;
  const int part = item % a.parts;
  item /= a.parts;
  const int kvh = item % a.num_kv_heads, s = item / a.num_kv_heads;
  const int cap = a.max_blocks_per_seq * kPage;
  int ctx = a.context_lens[s];
  if (ctx < 0 || ctx > cap) {
    if (threadIdx.x == 0 && part == 0 && kvh == 0) record_error(kErrContextLen, s);
    ctx = ctx < 0 ? 0 : cap;
  }
  const int t_begin = part * a.part, t_end = min(t_begin + a.part, ctx);
  if (t_begin >= t_end) return;
  const int group = a.group;
  const int first_page = t_begin / kPage;
  const int n_pages = (t_end - t_begin + kPage - 1) / kPage;   // <= 32: one id a lane
  const int my_pages = n_pages > warp ? (n_pages - warp + kWarps - 1) / kWarps : 0;
  const uint32_t stage0 = smem_addr(smem) + warp * NST * L::kStageBytes;
  const uint32_t bar0 = smem_addr(smem + L::kBarOffset) + warp * NST * 8;
  init_ring<NST>(bar0, lane);

  static_assert(kWeightsPart / kPage <= 32, "the pages of a partition: one id a lane");
  int id = -1;
  if (lane < n_pages) {
    const size_t at = static_cast<size_t>(s) * a.max_blocks_per_seq + first_page + lane;
    id = a.block_tables[at];
    if (id < 0 || id >= a.num_blocks) {
      if (warp == 0) record_error(kErrBlockId, static_cast<long long>(at));
      id = -1;   // a box at a negative row reads zeros
    }
  }
  const uint64_t once = evict_first_policy();
  auto issue = [&](int k) {   // whole warp; lane 0 loads this warp's page k
    const int row = __shfl_sync(0xffffffffu, id, warp + k * kWarps) * kPage;
    if (lane == 0) {
      const uint32_t bar = bar0 + (k % NST) * 8;
      const uint32_t dk = stage0 + (k % NST) * L::kStageBytes, dv = dk + L::kPageBytes;
      mbar_arrive_expect_tx(bar, L::kStageBytes);
#pragma unroll
      for (int b = 0; b < L::kBoxesPerRow; ++b)
        tma_load_4d_once(dk + b * kBoxBytes, &kmap, bar, 0, b, kvh, row, once);
#pragma unroll
      for (int b = 0; b < L::kBoxesPerRow; ++b)
        tma_load_4d_once(dv + b * kBoxBytes, &vmap, bar, 0, b, kvh, row, once);
    }
  };
  for (int k = 0; k < min(my_pages, NST); ++k) issue(k);

  WeightsWarp<D, BF16, NT> st;
  st.init(a.query + (static_cast<size_t>(s) * a.num_heads + static_cast<size_t>(kvh) * group) * D,
          group, lane);
  float* z = a.logits + (static_cast<size_t>(s) * a.num_kv_heads + kvh) * cap * group;
  bool ok = true;
  int k_stop = my_pages;
  for (int k = 0; k < my_pages; ++k) {
    if (!__all_sync(~0u, mbar_wait_bounded(bar0 + (k % NST) * 8, (k / NST) & 1))) {
      if (lane == 0) record_error(kErrWaitTimeout, blockIdx.x);
      ok = false;
      k_stop = k;
      break;
    }
    const uint32_t kb = stage0 + (k % NST) * L::kStageBytes;
    const int tok0 = t_begin + (warp + k * kWarps) * kPage;
    if (tok0 + kPage > ctx) zero_page_tail<L::kBoxesPerRow>(kb + L::kPageBytes, ctx - tok0, lane);
    st.page(kb, kb + L::kPageBytes, t_end - tok0, a.scale_log2, lane,
            z + static_cast<size_t>(tok0) * group, group);
    __syncwarp();
    if (k + NST < my_pages) issue(k + NST);
  }
  // (a warp that gave up first waits for the loads it still has in flight)
  if (!__syncthreads_and(drain_stages<NST>(ok, k_stop, my_pages, bar0))) return;
  float* red_acc = reinterpret_cast<float*>(smem);
  float* red_m = reinterpret_cast<float*>(smem + L::kRedMOffset);
  float* red_l = reinterpret_cast<float*>(smem + L::kRedLOffset);
  if (ok) {
    st.publish(red_acc + warp * group * D, red_m + warp * 16, red_l + warp * 16, group, lane);
  } else {
    for (int g = lane; g < group; g += 32) {
      red_m[warp * 16 + g] = -INFINITY;
      red_l[warp * 16 + g] = 0.f;
    }
  }
  __syncthreads();
  const size_t hrow0 = static_cast<size_t>(s) * a.num_heads + static_cast<size_t>(kvh) * group;
  merge_and_emit<D, NST>(smem, group, false, 1, 0,
                         [&](int g, int d, float o0, float o1, float big_m, float big_l) {
    const size_t p = (hrow0 + g) * a.parts + part;
    *reinterpret_cast<float2*>(a.tmp_out + p * D + d) = make_float2(o0, o1);
    if (d == 0) {
      a.part_m[p] = big_m;
      a.part_l[p] = big_l;
    }
  });
}

// weights[t] += sum_g 2^(z_tg - lse_g) for tokens t0 <= t < t1 (set from `fresh`
// on), by the kThreadsN threads of a CTA, kWeightsBatch tokens a thread at a time.
// Four heads a load: Q lanes share a token, so that a warp's loads are one piece.
// One such step from token b0; kWhole: all its tokens are before t1 and not new.
template <int kThreadsN, int Q, bool kWhole>
__device__ __forceinline__ void add_step_by_four(const float* z, float* w, int b0, int t1,
                                                 int fresh, int G, const float* lse_sh, int tid) {
  constexpr int kTokens = kThreadsN / Q;
  const int sub = tid % Q, first = b0 + tid / Q;
  float sum[kWeightsBatch], old[kWeightsBatch];
#pragma unroll
  for (int u = 0; u < kWeightsBatch; ++u) {
    const int t = first + u * kTokens;
    sum[u] = 0.f;
    old[u] = sub == 0 && (kWhole || (t < t1 && t < fresh)) ? w[t] : 0.f;
  }
  const float* zt = z + static_cast<size_t>(first) * G;
  for (int g = 4 * sub; g < G; g += 4 * Q) {
    const float4 l = *reinterpret_cast<const float4*>(lse_sh + g);
    float4 v[kWeightsBatch];
#pragma unroll
    for (int u = 0; u < kWeightsBatch; ++u)
      v[u] = kWhole || first + u * kTokens < t1
                 ? *reinterpret_cast<const float4*>(zt + u * kTokens * G + g)
                 : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
#pragma unroll
    for (int u = 0; u < kWeightsBatch; ++u)
      sum[u] += (ex2(v[u].x - l.x) + ex2(v[u].y - l.y)) +
                (ex2(v[u].z - l.z) + ex2(v[u].w - l.w));
  }
#pragma unroll
  for (int u = 0; u < kWeightsBatch; ++u) {
#pragma unroll
    for (int o = 1; o < Q; o <<= 1) sum[u] += __shfl_xor_sync(0xffffffffu, sum[u], o);
    const int t = first + u * kTokens;
    if (sub == 0 && (kWhole || t < t1)) w[t] = old[u] + sum[u];
  }
}

template <int kThreadsN, int Q>
__device__ __forceinline__ void add_weights_by_four(const float* z, float* w, int t0, int t1,
                                                    int fresh, int G, const float* lse_sh,
                                                    int tid) {
  constexpr int kStep = kThreadsN / Q * kWeightsBatch;
  int b0 = t0;
  for (; b0 + kStep <= min(t1, fresh); b0 += kStep)
    add_step_by_four<kThreadsN, Q, true>(z, w, b0, t1, fresh, G, lse_sh, tid);
  for (; b0 < t1; b0 += kStep)
    add_step_by_four<kThreadsN, Q, false>(z, w, b0, t1, fresh, G, lse_sh, tid);
}

template <int kThreadsN>
__device__ __forceinline__ void add_weights(const float* z, float* w, int t0, int t1, int fresh,
                                            int G, const float* lse_sh, int tid) {
  if (G == 16) return add_weights_by_four<kThreadsN, 4>(z, w, t0, t1, fresh, G, lse_sh, tid);
  if (G == 8) return add_weights_by_four<kThreadsN, 2>(z, w, t0, t1, fresh, G, lse_sh, tid);
  if ((G & 3) == 0) return add_weights_by_four<kThreadsN, 1>(z, w, t0, t1, fresh, G, lse_sh, tid);
  constexpr int kStep = kThreadsN * kWeightsBatch;
  for (int b0 = t0; b0 < t1; b0 += kStep) {
    float sum[kWeightsBatch] = {};
    for (int g = 0; g < G; ++g) {
      float v[kWeightsBatch];
#pragma unroll
      for (int u = 0; u < kWeightsBatch; ++u) {
        const int t = b0 + u * kThreadsN + tid;
        v[u] = t < t1 ? z[static_cast<size_t>(t) * G + g] : -INFINITY;
      }
#pragma unroll
      for (int u = 0; u < kWeightsBatch; ++u) sum[u] += ex2(v[u] - lse_sh[g]);
    }
#pragma unroll
    for (int u = 0; u < kWeightsBatch; ++u) {
      const int t = b0 + u * kThreadsN + tid;
      if (t < t1) w[t] = t < fresh ? w[t] + sum[u] : sum[u];
    }
  }
}

// ---------------------------------------------------------------------------
// One CTA a (sequence, KV head), the whole context: the heads' lse is known at
// the end of its own page loop, so the CTA turns its logits into weights itself
// and writes the outputs, with no partials and no second launch.
// Sequences are taken longest first (up to kLptMaxSeqs of them).
// ---------------------------------------------------------------------------
template <int D, int NST, bool BF16, int NT>
__global__ void __launch_bounds__(kThreads)
    weights_single_kernel(const __grid_constant__ CUtensorMap kmap,
                          const __grid_constant__ CUtensorMap vmap, const WeightsArgs a) {
  using L = DecodeSmem<D, NST>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(16) float lse_sh[16];
  __shared__ int chosen;
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  prefetch_tensormap(&kmap);
  prefetch_tensormap(&vmap);
  pdl_launch_dependents();
  pdl_wait();

  const int cap = a.max_blocks_per_seq * kPage;
  const int kvh = blockIdx.x % a.num_kv_heads;
  int s = blockIdx.x / a.num_kv_heads;
  if (a.num_seqs > 1 && a.num_seqs <= kLptMaxSeqs) {
    // the s-th longest sequence, ties by index: ranks counted on one 32-bit key
    // each, (length << 8 | 255 - index), four at a time
    unsigned* keys = reinterpret_cast<unsigned*>(smem);   // stage area, not in use yet
    const int n4 = (a.num_seqs + 3) / 4;
    for (int i = tid; i < 4 * n4; i += kThreads) {
      const int c = i < a.num_seqs ? min(max(a.context_lens[i], 0), (1 << 24) - 1) : 0;
      keys[i] = i < a.num_seqs ? static_cast<unsigned>(c) << 8 | (255 - i) : 0u;
    }
    __syncthreads();
    for (int i = tid; i < a.num_seqs; i += kThreads) {
      const unsigned key = keys[i];
      int rank = 0;
      for (int j = 0; j < n4; ++j) {
        const uint4 v = reinterpret_cast<const uint4*>(keys)[j];
        rank += (v.x > key) + (v.y > key) + (v.z > key) + (v.w > key);
      }
      if (rank == s) chosen = i;
    }
    __syncthreads();
    s = chosen;
    fence_proxy_async_smem();   // before TMA writes to the stage area
    __syncthreads();
  }
  int ctx = a.context_lens[s];
  if (ctx < 0 || ctx > cap) {
    if (tid == 0 && kvh == 0) record_error(kErrContextLen, s);
    ctx = ctx < 0 ? 0 : cap;
  }
  const int group = a.group;
  const size_t hrow0 = static_cast<size_t>(s) * a.num_heads + static_cast<size_t>(kvh) * group;
  if (ctx == 0) {
    for (int i = tid; i < group * D; i += kThreads) a.out[hrow0 * D + i] = 0;
    return;
  }
  const int n_pages = (ctx + kPage - 1) / kPage;
  const int my_pages = n_pages > warp ? (n_pages - warp + kWarps - 1) / kWarps : 0;
  const uint32_t stage0 = smem_addr(smem) + warp * NST * L::kStageBytes;
  const uint32_t bar0 = smem_addr(smem + L::kBarOffset) + warp * NST * 8;
  init_ring<NST>(bar0, lane);

  // block ids 32 at a time, one a lane, the next 32 on their way
  const size_t row_base = static_cast<size_t>(s) * a.max_blocks_per_seq;
  auto load_ids = [&](int win) -> int {
    const int k = win * 32 + lane;
    if (k >= my_pages) return -1;
    const size_t at = row_base + warp + static_cast<size_t>(k) * kWarps;
    const int id = a.block_tables[at];
    if (id >= 0 && id < a.num_blocks) return id;
    record_error(kErrBlockId, static_cast<long long>(at));
    return -1;   // a box at a negative row reads zeros
  };
  int win = 0, ids = load_ids(0), ids_next = my_pages > 32 ? load_ids(1) : -1;
  const uint64_t once = evict_first_policy();
  auto issue = [&](int k) {   // whole warp; lane 0 loads this warp's page k
    const int row = __shfl_sync(0xffffffffu, (k >> 5) == win ? ids : ids_next, k & 31) * kPage;
    if (lane == 0) {
      const uint32_t bar = bar0 + (k % NST) * 8;
      const uint32_t dk = stage0 + (k % NST) * L::kStageBytes, dv = dk + L::kPageBytes;
      mbar_arrive_expect_tx(bar, L::kStageBytes);
#pragma unroll
      for (int b = 0; b < L::kBoxesPerRow; ++b)
        tma_load_4d_once(dk + b * kBoxBytes, &kmap, bar, 0, b, kvh, row, once);
#pragma unroll
      for (int b = 0; b < L::kBoxesPerRow; ++b)
        tma_load_4d_once(dv + b * kBoxBytes, &vmap, bar, 0, b, kvh, row, once);
    }
  };
  for (int k = 0; k < min(my_pages, NST); ++k) issue(k);

  WeightsWarp<D, BF16, NT> st;
  st.init(a.query + hrow0 * D, group, lane);
  float* z = a.logits + (static_cast<size_t>(s) * a.num_kv_heads + kvh) * cap * group;
  bool ok = true;
  int k_stop = my_pages;
  for (int k = 0; k < my_pages; ++k) {
    if (k > 0 && (k & 31) == 0) {
      ++win;
      ids = ids_next;
      ids_next = my_pages > (win + 1) * 32 ? load_ids(win + 1) : -1;
    }
    if (!__all_sync(~0u, mbar_wait_bounded(bar0 + (k % NST) * 8, (k / NST) & 1))) {
      if (lane == 0) record_error(kErrWaitTimeout, blockIdx.x);
      ok = false;
      k_stop = k;
      break;
    }
    const uint32_t kb = stage0 + (k % NST) * L::kStageBytes;
    const int tok0 = (warp + k * kWarps) * kPage;
    if (tok0 + kPage > ctx) zero_page_tail<L::kBoxesPerRow>(kb + L::kPageBytes, ctx - tok0, lane);
    st.page(kb, kb + L::kPageBytes, ctx - tok0, a.scale_log2, lane,
            z + static_cast<size_t>(tok0) * group, group);
    __syncwarp();
    if (k + NST < my_pages) issue(k + NST);
  }
  // (a warp that gave up first waits for the loads it still has in flight; then
  // the CTA ends without a result)
  if (!__syncthreads_and(drain_stages<NST>(ok, k_stop, my_pages, bar0) && ok)) return;
  st.publish(reinterpret_cast<float*>(smem) + warp * group * D,
             reinterpret_cast<float*>(smem + L::kRedMOffset) + warp * 16,
             reinterpret_cast<float*>(smem + L::kRedLOffset) + warp * 16, group, lane);
  __syncthreads();
  merge_and_emit<D, NST>(smem, group, false, 1, 0,
                         [&](int g, int d, float o0, float o1, float big_m, float big_l) {
    const float inv = big_l > 0.f ? 1.f / big_l : (big_l == 0.f ? 0.f : big_l);
    *reinterpret_cast<uint32_t*>(a.out + (hrow0 + g) * D + d) = pack2<BF16>(o0 * inv, o1 * inv);
    if (d == 0) lse_sh[g] = big_l == 0.f ? INFINITY : big_m + __log2f(big_l);
  });
  __syncthreads();   // the lse, and every warp's logits
  if (ctx > a.max_tokens) {
    if (tid == 0 && kvh == 0) record_error(kErrContextLen, s);
    return;
  }
  add_weights<kThreads>(z, a.weights + (static_cast<size_t>(s) * a.num_kv_heads + kvh) *
                                           a.max_tokens,
                        0, ctx, max(ctx - a.new_tokens, 0), group, lse_sh, tid);
}

// lse (log2 units) of one head from its partitions, whole warp; +inf when no
// token has a finite logit, so that every weight comes out 0.
__device__ __forceinline__ float warp_lse(const float* m, const float* l, int np, int lane) {
  float big = -INFINITY;
  for (int p = lane; p < np; p += 32) big = fmaxf(big, m[p]);
#pragma unroll
  for (int o = 16; o; o >>= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, o));
  const float ref = big == -INFINITY ? 0.f : big;
  float sum = 0.f;
  for (int p = lane; p < np; p += 32) sum += ex2(m[p] - ref) * l[p];
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  return sum == 0.f ? INFINITY : ref + __log2f(sum);
}

template <int D, bool BF16>
__global__ void __launch_bounds__(kWeightsThreads)
    weights_merge_kernel(const WeightsArgs a) {
  constexpr int kWarpsM = kWeightsThreads / 32;
  __shared__ float part_sh[kWarpsM][D / 32][32];
  __shared__ __align__(16) float lse_sh[16];
  pdl_launch_dependents();
  pdl_wait();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cap = a.max_blocks_per_seq * kPage;
  const int run = blockIdx.x % a.runs, row = blockIdx.x / a.runs;   // row = s * Hk + kv
  const int s = row / a.num_kv_heads, kv = row % a.num_kv_heads;
  const int ctx = min(max(a.context_lens[s], 0), cap);
  const int t0 = run * a.run, t1 = min(t0 + a.run, ctx);
  if (t0 >= t1 && run > 0) return;
  const int np = (ctx + a.part - 1) / a.part;
  const int G = a.group;
  const size_t hrow = static_cast<size_t>(s) * a.num_heads + kv * G;
  for (int g = warp; g < G; g += kWarpsM) {
    const size_t base = (hrow + g) * a.parts;
    const float lse = warp_lse(a.part_m + base, a.part_l + base, np, lane);
    if (lane == 0) lse_sh[g] = lse;
  }
  __syncthreads();

  // ---- the weights of the run ----
  if (ctx > a.max_tokens) {
    if (tid == 0 && run == 0 && kv == 0) record_error(kErrContextLen, s);
  } else {
    const float* z = a.logits + static_cast<size_t>(row) * cap * G;
    float* w = a.weights + static_cast<size_t>(row) * a.max_tokens;
    const int fresh = max(ctx - a.new_tokens, 0);      // tokens from here on start anew
    add_weights<kWeightsThreads>(z, w, t0, t1, fresh, G, lse_sh, tid);
  }

  // ---- this run's share of the heads' outputs, a row a warp or several ----
  const int live_runs = max(1, (ctx + a.run - 1) / a.run);
  const int per = (G + live_runs - 1) / live_runs;
  const int g0 = min(run * per, G), g1 = min(g0 + per, G);
  // a row's partitions over `share` warps, so that few rows keep all warps busy
  const int share = np < 2 || g1 - g0 >= kWarpsM ? 1 : g1 - g0 >= 4 ? 2 : g1 - g0 >= 2 ? 4 : 8;
  constexpr int kVec = D / 32;                         // columns of a lane
  for (int gb = g0; gb < g1; gb += kWarpsM / share) {
    const int g = gb + warp / share, first = warp % share;
    float acc[kVec] = {};
    if (g < g1) {
      const size_t base = (hrow + g) * a.parts;
      const float lse = lse_sh[g];
      for (int p0 = first; p0 < np; p0 += share * kWeightsBatch) {
        float v[kWeightsBatch][kVec], m[kWeightsBatch];
#pragma unroll
        for (int i = 0; i < kWeightsBatch; ++i) {
          const int p = p0 + i * share;
          m[i] = -INFINITY;
          if (p < np) {
            m[i] = a.part_m[base + p];
            const float* src = a.tmp_out + (base + p) * D + lane * kVec;
            if constexpr (kVec == 4) {
              const float4 x = *reinterpret_cast<const float4*>(src);
              v[i][0] = x.x; v[i][1] = x.y; v[i][2] = x.z; v[i][3] = x.w;
            } else {
              const float2 x = *reinterpret_cast<const float2*>(src);
              v[i][0] = x.x; v[i][1] = x.y;
            }
          } else {
#pragma unroll
            for (int c = 0; c < kVec; ++c) v[i][c] = 0.f;
          }
        }
#pragma unroll
        for (int i = 0; i < kWeightsBatch; ++i) {
          const float e = ex2(m[i] - lse);
#pragma unroll
          for (int c = 0; c < kVec; ++c) acc[c] += e * v[i][c];
        }
      }
    }
    if (share > 1) {
      __syncthreads();
#pragma unroll
      for (int c = 0; c < kVec; ++c) part_sh[warp][c][lane] = acc[c];
      __syncthreads();
      for (int i = 1; i < share && first == 0; ++i)
#pragma unroll
        for (int c = 0; c < kVec; ++c) acc[c] += part_sh[warp + i][c][lane];
    }
    if (g < g1 && first == 0) {
      uint32_t* o = reinterpret_cast<uint32_t*>(a.out + (hrow + g) * D + lane * kVec);
#pragma unroll
      for (int c = 0; c < kVec; c += 2) o[c / 2] = pack2<BF16>(acc[c], acc[c + 1]);
    }
  }
}

}  // namespace pa
