// pa_evict.cuh -- eviction from a paged cache by accumulated attention weight:
// which tokens of every (sequence, KV head) stay (evict_select_kernel) and the
// move that packs them into the first slots of the sequence's blocks
// (evict_compact_kernel).
//
// Attention is a sum over the cached tokens, in any order, so the kept tokens
// need not keep their order.  A kept token whose slot is already below the new
// length stays where it is, and the r-th freed slot below it (a hole) takes
// the r-th kept token from above it.  That moves the fewest rows (in a steady
// state as many as were added since the last eviction, not the whole cache),
// and no row moved is overwritten and no slot written is read, so the moves
// need no order among themselves and repeating them changes nothing.
#pragma once

#include "pa_device.cuh"

namespace pa {

constexpr unsigned kErrSource = 9;

struct EvictArgs {
  int32_t* source;               // [S, Hk, budget]
  int32_t* new_lens;             // [S]
  float* weights;                // [S, Hk, max_tokens]
  int32_t* positions;            // [S, Hk, max_tokens]
  const int32_t* context_lens;   // [S]
  const int32_t* recorded_lens;  // [S]
  const int32_t* seq_lens;       // [S]
  int num_kv_heads;
  int max_tokens;
  int budget;
  int sink;
  int recent;
};

// Position in its sequence of slot i: recorded, or counted back from the
// sequence's length (slots filled in order since the last eviction).
__device__ __forceinline__ long long slot_position(const int32_t* positions, int recorded, int len,
                                                   int ctx, int i) {
  return i < recorded ? positions[i] : static_cast<long long>(len) - ctx + i;
}

// ---------------------------------------------------------------------------
// Select.  Every slot gets a 32-bit key that orders as its claim does: the
// weight's bits made monotone (-0 as +0, NaN below every number), all ones for
// a sink or a recent token.  The budget-th largest key T comes from a radix
// select over 11, 11 and 10 bits; kept are the keys above T and, of those
// equal to it, the lowest slots that fill the budget.
//
// One cluster of C CTAs takes a (sequence, KV head), each CTA a run of its
// slots, whose keys stay in shared memory between the digit passes (a run too
// long for it is read again from global memory).  The CTAs add up their
// histograms through distributed shared memory, and every one finds the same
// digit.  The kept flags then become one bit each, a warp's share of the run
// is counted by popcounts, and an exclusive scan over warps and CTAs gives
// every hole and every kept token behind the new length its rank.  The latter
// leave their slot numbers at their rank in a list spread over the cluster's
// shared memory (over the keys, which are done with), where the holes fetch
// theirs.
// ---------------------------------------------------------------------------
constexpr int kSelectThreads = 1024;
constexpr int kSelectWarps = kSelectThreads / 32;
constexpr int kDigitBits = 11;
constexpr int kBins = 1 << kDigitBits;

struct SelectSmem {
  // [bins] [bins summed over the cluster] [scan sums] [3 counts a warp] [totals] [flags] [keys]
  static constexpr int kHist = 0;
  static constexpr int kSum = kHist + kBins * 4;
  static constexpr int kScan = kSum + kBins * 4;
  static constexpr int kWarpCount = kScan + 2 * kSelectWarps * 4;
  static constexpr int kTotals = kWarpCount + 3 * kSelectWarps * 4;
  static constexpr int kPick = kTotals + 4 * 4;
  static constexpr int kFlags = kPick + 4 * 4;   // then flag words, then keys (or the list)
};

__device__ __forceinline__ uint32_t claim_key(float w) {
  if (w != w) return 0u;
  const uint32_t b = __float_as_uint(w + 0.f);    // -0 + 0 = +0
  return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ void st_cluster_u32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

// Bytes of shared memory for a run of `run` slots: flag words, and keys when
// `cached`, else room for this CTA's share of the list of moved slots.
__host__ __device__ constexpr int select_smem(int run, bool cached, int list) {
  return SelectSmem::kFlags + (run + 31) / 32 * 4 + 4 * (cached && run > list ? run : list);
}

__global__ void __launch_bounds__(kSelectThreads, 1)
    evict_select_kernel(const EvictArgs a, int max_run, int cached) {
  extern __shared__ __align__(16) uint8_t smem[];
  uint32_t* hist = reinterpret_cast<uint32_t*>(smem + SelectSmem::kHist);
  uint32_t* sum = reinterpret_cast<uint32_t*>(smem + SelectSmem::kSum);
  uint32_t* scan = reinterpret_cast<uint32_t*>(smem + SelectSmem::kScan);
  uint32_t* wcount = reinterpret_cast<uint32_t*>(smem + SelectSmem::kWarpCount);
  uint32_t* totals = reinterpret_cast<uint32_t*>(smem + SelectSmem::kTotals);
  uint32_t* pick = reinterpret_cast<uint32_t*>(smem + SelectSmem::kPick);
  uint32_t* flags = reinterpret_cast<uint32_t*>(smem + SelectSmem::kFlags);
  uint32_t* keys = flags + (max_run + 31) / 32;
  const int C = static_cast<int>(cluster_nctarank()), rank = static_cast<int>(cluster_ctarank());
  const int row = blockIdx.x / C;                      // s * Hk + kv
  const int s = row / a.num_kv_heads;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_launch_dependents();
  pdl_wait();

  int n = a.context_lens[s];
  const bool bad = n < 0 || n > a.max_tokens;
  if (bad) {
    if (tid == 0 && rank == 0 && row % a.num_kv_heads == 0) record_error(kErrContextLen, s);
    n = 0;
  }
  const int B = a.budget;
  const int kept = n < B ? n : B;
  if (tid == 0 && rank == 0 && row % a.num_kv_heads == 0) a.new_lens[s] = kept;
  int32_t* source = a.source + static_cast<size_t>(row) * B;
  if (n <= B) {                                        // everything stays
    for (int i = rank * kSelectThreads + tid; i < B; i += C * kSelectThreads)
      source[i] = i < n ? i : -1;
    return;
  }

  // ---- this CTA's run of slots, a multiple of 32 ----
  const int per = ((n + C - 1) / C + 31) & ~31;        // <= max_run
  const int lo = min(rank * per, n), run = min(per, n - lo);
  const size_t base = static_cast<size_t>(row) * a.max_tokens;
  const float* w = a.weights + base;
  const int32_t* pos = a.positions + base;
  const int recorded = min(max(a.recorded_lens[s], 0), n);
  const int len = a.seq_lens[s];
  const long long first_recent = static_cast<long long>(len) - a.recent;
  auto make_key = [&](int i) -> uint32_t {             // slot lo + i
    const long long p = slot_position(pos, recorded, len, n, lo + i);
    return (p < a.sink || p >= first_recent) ? 0xffffffffu : claim_key(w[lo + i]);
  };
  auto key_at = [&](int i) -> uint32_t { return cached ? keys[i] : make_key(i); };

  uint32_t prefix = 0;                                 // digits of T found so far
  uint32_t need = B;                                   // kept keys among those that share them
  uint32_t equal = 0;                                  // keys that share them
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
    const int bits = pass == 2 ? 10 : 11;
    for (int b = tid; b < kBins; b += kSelectThreads) hist[b] = 0;
    __syncthreads();
    for (int i = tid; i < run; i += kSelectThreads) {
      uint32_t k;
      if (pass == 0) {
        k = make_key(i);
        if (cached) keys[i] = k;
      } else {
        k = key_at(i);
        if ((k >> (shift + bits)) != prefix) continue;
      }
      atomicAdd(&hist[(k >> shift) & ((1u << bits) - 1)], 1u);
    }
    __syncthreads();
    if (C > 1) {
      cluster_sync();
      for (int b = tid; b < kBins; b += kSelectThreads) {
        uint32_t t = 0;
        for (int c = 0; c < C; ++c) t += ld_cluster_u32(map_cluster(smem_addr(&hist[b]), c));
        sum[b] = t;
      }
      cluster_sync();                                  // hist is cleared for the next digit
    } else {
      for (int b = tid; b < kBins; b += kSelectThreads) sum[b] = hist[b];
      __syncthreads();
    }
    // thread t: bins kBins - 1 - 2t and kBins - 2 - 2t, from the top
    const uint32_t c0 = sum[kBins - 1 - 2 * tid], c1 = sum[kBins - 2 - 2 * tid];
    uint32_t incl = c0 + c1;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const uint32_t v = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl += v;
    }
    if (lane == 31) scan[warp] = incl;
    __syncthreads();
    if (warp == 0) {
      uint32_t x = scan[lane];
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const uint32_t v = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d) x += v;
      }
      scan[kSelectWarps + lane] = x;
    }
    __syncthreads();
    const uint32_t above = (warp ? scan[kSelectWarps + warp - 1] : 0) + incl - c0 - c1;
    if (above < need && above + c0 >= need) {
      pick[0] = kBins - 1 - 2 * tid;
      pick[1] = need - above;
      pick[2] = c0;
    } else if (above + c0 < need && above + c0 + c1 >= need) {
      pick[0] = kBins - 2 - 2 * tid;
      pick[1] = need - above - c0;
      pick[2] = c1;
    }
    __syncthreads();
    prefix = (prefix << bits) | pick[0];
    need = pick[1];
    equal = pick[2];
    __syncthreads();
  }
  const uint32_t T = prefix;
  const bool cut = equal != need;                      // only some keys equal to T stay

  // ---- flags, a warp's share of the run at a time; words of 32 slots ----
  const int words = (run + 31) / 32, wper = (words + kSelectWarps - 1) / kSelectWarps;
  const int w0 = min(warp * wper, words), w1 = min(w0 + wper, words);
  const uint32_t below = (1u << lane) - 1;
  // exclusive scan of one count a warp over the cluster's warps, in order of
  // the slots; every CTA calls it (it holds cluster barriers)
  auto before = [&](uint32_t mine, int slot) -> uint32_t {
    if (lane == 0) wcount[slot * kSelectWarps + warp] = mine;
    __syncthreads();
    uint32_t v = wcount[slot * kSelectWarps + lane];
    const uint32_t own = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const uint32_t u = __shfl_up_sync(0xffffffffu, v, d);
      if (lane >= d) v += u;
    }
    const uint32_t total = __shfl_sync(0xffffffffu, v, 31);
    const uint32_t first = __shfl_sync(0xffffffffu, v - own, warp);
    if (C == 1) return first;
    if (tid == 0) totals[slot] = total;
    cluster_sync();
    uint32_t ahead = 0;
    for (int c = 0; c < rank; ++c) ahead += ld_cluster_u32(map_cluster(smem_addr(&totals[slot]), c));
    return ahead + first;
  };
  uint32_t ties = 0;
  if (cut) {
    uint32_t mine = 0;
    for (int q = w0; q < w1; ++q) {
      const int i = q * 32 + lane;
      mine += __popc(__ballot_sync(0xffffffffu, i < run && key_at(i) == T));
    }
    ties = before(mine, 0);
  }
  const int front = min(max(kept - lo, 0), run);       // slots of the run below the new length
  uint32_t holes = 0, tails = 0;
  for (int q = w0; q < w1; ++q) {
    const int i = q * 32 + lane;
    const uint32_t k = i < run ? key_at(i) : 0u;
    bool keep = i < run && k >= T;
    if (cut) {
      const uint32_t eq = __ballot_sync(0xffffffffu, i < run && k == T);
      if (keep && k == T) keep = ties + __popc(eq & below) < need;
      ties += __popc(eq);
    }
    const uint32_t f = __ballot_sync(0xffffffffu, keep);
    if (lane == 0) flags[q] = f;
    const uint32_t in = __ballot_sync(0xffffffffu, i < front);
    holes += __popc(in & ~f);
    tails += __popc(f & ~in);
  }
  holes = before(holes, 1);
  tails = before(tails, 2);                            // (its barrier: every key is done with)

  // ---- the list of moved slots, entry r in CTA r / lper ----
  const int lper = (min(B, n - B) + C - 1) / C;
  for (int q = w0; q < w1; ++q) {
    const int i = q * 32 + lane;
    const uint32_t f = flags[q];
    const uint32_t t = f & __ballot_sync(0xffffffffu, i >= front);
    if ((t >> lane) & 1u) {
      const int r = tails + __popc(t & below);
      st_cluster_u32(map_cluster(smem_addr(&keys[r % lper]), r / lper), lo + i);
    }
    tails += __popc(t);
  }
  cluster_sync();
  for (int q = w0; q < w1 && q * 32 < front; ++q) {
    const int i = q * 32 + lane;
    const uint32_t f = flags[q];
    const uint32_t h = ~f & __ballot_sync(0xffffffffu, i < front);
    int from = lo + i;
    if ((h >> lane) & 1u) {
      const int r = holes + __popc(h & below);
      from = ld_cluster_u32(map_cluster(smem_addr(&keys[r % lper]), r / lper));
    }
    holes += __popc(h);
    if (i < front) source[lo + i] = from;
  }
  if (C > 1) cluster_sync();                           // no CTA leaves while its list is read
}

// ---------------------------------------------------------------------------
// Compact: slot i < new_lens[s] takes the row of slot source[i].  A CTA takes
// kCompactSlots slots of one (sequence, KV head): each thread looks at one and
// moves its weight and position, the slots to move go into a list, and the CTA
// copies their K and V rows in 16-byte units, consecutive threads along a row.
// ---------------------------------------------------------------------------
constexpr int kCompactThreads = 256;
constexpr int kCompactSlots = 256;

struct CompactArgs {
  EvictArgs e;
  uint8_t* key_cache;            // [num_blocks, block_size, Hk, row_bytes]
  uint8_t* value_cache;
  const int32_t* block_tables;   // [S, MB]
  int block_size;
  int num_blocks;
  int max_blocks_per_seq;
  int row_units;                 // 16-byte units of a K row
  int chunks;                    // CTAs per (sequence, KV head)
};

__global__ void __launch_bounds__(kCompactThreads)
    evict_compact_kernel(const CompactArgs a) {
  __shared__ int2 list[kCompactSlots];       // (source, destination) rows of the flat cache
  __shared__ int moves;
  const int tid = threadIdx.x;
  const int row = blockIdx.x / a.chunks, chunk = blockIdx.x - row * a.chunks;
  const int s = row / a.e.num_kv_heads, kv = row - s * a.e.num_kv_heads;
  if (tid == 0) moves = 0;
  pdl_launch_dependents();
  pdl_wait();
  __syncthreads();
  const int n = a.e.context_lens[s], kept = a.e.new_lens[s];
  if (n < 0 || n > a.e.max_tokens || kept < 0 || kept > n || kept > a.e.budget) {
    if (tid == 0 && chunk == 0 && kv == 0) record_error(kErrContextLen, s);
    return;
  }
  const int recorded = min(max(a.e.recorded_lens[s], 0), n);
  const int len = a.e.seq_lens[s];
  const size_t base = static_cast<size_t>(row) * a.e.max_tokens;
  const int32_t* table = a.block_tables + static_cast<size_t>(s) * a.max_blocks_per_seq;
  // flat row of a slot, or -1 (reported) if its block id is out of range
  auto flat = [&](int i) -> int {
    const int b = i / a.block_size;
    const int id = b < a.max_blocks_per_seq ? table[b] : -1;
    if (id < 0 || id >= a.num_blocks) {
      record_error(kErrBlockId, static_cast<long long>(s) * a.max_blocks_per_seq + b);
      return -1;
    }
    return id * a.block_size + i % a.block_size;
  };
  const int i = chunk * kCompactSlots + tid;
  if (i < kept) {
    const int j = a.e.source[static_cast<size_t>(row) * a.e.budget + i];
    if (j != i && (j < kept || j >= n)) {
      record_error(kErrSource, static_cast<long long>(row) * a.e.budget + i);
    } else {
      if (j != i || i >= recorded)
        a.e.positions[base + i] = static_cast<int32_t>(
            slot_position(a.e.positions + base, recorded, len, n, j));
      if (j != i) {
        a.e.weights[base + i] = a.e.weights[base + j];
        const int src = flat(j), dst = flat(i);
        if (src >= 0 && dst >= 0) list[atomicAdd(&moves, 1)] = make_int2(src, dst);
      }
    }
  }
  __syncthreads();
  const int units = moves * a.row_units;
  const size_t stride = static_cast<size_t>(a.e.num_kv_heads) * a.row_units;
  const uint4* ks = reinterpret_cast<const uint4*>(a.key_cache);
  const uint4* vs = reinterpret_cast<const uint4*>(a.value_cache);
  uint4* kd = reinterpret_cast<uint4*>(a.key_cache);
  uint4* vd = reinterpret_cast<uint4*>(a.value_cache);
  for (int u = tid; u < units; u += kCompactThreads) {
    const int m = u / a.row_units, c = u - m * a.row_units + kv * a.row_units;
    const int2 e = list[m];
    const uint4 k = ks[e.x * stride + c], v = vs[e.x * stride + c];
    kd[e.y * stride + c] = k;
    vd[e.y * stride + c] = v;
  }
}

}  // namespace pa
