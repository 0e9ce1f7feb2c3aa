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
// select; kept are the keys above T and, of those equal to it, the lowest slots
// that fill the budget.
//
// One cluster of C CTAs takes a (sequence, KV head), each CTA a run of its
// slots, each warp a share of the run in words of 32 slots.  A long run is gone
// through twice: once for the histogram of the top digit (of 11, 11 and 10 bits),
// and once, that digit known, to flag the keys above it (a bit a slot) and to list
// those that share it, few as a rule, from which the other two digits follow.  (A
// warp with more of them than its list holds goes through its words again
// instead.)  A short run's keys stay in registers, for four digits of 8 bits,
// whose histograms are quicker to clear and to scan.  The CTAs add up their
// histograms through distributed shared memory, and every one finds the same
// digit.  Then a thread takes whole words: an exclusive scan of popcounts over threads and CTAs gives
// every hole and every kept token behind the new length its rank.  The latter
// leave their slot numbers at their rank in a list spread over the cluster's
// shared memory, where the holes fetch theirs.
//
// What bounds it is instructions and the barriers between the steps, not bytes
// (4 a slot).  8 x 8 rows of 32768 to 131072 slots: 30 to 32 us; 105 us when every key
// was built again for each digit and ranked a slot at a time (315 instructions
// a word).  128 x 8 rows of 1017 slots: 9.2 us; 31 us with 512 threads and three
// digits of 11 bits, 12.1 us with each word's bounds looked at in every pass.  One
// row of 131072 slots, eight CTAs with their keys in registers: 16.4 us; streamed,
// 19 us, in cycles about a tenth each for the top digit and its exchange, a fifth
// for flags and lists, the rest shared between the other digits and the ranks and
// list.
// ---------------------------------------------------------------------------

// kHeld: words of keys a warp keeps in registers, or 0: it loads them again
template <int kThreadsN, int kHeld>
struct SelectSmem {
  static constexpr int kWarpsN = kThreadsN / 32;
  static constexpr int kListed = kHeld ? 0 : 256;  // keys of T's first digit a warp lists
  static constexpr int kDigit = kHeld ? 8 : 11;    // bits of a digit (the last: what is left)
  static constexpr int kDigits = (32 + kDigit - 1) / kDigit;
  static constexpr int kBins = 1 << kDigit;
  // [a histogram a digit] [candidates: key, slot] [4 sums a warp] [totals] [pick]
  // [flag words] [equal words] [list of moved slots]
  static constexpr int kHist = 0;
  static constexpr int kCand = kHist + kDigits * kBins * 4;
  static constexpr int kScan = kCand + kWarpsN * kListed * 8;
  static constexpr int kTotals = kScan + 4 * kWarpsN * 4;
  static constexpr int kPick = kTotals + 4 * 4;
  static constexpr int kFlags = kPick + kDigits * 16;
  // bytes for a run of `run` slots and `list` entries of the list
  static __host__ __device__ constexpr int bytes(int run, int list) {
    return kFlags + (run + 31) / 32 * 8 + 4 * list;
  }
};

__device__ __forceinline__ uint32_t claim_key(float w) {
  const uint32_t b = __float_as_uint(w + 0.f);    // -0 + 0 = +0
  const uint32_t k = b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
  return w != w ? 0u : k;
}

__device__ __forceinline__ void st_cluster_u32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void add_cluster_u32(uint32_t addr, uint32_t v) {
  asm volatile("red.relaxed.cluster.shared::cluster.add.u32 [%0], %1;" ::"r"(addr), "r"(v)
               : "memory");
}

// Loads of what the kernel before may have written while this one had started
// already (a read-only load must not be used on it), and this one does not write:
// the compiler may move them over other accesses, but not before the pointer, which
// after_wait() makes once the other kernel's writes are there.
template <class T>
__device__ __forceinline__ const T* after_wait(const T* p) {
  const T* q;
  asm volatile("mov.u64 %0, %1;" : "=l"(q) : "l"(p));
  return q;
}
__device__ __forceinline__ float ld_plain(const float* p) {
  float v;
  asm("ld.global.f32 %0, [%1];" : "=f"(v) : "l"(p));
  return v;
}
__device__ __forceinline__ int ld_plain(const int32_t* p) {
  int v;
  asm("ld.global.s32 %0, [%1];" : "=r"(v) : "l"(p));
  return v;
}

template <int kThreadsN, int kHeld>
__global__ void __launch_bounds__(kThreadsN, kHeld > 18 ? 1 : 1024 / kThreadsN)
    evict_select_kernel(const EvictArgs a, int max_run, int list_shift) {
  using L = SelectSmem<kThreadsN, kHeld>;
  constexpr bool kReg = kHeld > 0;
  constexpr int kWarpsN = L::kWarpsN, kBins = L::kBins;
  constexpr int kBatch = kReg && kHeld % 9 == 0 ? 9 : 8;   // words a warp loads before it uses any
  static_assert(kHeld % kBatch == 0 && kHeld <= 32, "whole batches, a flag word a lane");
  extern __shared__ __align__(16) uint8_t smem[];
  uint2* cand = reinterpret_cast<uint2*>(smem + L::kCand);
  uint32_t* scan = reinterpret_cast<uint32_t*>(smem + L::kScan);
  uint32_t* totals = reinterpret_cast<uint32_t*>(smem + L::kTotals);
  uint4* pick = reinterpret_cast<uint4*>(smem + L::kPick);
  uint32_t* flags = reinterpret_cast<uint32_t*>(smem + L::kFlags);
  uint32_t* same = flags + (max_run + 31) / 32;
  uint32_t* list = same + (max_run + 31) / 32;
  const int C = static_cast<int>(cluster_nctarank()), rank = static_cast<int>(cluster_ctarank());
  const int row = blockIdx.x / C;                      // s * Hk + kv
  const int s = row / a.num_kv_heads;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  for (int b = tid; b < L::kDigits * kBins / 4; b += kThreadsN)
    reinterpret_cast<uint4*>(smem + L::kHist)[b] = make_uint4(0, 0, 0, 0);
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
    for (int i = rank * kThreadsN + tid; i < B; i += C * kThreadsN) source[i] = i < n ? i : -1;
    return;
  }

  // ---- this CTA's run of slots, a multiple of 32, and this warp's words of it ----
  const int per = ((n + C - 1) / C + 31) & ~31;        // <= max_run
  const int lo = min(rank * per, n), run = min(per, n - lo);
  const int words = (run + 31) / 32, wper = (words + kWarpsN - 1) / kWarpsN;
  const int w0 = min(warp * wper, words), w1 = min(w0 + wper, words);
  const size_t base = static_cast<size_t>(row) * a.max_tokens + lo;
  const float* w = after_wait(a.weights + base);
  const int32_t* pos = after_wait(a.positions + base);
  const int recorded = min(max(a.recorded_lens[s], 0), n) - lo;   // relative to the run, too
  // recorded positions are held below `sink` and from `first_recent` on; the
  // slots after them, whose positions follow their order, below `held_lo` and
  // from `held_hi` on
  auto clamp = [](long long x, int hi) { return static_cast<int>(x < 0 ? 0 : x > hi ? hi : x); };
  const long long len = a.seq_lens[s];
  const int first_recent = static_cast<int>(len - a.recent < INT32_MIN ? INT32_MIN : len - a.recent);
  const long long late = len - n + lo;                 // position of slot i: late + i
  const int held_lo = clamp(a.sink - late, run), held_hi = clamp(len - a.recent - late, run);

  // Keys of kBatch words from q of the warp's share (0 past its end); true if
  // they are whole words of slots that have only their weight.
  auto load = [&](int q, uint32_t (&k)[kBatch]) -> bool {
    const int i0 = q * 32 + lane;
    float x[kBatch];
    if (q + kBatch <= w1 && q * 32 >= recorded && q * 32 >= held_lo &&
        (q + kBatch) * 32 <= held_hi) {
#pragma unroll
      for (int u = 0; u < kBatch; ++u) x[u] = ld_plain(w + i0 + 32 * u);
#pragma unroll
      for (int u = 0; u < kBatch; ++u) k[u] = claim_key(x[u]);
      return true;
    }
    int p[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int i = i0 + 32 * u;
      const bool in = q + u < w1 && i < run;
      x[u] = in ? ld_plain(w + i) : 0.f;
      p[u] = in && i < recorded ? ld_plain(pos + i) : 0;
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int i = i0 + 32 * u;
      const bool held = i < recorded ? p[u] < a.sink || p[u] >= first_recent
                                     : i < held_lo || i >= held_hi;
      k[u] = q + u < w1 && i < run ? (held ? 0xffffffffu : claim_key(x[u])) : 0u;
    }
    return false;
  };
  // A short run's keys.  Those past its end, or in another warp's words, are 0.
  // None but NaN's keys are that low, so they can only make T's last bin look
  // fuller when T is 0; it then is cut, and the run's own slots come first.
  uint32_t held_keys[kReg ? kHeld : 1];
  if constexpr (kReg) {
    const int i0 = w0 * 32 + lane;
    const int mine = min(run, w1 * 32) - i0, noted = min(recorded, w1 * 32) - i0;
    const int at = static_cast<int>(late) + i0;
    // held: positions outside [sink, first_recent)
    const uint32_t open = first_recent > a.sink ? first_recent - a.sink : 0;
#pragma unroll
    for (int i = 0; i < kHeld; i += kBatch) {
      float x[kBatch];
      int p[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        x[u] = 32 * (i + u) < mine ? ld_plain(w + i0 + 32 * (i + u)) : 0.f;
        p[u] = 32 * (i + u) < noted ? ld_plain(pos + i0 + 32 * (i + u)) : at + 32 * (i + u);
      }
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const uint32_t k = static_cast<uint32_t>(p[u]) - a.sink >= open ? 0xffffffffu : claim_key(x[u]);
        held_keys[i + u] = 32 * (i + u) < mine ? k : 0u;
      }
    }
  }
  // f(first word, keys, whether every slot of the words is one of the run)
  auto each = [&](auto&& f) {
    for (int q = w0; q < w1; q += kBatch) {
      uint32_t k[kBatch];
      if (load(q, k)) f(q, k, true);
      else f(q, k, false);
    }
  };
  auto hist_of = [&](int pass) {
    return reinterpret_cast<uint32_t*>(smem + L::kHist) + pass * kBins;
  };
  // the slot of word q in this lane is one of this warp's (a key of 0 past the
  // end must not count)
  auto mine = [&](int q) { return q < w1 && q * 32 + lane < run; };

  // The digit of T from the cluster's summed histogram: (bin, how many of its
  // keys stay, how many there are).  The other CTAs add their bins that are not
  // empty, few of the 2048, to the first one's, which finds the digit for all (a
  // sum by every CTA over all bins took 5.5 k cycles with eight of them).
  // A CTA alone with few bins: every warp finds the digit for itself.
  uint32_t need = B;
  auto digit = [&](int pass) -> uint4 {
    __syncthreads();
    if constexpr (kBins == 256) {
      if (C == 1) {
        const uint4* bins = reinterpret_cast<const uint4*>(hist_of(pass)) + 62 - 2 * lane;
        const uint4 hi = bins[1], lo4 = bins[0];         // this lane's bins, from the top
        const uint32_t c[8] = {hi.w, hi.z, hi.y, hi.x, lo4.w, lo4.z, lo4.y, lo4.x};
        uint32_t own = 0;
#pragma unroll
        for (int q = 0; q < 8; ++q) own += c[q];
        uint32_t incl = own;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const uint32_t v = __shfl_up_sync(0xffffffffu, incl, d);
          if (lane >= d) incl += v;
        }
        // the first lane whose bins reach `need`, and the bin of them that does
        const int at = __ffs(__ballot_sync(0xffffffffu, incl >= need)) - 1;
        uint32_t above = incl - own, x = 0, y = 0, z = 0;
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          if (above < need && above + c[q] >= need) {
            x = 255 - 8 * lane - q;
            y = need - above;
            z = c[q];
          }
          above += c[q];
        }
        return make_uint4(__shfl_sync(0xffffffffu, x, at), __shfl_sync(0xffffffffu, y, at),
                          __shfl_sync(0xffffffffu, z, at), 0);
      }
    }
    constexpr int kPer = kBins > kThreadsN ? kBins / kThreadsN : 1;   // bins a thread
    uint32_t* hist = hist_of(pass);
    const int top = kBins - kPer * (tid + 1);          // this thread's bins, from the top
    const bool any = top >= 0;
    if (C > 1) {
      if (pass == 0) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
      if (rank != 0 && any) {
        const uint32_t to = map_cluster(smem_addr(&hist[top]), 0);
#pragma unroll
        for (int q = 0; q < kPer; ++q)
          if (hist[top + q]) add_cluster_u32(to + 4 * q, hist[top + q]);
      }
      cluster_sync();
    }
    if (rank == 0) {
      uint32_t c[kPer], own = 0;
#pragma unroll
      for (int q = 0; q < kPer; ++q) {
        c[q] = any ? hist[top + q] : 0u;
        own += c[q];
      }
      uint32_t incl = own;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const uint32_t v = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += v;
      }
      if (lane == 31) scan[warp] = incl;
      __syncthreads();
      uint32_t above = incl - own;
#pragma unroll
      for (int v = 0; v < kWarpsN; ++v)
        if (v < warp) above += scan[v];
      if (above < need && above + own >= need) {       // one thread
        uint4 found = make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int q = kPer - 1; q >= 0; --q) {
          if (above < need && above + c[q] >= need)
            found = make_uint4(top + q, need - above, c[q], 0);
          above += c[q];
        }
        pick[pass] = found;
        for (int r = 1; r < C; ++r) {
          const uint32_t to = map_cluster(smem_addr(&pick[pass]), r);
          st_cluster_u32(to, found.x);
          st_cluster_u32(to + 4, found.y);
          st_cluster_u32(to + 8, found.z);
        }
      }
    }
    if (C > 1) cluster_sync();
    else __syncthreads();
    return pick[pass];
  };

  // the histograms are clear; the cluster's are known to be before the first
  // CTA's is added to
  if (C > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  __syncthreads();
  const uint32_t below = (1u << lane) - 1;
  uint32_t T = 0;
  bool cut = false;                                    // only some keys equal to T stay
  if constexpr (kReg) {
    uint4 d = make_uint4(0, 0, 0, 0);
    int rest = 32;                                       // bits below T's digits so far
#pragma unroll
    for (int pass = 0; pass < L::kDigits; ++pass) {
      if (pass > 0 && d.z == need) break;                // all keys with these digits stay
      const int shift = 32 - L::kDigit * (pass + 1);
      uint32_t* h = hist_of(pass);
#pragma unroll
      for (int u = 0; u < kHeld; ++u)
        if (w0 + u < w1 && (pass == 0 || held_keys[u] >> (shift + L::kDigit) == T))
          atomicAdd(&h[(held_keys[u] >> shift) & (kBins - 1)], 1u);
      d = digit(pass);
      need = d.y;
      T = T << L::kDigit | d.x;
      rest = shift;
    }
    T <<= rest;
    cut = d.z != need;
    uint32_t f = 0, e = 0;                               // lane u: those of word w0 + u
    if (!cut) {
#pragma unroll
      for (int u = 0; u < kHeld; ++u) {
        const uint32_t v = __ballot_sync(0xffffffffu, held_keys[u] >= T);
        if (lane == u) f = v;
      }
    } else {
#pragma unroll
      for (int u = 0; u < kHeld; ++u) {
        const uint32_t v = __ballot_sync(0xffffffffu, held_keys[u] > T);
        const uint32_t z = __ballot_sync(0xffffffffu, held_keys[u] == T);
        if (lane == u) {
          f = v;
          e = z;
        }
      }
    }
    if (lane < w1 - w0) {
      flags[w0 + lane] = f;
      same[w0 + lane] = e;
    }
  } else {
    uint32_t* h0 = hist_of(0);
    each([&](int q, const uint32_t (&k)[kBatch], bool whole) {
#pragma unroll
      for (int u = 0; u < kBatch; ++u)
        if (whole || mine(q + u)) atomicAdd(&h0[k[u] >> 21], 1u);
    });
    const uint4 d0 = digit(0);
    need = d0.y;
    uint32_t* h1 = hist_of(1);
    uint2* wcand = cand + warp * L::kListed;             // this warp's list
    int listed_keys = 0;
    each([&](int q, const uint32_t (&k)[kBatch], bool whole) {
      uint32_t word = 0;                                 // lane u: the flags of word q + u
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const uint32_t top = k[u] >> 21;
        const uint32_t f = __ballot_sync(0xffffffffu, top > d0.x);
        if (lane == u) word = f;
        const bool c = top == d0.x && (whole || mine(q + u));
        const uint32_t m = __ballot_sync(0xffffffffu, c);
        if (m) {
          const int at = listed_keys + __popc(m & below);
          if (c && at < L::kListed) wcand[at] = make_uint2(k[u], (q + u) * 32 + lane);
          listed_keys += __popc(m);
        }
      }
      if (lane < kBatch && (whole || q + lane < w1)) {
        flags[q + lane] = word;
        same[q + lane] = 0;
      }
    });
    const bool listed = listed_keys <= L::kListed;     // else this warp goes through its words again
    __syncwarp();
    // f(key, slot) over this warp's keys that share T's first digit
    auto candidates = [&](auto&& f) {
      if (listed) {
        for (int i = lane; i < listed_keys; i += 32) f(wcand[i].x, static_cast<int>(wcand[i].y));
      } else {
        each([&](int q, const uint32_t (&k)[kBatch], bool) {
#pragma unroll
          for (int u = 0; u < kBatch; ++u)
            if ((k[u] >> 21) == d0.x && mine(q + u)) f(k[u], (q + u) * 32 + lane);
        });
      }
    };
    candidates([&](uint32_t k, int) { atomicAdd(&h1[(k >> 10) & 2047u], 1u); });
    const uint4 d1 = digit(1);
    need = d1.y;
    uint32_t* h2 = hist_of(2);
    const uint32_t prefix = d0.x << 11 | d1.x;
    T = prefix << 10;
    if (d1.z != need) {                                  // else all keys with these digits stay
      candidates([&](uint32_t k, int) {
        if ((k >> 10) == prefix) atomicAdd(&h2[k & 1023u], 1u);
      });
      const uint4 d2 = digit(2);
      need = d2.y;
      T |= d2.x;
      cut = d2.z != need;
    }
    candidates([&](uint32_t k, int i) {
      if (k >= T) atomicOr(cut && k == T ? &same[i >> 5] : &flags[i >> 5], 1u << (i & 31));
    });
  }
  __syncthreads();

  // ---- ranks, a thread a share of whole words ----
  // exclusive scan of a pair of counts over the cluster's threads, in order of
  // the slots; every CTA calls it (it holds cluster barriers)
  auto before = [&](uint32_t x, uint32_t y, int slot) -> uint2 {
    uint32_t* sums = scan + slot * 2 * kWarpsN;
    uint32_t ix = x, iy = y;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const uint32_t u = __shfl_up_sync(0xffffffffu, ix, d), v = __shfl_up_sync(0xffffffffu, iy, d);
      if (lane >= d) {
        ix += u;
        iy += v;
      }
    }
    if (lane == 31) {
      sums[warp] = ix;
      sums[kWarpsN + warp] = iy;
    }
    __syncthreads();
    ix -= x;
    iy -= y;
    uint32_t tx = 0, ty = 0;
#pragma unroll
    for (int v = 0; v < kWarpsN; ++v) {
      if (v == warp) {
        ix += tx;
        iy += ty;
      }
      tx += sums[v];
      ty += sums[kWarpsN + v];
    }
    if (C > 1) {
      if (tid == 0) {
        totals[2 * slot] = tx;
        totals[2 * slot + 1] = ty;
      }
      cluster_sync();
      tx = ty = 0;
      if (lane < rank) {
        tx = ld_cluster_u32(map_cluster(smem_addr(&totals[2 * slot]), lane));
        ty = ld_cluster_u32(map_cluster(smem_addr(&totals[2 * slot + 1]), lane));
      }
      ix += __reduce_add_sync(0xffffffffu, tx);
      iy += __reduce_add_sync(0xffffffffu, ty);
    }
    return make_uint2(ix, iy);
  };
  const int tper = (words + kThreadsN - 1) / kThreadsN;
  const int t0 = min(tid * tper, words), t1 = min(t0 + tper, words);
  if (cut) {
    uint32_t ties = 0;
    for (int q = t0; q < t1; ++q) ties += __popc(same[q]);
    ties = before(ties, 0, 0).x;
    for (int q = t0; q < t1; ++q) {                    // the first `need` of them stay
      uint32_t e = same[q], take = 0;
      for (; e && ties < need; ++ties, e &= e - 1) take |= e & (0u - e);
      ties += __popc(e);
      flags[q] |= take;
    }
  }
  const int front = min(max(kept - lo, 0), run);       // slots of the run below the new length
  // bits of word q below the new length
  auto front_bits = [&](int q) -> uint32_t {
    const int m = front - q * 32;
    return m >= 32 ? 0xffffffffu : m <= 0 ? 0u : (1u << m) - 1;
  };
  uint32_t holes = 0, tails = 0;
  for (int q = t0; q < t1; ++q) {
    const uint32_t f = flags[q], in = front_bits(q);
    holes += __popc(in & ~f);
    tails += __popc(f & ~in);
  }
  const uint2 first = before(holes, tails, 1);

  // ---- the list of moved slots, entry r in CTA r >> list_shift ----
  const uint32_t mask = (1u << list_shift) - 1;
  const uint32_t list_at = smem_addr(list);
  uint32_t r = first.y;
  for (int q = t0; q < t1; ++q) {
    for (uint32_t t = flags[q] & ~front_bits(q); t; t &= t - 1, ++r) {
      const uint32_t slot = lo + q * 32 + __ffs(t) - 1;
      if (C > 1) st_cluster_u32(map_cluster(list_at + 4 * (r & mask), r >> list_shift), slot);
      else list[r] = slot;
    }
  }
  // a word's holes take consecutive entries: the word's first rank goes where
  // the word's equal bits were, and a warp then writes whole words
  r = first.x;
  for (int q = t0; q < t1; ++q) {
    same[q] = r;
    r += __popc(front_bits(q) & ~flags[q]);
  }
  if (C > 1) cluster_sync();
  else __syncthreads();
  for (int q = warp; q * 32 < front; q += kWarpsN) {
    const uint32_t h = front_bits(q) & ~flags[q];
    int from = lo + q * 32 + lane;
    if ((h >> lane) & 1u) {
      const uint32_t e = same[q] + __popc(h & below);
      from = C > 1 ? ld_cluster_u32(map_cluster(list_at + 4 * (e & mask), e >> list_shift)) : list[e];
    }
    if (q * 32 + lane < front) source[lo + q * 32 + lane] = from;
  }
  if (C > 1) cluster_sync();                           // no CTA leaves while its list is read
}

// ---------------------------------------------------------------------------
// Compact: slot i < new_lens[s] takes the row of slot source[i].  A CTA takes
// 256 kPer slots of one (sequence, KV head): each thread looks at kPer of them
// and moves their weights and positions, the slots to move go into a list, and
// the CTA copies their K and V rows in 16-byte units, consecutive threads along a
// row.
//
// A moved token costs 8 D + 16 bytes (read and written), in rows of 2 D bytes at
// scattered places: 8 x 8 rows of 32768 to 131072 slots cut to 4096, D = 128, about
// all of them moved: 48 us for 263 MB, 84 % of the copy rate.  128 x 8
// rows of 1017 slots cut to 1000 move 17 rows each: 8.5 us, a chain of dependent
// loads (source, table, row) rather than bytes.
// ---------------------------------------------------------------------------
constexpr int kCompactThreads = 256;
constexpr int kCompactBatch = 4;      // units of K and of V a thread loads before it stores any

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

template <int kPer>
__global__ void __launch_bounds__(kCompactThreads)
    evict_compact_kernel(const CompactArgs a) {
  __shared__ int2 list[kCompactThreads * kPer];   // (source, destination) rows of the flat cache
  __shared__ int moves;
  const int tid = threadIdx.x;
  const int row = blockIdx.x / a.chunks, chunk = blockIdx.x - row * a.chunks;
  const int s = row / a.e.num_kv_heads, kv = row - s * a.e.num_kv_heads;
  if (tid == 0) moves = 0;
  pdl_launch_dependents();
  pdl_wait();
  const int n = a.e.context_lens[s], kept = a.e.new_lens[s];
  const int recorded = min(max(a.e.recorded_lens[s], 0), n);
  const int len = a.e.seq_lens[s];
  if (n < 0 || n > a.e.max_tokens || kept < 0 || kept > n || kept > a.e.budget) {
    if (tid == 0 && chunk == 0 && kv == 0) record_error(kErrContextLen, s);
    return;
  }
  const size_t base = static_cast<size_t>(row) * a.e.max_tokens;
  const int32_t* source = a.e.source + static_cast<size_t>(row) * a.e.budget;
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
  const int i0 = chunk * kCompactThreads * kPer + tid;
  int from[kPer];
#pragma unroll
  for (int u = 0; u < kPer; ++u) {
    const int i = i0 + u * kCompactThreads;
    from[u] = i < kept ? source[i] : i;
  }
  __syncthreads();                                // the count is clear
#pragma unroll
  for (int u = 0; u < kPer; ++u) {
    const int i = i0 + u * kCompactThreads;
    int j = from[u];
    if (i >= kept) continue;
    if (j != i && (j < kept || j >= n)) {
      record_error(kErrSource, static_cast<long long>(row) * a.e.budget + i);
      j = i;
    }
    bool move = j != i;
    if (move) {
      // (loaded beside the block ids, not after them)
      const float weight = a.e.weights[base + j];
      const int position =
          static_cast<int>(slot_position(a.e.positions + base, recorded, len, n, j));
      const int src = flat(j), dst = flat(i);
      move = src >= 0 && dst >= 0;
      if (move) {
        list[atomicAdd(&moves, 1)] = make_int2(src, dst);
        a.e.weights[base + i] = weight;
        a.e.positions[base + i] = position;
      }
    }
    // a token that stays, or whose move is left out, keeps its own position
    if (!move && i >= recorded)
      a.e.positions[base + i] =
          static_cast<int>(slot_position(a.e.positions + base, recorded, len, n, i));
  }
  __syncthreads();
  const int units = moves * a.row_units;
  const size_t stride = static_cast<size_t>(a.e.num_kv_heads) * a.row_units;
  const uint4* ks = reinterpret_cast<const uint4*>(a.key_cache);
  const uint4* vs = reinterpret_cast<const uint4*>(a.value_cache);
  uint4* kd = reinterpret_cast<uint4*>(a.key_cache);
  uint4* vd = reinterpret_cast<uint4*>(a.value_cache);
  for (int u0 = tid; u0 < units; u0 += kCompactThreads * kCompactBatch) {
    uint4 k[kCompactBatch], v[kCompactBatch];
    size_t to[kCompactBatch];
#pragma unroll
    for (int q = 0; q < kCompactBatch; ++q) {
      const int u = u0 + q * kCompactThreads;
      if (u < units) {
        const int m = u / a.row_units, c = u - m * a.row_units + kv * a.row_units;
        const int2 e = list[m];
        to[q] = e.y * stride + c;
        k[q] = ks[e.x * stride + c];
        v[q] = vs[e.x * stride + c];
      }
    }
#pragma unroll
    for (int q = 0; q < kCompactBatch; ++q) {
      if (u0 + q * kCompactThreads < units) {
        kd[to[q]] = k[q];
        vd[to[q]] = v[q];
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Commit: a thread a sequence; launch latency alone (128 x 8 rows of 1017 slots,
// select, compact and this: 15.4 us; with a copy for each of the lengths, 16.5).
// ---------------------------------------------------------------------------
constexpr int kCommitThreads = 128;

__global__ void __launch_bounds__(kCommitThreads)
    evict_commit_kernel(int32_t* context_lens, int32_t* recorded_lens, const int32_t* new_lens,
                        int num_seqs) {
  pdl_launch_dependents();
  pdl_wait();
  const long long s = static_cast<long long>(blockIdx.x) * kCommitThreads + threadIdx.x;
  if (s >= num_seqs) return;
  const int n = new_lens[s];
  if (n == 0 && context_lens[s] != 0) return;
  context_lens[s] = n;
  recorded_lens[s] = n;
}

}  // namespace pa
