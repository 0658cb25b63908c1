// moe_sample.cu — a token from each row of logits: temperature, top-k, top-p,
// min-p and one given random number per row.
//
// A cluster of CTAs holds a row in shared memory (read from HBM once).  Weights
// exp((l - max) / T) are fixed-point numbers of 45 bits at most, so that every sum
// of them is exact and does not depend on the order of its terms; whichever threads
// hold a row, the same token comes out.  Every filter keeps a prefix of the ranking
// by (l descending, index ascending), so the kept set is one bound on the 64-bit
// rank key (order of l, ~index).
//
// Where the bound is sought, tokens are first counted in bins of 1/32 octave of
// weight.  Few tokens down to the bin in question are brought to the first CTA and
// sorted there, which settles everything.  Otherwise the bin's range of values is
// divided by 512 until one value is left, with exact sums.

#include <algorithm>

#include "moe_common.cuh"
#include "moe_internal.h"

namespace moe {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kMaxCtas = 8;       // of a cluster (a row)
constexpr int kMaxSlice = 49152;  // elements of a CTA
constexpr int kMaxV = kMaxCtas * kMaxSlice;
constexpr float kNegInf = -INFINITY;

// 2^(j / 32) in units of 2^-31, rounded.
__constant__ uint32_t c_root[32] = {
    2147483648u, 2194507417u, 2242560872u, 2291666561u, 2341847524u, 2393127307u, 2445529972u, 2499080105u,
    2553802834u, 2609723834u, 2666869345u, 2725266179u, 2784941738u, 2845924021u, 2908241642u, 2971923842u,
    3037000500u, 3103502151u, 3171459999u, 3240905930u, 3311872529u, 3384393094u, 3458501653u, 3534232978u,
    3611622603u, 3690706840u, 3771522796u, 3854108391u, 3938502376u, 4024744348u, 4112874773u, 4202935003u};

__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ uint32_t peer_addr(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ void st_peer64(const void* p, uint32_t rank, uint64_t v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(peer_addr(smem_u32(p), rank)), "l"(v) : "memory");
}

template <int DT>
struct Stored {
  using T = uint16_t;
};
template <>
struct Stored<MOE_F32> {
  using T = float;
};

// A logit's value: NaN as -infinity, -0 as +0 (equal values rank by index).
template <int DT>
__device__ __forceinline__ float value(typename Stored<DT>::T v) {
  float f;
  if constexpr (DT == MOE_F32) f = v;
  else f = unpack2<DT>(v).x;
  return fmaxf(f, kNegInf) + 0.0f;
}

// A row's weights.  With c = 32 log2(e) / T in two terms, l c = n + e, n the nearest
// whole number, the weight is 2^(n / 32) 2^(e / 32): a root from a table of 32, a short
// polynomial for the rest, and a shift that puts the row's largest in [2^44, 2^45).
// e is off by 2^-25 (c has 48 bits and l c at most 17 before the point, or l - max is
// exact and taken first), so a weight by 2^-28 of itself.
struct Weights {
  float hi, lo;   // c
  float base;     // subtracted from l first: 0, or the largest where max * c is far
  int top;        // the largest's octave, n >> 5
  bool infinite;  // the row's largest is +infinity: those have weight 1 and the others 0
  __device__ __forceinline__ void init(float temperature, float largest) {
    const float t = fminf(fmaxf(temperature, 1e-30f), 3.0e38f);
    constexpr float kHi = 46.166241308446828f;  // 32 log2(e) and what fp32 leaves of it
    constexpr float kLo = static_cast<float>(46.16624130844682838 - static_cast<double>(kHi));
    hi = __fdiv_rn(kHi, t);
    lo = __fdiv_rn(fmaf(-hi, t, kHi) + kLo, t);
    infinite = largest == INFINITY;
    const float m = infinite ? 0.0f : largest;
    base = fabsf(m * hi) > 131072.0f ? m : 0.0f;
    top = 0;
    float e;
    top = split(m, e) >> 5;
  }
  // n and e of a logit
  __device__ __forceinline__ int split(float l, float& e) const {
    const float d = l - base;
    const float q = d * hi;
    const float rest = fmaf(d, lo, fmaf(d, hi, -q));
    const float a = fmaxf(q, -2097152.0f);  // (also for -infinity times 0)
    const float s = a + 12582912.0f;
    e = (a - (s - 12582912.0f)) + rest;
    return __float_as_int(s) - 0x4b400000;
  }
  // The bin of a logit, 32 to an octave of weight downwards from the largest's octave; from
  // 45 * 32 on the weight is zero.  (Of d * c as it is rounded, so never rising with l.)
  __device__ __forceinline__ int bin(float l) const {
    if (infinite) return l == INFINITY ? 31 : 1 << 20;
    float e;
    return 32 * top + 31 - split(l, e);
  }
  __device__ __forceinline__ uint64_t of(float l, const uint32_t* root, int* at = nullptr) const {
    if (at) *at = 31;
    if (infinite) return l == INFINITY ? 1ull << 44 : 0ull;
    float e;
    const int n = split(l, e);
    if (at) *at = 32 * top + 31 - n;
    const int down = top - (n >> 5);
    if (down > 44) return 0ull;
    // 2^(e / 32) - 1, |e| <= 0.51: terms of (ln 2 / 32)^i / i!
    const float p =
        e * fmaf(e, fmaf(e, fmaf(e, 9.1725e-9f, 1.69386395e-6f), 2.34607166e-4f), 2.16608494e-2f);
    const uint32_t r = root[n & 31];
    const uint32_t mant = r + static_cast<uint32_t>(__float2int_rn(static_cast<float>(r) * p));
    return (static_cast<uint64_t>(mant) << 13) >> down;
  }
};

__device__ __forceinline__ uint64_t warp_sum64(uint64_t v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// x * f for a fraction f in [0, 1), rounded down; *more: whether something was lost.
__device__ __forceinline__ uint64_t times_fraction(uint64_t x, float f, bool* more = nullptr) {
  // f as a multiple of 2^-64 (exact down to 2^-40; what lies below is lost)
  const uint32_t b = __float_as_uint(f);
  const int e = static_cast<int>(b >> 23) - 127;  // f = 1.m * 2^e, e <= -1
  uint64_t q = static_cast<uint64_t>((b & 0x7fffffu) | 0x800000u);
  const int up = 64 - 23 + e;
  q = b < 0x00800000u ? 0ull : up >= 0 ? q << up : up > -24 ? q >> -up : 0ull;
  if (more) *more = x * q != 0ull;
  return __umul64hi(x, q);
}

constexpr int kBins = 1536;        // counted: 45 octaves of weight by 32, a multiple of the threads
constexpr int kUsedBins = 45 * 32;
constexpr int kSub = kBins / 3;    // a value's range is divided by this, 3 words of 15 bits a sum
constexpr int kList = 2048;        // tokens that one CTA sorts
constexpr uint32_t kHistBytes = kBins * 4, kListBytes = kList * 8;

__device__ __forceinline__ uint32_t ld_peer32(const void* p, uint32_t rank) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(peer_addr(smem_u32(p), rank)) : "memory");
  return v;
}

// What the CTAs of a row exchange, and a CTA's warps.
struct Shared {
  uint64_t warp[kWarps];       // this CTA's sums by warp, of the last reduction
  uint64_t cta[2][kMaxCtas];   // every CTA's, two reductions in turn
  uint64_t said[2][4];         // the first CTA's findings, two in turn
  uint64_t found[2];           // an index found by one CTA
  float largest[kMaxCtas];
  uint32_t root[32];
  uint32_t listed;             // tokens in this CTA's list
};

template <int DT>
struct Row {
  using T = typename Stored<DT>::T;
  Shared& sh;
  const T* s;       // the slice
  uint32_t* hist;
  uint64_t* list;
  int C, rank, first, lo, hi;  // CTAs, this one, its first token, this warp's part of the slice
  int turn = 0;
  Weights wt;

  __device__ __forceinline__ int lane() const { return threadIdx.x & 31; }
  __device__ __forceinline__ int warp() const { return threadIdx.x >> 5; }
  __device__ __forceinline__ void sync_row() const {
    if (C > 1) cluster_sync_all();
    else __syncthreads();
  }
  static __device__ __forceinline__ uint64_t key_of(float v, int i) {
    return (static_cast<uint64_t>(order_key(v)) << 32) | static_cast<uint32_t>(~i);
  }
  __device__ __forceinline__ uint64_t weight(float v) const { return wt.of(v, sh.root); }

  // f(value, index) for this thread's tokens
  template <class F>
  __device__ __forceinline__ void each(F f) const {
    for (int i = lo + lane(); i < hi; i += 32) f(value<DT>(s[i]), first + i);
  }
  // the whole row's sum of what its threads have
  __device__ __forceinline__ uint64_t total(uint64_t v) {
    v = warp_sum64(v);
    turn ^= 1;
    __syncthreads();  // sh.warp may still be read
    if (lane() == 0) sh.warp[warp()] = v;
    __syncthreads();
    if (warp() == 0) {
      const uint64_t all = warp_sum64(lane() < kWarps ? sh.warp[lane()] : 0ull);
      if (lane() < C) st_peer64(&sh.cta[turn][rank], lane(), all);
    }
    sync_row();
    uint64_t t = 0;
    for (int r = 0; r < C; ++r) t += sh.cta[turn][r];
    return t;
  }
  template <class F>
  __device__ __forceinline__ uint64_t sum(F f) {
    uint64_t v = 0;
    each([&](float x, int i) { v += f(x, i); });
    return total(v);
  }
  // after sum(f): calls hit(value, index) in the one lane that holds the first index up to and
  // with which f sums to more than `target`
  template <class F, class H>
  __device__ __forceinline__ void locate(F f, uint64_t target, H hit) const {
    for (int r = 0; r < rank; ++r) {
      if (target < sh.cta[turn][r]) return;
      target -= sh.cta[turn][r];
    }
    if (target >= sh.cta[turn][rank]) return;
    for (int w = 0; w < warp(); ++w) {
      if (target < sh.warp[w]) return;
      target -= sh.warp[w];
    }
    if (target >= sh.warp[warp()]) return;
    for (int i0 = lo; i0 < hi; i0 += 32) {
      const int i = i0 + lane();
      const float x = i < hi ? value<DT>(s[i]) : kNegInf;
      uint64_t v = i < hi ? f(x, first + i) : 0ull;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint64_t p = __shfl_up_sync(0xffffffffu, v, o);
        if (lane() >= o) v += p;
      }
      const uint32_t over = __ballot_sync(0xffffffffu, v > target);
      if (over) {
        if (lane() == __ffs(over) - 1) hit(x, first + i);
        return;
      }
      target -= __shfl_sync(0xffffffffu, v, 31);
    }
  }

  // A thread's exclusive sum over the CTA's threads before it (each warp's total in sh.warp).
  __device__ __forceinline__ uint64_t scan(uint64_t v) const {
    uint64_t in = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint64_t p = __shfl_up_sync(0xffffffffu, in, o);
      if (lane() >= o) in += p;
    }
    __syncthreads();
    if (lane() == 31) sh.warp[warp()] = in;
    __syncthreads();
    for (int w = 0; w < warp(); ++w) in += sh.warp[w];
    return in - v;
  }
  // What the first CTA's threads put into sh.said[turn] of all (n words of its own), known to all.
  __device__ __forceinline__ void tell(int i, uint64_t v) const {
    for (int r = 0; r < C; ++r) st_peer64(&sh.said[turn][i], r, v);
  }
  __device__ __forceinline__ void clear_hist() const {
    for (int i = threadIdx.x; i < kBins; i += kThreads) hist[i] = 0;
    __syncthreads();
  }
  // A bin of every CTA's together.
  __device__ __forceinline__ uint64_t merged(int i) const {
    uint64_t v = hist[i];
    for (int r = 1; r < C; ++r) v += ld_peer32(hist + i, r);
    return v;
  }

  // The bins (first and last) in which a sum over the ranking reaches `need`, from counts, or
  // from sums of weights cut off to 15 or 16 bits (MASS: the true sums may be 2^-14 more, so
  // the two bins may differ), and about how many tokens lie down to the last.  kUsedBins
  // where it is not reached, with the number of all tokens.
  template <bool MASS>
  __device__ __forceinline__ void find_bins(uint64_t need, int& b0, int& b1, uint64_t& tokens) {
    turn ^= 1;
    sync_row();
    if (rank == 0) {
      uint64_t v[3], c[3], mine = 0, count = 0;
#pragma unroll
      for (int j = 0; j < 3; ++j) {
        const int i = 3 * threadIdx.x + j;
        c[j] = merged(i);
        v[j] = MASS ? (c[j] << 29) >> (i >> 5) : c[j];
        mine += v[j];
        count += c[j];
      }
      uint64_t at = scan(mine);
      uint64_t n = MASS ? scan(count) : at;
      // at most: a word is at least 2^14, and a bin's sum was rounded down once more
      const auto high = [](uint64_t x) { return MASS ? x + (x >> 14) + 2048 : x; };
#pragma unroll
      for (int j = 0; j < 3; ++j) {
        const uint64_t to = at + v[j];
        n += c[j];
        if ((at == 0 || high(at) < need) && high(to) >= need && to > at) tell(0, 3 * threadIdx.x + j);
        if (at < need && to >= need) {
          tell(1, 3 * threadIdx.x + j);
          tell(2, MASS ? n >> 15 : n);
        }
        at = to;
      }
      if (threadIdx.x == kThreads - 1) {
        if (high(at) < need) tell(0, kUsedBins);
        if (at < need) {
          tell(1, kUsedBins);
          tell(2, MASS ? n >> 15 : n);
        }
      }
    }
    sync_row();
    b0 = static_cast<int>(sh.said[turn][0]);
    b1 = static_cast<int>(sh.said[turn][1]);
    tokens = sh.said[turn][2];
  }

  // The keys between which the values of bins b0 to b1 lie, with some room.
  __device__ __forceinline__ void key_range(int b0, int b1, uint32_t& klo, uint32_t& khi) const {
    klo = khi = order_key(INFINITY);
    if (wt.infinite) return;
    const auto edge = [&](float n, float room) {
      const float x = n / wt.hi, v = wt.base + x;
      return order_key(fmaf(fabsf(wt.base) + fabsf(x), room, v + room * 1e-30f));
    };
    const int n0 = 32 * wt.top + 31;
    if (b0 > 0) khi = edge(static_cast<float>(n0 - b0) + 0.5f, 0x1p-20f);
    klo = b1 < kUsedBins ? edge(static_cast<float>(n0 - b1) - 0.5f, -0x1p-20f) : order_key(kNegInf);
    if (klo > khi) klo = khi;  // (not a number: no room was left)
  }

  // The smallest rank key of the ranking's first tokens, of those that `stays`, whose f sums
  // to `need` (at least 1, and reached) — known to lie between two values' keys.
  template <class S, class F>
  __device__ __forceinline__ uint64_t select(uint32_t klo, uint32_t khi, S stays, F f, uint64_t need) {
    constexpr int kGrain = DT == MOE_F32 ? 0 : DT == MOE_F16 ? 13 : 16;  // 2^this keys hold one value
    uint64_t above = sum([&](float v, int i) { return order_key(v) > khi && stays(v, i) ? f(v) : 0ull; });
    for (;;) {
      const int wide = 32 - __clz(static_cast<int>(khi - klo));  // bits of the range
      if (wide <= kGrain) break;
      const int sh_ = max(wide - 9, 0);  // kSub = 2^9
      clear_hist();
      each([&](float v, int i) {
        const uint32_t key = order_key(v);
        if (key >= klo && key <= khi && stays(v, i)) {
          const uint64_t w = f(v);
          const uint32_t at = (khi - key) >> sh_;
          atomicAdd(&hist[at], static_cast<uint32_t>(w) & 0x7fffu);
          if (w >> 15) {
            atomicAdd(&hist[kSub + at], static_cast<uint32_t>(w >> 15) & 0x7fffu);
            atomicAdd(&hist[2 * kSub + at], static_cast<uint32_t>(w >> 30));
          }
        }
      });
      turn ^= 1;
      sync_row();
      if (rank == 0) {
        const int t = threadIdx.x;  // kThreads = kSub
        const uint64_t v = merged(t) + (merged(kSub + t) << 15) + (merged(2 * kSub + t) << 30);
        const uint64_t at = above + scan(v);
        if (at < need && at + v >= need) {
          tell(0, t);
          tell(1, at);
        }
      }
      sync_row();
      const uint32_t t = static_cast<uint32_t>(sh.said[turn][0]);
      above = sh.said[turn][1];
      khi -= t << sh_;
      klo = max(klo, khi - ((1u << sh_) - 1u));
      if (sh_ <= kGrain) break;
    }
    const auto tie = [&](float v, int i) {
      const uint32_t key = order_key(v);
      return key >= klo && key <= khi && stays(v, i) ? f(v) : 0ull;
    };
    sum(tie);
    locate(tie, need - above - 1, [&](float v, int i) {
      for (int r = 0; r < C; ++r) st_peer64(&sh.found[turn], r, key_of(v, i));
    });
    sync_row();
    return sh.found[turn];
  }

  // The tokens for which `in` holds, from all CTAs to `all` of the first; how many there are,
  // or -1 for more than kList (nothing is written to `all` then).
  template <class P>
  __device__ __forceinline__ int gather(P in, uint64_t* all) {
    if (threadIdx.x == 0) sh.listed = 0;
    __syncthreads();
    for (int i0 = lo; i0 < hi; i0 += 32) {
      const int i = i0 + lane();
      const float v = i < hi ? value<DT>(s[i]) : kNegInf;
      const bool yes = i < hi && in(v);
      const uint32_t who = __ballot_sync(0xffffffffu, yes);
      if (!who) continue;
      uint32_t at = 0;
      if (lane() == 0) at = atomicAdd(&sh.listed, static_cast<uint32_t>(__popc(who)));
      at = __shfl_sync(0xffffffffu, at, 0) + static_cast<uint32_t>(__popc(who & ((1u << lane()) - 1u)));
      if (yes && at < kList) list[at] = key_of(v, first + i);
    }
    __syncthreads();
    const uint32_t n = sh.listed;
    turn ^= 1;
    if (threadIdx.x < C) st_peer64(&sh.cta[turn][rank], threadIdx.x, n);
    sync_row();
    uint64_t before = 0, sum = 0;
    for (int r = 0; r < C; ++r) {
      if (r < rank) before += sh.cta[turn][r];
      sum += sh.cta[turn][r];
    }
    if (sum > kList) return -1;
    for (uint32_t i = threadIdx.x; i < n; i += kThreads) st_peer64(all + before + i, 0, list[i]);
    sync_row();
    return static_cast<int>(sum);
  }
};

// Sorts keys[0 .. n) downwards in one CTA; n2: a power of two >= n, the room there is.
__device__ __forceinline__ void sort_down(uint64_t* keys, int n, int n2) {
  for (int i = n + threadIdx.x; i < n2; i += kThreads) keys[i] = 0;
  for (int k = 2; k <= n2; k <<= 1)
    for (int j = k >> 1; j > 0; j >>= 1) {
      __syncthreads();
      for (int t = threadIdx.x; t < n2 / 2; t += kThreads) {
        const int a = 2 * t - (t & (j - 1)), b = a + j;
        const uint64_t x = keys[a], y = keys[b];
        if ((x < y) == ((a & k) == 0)) {
          keys[a] = y;
          keys[b] = x;
        }
      }
    }
  __syncthreads();
}

__device__ __forceinline__ float value_of_key(uint64_t key) {
  const uint32_t o = static_cast<uint32_t>(key >> 32);
  return __uint_as_float(o & 0x80000000u ? o & 0x7fffffffu : ~o);
}

// ln(weight of v / all)
__device__ __forceinline__ float log_share(const Weights& wt, float v, uint64_t w, uint64_t all) {
  if (w >= all - w)  // at least half: from what is missing
    return log1pf(-(static_cast<float>(all - w) / static_cast<float>(all)));
  // by octaves: w = 2^((n + e) / 32 + 44 - top), all = 2^t m
  float e = 0.0f;
  const int n = wt.infinite ? 32 * wt.top : wt.split(v, e);
  const int t = 63 - __clzll(static_cast<long long>(all));
  const float m = static_cast<float>(all << (63 - t)) * 0x1p-63f;  // [1, 2]
  const int octaves = (n >> 5) - wt.top + 44 - t;
  return fmaf(static_cast<float>(octaves * 32 + (n & 31)) + e, 0.02166084939249829f, -logf(m));
}

template <int DT>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(moe_sampling_t a, int C, int per, uint32_t slice_bytes) {
  using T = typename Stored<DT>::T;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ Shared sh;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rank = static_cast<int>(blockIdx.x % C);
  const int64_t row = blockIdx.x / C;
  if (threadIdx.x < 32) sh.root[threadIdx.x] = c_root[threadIdx.x];
  pdl_launch_dependents();
  pdl_wait();

  // ---------------------------------------------------------------- the slice
  const int first = min(a.V, rank * per), n = min(a.V, first + per) - first;
  const T* g = static_cast<const T*>(a.logits) + row * a.logits_stride + first;
  constexpr int kVec = 16 / sizeof(T);
  const int off = static_cast<int>((reinterpret_cast<uintptr_t>(g) & 15u) / sizeof(T));
  T* s = reinterpret_cast<T*>(smem) + off;  // element i: where its 16-byte chunk is one in memory too
  float mine = kNegInf;
  {
    const int head = min(n, (kVec - off) % kVec), chunks = (n - head) / kVec;
    constexpr int kAhead = 4;
    for (int c0 = threadIdx.x; c0 < chunks; c0 += kThreads * kAhead) {
      uint4 v[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u)
        if (c0 + u * kThreads < chunks) v[u] = ld_ordered16(g + head + (c0 + u * kThreads) * kVec);
#pragma unroll
      for (int u = 0; u < kAhead; ++u)
        if (c0 + u * kThreads < chunks) {
          *reinterpret_cast<uint4*>(s + head + (c0 + u * kThreads) * kVec) = v[u];
          const uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if constexpr (DT == MOE_F32) {
              mine = fmaxf(mine, __uint_as_float(w[j]));
            } else {
              const float2 f = unpack2<DT>(w[j]);
              mine = fmaxf(mine, fmaxf(f.x, f.y));
            }
          }
        }
    }
    const int ends = n - chunks * kVec;  // elements before and behind the chunks
    if (static_cast<int>(threadIdx.x) < ends) {
      const int i = static_cast<int>(threadIdx.x) < head ? threadIdx.x : chunks * kVec + threadIdx.x;
      const T v = g[i];
      s[i] = v;
      mine = fmaxf(mine, value<DT>(v));
    }
  }
  const float temperature = a.temperature ? a.temperature[row] : 1.0f;
  int k = a.top_k ? a.top_k[row] : 0;
  const float top_p = a.top_p ? a.top_p[row] : 1.0f;
  const float min_p = a.min_p ? a.min_p[row] : 0.0f;
  float u = a.uniforms[row];
  float best = mine;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) best = fmaxf(best, __shfl_xor_sync(0xffffffffu, best, o));
  if (C > 1) cluster_sync_all();  // every CTA of the cluster runs
  if (lane == 0) sh.warp[warp] = __float_as_uint(best);
  __syncthreads();
  if (warp == 0) {
    best = lane < kWarps ? __uint_as_float(static_cast<uint32_t>(sh.warp[lane])) : kNegInf;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) best = fmaxf(best, __shfl_xor_sync(0xffffffffu, best, o));
    if (lane < C)
      asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(peer_addr(smem_u32(&sh.largest[rank]), lane)), "f"(best)
                   : "memory");
  }
  if (C > 1) cluster_sync_all();
  else __syncthreads();
  best = kNegInf;
  for (int r = 0; r < C; ++r) best = fmaxf(best, sh.largest[r]);
  best += 0.0f;
  if (best == kNegInf) {  // nothing to draw (the same in every CTA)
    if (rank == 0 && threadIdx.x == 0) {
      a.tokens[row] = -1;
      if (a.logprobs) a.logprobs[row] = kNegInf;
    }
    return;
  }

  // ------------------------------------------------------------ the parameters
  u = u > 0.0f ? fminf(u, 0.99999994f) : 0.0f;
  const bool greedy = temperature <= 0.0f;
  if (greedy || min_p > 1.0f || top_p <= 0.0f) k = 1;
  if (k <= 0 || k > a.V) k = a.V;
  const int chunk = per / kWarps;  // of a warp, a multiple of 32
  const int lo = min(n, warp * chunk), hi = min(n, lo + chunk);
  uint32_t* hist = reinterpret_cast<uint32_t*>(smem + slice_bytes);
  Row<DT> r{sh, s, hist, reinterpret_cast<uint64_t*>(smem + slice_bytes + kHistBytes), C, rank, first, lo, hi};
  r.turn = 0;
  r.wt.init(greedy || !(temperature == temperature) ? 1.0f : temperature, best);
  const Weights& wt = r.wt;

  if (k == 1) {  // rank 0: the first of the largest
    const auto is = [&](float v, int) { return static_cast<uint64_t>(v == best); };
    r.sum(is);
    r.locate(is, 0, [&](float, int i) {
      a.tokens[row] = i;
      if (a.logprobs) a.logprobs[row] = 0.0f;
    });
    return;
  }
  const uint64_t w_best = r.weight(best);
  bool more;
  uint64_t w_min = 0;  // weights below it do not stay
  if (min_p > 0.0f) w_min = min_p >= 1.0f ? w_best : times_fraction(w_best, min_p, &more) + more;

  // ------------------------------------------------------------ the filters
  uint64_t cut = 0;  // smallest rank key that stays
  const auto stays = [&](float v, int i) { return Row<DT>::key_of(v, i) >= cut; };
  const bool by_k = k < a.V, by_p = top_p < 1.0f;
  if (by_k || by_p) {
    int b0, b1;
    uint64_t tokens, sum = 0;
    const auto bin = [&](float v) { return wt.bin(v); };
    uint64_t* all = reinterpret_cast<uint64_t*>(smem);  // (over the slice, which is not read again then)
    int m = -1;
    // First every thread's largest is counted, not every token: at least k tokens lie in the bins
    // down to that in which the k-th of these does, and hardly more while threads are many.
    for (bool few = by_k && 3 * k <= kThreads * C;; few = false) {
      r.clear_hist();
      if (few) {
        const int b = bin(fmaxf(mine, kNegInf) + 0.0f);
        if (b < kUsedBins) atomicAdd(&hist[b], 1u);
        r.template find_bins<false>(k, b0, b1, tokens);
        if (b1 == kUsedBins) continue;
      } else if (by_k) {
        r.each([&](float v, int) {
          const int b = bin(v);
          if (b < kUsedBins) atomicAdd(&hist[b], 1u);
        });
        r.template find_bins<false>(k, b0, b1, tokens);
      } else {
        uint64_t v = 0;
        r.each([&](float x, int) {
          int b;
          const uint64_t w = wt.of(x, sh.root, &b);
          v += w;
          if (w) atomicAdd(&hist[b], static_cast<uint32_t>((w << (b >> 5)) >> 29));
        });
        sum = r.total(v);
        const uint64_t need = times_fraction(sum, top_p, &more);
        r.template find_bins<true>(max(need + more, static_cast<uint64_t>(1)), b0, b1, tokens);
      }
      const int last = min(b1, kUsedBins - 1);
      if (tokens <= kList) m = r.gather([&](float v) { return bin(v) <= last; }, all);
      if (m >= 0 || !few) break;
    }
    if (m >= 0) {  // ------------------------------- the first CTA does the rest
      if (rank != 0) return;
      uint64_t* weights = r.list;
      int n2 = 2;
      while (n2 < m) n2 <<= 1;
      sort_down(all, m, n2);
      constexpr int kPer = kList / kThreads;
      // by rank: sums of weights, how many stay
      uint64_t w[kPer], here = 0;
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const int i = kPer * threadIdx.x + j;
        w[j] = i < min(m, k) ? r.weight(value_of_key(all[i])) : 0ull;
        here += w[j];
      }
      uint64_t before = r.scan(here);
      if (by_k) {
        __syncthreads();
        if (threadIdx.x == kThreads - 1) sh.found[0] = before + here;
        __syncthreads();
        sum = sh.found[0];
      }
      uint64_t need = sum;
      if (by_p) need = max(times_fraction(sum, top_p, &more) + more, static_cast<uint64_t>(1));
      uint64_t kept = 0;
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        if (before >= need || w[j] < w_min) w[j] = 0;
        else kept += w[j];
        before += w[j];
      }
      r.scan(kept);
      uint64_t whole = 0;
      for (int i = 0; i < kWarps; ++i) whole += sh.warp[i];
      // by index: sort again, on (~index, place in the ranking) downwards
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const int i = kPer * threadIdx.x + j;
        if (i < n2) {
          weights[i] = w[j];
          if (i < m) all[i] = w[j] ? (all[i] << 32) | static_cast<uint32_t>(i) : static_cast<uint32_t>(i);
        }
      }
      // (the values leave the keys: by place they are wanted once more, for the logarithm)
      sort_down(all, m, n2);
      here = 0;
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const int i = kPer * threadIdx.x + j;
        w[j] = i < m && (all[i] >> 32) ? weights[static_cast<uint32_t>(all[i])] : 0ull;
        here += w[j];
      }
      before = r.scan(here);
      const uint64_t target = times_fraction(whole, u);
      if (target >= before && target < before + here) {
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
          if (target >= before && target < before + w[j]) {
            const int i = static_cast<int>(~static_cast<uint32_t>(all[kPer * threadIdx.x + j] >> 32));
            a.tokens[row] = i;
            if (a.logprobs) {
              const T* p = static_cast<const T*>(a.logits) + row * a.logits_stride + i;
              a.logprobs[row] = log_share(wt, value<DT>(*p), w[j], whole);
            }
          }
          before += w[j];
        }
      }
      return;
    }
    uint32_t klo, khi;
    if (by_k && b1 < kUsedBins) {
      r.key_range(b0, b1, klo, khi);
      cut = r.select(klo, khi, [](float, int) { return true; }, [](float) { return static_cast<uint64_t>(1); }, k);
    }
    if (by_p) {
      if (by_k) {
        r.clear_hist();
        uint64_t v = 0;
        r.each([&](float x, int i) {
          int b;
          const uint64_t w = stays(x, i) ? wt.of(x, sh.root, &b) : 0ull;
          v += w;
          if (w) atomicAdd(&hist[b], static_cast<uint32_t>((w << (b >> 5)) >> 29));
        });
        sum = r.total(v);
        const uint64_t need = times_fraction(sum, top_p, &more);
        r.template find_bins<true>(max(need + more, static_cast<uint64_t>(1)), b0, b1, tokens);
      }
      r.key_range(b0, b1, klo, khi);
      uint64_t need = times_fraction(sum, top_p, &more);
      need = max(need + more, static_cast<uint64_t>(1));
      cut = r.select(klo, khi, stays, [&](float v) { return r.weight(v); }, need);
    }
  }

  // --------------------------------------------------------------- the draw
  const auto kept = [&](float v, int i) {
    if (!stays(v, i)) return static_cast<uint64_t>(0);
    const uint64_t w = r.weight(v);
    return w >= w_min ? w : static_cast<uint64_t>(0);
  };
  const uint64_t all = r.sum(kept);
  r.locate(kept, times_fraction(all, u), [&](float v, int i) {
    a.tokens[row] = i;
    if (a.logprobs) a.logprobs[row] = log_share(wt, v, r.weight(v), all);
  });
}

template <int DT>
moe_status_t launch(const moe_sampling_t& a, cudaStream_t st) {
  // a row's CTAs: slices of at most 16384 elements where 8 of them do, and shorter ones
  // while SMs would be left without any
  const auto slice = [&](int C) { return ((a.V - 1) / C + 1 + kThreads - 1) / kThreads * kThreads; };
  int C = 1;
  while (C < kMaxCtas && (slice(C) > 16384 || (static_cast<int64_t>(a.B) * C * 2 <= sm_count() && slice(C) > 2048)))
    C *= 2;
  const int per = slice(C);
  // the slice with room for its alignment, or a list over it; the bins; a list
  const uint32_t slice_bytes =
      std::max(static_cast<uint32_t>(per * sizeof(typename Stored<DT>::T)) + 16u, kListBytes);
  const size_t smem = slice_bytes + kHistBytes + kListBytes;
  if (raise_smem_limit(sample_kernel<DT>, smem) != cudaSuccess) return check_launch("sample_kernel (smem)");
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.B) * C);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {static_cast<unsigned>(C), 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  if (cudaLaunchKernelEx(&cfg, sample_kernel<DT>, a, C, per, slice_bytes) != cudaSuccess) return check_launch("sample_kernel");
  stat_kernels(1);
  return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" moe_status_t moe_sample(const moe_sampling_t* s, void* stream) {
  if (!s) return set_error(MOE_ERR_INVALID_ARG, "moe_sampling_t is NULL");
  if (s->B < 0 || s->V < 1) return set_error(MOE_ERR_INVALID_ARG, "B must be >= 0 and V >= 1");
  if (s->V > kMaxV) return set_error(MOE_ERR_UNSUPPORTED, "V must be at most %d", kMaxV);
  if (s->B > (1 << 24)) return set_error(MOE_ERR_UNSUPPORTED, "B must be at most 2^24");
  if (s->dtype != MOE_F16 && s->dtype != MOE_BF16 && s->dtype != MOE_F32)
    return set_error(MOE_ERR_UNSUPPORTED, "dtype must be MOE_F16, MOE_BF16 or MOE_F32");
  if (s->B == 0) return MOE_OK;
  if (!s->logits || !s->uniforms || !s->tokens)
    return set_error(MOE_ERR_INVALID_ARG, "logits / uniforms / tokens is NULL");
  moe_sampling_t a = *s;
  if (a.B == 1) a.logits_stride = a.V;  // a single row's stride says nothing
  if (a.logits_stride < a.V) return set_error(MOE_ERR_INVALID_ARG, "the row stride must be at least V");
  const int size = a.dtype == MOE_F32 ? 4 : 2;
  const auto at = [](const void* p) { return reinterpret_cast<uintptr_t>(p); };
  if ((at(a.logits) & (size - 1)) ||
      ((at(a.uniforms) | at(a.temperature) | at(a.top_k) | at(a.top_p) | at(a.min_p) | at(a.logprobs)) & 3u) ||
      (at(a.tokens) & 7u))
    return set_error(MOE_ERR_INVALID_ARG, "a pointer is not aligned to its element type");
  Span in[6], t{at(a.tokens), 8ll * a.B}, lp{at(a.logprobs), 4ll * a.B};
  if (!row_span(a.logits, a.B, a.logits_stride, a.V, size, in[0]))
    return set_error(MOE_ERR_INVALID_ARG, "row strides reach past any memory");
  const void* params[5] = {a.uniforms, a.temperature, a.top_k, a.top_p, a.min_p};
  for (int i = 0; i < 5; ++i) in[1 + i] = Span{at(params[i]), 4ll * a.B};
  bool over = a.logprobs && meet(t, lp);
  for (int i = 0; i < 6; ++i)
    if (i == 0 || params[i - 1]) over |= meet(t, in[i]) || (a.logprobs && meet(lp, in[i]));
  if (over) return set_error(MOE_ERR_INVALID_ARG, "tokens and logprobs must not overlap the other tensors");
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (a.dtype == MOE_F32) return launch<MOE_F32>(a, st);
  return a.dtype == MOE_BF16 ? launch<MOE_BF16>(a, st) : launch<MOE_F16>(a, st);
}
