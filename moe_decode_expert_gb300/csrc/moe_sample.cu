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
// A top-k of few tokens needs no count: every CTA takes the j-th of its threads'
// largest, j = k / CTAs, and at least k tokens are not below the least of these.
// Else tokens are counted in bins of 1/32 octave of weight, which tells about where
// a filter ends.  Where few tokens lie above, they are brought to the first CTA, which
// settles everything; otherwise the range of values about the end is divided by 512
// until one value is left, with exact sums (and the whole range if the end was not
// in it).

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
    const float s = fmaxf((l - base) * hi, -2097152.0f) + 12582912.0f;
    return 32 * top + 31 - (__float_as_int(s) - 0x4b400000);
  }
  // sum + the weight of l
  __device__ __forceinline__ uint64_t add(uint64_t sum, float l, const uint2* root) const {
    if (infinite) return l == INFINITY ? sum + (1ull << 44) : sum;
    float e;
    const int n = split(l, e);
    // 2^(e / 32) - 1, |e| <= 0.51: terms of (ln 2 / 32)^i / i!
    const float p =
        e * fmaf(e, fmaf(e, fmaf(e, 9.1725e-9f, 1.69386395e-6f), 2.34607166e-4f), 2.16608494e-2f);
    const uint2 r = root[n & 31];
    const uint32_t mant = r.x + static_cast<uint32_t>(__float2int_rn(__uint_as_float(r.y) * p));
    // mant * 2^(13 - down): the shift right on 32 bits, the shift left in the product
    const int t = top - (n >> 5) - 13;
    const uint32_t m = __funnelshift_rc(mant, 0u, max(t, 0));  // (0 from 32 on: weights below 2^-44)
    return sum + static_cast<uint64_t>(m) * (1u << max(-t, 0));
  }
  __device__ __forceinline__ uint64_t of(float l, const uint2* root) const { return add(0, l, root); }
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
  uint64_t warp[kWarps];         // this CTA's sums by warp, of the last reduction
  uint64_t cta[2][kMaxCtas];     // every CTA's, two reductions in turn
  uint64_t other[2][kMaxCtas];   // of a second sum
  uint64_t said[2][4];           // the first CTA's findings, two in turn
  uint64_t found[2];             // a token found by one CTA
  uint64_t best[kMaxCtas];       // the largest logit, and the key that some of the threads' largest reach
  uint2 root[32];                // 2^(j / 32) in units of 2^-31, whole and in fp32
  uint32_t listed;               // tokens this CTA brought
  uint64_t spare[kWarps];
};

// A CTA's part of a row: its slice lies in shared memory as in global memory about 16-byte
// chunks, with -infinity in the places of the first and last chunk that are not its own.
// Slot i is token first + i.  Every warp has a run of the chunks.
template <int DT>
struct Row {
  using T = typename Stored<DT>::T;
  static constexpr int kVec = 16 / sizeof(T);
  static constexpr int kGrain = DT == MOE_F32 ? 0 : DT == MOE_F16 ? 13 : 16;  // 2^this keys hold one value
  Shared& sh;
  const uint4* s;
  uint32_t* hist;
  uint64_t* list;
  int C, rank, first, q0, q1;  // CTAs, this one, the token of slot 0, this warp's chunks
  int turn, chunks;
  const void* row;  // in global memory, from token 0
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

  static __device__ __forceinline__ void unpack(const uint4& c, float (&v)[kVec]) {
    const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (DT == MOE_F32) {
        v[j] = __uint_as_float(w[j]);  // (made sound when it was stored)
      } else {
        const float2 f = unpack2<DT>(w[j]);
        v[2 * j] = fmaxf(f.x, kNegInf) + 0.0f;
        v[2 * j + 1] = fmaxf(f.y, kNegInf) + 0.0f;
      }
    }
  }
  __device__ __forceinline__ float at(int slot) const {
    return value<DT>(reinterpret_cast<const T*>(s)[slot]);
  }
  // f(value, slot) for this thread's slots
  template <class F>
  __device__ __forceinline__ void each(F f) const {
    for (int q = q0 + lane(); q < q1; q += 32) {
      float v[kVec];
      unpack(s[q], v);
#pragma unroll
      for (int j = 0; j < kVec; ++j) f(v[j], q * kVec + j);
    }
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
  // The same of two sums, the second's into v2.
  __device__ __forceinline__ uint64_t total2(uint64_t v, uint64_t& v2) {
    const uint64_t w2 = warp_sum64(v2);
    __syncthreads();
    if (lane() == 0) sh.spare[warp()] = w2;
    __syncthreads();
    if (warp() == 0) {
      const uint64_t all = warp_sum64(lane() < kWarps ? sh.spare[lane()] : 0ull);
      if (lane() < C) st_peer64(&sh.other[turn ^ 1][rank], lane(), all);
    }
    v = total(v);
    v2 = 0;
    for (int r = 0; r < C; ++r) v2 += sh.other[turn][r];
    return v;
  }
  template <class F>
  __device__ __forceinline__ uint64_t sum(F f) {
    uint64_t v = 0;
    each([&](float x, int i) { v += f(x, i); });
    return total(v);
  }
  // A thread's exclusive sum over the CTA's threads before it; the CTA's sum in *all.
  __device__ __forceinline__ uint64_t scan(uint64_t v, uint64_t* all = nullptr) const {
    uint64_t in = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint64_t p = __shfl_up_sync(0xffffffffu, in, o);
      if (lane() >= o) in += p;
    }
    __syncthreads();
    if (lane() == 31) sh.spare[warp()] = in;
    __syncthreads();
    uint64_t before = 0, sum = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w == warp()) before = sum;
      sum += sh.spare[w];
    }
    if (all) *all = sum;
    return before + in - v;
  }
  // After total() of sums of f: calls hit(value, slot) in the one thread that holds the first slot
  // up to and with which f sums to more than `target`.  The warp's run of chunks that has it is
  // gone through once more by all threads of its CTA.
  template <class F, class H>
  __device__ __forceinline__ void locate(F f, uint64_t target, H hit) const {
    for (int r = 0; r < rank; ++r) {
      if (target < sh.cta[turn][r]) return;
      target -= sh.cta[turn][r];
    }
    if (target >= sh.cta[turn][rank]) return;
    int w = 0;
    for (; target >= sh.warp[w]; ++w) target -= sh.warp[w];
    const int per_warp = (chunks + kWarps - 1) / kWarps;
    const int a = w * per_warp * kVec, b = min(chunks, (w + 1) * per_warp) * kVec;
    const int run = (b - a + kThreads - 1) / kThreads;
    const int i0 = min(b, a + run * static_cast<int>(threadIdx.x)), i1 = min(b, i0 + run);
    uint64_t v = 0;
    for (int i = i0; i < i1; ++i) v += f(at(i), i);
    uint64_t before = scan(v);
    if (target < before || target >= before + v) return;
    for (int i = i0; i < i1; ++i) {
      const float x = at(i);
      before += f(x, i);
      if (target < before) {
        hit(x, i);
        return;
      }
    }
  }

  // The first CTA's threads put what they found into sh.said[turn] of all.
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

  // Counts the tokens that `stays` in their bins, and finds the first and last bin in which, by
  // those counts, the ranking's first k tokens, or the share p of the weight, may end (kUsedBins:
  // behind the last), and how many tokens lie down to the last.
  template <class S>
  __device__ __forceinline__ void find_bins(S stays, bool by_k, uint64_t k, float p, int& b0, int& b1,
                                            uint64_t& tokens) {
    clear_hist();
    each([&](float v, int i) {
      const int b = wt.bin(v);
      if (b < kUsedBins && stays(v, i)) atomicAdd(&hist[b], 1u);
    });
    turn ^= 1;
    sync_row();
    if (rank == 0) {
      uint64_t c[3], w[3], count = 0, mass = 0;
#pragma unroll
      for (int j = 0; j < 3; ++j) {
        const int i = 3 * threadIdx.x + j;
        c[j] = merged(i);
        w[j] = c[j] * ((static_cast<uint64_t>(sh.root[31 - (i & 31)].x) << 13) >> (i >> 5));
        count += c[j];
        mass += w[j];
      }
      uint64_t tokens_all, all;
      uint64_t n = scan(count, &tokens_all);
      uint64_t m = scan(mass, &all);
      // a token's weight is within 2^(1 / 64) of its bin's: two sums' ratio within 2^(1 / 32)
      const auto reached = [&](uint64_t n, uint64_t m, float room) {
        return by_k ? n >= k
                    : static_cast<float>(m) * room * (1.0f - p) >= static_cast<float>(all - m) * p;
      };
#pragma unroll
      for (int j = 0; j < 3; ++j) {
        const uint64_t n1 = n + c[j], m1 = m + w[j];
        const bool none = n == 0;  // (the share 0 of nothing is not reached)
        if (n1 != n) {
          if ((none || !reached(n, m, 1.025f)) && reached(n1, m1, 1.025f)) tell(0, 3 * threadIdx.x + j);
          if ((none || !reached(n, m, 0.975f)) && reached(n1, m1, 0.975f)) {
            tell(1, 3 * threadIdx.x + j);
            tell(2, n1);
          }
        }
        n = n1;
        m = m1;
      }
      if (threadIdx.x == kThreads - 1) {
        if (!reached(n, m, 1.025f)) tell(0, kUsedBins);
        if (!reached(n, m, 0.975f)) {
          tell(1, kUsedBins);
          tell(2, n);
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

  static __device__ __forceinline__ int range_shift(uint32_t klo, uint32_t khi) {
    return max(32 - __clz(static_cast<int>(khi - klo)) - 9, 0);  // kSub = 2^9
  }
  // Adds w to the sum of its part of the range, by 15 bits in three words.
  __device__ __forceinline__ void put(uint32_t part, uint64_t w) const {
    atomicAdd(&hist[part], static_cast<uint32_t>(w) & 0x7fffu);
    if (w >> 15) {
      atomicAdd(&hist[kSub + part], static_cast<uint32_t>(w >> 15) & 0x7fffu);
      atomicAdd(&hist[2 * kSub + part], static_cast<uint32_t>(w >> 30));
    }
  }
  // The rank key of the last of the ranking's first tokens, of those that `stays`, whose f sums to
  // `need` (at least 1).  The parts of the range [klo, khi] are in hist, `above` is what lies above
  // it; false if the end is not in the range.
  template <class S, class F>
  __device__ __forceinline__ bool select(uint32_t klo, uint32_t khi, uint64_t above, S stays, F f, uint64_t need,
                                         uint64_t& key) {
    for (bool filled = true;; filled = false) {
      const int shift = range_shift(klo, khi);
      if (!filled) {
        clear_hist();
        each([&](float v, int i) {
          const uint32_t key = order_key(v);
          if (key >= klo && key <= khi && stays(v, i)) put((khi - key) >> shift, f(v));
        });
      }
      turn ^= 1;
      sync_row();
      if (rank == 0) {
        const int t = threadIdx.x;  // kThreads = kSub
        const uint64_t v = merged(t) + (merged(kSub + t) << 15) + (merged(2 * kSub + t) << 30);
        uint64_t all;
        const uint64_t at = above + scan(v, &all);
        if (at < need && at + v >= need) {
          tell(0, t);
          tell(1, at);
        }
        if (t == 0 && (above >= need || above + all < need)) tell(0, kSub);
      }
      sync_row();
      const uint32_t t = static_cast<uint32_t>(sh.said[turn][0]);
      if (t == kSub) return false;
      above = sh.said[turn][1];
      khi -= t << shift;
      klo = max(klo, khi - ((1u << shift) - 1u));
      if (shift <= kGrain) break;
    }
    // one value is left: by index
    const auto tie = [&](float v, int i) {
      const uint32_t key = order_key(v);
      return key >= klo && key <= khi && stays(v, i) ? f(v) : 0ull;
    };
    sum(tie);
    locate(tie, need - above - 1, [&](float v, int i) {
      for (int r = 0; r < C; ++r) st_peer64(&sh.found[turn], r, key_of(v, first + i));
    });
    sync_row();
    key = sh.found[turn];
    return true;
  }

  // Brings the tokens that are not below `least` to the first CTA's list; how many there are, or -1
  // if a CTA has more than its share of the list.
  __device__ __forceinline__ int gather(float least, int n, int off) {
    const int share = kList / C;
    if (threadIdx.x == 0) sh.listed = 0;
    __syncthreads();
    for (int q = q0 + lane(); q < q1; q += 32) {
      float v[kVec];
      unpack(s[q], v);
      float m = v[0];
#pragma unroll
      for (int j = 1; j < kVec; ++j) m = fmaxf(m, v[j]);
      if (m >= least) {
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
          const int i = q * kVec + j;
          if (v[j] >= least && i >= off && i < off + n) {
            const int at = static_cast<int>(atomicAdd(&sh.listed, 1u));
            if (at < share) st_peer64(list + rank * share + at, 0, key_of(v[j], first + i));
          }
        }
      }
    }
    __syncthreads();
    turn ^= 1;
    if (threadIdx.x < C) st_peer64(&sh.cta[turn][rank], threadIdx.x, sh.listed);
    sync_row();
    int sum = 0;
    bool fits = true;
    for (int r = 0; r < C; ++r) {
      sum += static_cast<int>(sh.cta[turn][r]);
      fits &= sh.cta[turn][r] <= static_cast<uint64_t>(share);
    }
    return fits ? sum : -1;
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

// What a row asks for.
struct Asked {
  float temperature, top_p, u;
  uint64_t w_min;
  int k;  // 0: all
};

// The rest of a row by one CTA, from the m tokens that lead its ranking (their rank keys in
// `keys`, in any order; room for kList, as in `spare`).  `sum`: of all weights, for top_p
// without top_k.
template <int DT>
__device__ __forceinline__ void finish_list(const Row<DT>& r, const Asked& ask, uint64_t* keys, uint64_t* spare, int m,
                                            uint64_t sum, int64_t* token, float* logprob) {
  const Weights& wt = r.wt;
  const int k = ask.k ? min(m, ask.k) : m;
  bool more;
  const auto needed = [&](uint64_t sum) {
    return ask.top_p < 1.0f ? max(times_fraction(sum, ask.top_p, &more) + more, static_cast<uint64_t>(1)) : sum;
  };
  if (m <= 256) {
    // A thread per token: ranks and sums by comparing with every other (21 tokens: 0.5 us where
    // two sorts took 3.4; 256: 2 us).
    const bool in = static_cast<int>(threadIdx.x) < m;
    const uint64_t key = in ? keys[threadIdx.x] : 0ull;
    const float v = value_of_key(key);
    const uint64_t w = in ? r.weight(v) : 0ull;
    if (in) spare[threadIdx.x] = w;
    __syncthreads();
    int rank = 0;
    uint64_t before = 0;
    if (in)
      for (int j = 0; j < m; ++j)
        if (keys[j] > key) {
          ++rank;
          before += spare[j];
        }
    if (ask.k) r.scan(in && rank < k ? w : 0ull, &sum);
    const bool stays = in && rank < k && before < needed(sum) && (w >= ask.w_min || rank == 0);
    __syncthreads();
    if (in) spare[threadIdx.x] = stays ? w : 0ull;
    uint64_t whole;
    r.scan(stays ? w : 0ull, &whole);  // (also: spare is written)
    const uint64_t target = times_fraction(whole, ask.u);
    if (!stays) return;
    before = 0;
    const uint32_t at = static_cast<uint32_t>(key);  // ~index
    for (int j = 0; j < m; ++j)
      if (static_cast<uint32_t>(keys[j]) > at) before += spare[j];
    if (target >= before && target < before + w) {
      *token = static_cast<int>(~at);
      if (logprob) *logprob = log_share(wt, v, w, whole);
    }
    return;
  }
  int n2 = 512;
  while (n2 < m) n2 <<= 1;
  sort_down(keys, m, n2);
  constexpr int kPer = kList / kThreads;
  uint64_t w[kPer], here = 0;
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int i = kPer * threadIdx.x + j;
    w[j] = i < k ? r.weight(value_of_key(keys[i])) : 0ull;
    here += w[j];
  }
  uint64_t all;
  uint64_t before = r.scan(here, &all);
  const uint64_t need = needed(ask.k ? all : sum);
  here = 0;
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const uint64_t to = before + w[j];
    if (before >= need || (w[j] < ask.w_min && kPer * threadIdx.x + j != 0)) w[j] = 0;
    before = to;
    here += w[j];
  }
  uint64_t whole;
  r.scan(here, &whole);
  // by index: sort again, on (~index, place in the ranking) downwards
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int i = kPer * threadIdx.x + j;
    if (i < m) {
      spare[i] = w[j];
      keys[i] = w[j] ? (keys[i] << 32) | static_cast<uint32_t>(i) : static_cast<uint32_t>(i);
    }
  }
  sort_down(keys, m, n2);
  here = 0;
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int i = kPer * threadIdx.x + j;
    w[j] = i < m && (keys[i] >> 32) ? spare[static_cast<uint32_t>(keys[i])] : 0ull;
    here += w[j];
  }
  before = r.scan(here);
  const uint64_t target = times_fraction(whole, ask.u);
  if (target < before || target >= before + here) return;
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    if (target >= before && target < before + w[j]) {
      const int i = static_cast<int>(~static_cast<uint32_t>(keys[kPer * threadIdx.x + j] >> 32));
      *token = i;
      if (logprob) {
        // (its value has left the keys: it is in the row, whose first slot may be another CTA's)
        *logprob = log_share(wt, value<DT>(static_cast<const typename Stored<DT>::T*>(r.row)[i]), w[j], whole);
      }
    }
    before += w[j];
  }
}

template <int DT>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(moe_sampling_t a, int C, int per, uint32_t slice_bytes) {
  using T = typename Stored<DT>::T;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ Shared sh;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rank = static_cast<int>(blockIdx.x % C);
  const int64_t row = blockIdx.x / C;
  if (C > 1) asm volatile("barrier.cluster.arrive.release;" ::: "memory");  // this CTA runs
  if (threadIdx.x < 32) {
    const uint32_t v = c_root[threadIdx.x];
    sh.root[threadIdx.x] = make_uint2(v, __float_as_uint(static_cast<float>(v)));
  }
  pdl_launch_dependents();
  pdl_wait();

  // ---------------------------------------------------------------- the slice
  constexpr int kVec = 16 / sizeof(T);
  const int first = min(a.V, rank * per), n = min(a.V, first + per) - first;
  const T* g = static_cast<const T*>(a.logits) + row * a.logits_stride + first;
  const int off = static_cast<int>((reinterpret_cast<uintptr_t>(g) & 15u) / sizeof(T));
  const int chunks = n ? (off + n + kVec - 1) / kVec : 0;
  T* s = reinterpret_cast<T*>(smem);
  float mine = kNegInf;
  {
    const int c_lo = off ? 1 : 0, c_hi = (off + n) / kVec;  // whole chunks
    constexpr int kAhead = 4;
    for (int c0 = c_lo + threadIdx.x; c0 < c_hi; c0 += kThreads * kAhead) {
      uint4 v[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u)
        if (c0 + u * kThreads < c_hi) v[u] = ld_ordered16(g - off + (c0 + u * kThreads) * kVec);
#pragma unroll
      for (int u = 0; u < kAhead; ++u)
        if (c0 + u * kThreads < c_hi) {
          if constexpr (DT == MOE_F32) {  // NaN to -infinity, -0 to 0
            v[u].x = __float_as_uint(value<DT>(__uint_as_float(v[u].x)));
            v[u].y = __float_as_uint(value<DT>(__uint_as_float(v[u].y)));
            v[u].z = __float_as_uint(value<DT>(__uint_as_float(v[u].z)));
            v[u].w = __float_as_uint(value<DT>(__uint_as_float(v[u].w)));
          }
          *reinterpret_cast<uint4*>(s + (c0 + u * kThreads) * kVec) = v[u];
          float f[kVec];
          Row<DT>::unpack(v[u], f);
#pragma unroll
          for (int j = 0; j < kVec; ++j) mine = fmaxf(mine, f[j]);
        }
    }
    // the first and last chunk where they are not whole: 2 * kVec places
    if (threadIdx.x < 2 * kVec) {
      const int i = threadIdx.x < kVec ? threadIdx.x : (chunks - 1) * kVec + threadIdx.x - kVec;
      const bool whole = i / kVec >= c_lo && i / kVec < c_hi;
      if (chunks && !whole && (threadIdx.x < kVec || chunks > 1)) {
        const bool own = i >= off && i < off + n;
        float f = kNegInf;
        if (own) f = value<DT>(g[i - off]);
        if constexpr (DT == MOE_F32) s[i] = f;
        else s[i] = own ? g[i - off] : (DT == MOE_BF16 ? 0xff80u : 0xfc00u);
        mine = fmaxf(mine, f);
      }
    }
  }
  Asked ask;
  ask.temperature = a.temperature ? a.temperature[row] : 1.0f;
  int k = a.top_k ? a.top_k[row] : 0;
  ask.top_p = a.top_p ? a.top_p[row] : 1.0f;
  const float min_p = a.min_p ? a.min_p[row] : 0.0f;
  ask.u = a.uniforms[row];
  ask.u = ask.u > 0.0f ? fminf(ask.u, 0.99999994f) : 0.0f;
  const bool greedy = ask.temperature <= 0.0f;
  if (greedy || min_p > 1.0f || ask.top_p <= 0.0f) k = 1;
  if (k <= 0 || k >= a.V) k = 0;
  if (a.V == 1) k = 1;
  const bool by_k = k > 0, by_p = ask.top_p < 1.0f;
  ask.k = k;

  // ------------------------------------------- the largest, and what some threads' largest reach
  __syncthreads();
  float best = mine;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) best = fmaxf(best, __shfl_xor_sync(0xffffffffu, best, o));
  if (lane == 0) sh.warp[warp] = __float_as_uint(best);
  const int ctas = (a.V - 1) / per + 1;  // that have tokens
  const int share = (k - 1) / ctas + 1;
  const bool few = k > 1 && 3 * share <= kThreads;
  uint32_t reach = 0;
  if (few) {  // to 18 bits of the key, at most
    const uint32_t key = order_key(mine);
    for (int bit = 31; bit >= 14; --bit) {
      const uint32_t mid = reach | (1u << bit);
      if (__syncthreads_count(key >= mid) >= share) reach = mid;
    }
  } else {
    __syncthreads();
  }
  if (C > 1) asm volatile("barrier.cluster.wait.acquire;" ::: "memory");  // every CTA of the cluster runs
  if (warp == 0) {
    best = lane < kWarps ? __uint_as_float(static_cast<uint32_t>(sh.warp[lane])) : kNegInf;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) best = fmaxf(best, __shfl_xor_sync(0xffffffffu, best, o));
    if (lane < C) st_peer64(&sh.best[rank], lane, (static_cast<uint64_t>(__float_as_uint(best)) << 32) | reach);
  }
  if (C > 1) cluster_sync_all();
  else __syncthreads();
  best = kNegInf;
  for (int r = 0; r < C; ++r) {
    best = fmaxf(best, __uint_as_float(static_cast<uint32_t>(sh.best[r] >> 32)));
    if (r < ctas) reach = min(reach, static_cast<uint32_t>(sh.best[r]));
  }
  int64_t* token = a.tokens + row;
  float* logprob = a.logprobs ? a.logprobs + row : nullptr;
  if (best == kNegInf) {  // nothing to draw (the same in every CTA)
    if (rank == 0 && threadIdx.x == 0) {
      *token = -1;
      if (logprob) *logprob = kNegInf;
    }
    return;
  }

  Row<DT> r{sh, reinterpret_cast<const uint4*>(smem), reinterpret_cast<uint32_t*>(smem + slice_bytes),
            reinterpret_cast<uint64_t*>(smem + slice_bytes + kHistBytes), C, rank, first - off};
  r.chunks = chunks;
  const int per_warp = (chunks + kWarps - 1) / kWarps;
  r.q0 = min(chunks, warp * per_warp);
  r.q1 = min(chunks, r.q0 + per_warp);
  r.turn = 0;
  r.row = static_cast<const T*>(a.logits) + row * a.logits_stride;
  r.wt.init(greedy || !(ask.temperature == ask.temperature) ? 1.0f : ask.temperature, best);

  if (k == 1) {  // rank 0: the first of the largest
    const auto is = [&](float v, int) { return static_cast<uint64_t>(v == best); };
    r.sum(is);
    r.locate(is, 0, [&](float, int i) {
      *token = r.first + i;
      if (logprob) *logprob = 0.0f;
    });
    return;
  }
  bool more;
  ask.w_min = 0;  // weights below it do not stay
  if (min_p > 0.0f) {
    const uint64_t w = r.weight(best);
    ask.w_min = min_p >= 1.0f ? w : times_fraction(w, min_p, &more) + more;
  }

  // ------------------------------------------------------------ the filters
  uint64_t cut = 0;  // smallest rank key that stays
  const auto stays = [&](float v, int i) { return Row<DT>::key_of(v, r.first + i) >= cut; };
  const auto any = [](float, int) { return true; };
  const auto one = [](float) { return static_cast<uint64_t>(1); };
  const auto weigh = [&](float v) { return r.weight(v); };
  const auto needed = [&](uint64_t sum) { return max(times_fraction(sum, ask.top_p, &more) + more, static_cast<uint64_t>(1)); };
  uint64_t kept_above = 0;  // this thread's tokens above a range, if they are known to stay
  float v_hi = INFINITY;
  if (by_k || by_p) {
    int m = -1;
    uint64_t sum = 0, tokens;
    int b0, b1;
    uint32_t klo, khi;
    if (few) m = r.gather(reach > 0x007fffffu ? value_of_key(static_cast<uint64_t>(reach) << 32) : kNegInf, n, off);
    if (m < 0) {
      r.find_bins(any, by_k, k, ask.top_p, b0, b1, tokens);
      r.key_range(b0, b1, klo, khi);
      if (tokens <= kList) {
        if (!by_k) sum = r.sum([&](float v, int) { return r.weight(v); });
        uint32_t least, none;  // (tokens without weight are not wanted, nor those masked)
        r.key_range(b0, min(b1, kUsedBins - 1), least, none);
        m = r.gather(value_of_key(static_cast<uint64_t>(least) << 32), n, off);
      }
    }
    if (m >= 0) {  // the first CTA does the rest
      if (rank != 0) return;
      // its list lies in the CTAs' shares: together, over the slice, which is not read again
      uint64_t* keys = reinterpret_cast<uint64_t*>(smem);
      int at = 0;
      for (int c = 0; c < C; ++c) {
        const int many = static_cast<int>(sh.cta[r.turn][c]);
        for (int i = threadIdx.x; i < many; i += kThreads) keys[at + i] = r.list[c * (kList / C) + i];
        at += many;
      }
      __syncthreads();
      finish_list<DT>(r, ask, keys, r.list, m, sum, token, logprob);
      return;
    }
    if (by_k && b1 < kUsedBins) {
      for (;;) {
        const int shift = Row<DT>::range_shift(klo, khi);
        r.clear_hist();
        const uint64_t above = r.sum([&](float v, int) {
          const uint32_t key = order_key(v);
          if (key >= klo && key <= khi) r.put((khi - key) >> shift, 1);
          return static_cast<uint64_t>(key > khi);
        });
        if (r.select(klo, khi, above, any, one, k, cut)) break;
        klo = 0x007fffffu, khi = order_key(INFINITY);
      }
    }
    if (by_p) {
      if (by_k) {
        r.find_bins(stays, false, 0, ask.top_p, b0, b1, tokens);
        r.key_range(b0, b1, klo, khi);
      }
      for (;;) {
        const int shift = Row<DT>::range_shift(klo, khi);
        r.clear_hist();
        sum = 0;
        kept_above = 0;
        r.each([&](float v, int i) {
          if (!stays(v, i)) return;
          const uint32_t key = order_key(v);
          const uint64_t w = r.weight(v);
          sum += w;
          if (key > khi) kept_above += w;
          else if (key >= klo) r.put((khi - key) >> shift, w);
        });
        uint64_t above = kept_above;
        sum = r.total2(sum, above);
        v_hi = value_of_key(static_cast<uint64_t>(khi) << 32);
        uint64_t key;
        if (r.select(klo, khi, above, stays, weigh, needed(sum), key)) {
          cut = key;
          break;
        }
        klo = 0x007fffffu, khi = order_key(INFINITY);
      }
    }
  }

  // --------------------------------------------------------------- the draw
  const auto kept = [&](float v, int i) {
    if (!stays(v, i)) return static_cast<uint64_t>(0);
    const uint64_t w = r.weight(v);
    return w >= ask.w_min ? w : static_cast<uint64_t>(0);
  };
  uint64_t all = 0;
  if (v_hi < INFINITY && ask.w_min == 0) {  // what lies above the range was summed there
    all = kept_above;
    r.each([&](float v, int i) {
      if (v <= v_hi) all += kept(v, i);
    });
    all = r.total(all);
  } else {
    all = r.sum(kept);
  }
  r.locate(kept, times_fraction(all, ask.u), [&](float v, int i) {
    *token = r.first + i;
    if (logprob) *logprob = log_share(r.wt, v, r.weight(v), all);
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
      std::max(static_cast<uint32_t>(per * sizeof(typename Stored<DT>::T)) + 32u, kListBytes);
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
