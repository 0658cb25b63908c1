// moe_sample.cu — a token from each row of logits: temperature, top-k, top-p,
// min-p and one given random number per row.
//
// A cluster of CTAs has a row: in shared memory, read from HBM once, or, where rows are
// many and long, in L2.  Weights exp((l - max) / T) are fixed-point numbers of 45 bits at
// most, so that every sum of them is exact and does not depend on the order of its terms;
// whichever threads hold a row, the same token comes out.  Every filter keeps a prefix of
// the ranking by (l descending, index ascending), so the kept set is one bound on the
// 64-bit rank key (order of l, ~index).
//
// A top-k of few tokens needs no count: every CTA takes the j-th of its threads'
// largest, j = k / CTAs, and at least k tokens are not below the least of these.
// Else tokens are counted in bins of 1/32 octave of weight, which tells about where
// a filter ends.  Where few tokens lie above, they are brought to the first CTA, which
// settles everything.  Otherwise a pass sums what lies above a window about the end,
// and the first CTA gets the window's tokens; where these are too many (ties, or an
// end outside), the range of values is divided by 512 until one value is left.
//
// One row is a chain of latencies (151936 logits 9 us); many rows are bound by their
// instructions, about 50 a warp for 32 tokens where weights are summed: 256 rows of
// 131072, fp32, 81 us without filters, 155 with a top-p that ends among thousands.
// (64 registers, for two CTAs an SM, spill 56 to 96 bytes.)

#include <algorithm>

#include "moe_common.cuh"
#include "moe_exact.h"
#include "moe_internal.h"

namespace moe {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kMaxCtas = 8;       // of a cluster (a row)
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

// A logit's value.  NaN is never largest, has no weight and is not above or equal to anything, as
// -infinity; -0 is turned to 0 where keys are made.
template <int DT>
__device__ __forceinline__ float value(typename Stored<DT>::T v) {
  if constexpr (DT == MOE_F32) return v;
  else return unpack2<DT>(v).x;
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
  bool infinite;  // the row's largest is +infinity: those share it and the others have weight 0
  __device__ __forceinline__ void init(float temperature, float largest) {
    const float t = fminf(fmaxf(temperature, 1e-30f), 3.0e38f);
    constexpr float kHi = 46.166241308446828f;  // 32 log2(e) and what fp32 leaves of it
    constexpr float kLo = static_cast<float>(46.16624130844682838 - static_cast<double>(kHi));
    hi = __fdiv_rn(kHi, t);
    lo = __fdiv_rn(fmaf(-hi, t, kHi) + kLo, t);
    infinite = largest == INFINITY;
    // (infinite times a tiny c is far above every finite one, which has weight 0 below it; its
    // rest is not a number, which no whole number comes of)
    if (infinite) hi = 1e-36f, lo = 0.0f;
    base = !infinite && fabsf(largest * hi) > 131072.0f ? largest : 0.0f;
    top = 0;
    float e;
    top = split(largest, e) >> 5;
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
    const float s = fmaxf((l - base) * hi, -2097152.0f) + 12582912.0f;
    return 32 * top + 31 - (__float_as_int(s) - 0x4b400000);
  }
  // The weight of l is m * f.
  __device__ __forceinline__ void parts(float l, const uint2* root, uint32_t& m, uint32_t& f) const {
    float e;
    const int n = split(l, e);
    // 2^(e / 32) - 1, |e| <= 0.51: terms of (ln 2 / 32)^i / i!
    const float p =
        e * fmaf(e, fmaf(e, fmaf(e, 9.1725e-9f, 1.69386395e-6f), 2.34607166e-4f), 2.16608494e-2f);
    const uint2 r = root[n & 31];
    const uint32_t mant = r.x + static_cast<uint32_t>(__float2int_rn(__uint_as_float(r.y) * p));
    // mant * 2^(13 - down): a shift right on 32 bits, or a factor
    const int t = top - (n >> 5) - 13;
    m = __funnelshift_rc(mant, 0u, max(t, 0));  // (0 from 32 on: weights below 2^-44)
    f = 1u << max(-t, 0);
  }
  // sum + the weight of l
  __device__ __forceinline__ uint64_t add(uint64_t sum, float l, const uint2* root) const {
    uint32_t m, f;
    parts(l, root, m, f);
    return sum + static_cast<uint64_t>(m) * f;
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
constexpr int kUsedBins = kWeightBits * 32;
constexpr int kSub = 512;          // a value's range is divided by this
constexpr int kList = 1024;        // tokens that one CTA sorts
constexpr int kPer = kList / kThreads;
constexpr uint32_t kHistBytes = kBins * 4, kListBytes = kList * 8;
static_assert(kSub == kThreads && kList % kThreads == 0, "a part of a range per thread");
static_assert(kWords * kSub * 4 <= kHistBytes + kListBytes, "a range's sums lie over the counts and the first list");

__device__ __forceinline__ uint32_t ld_peer32(const void* p, uint32_t rank) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(peer_addr(smem_u32(p), rank)) : "memory");
  return v;
}
__device__ __forceinline__ uint4 ld_peer128(const void* p, uint32_t rank) {
  uint4 v;
  asm volatile("ld.shared::cluster.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(peer_addr(smem_u32(p), rank))
               : "memory");
  return v;
}

// What the CTAs of a row exchange, and a CTA's warps.
struct Shared {
  uint64_t warp[kWarps];               // this CTA's sums by warp, of the last reduction
  uint64_t spare[kWarps];
  uint64_t cta[2][kMaxCtas];           // every CTA's, two reductions in turn
  uint64_t other[2][kMaxCtas];         // of a second sum
  uint64_t region[kMaxCtas * kWarps];  // the first CTA's: every warp's sum in the row
  uint64_t said[2][4], finds[4];       // the first CTA's findings, two in turn; being made
  uint64_t found[2];                   // a token found by one CTA
  uint64_t best[kMaxCtas];             // the largest logit, and the key that some of the threads' largest reach
  uint4 edge[2];                       // the first and last chunk where they are not whole
  uint2 root[32];                      // 2^(j / 32) in units of 2^-31, whole and in fp32
  uint32_t listed;                     // tokens this CTA brought
  int middle;
  float place[2];
};

__device__ __forceinline__ float value_of_key(uint64_t key) {
  const uint32_t o = static_cast<uint32_t>(key >> 32);
  return __uint_as_float(o & 0x80000000u ? o & 0x7fffffffu : ~o);
}
__device__ __forceinline__ float value_of_order(uint32_t key) { return value_of_key(static_cast<uint64_t>(key) << 32); }

// A CTA's part of a row, in 16-byte chunks as they lie in global memory, with -infinity in
// the places of the first and last chunk that are not its own.  Slot i is token first + i.
// Every warp has a run of the chunks.  HELD: the chunks are in shared memory.
template <int DT, bool HELD>
struct Row {
  using T = typename Stored<DT>::T;
  static constexpr int kVec = 16 / sizeof(T);
  static constexpr int kGrain = DT == MOE_F32 ? 0 : DT == MOE_F16 ? 13 : 16;  // 2^this keys hold one value
  Shared& sh;
  const uint4* s;
  uint32_t* hist;
  uint64_t *list, *list2;
  int C, rank, first, off, n;  // CTAs, this one, the token of slot 0, its own slots: off to off + n
  int chunks, per_warp;
  int turn;
  Weights wt;

  __device__ __forceinline__ int lane() const { return threadIdx.x & 31; }
  __device__ __forceinline__ int warp() const { return threadIdx.x >> 5; }
  __device__ __forceinline__ void sync_row() const {
    if (C > 1) cluster_sync_all();
    else __syncthreads();
  }
  static __device__ __forceinline__ uint64_t key_of(float v, int i) {
    return (static_cast<uint64_t>(order_key(v + 0.0f)) << 32) | static_cast<uint32_t>(~i);
  }
  __device__ __forceinline__ uint64_t weight(float v) const { return wt.of(v, sh.root); }

  static __device__ __forceinline__ void unpack(const uint4& c, float (&v)[kVec]) {
    const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (DT == MOE_F32) {
        v[j] = __uint_as_float(w[j]);
      } else {
        const float2 f = unpack2<DT>(w[j]);
        v[2 * j] = f.x;
        v[2 * j + 1] = f.y;
      }
    }
  }
  __device__ __forceinline__ uint4 chunk(int q) const {
    if constexpr (HELD) return s[q];
    if (q == 0) return sh.edge[0];
    if (q == chunks - 1) return sh.edge[1];
    return ld_ordered16(s + q);
  }
  __device__ __forceinline__ float at(int slot) const {
    const uint4 c = chunk(slot / kVec);
    float v[kVec], x = 0.0f;
    unpack(c, v);
#pragma unroll
    for (int j = 0; j < kVec; ++j)
      if (j == slot % kVec) x = v[j];
    return x;
  }
  // f(values, first slot) for this thread's chunks
  template <class F>
  __device__ __forceinline__ void chunks_of(F f) const {
    const int q0 = min(chunks, warp() * per_warp), q1 = min(chunks, q0 + per_warp);
    float v[kVec];
    if constexpr (HELD) {
      for (int q = q0 + lane(); q < q1; q += 32) {
        unpack(s[q], v);
        f(v, q * kVec);
      }
    } else {  // two loads ahead
      uint4 a = make_uint4(0, 0, 0, 0), b = a;
      if (q0 + lane() < q1) a = chunk(q0 + lane());
      if (q0 + lane() + 32 < q1) b = chunk(q0 + lane() + 32);
      for (int q = q0 + lane(); q < q1; q += 32) {
        unpack(a, v);
        a = b;
        if (q + 64 < q1) b = chunk(q + 64);
        f(v, q * kVec);
      }
    }
  }
  // f(value, slot) for this thread's slots
  template <class F>
  __device__ __forceinline__ void each(F f) const {
    chunks_of([&](const float (&v)[kVec], int i) {
#pragma unroll
      for (int j = 0; j < kVec; ++j) f(v[j], i + j);
    });
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
  // Calls hit(value, slot) in the one thread that holds the first slot of warp w's run up to and
  // with which f sums to more than `target`.  All threads of the CTA go through the run once more.
  template <class F, class H>
  __device__ __forceinline__ void locate_in(int w, F f, uint64_t target, H hit) const {
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
  // The same of the whole row, after total() of sums of f.
  template <class F, class H>
  __device__ __forceinline__ void locate(F f, uint64_t target, H hit) const {
    for (int r = 0; r < rank; ++r) {
      if (target < sh.cta[turn][r]) return;
      target -= sh.cta[turn][r];
    }
    if (target >= sh.cta[turn][rank]) return;
    int w = 0;
    for (; target >= sh.warp[w]; ++w) target -= sh.warp[w];
    locate_in(w, f, target, hit);
  }

  // What threads of the first CTA left in sh.finds, to all CTAs; with a barrier of the row.
  __device__ __forceinline__ void tell(int words) const {
    if (rank == 0) {
      __syncthreads();
      if (static_cast<int>(threadIdx.x) < C)
        for (int i = 0; i < words; ++i) st_peer64(&sh.said[turn][i], threadIdx.x, sh.finds[i]);
    }
    sync_row();
  }
  template <int N = kBins>
  __device__ __forceinline__ void clear_hist() const {
    for (int i = threadIdx.x; i < N; i += kThreads) hist[i] = 0;
    __syncthreads();
  }

  // The key of the value n / 32 octaves of weight up from weight 1, with some room to either side.
  __device__ __forceinline__ uint32_t key_at(float n, float room) const {
    if (wt.infinite || n == INFINITY) return order_key(INFINITY);
    if (n == -INFINITY) return order_key(kNegInf);
    const float x = n / wt.hi, v = wt.base + x;
    // (-0 as 0, as the tokens' keys have it; past the largest float: infinity, not a number's key)
    return min(order_key(fmaf(fabsf(wt.base) + fabsf(x), room, v + room * 1e-30f) + 0.0f), order_key(INFINITY));
  }
  // The least value that a token with some weight, down to bin b, has.
  __device__ __forceinline__ float least_of(int b) const {
    return value_of_order(key_at(static_cast<float>(32 * wt.top + 31 - min(b, kUsedBins - 1)) - 0.5f, -0x1p-20f));
  }

  // Counts the tokens that `stays` in their bins, and finds by those counts a window of keys in which
  // the ranking's first k tokens, or the share p of the weight, should end; the last bin where they
  // may (kUsedBins: behind the last), and how many tokens lie down to it.
  template <bool ALL, class S>
  __device__ __forceinline__ void find_bins(S stays, bool by_k, uint64_t k, float p, uint32_t& klo, uint32_t& khi, int& b1,
                                            uint64_t& tokens) {
    clear_hist();
    each([&](float v, int i) {
      const int b = wt.bin(v);
      if (b < kUsedBins && (ALL || stays(v, i))) atomicAdd(&hist[b], 1u);
    });
    turn ^= 1;
    sync_row();
    if (rank == 0) {
      uint64_t count = 0, mass = 0, w[4];
      uint32_t c[4] = {};
      if (threadIdx.x < kBins / 4) {
        uint4 h = reinterpret_cast<const uint4*>(hist)[threadIdx.x];
#pragma unroll
        for (int r0 = 1; r0 < kMaxCtas; r0 += 4) {  // several on their way: one takes most of a microsecond
          uint4 o[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            o[u] = make_uint4(0, 0, 0, 0);
            if (r0 + u < C) o[u] = ld_peer128(hist + 4 * threadIdx.x, r0 + u);
          }
#pragma unroll
          for (int u = 0; u < 4; ++u) h.x += o[u].x, h.y += o[u].y, h.z += o[u].z, h.w += o[u].w;
        }
        c[0] = h.x, c[1] = h.y, c[2] = h.z, c[3] = h.w;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int i = 4 * threadIdx.x + j;
        // (rounded up: what lies behind the end is not to be taken for less than it is)
        w[j] = c[j] * (((static_cast<uint64_t>(sh.root[31 - (i & 31)].x) << 13) >> min(i >> 5, 63)) + 1);
        count += c[j];
        mass += w[j];
      }
      uint64_t all;
      uint64_t n = scan(count);
      uint64_t m = scan(mass, &all);
      // the share p is reached where m (1 - p) >= (all - m) p: where at most this lies behind; a
      // token's weight is within 2^(1 / 64) of its bin's, so two sums' ratio within 2^(1 / 32)
      uint64_t behind[3];
#pragma unroll
      for (int j = 0; j < 3; ++j) {
        const float room = (j == 0 ? 1.025f : j == 1 ? 1.0f : 0.975f) * (1.0f - p);
        behind[j] = by_k ? 0 : times_fraction(all, fminf(__fdividef(room, room + p), 0.99999994f));
      }
      const auto reached = [&](uint64_t n, uint64_t m, int j) { return by_k ? n >= k : all - m <= behind[j]; };
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint64_t n1 = n + c[j], m1 = m + w[j];
        const bool none = n == 0;  // (the share 0 of nothing is not reached)
        if (c[j]) {
          if ((none || !reached(n, m, 0)) && reached(n1, m1, 0)) {
            sh.finds[0] = 4 * threadIdx.x + j;
            sh.finds[3] = n;
          }
          if ((none || !reached(n, m, 1)) && reached(n1, m1, 1)) {
            sh.middle = 4 * threadIdx.x + j;
            // where in the bin, if its tokens are spread evenly, and half of a window for 512 of them
            sh.place[0] = by_k ? __fdividef(static_cast<float>(k - n), static_cast<float>(c[j]))
                               : __fdividef(static_cast<float>(all - behind[1] - m), static_cast<float>(w[j]));
            sh.place[1] = __fdividef(256.0f, static_cast<float>(c[j]));
          }
          if ((none || !reached(n, m, 2)) && reached(n1, m1, 2)) {
            sh.finds[1] = 4 * threadIdx.x + j;
            sh.finds[2] = n1;
          }
        }
        n = n1;
        m = m1;
      }
      if (threadIdx.x == kThreads - 1) {
        if (!reached(n, m, 0)) sh.finds[0] = kUsedBins;
        if (!reached(n, m, 2)) {
          sh.finds[1] = kUsedBins;
          sh.finds[2] = n;
        }
      }
      __syncthreads();
      // Fewer tokens than a list holds, or about as many, are all taken; of more, those about the
      // place where the end lies if every weight is its bin's, as it nearly always does where
      // tokens are many (and else it is found out).
      if (threadIdx.x == 0) {
        const int n0 = 32 * wt.top + 31;
        float hi = INFINITY, lo = -INFINITY;
        if (sh.finds[1] < kUsedBins && sh.finds[2] - sh.finds[3] > kList * 3 / 4) {
          const float at = static_cast<float>(n0 - sh.middle) + 0.5f - sh.place[0];
          hi = at + sh.place[1];
          lo = at - sh.place[1];
        } else {
          if (sh.finds[0] > 0) hi = static_cast<float>(n0 - static_cast<int>(sh.finds[0])) + 0.5f;
          if (sh.finds[1] < kUsedBins) lo = static_cast<float>(n0 - static_cast<int>(sh.finds[1])) - 0.5f;
        }
        sh.finds[0] = __float_as_uint(hi);
        sh.finds[3] = __float_as_uint(lo);
      }
    }
    tell(4);
    b1 = static_cast<int>(sh.said[turn][1]);
    tokens = sh.said[turn][2];
    klo = key_at(__uint_as_float(static_cast<uint32_t>(sh.said[turn][3])), -0x1p-20f);
    khi = max(klo, key_at(__uint_as_float(static_cast<uint32_t>(sh.said[turn][0])), 0x1p-20f));
  }

  // ------------------------------------------------------- ranges by parts
  // The rank key of the last of the ranking's first tokens, of those that `stays`, whose f sums to
  // `need` (at least 1, and reached): the range of keys, between those of the infinities, is divided
  // until one value is left.  `above`
  // is the sum above the range; where the end is not in it, all begins again with all keys, once: 0
  // if it is not among those, which no exact sums lead to.
  template <class S, class F>
  __device__ __forceinline__ uint64_t select(uint32_t klo, uint32_t khi, uint64_t above, S stays, F f, uint64_t need) {
    for (bool again = false;;) {
      const int shift = part_shift(klo, khi);
      static_assert(kSub == 512, "what part_shift() divides by");
      clear_hist<kWords * kSub>();
      each([&](float v, int i) {
        const uint32_t key = order_key(v + 0.0f);
        if (in_range(key, klo, khi) && i >= off && i < off + n && stays(v, i)) {
          const uint64_t w = f(v);
          const uint32_t part = part_of(key, khi, shift);
#pragma unroll
          for (int j = 0; j < kWords; ++j)
            if (word_of(w, j)) atomicAdd(&hist[j * kSub + part], word_of(w, j));
        }
      });
      turn ^= 1;
      sync_row();
      if (rank == 0) {
        const int t = threadIdx.x;  // kThreads = kSub
        uint64_t v = 0, all;
#pragma unroll
        for (int r0 = 0; r0 < kMaxCtas; r0 += 4) {
          uint32_t o[4][kWords] = {};
#pragma unroll
          for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int j = 0; j < kWords; ++j)
              if (r0 + u < C) o[u][j] = ld_peer32(hist + j * kSub + t, r0 + u);
#pragma unroll
          for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int j = 0; j < kWords; ++j) v += of_word(o[u][j], j);
        }
        const uint64_t at = above + scan(v, &all);
        if (at < need && at + v >= need) {
          sh.finds[0] = t;
          sh.finds[1] = at;
        }
        if (t == 0 && (above >= need || above + all < need)) sh.finds[0] = kSub;
      }
      tell(2);
      const uint32_t t = static_cast<uint32_t>(sh.said[turn][0]);
      if (t == kSub) {
        if (again) return 0;
        again = true;
        klo = order_key(kNegInf), khi = order_key(INFINITY);
        above = 0;
        continue;
      }
      above = sh.said[turn][1];
      khi -= t << shift;
      klo = max(klo, khi - ((1u << shift) - 1u));
      if (shift <= kGrain) break;
    }
    // one value is left: by index
    const auto tie = [&](float v, int i) {
      const uint32_t key = order_key(v + 0.0f);
      return in_range(key, klo, khi) && i >= off && i < off + n && stays(v, i) ? f(v) : 0ull;
    };
    sum(tie);
    locate(tie, need - above - 1, [&](float v, int i) {
      for (int r = 0; r < C; ++r) st_peer64(&sh.found[turn], r, key_of(v, first + i));
    });
    sync_row();
    return sh.found[turn];
  }

  // --------------------------------------------------------- lists of tokens
  // A token to this CTA's part of a list.
  __device__ __forceinline__ void bring(float v, int i) const {
    const int at = static_cast<int>(atomicAdd(&sh.listed, 1u));
    if (at < kList) list2[at] = key_of(v, first + i);
  }
  // Those of a chunk that lie between two values, and of the value `tie` only the slots up to `last`.
  __device__ __forceinline__ void bring_some(const float (&v)[kVec], int i, float v_lo, float v_hi,
                                             float tie = 0.0f, int last = INT32_MAX) const {
#pragma unroll
    for (int j = 0; j < kVec; ++j)
      if (v[j] >= v_lo && v[j] <= v_hi && i + j >= off && i + j < off + n && (v[j] != tie || i + j <= last))
        bring(v[j], i + j);
  }
  __device__ __forceinline__ void begin_list() const {
    if (threadIdx.x == 0) sh.listed = 0;
    __syncthreads();
  }
  // The parts together, in the first CTA's list; how many tokens there are, or -1 for more than
  // kList, known to all.
  __device__ __forceinline__ int end_list() {
    __syncthreads();
    const int mine = static_cast<int>(sh.listed);
    turn ^= 1;
    if (static_cast<int>(threadIdx.x) < C) st_peer64(&sh.cta[turn][rank], threadIdx.x, static_cast<uint64_t>(mine));
    sync_row();
    uint64_t before = 0, sum = 0;
    for (int r = 0; r < C; ++r) {
      if (r < rank) before += sh.cta[turn][r];
      sum += sh.cta[turn][r];
    }
    if (sum > kList) return -1;
    for (int i = threadIdx.x; i < mine; i += kThreads) st_peer64(list + before + i, 0, list2[i]);
    sync_row();
    return static_cast<int>(sum);
  }
  // The first CTA, after end_list(): into list2, which sort() takes.
  __device__ __forceinline__ void close_list(int m) const {
    for (int i = threadIdx.x; i < m; i += kThreads) list2[i] = list[i];
    __syncthreads();
  }
  // Brings the tokens that are not below `least`; with SUM, the sum of all weights into `sum`.
  template <bool SUM>
  __device__ __forceinline__ int gather(float least, uint64_t& sum) {
    begin_list();
    uint64_t all = 0;
    chunks_of([&](const float (&v)[kVec], int i) {
      float m = v[0];
#pragma unroll
      for (int j = 1; j < kVec; ++j) m = fmaxf(m, v[j]);
      if constexpr (SUM) {
#pragma unroll
        for (int j = 0; j < kVec; ++j) all = wt.add(all, v[j], sh.root);
      }
      if (m >= least) bring_some(v, i, least, INFINITY);
    });
    if constexpr (SUM) sum = total(all);
    return end_list();
  }

  // Sorts the keys in list2[0 .. m) downwards, in one CTA: by their part of the range of the first
  // words, then by comparing within a part; by exchanges where a part has many.
  __device__ __forceinline__ void sort(int m) const {
    uint32_t most = 0, least = 0xffffffffu;
    uint64_t key[kPer];
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int i = threadIdx.x + j * kThreads;
      key[j] = i < m ? list2[i] : 0ull;
      if (i < m) {
        most = max(most, static_cast<uint32_t>(key[j] >> 32));
        least = min(least, static_cast<uint32_t>(key[j] >> 32));
      }
    }
    most = __reduce_max_sync(0xffffffffu, most);
    least = __reduce_min_sync(0xffffffffu, least);
    __syncthreads();
    if (lane() == 0) sh.spare[warp()] = (static_cast<uint64_t>(most) << 32) | least;
    hist[threadIdx.x] = 0;
    __syncthreads();
    for (int w = 0; w < kWarps; ++w) {
      most = max(most, static_cast<uint32_t>(sh.spare[w] >> 32));
      least = min(least, static_cast<uint32_t>(sh.spare[w]));
    }
    const int shift = max(32 - __clz(static_cast<int>(most - least)) - 9, 0);
    int at[kPer];
#pragma unroll
    for (int j = 0; j < kPer; ++j)
      if (static_cast<int>(threadIdx.x) + j * kThreads < m)
        at[j] = static_cast<int>(atomicAdd(&hist[(most - static_cast<uint32_t>(key[j] >> 32)) >> shift], 1u));
    __syncthreads();
    const uint32_t mine = hist[threadIdx.x];
    if (__syncthreads_or(mine > 64u)) {
      int n2 = 2;
      while (n2 < m) n2 <<= 1;
      for (int i = m + threadIdx.x; i < n2; i += kThreads) list2[i] = 0;
      for (int k = 2; k <= n2; k <<= 1)
        for (int j = k >> 1; j > 0; j >>= 1) {
          __syncthreads();
          for (int t = threadIdx.x; t < n2 / 2; t += kThreads) {
            const int a = 2 * t - (t & (j - 1)), b = a + j;
            const uint64_t x = list2[a], y = list2[b];
            if ((x < y) == ((a & k) == 0)) {
              list2[a] = y;
              list2[b] = x;
            }
          }
        }
      __syncthreads();
      return;
    }
    hist[kSub + threadIdx.x] = static_cast<uint32_t>(scan(mine));
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kPer; ++j)
      if (static_cast<int>(threadIdx.x) + j * kThreads < m)
        list[hist[kSub + ((most - static_cast<uint32_t>(key[j] >> 32)) >> shift)] + at[j]] = key[j];
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kPer; ++j)
      if (static_cast<int>(threadIdx.x) + j * kThreads < m) {
        const uint32_t part = (most - static_cast<uint32_t>(key[j] >> 32)) >> shift;
        const uint32_t from = hist[kSub + part], many = hist[part];
        uint32_t to = from;
        for (uint32_t i = 0; i < many; ++i) to += list[from + i] > key[j];
        list2[to] = key[j];
      }
    __syncthreads();
  }
};

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
  __device__ __forceinline__ uint64_t needed(uint64_t sum) const {  // of a sum of weights
    bool more;
    if (!(top_p < 1.0f)) return sum;
    const uint64_t n = times_fraction(sum, top_p, &more);
    return max(n + more, static_cast<uint64_t>(1));
  }
};

// The rest of a row by one CTA, from the m tokens that lead its ranking (their rank keys in
// r.list2, in any order).  `sum`: of all weights, for top_p without top_k.
template <int DT, bool HELD>
__device__ __forceinline__ void finish_list(const Row<DT, HELD>& r, const Asked& ask, int m, uint64_t sum,
                                            int64_t* token, float* logprob) {
  const Weights& wt = r.wt;
  const int k = ask.k ? min(m, ask.k) : m;
  uint64_t *keys = r.list2, *spare = r.list;
  if (m <= 64) {
    // Eight threads per token: ranks and sums by comparing with every other.
    const int t = threadIdx.x >> 3, part = threadIdx.x & 7;
    const bool in = t < m;
    const uint64_t key = in ? keys[t] : 0ull;
    const float v = value_of_key(key);
    const uint64_t w = in ? r.weight(v) : 0ull;
    if (in && part == 0) spare[t] = w;
    __syncthreads();
    const auto add8 = [](uint64_t v) {
#pragma unroll
      for (int o = 1; o < 8; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
      return v;
    };
    uint64_t before = 0, ahead = 0;
    for (int j = part; j < m; j += 8)
      if (keys[j] > key) {
        ++ahead;
        before += spare[j];
      }
    before = add8(before);
    const int rank = static_cast<int>(add8(ahead));
    if (ask.k) {  // the sum of the first k: every eight threads add it up for themselves
      if (in && part == 0) r.hist[t] = static_cast<uint32_t>(rank);
      __syncthreads();
      sum = 0;
      for (int j = part; j < m; j += 8)
        if (static_cast<int>(r.hist[j]) < k) sum += spare[j];
      sum = add8(sum);
    }
    const bool stays = in && rank < k && before < ask.needed(sum) && (w >= ask.w_min || rank == 0);
    __syncthreads();
    if (in && part == 0) spare[t] = stays ? w : 0ull;
    __syncthreads();
    const uint32_t at = static_cast<uint32_t>(key);  // ~index
    uint64_t whole = 0;
    before = 0;
    for (int j = part; j < m; j += 8) {
      whole += spare[j];
      if (static_cast<uint32_t>(keys[j]) > at) before += spare[j];
    }
    whole = add8(whole);
    before = add8(before);
    const uint64_t target = times_fraction(whole, ask.u);
    if (stays && part == 0 && target >= before && target < before + w) {
      *token = static_cast<int>(~at);
      if (logprob) *logprob = log_share(wt, v, w, whole);
    }
    return;
  }
  r.sort(m);
  uint64_t w[kPer], here = 0;
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int i = kPer * threadIdx.x + j;
    w[j] = i < k ? r.weight(value_of_key(keys[i])) : 0ull;
    here += w[j];
  }
  uint64_t all;
  uint64_t before = r.scan(here, &all);
  const uint64_t need = ask.needed(ask.k ? all : sum);
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
  // by index: sorted again, on (~index, order of the value, or 0 where the token does not stay)
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int i = kPer * threadIdx.x + j;
    if (i < m) keys[i] = (keys[i] << 32) | (w[j] ? keys[i] >> 32 : 0ull);
  }
  __syncthreads();
  r.sort(m);
  here = 0;
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int i = kPer * threadIdx.x + j;
    w[j] = i < m && static_cast<uint32_t>(keys[i]) ? r.weight(value_of_key(keys[i] << 32)) : 0ull;
    here += w[j];
  }
  before = r.scan(here);
  const uint64_t target = times_fraction(whole, ask.u);
  if (target < before || target >= before + here) return;
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    if (target >= before && target < before + w[j]) {
      const uint64_t key = keys[kPer * threadIdx.x + j];
      *token = static_cast<int>(~static_cast<uint32_t>(key >> 32));
      if (logprob) *logprob = log_share(wt, value_of_key(key << 32), w[j], whole);
    }
    before += w[j];
  }
}

template <int DT, bool HELD>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(moe_sampling_t a, int C, int per, uint32_t slice_bytes) {
  using T = typename Stored<DT>::T;
  using R = Row<DT, HELD>;
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
  constexpr int kVec = R::kVec;
  const int first = min(a.V, rank * per), n = min(a.V, first + per) - first;
  const T* g = static_cast<const T*>(a.logits) + row * a.logits_stride + first;
  const int off = static_cast<int>((reinterpret_cast<uintptr_t>(g) & 15u) / sizeof(T));
  const int chunks = n ? (off + n + kVec - 1) / kVec : 0;
  T* s = reinterpret_cast<T*>(smem);
  float mine = kNegInf;  // this thread's largest, and the first of its whole chunks that has it
  int where = -1;
  float mine_edge = kNegInf;  // and its place in the first or last chunk, where these are not whole
  int i_edge = 0;
  {
    // whole chunks; in global memory the first and last are edges whether whole or not
    const int c_lo = HELD ? (off ? 1 : 0) : 1, c_hi = HELD ? (off + n) / kVec : chunks - 1;
    constexpr int kAhead = 4;
    for (int c0 = c_lo + threadIdx.x; c0 < c_hi; c0 += kThreads * kAhead) {
      uint4 v[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u)
        if (c0 + u * kThreads < c_hi) v[u] = ld_ordered16(g - off + (c0 + u * kThreads) * kVec);
#pragma unroll
      for (int u = 0; u < kAhead; ++u)
        if (c0 + u * kThreads < c_hi) {
          float f[kVec];
          if constexpr (HELD) *reinterpret_cast<uint4*>(s + (c0 + u * kThreads) * kVec) = v[u];
          R::unpack(v[u], f);
          float m = f[0];
#pragma unroll
          for (int j = 1; j < kVec; ++j) m = fmaxf(m, f[j]);
          if (m > mine) {
            mine = m;
            where = c0 + u * kThreads;
          }
        }
    }
    // the first and last chunk: 2 * kVec places
    if (threadIdx.x < 2 * kVec && chunks) {
      const int e = threadIdx.x >= kVec, c = e ? chunks - 1 : 0, i = c * kVec + (threadIdx.x & (kVec - 1));
      if (!(c >= c_lo && c < c_hi)) {  // (one chunk alone is written twice, alike)
        const bool own = i >= off && i < off + n;
        T raw;
        float f = kNegInf;
        if constexpr (DT == MOE_F32) raw = kNegInf;
        else raw = DT == MOE_BF16 ? 0xff80u : 0xfc00u;
        if (own) {
          raw = g[i - off];
          f = value<DT>(raw);
        }
        if constexpr (HELD) s[i] = raw;
        else reinterpret_cast<T*>(&sh.edge[e])[threadIdx.x & (kVec - 1)] = raw;
        if (!e || chunks > 1) {  // (of one chunk alone each token is one thread's)
          mine_edge = f;
          i_edge = i;
        }
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
  if (greedy || min_p > 1.0f || ask.top_p <= 0.0f || a.V == 1) k = 1;
  else if (k <= 0 || k >= a.V) k = 0;
  const bool by_k = k > 0, by_p = ask.top_p < 1.0f;
  ask.k = k;

  // ------------------------------------------- the largest, and what some threads' largest reach
  __syncthreads();
  const float mine_whole = mine;
  mine = fmaxf(mine, mine_edge);
  float best = mine;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) best = fmaxf(best, __shfl_xor_sync(0xffffffffu, best, o));
  if (lane == 0) sh.warp[warp] = __float_as_uint(best);
  const int ctas = (a.V - 1) / per + 1;  // that have tokens
  const int share = (k - 1) / ctas + 1;
  const bool few = k > 1 && 3 * share <= kThreads && 2 * k <= kList;
  uint32_t reach = 0;
  if (few) {  // to 18 bits of the key, at most
    const uint32_t key = order_key(mine + 0.0f);
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

  uint8_t* behind = smem + slice_bytes;
  R r{sh, HELD ? reinterpret_cast<const uint4*>(smem) : reinterpret_cast<const uint4*>(g - off),
      reinterpret_cast<uint32_t*>(behind), reinterpret_cast<uint64_t*>(behind + kHistBytes),
      reinterpret_cast<uint64_t*>(behind + kHistBytes + kListBytes), C, rank, first - off, off, n, chunks,
      (chunks + kWarps - 1) / kWarps, 0};
  r.wt.init(greedy || !(ask.temperature == ask.temperature) ? 1.0f : ask.temperature, best);

  if (k == 1) {  // rank 0: the first of the largest
    int i = INT32_MAX;
    if (mine_whole == best) {
      float v[kVec];
      R::unpack(r.chunk(where), v);
#pragma unroll
      for (int j = kVec - 1; j >= 0; --j)
        if (v[j] == best) i = where * kVec + j;
    }
    if (mine_edge == best) i = min(i, i_edge);
    i = __reduce_min_sync(0xffffffffu, i);
    __syncthreads();
    if (lane == 0) sh.warp[warp] = static_cast<uint64_t>(i);
    __syncthreads();
    if (warp == 0) {
      i = __reduce_min_sync(0xffffffffu, lane < kWarps ? static_cast<int>(sh.warp[lane]) : INT32_MAX);
      if (lane == 0) st_peer64(&sh.cta[0][rank], 0, i == INT32_MAX ? ~0ull : static_cast<uint64_t>(r.first + i));
    }
    r.sync_row();
    if (rank == 0 && threadIdx.x == 0) {
      uint64_t least = ~0ull;
      for (int c = 0; c < C; ++c) least = min(least, sh.cta[0][c]);
      *token = static_cast<int64_t>(least);
      if (logprob) *logprob = 0.0f;
    }
    return;
  }
  ask.w_min = 0;  // weights below it do not stay
  if (min_p > 0.0f) {
    bool more;
    const uint64_t w = r.weight(best);
    ask.w_min = min_p >= 1.0f ? w : times_fraction(w, min_p, &more) + more;
  }

  // ------------------------------------------------------------ the filters
  uint64_t cut = 0;  // smallest rank key that stays
  float v_cut = kNegInf;
  const auto stays = [&](float v, int i) { return v > v_cut || (v == v_cut && R::key_of(v, r.first + i) >= cut); };
  const auto any = [](float, int) { return true; };
  const auto lost = [&] {  // (a border that was not found: no token, the same in every CTA)
    if (rank == 0 && threadIdx.x == 0) {
      *token = -1;
      if (logprob) *logprob = NAN;
    }
  };
  const auto set_cut = [&](uint64_t key) {
    cut = key;
    v_cut = value_of_key(key);
  };
  const auto kept = [&](float v, int i) {
    const uint64_t w = r.weight(v);
    return w >= ask.w_min && stays(v, i) ? w : static_cast<uint64_t>(0);
  };
  const auto write = [&](float v, int i, uint64_t all) {
    *token = r.first + i;
    if (logprob) *logprob = log_share(r.wt, v, r.weight(v), all);
  };
  uint64_t known = 0;  // this thread's weights above v_known, which all stay
  float v_known = INFINITY;
  if (by_k || by_p) {
    int m = -1, b1;
    uint64_t sum = 0, tokens;
    uint32_t klo, khi;
    if (few) {
      m = r.template gather<false>(reach > 0x007fffffu ? value_of_order(reach) : kNegInf, sum);
    } else if (a.V <= kList) {  // all that have weight
      const float least = r.least_of(kUsedBins);
      m = by_p && !by_k ? r.template gather<true>(least, sum) : r.template gather<false>(least, sum);
    }
    if (m < 0) {
      r.template find_bins<true>(any, by_k, k, ask.top_p, klo, khi, b1, tokens);
      if (tokens <= kList) {
        const float least = r.least_of(b1);
        m = by_k ? r.template gather<false>(least, sum) : r.template gather<true>(least, sum);
      }
    }
    if (m >= 0) {  // the first CTA does the rest
      if (rank != 0) return;
      r.close_list(m);
      finish_list<DT, HELD>(r, ask, m, sum, token, logprob);
      return;
    }
    if (by_k && b1 < kUsedBins) {
      // what lies above the window is counted, its tokens are brought and sorted
      const float v_lo = value_of_order(klo), v_hi = value_of_order(khi);
      r.begin_list();
      uint64_t above = 0;
      r.chunks_of([&](const float (&v)[R::kVec], int i) {
        bool near = false;
#pragma unroll
        for (int j = 0; j < R::kVec; ++j) {
          above += v[j] > v_hi;
          near |= v[j] >= v_lo && v[j] <= v_hi;
        }
        if (near) r.bring_some(v, i, v_lo, v_hi);
      });
      above = r.total(above);
      m = r.end_list();
      if (m >= 0) {
        r.turn ^= 1;
        if (rank == 0) {
          r.close_list(m);
          r.sort(m);
          if (threadIdx.x == 0) {
            const uint64_t at = static_cast<uint64_t>(k) - above - 1;  // (past the end: wraps, is not below m)
            sh.finds[0] = at < static_cast<uint64_t>(m) ? r.list2[at] : 0ull;
          }
        }
        r.tell(1);
        set_cut(sh.said[r.turn][0]);
      }
      if (m < 0 || cut == 0)
        set_cut(r.select(klo, khi, above, any, [](float) { return static_cast<uint64_t>(1); }, k));
      if (cut == 0) return lost();
    }
    if (by_p) {
      if (by_k) {
        r.template find_bins<false>(stays, false, 0, ask.top_p, klo, khi, b1, tokens);
        khi = max(khi, order_key(v_cut));  // (so that all above the window stay)
      }
      // the same with weights; what stays above the window is kept by warp as well
      const float v_lo = value_of_order(klo), v_hi = value_of_order(khi);
      uint64_t high = 0, low = 0;  // low: all
      const int i_cut = cut ? static_cast<int>(~static_cast<uint32_t>(cut)) - r.first : INT32_MAX;
      r.begin_list();
      if (cut == 0) {  // (every weight is computed, whatever becomes of it: no branches in between)
        r.chunks_of([&](const float (&v)[R::kVec], int i) {
          bool near = false;
#pragma unroll
          for (int j = 0; j < R::kVec; ++j) {
            uint32_t m, f;
            r.wt.parts(v[j], sh.root, m, f);
            low += static_cast<uint64_t>(m) * f;
            high += static_cast<uint64_t>(v[j] > v_hi ? m : 0u) * f;
            near |= v[j] >= v_lo && v[j] <= v_hi;
          }
          if (near) r.bring_some(v, i, v_lo, v_hi);
        });
      } else {
        r.chunks_of([&](const float (&v)[R::kVec], int i) {
          bool near = false;
#pragma unroll
          for (int j = 0; j < R::kVec; ++j) {
            const bool in = v[j] > v_cut || (v[j] == v_cut && i + j <= i_cut);
            uint32_t m, f;
            r.wt.parts(v[j], sh.root, m, f);
            low += static_cast<uint64_t>(in ? m : 0u) * f;
            high += static_cast<uint64_t>(v[j] > v_hi ? m : 0u) * f;  // (above the window all stay)
            near |= in && v[j] >= v_lo && v[j] <= v_hi;
          }
          if (near) r.bring_some(v, i, fmaxf(v_lo, v_cut), v_hi, v_cut, i_cut);
        });
      }
      const uint64_t stay = warp_sum64(high);
      uint64_t above = high;
      sum = r.total2(low, above);
      if (lane == 0) st_peer64(&sh.region[rank * kWarps + warp], 0, stay);
      m = r.end_list();
      const uint64_t need = ask.needed(sum);
      if (m >= 0) {
        uint64_t* said = sh.said[r.turn ^ 1];
        if (rank == 0) {
          r.close_list(m);
          r.sort(m);
          uint64_t w[kPer], here = 0, all, keep = 0;
#pragma unroll
          for (int j = 0; j < kPer; ++j) {
            const int i = kPer * threadIdx.x + j;
            w[j] = i < m ? r.weight(value_of_key(r.list2[i])) : 0ull;
            here += w[j];
          }
          uint64_t before = above + r.scan(here, &all);
          const bool inside = above < need && above + all >= need;
          if (threadIdx.x == 0) sh.finds[0] = 0;
          r.clear_hist();
#pragma unroll
          for (int j = 0; j < kPer; ++j) {
            const int i = kPer * threadIdx.x + j;
            if (inside && i < m && before < need) {
              const uint64_t key = r.list2[i];
              if (w[j] && before + w[j] >= need) sh.finds[0] = key;
              {  // to the sum of the warp that has it
                const int at = static_cast<int>(~static_cast<uint32_t>(key)), c = at / per;
                const int o = static_cast<int>((reinterpret_cast<uintptr_t>(g) / sizeof(T) + c * per) % kVec);
                const int its = min(a.V, (c + 1) * per) - c * per;
                const int pw = ((o + its + kVec - 1) / kVec + kWarps - 1) / kWarps;
                const int of = kWords * (c * kWarps + (at - c * per + o) / kVec / pw);  // in words, as no
#pragma unroll
                for (int u = 0; u < kWords; ++u) atomicAdd(&r.hist[of + u], word_of(w[j], u));  // 64-bit sums are made there
              }
            }
            before += w[j];
          }
          __syncthreads();
          // the warp that has the token drawn
          const int regions = C * kWarps;
          if (static_cast<int>(threadIdx.x) < regions) {
            keep = sh.region[threadIdx.x];
#pragma unroll
            for (int u = 0; u < kWords; ++u) keep += of_word(r.hist[kWords * threadIdx.x + u], u);
          }
          const uint64_t from = r.scan(keep, &all);
          const uint64_t target = times_fraction(all, ask.u);
          if (target >= from && target < from + keep) {
            sh.finds[1] = threadIdx.x;
            sh.finds[2] = target - from;
          }
          if (threadIdx.x == 0) sh.finds[3] = all;
        }
        r.turn ^= 1;
        r.tell(4);
        if (said[0]) set_cut(said[0]);
        if (said[0] && ask.w_min == 0) {
          const int region = static_cast<int>(said[1]);
          if (region / kWarps != rank) return;
          const uint64_t all = said[3];
          r.locate_in(region % kWarps, kept, said[2], [&](float v, int i) { write(v, i, all); });
          return;
        }
      }
      if (m < 0 || sh.said[r.turn][0] == 0) {
        set_cut(r.select(klo, khi, above, stays, [&](float v) { return r.weight(v); }, need));
        if (cut == 0) return lost();
        if (v_cut <= v_hi) {  // all above the window stay, and were added up
          known = high;
          v_known = v_hi;
        }
      }
    }
  }

  // --------------------------------------------------------------- the draw
  uint64_t all = 0;
  if (ask.w_min == 0 && v_known < INFINITY) {
    all = known;
    r.each([&](float v, int i) {
      if (v <= v_known && v >= v_cut) all += kept(v, i);
    });
  } else if (cut != 0) {
    r.each([&](float v, int i) { all += kept(v, i); });
  } else if (ask.w_min != 0) {
    r.each([&](float v, int) {
      const uint64_t w = r.weight(v);
      all += w >= ask.w_min ? w : 0ull;
    });
  } else {
    r.each([&](float v, int) { all = r.wt.add(all, v, sh.root); });
  }
  all = r.total(all);
  r.locate(kept, times_fraction(all, ask.u), [&](float v, int i) { write(v, i, all); });
}

template <int DT, bool HELD>
moe_status_t launch_as(const moe_sampling_t& a, int C, int per, cudaStream_t st) {
  const uint32_t slice_bytes = HELD ? static_cast<uint32_t>(per * sizeof(typename Stored<DT>::T)) + 32u : 0u;
  const size_t smem = slice_bytes + kHistBytes + 2 * kListBytes;
  if (raise_smem_limit(sample_kernel<DT, HELD>, smem) != cudaSuccess) return check_launch("sample_kernel (smem)");
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
  if (cudaLaunchKernelEx(&cfg, sample_kernel<DT, HELD>, a, C, per, slice_bytes) != cudaSuccess)
    return check_launch("sample_kernel");
  stat_kernels(1);
  return MOE_OK;
}

template <int DT>
moe_status_t launch(const moe_sampling_t& a, cudaStream_t st) {
  const auto slice = [&](int C) { return ((a.V - 1) / C + 1 + kThreads - 1) / kThreads * kThreads; };
  // A row's CTAs, of slices that are worth it: about the two that an SM holds of every SM, or, of long
  // slices, half as many again, as rows that ask for different things end at different times (64
  // mixed rows of 151936 take 87 us by 4 CTAs, 67 by 8; 64 of 32000 take 26 by 4, 34 by 8).
  int C = 1;
  while (C < kMaxCtas && slice(C) > 2048 &&
         static_cast<int64_t>(a.B) * C * 10 <= (slice(C) > 32768 ? 17 : 10) * sm_count())
    C *= 2;
  const int per = slice(C);
  // Held in shared memory where two CTAs still fit an SM, or one where there are no more CTAs.
  constexpr int size = sizeof(typename Stored<DT>::T);
  const int64_t held = static_cast<int64_t>(per) * size, fits = a.B * static_cast<int64_t>(C) <= sm_count() ? 200000 : 90000;
  return held <= fits ? launch_as<DT, true>(a, C, per, st) : launch_as<DT, false>(a, C, per, st);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" moe_status_t moe_sample(const moe_sampling_t* s, void* stream) {
  if (!s) return set_error(MOE_ERR_INVALID_ARG, "moe_sampling_t is NULL");
  if (s->B < 0 || s->V < 1) return set_error(MOE_ERR_INVALID_ARG, "B must be >= 0 and V >= 1");
  if (s->V > kMaxLogits) return set_error(MOE_ERR_UNSUPPORTED, "V must be at most %d", kMaxLogits);
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
