// moe_sample.cu — a token from each row of logits: temperature, top-k, top-p,
// min-p and one given random number per row.
//
// A cluster of CTAs holds a row in shared memory (read from HBM once).  Weights
// exp((l - max) / T) are fixed-point numbers of 45 bits at most, so that every sum
// of them is exact and does not depend on the order of its terms; whichever threads
// hold a row, the same token comes out.  Every filter keeps a prefix of the ranking
// by (l descending, index ascending), so the kept set is one bound on the 64-bit
// rank key (order of l, ~index), found by bisection with sums over the cluster.

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
  __device__ __forceinline__ uint64_t of(float l, const uint32_t* root) const {
    if (infinite) return l == INFINITY ? 1ull << 44 : 0ull;
    float e;
    const int n = split(l, e);
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

// The sums of a row's cluster and where they lie.
struct Shared {
  uint64_t warp[kWarps];       // this CTA's sums by warp, of the last reduction
  uint64_t cta[2][kMaxCtas];   // every CTA's, two reductions in turn
  uint64_t found[2];           // an index found by one CTA
  float largest[kMaxCtas];
  uint32_t root[32];
};

template <int DT>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(moe_sampling_t a, int C, int per) {
  using T = typename Stored<DT>::T;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ Shared sh;
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rank = static_cast<int>(blockIdx.x % C);
  const int64_t row = blockIdx.x / C;
  if (threadIdx.x < 32) sh.root[threadIdx.x] = c_root[threadIdx.x];
  pdl_wait();

  // ---------------------------------------------------------------- the slice
  const int first = min(a.V, rank * per), n = min(a.V, first + per) - first;
  const T* g = static_cast<const T*>(a.logits) + row * a.logits_stride + first;
  constexpr int kVec = 16 / sizeof(T);
  const int off = static_cast<int>((reinterpret_cast<uintptr_t>(g) & 15u) / sizeof(T));
  T* s = reinterpret_cast<T*>(smem) + off;  // element i: where its 16-byte chunk is one in memory too
  float best = kNegInf;
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
              best = fmaxf(best, __uint_as_float(w[j]));
            } else {
              const float2 f = unpack2<DT>(w[j]);
              best = fmaxf(best, fmaxf(f.x, f.y));
            }
          }
        }
    }
    const int ends = n - chunks * kVec;  // elements before and behind the chunks
    if (static_cast<int>(threadIdx.x) < ends) {
      const int i = static_cast<int>(threadIdx.x) < head ? threadIdx.x : chunks * kVec + threadIdx.x;
      const T v = g[i];
      s[i] = v;
      best = fmaxf(best, value<DT>(v));
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) best = fmaxf(best, __shfl_xor_sync(0xffffffffu, best, o));
  if (lane == 0) sh.warp[warp] = __float_as_uint(best);
  __syncthreads();
  if (warp == 0) {
    best = lane < kWarps ? __uint_as_float(static_cast<uint32_t>(sh.warp[lane])) : kNegInf;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) best = fmaxf(best, __shfl_xor_sync(0xffffffffu, best, o));
    if (C > 1) cluster_sync_all();  // every CTA of the cluster runs
    if (lane < C)
      asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(peer_addr(smem_u32(&sh.largest[rank]), lane)), "f"(best)
                   : "memory");
  } else if (C > 1) {
    cluster_sync_all();
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
  const float temperature = a.temperature ? a.temperature[row] : 1.0f;
  int k = a.top_k ? a.top_k[row] : 0;
  float top_p = a.top_p ? a.top_p[row] : 1.0f;
  const float min_p = a.min_p ? a.min_p[row] : 0.0f;
  float u = a.uniforms[row];
  u = u > 0.0f ? fminf(u, 0.99999994f) : 0.0f;
  const bool greedy = temperature <= 0.0f;
  if (greedy || min_p > 1.0f || top_p <= 0.0f) k = 1;
  if (k <= 0 || k > a.V) k = a.V;
  Weights wt;
  wt.init(greedy || !(temperature == temperature) ? 1.0f : temperature, best);
  const uint64_t w_best = wt.of(best, sh.root);
  bool more;
  uint64_t w_min = 0;  // weights below it do not stay
  if (min_p > 0.0f) w_min = min_p >= 1.0f ? w_best : times_fraction(w_best, min_p, &more) + more;

  // ------------------------------------------------------ sums over the row
  const int chunk = per / kWarps;  // of a warp, a multiple of 32
  const int lo = min(n, warp * chunk), hi = min(n, lo + chunk);
  int turn = 0;
  // the sum of f(value, index) over the row, by warp and CTA in sh
  const auto sum = [&](auto f) {
    uint64_t v = 0;
    for (int i = lo + lane; i < hi; i += 32) v += f(value<DT>(s[i]), first + i);
    v = warp_sum64(v);
    turn ^= 1;
    __syncthreads();  // sh.warp may still be read
    if (lane == 0) sh.warp[warp] = v;
    __syncthreads();
    if (warp == 0) {
      const uint64_t all = warp_sum64(lane < kWarps ? sh.warp[lane] : 0ull);
      if (lane < C) st_peer64(&sh.cta[turn][rank], lane, all);
    }
    if (C > 1) cluster_sync_all();
    else __syncthreads();
    uint64_t total = 0;
    for (int r = 0; r < C; ++r) total += sh.cta[turn][r];
    return total;
  };
  // after sum(f): calls hit(i) in the one lane that holds the first index i up to and with
  // which f sums to more than `target`
  const auto locate = [&](auto f, uint64_t target, auto hit) {
    for (int r = 0; r < rank; ++r) {
      if (target < sh.cta[turn][r]) return;
      target -= sh.cta[turn][r];
    }
    if (target >= sh.cta[turn][rank]) return;
    for (int w = 0; w < warp; ++w) {
      if (target < sh.warp[w]) return;
      target -= sh.warp[w];
    }
    if (target >= sh.warp[warp]) return;
    for (int i0 = lo; i0 < hi; i0 += 32) {
      const int i = i0 + lane;
      uint64_t v = i < hi ? f(value<DT>(s[i]), first + i) : 0ull;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint64_t p = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += p;
      }
      const uint32_t over = __ballot_sync(0xffffffffu, v > target);
      if (over) {
        if (lane == __ffs(over) - 1) hit(first + i);
        return;
      }
      target -= __shfl_sync(0xffffffffu, v, 31);
    }
  };
  const auto locate_all = [&](auto f, uint64_t target) {  // the index, in every CTA
    locate(f, target, [&](int i) {
      for (int r = 0; r < C; ++r) st_peer64(&sh.found[turn], r, static_cast<uint64_t>(i));
    });
    if (C > 1) cluster_sync_all();
    else __syncthreads();
    return static_cast<int>(sh.found[turn]);
  };
  const auto rank_key_of = [](float v, int i) {
    return (static_cast<uint64_t>(order_key(v)) << 32) | static_cast<uint32_t>(~i);
  };

  // ------------------------------------------------------------ the filters
  uint64_t cut = 0;  // smallest rank key that stays
  if (k < a.V) {
    uint32_t key = 0;
    for (int bit = 31; bit >= 0; --bit) {
      const uint32_t mid = key | (1u << bit);
      if (sum([&](float v, int) { return static_cast<uint64_t>(order_key(v) >= mid); }) >= static_cast<uint64_t>(k))
        key = mid;
    }
    const uint64_t above = sum([&](float v, int) { return static_cast<uint64_t>(order_key(v) > key); });
    const auto tie = [&](float v, int) { return static_cast<uint64_t>(order_key(v) == key); };
    sum(tie);
    const int i = locate_all(tie, static_cast<uint64_t>(k) - above - 1);
    cut = (static_cast<uint64_t>(key) << 32) | static_cast<uint32_t>(~i);
  }
  if (top_p < 1.0f && k > 1) {
    const uint64_t old = cut;
    const auto stays = [&](float v, int i) { return rank_key_of(v, i) >= old; };
    const uint64_t all = sum([&](float v, int i) { return stays(v, i) ? wt.of(v, sh.root) : 0ull; });
    uint64_t need = times_fraction(all, top_p, &more);
    need = max(need + more, static_cast<uint64_t>(1));
    uint32_t key = 0;
    for (int bit = 31; bit >= 0; --bit) {
      const uint32_t mid = key | (1u << bit);
      if (sum([&](float v, int i) { return order_key(v) >= mid && stays(v, i) ? wt.of(v, sh.root) : 0ull; }) >= need)
        key = mid;
    }
    const uint64_t above =
        sum([&](float v, int i) { return order_key(v) > key && stays(v, i) ? wt.of(v, sh.root) : 0ull; });
    const auto tie = [&](float v, int i) { return order_key(v) == key && stays(v, i) ? wt.of(v, sh.root) : 0ull; };
    sum(tie);
    const int i = locate_all(tie, need - above - 1);
    cut = (static_cast<uint64_t>(key) << 32) | static_cast<uint32_t>(~i);
  }

  // --------------------------------------------------------------- the draw
  const auto kept = [&](float v, int i) {
    const uint64_t w = wt.of(v, sh.root);
    return rank_key_of(v, i) >= cut && w >= w_min ? w : 0ull;
  };
  const uint64_t all = sum(kept);
  locate(kept, times_fraction(all, u), [&](int i) {
    a.tokens[row] = i;
    if (a.logprobs) {
      const float v = value<DT>(s[i - first]);
      const uint64_t w = wt.of(v, sh.root);
      float lp;
      if (w >= all - w) {  // at least half: from what is missing
        lp = log1pf(-(static_cast<float>(all - w) / static_cast<float>(all)));
      } else {
        // ln(w / all) by octaves: w = 2^(n / 32 + e / 32 + 44 - top), all = 2^t m
        float e;
        const int nn = wt.infinite ? wt.top * 32 : wt.split(v, e);
        if (wt.infinite) e = 0.0f;
        const int t = 63 - __clzll(static_cast<long long>(all));
        const float m = static_cast<float>(all << (63 - t)) * 0x1p-63f;  // [1, 2]
        const int octaves = (nn >> 5) - wt.top + 44 - t;
        lp = fmaf(static_cast<float>(octaves * 32 + (nn & 31)) + e, 0.02166084939249829f, -logf(m));
      }
      a.logprobs[row] = lp;
    }
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
  const size_t smem = (static_cast<size_t>(per) * sizeof(typename Stored<DT>::T)) + 16;
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
  if (cudaLaunchKernelEx(&cfg, sample_kernel<DT>, a, C, per) != cudaSuccess) return check_launch("sample_kernel");
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
