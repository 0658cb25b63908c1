// moe_rope.cu — rotation of new queries and keys, and append of keys and
// values to a paged cache, with the optional per-head RMS norm before it.
//
// A token's heads are walked by a group of 8, 16 or 32 neighbouring lanes, one
// 16-byte chunk of 8 elements each: one wide load, the norm's sum by shuffles
// within the group, the partner half of the rotation by a shuffle, one wide store
// (8 bytes to an e4m3 cache).  Every element is read and written once.  What
// belongs to the token (its angles, cache slot) or to the column (norm weights)
// stays in registers from head to head, and the norm weights go into the
// rotation's factors: with all of it formed per head the kernel was bound by
// instructions (284 per head and warp).  8192 tokens of 20 heads of 256, a quarter
// rotated, per-head norms: 31.3 us, 79 % of the 6787 GB/s copy (57 us before), of
// which the instructions are still about 20.
//
// Angles.  a = pos * f.  f / 2pi is formed as a 64-bit binary fraction of a
// turn (the 24-bit mantissa of f times the leading 64 bits of 1 / 2pi, shifted
// by its exponent); pos times that fraction, modulo 2^64, is the angle's
// fraction of a turn with the whole turns gone exactly, and sincospif takes it
// from there.  Far positions cost no accuracy and no fp64 arithmetic: the
// fraction is off by at most |pos| * max(1, |f|) * 2^-63 turns.

#include <cuda_fp8.h>

#include <type_traits>

#include "moe_common.cuh"
#include "moe_kv.h"

namespace moe {
namespace {

constexpr int kThreads = 128;
constexpr int kTableMax = 512;   // tokens of a block times rot_dim / 2
// Heads in hand, and heads loaded ahead (8192 tokens: 1 took 38.8 us, 2 33.8, and 3
// cost registers, 38.0).
constexpr int kAhead = 2;
constexpr int kFill = 4;  // blocks per SM that fill it (777 tokens: 8 took 11.8 us, 4 7.1, 1 9.9)

struct RopeArgs {
  moe_kv_cache_t c;
  moe_rope_t r;
  Control* ctrl;
  int32_t heads;   // query + key + value heads of a token
  int32_t share;   // lane groups that share a token (a power of two)
  int32_t each;    // heads of a block's token: the block takes heads [y * each, (y + 1) * each)
  int64_t slots;   // n_pages * page_size
  FastDiv by_page;
};

// 1 / 2pi = 0.28be60db9391054a7f09... in base 16: its first 64 fraction bits.
constexpr uint64_t kInv2Pi = 0x28be60db9391054aull;

// f / 2pi modulo 1 as a 64-bit fraction.
__device__ __forceinline__ uint64_t turn_fraction(float f) {
  const uint32_t b = __float_as_uint(f);
  const int e = static_cast<int>((b >> 23) & 0xff);
  const uint64_t m = (b & 0x7fffffu) | (e ? 0x800000u : 0u);
  const int sh = 150 - (e ? e : 1);  // f = m * 2^-sh
  const uint64_t lo = m * kInv2Pi, hi = __umul64hi(m, kInv2Pi);
  uint64_t t;
  if (sh <= 0)
    t = sh > -64 ? lo << -sh : 0ull;
  else if (sh < 64)
    t = (lo >> sh) | (hi << (64 - sh));
  else
    t = sh < 128 ? hi >> (sh - 64) : 0ull;
  return (b >> 31) ? 0ull - t : t;
}

// cos and sin of pos * f.
__device__ __forceinline__ float2 rotation(int64_t pos, float f) {
  const uint64_t turn = turn_fraction(f) * static_cast<uint64_t>(pos);
  const float half_turns = static_cast<float>(static_cast<int32_t>(turn >> 32)) * 4.656612873077393e-10f;  // 2^-31
  float2 cs;
  sincospif(half_turns, &cs.y, &cs.x);
  return cs;
}

__device__ __forceinline__ uint32_t pack2(int dt, float a, float b) {
  if (dt == MOE_BF16) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
  const __half2 v = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// Blocks along the tokens when `share` of a block's groups share a token.
inline int64_t r_blocks(const RopeArgs& a, int groups, int share) {
  const int tokens = groups / share;
  return (static_cast<int64_t>(a.r.T) + tokens - 1) / tokens;
}

// LPH lanes per group.  Blocks per SM: seven, 72 registers (8192 tokens: 31.3 us,
// 35.4 with six); the e4m3 form needs more (777 tokens: 6.3 us with six, 7.4).
template <int DT, int LPH, bool F8, bool PAIRS>
__global__ void __launch_bounds__(kThreads, F8 ? 6 : 7) rope_append_kernel(RopeArgs a) {
  __shared__ float2 table[kTableMax];  // [token of the block][frequency]
  const moe_rope_t& r = a.r;
  const int tid = threadIdx.x, lane = tid & 31, c = tid % LPH;
  const int tokens = kThreads / LPH / a.share;  // of a block
  const int my_tok = tid / LPH / a.share, sub = (tid / LPH) & (a.share - 1);
  const int t0 = blockIdx.x * tokens, t = t0 + my_tok;
  const bool live = t < r.T;
  const int D = a.c.head_dim, half = r.rot_dim >> 1, hq = r.n_q_heads, hkv = a.c.n_kv_heads;
  const int h_lo = blockIdx.y * a.each, h_hi = min(a.heads, h_lo + a.each);
  const bool col_in = live && c * 8 < D;
  pdl_launch_dependents();
  pdl_wait();

  // Which of this lane's elements turn, and with which lane's elements (halves).
  const int hc = half >> 3;  // chunks of a half
  const bool turns = PAIRS ? c * 4 < half : c < 2 * hc;
  const int partner = (lane & ~(LPH - 1)) + (PAIRS || !turns ? c : c < hc ? c + hc : c - hc);
  const int pc = partner & (LPH - 1);  // that lane's chunk

  // The next heads, and their kind's norm weights (this chunk's and the
  // partner's), are loaded while the ones before are worked on; the first ones
  // before anything else is waited for.  Kinds: 0 queries, 1 keys, 2 values.
  uint4 next[kAhead], wnext[2];
  const uint16_t* src = nullptr;
  auto begin = [&](int kind) {
    const int r0 = kind == 0 ? 0 : kind == 1 ? hq : hq + hkv, r1 = kind == 0 ? hq : kind == 1 ? hq + hkv : a.heads;
    const int lo = max(r0, h_lo), hi = min(r1, h_hi);
    if (lo >= hi) return;
    const void* in = kind == 0 ? r.q : kind == 1 ? r.k : r.v;
    const int64_t ts = kind == 0 ? r.q_token_stride : kind == 1 ? r.k_token_stride : r.v_token_stride;
    const int64_t hs = kind == 0 ? r.q_head_stride : kind == 1 ? r.k_head_stride : r.v_head_stride;
    const int first = h_lo + (lo - h_lo) / a.share * a.share + sub;
    src = static_cast<const uint16_t*>(in) + t * ts + (first - r0) * hs + c * 8;
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int h = first + i * a.share;
      next[i] = make_uint4(0, 0, 0, 0);
      if (col_in && h >= lo && h < hi) next[i] = ld_ordered16(src);
      src += a.share * hs;
    }
    const uint16_t* w = static_cast<const uint16_t*>(kind == 0 ? r.q_norm_w : r.k_norm_w);
    if (kind < 2 && w && c * 8 < D) {
      wnext[0] = ld_ordered16(w + c * 8);
      wnext[1] = ld_ordered16(w + pc * 8);
    }
  };
  begin(h_lo < hq ? 0 : h_lo < hq + hkv ? 1 : 2);
  int64_t slot = -1;
  if (live) asm volatile("ld.global.s64 %0, [%1];" : "=l"(slot) : "l"(r.slots + t) : "memory");

  const int ntab = min(tokens, r.T - t0) * half;
  for (int i = tid; i < ntab; i += kThreads) table[i] = rotation(r.positions[t0 + i / half], r.inv_freq[i % half]);
  __syncthreads();

  // the token's place in the cache
  int64_t page = -1, off = 0;
  if (slot >= a.slots) {
    if (c == 0 && sub == 0 && blockIdx.y == 0) report_error(a.ctrl, kDevBadSlot, static_cast<uint32_t>(t));
  } else if (slot >= 0) {
    page = a.slots <= 0x7fffffffll ? a.by_page(static_cast<int>(slot)) : slot / a.c.page_size;
    off = slot - page * a.c.page_size;
  }
  const float inv_d = __frcp_rn(static_cast<float>(D));

  // Heads r0 .. r1 - 1 of the token's row of heads, of one kind.  All groups of a
  // warp make the same number of rounds.
  auto walk = [&](auto kind, int r0, int r1, int64_t in_hs, void* outp, int64_t at,
                  int64_t out_hs, bool store, const void* norm_w, const float* scales) {
    constexpr int kKind = decltype(kind)::value;
    constexpr bool kToF8 = F8 && kKind != 0;
    const int lo = max(r0, h_lo), hi = min(r1, h_hi);
    if (lo >= hi) return;
    const int first = h_lo + (lo - h_lo) / a.share * a.share;
    const int64_t step = a.share * in_hs, out_step = a.share * out_hs;
    int64_t to = at + (first + sub - r0) * out_hs + c * 8;
    // A turned element is (its own value times ca + its partner's times cb) *
    // 1/rms: the norm weights and the angle's sign go into the factors.
    float ca[8], cb[8];
    if constexpr (kKind != 2) {
      const bool in_d = c * 8 < D;
      float wp[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) ca[j] = wp[j] = 1.0f;
      if (norm_w && in_d) {
        unpack8<DT>(wnext[0], ca);
        unpack8<DT>(wnext[1], wp);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int p = PAIRS ? c * 4 + (j >> 1) : (c < hc ? c : c - hc) * 8 + j;
        cb[j] = 0.0f;
        if (live && turns && p < half) {
          const float2 t2 = table[my_tok * half + p];
          const bool minus = PAIRS ? (j & 1) == 0 : c < hc;
          ca[j] *= t2.x;
          cb[j] = (minus ? -t2.y : t2.y) * (PAIRS ? wp[j ^ 1] : wp[j]);
        }
      }
    }
    uint4 raw[kAhead];
    for (int hb = first; hb < hi; hb += kAhead * a.share) {
#pragma unroll
      for (int i = 0; i < kAhead; ++i) raw[i] = next[i];
      if (hb + kAhead * a.share < hi) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          const int h = hb + (kAhead + i) * a.share + sub;
          next[i] = make_uint4(0, 0, 0, 0);
          if (col_in && h < hi) next[i] = ld_ordered16(src);
          src += step;
        }
      } else if (kKind < 2) {
        begin(kKind + 1);
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i, to += out_step) {
        if (hb + i * a.share >= hi) break;  // the same for the whole warp
        const int h = hb + i * a.share + sub;
        float f[8];
        unpack8<DT>(raw[i], f);
        if constexpr (kKind != 2) {
          float rstd = 1.0f;
          if (norm_w) {
            float ss = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j) ss = fmaf(f[j], f[j], ss);
#pragma unroll
            for (int o = LPH / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            rstd = rsqrtf(fmaf(ss, inv_d, r.eps));
          }
          float g[8];
          if constexpr (PAIRS) {
#pragma unroll
            for (int j = 0; j < 8; ++j) g[j] = f[j ^ 1];
          } else if (half) {
            uint4 other;
            other.x = __shfl_sync(0xffffffffu, raw[i].x, partner);
            other.y = __shfl_sync(0xffffffffu, raw[i].y, partner);
            other.z = __shfl_sync(0xffffffffu, raw[i].z, partner);
            other.w = __shfl_sync(0xffffffffu, raw[i].w, partner);
            unpack8<DT>(other, g);
          }
#pragma unroll
          for (int j = 0; j < 8; ++j) f[j] *= ca[j];
          if (turns) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
              if (!PAIRS || c * 4 + (j >> 1) < half) f[j] = fmaf(g[j], cb[j], f[j]);
          }
#pragma unroll
          for (int j = 0; j < 8; ++j) f[j] *= rstd;
        }
        if (!col_in || !store || h < lo || h >= hi) continue;
        if constexpr (kToF8) {
          const float s8 = scales ? __frcp_rn(scales[h - r0]) : 1.0f;
          uint32_t q[4];
#pragma unroll
          for (int j = 0; j < 4; ++j)
            q[j] = __nv_cvt_float2_to_fp8x2(make_float2(f[2 * j] * s8, f[2 * j + 1] * s8),
                                            __NV_SATFINITE, __NV_E4M3);
          *reinterpret_cast<uint2*>(static_cast<uint8_t*>(outp) + to) =
              make_uint2(q[0] | (q[1] << 16), q[2] | (q[3] << 16));
        } else {
          *reinterpret_cast<uint4*>(static_cast<uint16_t*>(outp) + to) =
              kKind == 2 ? raw[i]
                         : make_uint4(pack2(DT, f[0], f[1]), pack2(DT, f[2], f[3]), pack2(DT, f[4], f[5]),
                                      pack2(DT, f[6], f[7]));
        }
      }
    }
  };
  walk(std::integral_constant<int, 0>(), 0, hq, r.q_head_stride, r.q_out,
       t * r.out_token_stride, r.out_head_stride, true, r.q_norm_w, nullptr);
  walk(std::integral_constant<int, 1>(), hq, hq + hkv, r.k_head_stride, a.c.k,
       page * a.c.k_page_stride + off * a.c.k_token_stride, a.c.k_head_stride, page >= 0, r.k_norm_w, a.c.k_scale);
  walk(std::integral_constant<int, 2>(), hq + hkv, a.heads, r.v_head_stride, a.c.v,
       page * a.c.v_page_stride + off * a.c.v_token_stride, a.c.v_head_stride, page >= 0, nullptr, a.c.v_scale);
}

template <int DT, int LPH, bool F8, bool PAIRS>
moe_status_t launch(RopeArgs a, cudaStream_t st) {
  constexpr int kGroups = kThreads / LPH;
  // Few tokens: their heads over all groups of a block and over blocks, one head
  // each.  Many: a group per token walks all its heads, as soon as that fills
  // kFill blocks per SM; between them, fewer groups share a token.
  const int64_t fill = kFill * static_cast<int64_t>(sm_count());
  a.share = kGroups;
  while (a.share > 1 && (r_blocks(a, kGroups, a.share / 2)) >= fill) a.share >>= 1;
  int rounds = (a.heads + a.share - 1) / a.share;  // heads of a group
  const int64_t bx = r_blocks(a, kGroups, a.share);
  int by = 1;
  while (by < rounds && bx * by < fill) ++by;
  rounds = (rounds + by - 1) / by;
  a.each = rounds * a.share;
  by = (a.heads + a.each - 1) / a.each;
  if (bx > 0x7fffffff || by > 65535) return set_error(MOE_ERR_UNSUPPORTED, "too many (token, head) pairs");
  if (launch_pdl(rope_append_kernel<DT, LPH, F8, PAIRS>, dim3(static_cast<unsigned>(bx), static_cast<unsigned>(by)),
                 dim3(kThreads), 0, st, a) != cudaSuccess)
    return check_launch("rope_append_kernel");
  stat_kernels(1);
  return MOE_OK;
}

template <int DT, bool F8, bool PAIRS>
moe_status_t dispatch(const RopeArgs& a, cudaStream_t st) {
  if (a.c.head_dim <= 64) return launch<DT, 8, F8, PAIRS>(a, st);
  if (a.c.head_dim <= 128) return launch<DT, 16, F8, PAIRS>(a, st);
  return launch<DT, 32, F8, PAIRS>(a, st);
}

template <int DT>
moe_status_t dispatch(const RopeArgs& a, cudaStream_t st) {
  if (a.c.dtype == MOE_E4M3) return a.r.interleaved ? dispatch<DT, true, true>(a, st) : dispatch<DT, true, false>(a, st);
  return a.r.interleaved ? dispatch<DT, false, true>(a, st) : dispatch<DT, false, false>(a, st);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" moe_status_t moe_rope_append(const moe_kv_cache_t* cache, const moe_rope_t* r, void* ws, size_t ws_bytes,
                                        void* stream) {
  if (!r) return set_error(MOE_ERR_INVALID_ARG, "moe_rope_t is NULL");
  if (moe_status_t s = check_cache(cache, r->dtype)) return s;
  if (r->T < 0 || r->n_q_heads < 1) return set_error(MOE_ERR_INVALID_ARG, "T must be >= 0 and n_q_heads >= 1");
  if (r->rot_dim < 0 || r->rot_dim > cache->head_dim || r->rot_dim % 2)
    return set_error(MOE_ERR_INVALID_ARG, "rot_dim must be even, from 0 to head_dim");
  if (!r->interleaved && r->rot_dim % 16)
    return set_error(MOE_ERR_UNSUPPORTED, "rot_dim must be a multiple of 16 unless interleaved");
  if (!(r->eps >= 0.0f)) return set_error(MOE_ERR_INVALID_ARG, "eps must be >= 0");
  if (!r->q_norm_w != !r->k_norm_w) return set_error(MOE_ERR_INVALID_ARG, "q_norm_w and k_norm_w go together");
  if (!ws || ws_bytes < sizeof(Control)) return set_error(MOE_ERR_WORKSPACE, "workspace NULL or too small");
  if (reinterpret_cast<uintptr_t>(ws) % kWsAlign)
    return set_error(MOE_ERR_WORKSPACE, "workspace must be 256-byte aligned");
  if (r->T == 0) return MOE_OK;
  if (!r->q || !r->k || !r->v || !r->q_out || !r->positions || !r->slots || (r->rot_dim && !r->inv_freq))
    return set_error(MOE_ERR_INVALID_ARG, "q / k / v / q_out / positions / slots / inv_freq is NULL");
  if (!ptr16(r->q) || !ptr16(r->k) || !ptr16(r->v) || !ptr16(r->q_out) || !ptr16(r->q_norm_w) || !ptr16(r->k_norm_w))
    return set_error(MOE_ERR_INVALID_ARG, "q, k, v, q_out and the norm weights must be 16-byte aligned");
  if ((reinterpret_cast<uintptr_t>(r->positions) | reinterpret_cast<uintptr_t>(r->slots)) & 7u ||
      reinterpret_cast<uintptr_t>(r->inv_freq) & 3u)
    return set_error(MOE_ERR_INVALID_ARG, "positions, slots or inv_freq is not aligned to its element type");
  if ((r->q_token_stride | r->q_head_stride | r->k_token_stride | r->k_head_stride | r->v_token_stride |
       r->v_head_stride | r->out_token_stride | r->out_head_stride) & 7)
    return set_error(MOE_ERR_UNSUPPORTED, "strides of q, k, v and q_out must be multiples of 16 bytes");
  if (r->T > (1 << 30)) return set_error(MOE_ERR_UNSUPPORTED, "T must be <= 2^30");
  if (static_cast<int64_t>(r->n_q_heads) + 2 * static_cast<int64_t>(cache->n_kv_heads) > (1 << 20))
    return set_error(MOE_ERR_UNSUPPORTED, "too many heads");
  RopeArgs a;
  a.c = *cache;
  a.r = *r;
  a.ctrl = static_cast<Control*>(ws);
  a.heads = r->n_q_heads + 2 * cache->n_kv_heads;
  a.slots = static_cast<int64_t>(cache->n_pages) * cache->page_size;
  a.by_page = FastDiv(cache->page_size);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  return r->dtype == MOE_BF16 ? dispatch<MOE_BF16>(a, st) : dispatch<MOE_F16>(a, st);
}
