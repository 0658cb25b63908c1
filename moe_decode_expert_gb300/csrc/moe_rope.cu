// moe_rope.cu — rotation of new queries and keys, and append of keys and
// values to a paged cache, with the optional per-head RMS norm before it.
//
// A (token, head) item — query, key or value head — takes 8, 16 or 32
// neighbouring lanes, one 16-byte chunk of 8 elements each: one wide load, the
// norm's sum by shuffles within the item, the partner half of the rotation by
// a shuffle, one wide store (8 bytes to an e4m3 cache).  Every element is read
// and written once.
//
// Angles.  a = pos * f.  f / 2pi is formed as a 64-bit binary fraction of a
// turn (the 24-bit mantissa of f times the leading 64 bits of 1 / 2pi, shifted
// by its exponent); pos times that fraction, modulo 2^64, is the angle's
// fraction of a turn with the whole turns gone exactly, and sincospif takes it
// from there.  Far positions cost no accuracy and no fp64 arithmetic: the
// fraction is off by at most |pos| * max(1, |f|) * 2^-63 turns.

#include <cuda_fp8.h>

#include "moe_common.cuh"
#include "moe_kv.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
// Tokens of a block's items times rot_dim / 2: at least 3 items per token.
constexpr int kTableMax = 1536;

struct RopeArgs {
  moe_kv_cache_t c;
  moe_rope_t r;
  Control* ctrl;
  int32_t heads;    // query + key + value heads of a token
  int64_t items;    // T * heads
  int64_t slots;    // n_pages * page_size
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

// LPH lanes per item, NI items per thread.
template <int DT, int LPH, int NI, bool F8>
__global__ void __launch_bounds__(kThreads) rope_append_kernel(RopeArgs a) {
  __shared__ float2 table[kTableMax];  // [token of the block][frequency]
  constexpr int kPer = kThreads / LPH;  // items per pass
  const int tid = threadIdx.x, lane = tid & 31, c = tid % LPH;
  const moe_rope_t& r = a.r;
  const int D = a.c.head_dim, half = r.rot_dim >> 1, hq = r.n_q_heads, hkv = a.c.n_kv_heads;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * (kPer * NI);
  const int t0 = static_cast<int>(first / a.heads);
  const int rem0 = static_cast<int>(first - static_cast<int64_t>(t0) * a.heads);
  pdl_launch_dependents();
  pdl_wait();

  uint4 raw[NI];
  int tok[NI], head[NI];
  int64_t slot[NI];
  const bool col_in = c * 8 < D;
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int k = rem0 + i * kPer + tid / LPH;
    tok[i] = k / a.heads;  // relative to t0
    head[i] = k - tok[i] * a.heads;
    raw[i] = make_uint4(0, 0, 0, 0);
    slot[i] = -1;
    if (first + i * kPer + tid / LPH < a.items) {
      const int64_t t = t0 + tok[i];
      const void* base;
      int64_t off;
      if (head[i] < hq) {
        base = r.q;
        off = t * r.q_token_stride + head[i] * r.q_head_stride;
      } else if (head[i] < hq + hkv) {
        base = r.k;
        off = t * r.k_token_stride + (head[i] - hq) * r.k_head_stride;
      } else {
        base = r.v;
        off = t * r.v_token_stride + (head[i] - hq - hkv) * r.v_head_stride;
      }
      if (col_in) raw[i] = ld_ordered16(static_cast<const uint16_t*>(base) + off + c * 8);
      if (head[i] >= hq) slot[i] = r.slots[t];
    } else {
      head[i] = -1;
    }
  }

  const int last = rem0 + kPer * NI - 1;
  int ntok = last / a.heads + 1;
  if (t0 + static_cast<int64_t>(ntok) > r.T) ntok = r.T - t0;
  for (int i = tid; i < ntok * half; i += kThreads)
    table[i] = rotation(r.positions[t0 + i / half], r.inv_freq[i % half]);
  __syncthreads();

#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const bool is_q = head[i] >= 0 && head[i] < hq, is_v = head[i] >= hq + hkv;
    float f[8];
    unpack8<DT>(raw[i], f);
    if (r.q_norm_w) {
      float ss = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) ss = fmaf(f[j], f[j], ss);
#pragma unroll
      for (int o = LPH / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      if (!is_v && head[i] >= 0 && col_in) {
        const float rstd = __frcp_rn(sqrtf(__fdiv_rn(ss, static_cast<float>(D)) + r.eps));
        float w[8];
        unpack8<DT>(ld_ordered16(static_cast<const uint16_t*>(is_q ? r.q_norm_w : r.k_norm_w) + c * 8), w);
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = f[j] * rstd * w[j];
      }
    }
    const float2* cs = table + tok[i] * half;
    if (r.interleaved) {
      if (head[i] >= 0 && !is_v) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int p = c * 4 + j;
          if (p < half) {
            const float2 t = cs[p];
            const float u = f[2 * j], v = f[2 * j + 1];
            f[2 * j] = u * t.x - v * t.y;
            f[2 * j + 1] = v * t.x + u * t.y;
          }
        }
      }
    } else if (half) {
      const int hc = half >> 3;  // chunks of a half
      const int src = (lane & ~(LPH - 1)) + (c < hc ? c + hc : c < 2 * hc ? c - hc : c);
      float g[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) g[j] = __shfl_sync(0xffffffffu, f[j], src);
      if (head[i] >= 0 && !is_v && c < 2 * hc) {
        const int p = (c < hc ? c : c - hc) * 8;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float2 t = cs[p + j];
          f[j] = c < hc ? f[j] * t.x - g[j] * t.y : f[j] * t.x + g[j] * t.y;
        }
      }
    }
    if (head[i] < 0 || !col_in) continue;
    if (is_q) {
      uint16_t* o = static_cast<uint16_t*>(r.q_out) + (t0 + static_cast<int64_t>(tok[i])) * r.out_token_stride +
                    head[i] * r.out_head_stride + c * 8;
      *reinterpret_cast<uint4*>(o) =
          make_uint4(pack2(DT, f[0], f[1]), pack2(DT, f[2], f[3]), pack2(DT, f[4], f[5]), pack2(DT, f[6], f[7]));
      continue;
    }
    const int64_t s = slot[i];
    if (s < 0) continue;
    if (s >= a.slots) {
      if (c == 0 && a.ctrl) report_error(a.ctrl, kDevBadSlot, static_cast<uint32_t>(t0 + tok[i]));
      continue;
    }
    int64_t page, off;
    if (a.slots <= 0xffffffffll) {
      page = static_cast<uint32_t>(s) / static_cast<uint32_t>(a.c.page_size);
      off = static_cast<uint32_t>(s) % static_cast<uint32_t>(a.c.page_size);
    } else {
      page = s / a.c.page_size;
      off = s % a.c.page_size;
    }
    const int hd = is_v ? head[i] - hq - hkv : head[i] - hq;
    const int64_t at = is_v ? page * a.c.v_page_stride + off * a.c.v_token_stride + hd * a.c.v_head_stride
                            : page * a.c.k_page_stride + off * a.c.k_token_stride + hd * a.c.k_head_stride;
    void* cache = is_v ? a.c.v : a.c.k;
    if constexpr (F8) {
      const float* sc = is_v ? a.c.v_scale : a.c.k_scale;
      const float s8 = sc ? sc[hd] : 1.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = __fdiv_rn(f[j], s8);
      uint32_t q[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        q[j] = __nv_cvt_float2_to_fp8x2(make_float2(f[2 * j], f[2 * j + 1]), __NV_SATFINITE, __NV_E4M3);
      *reinterpret_cast<uint2*>(static_cast<uint8_t*>(cache) + at + c * 8) =
          make_uint2(q[0] | (q[1] << 16), q[2] | (q[3] << 16));
    } else {
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(cache) + at + c * 8) =
          make_uint4(pack2(DT, f[0], f[1]), pack2(DT, f[2], f[3]), pack2(DT, f[4], f[5]), pack2(DT, f[6], f[7]));
    }
  }
}

template <int DT, int LPH, bool F8>
moe_status_t launch(const RopeArgs& a, cudaStream_t st) {
  constexpr int kPer = kThreads / LPH;
  const int64_t grid = (a.items + kPer - 1) / kPer;
  if (grid > 0x7fffffff) return set_error(MOE_ERR_UNSUPPORTED, "too many (token, head) pairs");
  if (launch_pdl(rope_append_kernel<DT, LPH, 1, F8>, dim3(static_cast<unsigned>(grid)), dim3(kThreads), 0, st, a) !=
      cudaSuccess)
    return check_launch("rope_append_kernel");
  stat_kernels(1);
  return MOE_OK;
}

template <int DT, bool F8>
moe_status_t dispatch(const RopeArgs& a, cudaStream_t st) {
  if (a.c.head_dim <= 64) return launch<DT, 8, F8>(a, st);
  if (a.c.head_dim <= 128) return launch<DT, 16, F8>(a, st);
  return launch<DT, 32, F8>(a, st);
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
  if (static_cast<int64_t>(r->n_q_heads) + 2 * static_cast<int64_t>(cache->n_kv_heads) > (1 << 20))
    return set_error(MOE_ERR_UNSUPPORTED, "too many heads");
  RopeArgs a;
  a.c = *cache;
  a.r = *r;
  a.ctrl = static_cast<Control*>(ws);
  a.heads = r->n_q_heads + 2 * cache->n_kv_heads;
  a.items = static_cast<int64_t>(r->T) * a.heads;
  a.slots = static_cast<int64_t>(cache->n_pages) * cache->page_size;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool f8 = cache->dtype == MOE_E4M3;
  if (r->dtype == MOE_BF16) return f8 ? dispatch<MOE_BF16, true>(a, st) : dispatch<MOE_BF16, false>(a, st);
  return f8 ? dispatch<MOE_F16, true>(a, st) : dispatch<MOE_F16, false>(a, st);
}
