// moe_norm.cu — RMS norm with the residual's addition, 16-bit or e4m3 output.
//
//   h = x (+ r);  r_out = rn(h);  y = h * rsqrt(mean(h^2) + eps) * w;
//   out = rn(y), or q = e4m3(y / s) with s = max(max|y|, 2^-96) / 448 per row
//   or per group of columns.
//
// One pass: a row's h values stay in registers between the reduction and the
// output, so every input is read once.  max|y| = rsqrt(..) * max|h w|, so the
// sum of squares and the row's largest magnitude come out of one reduction.
// Magnitudes are reduced as unsigned bit patterns: their order is that of the
// floats, with NaN above infinity, so a NaN reaches the row's scale.
//
// HBM bounds it: 16384 rows of 4096 with residual to e4m3 groups of 128 take 76 us,
// 91 % of the 6787 GB/s copy; 16384 x 2048 in bf16 39.5 us (100 %), 2047 43 (91 %).

#include <cuda_fp8.h>

#include "moe_common.cuh"
#include "moe_internal.h"

namespace moe {
namespace {

constexpr float kE4m3Max = 448.0f;
constexpr float kAmaxFloor = 1.26217744835361888865876570445e-29f;  // 2^-96

enum { kOutSame = 0, kOutRow = 1, kOutGroup = 2 };

__device__ __forceinline__ uint32_t pack2(int dt, float a, float b) {
  if (dt == MOE_BF16) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
  const __half2 v = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}

// Scale of a row or group from its largest |y| (kept NaN if that is NaN).
__device__ __forceinline__ float scale_of(float amax) { return (amax < kAmaxFloor ? kAmaxFloor : amax) * (1.0f / kE4m3Max); }

// 1 / s to one unit in the last place (s is at least 2^-105 here).
__device__ __forceinline__ float reciprocal(float s) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
  return r;
}

// Threads of a block at most: rows of one or two vectors per thread take
// kThreads, of four or eight 512, pairs and scalar ones 1024 (eight pairs 512).
// 256 threads leave an SM more rows in flight than 512 (16384 x 4096 e4m3: 76 us
// against 89); a warp per row needs no barrier (16384 x 512: 11.4 us against 16.9).
constexpr int kThreads = 256;
constexpr int kWarpVecs = 128;  // rows of up to this many vectors: a warp each
template <int VEC, int NV>
constexpr int kMaxThreads = VEC == 1 ? 1024 : VEC == 2 ? (NV == 8 ? 512 : 1024) : NV < 4 ? kThreads : 512;

// A row's pairs of one tensor: as 4-byte words where `like` (they lie on word
// boundaries), else as two elements each.  Branches are uniform and hold nothing
// that waits for a load: with a choice per pair, converted there, 9537 rows of 6221
// took 229 us, with single elements 136, so 103.
template <int NV>
struct Pairs {
  uint32_t lo[NV], hi[NV];
  __device__ __forceinline__ void load(const uint16_t* p, bool like, int c, int step, int H) {
    if (like) {
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        lo[v] = hi[v] = 0u;
        if (c + v * step + 1 < H) lo[v] = *reinterpret_cast<const uint32_t*>(p + c + v * step);
      }
    } else {
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        lo[v] = hi[v] = 0u;
        if (c + v * step + 1 < H) {
          lo[v] = p[c + v * step];
          hi[v] = p[c + v * step + 1];
        }
      }
    }
  }
  template <int DT>
  __device__ __forceinline__ float2 get(int v) const {
    return unpack2<DT>(lo[v] | (hi[v] << 16));
  }
};

// VEC elements (8: one 16-byte load; 2: a pair, at any alignment; 1: any
// alignment) NV times per thread.
// WARP: a warp per row; else a CTA per row.
template <int DT, int VEC, int NV, int OUT, bool WARP>
__global__ void __launch_bounds__(WARP ? 128 : kMaxThreads<VEC, NV>) norm_kernel(moe_norm_t a) {
  __shared__ float s_sum[32];
  __shared__ uint32_t s_max[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int nthr = WARP ? 32 : blockDim.x;
  const int tid = WARP ? lane : threadIdx.x;
  const int64_t row = WARP ? static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + warp : blockIdx.x;
  pdl_launch_dependents();
  pdl_wait();
  if (row >= a.T) return;
  const uint16_t* x = static_cast<const uint16_t*>(a.x) + row * a.x_stride;
  const uint16_t* r = static_cast<const uint16_t*>(a.residual) + row * a.residual_stride;
  const uint16_t* w = static_cast<const uint16_t*>(a.weight);
  uint16_t* ro = static_cast<uint16_t*>(a.residual_out) + row * a.residual_out_stride;
  const bool res = a.residual != nullptr, res_out = a.residual_out != nullptr;

  // Pairs begin where x has a word boundary: at column `early`.  What they leave,
  // column 0 or the last one, is one thread's extra element.
  const auto at = [](const void* p) { return static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p)); };
  const auto like_x = [&](const void* p) { return ((at(x) ^ at(p)) & 2u) == 0; };
  const int early = VEC == 2 ? (at(x) >> 1) & 1 : 0;
  [[maybe_unused]] const int c0 = early + 2 * tid, step = 2 * nthr;
  [[maybe_unused]] const int extra = tid == 0 && early ? 0 : tid == nthr - 1 && ((a.H - early) & 1) ? a.H - 1 : -1;
  [[maybe_unused]] float hx = 0.0f;

  float h[NV * VEC];
  [[maybe_unused]] uint4 wv[VEC == 8 ? NV : 1];  // weights stay packed
  if constexpr (VEC == 8) {
    uint4 xv[NV], rv[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = (v * nthr + tid) * 8;
      xv[v] = rv[v] = wv[v] = make_uint4(0, 0, 0, 0);
      if (c < a.H) {
        xv[v] = ld_ordered16(x + c);
        if (res) rv[v] = ld_ordered16(r + c);
        wv[v] = ld_ordered16(w + c);
      }
    }
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      float xf[8], rf[8];
      unpack8<DT>(xv[v], xf);
      unpack8<DT>(rv[v], rf);
#pragma unroll
      for (int j = 0; j < 8; ++j) h[v * 8 + j] = res ? xf[j] + rf[j] : xf[j];
    }
  } else if constexpr (VEC == 2) {
    Pairs<NV> xp, rp;
    xp.load(x, true, c0, step, a.H);
    if (res) rp.load(r, like_x(r), c0, step, a.H);
    if (extra >= 0) {
      hx = load_scalar<DT>(x, extra);
      if (res) hx += load_scalar<DT>(r, extra);
    }
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      float2 p = xp.template get<DT>(v);
      if (res) {
        const float2 q = rp.template get<DT>(v);
        p.x += q.x, p.y += q.y;
      }
      h[2 * v] = p.x, h[2 * v + 1] = p.y;
    }
  } else {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = v * nthr + tid;
      h[v] = 0.0f;
      if (c < a.H) {
        h[v] = load_scalar<DT>(x, c);
        if (res) h[v] += load_scalar<DT>(r, c);
      }
    }
  }

  float sum = 0.0f;
  uint32_t mx = 0u;
#pragma unroll
  for (int i = 0; i < NV * VEC; ++i) sum = fmaf(h[i], h[i], sum);
  if constexpr (VEC == 2) sum = fmaf(hx, hx, sum);
  [[maybe_unused]] Pairs<VEC == 2 ? NV : 1> wp;
  if constexpr (VEC == 2 && OUT == kOutRow) {
    wp.load(w, like_x(w), c0, step, a.H);
    if (extra >= 0) mx = __float_as_uint(hx * load_scalar<DT>(w, extra)) & 0x7fffffffu;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const float2 p = wp.template get<DT>(v);
      mx = max(mx, max(__float_as_uint(h[2 * v] * p.x) & 0x7fffffffu, __float_as_uint(h[2 * v + 1] * p.y) & 0x7fffffffu));
    }
  } else if (OUT == kOutRow) {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      float w8[VEC];
      if constexpr (VEC == 8) unpack8<DT>(wv[v], w8);
      else w8[0] = v * nthr + tid < a.H ? load_scalar<DT>(w, v * nthr + tid) : 0.0f;
#pragma unroll
      for (int j = 0; j < VEC; ++j) mx = max(mx, __float_as_uint(h[v * VEC + j] * w8[j]) & 0x7fffffffu);
    }
  }
  sum = warp_sum(sum);
  if (OUT == kOutRow) mx = __reduce_max_sync(0xffffffffu, mx);
  if constexpr (!WARP) {
    if (lane == 0) {
      s_sum[warp] = sum;
      s_max[warp] = mx;
    }
    __syncthreads();
    const int nw = blockDim.x >> 5;
    sum = warp_sum(lane < nw ? s_sum[lane] : 0.0f);
    if (OUT == kOutRow) mx = __reduce_max_sync(0xffffffffu, lane < nw ? s_max[lane] : 0u);
  }
  const float rstd = rsqrtf(__fdiv_rn(sum, static_cast<float>(a.H)) + a.eps);

  float inv = 1.0f;
  if (OUT == kOutRow) {
    const float s = scale_of(__uint_as_float(mx) * rstd);
    inv = reciprocal(s);
    if (tid == 0) a.scales[row] = s;
  }

  uint8_t* o8 = static_cast<uint8_t*>(a.out) + row * a.out_stride;
  uint16_t* o16 = static_cast<uint16_t*>(a.out) + row * a.out_stride;
  if constexpr (VEC == 2) {
    // A row's pairs out again, u(v) of pair v.
    const auto store = [&](uint16_t* p, auto u) {
      if (like_x(p)) {
#pragma unroll
        for (int v = 0; v < NV; ++v) {
          const float2 q = u(v);
          if (c0 + v * step + 1 < a.H) *reinterpret_cast<uint32_t*>(p + c0 + v * step) = pack2(DT, q.x, q.y);
        }
      } else {
#pragma unroll
        for (int v = 0; v < NV; ++v) {
          const float2 q = u(v);
          if (c0 + v * step + 1 < a.H) {
            store_out(p, c0 + v * step, q.x, DT);
            store_out(p, c0 + v * step + 1, q.y, DT);
          }
        }
      }
    };
    // (for 16-bit outputs the weights are loaded only now, from L1: beside x and r their
    // loads delayed those, 16384 x 2047 in single elements 133 us against 73)
    if constexpr (OUT == kOutSame) wp.load(w, like_x(w), c0, step, a.H);
    if (res_out) store(ro, [&](int v) { return make_float2(h[2 * v], h[2 * v + 1]); });
    const auto y = [&](int v) {
      const float2 p = wp.template get<DT>(v);
      return make_float2(h[2 * v] * rstd * p.x, h[2 * v + 1] * rstd * p.y);
    };
    if (extra >= 0) {
      const float ye = hx * rstd * load_scalar<DT>(w, extra);
      if (res_out) store_out(ro, extra, hx, DT);
      if (OUT == kOutSame) store_out(o16, extra, ye, DT);
      else o8[extra] = static_cast<uint8_t>(__nv_cvt_float_to_fp8(ye * inv, __NV_SATFINITE, __NV_E4M3));
    }
    if constexpr (OUT == kOutSame) {
      store(o16, y);
    } else {
      const bool even = ((at(o8) + early) & 1u) == 0;  // pairs of bytes on 2-byte boundaries
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const float2 q = y(v);
        const uint32_t two = __nv_cvt_float2_to_fp8x2(make_float2(q.x * inv, q.y * inv), __NV_SATFINITE, __NV_E4M3);
        uint8_t* o = o8 + c0 + v * step;
        if (c0 + v * step + 1 < a.H) {
          if (even) {
            *reinterpret_cast<uint16_t*>(o) = static_cast<uint16_t>(two);
          } else {
            o[0] = static_cast<uint8_t>(two);
            o[1] = static_cast<uint8_t>(two >> 8);
          }
        }
      }
    }
  } else {
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    if constexpr (VEC == 8) {
      const int c = (v * nthr + tid) * 8;
      const bool in = c < a.H;
      float y[8];
      unpack8<DT>(wv[v], y);
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] *= h[v * 8 + j] * rstd;
      if (in && res_out) {
        const float* p = h + v * 8;
        *reinterpret_cast<uint4*>(ro + c) =
            make_uint4(pack2(DT, p[0], p[1]), pack2(DT, p[2], p[3]), pack2(DT, p[4], p[5]), pack2(DT, p[6], p[7]));
      }
      if (OUT == kOutSame) {
        if (in)
          *reinterpret_cast<uint4*>(o16 + c) =
              make_uint4(pack2(DT, y[0], y[1]), pack2(DT, y[2], y[3]), pack2(DT, y[4], y[5]), pack2(DT, y[6], y[7]));
      } else {
        if (OUT == kOutGroup) {
          // group / 8 neighbouring lanes hold a group (groups start at
          // multiples of their size, and so do those lanes)
          uint32_t g = 0u;
#pragma unroll
          for (int j = 0; j < 8; ++j) g = max(g, __float_as_uint(y[j]) & 0x7fffffffu);
          for (int o = 1; o < (a.group >> 3); o <<= 1) g = max(g, __shfl_xor_sync(0xffffffffu, g, o));
          const float s = scale_of(__uint_as_float(g));
          inv = reciprocal(s);
          if (in && (c % a.group) == 0)
            a.scales[row * ((a.H + a.group - 1) / a.group) + c / a.group] = s;
        }
        if (in)
          *reinterpret_cast<uint2*>(o8 + c) = make_uint2(e4m3x4(y[0] * inv, y[1] * inv, y[2] * inv, y[3] * inv),
                                                         e4m3x4(y[4] * inv, y[5] * inv, y[6] * inv, y[7] * inv));
      }
    } else {
      const int c = v * nthr + tid;
      if (c < a.H) {
        // the weight comes from L1 again, as above
        const float y = h[v] * rstd * load_scalar<DT>(w, c);
        if (res_out) store_out(ro, c, h[v], DT);
        if (OUT == kOutSame)
          store_out(o16, c, y, DT);
        else
          o8[c] = static_cast<uint8_t>(__nv_cvt_float_to_fp8(y * inv, __NV_SATFINITE, __NV_E4M3));
      }
    }
  }
  }
}

template <int DT, int VEC, int NV, int OUT, bool WARP>
moe_status_t launch(const moe_norm_t& n, int threads, cudaStream_t st) {
  const unsigned grid = WARP ? static_cast<unsigned>((static_cast<int64_t>(n.T) + threads / 32 - 1) / (threads / 32))
                             : static_cast<unsigned>(n.T);
  if (launch_pdl(norm_kernel<DT, VEC, NV, OUT, WARP>, dim3(grid), dim3(threads), 0, st, n) != cudaSuccess)
    return check_launch("norm_kernel");
  stat_kernels(1);
  return MOE_OK;
}

template <int DT, int OUT>
moe_status_t dispatch(const moe_norm_t& n, bool wide, cudaStream_t st) {
  if (!wide) {
    if constexpr (OUT != kOutGroup) {
      // Many rows: as many elements per thread as registers allow, so that an SM holds
      // more rows at a time (16384 x 2047 with residual: 43 us with 16, 45 with 8, 68
      // with 4; 9537 x 6221: 103 with 16, 112 with 32).  Up to 512 elements a warp per
      // row (11874 x 203: 4.5 us against 12.4, 5000 x 333 3.4 against 5.4), up to 128
      // in single ones (11874 x 115: 3.5 against 4.2 in pairs).
      const bool many = n.T >= 4 * sm_count();
      if (n.H <= 4 * 32) return launch<DT, 1, 4, OUT, true>(n, 128, st);
      if (many && n.H <= 8 * 32) return launch<DT, 2, 4, OUT, true>(n, 128, st);
      if (many && n.H <= 16 * 32) return launch<DT, 2, 8, OUT, true>(n, 128, st);
      if (many && n.H <= 16 * 512)
        return launch<DT, 2, 8, OUT, false>(n, ((n.H + 15) / 16 + 31) / 32 * 32, st);
      // Few rows: few elements per thread (300 x 203: 1.9 us, 2.6 with a warp each).
      if (n.H <= 4 * 512) return launch<DT, 2, 2, OUT, false>(n, ((n.H + 3) / 4 + 31) / 32 * 32, st);
      if (n.H <= 8 * 1024) return launch<DT, 2, 4, OUT, false>(n, ((n.H + 7) / 8 + 31) / 32 * 32, st);
      return launch<DT, 1, 32, OUT, false>(n, 1024, st);
    }
  }
  const int vecs = (n.H + 7) / 8;
  if (vecs <= kWarpVecs) {
    const int nv = (vecs + 31) / 32;
    if (nv == 1) return launch<DT, 8, 1, OUT, true>(n, 128, st);
    if (nv == 2) return launch<DT, 8, 2, OUT, true>(n, 128, st);
    return launch<DT, 8, 4, OUT, true>(n, 128, st);
  }
  const int nv = vecs <= kThreads ? 1 : vecs <= 2 * kThreads ? 2 : vecs <= 4 * 512 ? 4 : 8;
  const int thr = ((vecs + nv - 1) / nv + 31) / 32 * 32;
  if (nv == 1) return launch<DT, 8, 1, OUT, false>(n, thr, st);
  if (nv == 2) return launch<DT, 8, 2, OUT, false>(n, thr, st);
  if (nv == 4) return launch<DT, 8, 4, OUT, false>(n, thr, st);
  return launch<DT, 8, 8, OUT, false>(n, thr, st);
}

// A tensor's rows by their bytes.
struct Rows {
  const void* at;
  int64_t step;   // from row to row
  int64_t bytes;  // of a row, at most step
};

// Whether a row of `a` shares a byte with a row of `b` other than (same_row: or the same as)
// its own number's.  A row is read whole before any of it is written, so in place is fine
// row by row; other rows are other CTAs'.  At different distances any overlap counts.
bool overlap(const Rows& a, const Rows& b, int32_t T, bool same_row) {
  const int64_t p = static_cast<int64_t>(reinterpret_cast<uintptr_t>(a.at));
  const int64_t q = static_cast<int64_t>(reinterpret_cast<uintptr_t>(b.at));
  const int64_t last = T - 1;
  if (p + last * a.step + a.bytes <= q || q + last * b.step + b.bytes <= p) return false;
  if (last == 0) return same_row;
  if (a.step != b.step) return true;
  // row i + k of b begins d + k * step bytes behind row i of a
  const int64_t d = q - p, s = a.step, near = -d / s;
  for (int64_t k = near - 1; k <= near + 1; ++k)
    if ((k != 0 || same_row) && k >= -last && k <= last && d + k * s < a.bytes && d + k * s + b.bytes > 0) return true;
  return false;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" moe_status_t moe_add_rmsnorm(const moe_norm_t* n, void* stream) {
  if (!n) return set_error(MOE_ERR_INVALID_ARG, "moe_norm_t is NULL");
  if (n->T < 0 || n->H < 1) return set_error(MOE_ERR_INVALID_ARG, "T must be >= 0 and H >= 1");
  if (n->H > 32768) return set_error(MOE_ERR_UNSUPPORTED, "H must be <= 32768");
  if (n->dtype != MOE_F16 && n->dtype != MOE_BF16)
    return set_error(MOE_ERR_UNSUPPORTED, "dtype must be MOE_F16 or MOE_BF16");
  if (n->out_dtype != n->dtype && n->out_dtype != MOE_E4M3)
    return set_error(MOE_ERR_UNSUPPORTED, "out_dtype must equal dtype or be MOE_E4M3");
  const bool e4m3 = n->out_dtype == MOE_E4M3;
  if (n->group != 0 && (!e4m3 || n->group < 16 || n->group > 256 || (n->group & (n->group - 1))))
    return set_error(MOE_ERR_INVALID_ARG, "group must be 0, or with MOE_E4M3 a power of two from 16 to 256");
  if (!(n->eps >= 0.0f)) return set_error(MOE_ERR_INVALID_ARG, "eps must be >= 0");
  if (!n->residual && n->residual_out) return set_error(MOE_ERR_INVALID_ARG, "residual_out given without residual");
  if (n->T == 0) return MOE_OK;
  if (!n->x || !n->weight || !n->out) return set_error(MOE_ERR_INVALID_ARG, "x / weight / out is NULL");
  if (e4m3 != (n->scales != nullptr)) return set_error(MOE_ERR_INVALID_ARG, "scales goes with MOE_E4M3, and only with it");
  if (n->x_stride < n->H || n->out_stride < n->H || (n->residual && n->residual_stride < n->H) ||
      (n->residual_out && n->residual_out_stride < n->H))
    return set_error(MOE_ERR_INVALID_ARG, "row strides must be at least H");
  const uintptr_t p16 = reinterpret_cast<uintptr_t>(n->x) | reinterpret_cast<uintptr_t>(n->residual) |
                        reinterpret_cast<uintptr_t>(n->weight) | reinterpret_cast<uintptr_t>(n->residual_out) |
                        (e4m3 ? 0 : reinterpret_cast<uintptr_t>(n->out));
  if ((p16 & 1u) || (reinterpret_cast<uintptr_t>(n->scales) & 3u))
    return set_error(MOE_ERR_INVALID_ARG, "a pointer is not aligned to its element type");
  const int64_t strides = n->x_stride | n->out_stride | (n->residual ? n->residual_stride : 0) |
                          (n->residual_out ? n->residual_out_stride : 0);
  const bool wide = n->H % 8 == 0 && (p16 & 15u) == 0 && (reinterpret_cast<uintptr_t>(n->out) & 7u) == 0 &&
                    (strides & 7) == 0;
  if (n->group && !wide)
    return set_error(MOE_ERR_UNSUPPORTED, "group scales need H %% 8 == 0 and 16-byte aligned rows");
  const int64_t width = 2ll * n->H;
  const Rows x{n->x, 2 * n->x_stride, width}, r{n->residual, 2 * n->residual_stride, width};
  const Rows o{n->out, (e4m3 ? 1 : 2) * n->out_stride, e4m3 ? n->H : width};
  const Rows ro{n->residual_out, 2 * n->residual_out_stride, width};
  if (overlap(x, o, n->T, false) || (n->residual && overlap(r, o, n->T, false)) ||
      (n->residual_out && (overlap(x, ro, n->T, false) || overlap(r, ro, n->T, false) || overlap(o, ro, n->T, true))))
    return set_error(MOE_ERR_INVALID_ARG, "rows of out or residual_out overlap other rows that are read or written");
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int out = !e4m3 ? kOutSame : n->group ? kOutGroup : kOutRow;
  if (n->dtype == MOE_BF16)
    return out == kOutSame  ? dispatch<MOE_BF16, kOutSame>(*n, wide, st)
           : out == kOutRow ? dispatch<MOE_BF16, kOutRow>(*n, wide, st)
                            : dispatch<MOE_BF16, kOutGroup>(*n, wide, st);
  return out == kOutSame  ? dispatch<MOE_F16, kOutSame>(*n, wide, st)
         : out == kOutRow ? dispatch<MOE_F16, kOutRow>(*n, wide, st)
                          : dispatch<MOE_F16, kOutGroup>(*n, wide, st);
}
