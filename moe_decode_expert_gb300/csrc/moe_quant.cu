// moe_quant.cu — quantisation of rows or weights to e4m3 with an fp32 scale for
// each block of 1 or 128 rows by 128 columns.
//
//   s = max(max|x|, 2^-96) / 448 over the block;  out = e4m3(x / s)
//
// A block's values stay in registers between its largest magnitude and the
// output, so every input is read once.  Magnitudes are reduced as unsigned bit
// patterns: their order is that of the floats, with NaN above infinity, so a NaN
// reaches its block's scale.

#include <cuda_fp8.h>

#include "moe_common.cuh"
#include "moe_internal.h"

namespace moe {
namespace {

constexpr int kBlock = 128;  // columns of a scale
constexpr float kE4m3Max = 448.0f;
constexpr float kAmaxFloor = 1.26217744835361888865876570445e-29f;  // 2^-96

__device__ __forceinline__ float scale_of(uint32_t amax) {
  const float a = __uint_as_float(amax);
  return __fdiv_rn(a < kAmaxFloor ? kAmaxFloor : a, kE4m3Max);
}
__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7fffffffu; }

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}

template <int DT>
__device__ __forceinline__ uint32_t amax8(const uint4& v) {
  float f[8];
  unpack8<DT>(v, f);
  uint32_t m = 0u;
#pragma unroll
  for (int j = 0; j < 8; ++j) m = max(m, magnitude(f[j]));
  return m;
}
template <int DT>
__device__ __forceinline__ uint2 codes8(const uint4& v, float inv) {
  float f[8];
  unpack8<DT>(v, f);
#pragma unroll
  for (int j = 0; j < 8; ++j) f[j] *= inv;
  return make_uint2(e4m3x4(f[0], f[1], f[2], f[3]), e4m3x4(f[4], f[5], f[6], f[7]));
}

// Blocks of one row, 16-byte loads: 16 neighbouring lanes hold a block, and a
// thread NV of them, blockDim / 16 blocks apart in the [T, blocks] order.
template <int DT, int NV>
__global__ void __launch_bounds__(256) quant_rows_wide_kernel(moe_quant_t a, int blocks, int64_t total) {
  pdl_launch_dependents();
  pdl_wait();
  const int sub = threadIdx.x & 15;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * (16 * NV) + (threadIdx.x >> 4);
  uint4 v[NV];
  int64_t row[NV];
  int col[NV];
#pragma unroll
  for (int u = 0; u < NV; ++u) {
    const int64_t at = first + 16 * u;
    row[u] = at / blocks;
    col[u] = static_cast<int>(at - row[u] * blocks) * kBlock + sub * 8;
    v[u] = make_uint4(0, 0, 0, 0);
    if (at < total && col[u] < a.H)
      v[u] = ld_ordered16(static_cast<const uint16_t*>(a.x) + row[u] * a.x_stride + col[u]);
  }
#pragma unroll
  for (int u = 0; u < NV; ++u) {
    const int64_t at = first + 16 * u;
    uint32_t m = amax8<DT>(v[u]);
#pragma unroll
    for (int o = 1; o < 16; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float s = scale_of(m);
    if (at < total) {
      if (sub == 0) a.scales[at] = s;
      if (col[u] < a.H)
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.out) + row[u] * a.out_stride + col[u]) =
            codes8<DT>(v[u], __frcp_rn(s));
    }
  }
}

// Blocks of one row at any alignment: a warp per block, 4 elements per lane.
template <int DT>
__global__ void __launch_bounds__(256) quant_rows_kernel(moe_quant_t a, int blocks, int64_t total) {
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int64_t at = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  if (at >= total) return;
  const int64_t row = at / blocks;
  const int c0 = static_cast<int>(at - row * blocks) * kBlock + lane;
  const uint16_t* x = static_cast<const uint16_t*>(a.x) + row * a.x_stride;
  uint8_t* o = static_cast<uint8_t*>(a.out) + row * a.out_stride;
  float f[4];
  uint32_t m = 0u;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    f[j] = c0 + 32 * j < a.H ? load_scalar<DT>(x, c0 + 32 * j) : 0.0f;
    m = max(m, magnitude(f[j]));
  }
  const float s = scale_of(__reduce_max_sync(0xffffffffu, m));
  const float inv = __frcp_rn(s);
  if (lane == 0) a.scales[at] = s;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (c0 + 32 * j < a.H)
      o[c0 + 32 * j] = static_cast<uint8_t>(__nv_cvt_float_to_fp8(f[j] * inv, __NV_SATFINITE, __NV_E4M3));
}

// Blocks of 128 rows: a CTA each, 16 threads (WIDE: 16-byte loads) or a warp (any
// alignment) per row and pass.
template <int DT, bool WIDE>
__global__ void __launch_bounds__(256) quant_blocks_kernel(moe_quant_t a, int blocks) {
  constexpr int kPer = WIDE ? 16 : 8, kPass = kBlock / kPer;  // rows of a pass, passes
  __shared__ uint32_t s_max[8];
  pdl_launch_dependents();
  pdl_wait();
  const int64_t at = blockIdx.x;
  const int64_t r0 = at / blocks * kBlock;
  const int c0 = static_cast<int>(at % blocks) * kBlock;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int sub = WIDE ? threadIdx.x & 15 : lane, r = WIDE ? threadIdx.x >> 4 : warp;
  const uint16_t* x = static_cast<const uint16_t*>(a.x);
  uint8_t* o = static_cast<uint8_t*>(a.out);
  uint32_t m = 0u;
  uint4 v[WIDE ? kPass : 1];
  uint16_t e[WIDE ? 1 : kPass][4];
#pragma unroll
  for (int p = 0; p < kPass; ++p) {
    const int64_t row = r0 + r + kPer * p;
    if constexpr (WIDE) {
      v[p] = make_uint4(0, 0, 0, 0);
      if (row < a.T && c0 + sub * 8 < a.H) v[p] = ld_ordered16(x + row * a.x_stride + c0 + sub * 8);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        e[p][j] = row < a.T && c0 + lane + 32 * j < a.H ? x[row * a.x_stride + c0 + lane + 32 * j] : 0;
    }
  }
#pragma unroll
  for (int p = 0; p < kPass; ++p) {
    if constexpr (WIDE) {
      m = max(m, amax8<DT>(v[p]));
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) m = max(m, magnitude(unpack2<DT>(e[p][j]).x));
    }
  }
  m = __reduce_max_sync(0xffffffffu, m);
  if (lane == 0) s_max[warp] = m;
  __syncthreads();
  const float s = scale_of(__reduce_max_sync(0xffffffffu, s_max[lane & 7]));
  const float inv = __frcp_rn(s);
  if (threadIdx.x == 0) a.scales[at] = s;
#pragma unroll
  for (int p = 0; p < kPass; ++p) {
    const int64_t row = r0 + r + kPer * p;
    if (row >= a.T) continue;
    if constexpr (WIDE) {
      if (c0 + sub * 8 < a.H) *reinterpret_cast<uint2*>(o + row * a.out_stride + c0 + sub * 8) = codes8<DT>(v[p], inv);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int c = c0 + lane + 32 * j;
        if (c < a.H)
          o[row * a.out_stride + c] = static_cast<uint8_t>(
              __nv_cvt_float_to_fp8(unpack2<DT>(e[p][j]).x * inv, __NV_SATFINITE, __NV_E4M3));
      }
    }
  }
}

template <int DT>
cudaError_t launch(const moe_quant_t& q, bool wide, int blocks, int64_t total, cudaStream_t st) {
  if (q.rows == kBlock)
    return launch_pdl(wide ? quant_blocks_kernel<DT, true> : quant_blocks_kernel<DT, false>,
                      dim3(static_cast<unsigned>(total)), dim3(256), 0, st, q, blocks);
  if (!wide)
    return launch_pdl(quant_rows_kernel<DT>, dim3(static_cast<unsigned>((total + 7) / 8)), dim3(256), 0, st, q, blocks,
                      total);
  if (total <= 16 * 4 * sm_count())
    return launch_pdl(quant_rows_wide_kernel<DT, 1>, dim3(static_cast<unsigned>((total + 15) / 16)), dim3(256), 0, st,
                      q, blocks, total);
  return launch_pdl(quant_rows_wide_kernel<DT, 4>, dim3(static_cast<unsigned>((total + 63) / 64)), dim3(256), 0, st, q,
                    blocks, total);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" moe_status_t moe_quantize_e4m3(const moe_quant_t* q, void* stream) {
  if (!q) return set_error(MOE_ERR_INVALID_ARG, "moe_quant_t is NULL");
  if (q->T < 0 || q->H < 1) return set_error(MOE_ERR_INVALID_ARG, "T must be >= 0 and H >= 1");
  if (q->rows != 1 && q->rows != kBlock) return set_error(MOE_ERR_INVALID_ARG, "rows must be 1 or 128");
  if (q->dtype != MOE_F16 && q->dtype != MOE_BF16)
    return set_error(MOE_ERR_UNSUPPORTED, "dtype must be MOE_F16 or MOE_BF16");
  if (q->T == 0) return MOE_OK;
  if (!q->x || !q->out || !q->scales) return set_error(MOE_ERR_INVALID_ARG, "x / out / scales is NULL");
  const int64_t xs = q->T > 1 ? q->x_stride : q->H, os = q->T > 1 ? q->out_stride : q->H;
  if (xs < q->H || os < q->H) return set_error(MOE_ERR_INVALID_ARG, "row strides must be at least H");
  const uintptr_t x = reinterpret_cast<uintptr_t>(q->x), o = reinterpret_cast<uintptr_t>(q->out),
                  s = reinterpret_cast<uintptr_t>(q->scales);
  if ((x & 1u) || (s & 3u)) return set_error(MOE_ERR_INVALID_ARG, "a pointer is not aligned to its element type");
  const int blocks = (q->H - 1) / kBlock + 1;
  const int64_t total = (static_cast<int64_t>(q->T) - 1) / q->rows * blocks + blocks;
  if (total > INT32_MAX) return set_error(MOE_ERR_UNSUPPORTED, "ceil(T / rows) * ceil(H / 128) must be below 2^31");
  Span xspan, ospan;
  const Span sspan{s, 4 * total};
  if (!row_span(q->x, q->T, xs, q->H, 2, xspan) || !row_span(q->out, q->T, os, q->H, 1, ospan))
    return set_error(MOE_ERR_INVALID_ARG, "row strides reach past any memory");
  if (meet(xspan, ospan) || meet(xspan, sspan) || meet(ospan, sspan))
    return set_error(MOE_ERR_INVALID_ARG, "out and scales must not overlap x or each other");
  moe_quant_t a = *q;
  a.x_stride = xs;
  a.out_stride = os;
  const bool wide = q->H % 8 == 0 && (x & 15u) == 0 && (o & 7u) == 0 && ((xs | os) & 7) == 0;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if ((q->dtype == MOE_BF16 ? launch<MOE_BF16>(a, wide, blocks, total, st)
                            : launch<MOE_F16>(a, wide, blocks, total, st)) != cudaSuccess)
    return check_launch("quantisation kernel");
  stat_kernels(1);
  return MOE_OK;
}
