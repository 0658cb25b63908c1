// moe_quant.cu — quantisation of rows or weights to e4m3 with an fp32 scale for
// each block of 1 or 128 rows by 128 columns.
//
//   s = max(max|x|, 2^-96) / 448 over the block;  out = e4m3(x / s)
//
// with the quotient rounded to fp32 first.
// A block's values stay in registers between its largest magnitude and the
// output, so every input is read once.  Magnitudes are reduced as unsigned 16-bit
// patterns, two an instruction: their order is that of the floats, with NaN above
// infinity, so a NaN reaches its block's scale.
//
// HBM bounds it: 8192 rows of 4096 in bf16 16.9 us, 6020 GB/s, 90 % of the copy.

#include <cuda_fp8.h>

#include <type_traits>

#include "moe_common.cuh"
#include "moe_exact.h"
#include "moe_internal.h"
#include "moe_kv.h"

namespace moe {
namespace {

constexpr int kBlock = 128;  // columns of a scale
constexpr float kE4m3Max = 448.0f;
constexpr float kAmaxFloor = 1.26217744835361888865876570445e-29f;  // 2^-96

__device__ __forceinline__ float scale_of(uint32_t amax) {
  const float a = __uint_as_float(amax);
  return __fdiv_rn(a < kAmaxFloor ? kAmaxFloor : a, kE4m3Max);
}
__device__ __forceinline__ uint32_t max16x2(uint32_t a, uint32_t b) {
  uint32_t m;
  asm("max.u16x2 %0, %1, %2;" : "=r"(m) : "r"(a), "r"(b));
  return m;
}
// fp32 bits of a 16-bit magnitude
template <int DT>
__device__ __forceinline__ uint32_t wide(uint32_t m) {
  return __float_as_uint(unpack2<DT>(m).x);
}

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}

// The largest magnitudes of the even and of the odd values.
__device__ __forceinline__ uint32_t amax8(const uint4& v) {
  return max16x2(max16x2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu), max16x2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu));
}
// f, of a constant: whether the block's values are scaled up to be divided.
template <int DT, class F>
__device__ __forceinline__ void by_size(const Quotient& by, F f) {
  if (DT == MOE_BF16 && by.tiny) f(std::true_type());
  else f(std::false_type());
}
__device__ __forceinline__ uint32_t either(uint32_t m) { return max(m & 0xffffu, m >> 16); }
template <int DT, bool UP>
__device__ __forceinline__ uint2 codes8(const uint4& v, const Quotient& by) {
  float f[8];
  unpack8<DT>(v, f);
  by.divide<UP>(f);
  return make_uint2(e4m3x4(f[0], f[1], f[2], f[3]) ^ 0x80808080u, e4m3x4(f[4], f[5], f[6], f[7]) ^ 0x80808080u);
}

// Blocks of one row, 16-byte loads: 8 neighbouring lanes hold a block, 16 columns
// each, and a thread NV of them, blockDim / 8 blocks apart in the [T, blocks] order.
// EVEN: rows of out begin on 16 bytes too.
template <int DT, int NV, bool EVEN>
__global__ void __launch_bounds__(256) quant_rows_wide_kernel(moe_quant_t a, int blocks, FastDiv by_blocks, int total) {
  pdl_launch_dependents();
  pdl_wait();
  const int sub = threadIdx.x & 7;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * (32 * NV) + (threadIdx.x >> 3);
  uint4 v[NV][2];
  int row[NV], col[NV];
#pragma unroll
  for (int u = 0; u < NV; ++u) {
    const int at = static_cast<int>(min(first + 32 * u, static_cast<int64_t>(total) - 1));  // (past the end: the last again)
    row[u] = by_blocks(at);
    col[u] = (at - row[u] * blocks) * kBlock + sub * 16;
    const uint16_t* x = static_cast<const uint16_t*>(a.x) + static_cast<int64_t>(row[u]) * a.x_stride + col[u];
    v[u][0] = v[u][1] = make_uint4(0, 0, 0, 0);
    if (col[u] < a.H) v[u][0] = ld_ordered16(x);
    if (col[u] + 8 < a.H) v[u][1] = ld_ordered16(x + 8);
  }
#pragma unroll
  for (int u = 0; u < NV; ++u) {
    uint32_t m = max16x2(amax8(v[u][0]), amax8(v[u][1]));
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) m = max16x2(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float s = scale_of(wide<DT>(either(m)));
    const Quotient by(s);
    if (first + 32 * u >= total) break;
    if (sub == 0) a.scales[first + 32 * u] = s;
    uint8_t* o = static_cast<uint8_t*>(a.out) + static_cast<int64_t>(row[u]) * a.out_stride + col[u];
    uint2 lo, hi;
    by_size<DT>(by, [&](auto up) {
      lo = codes8<DT, up>(v[u][0], by);
      hi = codes8<DT, up>(v[u][1], by);
    });
    if (EVEN && col[u] + 8 < a.H) {
      *reinterpret_cast<uint4*>(o) = make_uint4(lo.x, lo.y, hi.x, hi.y);
    } else {
      if (col[u] < a.H) *reinterpret_cast<uint2*>(o) = lo;
      if (col[u] + 8 < a.H) *reinterpret_cast<uint2*>(o + 8) = hi;
    }
  }
}

// At any alignment a warp has a row's part of a block, lane l its columns l, l + 32, l + 64 and
// l + 96: neighbouring lanes write neighbouring bytes.  Bound by the memory instructions, one per
// 32 elements: 5120 x 2003 by blocks of 128 rows 9.9 us, 47 % of the 6680 GB/s copy.  (Eight columns a
// lane, stored in words put together from two lanes' bytes: 20 us.)
// (The four stay apart until all loads are out: put together at once, each load was waited for, 28 us.)
struct Spread {
  uint16_t v[4];
  __device__ __forceinline__ void load(const uint16_t* p, int n) {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = 32 * j < n ? p[32 * j] : 0;
  }
  // The largest magnitude's fp32 bits, or what gives them to wide().  (Of bf16 as it is stored: through
  // fp32 the loads were waited for one by one, 5120 x 2003 25.2 us, so 11.6; of fp16 by its
  // conversions, which keep the loads together: 11.2 us, as it is stored 11.6.)
  template <int DT>
  __device__ __forceinline__ uint32_t amax() const {
    uint32_t m = 0u;
#pragma unroll
    for (int j = 0; j < 4; ++j) m = max(m, DT == MOE_BF16 ? v[j] & 0x7fffu : __float_as_uint(unpack2<DT>(v[j]).x) & 0x7fffffffu);
    return m;
  }
  template <int DT>
  static __device__ __forceinline__ uint32_t bits(uint32_t amax) {
    return DT == MOE_BF16 ? wide<DT>(amax) : amax;
  }
  template <int DT, bool UP>
  __device__ __forceinline__ void store(uint8_t* o, int n, const Quotient& by) const {
    float f[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) f[j] = unpack2<DT>(v[j]).x;
    by.divide<UP>(f);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (32 * j < n) o[32 * j] = static_cast<uint8_t>(__nv_cvt_float_to_fp8(f[j], __NV_SATFINITE, __NV_E4M3) ^ 0x80);
  }
};

// Blocks of one row at any alignment: a warp has NV of them at a time.
template <int DT, int NV>
__global__ void __launch_bounds__(256) quant_rows_kernel(moe_quant_t a, int blocks, FastDiv by_blocks, int total) {
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * (8 * NV) + (threadIdx.x >> 5);
  Spread v[NV];
  int row[NV], col[NV];
#pragma unroll
  for (int u = 0; u < NV; ++u) {
    const int at = static_cast<int>(min(first + 8 * u, static_cast<int64_t>(total) - 1));
    row[u] = by_blocks(at);
    col[u] = (at - row[u] * blocks) * kBlock + lane;
    v[u].load(static_cast<const uint16_t*>(a.x) + static_cast<int64_t>(row[u]) * a.x_stride + col[u], a.H - col[u]);
  }
#pragma unroll
  for (int u = 0; u < NV; ++u) {
    if (first + 8 * u >= total) break;
    const float s = scale_of(Spread::bits<DT>(__reduce_max_sync(0xffffffffu, v[u].template amax<DT>())));
    if (lane == 0) a.scales[first + 8 * u] = s;
    uint8_t* o = static_cast<uint8_t*>(a.out) + static_cast<int64_t>(row[u]) * a.out_stride + col[u];
    const Quotient by(s);
    by_size<DT>(by, [&](auto up) { v[u].template store<DT, up>(o, a.H - col[u], by); });
  }
}

// Blocks of 128 rows: a CTA each, 16 threads (WIDE: 16-byte loads) or a warp (any alignment) per
// row and pass.
template <int DT, bool WIDE>
__global__ void __launch_bounds__(WIDE ? 256 : 512) quant_blocks_kernel(moe_quant_t a, int blocks) {
  constexpr int kPer = 16, kPass = kBlock / kPer;  // rows of a pass, passes
  constexpr int kWarps = WIDE ? 8 : 16;
  __shared__ uint32_t s_max[kWarps];
  pdl_launch_dependents();
  pdl_wait();
  const int64_t at = blockIdx.x;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t r0 = at / blocks * kBlock + (WIDE ? threadIdx.x >> 4 : warp);
  const int c0 = static_cast<int>(at % blocks) * kBlock + (WIDE ? (threadIdx.x & 15) * 8 : lane);
  const uint16_t* x = static_cast<const uint16_t*>(a.x);
  uint8_t* o = static_cast<uint8_t*>(a.out);
  uint32_t m = 0u;
  uint4 v[WIDE ? kPass : 1];
  Spread e[WIDE ? 1 : kPass];
#pragma unroll
  for (int p = 0; p < kPass; ++p) {
    const int64_t row = r0 + kPer * p;
    if constexpr (WIDE) {
      v[p] = make_uint4(0, 0, 0, 0);
      if (row < a.T && c0 < a.H) v[p] = ld_ordered16(x + row * a.x_stride + c0);
    } else {
      e[p].load(x + (row < a.T ? row * a.x_stride + c0 : 0), row < a.T ? a.H - c0 : 0);
    }
  }
#pragma unroll
  for (int p = 0; p < kPass; ++p) {
    if constexpr (WIDE) m = max16x2(m, amax8(v[p]));
    else m = max(m, e[p].template amax<DT>());
  }
  m = __reduce_max_sync(0xffffffffu, WIDE ? either(m) : m);
  if (lane == 0) s_max[warp] = m;
  __syncthreads();
  m = __reduce_max_sync(0xffffffffu, s_max[lane & (kWarps - 1)]);
  const float s = scale_of(WIDE ? wide<DT>(m) : Spread::bits<DT>(m));
  const Quotient by(s);
  if (threadIdx.x == 0) a.scales[at] = s;
  by_size<DT>(by, [&](auto up) {
#pragma unroll
    for (int p = 0; p < kPass; ++p) {
      const int64_t row = r0 + kPer * p;
      if (row >= a.T || c0 >= a.H) continue;
      if constexpr (WIDE) *reinterpret_cast<uint2*>(o + row * a.out_stride + c0) = codes8<DT, up>(v[p], by);
      else e[p].template store<DT, up>(o + row * a.out_stride + c0, a.H - c0, by);
    }
  });
}

template <int DT>
cudaError_t launch(const moe_quant_t& q, bool wide, int blocks, int64_t total, cudaStream_t st) {
  if (q.rows == kBlock)
    return launch_pdl(wide ? quant_blocks_kernel<DT, true> : quant_blocks_kernel<DT, false>,
                      dim3(static_cast<unsigned>(total)), dim3(wide ? 256 : 512), 0, st, q, blocks);
  if (!wide)
    return launch_pdl(quant_rows_kernel<DT, 4>, dim3(static_cast<unsigned>((total + 31) / 32)), dim3(256), 0, st, q, blocks,
                      FastDiv(blocks), static_cast<int>(total));
  const bool even = (reinterpret_cast<uintptr_t>(q.out) & 15u) == 0 && (q.out_stride & 15) == 0;
  const auto run = [&](auto kernel, int nv) {
    return launch_pdl(kernel, dim3(static_cast<unsigned>((total + 32 * nv - 1) / (32 * nv))), dim3(256), 0, st, q, blocks,
                      FastDiv(blocks), static_cast<int>(total));
  };
  // A block each while SMs would be left without any, then two: 64 bytes in flight per thread.
  if (total <= 32 * 4 * sm_count())
    return even ? run(quant_rows_wide_kernel<DT, 1, true>, 1) : run(quant_rows_wide_kernel<DT, 1, false>, 1);
  return even ? run(quant_rows_wide_kernel<DT, 2, true>, 2) : run(quant_rows_wide_kernel<DT, 2, false>, 2);
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
