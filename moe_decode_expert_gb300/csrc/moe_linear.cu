// moe_linear.cu — product of e4m3 rows with an e4m3 weight, both with fp32 scales
// of blocks of 128 (x: per row and 128 columns; w: per 128 x 128), on tcgen05.
//
//   out[t][n] = sum_b xs[t][b] ws[n / 128][b] P_b[t][n],
//   P_b[t][n] = sum_{k in block b} x[t][k] w[n][k]
//
// A block's product P_b is four tensor-core steps of 32 into an fp32 accumulator in
// tensor memory that starts at zero; an epilogue warp reads it and adds it, times
// its two scales, to fp32 sums in registers while the next block's product is made
// in another accumulator.  A block of K is 128 bytes, one row of the 128-byte
// swizzle, so a stage of the ring is one block of both operands.  The two scales
// are applied as their product; a chunk of blocks in which some product is no
// normal number is summed by another loop, which applies them one after the other.
//
// Few rows stream the weight: 8 x 151936 x 2048 51 us, 6200 GB/s, 93 % of the copy;
// one row x 5120 x 2048 3.9 us in a graph, launch and latency.  Many rows are bound by
// the sums: reading a 256 x 256 accumulator and adding it takes as long as the MMAs
// that make it (8192 x 5120 x 4096 136 us, 2530 TFLOP/s; 116 with no accumulator read).

#include <algorithm>

#include "moe_common.cuh"
#include "moe_exact.h"
#include "moe_internal.h"
#include "moe_tc.cuh"

namespace moe {
namespace {

constexpr int kBlock = 128;               // columns (and weight rows) of a scale
constexpr uint32_t kTile = 128 * kBlock;  // bytes of 128 rows of a block

// Instruction descriptor, kind::f8f6f4: fp32 accumulator, A and B e4m3, both
// K-major, M = 128, N.
template <int N>
constexpr uint32_t idesc_e4m3() {
  return (1u << 4) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(128 >> 4) << 24);
}
__device__ __forceinline__ void mma_e4m3(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                         uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// One thread of a converged warp, always the same.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}
// Fetch a tile into L2 (may come before griddepcontrol.wait: L2 is where writes meet).
__device__ __forceinline__ void tma_prefetch_2d(const CUtensorMap* map, int c0, int c1) {
  asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global [%0, {%1, %2}];" ::"l"(map), "r"(c0), "r"(c1) : "memory");
}

__device__ __forceinline__ uint32_t pack2(int dt, float a, float b) {
  if (dt == MOE_BF16) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
  const __half2 v = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// Cluster-wide barrier in two halves; every thread of every CTA takes part in both.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
// (after the fence of set-up barriers, which is all that it has to order)
__device__ __forceinline__ void cluster_arrive_relaxed() { asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }
// The address in CTA `rank`'s shared memory that `addr` is in this one's.
__device__ __forceinline__ uint32_t peer_addr(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
// 8 or 16 bytes into another CTA's shared memory, counted on a barrier there.
__device__ __forceinline__ void send8(uint32_t dst, float a, float b, uint32_t bar) {
  asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], {%1,%2}, [%3];" ::"r"(dst), "f"(a),
               "f"(b), "r"(bar)
               : "memory");
}
__device__ __forceinline__ void send16(uint32_t dst, float a, float b, float c, float d, uint32_t bar) {
  asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1,%2,%3,%4}, [%5];" ::"r"(dst),
               "f"(a), "f"(b), "f"(c), "f"(d), "r"(bar)
               : "memory");
}

// ============================================================ few rows
// The weight's rows are the MMA's M (128 per tile) and NT tokens its N, so the
// weight, the larger operand, is streamed once for them.  S CTAs of a cluster share
// a tile's blocks of K; each then adds the S partial sums (in the order of K) of 1 / S
// of the columns, which the others send from their registers to its shared memory.
template <int NT>
struct Few {
  static constexpr uint32_t kStage = kTile + NT * kBlock;
  static constexpr int kAcc = NT <= 32 ? 4 : 2;  // accumulators in tensor memory
  static constexpr uint32_t kCols = NT * kAcc;
  static constexpr int kChunk = 16;       // blocks whose scales are staged at a time
  static constexpr int kPitch = NT + 4;   // floats per block of staged scales
  static constexpr uint32_t kScales = kChunk * kPitch * 4;
  static constexpr uint32_t kParts = NT * 512;  // sums of this CTA's columns, S > 1
  static constexpr int kMaxStages = 5;
  // Of a CTA's shared memory: the ring, one or two chunks of scales, the sums.  At least the
  // share that its columns are of the SM's 512, so that no CTA waits for columns that another
  // holds.
  static size_t smem(int stages, int nkb, int S) {
    const size_t n = stages * kStage + (nkb > kChunk ? 2 : 1) * kScales + (S > 1 ? kParts : 0) + 1024;
    const size_t least = static_cast<size_t>(kCols) * 227 * 1024 / 512;
    return n < least ? least : n;
  }
  static int stages(int nkb, int S) {
    int n = std::min(kMaxStages, std::max(nkb, 2));
    while (n > 2 && smem(n, nkb, S) > 113 * 1024) --n;  // two CTAs fit an SM
    return n;
  }
};

template <int NT>
__global__ void __launch_bounds__(192, 2)
    linear_few_kernel(const __grid_constant__ CUtensorMap mapW, const __grid_constant__ CUtensorMap mapX,
                      moe_linear_t a, int KB, int S, int mtiles, int stages, Control* ctrl, uint64_t timeout) {
  using F = Few<NT>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* scales = reinterpret_cast<float*>(smem + stages * F::kStage);
  __shared__ __align__(8) uint64_t full[F::kMaxStages], empty[F::kMaxStages], tfull[F::kAcc], tempty[F::kAcc], done, inbox;
  __shared__ uint32_t tmem_base_s;
  __shared__ volatile int s_abort, s_odd[2];

  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const int rank = static_cast<int>(blockIdx.x % S);
  const int tile = static_cast<int>(blockIdx.x / S);
  const int m0 = tile % mtiles * NT, nt = tile / mtiles, n0 = nt * 128;
  const int kb0 = static_cast<int>(static_cast<int64_t>(KB) * rank / S);
  const int nkb = static_cast<int>(static_cast<int64_t>(KB) * (rank + 1) / S) - kb0;
  float* parts = scales + ((KB + S - 1) / S > F::kChunk ? 2 : 1) * (F::kScales / 4);
  const int width = NT / S, wshift = __ffs(width) - 1;  // columns whose sums this CTA adds: fours, or two
  constexpr int kMinVec = NT == 16 ? 2 : 4;
  const int vec = NT == 16 && width == 2 ? 2 : 4;
  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) { mbar_init(&full[s], 1); mbar_init(&empty[s], 1); }
    for (int b = 0; b < F::kAcc; ++b) { mbar_init(&tfull[b], 1); mbar_init(&tempty[b], 4); }
    mbar_init(&done, 1);
    mbar_init(&inbox, 1);
    mbar_fence_init();
    s_abort = s_odd[0] = s_odd[1] = 0;
    // (others' sums of this CTA's columns, fours or twos with a token)
    if (S > 1)
      mbar_arrive_expect_tx(&inbox, static_cast<uint32_t>((max(min(a.M - m0 - rank * width, width), 0) + vec - 1) / vec * (S - 1) * vec) * 512u);
    tensormap_prefetch(&mapW);
    tensormap_prefetch(&mapX);
    for (int i = 0; i < min(nkb, stages); ++i) tma_prefetch_2d(&mapW, (kb0 + i) * kBlock, n0);
  }
  if (threadIdx.x == 64)  // (the weight's scales to L2, as the weight; of a row of scales' 128 bytes)
    asm volatile("prefetch.global.L2 [%0];" ::"l"(a.w_scales + static_cast<int64_t>(nt) * KB + kb0));
  if (warp == 1) {
    tmem_alloc(&tmem_base_s, F::kCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // (after the allocation: a CTA of the next kernel that got its columns first would wait for
  // this one, and this one for those columns)
  pdl_launch_dependents();
  if (S > 1) cluster_arrive_relaxed();
  pdl_wait();
  const uint32_t tbase = tmem_base_s;

  if (warp == 0) {
    if (lane == 0) {  // ---------------------------------------------- TMA producer
      int stage = 0;
      uint32_t phase = 0, issued_mask = 0, issued_phase = 0;
      for (int i = 0; i < nkb; ++i) {
        if (i >= stages && !tc_wait_polled(&empty[stage], phase ^ 1u, timeout, &s_abort)) {
          s_abort = 1;
          report_error(ctrl, kDevTimeoutCopy, blockIdx.x);
          break;
        }
        uint8_t* st = smem + stage * F::kStage;
        mbar_arrive_expect_tx(&full[stage], F::kStage);
        tma_load_2d(st, &mapW, &full[stage], (kb0 + i) * kBlock, n0);
        tma_load_2d(st + kTile, &mapX, &full[stage], (kb0 + i) * kBlock, m0);
        issued_mask |= 1u << stage;
        issued_phase = (issued_phase & ~(1u << stage)) | (phase << stage);
        if (++stage == stages) { stage = 0; phase ^= 1u; }
      }
      // let every copy this thread issued land before the CTA exits
      for (int s = 0; s < stages; ++s)
        if (issued_mask & (1u << s)) mbar_wait_until(&full[s], (issued_phase >> s) & 1u, global_ns() + timeout);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ----------------------------------------------------------------- MMA issuer
    // (the whole warp goes through the loop and one thread of it issues: with the others gone, an
    // MMA's descriptors are moved to the uniform registers it takes them from one by one)
    constexpr uint32_t idesc = idesc_e4m3<NT>();
    const uint64_t adesc = sw128_desc(smem_u32(smem)), bdesc = sw128_desc(smem_u32(smem) + kTile);
    int stage = 0;
    uint32_t phase = 0;
    for (int i = 0; i < nkb; ++i) {
      const int b = i % F::kAcc;
      if (!__all_sync(0xffffffffu, (i < F::kAcc || tc_wait_polled(&tempty[b], ((i / F::kAcc) & 1) ^ 1u, timeout, &s_abort)) &&
                                       tc_wait_polled(&full[stage], phase, timeout, &s_abort))) {
        s_abort = 1;
        if (lane == 0) report_error(ctrl, kDevTimeoutCopy, blockIdx.x);
        break;
      }
      tc_fence_after();
      const uint64_t at = static_cast<uint64_t>(stage) * (F::kStage >> 4);  // of a descriptor's address
      if (elect_one()) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          mma_e4m3(tbase + static_cast<uint32_t>(b * NT), adesc + at + 2 * k, bdesc + at + 2 * k, idesc, k != 0);
        tc_commit(&empty[stage]);
        tc_commit(&tfull[b]);
      }
      __syncwarp();
      if (++stage == stages) { stage = 0; phase ^= 1u; }
    }
    if (elect_one()) {
      tc_commit(&done);  // completes once every MMA issued above has completed
      mbar_wait_until(&done, 0, global_ns() + timeout);
    }
    __syncwarp();
  } else {  // ---------------------------------------------------- epilogue, 128 threads
    const int q = warp & 3;
    const int row = 32 * q + lane;      // weight row of the tile = TMEM lane
    const int etid = threadIdx.x - 64;  // 0..127
    constexpr int kPer = NT * F::kChunk / 128, kChunkBits = 4, kStep = NT == 16 ? 16 : 32;
    static_assert(F::kChunk == 1 << kChunkBits, "chunks of a power of two");
    float acc[NT];
#pragma unroll
    for (int c = 0; c < NT; ++c) acc[c] = 0.0f;
    float next[kPer];
    // A chunk's blocks are 2^cb, of kChunk at most: where there are few, no thread asks for others.
    const int cb = min(32 - __clz(nkb - 1), kChunkBits), cmask = (1 << cb) - 1;
    // products of both scales for blocks [c << cb, ..), anything normal beyond M and the last block
    const auto fetch = [&](int chunk) {
#pragma unroll
      for (int u = 0; u < kPer; ++u) {
        const int at = etid + 128 * u, t = at >> cb, i = (chunk << cb) + (at & cmask);
        next[u] = 1.0f;
        if (t < NT && i < nkb && m0 + t < a.M)
          next[u] = a.x_scales[static_cast<int64_t>(m0 + t) * KB + kb0 + i] *
                    a.w_scales[static_cast<int64_t>(nt) * KB + kb0 + i];
      }
    };
    // (s_odd says of a chunk whether some product is infinite or below the normal numbers)
    const auto stage_scales = [&](int chunk) {
      float least = 1.0f, most = 1.0f;
#pragma unroll
      for (int u = 0; u < kPer; ++u) {
        const int at = etid + 128 * u, t = at >> cb;
        least = fminf(least, fabsf(next[u]));
        most = fmaxf(most, fabsf(next[u]));
        if (t < NT) scales[((chunk & 1) * F::kChunk + (at & cmask)) * F::kPitch + t] = next[u];
      }
      if (!normal(least) || !normal(most)) s_odd[chunk & 1] = chunk + 1;
    };
    bool ok = true;
    // Waits for block i's sums (a wait that ran out leaves the loop running without it, so that all
    // warps meet at the barriers); their address.
    const auto begin = [&](int i) {
      const int b = i % F::kAcc;
      ok = __all_sync(0xffffffffu, ok && tc_wait_polled(&tfull[b], (i / F::kAcc) & 1, timeout, &s_abort));
      if (ok) tc_fence_after();
      else s_abort = 1;
      return tbase + (static_cast<uint32_t>(32 * q) << 16) + static_cast<uint32_t>(b * NT);
    };
    const auto release = [&](int i) {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&tempty[i % F::kAcc]);
    };
    // Blocks [i0, i1), a chunk with such products: small code with the sums in local memory, as it
    // seldom runs and lies between what does.
    const auto add_odd = [&](int i0, int i1) {
      float sum[NT];
#pragma unroll
      for (int c = 0; c < NT; ++c) sum[c] = acc[c];
#pragma unroll 1
      for (int i = i0; i < i1; ++i) {
        const uint32_t ta = begin(i);
        if (!ok) continue;
#pragma unroll 1
        for (int c = 0; c < NT && m0 + c < a.M; ++c)
          sum[c] = add_scaled(sum[c], tmem_ld1(ta + c), a.x_scales[static_cast<int64_t>(m0 + c) * KB + kb0 + i],
                              a.w_scales[static_cast<int64_t>(nt) * KB + kb0 + i]);
        release(i);
      }
#pragma unroll
      for (int c = 0; c < NT; ++c) acc[c] = sum[c];
    };
    fetch(0);
    for (int i = 0; i < nkb; ++i) {
      const int chunk = i >> cb, in = i & cmask;
      if (in == 0) {
        stage_scales(chunk);
        named_bar_sync(1, 128);  // (also: every warp is past the chunk before the last, whose place this was)
        const int next_i = (chunk + 1) << cb;
        const bool odd = s_odd[chunk & 1] == chunk + 1;
        if (odd) add_odd(i, min(nkb, next_i));
        if (next_i < nkb) fetch(chunk + 1);
        if (odd) {
          i = next_i - 1;
          continue;
        }
      }
      const uint32_t ta = begin(i);
      if (!ok) continue;
      const float4* sc = reinterpret_cast<const float4*>(scales + ((chunk & 1) * F::kChunk + in) * F::kPitch);
#pragma unroll
      for (int c0 = 0; c0 < NT; c0 += kStep) {
        uint32_t v[kStep];
        if constexpr (kStep == 32) tmem_ld32_issue(ta + c0, v);
        else tmem_ld16_issue(ta + c0, v);
        tmem_ld_wait();
        tmem_ld_tie(v);
        if (c0 + kStep == NT) release(i);
#pragma unroll
        for (int j = 0; j < kStep / 4; ++j) {
          const float4 s = sc[c0 / 4 + j];
          acc[c0 + 4 * j] = fmaf(__uint_as_float(v[4 * j]), s.x, acc[c0 + 4 * j]);
          acc[c0 + 4 * j + 1] = fmaf(__uint_as_float(v[4 * j + 1]), s.y, acc[c0 + 4 * j + 1]);
          acc[c0 + 4 * j + 2] = fmaf(__uint_as_float(v[4 * j + 2]), s.z, acc[c0 + 4 * j + 2]);
          acc[c0 + 4 * j + 3] = fmaf(__uint_as_float(v[4 * j + 3]), s.w, acc[c0 + 4 * j + 3]);
        }
      }
    }
    if (!ok && lane == 0) report_error(ctrl, kDevTimeoutCopy, blockIdx.x);
    const int n = n0 + row;
    if (S == 1) {
      if (n < a.N) {
#pragma unroll
        for (int c = 0; c < NT; ++c)
          if (m0 + c < a.M) store_out(a.out, static_cast<size_t>((m0 + c) * a.out_stride + n), acc[c], a.out_dtype);
      }
    } else {
      cluster_wait();  // every CTA of the cluster runs
      // sums as [CTA that has them][fours or twos of columns][row] in the CTA whose columns they are
      const uint32_t bar = smem_u32(&inbox);
      const uint32_t mine = smem_u32(parts) + static_cast<uint32_t>((rank * width * 128 + row * vec) * 4);
#pragma unroll
      for (int c = 0; c < NT; c += kMinVec) {
        if (m0 + c >= a.M) break;
        const int to = c >> wshift;
        const uint32_t at = mine + static_cast<uint32_t>((c - to * width) * 512);
        float* here = parts + (rank * width + c - to * width) * 128 + row * vec;
        if (kMinVec == 2 && vec == 2) {
          if (to == rank) *reinterpret_cast<float2*>(here) = make_float2(acc[c], acc[c + 1]);
          else if (!s_abort) send8(peer_addr(at, to), acc[c], acc[c + 1], peer_addr(bar, to));
        } else if (c % 4 == 0) {
          if (to == rank) *reinterpret_cast<float4*>(here) = make_float4(acc[c], acc[c + 1], acc[c + 2], acc[c + 3]);
          else if (!s_abort) send16(peer_addr(at, to), acc[c], acc[c + 1], acc[c + 2], acc[c + 3], peer_addr(bar, to));
        }
      }
      const bool here = tc_wait_polled(&inbox, 0, timeout, &s_abort);
      if (!here) {
        s_abort = 1;
        report_error(ctrl, kDevTimeoutCopy, blockIdx.x);
      }
      const int c0 = m0 + rank * width, many = here && n < a.N ? min(a.M - c0, width) : 0;
      const auto write = [&](int j, float v) {
        if (j < many) store_out(a.out, static_cast<size_t>((c0 + j) * a.out_stride + n), v, a.out_dtype);
      };
      if (kMinVec == 2 && vec == 2) {
        float2 sum = make_float2(0.0f, 0.0f);
        for (int r = 0; r < S; ++r) {
          const float2 v = reinterpret_cast<const float2*>(parts)[r * 128 + row];
          sum.x += v.x, sum.y += v.y;
        }
        write(0, sum.x), write(1, sum.y);
      } else {
        for (int j = 0; j < many; j += 4) {
          const float4* from = reinterpret_cast<const float4*>(parts) + j / 4 * 128 + row;
          float4 sum = from[0];
#pragma unroll
          for (int r = 1; r < 8; ++r)
            if (r < S) {
              const float4 v = from[r * (width / 4) * 128];
              sum.x += v.x, sum.y += v.y, sum.z += v.z, sum.w += v.w;
            }
          write(j, sum.x), write(j + 1, sum.y), write(j + 2, sum.z), write(j + 3, sum.w);
        }
      }
    }
  }
  if (S > 1 && warp < 2) cluster_wait();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tbase, F::kCols);
  }
  // A CTA that gave up is not left before the others have: what they sent may be on its way.
  if (S > 1 && s_abort) {
    cluster_arrive();
    cluster_wait();
  }
}

// =========================================================== many rows
// Tiles of 256 tokens by N weight rows, each of a pair of CTAs: the tokens are the
// MMA's M (128 per CTA), the weight rows its N, and each CTA stages half of both, so that
// a pair reads every byte once.  Accumulators fill the tensor memory.  A row's sums of a
// tile are in N / 64 threads' registers, 64 each.
template <int N>
struct Many {
  static constexpr uint32_t kStage = kTile + N / 2 * kBlock;
  static constexpr int kStages = N == 256 ? 4 : 7;
  static constexpr int kAcc = 512 / N;
  // Warps that issue MMAs, block by block in turn: what one does for a block (two waits, four
  // MMAs, two commits) takes longer than the block's MMAs (N = 128: 272 us with one warp, 202
  // with two, for 8192 x 5120 x 4096).
  static constexpr int kIssuers = 2;
  static constexpr int kWarps = N / 16;  // of the epilogue
  static constexpr int kThreads = 128 + 32 * kWarps;
  static constexpr int kLoads = N == 256 ? 1 : 2;        // loads of 32 columns in flight: what registers allow
  static constexpr int kChunk = 16;                      // blocks whose scales are staged at a time,
  static constexpr int kScales = kChunk * (128 + N / 128);  // floats: the rows' and the weight blocks'
  static constexpr uint32_t kTurn = 32 * 128;            // bytes a warp turns its results in
  static constexpr size_t kSmem = kStages * kStage + 2 * kScales * 4 + kWarps * kTurn + 1024;
};

__device__ __forceinline__ void tma_load_2d_pair(void* dst, const CUtensorMap* map, uint32_t bar, int c0, int c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], "
      "[%2];" ::"r"(smem_u32(dst)),
      "l"(map), "r"(bar), "r"(c0), "r"(c1)
      : "memory");
}
__device__ __forceinline__ void mma_e4m3_pair(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                              uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Arrives on the barrier at this offset in both CTAs once the MMAs issued so far are done.
__device__ __forceinline__ void tc_commit_pair(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
          smem_u32(bar)),
      "h"(static_cast<uint16_t>(3))
      : "memory");
}
// (Released to the CTA only: what it orders, reads of tensor memory, the fence before it has
// ordered; a release to the cluster waits for the thread's memory operations, 335 us against 212
// for 8192 x 5120 x 4096.)
__device__ __forceinline__ void mbar_arrive_at(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// (a, b) += (x, y) * s, in one instruction (in two: 140 us for 8192 x 5120 x 4096, 136)
__device__ __forceinline__ void fma2(float& a, float& b, uint32_t x, uint32_t y, float s) {
  asm("{\n\t.reg .b64 c, d, e;\n\tmov.b64 c, {%2, %3};\n\tmov.b64 d, {%4, %4};\n\tmov.b64 e, {%0, %1};\n\t"
      "fma.rn.f32x2 e, c, d, e;\n\tmov.b64 {%0, %1}, e;\n\t}"
      : "+f"(a), "+f"(b)
      : "r"(x), "r"(y), "f"(s));
}

__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, const void* src, int c0, int c1) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];" ::"l"(map), "r"(smem_u32(src)),
               "r"(c0), "r"(c1)
               : "memory");
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}

// A warp's 32 rows of 64 results to memory, 128 bytes of each row at a time: through shared
// memory, in 16-byte pieces whose order is turned by the row as the 128-byte swizzle has it, and
// from there by a bulk copy that goes on while the next tile is summed (stores of the warps' own
// took 2.7 us of a tile's 17: 8192 x 5120 x 4096 151 us, so 136).  Rows that do not begin on 16 bytes, and their ends, are
// written by the warp.
// SIZE: bytes of an output.
template <int SIZE>
__device__ __forceinline__ void many_store(const moe_linear_t& a, const CUtensorMap* map, const float (&acc)[64],
                                           uint8_t* turn, int m0, int n0, int lane, int bulk) {
  constexpr int kCols = 128 / SIZE, kPiece = 16 / SIZE;  // of a pass, of a piece
#pragma unroll
  for (int c0 = 0; c0 < 64; c0 += kCols) {
    const int n = n0 + c0;
    if (n >= a.N) break;
    if (bulk && lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
    __syncwarp();
#pragma unroll
    for (int p = 0; p < 8; ++p) {
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (SIZE == 4) w[j] = __float_as_uint(acc[c0 + 4 * p + j]);
        else w[j] = pack2(a.out_dtype, acc[8 * p + 2 * j], acc[8 * p + 2 * j + 1]);
      }
      *reinterpret_cast<uint4*>(turn + lane * 128 + ((p ^ lane) & 7) * 16) = make_uint4(w[0], w[1], w[2], w[3]);
    }
    if (bulk && n + kCols <= a.N) {  // (the copy would fill up the last 16 bytes of a row)
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) tma_store_2d(map, turn, n, m0);
    } else {
      __syncwarp();
      for (int i = lane; i < 32 * kCols; i += 32) {
        const int r = i / kCols, c = i % kCols;
        const uint8_t* at = turn + r * 128 + ((c / kPiece ^ r) & 7) * 16 + c % kPiece * SIZE;
        if (m0 + r < a.M && n + c < a.N) {
          uint8_t* o = static_cast<uint8_t*>(a.out) + ((m0 + r) * a.out_stride + n + c) * SIZE;
          if constexpr (SIZE == 4) *reinterpret_cast<uint32_t*>(o) = *reinterpret_cast<const uint32_t*>(at);
          else *reinterpret_cast<uint16_t*>(o) = *reinterpret_cast<const uint16_t*>(at);
        }
      }
    }
  }
}

template <int N>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(Many<N>::kThreads, 1)
    linear_many_kernel(const __grid_constant__ CUtensorMap mapX, const __grid_constant__ CUtensorMap mapW,
                       const __grid_constant__ CUtensorMap mapOut, moe_linear_t a, int KB, int mtiles, int tiles, int bulk, Control* ctrl, uint64_t timeout) {
  using G = Many<N>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ __align__(8) uint64_t full[G::kStages], empty[G::kStages], tfull[G::kAcc], tempty[G::kAcc], sfull[2], sempty[2],
      done[G::kIssuers];
  __shared__ uint32_t tmem_base_s;
  __shared__ volatile int s_abort, s_far[2];  // (of a chunk of scales: whether some are far from 1)

  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const int rank = static_cast<int>(blockIdx.x & 1u);  // in the pair; 0 issues the MMAs
  const int first = static_cast<int>(blockIdx.x >> 1), step = static_cast<int>(gridDim.x >> 1);
  if (threadIdx.x == 0) {
    for (int s = 0; s < G::kStages; ++s) { mbar_init(&full[s], 1); mbar_init(&empty[s], 1); }
    for (int b = 0; b < G::kAcc; ++b) { mbar_init(&tfull[b], 1); mbar_init(&tempty[b], 2 * G::kWarps); }
    for (int b = 0; b < 2; ++b) { mbar_init(&sfull[b], 32); mbar_init(&sempty[b], G::kWarps); }
    for (int i = 0; i < G::kIssuers; ++i) mbar_init(&done[i], 1);
    mbar_fence_init();
    s_abort = 0;
    tensormap_prefetch(&mapX);
    tensormap_prefetch(&mapW);
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_base_s)),
                 "r"(512u)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  cluster_arrive();  // both CTAs' barriers are set up before either signals the other's
  cluster_wait();
  tc_fence_after();
  pdl_launch_dependents();
  pdl_wait();
  const uint32_t tbase = tmem_base_s;
  // (N = 256: 640 threads of 96 registers at launch, 128 * 32 + 512 * 112 then)
  if constexpr (N == 256)
    if (warp < 4) asm volatile("setmaxnreg.dec.sync.aligned.u32 32;");

  if (warp == 0) {
    if (lane == 0) {  // ---------------------------------------------- TMA producer
      int stage = 0;
      uint32_t phase = 0, issued_mask = 0, issued_phase = 0;
      for (int t = first; t < tiles && !s_abort; t += step) {
        const int m0 = t % mtiles * 256 + rank * 128, n0 = t / mtiles * N + rank * (N / 2);
        for (int kb = 0; kb < KB; ++kb) {
          if (!tc_wait_polled(&empty[stage], phase ^ 1u, timeout, &s_abort)) {
            s_abort = 1;
            report_error(ctrl, kDevTimeoutCopy, blockIdx.x);
            break;
          }
          uint8_t* st = smem + stage * G::kStage;
          const uint32_t bar = peer_addr(smem_u32(&full[stage]), 0);  // rank 0's, for both
          if (rank == 0) mbar_arrive_expect_tx(&full[stage], 2 * G::kStage);
          tma_load_2d_pair(st, &mapX, bar, kb * kBlock, m0);
          tma_load_2d_pair(st + kTile, &mapW, bar, kb * kBlock, n0);
          issued_mask |= 1u << stage;
          issued_phase = (issued_phase & ~(1u << stage)) | (phase << stage);
          if (++stage == G::kStages) { stage = 0; phase ^= 1u; }
        }
      }
      // let every copy of the pair land before a CTA exits (rank 1 leaves after rank 0)
      if (rank == 0)
        for (int s = 0; s < G::kStages; ++s)
          if (issued_mask & (1u << s)) mbar_wait_until(&full[s], (issued_phase >> s) & 1u, global_ns() + timeout);
    }
    __syncwarp();
  } else if (warp <= G::kIssuers) {
    if (rank == 0) {  // ---------------------------------------------- MMA issuers
      // (the whole warp goes through the loop and one thread of it issues: with the others gone, an
      // MMA's descriptors are moved to the uniform registers it takes them from one by one)
      constexpr uint32_t idesc = (1u << 4) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(256 >> 4) << 24);
      const int blocks = first < tiles ? ((tiles - 1 - first) / step + 1) * KB : 0;
      const uint64_t adesc = sw128_desc(smem_u32(smem)), bdesc = sw128_desc(smem_u32(smem) + kTile);
      int stage = warp - 1, b = warp - 1;
      uint32_t phase = 0, bphase = 0;
      for (int i = warp - 1; i < blocks; i += G::kIssuers) {
        if (!__all_sync(0xffffffffu, tc_wait_polled(&tempty[b], bphase ^ 1u, timeout, &s_abort) &&
                                         tc_wait_polled(&full[stage], phase, timeout, &s_abort))) {
          s_abort = 1;
          if (lane == 0) report_error(ctrl, kDevTimeoutCopy, blockIdx.x);
          break;
        }
        tc_fence_after();
        const uint64_t at = static_cast<uint64_t>(stage) * (G::kStage >> 4);  // of a descriptor's address
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma_e4m3_pair(tbase + static_cast<uint32_t>(b * N), adesc + at + 2 * k, bdesc + at + 2 * k, idesc, k != 0);
          tc_commit_pair(&empty[stage]);
          tc_commit_pair(&tfull[b]);
        }
        __syncwarp();
        stage += G::kIssuers;
        if (stage >= G::kStages) { stage -= G::kStages; phase ^= 1u; }
        b += G::kIssuers;
        if (b >= G::kAcc) { b -= G::kAcc; bphase ^= 1u; }
      }
      if (elect_one()) {
        // completes once every MMA that this thread issued has completed
        asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                         smem_u32(&done[warp - 1]))
                     : "memory");
        mbar_wait_until(&done[warp - 1], 0, global_ns() + timeout);
      }
    }
    __syncwarp();
  } else if (warp < 4) {  // ------------------------------------------- scales
    // A chunk's scales, two chunks in turn: four rows a thread, and the weight block's.  (Loaded by each
    // thread of the epilogue for its own row they missed L1, which 128 rows a line apart overflow.)
    float* scales = reinterpret_cast<float*>(smem + G::kStages * G::kStage + G::kWarps * G::kTurn);
    int buf = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int t = first; t < tiles && ok; t += step) {
      const int m0 = t % mtiles * 256 + rank * 128, nb = t / mtiles * (N / 128);
      for (int kb0 = 0; kb0 < KB; kb0 += G::kChunk) {
        ok = __all_sync(0xffffffffu, tc_wait_polled(&sempty[buf], phase ^ 1u, timeout, &s_abort));
        if (!ok) break;
        float* sc = scales + buf * G::kScales;
        float least = 1.0f, most = 1.0f;  // magnitudes of this lane's scales
        if (lane % G::kChunk + kb0 < KB && lane < N / 128 * G::kChunk) {  // (past the last weight block: any)
          const float w =
              a.w_scales[static_cast<int64_t>(min(nb + lane / G::kChunk, (a.N - 1) / 128)) * KB + kb0 + lane % G::kChunk];
          sc[G::kChunk * 128 + lane] = w;
          least = most = fabsf(w);
        }
#pragma unroll 1
        for (int r = lane; r < 128; r += 32) {
          const float* from = a.x_scales + static_cast<int64_t>(min(m0 + r, a.M - 1)) * KB + kb0;
          float v[G::kChunk];
#pragma unroll
          for (int i = 0; i < G::kChunk; ++i) v[i] = kb0 + i < KB ? from[i] : 1.0f;
#pragma unroll
          for (int i = 0; i < G::kChunk; ++i) {
            sc[i * 128 + r] = v[i];
            least = fminf(least, fabsf(v[i]));
            most = fmaxf(most, fabsf(v[i]));
          }
        }
        const bool far = __any_sync(0xffffffffu, least < kNearScale || most >= 1.0f / kNearScale);
        if (lane == 0) s_far[buf] = far;
        mbar_arrive(&sfull[buf]);
        buf ^= 1;
        phase ^= buf == 0;
      }
    }
    if (!ok) {
      s_abort = 1;
      if (lane == 0) report_error(ctrl, kDevTimeoutCopy, blockIdx.x);
    }
  } else {  // ------------------------------------------------------- epilogue
    if constexpr (N == 256) asm volatile("setmaxnreg.inc.sync.aligned.u32 112;");
    const int q = warp & 3, g = (warp - 4) >> 2;  // quarter of the TMEM lanes, 64 of the columns
    const uint32_t lane0 = tbase + (static_cast<uint32_t>(32 * q) << 16) + static_cast<uint32_t>(64 * g);
    const uint32_t free_bar = peer_addr(smem_u32(&tempty[0]), 0);
    float* scales = reinterpret_cast<float*>(smem + G::kStages * G::kStage + G::kWarps * G::kTurn);
    uint8_t* turn = smem + G::kStages * G::kStage + (warp - 4) * G::kTurn;
    int b = 0, buf = 0;  // accumulator; chunk of scales
    uint32_t bphase = 0, sphase = 0;
    bool ok = true;
    for (int t = first; t < tiles; t += step) {
      float acc[64];
#pragma unroll
      for (int c = 0; c < 64; ++c) acc[c] = 0.0f;
      for (int kb0 = 0; kb0 < KB; kb0 += G::kChunk) {
        // (a wait that ran out leaves the loops running without it, so that all warps end together)
        ok = __all_sync(0xffffffffu, ok && tc_wait_polled(&sfull[buf], sphase, timeout, &s_abort));
        const float* sc = scales + buf * G::kScales;
        const int n = min(G::kChunk, KB - kb0);
        // Reads this row's scales, and waits for the block's sums.
        const auto begin = [&](int in, float& sx, float& sw) {
          sx = sc[in * 128 + 32 * q + lane], sw = sc[G::kChunk * (128 + (g >> 1)) + in];
          if (in + 1 == n) {
            __syncwarp();
            if (lane == 0) mbar_arrive(&sempty[buf]);
          }
          ok = __all_sync(0xffffffffu, ok && tc_wait_polled(&tfull[b], bphase, timeout, &s_abort));
          if (ok) tc_fence_after();
          else s_abort = 1;
        };
        const auto release = [&] {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_at(free_bar + static_cast<uint32_t>(8 * b));
        };
        if (!s_far[buf]) {
          for (int in = 0; in < n; ++in) {
            float s, sw;
            begin(in, s, sw);
            if (!ok) continue;
            s *= sw;
#pragma unroll
            for (int c = 0; c < 64; c += 32 * G::kLoads) {
              uint32_t v[G::kLoads][32];
#pragma unroll
              for (int u = 0; u < G::kLoads; ++u) tmem_ld32_issue(lane0 + static_cast<uint32_t>(b * N + c + 32 * u), v[u]);
              tmem_ld_wait();
#pragma unroll
              for (int u = 0; u < G::kLoads; ++u) tmem_ld_tie(v[u]);
              if (c + 32 * G::kLoads == 64) release();
#pragma unroll
              for (int j = 0; j < 32 * G::kLoads; j += 2)
                fma2(acc[c + j], acc[c + j + 1], v[j / 32][j % 32], v[j / 32][j % 32 + 1], s);
            }
            if (++b == G::kAcc) { b = 0; bphase ^= 1u; }
          }
        } else {  // (seldom: small code, with the sums in local memory)
          float sum[64];
#pragma unroll
          for (int c = 0; c < 64; ++c) sum[c] = acc[c];
#pragma unroll 1
          for (int in = 0; in < n; ++in) {
            float sx, sw;
            begin(in, sx, sw);
            if (!ok) continue;
#pragma unroll 1
            for (int c = 0; c < 64; ++c)
              sum[c] = add_scaled(sum[c], tmem_ld1(lane0 + static_cast<uint32_t>(b * N + c)), sx, sw);
            release();
            if (++b == G::kAcc) { b = 0; bphase ^= 1u; }
          }
#pragma unroll
          for (int c = 0; c < 64; ++c) acc[c] = sum[c];
        }
        buf ^= 1;
        sphase ^= buf == 0;
      }
      if (!ok) continue;
      const int m0 = t % mtiles * 256 + rank * 128 + 32 * q, n0 = t / mtiles * N + 64 * g;
      if (m0 >= a.M || n0 >= a.N) continue;
      if (a.out_dtype == MOE_F32) many_store<4>(a, &mapOut, acc, turn, m0, n0, lane, bulk);
      else many_store<2>(a, &mapOut, acc, turn, m0, n0, lane, bulk);
    }
    if (bulk && lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    if (!ok) {
      s_abort = 1;
      if (lane == 0) report_error(ctrl, kDevTimeoutCopy, blockIdx.x);
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_arrive();  // neither CTA's memory goes while the other's MMAs or arrivals may touch it
  cluster_wait();
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tbase), "r"(512u) : "memory");
  }
}

// ================================================================ host
// 2-D map of `outer` rows of `inner` elements of `size` bytes, `stride` bytes apart; box of
// 128 bytes x box_rows, 128-byte swizzle; zeros outside.
bool map_2d(CUtensorMap* m, CUtensorMapDataType type, uint32_t size, const void* base, uint64_t inner, uint64_t outer,
            uint64_t stride, uint32_t box_rows) {
  const auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[2] = {inner, outer}, strides[1] = {stride};
  cuuint32_t box[2] = {128 / size, box_rows}, estr[2] = {1, 1};
  return fn(m, type, 2, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool byte_map(CUtensorMap* m, const void* base, uint64_t inner, uint64_t outer, uint64_t stride, uint32_t box_rows) {
  return map_2d(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, base, inner, outer, stride, box_rows);
}

template <int NT>
moe_status_t launch_few(const moe_linear_t& l, int KB, Control* ctrl, cudaStream_t st) {
  const int mtiles = (l.M - 1) / NT + 1;
  const int64_t tiles = static_cast<int64_t>(mtiles) * ((l.N - 1) / 128 + 1);
  int S = 1;
  while (S < 8 && tiles * S <= sm_count() && KB >= 4 * S) S *= 2;
  const int nkb = (KB + S - 1) / S, stages = Few<NT>::stages(nkb, S);
  CUtensorMap mw, mx;
  if (!byte_map(&mw, l.w, l.K, l.N, l.w_stride, 128) || !byte_map(&mx, l.x, l.K, l.M, l.x_stride, NT))
    return set_error(MOE_ERR_CUDA, "cuTensorMapEncodeTiled failed (linear)");
  const size_t smem = Few<NT>::smem(stages, nkb, S);
  if (raise_smem_limit(linear_few_kernel<NT>, smem) != cudaSuccess) return check_launch("linear_few_kernel (smem)");
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(tiles * S));
  cfg.blockDim = dim3(192);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {static_cast<unsigned>(S), 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  if (cudaLaunchKernelEx(&cfg, linear_few_kernel<NT>, mw, mx, l, KB, S, mtiles, stages, ctrl, tc_wait_timeout_ns()) != cudaSuccess)
    return check_launch("linear_few_kernel");
  stat_kernels(1);
  return MOE_OK;
}

template <int N>
moe_status_t launch_many(const moe_linear_t& l, int KB, Control* ctrl, cudaStream_t st) {
  const int mtiles = (l.M - 1) / 256 + 1;
  const int tiles = mtiles * ((l.N - 1) / N + 1);
  CUtensorMap mx, mw;
  if (!byte_map(&mx, l.x, l.K, l.M, l.x_stride, 128) || !byte_map(&mw, l.w, l.K, l.N, l.w_stride, N / 2))
    return set_error(MOE_ERR_CUDA, "cuTensorMapEncodeTiled failed (linear)");
  if (raise_smem_limit(linear_many_kernel<N>, Many<N>::kSmem) != cudaSuccess)
    return check_launch("linear_many_kernel (smem)");
  const int size = l.out_dtype == MOE_F32 ? 4 : 2;
  const int bulk = (reinterpret_cast<uintptr_t>(l.out) & 15u) == 0 && l.out_stride * size % 16 == 0 &&
                   l.out_stride * size < int64_t(1) << 40;
  CUtensorMap mo = mx;
  if (bulk && !map_2d(&mo, size == 4 ? CU_TENSOR_MAP_DATA_TYPE_UINT32 : CU_TENSOR_MAP_DATA_TYPE_UINT16, size, l.out, l.N, l.M,
                      l.out_stride * size, 32))
    return set_error(MOE_ERR_CUDA, "cuTensorMapEncodeTiled failed (linear)");
  const int pairs = sm_count() / 2;
  if (launch_pdl(linear_many_kernel<N>, dim3(2 * (tiles < pairs ? tiles : pairs)), dim3(Many<N>::kThreads), Many<N>::kSmem,
                 st, mx, mw, mo, l, KB, mtiles, tiles, bulk, ctrl, tc_wait_timeout_ns()) != cudaSuccess)
    return check_launch("linear_many_kernel");
  stat_kernels(1);
  return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" moe_status_t moe_linear_e4m3(const moe_linear_t* l, void* ws, size_t ws_bytes, void* stream) {
  if (!l) return set_error(MOE_ERR_INVALID_ARG, "moe_linear_t is NULL");
  if (l->M < 0 || l->N < 0 || l->K < 1) return set_error(MOE_ERR_INVALID_ARG, "M and N must be >= 0 and K >= 1");
  if (l->out_dtype != MOE_F16 && l->out_dtype != MOE_BF16 && l->out_dtype != MOE_F32)
    return set_error(MOE_ERR_UNSUPPORTED, "out_dtype must be MOE_F16, MOE_BF16 or MOE_F32");
  if (l->M == 0 || l->N == 0) return MOE_OK;
  if (!l->x || !l->x_scales || !l->w || !l->w_scales || !l->out)
    return set_error(MOE_ERR_INVALID_ARG, "x / x_scales / w / w_scales / out is NULL");
  if (!ws || ws_bytes < sizeof(Control) || reinterpret_cast<uintptr_t>(ws) % kWsAlign)
    return set_error(MOE_ERR_WORKSPACE, "a 256-byte aligned workspace of this library is needed");
  moe_linear_t a = *l;
  // a single row's stride says nothing
  if (a.M == 1) a.x_stride = (a.K + 15ll) & ~15ll, a.out_stride = a.N;
  if (a.N == 1) a.w_stride = (a.K + 15ll) & ~15ll;
  if (a.x_stride < a.K || a.w_stride < a.K || a.out_stride < a.N)
    return set_error(MOE_ERR_INVALID_ARG, "row strides must be at least the rows' lengths");
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.x), w = reinterpret_cast<uintptr_t>(a.w),
                  o = reinterpret_cast<uintptr_t>(a.out);
  if ((x | w) & 15u) return set_error(MOE_ERR_UNSUPPORTED, "x and w must begin on 16 bytes");
  if ((a.x_stride | a.w_stride) & 15)
    return set_error(MOE_ERR_UNSUPPORTED, "the row strides of x and w must be multiples of 16");
  const int size = a.out_dtype == MOE_F32 ? 4 : 2;
  if ((o & (size - 1)) || ((reinterpret_cast<uintptr_t>(a.x_scales) | reinterpret_cast<uintptr_t>(a.w_scales)) & 3u))
    return set_error(MOE_ERR_INVALID_ARG, "a pointer is not aligned to its element type");
  const int KB = (a.K - 1) / kBlock + 1, nb = (a.N - 1) / 128 + 1;
  if (((a.M - 1ll) / 16 + 1) * nb >= int64_t(1) << 28)
    return set_error(MOE_ERR_UNSUPPORTED, "ceil(M / 16) * ceil(N / 128) must be below 2^28");
  Span xs, wsp, os;
  if (!row_span(a.x, a.M, a.x_stride, a.K, 1, xs) || !row_span(a.w, a.N, a.w_stride, a.K, 1, wsp) ||
      !row_span(a.out, a.M, a.out_stride, a.N, size, os) || a.x_stride >= int64_t(1) << 40 ||
      a.w_stride >= int64_t(1) << 40)
    return set_error(MOE_ERR_INVALID_ARG, "row strides reach past any memory");
  const Span ss{reinterpret_cast<uintptr_t>(a.x_scales), 4ll * a.M * KB};
  const Span ts{reinterpret_cast<uintptr_t>(a.w_scales), 4ll * nb * KB};
  if (meet(os, xs) || meet(os, wsp) || meet(os, ss) || meet(os, ts) ||
      meet(os, Span{reinterpret_cast<uintptr_t>(ws), sizeof(Control)}))
    return set_error(MOE_ERR_INVALID_ARG, "out must not overlap the other tensors");
  Control* ctrl = static_cast<Control*>(ws);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  // Few rows, or so few tiles of many that most pairs of SMs would have none (256 x 2048 x 4096,
  // 16 tiles for 76 pairs: 14.0 us, 9.6 by tiles of 64 rows and parts of K).
  const int64_t pairs = sm_count() / 2, m256 = (a.M - 1) / 256 + 1;
  if (a.M <= 16) return launch_few<16>(a, KB, ctrl, st);
  // (Tiles of 64 rows exchange twice the sums, and of 32 read the weight from L2 twice as often: 64 x
  // 5120 x 2048 7.4 us by 64, 6.7 by 32; 64 x 5120 x 8192 13.7 by 64, 14.9 by 32.)
  if (a.M <= 32 || (a.M <= 128 && static_cast<int64_t>(nb) * KB <= 8 * sm_count())) return launch_few<32>(a, KB, ctrl, st);
  if (a.M <= 128 || m256 * nb * 4 <= pairs) return launch_few<64>(a, KB, ctrl, st);
  // A wider tile takes about 1.5 times as long as a narrower: 8192 x 5120 x 4096 136 us against
  // 173, but 256 x 5120 x 2048, 20 tiles or 40 for 76 pairs, 12.7 against 10.3.
  const auto rounds = [&](int n) { return (m256 * ((a.N - 1) / n + 1) + pairs - 1) / pairs; };
  if (3 * rounds(256) <= 2 * rounds(128)) return launch_many<256>(a, KB, ctrl, st);
  return launch_many<128>(a, KB, ctrl, st);
}
