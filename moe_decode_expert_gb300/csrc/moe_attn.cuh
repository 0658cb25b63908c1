// moe_attn.cuh — attention of one new token per sequence over a paged cache: the
// kernel and its launch.
//
// Per sequence and key/value head, the G = n_q_heads / n_kv_heads query heads
// of its group share every key and value row, which is read once: 4 G flops
// per element of the cache, so HBM bounds the kernel (8 flops per byte at
// G = 8 in 16 bits; the tensor cores have two orders of magnitude more).
//
// Scores are formed transposed, S^T = K Q^T (tokens x heads), so that a group
// of up to 8 heads fills the n = 8 side of mma.m16n8k16 and K rows are its A
// operand straight from shared memory; the output O^T = V^T P^T has the heads
// in the same columns, so the running maximum and sum of a head live in the
// lanes that hold its column.  movmatrix turns S^T fragments into P^T ones.
//
// Weights go into the second product as bf16 in two terms (2^-17) or as fp16 in
// one, 2^14 above their true value (2^-11, and normal down to 2^-28 of the
// largest; below that 2^-39 of it, absolute).  One fp16 term is no coarser than the
// half step of an fp16 output, an eighth of a bf16 one's; a second term would
// be a second product for every value.  Scores, references, sums and outputs are fp32
// throughout.
//
// Work is split evenly over workers whatever the lengths: the (sequence, kv
// head, unit of U tokens) triples form one line, with kVoid empty places before
// each segment, that is each (sequence, kv head), for its fixed cost; worker c of
// n takes the c-th n-th of it and finds its place from seq_lens itself.  A
// segment that ends up with several workers is joined by the last of them to
// arrive, in groups of kJoin parts and then over the groups, always in the same
// order: one launch, results independent of timing.  Where every segment is short
// and has a worker of its own, the line is not cut inside segments.
//
// Head chunks of a kv head beyond the first are further segments, or, up to
// kMaxSides of them, lines of their own side by side (blockIdx.y), on which as many
// workers read the same rows at about the same time.  Neighbouring kv heads, whose rows
// of a token are neighbours in memory, get lines side by side too (kv_sides).
//
// A worker is a CTA, or, where segments are few, a team: a cluster of 8 CTAs whose
// warps share each segment and sum their outputs through distributed shared
// memory, which spares a short sequence the join through global memory (1531
// tokens of 2 kv heads: 8.4 to 8.7 us against 13.7 with CTAs).
//
// A warp owns whole units: K and V of a unit are two slots of its own ring in
// shared memory, filled by cp.async two slots ahead, across segment ends; only the
// end of a long segment's part meets at a CTA barrier.
//
// Measured (fraction of the 6787 GB/s copy): 64 sequences of up to 32k tokens,
// 16 over 2 heads of 256, bf16: 320 to 331 us by GPU (100 to 97 %); 285k tokens of 8 e4m3 heads of
// 128, groups of 5: 100 us (86 %); 250 windows of 512 over 12 fp16 heads of 64,
// pages of 24: 69 us (77 %, bound by instructions: 8 columns for one head).

#pragma once

#include <atomic>

#include "moe_common.cuh"
#include "moe_kv.h"

namespace moe {
namespace {

constexpr int kRing = 3;         // slots of a warp's ring
constexpr int kMaxSms = 160;     // SMs that a launch fills
constexpr int kMaxCtas = 4 * kMaxSms;
constexpr int kSmallPer = 2;     // small chunks per CTA of a long line
constexpr int kMaxChunks = kMaxCtas * (1 + kSmallPer);  // partial slots in the workspace: two per chunk
// Chunks of all lines of a launch: four CTAs an SM at head_dim <= 64, else two.
constexpr int max_chunks(int dp) { return dp > 64 ? kMaxChunks / 2 : kMaxChunks; }
constexpr int kTeamCtas = 8;     // CTAs of a team (a cluster), and the most teams
constexpr int kMaxTeams = 40;
constexpr int kMaxSides = 8;     // lines side by side
constexpr int kMaxParts = 64;    // partial results combined at a time
// Places of the line that a team takes at least (one short sequence in one team:
// 256 cost 16.3 us where 128 cost 9.4, the two heads then sharing a team).
constexpr int kTeamMin = 128;
// Units up to which a segment is left whole where every one has a worker of its own:
// what a join costs goes into 32 units of a CTA (16 or 48 the same; 64 segments of
// up to 5 units 9.7 us against 13.8) and 256 of a team.
constexpr int kWholeCta = 32;
constexpr int kWholeTeam = 256;
// Units up to which a segment is one warp's alone (8 made 32 heads over 2 kv heads
// of ragged 8k tokens 12 % slower; none made 20 short segments 1.7 times slower).
constexpr int kSolo = 4;
// ... and where each has a CTA anyway (35 of up to 7 units 5.5 us, 6.6 with 2 and 8.6 with 4).
constexpr int kSoloWhole = 1;
// A line of kLong places per CTA and more keeps kBack per cent of them back for the
// CTAs that get done first: 327 to 320 us at 438 places per CTA; at 117 places the
// extra joins cost more than the balance gains (98 to 103 us).
constexpr int kLong = 256;
constexpr int kBack = 20;
// CTAs of an SM.  Rows of 64 elements leave registers for four, with units of half
// the bytes (the window case: 75 us against 81 with three and 90 with two); wider
// ones stay with two (three CTAs of half units at 128: within 2 % either way).
constexpr int kCtas64 = 4;
constexpr int kCtas128 = 2;
constexpr int kCtas256 = 2;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// Workspace: control block, join counters [kMaxChunks][4] (teams: [team][8]) and
// the number of small chunks taken, partial statistics [kMaxChunks * 2][16][2]
// fp32 (teams: [team * 2][8][16][2]), partial outputs [chunks * 2][heads][DP] fp32.
constexpr size_t kCountersAt = 256;
constexpr size_t kStatsAt = kCountersAt + kMaxChunks * 4 * sizeof(uint32_t) + 256;
constexpr size_t kPartsAt = kStatsAt + kMaxChunks * 2 * 16 * 2 * sizeof(float);
static_assert(kPartsAt % 256 == 0, "partials are 256-byte aligned");
static_assert(kMaxTeams * 8 <= kMaxCtas, "teams fit where CTAs do");

}  // namespace

struct AttnArgs {
  moe_kv_cache_t c;
  moe_attention_t a;
  uint8_t* ws;
  int32_t chunks;  // head chunks of a kv head on a line
  int32_t sides;   // lines side by side, one per further head chunk ...
  int32_t kv_sides;  // ... times those over neighbouring kv heads (a divisor of n_kv_heads)
  int32_t hpc;     // query heads of a chunk (<= 8 * NT)
  int32_t group;   // query heads of a kv head
  int32_t max_len; // max_pages * page_size, saturated
  FastDiv by_page;
  uint32_t k_page, k_token, k_head, v_page, v_token, v_head;  // the cache's strides in bytes
  int32_t blocks;  // page_size % 16 == 0: 16 neighbouring tokens share a page
};

namespace {

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// cp.async of 16 bytes, or zeros where `bytes` is 0 (nothing is read then).
__device__ __forceinline__ void cp16_or_zero(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint32_t movm_t(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

// D (16x8 fp32) += A (16x16) * B (16x8) in bf16 or fp16.
template <bool BF16>
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  if constexpr (BF16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

template <bool BF16>
__device__ __forceinline__ uint32_t pack(float a, float b) {
  if constexpr (BF16) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
  } else {
    const __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
}

// A bf16 pair with the largest finite value in an infinity's place.
__device__ __forceinline__ uint32_t finite2(uint32_t v) {
  uint32_t r;
  asm("min.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(v), "r"(0x7f7f7f7fu));
  return r;
}

// Four e4m3 values -> the low two and the high two as fp16 pairs, exact.
__device__ __forceinline__ void e4m3_half4(uint32_t four, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(four));
}

// What a combination of partial results keeps in shared memory (kThreads
// float4 follow it).
template <int HEADS>
struct Combine {
  float w[kMaxParts][HEADS], lp[kMaxParts][HEADS];  // references, then weights; partial sums
  float m[HEADS], l[HEADS];
};

// Everything of a kernel that does not depend on its place in the line.
template <int QT, bool F8, int DP, int NT, bool TEAM>
struct Shape {
  static constexpr int kWarps = 4;
  static constexpr int kThreads = kWarps * 32;
  static constexpr int kTeam = TEAM ? kTeamCtas : 1;  // CTAs of a worker
  static constexpr int kTw = kTeam * kWarps;          // its warps
  // places before a segment's units: its fixed cost, in units (2, 4, 6, 8 differ by
  // 2 %; without any the window case took a third longer)
  static constexpr int kVoid = TEAM ? 0 : 4;
  // places of the line a worker takes at least (CTAs: 4 and 6 cost short batches 2
  // us in joins, 16 and 20 2 us in streaming)
  static constexpr int kMinUnits = TEAM ? kTeamMin : 12;
  // units up to which a segment is left whole where every one has a worker
  static constexpr int kWhole = TEAM ? kWholeTeam : kWholeCta;
  static constexpr int kBytes = F8 ? 1 : 2;
  static constexpr int kFill = (TEAM || DP > 64 ? 8192 : 4096) / (DP * kBytes);
  static constexpr int kU = kFill < 16 ? 16 : kFill < 64 ? kFill : 64;  // tokens of a unit
  static constexpr int kCtas = TEAM ? 2 : DP == 256 ? kCtas256 : DP == 128 ? kCtas128 : NT == 1 ? kCtas64 : 3;  // CTAs of an SM
  static constexpr int kHeads = 8 * NT;
  // parts joined at a time: kMaxParts groups hold every chunk of a launch
  static constexpr int kJoin = DP > 64 ? 32 : 64;
  static_assert(kCtas * kMaxSms * (1 + kSmallPer) <= max_chunks(DP), "every chunk has its slots in the workspace");
  static_assert(kJoin <= kMaxParts && kCtas * kMaxSms * (1 + kSmallPer) <= kJoin * kMaxParts, "two levels of joins do");
  static constexpr int kRow = DP * kBytes;                                            // bytes of a row
  static constexpr int kSlot = kU * kRow;
  static constexpr int kCpr = kRow / 16;   // 16-byte chunks of a row
  static constexpr int kMt = kU / 16;      // m tiles of a unit's scores
  static constexpr int kDm = DP / 16;      // m tiles of the output
  static constexpr int kCols = NT == 1 && DP > 64 ? 64 : 32;  // output columns the warps merge at a time
  static constexpr int kPitch = kCols + 4;         // their fp32 pitch: conflict-free
  static constexpr bool kBf16 = !F8 && QT == MOE_BF16;  // type of the matrix products
  // Shared memory: the warps' rings, then the merge buffer (single CTAs) or what
  // a combination needs, whichever is larger.
  static constexpr int kRingBytes = kRing * kSlot;  // of a warp
  static constexpr int kMergeAt = kWarps * kRingBytes;
  static constexpr int kMerge = TEAM ? 0 : kWarps * kHeads * kPitch * 4;
  static constexpr int kCombine = static_cast<int>(sizeof(Combine<kHeads>)) + kThreads * 16;
  // what a team CTA receives: its columns and all statistics from every rank
  static constexpr int kShare = kHeads * DP / 4 / kTeamCtas;  // column quads
  static constexpr int kReceive = TEAM ? kTeam * (kShare * 16 + 16 * 8) : 0;
  static constexpr int kMost = kMerge > kCombine ? kMerge : kCombine;
  static constexpr int kSmem = kMergeAt + (kMost > kReceive ? kMost : kReceive);
  static constexpr int kPart = DP + 4;  // fp32 pitch of a team warp's output in its ring: conflict-free
  static_assert(kHeads * kPart * 4 <= kRingBytes, "a warp's output fits its ring");
};

// Byte offset of 16-byte chunk c of row r in a slot: chunks are permuted so
// that 8 rows at one chunk column lie in 8 different bank groups.
template <int kCpr>
__device__ __forceinline__ uint32_t swz(int r, int c) {
  if constexpr (kCpr >= 8) return static_cast<uint32_t>(r * kCpr * 16 + ((c ^ (r & 7)) << 4));
  // rows of 64 bytes: two to a 128-byte line
  return static_cast<uint32_t>((r >> 1) * 128 + ((((r & 1) * 4 + c) ^ ((r >> 1) & 3)) << 4));
}

// The line in chunks.  The n workers begin with a chunk each, of `each` places,
// the first `more` of one more.  A long line keeps its last part back: from
// `wide` on, chunks of `small` places that CTAs take as they get done, because SMs
// do not get equal shares of the memory's bandwidth (with equal chunks the last CTA
// of 304 was done at 96 us where the median was at 82).
struct Line {
  int total, n, each, more, wide, small, chunks;
  __device__ __forceinline__ int start(int c) const {
    return c <= n ? each * c + min(c, more) : min(wide + (c - n) * small, total);
  }
  __device__ __forceinline__ int owner(int x) const {
    const int first = more * (each + 1);
    if (x < first) return static_cast<int>(static_cast<unsigned>(x) / static_cast<unsigned>(each + 1));
    if (x < wide) return more + static_cast<int>(static_cast<unsigned>(x - first) / static_cast<unsigned>(each));
    return n + static_cast<int>(static_cast<unsigned>(x - wide) / static_cast<unsigned>(small));
  }
};

// A CTA of another rank of the cluster: its shared memory and the barrier.
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ uint32_t at_rank(const void* p, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  return a;
}
__device__ __forceinline__ void st_rank2(uint32_t a, float2 v) {
  asm volatile("st.shared::cluster.v2.f32 [%0], {%1,%2};" ::"r"(a), "f"(v.x), "f"(v.y) : "memory");
}
__device__ __forceinline__ void st_rank4(uint32_t a, float4 v) {
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1,%2,%3,%4};" ::"r"(a), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w)
               : "memory");
}

template <int QT, bool F8, int DP, int NT, bool TEAM>
__global__ void __launch_bounds__(Shape<QT, F8, DP, NT, TEAM>::kThreads, (Shape<QT, F8, DP, NT, TEAM>::kCtas))
    paged_attention_kernel(AttnArgs g) {
  using S = Shape<QT, F8, DP, NT, TEAM>;
  constexpr int kWarps = S::kWarps, kThreads = S::kThreads, kVoid = S::kVoid, kMinUnits = S::kMinUnits;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float s_m[kWarps][16], s_l[kWarps][16];
  __shared__ int s_scan[kWarps], s_most[kWarps], s_b, s_prefix, s_flag;

  const moe_attention_t& a = g.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int gr = lane >> 2, tq = lane & 3;  // row group and column pair of a fragment
  Control* ctrl = reinterpret_cast<Control*>(g.ws);
  uint32_t* counters = reinterpret_cast<uint32_t*>(g.ws + kCountersAt);
  float* stats = reinterpret_cast<float*>(g.ws + kStatsAt);
  float* parts = reinterpret_cast<float*>(g.ws + kPartsAt);

  pdl_launch_dependents();
  pdl_wait();

  // A sequence's token range and its places on the line: the void ones, then
  // its units (at least one, so that an empty sequence is written too).
  auto clamp_len = [&](int len) { return len < 0 ? 0 : min(len, g.max_len); };
  auto low = [&](int len) { return a.window > 0 && len > a.window ? len - a.window : 0; };
  auto places_of = [&](int lo, int len) { return kVoid + (len > lo ? (len + S::kU - 1) / S::kU - lo / S::kU : 1); };
  auto places = [&](int b) {
    const int len = clamp_len(a.seq_lens[b]);
    return places_of(low(len), len);
  };

  // The line's length and shape.  Up to 32 sequences: every warp by itself, a
  // sequence per lane.
  const int segs = g.c.n_kv_heads / g.kv_sides * g.chunks;  // segments of a sequence on this line
  const int side = static_cast<int>(blockIdx.y) / g.kv_sides, kv_side = static_cast<int>(blockIdx.y) - side * g.kv_sides;
  // the worker, and this CTA's and warp's number in it
  const int worker = static_cast<int>(blockIdx.x) / S::kTeam;
  const int rank = TEAM ? static_cast<int>(cluster_rank()) : 0;
  const int tw = rank * kWarps + warp;
  int my_len = 0, my_u = 0, my_inc = 0;  // a lane's sequence: length, places, places up to its end
  int sum = 0, most = 0;  // places of all sequences (before * segs), and of the longest
  if (a.B <= 32) {
    if (lane < a.B) {
      my_len = clamp_len(a.seq_lens[lane]);
      my_u = places_of(low(my_len), my_len);
    }
    my_inc = my_u;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, my_inc, o);
      if (lane >= o) my_inc += v;
    }
    sum = __shfl_sync(0xffffffffu, my_inc, 31);
    most = __reduce_max_sync(0xffffffffu, my_u);
  } else {
    for (int i = tid; i < a.B; i += kThreads) {
      const int u = places(i);
      sum += u;
      most = max(most, u);
    }
    sum = __reduce_add_sync(0xffffffffu, sum);
    most = __reduce_max_sync(0xffffffffu, most);
    if (lane == 0) {
      s_scan[warp] = sum;
      s_most[warp] = most;
    }
    __syncthreads();
    sum = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      sum += s_scan[w];
      most = max(most, s_most[w]);
    }
  }
  Line ln;
  ln.total = sum * segs;
  ln.n = (ln.total + kMinUnits - 1) / kMinUnits;
  // This line's slots and counters.
  const int at0 = static_cast<int>(blockIdx.y * gridDim.x) * (1 + kSmallPer);
  // a worker per segment, as long as there are workers: a segment of one unit
  // costs several units' time
  const int fit = static_cast<int>(gridDim.x) / S::kTeam;
  ln.n = min(max(ln.n, a.B * segs), fit);
  // Few and short segments: one worker each, with nothing to join.
  const bool whole_segs = a.B * segs <= fit && most <= kVoid + S::kWhole;
  if (whole_segs) ln.n = a.B * segs;
  if (worker >= ln.n) return;
  ln.each = static_cast<int>(static_cast<unsigned>(ln.total) / static_cast<unsigned>(ln.n));
  ln.more = ln.total - ln.each * ln.n;
  ln.wide = ln.total;
  ln.small = 1;
  ln.chunks = ln.n;
  if (!TEAM && !whole_segs && ln.each >= kLong) {
    ln.each -= static_cast<int>(static_cast<unsigned>(ln.each) * kBack / 100u);
    ln.more = 0;
    ln.wide = ln.each * ln.n;
    ln.small = (ln.total - ln.wide + kSmallPer * ln.n - 1) / (kSmallPer * ln.n);
    ln.chunks = ln.n + (ln.total - ln.wide + ln.small - 1) / ln.small;
  }

  const uint32_t ring = smem_u32(smem + warp * (kRing * S::kSlot));
  float* merge = reinterpret_cast<float*>(smem + S::kMergeAt);
  using Comb = Combine<S::kHeads>;
  Comb& cb_s = *reinterpret_cast<Comb*>(smem + S::kMergeAt);
  float4* cb_x = reinterpret_cast<float4*>(smem + S::kMergeAt + sizeof(Comb));
  const int D = g.c.head_dim;

  // ------------------------------------------------------------------ loads
  // The loads of this warp's units run ahead of the arithmetic: a cursor walks
  // the units to load, across segment ends (a team's within a segment: its rings hold the outputs
  // at the end of one).
  constexpr int kRr = (S::kU + 31) / 32;  // rows of a unit per lane
  constexpr int kStep = 32 / S::kCpr;     // rows of one pass of the warp
  const int col = lane % S::kCpr, row0 = lane / S::kCpr;
  const bool col_in = col * 16 < D * S::kBytes;
  int b = 0, prefix = 0, len = 0, lo = 0, nb = 0, p, p_end;
  int cb, cseg, clen, clo, cnb, next_len;  // the cursor's sequence and segment
  int cu, cue, cstep, cleft;  // its next unit, the end and step there; places left after that part
  // Which units of a segment's part at places [ub, ue) are this warp's: units
  // u, u + step, ... below `end`.  A short segment in one piece is one warp's
  // alone (solo), so that its end needs no barrier and the other warps go on;
  // else the warps take turns, beginning with another one in each segment.
  auto mine = [&](int sidx, int places_of_seg, int ub, int ue, int& u, int& end, int& step) {
    const int u0 = max(ub - kVoid, 0);
    end = ue - kVoid;
    if (!TEAM && places_of_seg <= kVoid + (whole_segs ? kSoloWhole : kSolo) && u0 == 0 && ue == places_of_seg) {
      u = 0;
      step = 1;
      if ((sidx & (kWarps - 1)) != warp) end = 0;
      return true;
    }
    u = u0 + ((tw - sidx) & (S::kTw - 1));
    step = S::kTw;
    return false;
  };
  auto enter = [&](int ub, int n) {  // the cursor's segment from place ub on, n places left
    const int ue = min(cnb, ub + n);
    cleft = n - (ue - ub);
    mine(cb * segs + cseg, cnb, ub, ue, cu, cue, cstep);
  };
  // Where the rows of a unit are: lane l holds rows l (and l + 32); the unit
  // looked up (n...) is the one after the unit being loaded.
  int page[kRr], off[kRr], npage[kRr], noff[kRr];
  int kvh_l = 0, nkvh = 0;  // their kv heads
  bool have = false, nhave = false, nvalid[kRr];
  auto look_up = [&]() {
    while (cu >= cue && cleft > 0) {
      if (++cseg == segs) {
        cseg = 0;
        ++cb;
        clen = clamp_len(next_len);
        clo = low(clen);
        cnb = places_of(clo, clen);
        next_len = cb + 1 < a.B ? a.seq_lens[cb + 1] : 0;
      }
      enter(0, cleft);
    }
    nhave = cu < cue;
#pragma unroll
    for (int r = 0; r < kRr; ++r) npage[r] = -1, noff[r] = 0, nvalid[r] = false;
    if (!nhave) return;
    nkvh = (g.chunks == 1 ? cseg : cseg / g.chunks) * g.kv_sides + kv_side;
    const int32_t* table = a.block_table + cb * a.table_stride;
#pragma unroll
    for (int r = 0; r < kRr; ++r) {
      const int row = lane + 32 * r;
      // unsigned: the last unit may reach past the largest int
      const uint32_t tok = static_cast<uint32_t>(clo / S::kU + cu) * S::kU + row;
      const uint32_t first = g.blocks ? tok | 15u : tok, last = g.blocks ? tok & ~15u : tok;
      nvalid[r] = row < S::kU && tok >= static_cast<uint32_t>(clo) && tok < static_cast<uint32_t>(clen);
      // rows beside those that count are placed too where a block shares a page
      if (row < S::kU && first >= static_cast<uint32_t>(clo) && last < static_cast<uint32_t>(clen)) {
        const int idx = g.by_page(static_cast<int>(tok));
        noff[r] = static_cast<int>(tok) - idx * g.c.page_size;
        npage[r] = table[idx];
        if (static_cast<uint32_t>(npage[r]) >= static_cast<uint32_t>(g.c.n_pages)) {
          npage[r] = -1;
          report_error(ctrl, kDevBadPage, static_cast<uint32_t>(cb));
        }
      }
    }
    cu += cstep;
  };
  uint64_t vm0 = 0, vm1 = 0;  // tokens of the unit in hand and of the next that count
  bool keys = true;           // what is loaded next: keys, then the same unit's values
  // Issue the next item, one unit's rows of K or of V, into `slot`; rows that do
  // not count (and columns past head_dim) become zeros without being read.
  auto issue = [&](uint32_t slot) {
    if (keys) {
      vm0 = vm1;
      vm1 = 0;
      have = nhave;
      kvh_l = nkvh;
#pragma unroll
      for (int r = 0; r < kRr; ++r) {
        page[r] = npage[r];
        off[r] = noff[r];
        vm1 |= static_cast<uint64_t>(__ballot_sync(0xffffffffu, nvalid[r] && page[r] >= 0)) << (32 * r);
      }
    }
    if (!have) {
      keys = !keys;
      cp_commit();
      return;
    }
    const uint64_t vm = vm1;
    // 32 by 32 bit products: one instruction each
    const uint32_t ps = keys ? g.k_page : g.v_page, ts = keys ? g.k_token : g.v_token, hs = keys ? g.k_head : g.v_head;
    const uint8_t* at = static_cast<const uint8_t*>(keys ? g.c.k : g.c.v) +
                        static_cast<uint64_t>(static_cast<uint32_t>(kvh_l)) * hs + col * 16;
    if (g.blocks) {
      // 16 rows on one page: one address, then steps
      at += static_cast<uint64_t>(static_cast<uint32_t>(row0)) * ts;
#pragma unroll
      for (int bl = 0; bl < S::kU / 16; ++bl) {
        const uint32_t pg = static_cast<uint32_t>(max(__shfl_sync(0xffffffffu, page[bl >> 1], (bl & 1) * 16), 0));
        const uint32_t of = static_cast<uint32_t>(__shfl_sync(0xffffffffu, off[bl >> 1], (bl & 1) * 16));
        const uint32_t bits = col_in ? static_cast<uint32_t>(vm >> (bl * 16 + row0)) : 0u;
        const uint8_t* src = at + static_cast<uint64_t>(pg) * ps + static_cast<uint64_t>(of) * ts;
        const uint64_t step = static_cast<uint64_t>(ts) * kStep;
#pragma unroll
        for (int i = 0; i < 16 / kStep; ++i, src += step)
          cp16_or_zero(slot + swz<S::kCpr>(bl * 16 + i * kStep + row0, col), src, ((bits >> (i * kStep)) & 1u) << 4);
      }
    } else {
      const uint64_t bits = col_in ? vm >> row0 : 0u;
#pragma unroll
      for (int i = 0; i < S::kU / kStep; ++i) {
        const int r = i * kStep + row0;
        const uint32_t pg = static_cast<uint32_t>(max(__shfl_sync(0xffffffffu, page[i * kStep / 32], r & 31), 0));
        const uint32_t of = static_cast<uint32_t>(__shfl_sync(0xffffffffu, off[i * kStep / 32], r & 31));
        const uint8_t* src = at + static_cast<uint64_t>(pg) * ps + static_cast<uint64_t>(of) * ts;
        cp16_or_zero(slot + swz<S::kCpr>(r, col), src, (static_cast<uint32_t>(bits >> (i * kStep)) & 1u) << 4);
      }
    }
    cp_commit();
    if (keys) look_up();
    keys = !keys;
  };
  int slot = 0;  // ring slot in hand
  auto slot_at = [&](int ahead) {
    int s = slot + ahead;
    if (s >= kRing) s -= kRing;
    return ring + s * S::kSlot;
  };
  // Start on `n` places from place `u` of segment `seg` of sequence b.
  auto start_loads = [&](int n, int seg, int u) {
    cb = b, cseg = seg;
    clen = len, clo = lo, cnb = nb;
    enter(u, n);
    next_len = cb + 1 < a.B ? a.seq_lens[cb + 1] : 0;
    look_up();
#pragma unroll 1
    for (int k = 0; k < kRing; ++k) issue(slot_at(k));  // K, V, K: vm0 is the first unit's mask, vm1 the second's
  };
  [[maybe_unused]] bool again = false;  // a team that has combined a segment before
  if constexpr (TEAM) cluster_arrive();  // waited for before the first write to another rank

  for (int cta = worker;;) {  // the chunk in hand
  p = ln.start(cta);
  p_end = ln.start(cta + 1);
  // The sequence that holds p: the one whose places, before * segs, reach it.
  if (whole_segs) {
    b = cta / segs;
    prefix = 0;  // places count from the sequence's first
    len = a.B <= 32 ? __shfl_sync(0xffffffffu, my_len, b) : clamp_len(a.seq_lens[b]);
  } else if (a.B <= 32) {
    b = 31 - __clz(__ballot_sync(0xffffffffu, my_u > 0 && (my_inc - my_u) * segs <= p));
    prefix = __shfl_sync(0xffffffffu, my_inc - my_u, b);
    len = __shfl_sync(0xffffffffu, my_len, b);
  } else {
    int before = 0;
    for (int b0 = 0;; b0 += kThreads) {
      const int i = b0 + tid;
      const int u = i < a.B ? places(i) : 0;
      int inc = u;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += v;
      }
      __syncthreads();
      if (lane == 31) s_scan[warp] = inc;
      if (tid == 0) s_b = -1;
      __syncthreads();
      int ex = before + inc - u;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        if (w < warp) ex += s_scan[w];
        before += s_scan[w];
      }
      if (u > 0 && ex * segs <= p && p < (ex + u) * segs) {
        s_b = i;
        s_prefix = ex;
      }
      __syncthreads();
      if (s_b >= 0) break;
    }
    b = s_b;
    prefix = s_prefix;
    len = clamp_len(a.seq_lens[b]);
  }
  lo = low(len);
  nb = places_of(lo, len);
  if (whole_segs) {
    p = (cta - b * segs) * nb;
    p_end = p + nb;
  }
  if constexpr (!TEAM) {
    keys = true;
    slot = 0;
    const int seg = (p - prefix * segs) / nb;
    start_loads(p_end - p, seg, p - prefix * segs - seg * nb);
  }

  while (p < p_end) {
    // ------------------------------------------ the part at places [ub, ue)
    const int local = p - prefix * segs;
    const int seg = static_cast<int>(static_cast<unsigned>(local) / static_cast<unsigned>(nb));
    const int ub = local - seg * nb;
    const int ue = min(nb, ub + p_end - p);
    const int seg_start = p - ub;
    if (ue <= kVoid) break;  // the share ends before the segment's first unit: it is the next CTA's
    const int kv = g.chunks == 1 ? seg : seg / g.chunks, chunk = seg - kv * g.chunks;
    const int kvh = kv * g.kv_sides + kv_side;
    const int h_in = (chunk * g.sides + side) * g.hpc;
    const int heads = min(g.hpc, g.group - h_in);  // query heads of this segment
    const int h0 = kvh * g.group + h_in;
    if constexpr (TEAM) {
      keys = true;
      slot = 0;
      start_loads(ue - ub, seg, ub);
    }
    if (tid == 0 && rank == 0) {
      const int raw = a.seq_lens[b];
      if (raw < 0 || raw > g.max_len) report_error(ctrl, kDevBadLength, static_cast<uint32_t>(b));
    }

    int u, u_end, u_step;
    const bool solo = mine(b * segs + seg, nb, ub, ue, u, u_end, u_step);
    const float vscale = F8 && g.c.v_scale ? g.c.v_scale[kvh] : 1.0f;
    float o[NT][S::kDm][4];
    float m[NT][2], l[NT][2];  // a head's reference (log2) and this lane's share of its sum
    if (!solo || u < u_end) {
    // Q fragments (the B operand): head gr of an n tile, its elements in the
    // order in which K fragments bring theirs.
    uint32_t qf[NT][DP / 16][2];
    float qscale[NT][2];  // what undoes the fp16 scaling of a bf16 query (e4m3 cache)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int h = nt * 8 + gr;
      const uint16_t* q = static_cast<const uint16_t*>(a.q) + b * a.q_seq_stride +
                          static_cast<int64_t>(h0 + (h < heads ? h : 0)) * a.q_head_stride;
#pragma unroll
      for (int ks = 0; ks < DP / 16; ++ks) {
        const int d0 = ks * 16 + (F8 ? 4 * tq : 2 * tq), d1 = d0 + (F8 ? 2 : 8);
        qf[nt][ks][0] = h < heads && d0 < D ? *reinterpret_cast<const uint32_t*>(q + d0) : 0u;
        qf[nt][ks][1] = h < heads && d1 < D ? *reinterpret_cast<const uint32_t*>(q + d1) : 0u;
      }
      qscale[nt][0] = qscale[nt][1] = 1.0f;
      if constexpr (F8 && QT == MOE_BF16) {
        // bf16 queries enter the fp16 products scaled by a power of two that
        // brings the head's largest element to [2^14, 2^15): exact but for
        // elements 2^-29 times smaller than it.
        uint32_t mx = 0;
#pragma unroll
        for (int ks = 0; ks < DP / 16; ++ks)
#pragma unroll
          for (int j = 0; j < 2; ++j)
            mx = max(mx, max(qf[nt][ks][j] & 0x7fffu, (qf[nt][ks][j] >> 16) & 0x7fffu));
        mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        const int e = static_cast<int>(mx >> 7);  // biased exponent of the largest
        const int up = e == 0 || e == 255 ? 0 : 141 - e;  // -113 .. 140
        // two factors, so that neither leaves the range of fp32
        const float f1 = __uint_as_float(static_cast<uint32_t>(127 + up / 2) << 23);
        const float f2 = __uint_as_float(static_cast<uint32_t>(127 + up - up / 2) << 23);
#pragma unroll
        for (int ks = 0; ks < DP / 16; ++ks)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float2 v = unpack2<MOE_BF16>(qf[nt][ks][j]);
            qf[nt][ks][j] = pack<false>(v.x * f1 * f2, v.y * f1 * f2);
          }
        const int u0 = __shfl_sync(0xffffffffu, up, (2 * tq) * 4), u1 = __shfl_sync(0xffffffffu, up, (2 * tq + 1) * 4);
        qscale[nt][0] = exp2f(static_cast<float>(-u0));
        qscale[nt][1] = exp2f(static_cast<float>(-u1));
      }
    }
    const float s2 = a.scale * kLog2e * (F8 && g.c.k_scale ? g.c.k_scale[kvh] : 1.0f);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) qscale[nt][0] *= s2, qscale[nt][1] *= s2;

#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int dm = 0; dm < S::kDm; ++dm)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[nt][dm][j] = 0.0f;
      m[nt][0] = m[nt][1] = -INFINITY;
      l[nt][0] = l[nt][1] = 0.0f;
    }

    // ----------------------------------------------------------- compute
    const int kr = (lane & 7) + 8 * ((lane >> 3) & 1);  // K row of this lane's matrix
    const int kc = lane >> 4;                           // and its chunk
    const int vr = F8 ? (lane & 7) + 8 * ((lane >> 3) & 1) : (lane & 7) + 8 * (lane >> 4);
    const int vc = F8 ? lane >> 4 : (lane >> 3) & 1;
    for (; u < u_end; u += u_step) {
      const uint64_t vm = vm0;
      cp_wait<kRing - 1>();
      __syncwarp();
      float s[S::kMt][NT][4];
#pragma unroll
      for (int mt = 0; mt < S::kMt; ++mt) {
        float acc2[NT][4];  // a second chain, where one m tile alone would wait on itself
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int j = 0; j < 4; ++j) s[mt][nt][j] = acc2[nt][j] = 0.0f;
        const uint32_t kslot = slot_at(0);
        if constexpr (!F8) {
#pragma unroll
          for (int ks = 0; ks < DP / 16; ++ks) {
            uint32_t f[4];
            ldsm4(f, kslot + swz<S::kCpr>(mt * 16 + kr, ks * 2 + kc));
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              mma<S::kBf16>((ks & 1) && S::kMt == 1 ? acc2[nt] : s[mt][nt], f[0], f[1], f[2], f[3], qf[nt][ks][0],
                            qf[nt][ks][1]);
          }
        } else {
#pragma unroll
          for (int ks = 0; ks < DP / 16; ks += 2) {
            uint32_t f[4];
            ldsm4(f, kslot + swz<S::kCpr>(mt * 16 + kr, ks + kc));
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              uint32_t a0, a1, a2, a3;
              e4m3_half4(f[2 * j], a0, a2);
              e4m3_half4(f[2 * j + 1], a1, a3);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                mma<false>(s[mt][nt], a0, a1, a2, a3, qf[nt][ks + j][0], qf[nt][ks + j][1]);
            }
          }
        }
        if constexpr (S::kMt == 1)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 4; ++j) s[mt][nt][j] += acc2[nt][j];
      }
      __syncwarp();
      issue(slot_at(0));
      if (++slot == kRing) slot = 0;

      // softmax step: new reference, weights, sums
      const bool whole = vm == (S::kU == 64 ? ~0ull : (1ull << (S::kU & 63)) - 1);
      uint32_t pf[S::kMt][NT][2];
      [[maybe_unused]] uint32_t pl[S::kMt][NT][2];
      float alpha[NT][2];
      bool moved = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int mt = 0; mt < S::kMt; ++mt)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float v = s[mt][nt][j] * (F8 && QT == MOE_BF16 ? qscale[nt][j & 1] : s2);
            if (!whole && !((vm >> (mt * 16 + gr + 8 * (j >> 1))) & 1)) v = -INFINITY;
            s[mt][nt][j] = v;
            mx[j & 1] = fmaxf(mx[j & 1], v);
          }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          mx[j] = fmaxf(mx[j], __shfl_xor_sync(0xffffffffu, mx[j], 4));
          mx[j] = fmaxf(mx[j], __shfl_xor_sync(0xffffffffu, mx[j], 8));
          mx[j] = fmaxf(mx[j], __shfl_xor_sync(0xffffffffu, mx[j], 16));
          // fp16 weights are kept 2^14 above their true value: the largest is
          // 2^14, and those down to 2^-28 of it are normal fp16 numbers.
          if (!S::kBf16) mx[j] -= 14.0f;
          const float mn = fmaxf(m[nt][j], mx[j]);
          const float ref = mn == -INFINITY ? 0.0f : mn;
          alpha[nt][j] = ex2(m[nt][j] - ref);
          moved |= m[nt][j] != mn;
          m[nt][j] = mn;
          l[nt][j] *= alpha[nt][j];
#pragma unroll
          for (int mt = 0; mt < S::kMt; ++mt)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const float w = ex2(s[mt][nt][2 * k + j] - ref);
              s[mt][nt][2 * k + j] = w;
              l[nt][j] += w;
            }
        }
#pragma unroll
        for (int mt = 0; mt < S::kMt; ++mt)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const float w0 = s[mt][nt][2 * k], w1 = s[mt][nt][2 * k + 1];
            const uint32_t hi = pack<S::kBf16>(w0, w1);
            pf[mt][nt][k] = movm_t(hi);
            if constexpr (S::kBf16) {
              // bf16 weights go as two terms (16 significant bits)
              const float2 f = unpack2<MOE_BF16>(hi);
              pl[mt][nt][k] = movm_t(pack<true>(w0 - f.x, w1 - f.y));
            }
          }
      }
      if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int dm = 0; dm < S::kDm; ++dm)
#pragma unroll
            for (int j = 0; j < 4; ++j) o[nt][dm][j] *= alpha[nt][j & 1];
      }

      cp_wait<kRing - 1>();
      __syncwarp();
      const uint32_t vslot = slot_at(0);
#pragma unroll
      for (int mt = 0; mt < S::kMt; ++mt) {
        if constexpr (!F8) {
#pragma unroll
          for (int dm = 0; dm < S::kDm; ++dm) {
            uint32_t f[4];
            ldsm4t(f, vslot + swz<S::kCpr>(mt * 16 + vr, dm * 2 + vc));
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              mma<S::kBf16>(o[nt][dm], f[0], f[1], f[2], f[3], pf[mt][nt][0], pf[mt][nt][1]);
            if constexpr (S::kBf16) {
              // A weight's low term is zero or of either sign: an infinite value times it
              // would turn the high term's infinity into NaN.  (0 to 2 % of a call's time:
              // 64 sequences up to 32k 328.5 us with and without, 100 of up to 700 over groups
              // of 20 heads of 64 15.25 against 14.97.)
#pragma unroll
              for (int i = 0; i < 4; ++i) f[i] = finite2(f[i]);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                mma<true>(o[nt][dm], f[0], f[1], f[2], f[3], pl[mt][nt][0], pl[mt][nt][1]);
            }
          }
        } else {
#pragma unroll
          for (int dm = 0; dm < S::kDm; dm += 2) {
            uint32_t f[4];
            ldsm4t(f, vslot + swz<S::kCpr>(mt * 16 + vr, dm + vc));
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              // 16-bit transposition leaves (token, token + 1) x (d, d + 1)
              // bytes in a register: pair the tokens of one d
              uint32_t a0, a1, a2, a3;
              e4m3_half4(__byte_perm(f[2 * j], 0, 0x3120), a0, a1);
              e4m3_half4(__byte_perm(f[2 * j + 1], 0, 0x3120), a2, a3);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                mma<false>(o[nt][dm + j], a0, a1, a2, a3, pf[mt][nt][0], pf[mt][nt][1]);
            }
          }
        }
      }
      __syncwarp();
      issue(slot_at(0));
      if (++slot == kRing) slot = 0;
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        l[nt][j] += __shfl_xor_sync(0xffffffffu, l[nt][j], 4);
        l[nt][j] += __shfl_xor_sync(0xffffffffu, l[nt][j], 8);
        l[nt][j] += __shfl_xor_sync(0xffffffffu, l[nt][j], 16);
      }
    if (solo) {
      // straight from the registers, two neighbouring columns at a time
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int h = nt * 8 + 2 * tq;  // this lane's first head
        float inv[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          inv[j] = l[nt][j] == 0.0f ? 0.0f : __fdiv_rn(vscale, l[nt][j]);
          if (gr == 0 && h + j < heads && a.lse)
            a.lse[static_cast<int64_t>(b) * a.n_q_heads + h0 + h + j] =
                l[nt][j] == 0.0f ? -INFINITY : (m[nt][j] + log2f(l[nt][j])) * kLn2;
        }
        uint16_t* out = static_cast<uint16_t*>(a.out) + b * a.out_seq_stride + (h0 + h) * a.out_head_stride;
#pragma unroll
        for (int dm = 0; dm < S::kDm; ++dm) {
          const float* v = o[nt][dm];
          if constexpr (F8) {
            // rows 2 gr and 2 gr + 1 of either head
            const int d = dm * 16 + 2 * gr;
#pragma unroll
            for (int j = 0; j < 2; ++j)
              if (h + j < heads && d < D)
                *reinterpret_cast<uint32_t*>(out + j * a.out_head_stride + d) =
                    pack<QT == MOE_BF16>(v[j] * inv[j], v[2 + j] * inv[j]);
          } else {
            // rows gr and gr + 8: an even row's lane takes both rows of the first
            // head, the odd one's both of the second
            const int odd = gr & 1, d = dm * 16 + (gr & ~1);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const float x = v[2 * k] * inv[0], y = v[2 * k + 1] * inv[1];
              const float got = __shfl_xor_sync(0xffffffffu, odd ? x : y, 4);
              if (h + odd < heads && d + 8 * k < D)
                *reinterpret_cast<uint32_t*>(out + odd * a.out_head_stride + d + 8 * k) =
                    odd ? pack<QT == MOE_BF16>(got, y) : pack<QT == MOE_BF16>(x, got);
            }
          }
        }
      }
    }
    }

    // ------------------------------------------------ the four warps meet
    if (!solo) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j)
        if (gr == 0) {
          s_m[warp][nt * 8 + 2 * tq + j] = m[nt][j];
          s_l[warp][nt * 8 + 2 * tq + j] = l[nt][j];
        }
    const bool split = ub > kVoid || ue < nb;
    constexpr int kQuads = DP / 4;
    const int part = cta - (split ? ln.owner(seg_start + kVoid) : cta);
    const int my_slot = (at0 + cta) * 2 + (part == 0 ? 1 : 0);
    // this CTA's share of the segment's column quads, and the heads it touches
    const int all = heads * kQuads, per = TEAM ? (all + S::kTeam - 1) / S::kTeam : all;
    const int e_lo = min(rank * per, all), e_hi = min(e_lo + per, all);
    auto holds = [&](int h) { return h * kQuads < e_hi && (h + 1) * kQuads > e_lo; };
    // statistics of a slot (teams: one copy per rank, written and read by that rank)
    auto stat = [&](int sl) { return reinterpret_cast<float2*>(stats) + (static_cast<int64_t>(sl) * S::kTeam + rank) * 16; };
    auto quad = [&](int sl, int e) {
      return reinterpret_cast<float4*>(parts) + static_cast<int64_t>(sl) * (S::kHeads * kQuads) + e;
    };
    // One column quad in sum: the finished output, or a part in `sl`.
    auto finish = [&](int e, float4 v, float ref, float lsum) {
      const int h = e / kQuads, d = (e % kQuads) * 4;
      const float inv = lsum == 0.0f ? 0.0f : __fdiv_rn(vscale, lsum);
      if (d == 0 && a.lse)
        a.lse[static_cast<int64_t>(b) * a.n_q_heads + h0 + h] =
            lsum == 0.0f ? -INFINITY : (ref + log2f(lsum)) * kLn2;
      if (d >= D) return;
      uint16_t* out = static_cast<uint16_t*>(a.out) + b * a.out_seq_stride +
                      static_cast<int64_t>(h0 + h) * a.out_head_stride + d;
      *reinterpret_cast<uint2*>(out) = make_uint2(pack<QT == MOE_BF16>(v.x * inv, v.y * inv),
                                                  pack<QT == MOE_BF16>(v.z * inv, v.w * inv));
    };
    auto emit = [&](bool final, int sl, int e, float4 v, float ref, float lsum) {
      if (final) {
        finish(e, v, ref, lsum);
      } else {
        *quad(sl, e) = v;
        if (TEAM || e % kQuads == 0) stat(sl)[e / kQuads] = make_float2(ref, lsum);
      }
    };
    // One column quad of a head over the CTA's four warps, and the head's
    // reference and sum.
    auto four_warps = [&](int h, auto quad_at, float2& ml) {
      ml.x = s_m[0][h];
#pragma unroll
      for (int w = 1; w < kWarps; ++w) ml.x = fmaxf(ml.x, s_m[w][h]);
      const float ref = ml.x == -INFINITY ? 0.0f : ml.x;
      float4 v = make_float4(0, 0, 0, 0);
      ml.y = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float f = ex2(s_m[w][h] - ref);
        const float4 x = *reinterpret_cast<const float4*>(quad_at(w));
        v.x = fmaf(f, x.x, v.x);
        v.y = fmaf(f, x.y, v.y);
        v.z = fmaf(f, x.z, v.z);
        v.w = fmaf(f, x.w, v.w);
        ml.y = fmaf(f, s_l[w][h], ml.y);
      }
      return v;
    };
    // Combine `count` partial results in order: stat_of(k, h) gives part k's
    // (reference, sum) of a head, quad_of(k, e) its column quad e.  Few columns
    // are shared out over the threads by parts as well.
    auto combine = [&](int count, bool final, int sl, auto stat_of, auto quad_of) {
      for (int e = tid; e < count * S::kHeads; e += kThreads) {
        const float2 ml = holds(e % S::kHeads) ? stat_of(e / S::kHeads, e % S::kHeads) : make_float2(-INFINITY, 0.0f);
        cb_s.w[e / S::kHeads][e % S::kHeads] = ml.x;
        cb_s.lp[e / S::kHeads][e % S::kHeads] = ml.y;
      }
      __syncthreads();
      {
        // kThreads / kHeads neighbouring lanes per head
        constexpr int kPer = kThreads / S::kHeads;
        const int h = tid / kPer, sub = tid % kPer;
        float mm = -INFINITY;
        for (int k = sub; k < count; k += kPer) mm = fmaxf(mm, cb_s.w[k][h]);
#pragma unroll
        for (int o = 1; o < kPer; o <<= 1) mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, o));
        const float ref = mm == -INFINITY ? 0.0f : mm;
        float lsum = 0.0f;
        for (int k = sub; k < count; k += kPer) {
          const float f = ex2(cb_s.w[k][h] - ref);
          cb_s.w[k][h] = f;
          lsum = fmaf(f, cb_s.lp[k][h], lsum);
        }
#pragma unroll
        for (int o = 1; o < kPer; o <<= 1) lsum += __shfl_xor_sync(0xffffffffu, lsum, o);
        if (sub == 0) {
          cb_s.m[h] = mm;
          cb_s.l[h] = lsum;
        }
      }
      __syncthreads();
      const int cols = max(e_hi - e_lo, 1);
      const int ng = max(1, min(kThreads / cols, count));  // threads per column quad
      const int gi = ng > 1 ? tid / cols : 0, e0 = ng > 1 ? tid - gi * cols : tid;
      // kQ quads by kK parts in flight per thread, as registers allow (32 loads
      // in flight spilled and cost 1 to 4 % over all)
      constexpr int kFew = S::kHeads * kQuads / (TEAM ? S::kTeam : 1) / kThreads;
      constexpr int kFit = S::kCtas > 2 ? 8 : 16;
      constexpr int kQ = kFew < 1 ? 1 : kFew > 4 ? 4 : kFew, kK = kFit / kQ < 16 ? kFit / kQ : 16;
      for (int eb = e_lo + e0; eb < e_hi; eb += kQ * kThreads) {
        float4 v[kQ];
#pragma unroll
        for (int i = 0; i < kQ; ++i) v[i] = make_float4(0, 0, 0, 0);
        if (gi < ng)
          for (int k0 = gi; k0 < count; k0 += kK * ng) {
            float4 x[kK][kQ];
#pragma unroll
            for (int k = 0; k < kK; ++k)
#pragma unroll
              for (int i = 0; i < kQ; ++i) {
                x[k][i] = make_float4(0, 0, 0, 0);
                if (k0 + k * ng < count && eb + i * kThreads < e_hi) x[k][i] = quad_of(k0 + k * ng, eb + i * kThreads);
              }
#pragma unroll
            for (int k = 0; k < kK; ++k)
#pragma unroll
              for (int i = 0; i < kQ; ++i) {
                const float f = k0 + k * ng < count ? cb_s.w[k0 + k * ng][((eb + i * kThreads) / kQuads) % S::kHeads] : 0.0f;
                v[i].x = fmaf(f, x[k][i].x, v[i].x);
                v[i].y = fmaf(f, x[k][i].y, v[i].y);
                v[i].z = fmaf(f, x[k][i].z, v[i].z);
                v[i].w = fmaf(f, x[k][i].w, v[i].w);
              }
          }
#pragma unroll
        for (int i = 0; i < kQ; ++i) {
          const int e = eb + i * kThreads, h = e / kQuads;
          if (ng > 1) {
            if (i == 0) cb_x[tid] = v[0];
          } else if (e < e_hi) {
            emit(final, sl, e, v[i], cb_s.m[h], cb_s.l[h]);
          }
        }
      }
      if (ng > 1) {
        __syncthreads();
        if (tid < e_hi - e_lo) {
          float4 v = cb_x[tid];
          for (int j = 1; j < ng; ++j) {
            const float4 x = cb_x[j * cols + tid];
            v.x += x.x;
            v.y += x.y;
            v.z += x.z;
            v.w += x.w;
          }
          const int h = (e_lo + tid) / kQuads;
          emit(final, sl, e_lo + tid, v, cb_s.m[h], cb_s.l[h]);
        }
      }
    };

    if constexpr (TEAM) {
      // Every warp's output to its ring; the CTA's four in sum to the ranks
      // that hold the columns; there the eight ranks' in sum.
      float* mine = reinterpret_cast<float*>(smem + warp * S::kRingBytes);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int dm = 0; dm < S::kDm; ++dm)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int d = dm * 16 + (F8 ? 2 * gr + (j >> 1) : gr + 8 * (j >> 1));
            mine[(nt * 8 + 2 * tq + (j & 1)) * S::kPart + d] = o[nt][dm][j];
          }
      float4* got = reinterpret_cast<float4*>(smem + S::kMergeAt);          // [rank][kShare]
      float2* got_ml = reinterpret_cast<float2*>(got + S::kTeam * S::kShare);  // [rank][16]
      // the ranks run, and are done with what they received before
      if (again) cluster_arrive();
      again = true;
      cluster_wait();
      __syncthreads();
      for (int e = tid; e < all; e += kThreads) {
        const int h = e / kQuads;
        float2 ml;
        const float4 v = four_warps(h, [&](int w) {
          return reinterpret_cast<const float*>(smem + w * S::kRingBytes) + h * S::kPart + (e % kQuads) * 4;
        }, ml);
        const int to = e / per;
        st_rank4(at_rank(got + rank * S::kShare + (e - to * per), to), v);
        st_rank2(at_rank(got_ml + rank * 16 + h, to), ml);
      }
      cluster_arrive();
      cluster_wait();
      for (int e = e_lo + tid; e < e_hi; e += kThreads) {
        const int h = e / kQuads;
        float mm = got_ml[h].x;
#pragma unroll
        for (int r = 1; r < S::kTeam; ++r) mm = fmaxf(mm, got_ml[r * 16 + h].x);
        const float ref = mm == -INFINITY ? 0.0f : mm;
        float4 v = make_float4(0, 0, 0, 0);
        float lsum = 0.0f;
#pragma unroll
        for (int r = 0; r < S::kTeam; ++r) {
          const float2 ml = got_ml[r * 16 + h];
          const float4 x = got[r * S::kShare + e - e_lo];
          const float f = ex2(ml.x - ref);
          v.x = fmaf(f, x.x, v.x);
          v.y = fmaf(f, x.y, v.y);
          v.z = fmaf(f, x.z, v.z);
          v.w = fmaf(f, x.w, v.w);
          lsum = fmaf(f, ml.y, lsum);
        }
        emit(!split, my_slot, e, v, mm, lsum);
      }
    } else {
      constexpr int kPasses = DP / S::kCols, kPq = S::kCols / 4;
#pragma unroll
      for (int pass = 0; pass < kPasses; ++pass) {
        if (pass) __syncthreads();
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int dm = 0; dm < S::kCols / 16; ++dm)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int d = dm * 16 + (F8 ? 2 * gr + (j >> 1) : gr + 8 * (j >> 1));
              merge[(warp * S::kHeads + nt * 8 + 2 * tq + (j & 1)) * S::kPitch + d] =
                  o[nt][pass * (S::kCols / 16) + dm][j];
            }
        __syncthreads();
        for (int i = tid; i < heads * kPq; i += kThreads) {
          const int h = i / kPq, dc = (i % kPq) * 4;
          float2 ml;
          const float4 v = four_warps(h, [&](int w) { return merge + (w * S::kHeads + h) * S::kPitch + dc; }, ml);
          emit(!split, my_slot, h * kQuads + (pass * S::kCols + dc) / 4, v, ml.x, ml.y);
        }
      }
    }

    // --------------------------------------- parts of other workers join
    if (split) {
      const int first = at0 + cta - part;  // the segment's first worker's slots
      const int n_parts = ln.owner(seg_start + nb - 1) + at0 - first + 1;
      // Arrive at a counter; true for the whole CTA if it is the last of n.
      // (release and acquire by one thread; the barriers extend them to the CTA)
      auto arrive = [&](uint32_t* counter, int n) {
        __syncthreads();
        if (tid == 0) {
          uint32_t was;
          asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(was) : "l"(counter) : "memory");
          s_flag = was == static_cast<uint32_t>(n - 1);
          if (s_flag) *counter = 0u;  // for the next launch
        }
        __syncthreads();
        return s_flag != 0;
      };
      // Join parts from, from + step, ... (count of them) into the first one's
      // slot, or into the output.
      auto join = [&](int from, int step, int count, bool final) {
        auto slot_of = [&](int k) { return (first + from + k * step) * 2 + (from + k * step == 0 ? 1 : 0); };
        combine(count, final, slot_of(0), [&](int k, int h) { return __ldcg(stat(slot_of(k)) + h); },
                [&](int k, int e) { return __ldcg(quad(slot_of(k), e)); });
      };
      if constexpr (TEAM) {
        // every rank joins its own columns of the teams' slots
        if (arrive(counters + first * 8 + rank, n_parts)) join(0, 1, n_parts, true);
      } else {
        const int n_groups = (n_parts + S::kJoin - 1) / S::kJoin, from = part / S::kJoin * S::kJoin;
        const int count = min(S::kJoin, n_parts - from);
        uint32_t* at = counters + (first + from) * 4 + (from == 0 ? 1 : 0);
        if (arrive(at, count)) {
          join(from, 1, count, n_groups == 1);
          if (n_groups > 1 && arrive(counters + first * 4 + 2, n_groups)) join(0, S::kJoin, n_groups, true);
        }
      }
    }
    if constexpr (!TEAM) __syncthreads();  // the merge buffer and the statistics are free again
    }

    // ---------------------------------------------------- the next segment
    p += ue - ub;
    if (p < p_end && seg == segs - 1 && ue == nb) {
      prefix += nb;
      ++b;
      len = clamp_len(a.seq_lens[b]);
      lo = low(len);
      nb = places_of(lo, len);
    }
  }
  cp_wait<0>();
  if (TEAM || ln.chunks == ln.n) break;
  // the next small chunk, if any is left; the last CTA to find none clears the count
  __syncthreads();
  if (tid == 0) s_flag = ln.n + static_cast<int>(atomicAdd(counters + kMaxChunks * 4 + blockIdx.y, 1u));
  __syncthreads();
  cta = s_flag;
  if (cta >= ln.chunks) {
    if (tid == 0 && cta == ln.chunks + ln.n - 1) counters[kMaxChunks * 4 + blockIdx.y] = 0u;
    break;
  }
  }
}

template <int QT, bool F8, int DP, int NT, bool TEAM>
moe_status_t launch(const AttnArgs& g, cudaStream_t st) {
  using S = Shape<QT, F8, DP, NT, TEAM>;
  const auto kernel = paged_attention_kernel<QT, F8, DP, NT, TEAM>;
  // A kernel's shared-memory limit is raised and its grid found once per
  // device: asking costs microseconds.
  static std::atomic<int> grid_of[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return check_launch("cudaGetDevice");
  if (dev >= 64) return set_error(MOE_ERR_UNSUPPORTED, "device number above 63");
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(S::kThreads);
  cfg.dynamicSmemBytes = S::kSmem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = S::kTeam;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = TEAM ? attr : attr + 1;
  int grid = grid_of[dev].load(std::memory_order_acquire);
  if (!grid) {
    if (raise_smem_limit(kernel, S::kSmem) != cudaSuccess) return check_launch("paged_attention_kernel attributes");
    if (TEAM) {
      int teams = 0;
      cfg.gridDim = dim3(S::kTeam);
      cfg.numAttrs = 1;
      if (cudaOccupancyMaxActiveClusters(&teams, kernel, &cfg) != cudaSuccess)
        return check_launch("paged_attention_kernel occupancy");
      if (teams < 1) return set_error(MOE_ERR_UNSUPPORTED, "the device cannot hold a cluster of the kernel");
      grid = (teams < kMaxTeams ? teams : kMaxTeams) * S::kTeam;
    } else {
      grid = S::kCtas * (sm_count() < kMaxSms ? sm_count() : kMaxSms);
    }
    grid_of[dev].store(grid, std::memory_order_release);
  }
  cfg.gridDim = dim3(static_cast<unsigned>(grid / (g.sides * g.kv_sides)), static_cast<unsigned>(g.sides * g.kv_sides));
  cfg.numAttrs = TEAM ? 2 : 1;
  if (cudaLaunchKernelEx(&cfg, kernel, g) != cudaSuccess) return check_launch("paged_attention_kernel");
  stat_kernels(1);
  return MOE_OK;
}

template <int QT, bool F8, bool TEAM>
moe_status_t pick(const AttnArgs& g, int nt, cudaStream_t st) {
  const int D = g.c.head_dim;
  if (nt == 1) {
    if (D <= 64) return launch<QT, F8, 64, 1, TEAM>(g, st);
    if (D <= 128) return launch<QT, F8, 128, 1, TEAM>(g, st);
    return launch<QT, F8, 256, 1, TEAM>(g, st);
  }
  return D <= 64 ? launch<QT, F8, 64, 2, TEAM>(g, st) : launch<QT, F8, 128, 2, TEAM>(g, st);
}

template <bool TEAM>
moe_status_t pick(const AttnArgs& g, int nt, cudaStream_t st) {
  const bool f8 = g.c.dtype == MOE_E4M3;
  if (g.a.dtype == MOE_BF16) return f8 ? pick<MOE_BF16, true, TEAM>(g, nt, st) : pick<MOE_BF16, false, TEAM>(g, nt, st);
  return f8 ? pick<MOE_F16, true, TEAM>(g, nt, st) : pick<MOE_F16, false, TEAM>(g, nt, st);
}

}  // namespace

// One CTA per worker of the line (moe_attn.cu), or a team of CTAs (moe_attn_team.cu).
moe_status_t launch_attention_ctas(const AttnArgs& g, int nt, cudaStream_t st);
moe_status_t launch_attention_teams(const AttnArgs& g, int nt, cudaStream_t st);

}  // namespace moe
