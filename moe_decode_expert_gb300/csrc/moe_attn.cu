// moe_attn.cu — attention of one new token per sequence over a paged cache.
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
// Work is split evenly over the CTAs whatever the lengths: the (sequence,
// kv head, unit of U tokens) triples form one line, with kVoid empty places
// before each (sequence, kv head) for its fixed cost, and CTA c of n takes the
// c-th n-th of it (every CTA finds its place from seq_lens itself).  A (sequence,
// kv head) that ends up in several CTAs is joined by the last of them to arrive,
// in groups of kJoin parts and then over the groups, always in the same order:
// one launch, results independent of timing.
//
// A warp owns whole units: K and V of a unit are two slots of its own ring in
// shared memory, filled by cp.async two slots ahead; only a part's end meets
// at a CTA barrier.

#include <atomic>

#include "moe_common.cuh"
#include "moe_kv.h"

namespace moe {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kRing = 3;         // slots of a warp's ring
constexpr int kMaxCtas = 640;    // partial slots in the workspace: two per CTA
constexpr int kJoin = 16;        // parts joined by one CTA at a time
constexpr int kMaxGroups = (kMaxCtas + kJoin - 1) / kJoin;
constexpr int kMinUnits = 4;     // places of the line a CTA takes at least: one per warp
constexpr int kVoid = 4;         // places before a segment's units: its fixed cost, in units
constexpr int kSlotTarget = 8192;
constexpr int kCtas64 = 2;
constexpr int kCtas128 = 2;
constexpr int kCtas256 = 2;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// Workspace: control block, join counters [kMaxCtas][4], partial statistics
// [kMaxCtas * 2][16][2] fp32, partial outputs [kMaxCtas * 2][heads][DP] fp32.
constexpr size_t kCountersAt = 256;
constexpr size_t kStatsAt = kCountersAt + kMaxCtas * 4 * sizeof(uint32_t);
constexpr size_t kPartsAt = kStatsAt + kMaxCtas * 2 * 16 * 2 * sizeof(float);
static_assert(kPartsAt % 256 == 0, "partials are 256-byte aligned");

struct AttnArgs {
  moe_kv_cache_t c;
  moe_attention_t a;
  uint8_t* ws;
  int32_t chunks;  // head chunks of a kv head
  int32_t hpc;     // query heads of a chunk (<= 8 * NT)
  int32_t group;   // query heads of a kv head
  int32_t max_len; // max_pages * page_size, saturated
  // token / page_size = umulhi(token, page_mul) >> page_shift (page_mul 0: page_size 1)
  uint32_t page_mul;
  int32_t page_shift;
  int32_t blocks;  // page_size % 16 == 0: 16 neighbouring tokens share a page
};

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

// Two e4m3 values (low 16 bits) -> two fp16 values, exact.
__device__ __forceinline__ uint32_t e4m3_half2(uint32_t two) {
  uint32_t r;
  asm("{\n\t.reg .b16 t;\n\tcvt.u16.u32 t, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}" : "=r"(r) : "r"(two));
  return r;
}

// The statistics of a join, in shared memory.
struct JoinSmem {
  float w[kMaxGroups > kJoin ? kMaxGroups : kJoin][16];
  float m[16], l[16];
};

// Everything of a kernel that does not depend on its place in the line.
template <int QT, bool F8, int DP, int NT>
struct Shape {
  static constexpr int kBytes = F8 ? 1 : 2;
  static constexpr int kFill = kSlotTarget / (DP * kBytes);
  static constexpr int kU = kFill < 16 ? 16 : kFill < 64 ? kFill : 64;  // tokens of a unit
  static constexpr int kCtas = DP == 256 ? kCtas256 : DP == 128 ? kCtas128 : kCtas64;  // CTAs of an SM
  static constexpr int kRow = DP * kBytes;                                            // bytes of a row
  static constexpr int kSlot = kU * kRow;
  static constexpr int kCpr = kRow / 16;   // 16-byte chunks of a row
  static constexpr int kMt = kU / 16;      // m tiles of a unit's scores
  static constexpr int kDm = DP / 16;      // m tiles of the output
  static constexpr int kHeads = 8 * NT;
  static constexpr int kCols = NT == 1 ? 64 : 32;  // output columns the warps merge at a time
  static constexpr int kPitch = kCols + 4;         // their fp32 pitch: conflict-free
  static constexpr bool kBf16 = !F8 && QT == MOE_BF16;  // type of the matrix products
  static constexpr int kMergeAt = kWarps * kRing * kSlot;
  static constexpr int kSmem = kMergeAt + kWarps * kHeads * kPitch * 4;
};

// Byte offset of 16-byte chunk c of row r in a slot: chunks are permuted so
// that 8 rows at one chunk column lie in 8 different bank groups.
template <int kCpr>
__device__ __forceinline__ uint32_t swz(int r, int c) {
  if constexpr (kCpr >= 8) return static_cast<uint32_t>(r * kCpr * 16 + ((c ^ (r & 7)) << 4));
  // rows of 64 bytes: two to a 128-byte line
  return static_cast<uint32_t>((r >> 1) * 128 + ((((r & 1) * 4 + c) ^ ((r >> 1) & 3)) << 4));
}

// The line of units: CTA c of n takes `each` of them, the first `more` CTAs one
// more.
struct Line {
  int total, n, each, more;
  __device__ __forceinline__ int start(int c) const { return each * c + min(c, more); }
  __device__ __forceinline__ int owner(int x) const {
    const int wide = more * (each + 1);
    return x < wide ? static_cast<int>(static_cast<unsigned>(x) / static_cast<unsigned>(each + 1))
                    : more + static_cast<int>(static_cast<unsigned>(x - wide) / static_cast<unsigned>(each));
  }
};

template <int QT, bool F8, int DP, int NT>
__global__ void __launch_bounds__(kThreads, (Shape<QT, F8, DP, NT>::kCtas)) paged_attention_kernel(AttnArgs g) {
  using S = Shape<QT, F8, DP, NT>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float s_m[kWarps][16], s_l[kWarps][16];
  __shared__ JoinSmem s_join;
  __shared__ int s_scan[kWarps], s_b, s_prefix, s_flag;

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

  // The line's length, then this CTA's share of it, then the sequence that
  // holds its start.  The first kThreads sequences stay in registers.
  const int segs = g.c.n_kv_heads * g.chunks;  // segments of a sequence
  const int u0 = tid < a.B ? places(tid) : 0;
  int sum = u0;
  for (int b = tid + kThreads; b < a.B; b += kThreads) sum += places(b);
  sum = __reduce_add_sync(0xffffffffu, sum);
  if (lane == 0) s_scan[warp] = sum;
  __syncthreads();
  Line ln;
  ln.total = (s_scan[0] + s_scan[1] + s_scan[2] + s_scan[3]) * segs;
  ln.n = min((ln.total + kMinUnits - 1) / kMinUnits, static_cast<int>(gridDim.x));
  const int cta = blockIdx.x;
  if (cta >= ln.n) return;
  ln.each = static_cast<int>(static_cast<unsigned>(ln.total) / static_cast<unsigned>(ln.n));
  ln.more = ln.total - ln.each * ln.n;
  int p = ln.start(cta);
  const int p_end = ln.start(cta + 1);
  int before = 0;
  for (int b0 = 0;; b0 += kThreads) {
    const int b = b0 + tid;
    const int u = b0 == 0 ? u0 : b < a.B ? places(b) : 0;
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
      s_b = b;
      s_prefix = ex;
    }
    __syncthreads();
    if (s_b >= 0) break;
  }
  int b = s_b, prefix = s_prefix;
  int len = clamp_len(a.seq_lens[b]), lo = low(len), nb = places_of(lo, len);

  const uint32_t ring = smem_u32(smem + warp * (kRing * S::kSlot));
  float* merge = reinterpret_cast<float*>(smem + S::kMergeAt);
  const int D = g.c.head_dim;

  // ------------------------------------------------------------------ loads
  // This warp's units are at places p + warp, p + warp + kWarps, ... of the line.
  // Their loads run ahead of the arithmetic, across segment ends: a cursor
  // walks the units to load.
  constexpr int kRr = (S::kU + 31) / 32;  // rows of a unit per lane
  constexpr int kStep = 32 / S::kCpr;     // rows of one pass of the warp
  const int col = lane % S::kCpr, row0 = lane / S::kCpr;
  const bool col_in = col * 16 < D * S::kBytes;
  int left = (p_end - p - warp + kWarps - 1) / kWarps;  // places still to look at
  if (p_end - p <= warp) left = 0;
  int cb = b, cseg = (p - prefix * segs) / nb, cu = p - prefix * segs - cseg * nb + warp;
  int clen = len, clo = lo, cnb = nb;
  int next_len = cb + 1 < a.B ? a.seq_lens[cb + 1] : 0;
  auto settle = [&]() {  // bring the cursor's place into its segment
    while (cu >= cnb) {
      cu -= cnb;
      if (++cseg == segs) {
        cseg = 0;
        ++cb;
        clen = clamp_len(next_len);
        clo = low(clen);
        cnb = places_of(clo, clen);
        next_len = cb + 1 < a.B ? a.seq_lens[cb + 1] : 0;
      }
    }
  };
  auto page_of = [&](int tok) {
    return g.page_mul ? static_cast<int>(__umulhi(static_cast<uint32_t>(tok), g.page_mul) >> g.page_shift) : tok;
  };
  // Where the rows of a unit are: lane l holds rows l (and l + 32); the unit
  // looked up (n...) is the one after the unit being loaded.
  int page[kRr], off[kRr], npage[kRr], noff[kRr];
  int kvh_l = 0, nkvh = 0;  // their kv heads
  bool have = false, nhave = false, nvalid[kRr];
  auto look_up = [&]() {
    nhave = false;
    while (left > 0 && !nhave) {
      --left;
      settle();
      nhave = cu >= kVoid;
      if (!nhave) cu += kWarps;
    }
#pragma unroll
    for (int r = 0; r < kRr; ++r) npage[r] = -1, noff[r] = 0, nvalid[r] = false;
    if (!nhave) return;
    nkvh = g.chunks == 1 ? cseg : cseg / g.chunks;
    const int32_t* table = a.block_table + cb * a.table_stride;
#pragma unroll
    for (int r = 0; r < kRr; ++r) {
      const int row = lane + 32 * r;
      // unsigned: the last unit may reach past the largest int
      const uint32_t tok = static_cast<uint32_t>(clo / S::kU + cu - kVoid) * S::kU + row;
      const uint32_t first = g.blocks ? tok | 15u : tok, last = g.blocks ? tok & ~15u : tok;
      nvalid[r] = row < S::kU && tok >= static_cast<uint32_t>(clo) && tok < static_cast<uint32_t>(clen);
      // rows beside those that count are placed too where a block shares a page
      if (row < S::kU && first >= static_cast<uint32_t>(clo) && last < static_cast<uint32_t>(clen)) {
        const int idx = page_of(static_cast<int>(tok));
        noff[r] = static_cast<int>(tok) - idx * g.c.page_size;
        npage[r] = table[idx];
        if (static_cast<uint32_t>(npage[r]) >= static_cast<uint32_t>(g.c.n_pages)) {
          npage[r] = -1;
          report_error(ctrl, kDevBadPage, static_cast<uint32_t>(cb));
        }
      }
    }
    cu += kWarps;
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
    const int64_t ps = keys ? g.c.k_page_stride : g.c.v_page_stride;
    const int64_t ts = keys ? g.c.k_token_stride : g.c.v_token_stride;
    const int64_t hs = keys ? g.c.k_head_stride : g.c.v_head_stride;
    const uint8_t* at = static_cast<const uint8_t*>(keys ? g.c.k : g.c.v) + kvh_l * hs * S::kBytes + col * 16;
    if (g.blocks) {
      // 16 rows on one page: one address, then steps
#pragma unroll
      for (int bl = 0; bl < S::kU / 16; ++bl) {
        const int pg = __shfl_sync(0xffffffffu, page[bl >> 1], (bl & 1) * 16);
        const int of = __shfl_sync(0xffffffffu, off[bl >> 1], (bl & 1) * 16);
        const uint32_t bits = col_in ? static_cast<uint32_t>(vm >> (bl * 16 + row0)) : 0u;
        const uint8_t* src = at + (max(pg, 0) * ps + (of + row0) * ts) * S::kBytes;
#pragma unroll
        for (int i = 0; i < 16 / kStep; ++i)
          cp16_or_zero(slot + swz<S::kCpr>(bl * 16 + i * kStep + row0, col), src + i * kStep * ts * S::kBytes,
                       ((bits >> (i * kStep)) & 1u) << 4);
      }
    } else {
#pragma unroll
      for (int i = 0; i < S::kU / kStep; ++i) {
        const int r = i * kStep + row0;
        const int pg = __shfl_sync(0xffffffffu, page[i * kStep / 32], r & 31);
        const int of = __shfl_sync(0xffffffffu, off[i * kStep / 32], r & 31);
        const bool in = ((vm >> r) & 1) && col_in;
        cp16_or_zero(slot + swz<S::kCpr>(r, col), at + (in ? (pg * ps + of * ts) * S::kBytes : 0), in ? 16u : 0u);
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
  look_up();
#pragma unroll 1
  for (int k = 0; k < kRing; ++k) issue(slot_at(k));  // K, V, K: vm0 is the first unit's mask, vm1 the second's
  int turn = warp;      // line places before this warp's next unit, from p on

  while (p < p_end) {
    // ------------------------------------------ the part at places [ub, ue)
    const int local = p - prefix * segs;
    const int seg = static_cast<int>(static_cast<unsigned>(local) / static_cast<unsigned>(nb));
    const int ub = local - seg * nb;
    const int ue = min(nb, ub + p_end - p);
    const int seg_start = p - ub;
    if (ue <= kVoid) break;  // the share ends before the segment's first unit: it is the next CTA's
    const int kvh = g.chunks == 1 ? seg : seg / g.chunks, chunk = seg - kvh * g.chunks;
    const int heads = min(g.hpc, g.group - chunk * g.hpc);  // query heads of this segment
    const int h0 = kvh * g.group + chunk * g.hpc;
    if (tid == 0) {
      const int raw = a.seq_lens[b];
      if (raw < 0 || raw > g.max_len) report_error(ctrl, kDevBadLength, static_cast<uint32_t>(b));
    }

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

    float o[NT][S::kDm][4];
    float m[NT][2], l[NT][2];  // a head's reference (log2) and this lane's share of its sum
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
    for (; turn < ue - ub; turn += kWarps) {
      if (ub + turn < kVoid) continue;
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
              const uint32_t a0 = e4m3_half2(f[2 * j]), a2 = e4m3_half2(f[2 * j] >> 16);
              const uint32_t a1 = e4m3_half2(f[2 * j + 1]), a3 = e4m3_half2(f[2 * j + 1] >> 16);
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
            float v = s[mt][nt][j] * s2;
            if constexpr (F8 && QT == MOE_BF16) v *= qscale[nt][j & 1];
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
            for (int nt = 0; nt < NT; ++nt) {
              mma<S::kBf16>(o[nt][dm], f[0], f[1], f[2], f[3], pf[mt][nt][0], pf[mt][nt][1]);
              if constexpr (S::kBf16) mma<true>(o[nt][dm], f[0], f[1], f[2], f[3], pl[mt][nt][0], pl[mt][nt][1]);
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
              const uint32_t x = __byte_perm(f[2 * j], 0, 0x3120), y = __byte_perm(f[2 * j + 1], 0, 0x3120);
              const uint32_t a0 = e4m3_half2(x), a1 = e4m3_half2(x >> 16);
              const uint32_t a2 = e4m3_half2(y), a3 = e4m3_half2(y >> 16);
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
    turn -= ue - ub;

    // ------------------------------------------------ the four warps meet
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float t = l[nt][j];
        t += __shfl_xor_sync(0xffffffffu, t, 4);
        t += __shfl_xor_sync(0xffffffffu, t, 8);
        t += __shfl_xor_sync(0xffffffffu, t, 16);
        if (gr == 0) {
          s_m[warp][nt * 8 + 2 * tq + j] = m[nt][j];
          s_l[warp][nt * 8 + 2 * tq + j] = t;
        }
      }
    const bool split = ub > kVoid || ue < nb;
    const float vscale = F8 && g.c.v_scale ? g.c.v_scale[kvh] : 1.0f;
    constexpr int kQuads = DP / 4;
    // Write one head's four columns: the finished output.
    auto finish = [&](int h, int d, float4 v, float lsum) {
      const float inv = (lsum == 0.0f ? 0.0f : __fdiv_rn(vscale, lsum));
      if (d >= D) return;
      uint16_t* out = static_cast<uint16_t*>(a.out) + b * a.out_seq_stride +
                      static_cast<int64_t>(h0 + h) * a.out_head_stride + d;
      *reinterpret_cast<uint2*>(out) = make_uint2(pack<QT == MOE_BF16>(v.x * inv, v.y * inv),
                                                  pack<QT == MOE_BF16>(v.z * inv, v.w * inv));
    };
    auto finish_lse = [&](int h, float ref, float lsum) {
      if (a.lse)
        a.lse[static_cast<int64_t>(b) * a.n_q_heads + h0 + h] =
            lsum == 0.0f ? -INFINITY : (ref + log2f(lsum)) * kLn2;
    };
    const int part = cta - (split ? ln.owner(seg_start + kVoid) : cta);
    const int role = part == 0 ? 1 : 0;
    const int my_slot = cta * 2 + role;
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
      for (int e = tid; e < heads * kPq; e += kThreads) {
        const int h = e / kPq, dc = (e % kPq) * 4, d = pass * S::kCols + dc;
        float mm = s_m[0][h];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) mm = fmaxf(mm, s_m[w][h]);
        const float ref = mm == -INFINITY ? 0.0f : mm;
        float4 v = make_float4(0, 0, 0, 0);
        float lsum = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float f = ex2(s_m[w][h] - ref);
          const float4 x = *reinterpret_cast<const float4*>(merge + (w * S::kHeads + h) * S::kPitch + dc);
          v.x = fmaf(f, x.x, v.x);
          v.y = fmaf(f, x.y, v.y);
          v.z = fmaf(f, x.z, v.z);
          v.w = fmaf(f, x.w, v.w);
          lsum = fmaf(f, s_l[w][h], lsum);
        }
        if (!split) {
          finish(h, d, v, lsum);
          if (d == 0) finish_lse(h, mm, lsum);
        } else {
          *reinterpret_cast<float4*>(parts + (static_cast<int64_t>(my_slot) * S::kHeads + h) * DP + d) = v;
          if (d == 0) {
            stats[(my_slot * 16 + h) * 2] = mm;
            stats[(my_slot * 16 + h) * 2 + 1] = lsum;
          }
        }
      }
    }

    // ------------------------------------------- parts of other CTAs join
    if (split) {
      const int first_cta = cta - part;
      const int n_parts = ln.owner(seg_start + nb - 1) - first_cta + 1;
      const int n_groups = (n_parts + kJoin - 1) / kJoin;
      // Join parts from, from + step, ... (count of them) into the first one's
      // slot, or finish the segment.
      auto join = [&](int from, int step, int count, bool final) {
        auto slot_of = [&](int k) {
          const int pt = from + k * step;
          return (first_cta + pt) * 2 + (pt == 0 ? 1 : 0);
        };
        for (int e = tid; e < count * 16; e += kThreads)
          s_join.w[e >> 4][e & 15] = (e & 15) < heads ? __ldcg(stats + (slot_of(e >> 4) * 16 + (e & 15)) * 2) : 0.0f;
        __syncthreads();
        if (tid < heads) {
          float mm = -INFINITY;
          for (int k = 0; k < count; ++k) mm = fmaxf(mm, s_join.w[k][tid]);
          const float ref = mm == -INFINITY ? 0.0f : mm;
          float lsum = 0.0f;
          for (int k = 0; k < count; ++k) {
            const float f = ex2(s_join.w[k][tid] - ref);
            s_join.w[k][tid] = f;
            lsum = fmaf(f, __ldcg(stats + (slot_of(k) * 16 + tid) * 2 + 1), lsum);
          }
          s_join.m[tid] = mm;
          s_join.l[tid] = lsum;
        }
        __syncthreads();
        for (int e = tid; e < heads * kQuads; e += kThreads) {
          const int h = e / kQuads, d = (e % kQuads) * 4;
          float4 v = make_float4(0, 0, 0, 0);
#pragma unroll 8
          for (int k = 0; k < count; ++k) {
            const float4 x = __ldcg(reinterpret_cast<const float4*>(
                parts + (static_cast<int64_t>(slot_of(k)) * S::kHeads + h) * DP + d));
            const float f = s_join.w[k][h];
            v.x = fmaf(f, x.x, v.x);
            v.y = fmaf(f, x.y, v.y);
            v.z = fmaf(f, x.z, v.z);
            v.w = fmaf(f, x.w, v.w);
          }
          if (final) {
            finish(h, d, v, s_join.l[h]);
            if (d == 0) finish_lse(h, s_join.m[h], s_join.l[h]);
          } else {
            *reinterpret_cast<float4*>(parts + (static_cast<int64_t>(slot_of(0)) * S::kHeads + h) * DP + d) = v;
          }
        }
        if (!final) {
          if (tid < heads) {
            stats[(slot_of(0) * 16 + tid) * 2] = s_join.m[tid];
            stats[(slot_of(0) * 16 + tid) * 2 + 1] = s_join.l[tid];
          }
        }
      };
      // Arrive at a counter; true for the whole CTA if it is the last of n.
      auto arrive = [&](uint32_t* counter, int n) {
        __threadfence();
        __syncthreads();
        if (tid == 0) {
          const uint32_t was = atomicAdd(counter, 1u);
          s_flag = was == static_cast<uint32_t>(n - 1);
          if (s_flag) *counter = 0u;  // for the next launch
          __threadfence();
        }
        __syncthreads();
        return s_flag != 0;
      };
      const int grp = part / kJoin, grp_first = grp * kJoin;
      const int grp_n = min(kJoin, n_parts - grp_first);
      uint32_t* at = counters + (first_cta + grp_first) * 4;
      if (arrive(at + (grp_first == 0 ? 1 : 0), grp_n)) {
        join(grp_first, 1, grp_n, n_groups == 1);
        if (n_groups > 1) {
          uint32_t* top = counters + first_cta * 4 + 2;
          if (arrive(top, n_groups)) join(0, kJoin, n_groups, true);
        }
      }
    }
    __syncthreads();  // the merge buffer and the statistics are free again

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
}

template <int QT, bool F8, int DP, int NT>
moe_status_t launch(const AttnArgs& g, cudaStream_t st) {
  using S = Shape<QT, F8, DP, NT>;
  const auto kernel = paged_attention_kernel<QT, F8, DP, NT>;
  // the limit of a kernel is raised once per device: asking costs microseconds
  static std::atomic<uint64_t> raised{0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return check_launch("cudaGetDevice");
  const uint64_t bit = dev < 64 ? 1ull << dev : 0ull;
  if (!(raised.load(std::memory_order_acquire) & bit)) {
    if (raise_smem_limit(kernel, S::kSmem) != cudaSuccess) return check_launch("paged_attention_kernel attributes");
    raised.fetch_or(bit, std::memory_order_release);
  }
  const int fit = S::kCtas * sm_count(), grid = fit < kMaxCtas ? fit : kMaxCtas;
  if (launch_pdl(kernel, dim3(static_cast<unsigned>(grid)), dim3(kThreads), S::kSmem, st, g) != cudaSuccess)
    return check_launch("paged_attention_kernel");
  stat_kernels(1);
  return MOE_OK;
}

template <int QT, bool F8>
moe_status_t dispatch(const AttnArgs& g, int nt, cudaStream_t st) {
  const int D = g.c.head_dim;
  if (nt == 1) {
    if (D <= 64) return launch<QT, F8, 64, 1>(g, st);
    if (D <= 128) return launch<QT, F8, 128, 1>(g, st);
    return launch<QT, F8, 256, 1>(g, st);
  }
  if (D <= 64) return launch<QT, F8, 64, 2>(g, st);
  if (D <= 128) return launch<QT, F8, 128, 2>(g, st);
  return launch<QT, F8, 256, 2>(g, st);
}

// n tiles of 8 heads of a segment: two when a group has more than 8 heads.
int n_tiles(int group) { return group > 8 ? 2 : 1; }
int padded_dim(int D) { return D <= 64 ? 64 : D <= 128 ? 128 : 256; }

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" size_t moe_attention_workspace_bytes(const moe_kv_cache_t* cache, int32_t n_q_heads) {
  if (!cache || cache->n_kv_heads < 1 || cache->head_dim < 1 || cache->head_dim > 256 || n_q_heads < 1 ||
      n_q_heads % cache->n_kv_heads)
    return 0;
  const int nt = n_tiles(n_q_heads / cache->n_kv_heads);
  return kPartsAt + static_cast<size_t>(kMaxCtas) * 2 * 8 * nt * padded_dim(cache->head_dim) * sizeof(float);
}

extern "C" moe_status_t moe_paged_attention(const moe_kv_cache_t* cache, const moe_attention_t* a, void* ws,
                                            size_t ws_bytes, void* stream) {
  if (!a) return set_error(MOE_ERR_INVALID_ARG, "moe_attention_t is NULL");
  if (moe_status_t s = check_cache(cache, a->dtype)) return s;
  if (a->B < 0 || a->n_q_heads < 1 || a->max_pages < 0 || a->window < 0)
    return set_error(MOE_ERR_INVALID_ARG, "B, max_pages and window must be >= 0 and n_q_heads >= 1");
  if (a->n_q_heads % cache->n_kv_heads)
    return set_error(MOE_ERR_INVALID_ARG, "n_q_heads must be a multiple of the cache's n_kv_heads");
  if (a->n_q_heads > 65536) return set_error(MOE_ERR_UNSUPPORTED, "too many heads");
  if (!ws || ws_bytes < moe_attention_workspace_bytes(cache, a->n_q_heads))
    return set_error(MOE_ERR_WORKSPACE, "workspace is NULL or has %zu bytes, %zu needed", ws_bytes,
                     moe_attention_workspace_bytes(cache, a->n_q_heads));
  if (reinterpret_cast<uintptr_t>(ws) % kWsAlign)
    return set_error(MOE_ERR_WORKSPACE, "workspace must be 256-byte aligned");
  if (a->B == 0) return MOE_OK;
  if (!a->q || !a->out || !a->seq_lens || (a->max_pages > 0 && !a->block_table))
    return set_error(MOE_ERR_INVALID_ARG, "q / out / seq_lens / block_table is NULL");
  if (!ptr16(a->q) || !ptr16(a->out)) return set_error(MOE_ERR_INVALID_ARG, "q / out is not 16-byte aligned");
  if ((reinterpret_cast<uintptr_t>(a->block_table) | reinterpret_cast<uintptr_t>(a->seq_lens) |
       reinterpret_cast<uintptr_t>(a->lse)) & 3u)
    return set_error(MOE_ERR_INVALID_ARG, "block_table, seq_lens or lse is not 4-byte aligned");
  if ((a->q_seq_stride | a->q_head_stride | a->out_seq_stride | a->out_head_stride) & 7)
    return set_error(MOE_ERR_UNSUPPORTED, "strides of q and out must be multiples of 16 bytes");
  AttnArgs g;
  g.c = *cache;
  g.a = *a;
  g.ws = static_cast<uint8_t*>(ws);
  g.group = a->n_q_heads / cache->n_kv_heads;
  const int nt = n_tiles(g.group);
  g.chunks = (g.group + 8 * nt - 1) / (8 * nt);
  g.hpc = (g.group + g.chunks - 1) / g.chunks;
  // Tokens are 32-bit numbers; units round a length up by less than 64.
  const int64_t cap = static_cast<int64_t>(a->max_pages) * cache->page_size;
  // The line of units is counted in 32 bits.
  if (cap / 16 + 2 + kVoid > 0x7fffffffll / g.chunks / cache->n_kv_heads / a->B)
    return set_error(MOE_ERR_UNSUPPORTED, "batch * kv heads * table tokens too large");
  // ceil(2^(31 + s) / page_size), s = ceil(log2 page_size): exact for 31-bit tokens
  int sh = 0;
  while ((1ll << sh) < cache->page_size) ++sh;
  g.page_mul = sh ? static_cast<uint32_t>(((1ull << (31 + sh)) + cache->page_size - 1) / cache->page_size) : 0u;
  g.page_shift = sh - 1;
  g.blocks = cache->page_size % 16 == 0;
  g.max_len = static_cast<int32_t>(cap < 0x7fffff00 ? cap : 0x7fffff00);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool f8 = cache->dtype == MOE_E4M3;
  if (a->dtype == MOE_BF16) return f8 ? dispatch<MOE_BF16, true>(g, nt, st) : dispatch<MOE_BF16, false>(g, nt, st);
  return f8 ? dispatch<MOE_F16, true>(g, nt, st) : dispatch<MOE_F16, false>(g, nt, st);
}
