// moe_attn.cu — the C entries of paged attention, and the kernels whose workers
// are single CTAs.

#include "moe_attn.cuh"

namespace moe {

moe_status_t launch_attention_ctas(const AttnArgs& g, int nt, cudaStream_t st) { return pick<false>(g, nt, st); }

namespace {

int padded_dim(int D) { return D <= 64 ? 64 : D <= 128 ? 128 : 256; }
// n tiles of 8 heads of a segment: two when a group has more than 8 heads, but one
// for rows of more than 128 elements, where two leave no room for a second CTA on
// an SM; there the tiles' lines lie side by side and read the rows at about the
// same time, the later ones from L2 (32 heads over 2 of 256: 4 sequences of up to
// 8k tokens 25 us against 48, 64 of them 143 against 142; rows of 96, 53 sequences
// of 16k: 154 against 126).
int n_tiles(int group, int dp) { return group > 8 && dp <= 128 ? 2 : 1; }
// Segments up to which teams are the workers: 8 segments of 4k tokens took 16.9 us
// with teams against 15.4 with CTAs, 2 of 8k tokens 13.3 against 16.9.
constexpr int kTeamSegments = 4;
// Up to this many segments have a team each, if the table (or the window) keeps
// them short enough: 32 of 128 units 12.9 us against 16.8 with CTAs, 16 of 64 units
// 8.8 against 15.0; 8 of 256 units 15.7 against 15.0.
constexpr int kTeamsEach = 32;
constexpr int kTeamsEachUnits = 160;
// Groups of more than 8 heads whose segments are few and short are split into one
// tile of heads each, up to this many segments: 7 windows of 76 over 64 heads of 256
// 7.6 us against 12.9, 70 sequences of 100 over 32 e4m3 heads of 128 6.9 against
// 8.8; 300 of 60 stay (7.4 us, 11.7 as 600).
constexpr int kSplit = 304;
constexpr int kSplitUnits = 32;
// Lines over neighbouring kv heads, whose CTAs together read longer pieces of memory:
// 5 sequences of 120k tokens, 8 e4m3 heads of 96 171 us against 302 (162 where each
// head's rows are together), 250 windows of 512 over 12 heads of 64 69 against 73; 8
// such lines gain no more and cost short batches 2 %.
constexpr int kKvSides = 4;

// Tokens that a table of this many pages holds, as the kernel counts them.
int32_t longest(const moe_kv_cache_t* c, int32_t max_pages) {
  const int64_t cap = static_cast<int64_t>(max_pages) * c->page_size;
  return static_cast<int32_t>(cap < 0x7fffff00 ? cap : 0x7fffff00);
}

// How a batch is launched: from its sizes alone, as the lengths are the device's.
struct Plan {
  int nt;      // tiles of 8 heads of a segment
  int hpc, chunks, sides, kv_sides;  // as in AttnArgs
  bool teams;  // workers are teams of CTAs
};

Plan plan_of(const moe_kv_cache_t* c, int32_t B, int32_t n_q_heads, int32_t max_len, int32_t window) {
  Plan p;
  const int group = n_q_heads / c->n_kv_heads, tiles = (group + 7) / 8, dp = padded_dim(c->head_dim);
  const int fill = 8192 / (dp * (c->dtype == MOE_E4M3 ? 1 : 2));
  const int unit = fill < 16 ? 16 : fill < 64 ? fill : 64;  // tokens of a team's unit
  // the same of a CTA's unit
  const int cta_fill = dp <= 64 ? fill / 2 : fill;
  const int cta_unit = cta_fill < 16 ? 16 : cta_fill < 64 ? cta_fill : 64;
  const int most = window > 0 && window < max_len ? window : max_len;  // tokens of a sequence
  p.nt = n_tiles(group, dp);
  p.chunks = (tiles + p.nt - 1) / p.nt;
  const int64_t kv = static_cast<int64_t>(B) * c->n_kv_heads;
  // (not where that takes segments their teams: 18 of 300 tokens 7.0 us, 36 8.1 with CTAs)
  if (p.nt == 2 && kv * tiles <= kSplit && most / cta_unit + 2 <= kSplitUnits &&
      (kv * p.chunks > kTeamsEach || kv * tiles <= kTeamsEach)) {
    p.nt = 1;
    p.chunks = tiles;
  }
  p.hpc = (group + p.chunks - 1) / p.chunks;
  const int64_t segments = kv * p.chunks;
  p.teams = segments <= kTeamSegments || (segments <= kTeamsEach && most / unit + 2 <= kTeamsEachUnits);
  // (48 heads over 1 of 128, 64 sequences of up to 32k tokens: 243 us, 292 with the
  // chunks' segments one after the other on one line)
  p.sides = !p.teams && p.chunks <= kMaxSides ? p.chunks : 1;
  p.chunks /= p.sides;
  // neighbouring kv heads side by side, where their rows are neighbours in memory
  p.kv_sides = 1;
  if (!p.teams && c->k_head_stride < c->k_token_stride)
    for (int n = kKvSides / p.sides; n > 1 && p.kv_sides == 1; --n)
      if (c->n_kv_heads % n == 0) p.kv_sides = n;
  return p;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" size_t moe_attention_workspace_bytes(const moe_kv_cache_t* cache, int32_t n_q_heads) {
  if (!cache || cache->n_kv_heads < 1 || cache->head_dim < 1 || cache->head_dim > 256 || n_q_heads < 1 ||
      n_q_heads % cache->n_kv_heads)
    return 0;
  const int dp = padded_dim(cache->head_dim), nt = n_tiles(n_q_heads / cache->n_kv_heads, dp);
  return kPartsAt + static_cast<size_t>(max_chunks(dp)) * 2 * 8 * nt * dp * sizeof(float);
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
  const int tiles = (g.group + 7) / 8;
  // Tokens are 32-bit numbers; units round a length up by less than 64.
  const int64_t cap = static_cast<int64_t>(a->max_pages) * cache->page_size;
  // The line of units is counted in 32 bits.
  if (cap / 16 + 2 + 4 > 0x7fffffffll / tiles / cache->n_kv_heads / a->B)
    return set_error(MOE_ERR_UNSUPPORTED, "batch * kv heads * table tokens too large");
  g.by_page = FastDiv(cache->page_size);
  const int64_t size = cache->dtype == MOE_E4M3 ? 1 : 2;
  g.k_page = static_cast<uint32_t>(cache->k_page_stride * size);
  g.k_token = static_cast<uint32_t>(cache->k_token_stride * size);
  g.k_head = static_cast<uint32_t>(cache->k_head_stride * size);
  g.v_page = static_cast<uint32_t>(cache->v_page_stride * size);
  g.v_token = static_cast<uint32_t>(cache->v_token_stride * size);
  g.v_head = static_cast<uint32_t>(cache->v_head_stride * size);
  g.blocks = cache->page_size % 16 == 0;
  g.max_len = longest(cache, a->max_pages);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const Plan plan = plan_of(cache, a->B, a->n_q_heads, g.max_len, a->window);
  g.hpc = plan.hpc;
  g.chunks = plan.chunks;
  g.sides = plan.sides;
  g.kv_sides = plan.kv_sides;
  return plan.teams ? launch_attention_teams(g, plan.nt, st) : launch_attention_ctas(g, plan.nt, st);
}

extern "C" int32_t moe_attention_form(const moe_kv_cache_t* cache, int32_t B, int32_t n_q_heads, int32_t max_pages,
                                      int32_t window) {
  if (!cache || cache->n_kv_heads < 1 || cache->page_size < 1 || cache->head_dim < 1 || cache->head_dim > 256 ||
      B < 1 || n_q_heads < 1 || n_q_heads % cache->n_kv_heads || max_pages < 0 || window < 0)
    return 0;
  return plan_of(cache, B, n_q_heads, longest(cache, max_pages), window).teams ? 2 : 1;
}
