// moe_attn_team.cu — the paged-attention kernels whose workers are teams of CTAs.

#include "moe_attn.cuh"

namespace moe {

moe_status_t launch_attention_teams(const AttnArgs& g, int nt, cudaStream_t st) { return pick<true>(g, nt, st); }

}  // namespace moe
