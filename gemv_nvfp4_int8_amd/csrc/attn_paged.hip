// attn_paged.hip -- which kernel serves a call of paged_attention.
#include "attn_common.hpp"
#include "qp_launch.hpp"

namespace qp {

static bool few_rows(uint32_t max_q, uint32_t group)
{
    return (uint64_t)max_q * group <= attn::DECODE_ROWS;
}

uint64_t paged_attention_work(uint32_t, uint32_t, uint32_t max_q, uint32_t q_heads, uint32_t kv_heads, uint32_t d)
{
    return few_rows(max_q, q_heads / kv_heads) ? attn::decode_work(d) : attn::tiles_work(d);
}

hipError_t launch_paged_attention(const AttnArgs &a, hipStream_t st)
{
    return few_rows(a.max_q, a.q_heads / a.cache.heads) ? attn::launch_attn_decode(a, st) : attn::launch_attn_tiles(a, st);
}

} // namespace qp
