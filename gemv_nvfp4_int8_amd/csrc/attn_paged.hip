// attn_paged.hip -- which kernel serves a call of paged_attention.
#include "attn_common.hpp"
#include "qp_launch.hpp"

namespace qp {

uint64_t paged_attention_work(uint32_t, uint32_t, uint32_t max_q, uint32_t q_heads, uint32_t kv_heads, uint32_t d)
{
    const uint64_t rows = (uint64_t)max_q * (q_heads / kv_heads);
    // the format is not an argument: enough for either
    const uint64_t few = rows <= attn::decode_rows(d, true) ? attn::decode_work((uint32_t)rows, d) : 0;
    return rows > attn::decode_rows(d, false) ? max(few, attn::tiles_work(d)) : few;
}

hipError_t launch_paged_attention(const AttnArgs &a, hipStream_t st)
{
    const uint64_t rows = (uint64_t)a.max_q * (a.q_heads / a.cache.heads);
    return rows <= attn::decode_rows(a.cache.d, a.cache.fp8) ? attn::launch_attn_decode(a, st) : attn::launch_attn_tiles(a, st);
}

} // namespace qp
