// attention.cu -- h3fp4_kv_attention: which kernel takes a call, and its
// workspace.
#include "attention.cuh"

namespace h3fp4 {
namespace {

// Most rows (query tokens times query heads of a cache head) of a sequence
// that the row kernel takes.  It reads the codes once for 16 rows, the tile
// kernel once for 256 but with all of a tile's work for one row.  32 rows: 32
// sequences of up to 8,192 keys, 8 heads, 144 us (tile kernel 252), 131,072
// keys 116 us (137), 8 of 1,000 keys 12.3 us (13.1), one of 8,192 keys 21.5 us
// (20.4).  48 rows: 207 us (253), 167 (138), 14.8 (13.4), 27.0 (21.1).
constexpr int64_t kMostRows = 32;

bool few_rows(const AttnShape &s) { return static_cast<int64_t>(s.max_tokens) * (s.heads / s.kv_heads) <= kMostRows; }

AttnShape shape_of(const AttnArgs &a)
{
    return AttnShape{a.tokens, a.heads, a.cache.heads, a.cache.head_dim, a.batch.batch, a.batch.max_tokens, a.max_kv,
                     a.causal ? a.window : 0};
}

SplitPlan plan_of(const AttnShape &s) { return few_rows(s) ? plan_rows(s) : plan_tile(s); }

}  // namespace

int64_t attention_workspace(const AttnShape &s)
{
    const int64_t rows = s.tokens == 0 || s.batch == 0 || s.max_tokens == 0 ? 0 : plan_of(s).part_rows;
    return rows > (int64_t(1) << 50) ? -1 : rows * (4 * s.head_dim + 8);   // a mean, and its sum's logarithm (or the sum and what it is kept against)
}

cudaError_t launch_attention(const AttnArgs &a, void *workspace, cudaStream_t st)
{
    const AttnShape s = shape_of(a);   // (the parts are no more than without the reach: the workspace does for both)
    const SplitPlan plan = plan_of(s);
    float *part = static_cast<float *>(workspace);
    float *stat = part + plan.part_rows * s.head_dim;
    return few_rows(s) ? launch_attention_rows(a, plan, stat, part, st)
                       : launch_attention_tile(a, plan, reinterpret_cast<float2 *>(stat), part, st);
}

bool attention_timeout_ok(const AttnArgs &a)
{
    return a.cache.head_dim == 128 && int64_t(a.batch.max_tokens) * (a.heads / a.cache.heads) <= 8;
}

cudaError_t launch_attention_wait_timeout(const AttnArgs &a, void *workspace, uint64_t wait_ns, cudaStream_t st)
{
    const SplitPlan plan = plan_of(shape_of(a));
    float *part = static_cast<float *>(workspace);
    return launch_attention_rows_timeout(a, plan, part + plan.part_rows * a.cache.head_dim, part, wait_ns, st);
}

cudaError_t read_attention_error(uint32_t *code)
{
    uint32_t rows = 0, tile = 0;
    cudaError_t e = read_attention_rows_error(&rows);
    if (e == cudaSuccess)
        e = read_attention_tile_error(&tile);
    *code = rows | tile;
    return e;
}

}  // namespace h3fp4
