// attention.cu -- h3fp4_kv_attention: which kernel takes a call, its split over
// the keys and its workspace.
#include "attention.cuh"

namespace h3fp4 {
namespace {

constexpr int64_t kMostWorkspace = int64_t(1) << 50;

// Most rows (query tokens times query heads of a cache head) of a sequence
// that the row kernel takes.
constexpr int64_t kMostRows = 16;

bool few_rows(const AttnShape &s) { return static_cast<int64_t>(s.max_tokens) * (s.heads / s.kv_heads) <= kMostRows; }

SplitPlan plan_of(const AttnShape &s) { return few_rows(s) ? plan_rows(s) : plan_tile(s); }

// Rows of parts that the workspace holds: an output and (maximum, sum) for each row and part.
int64_t part_rows(const AttnShape &s, const SplitPlan &p)
{
    if (p.splits == 1 || s.tokens == 0)
        return 0;
    const int64_t per = static_cast<int64_t>(s.heads) * p.splits;   // < 2^16 * 2^18
    return s.tokens > kMostWorkspace / per ? -1 : s.tokens * per;
}

AttnShape shape_of(const AttnArgs &a)
{
    return AttnShape{a.tokens, a.heads, a.cache.heads, a.cache.head_dim, a.batch.batch, a.batch.max_tokens, a.max_kv};
}

}  // namespace

int64_t attention_workspace(const AttnShape &s)
{
    const int64_t rows = part_rows(s, plan_of(s));
    return rows < 0 || rows > kMostWorkspace / 1024 ? -1 : rows * (4 * s.head_dim + 8);
}

cudaError_t launch_attention(const AttnArgs &a, void *workspace, cudaStream_t st)
{
    const AttnShape s = shape_of(a);
    const SplitPlan plan = plan_of(s);
    float *part = static_cast<float *>(workspace);
    float2 *stat = reinterpret_cast<float2 *>(part + part_rows(s, plan) * s.head_dim);
    cudaError_t e = few_rows(s) ? launch_attention_rows(a, plan, stat, part, st) : launch_attention_tile(a, plan, stat, part, st);
    if (e == cudaSuccess && plan.splits > 1)
        e = launch_attention_join(a, plan, stat, part, st);
    return e;
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
