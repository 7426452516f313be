// kvtables.cu -- h3fp4_kv_tables: offsets, lengths, pages and slots of a
// batch's new tokens, from its requests' lengths.
//
// One launch and no workspace.  A tile is 1,024 sequences; several CTAs share
// one, each scanning the tile's tokens and pages in shared memory and writing
// its share of the rows, whose sequence a binary search finds.  What lies
// before the tile and the batch's total each CTA sums up for itself (8 bytes a
// sequence out of L2), which costs less than a second launch or a wait.  Bound
// by a launch and a chain of dependent loads: lengths, the table's entry or the
// free list's, the stores (64 requests of one token 5.0 us in a graph).
#include <algorithm>

#include "kvcache.cuh"
#include "kvtables.cuh"

namespace h3fp4 {
namespace {

__device__ uint32_t g_error;

// 512 threads and two sequences each: 64 requests 5.0 us, 1,000 prompts (314,388 tokens) 7.0; 256 and four 5.3 and 7.9, 1,024
// and one 6.4 and 8.4, 128 and eight 6.1 and 10.9.
constexpr int kThreads = 512;
constexpr int kEach = 2;                    // sequences a thread
constexpr int kTile = kThreads * kEach;
constexpr int kRows = 4;                    // rows of slots a thread takes at a time

struct Request {
    int held, count, first, pages;   // first: the first new page; pages: how many
    bool ok;
};

__device__ __forceinline__ Request request(const h3fp4_kv_requests &q, int b, int shift)
{
    Request r{q.held[b], q.count[b], 0, 0, false};
    const int64_t page = int64_t(1) << shift, end = static_cast<int64_t>(r.held) + r.count;
    const int64_t last = (end + page - 1) >> shift;
    if (r.held < 0 || r.count < 0 || r.count > q.max_tokens || end > INT32_MAX || last > q.ld_table)
        return Request{0, 0, 0, 0, false};
    r.first = static_cast<int>((r.held + page - 1) >> shift);
    r.pages = static_cast<int>(last) - r.first;
    r.ok = true;
    return r;
}

template <class T>
__device__ __forceinline__ T warp_sum_up_to(T v, int lane)
{
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const T y = __shfl_up_sync(0xFFFFFFFFu, v, o);
        v += lane >= o ? y : 0;
    }
    return v;
}

// Sequence of element x among those that begin at at[0 .. n - 1], of which x is at or past the first: the last that begins at
// or before it.  first_step: the largest power of two below n (or 0).
__device__ __forceinline__ int owner(const int *at, int n, int first_step, int x)
{
    int lo = 0;
    for (int step = first_step; step > 0; step >>= 1)
        if (lo + step < n && at[lo + step] <= x)
            lo += step;
    return lo;
}

__global__ void __launch_bounds__(kThreads) tables_kernel(h3fp4_kv_requests q, int shift)
{
    __shared__ int tokens_at[kTile], pages_at[kTile], held[kTile], first[kTile], begun[kTile];
    __shared__ int warp_tokens[kThreads / 32], warp_pages[kThreads / 32];
    __shared__ long long ahead[2], total[2];   // tokens and pages of the sequences before the tile, and of all
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int b0 = blockIdx.y * kTile, n = min(kTile, q.batch - b0);
    uint32_t error = 0;
    const int free_at = *q.free_at;

    // The tile: tokens and pages of each thread's sequences, summed up.
    Request mine[kEach];
    int t = 0, p = 0, page_begun[kEach];
    bool begins[kEach];
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const int at = threadIdx.x * kEach + i;
        mine[i] = at < n ? request(q, b0 + at, shift) : Request{0, 0, 0, 0, true};
    }
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        begins[i] = mine[i].count > 0 && (mine[i].held & ((1 << shift) - 1)) != 0;   // within a page
        page_begun[i] = begins[i] ? q.page_table[(b0 + threadIdx.x * kEach + i) * q.ld_table + (mine[i].held >> shift)] : -1;
        error |= mine[i].ok ? 0u : ERR_KV_RANGE;
        t += mine[i].count;   // below 2^30 in a tile
        p += mine[i].pages;
    }
    const int my_tokens = warp_sum_up_to(t, lane), my_pages = warp_sum_up_to(p, lane);
    if (lane == 31) {
        warp_tokens[warp] = my_tokens;
        warp_pages[warp] = my_pages;
    }
    if (threadIdx.x == 0)
        ahead[0] = ahead[1] = total[0] = total[1] = 0;
    __syncthreads();
    int tile_tokens = 0, tile_pages = 0, tokens_to = my_tokens - t, pages_to = my_pages - p;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
        tokens_to += w < warp ? warp_tokens[w] : 0;
        pages_to += w < warp ? warp_pages[w] : 0;
        tile_tokens += warp_tokens[w];
        tile_pages += warp_pages[w];
    }
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const int at = threadIdx.x * kEach + i;
        tokens_at[at] = tokens_to;
        pages_at[at] = pages_to;
        held[at] = mine[i].held;
        first[at] = mine[i].first;
        const bool in = page_begun[i] >= 0 && page_begun[i] < q.num_pages;
        begun[at] = in ? page_begun[i] : -1;
        error |= begins[i] && !in ? ERR_KV_RANGE : 0u;
        tokens_to += mine[i].count;
        pages_to += mine[i].pages;
    }
    // The sequences outside the tile.
    if (gridDim.y > 1) {
        long long sum[4] = {0, 0, 0, 0};   // tokens and pages before, after
        for (int b = threadIdx.x; b < q.batch; b += kThreads) {
            const bool before = b < b0;
            if (!before && b < b0 + kTile)
                continue;
            const Request r = request(q, b, shift);
            sum[0] += before ? r.count : 0;
            sum[1] += before ? r.pages : 0;
            sum[2] += before ? 0 : r.count;
            sum[3] += before ? 0 : r.pages;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
                sum[i] += __shfl_xor_sync(0xFFFFFFFFu, sum[i], o);
            if (lane == 0)
                atomicAdd(reinterpret_cast<unsigned long long *>(i < 2 ? &ahead[i] : &total[i - 2]), static_cast<unsigned long long>(sum[i]));
        }
    }
    __syncthreads();
    const int64_t tokens0 = ahead[0], pages0 = ahead[1];
    const int64_t tokens_all = tokens0 + tile_tokens + total[0], pages_all = pages0 + tile_pages + total[1];
    const int first_step = n > 1 ? 1 << (31 - __clz(n - 1)) : 0;
    const auto page_of = [&](int64_t k) {   // number of the k-th page taken; -1 where there is none
        const int64_t at = free_at + k;
        const int id = at >= 0 && at < q.num_free ? q.free_pages[at] : -1;
        return id >= 0 && id < q.num_pages ? id : -1;
    };

    if (blockIdx.x == 0) {   // offsets and lengths
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const int at = threadIdx.x * kEach + i;
            if (at < n) {
                q.cu_tokens[b0 + at + 1] = static_cast<int>(min(tokens0 + tokens_at[at] + mine[i].count, static_cast<int64_t>(INT32_MAX)));
                q.kv_len[b0 + at] = mine[i].held + mine[i].count;
            }
        }
        if (blockIdx.y == 0 && threadIdx.x == 0) {
            q.cu_tokens[0] = 0;
            const int64_t left = max(static_cast<int64_t>(q.num_free) - free_at, static_cast<int64_t>(0));   // (places before the list too)
            *q.free_at_out = static_cast<int>(free_at + min(pages_all, left));
            if (tokens_all > INT32_MAX || (q.slots != nullptr || q.positions != nullptr ? tokens_all > q.tokens : false))
                error |= ERR_KV_RANGE;
        }
    }
    const int64_t thread = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x, threads = static_cast<int64_t>(gridDim.x) * kThreads;
    for (int64_t i = thread; i < tile_pages; i += threads) {
        const int s = owner(pages_at, n, first_step, static_cast<int>(i));
        const int id = page_of(pages0 + i);
        error |= id < 0 ? ERR_KV_RANGE : 0u;
        q.page_table[(b0 + s) * q.ld_table + first[s] + (i - pages_at[s])] = id;
    }
    if (error != 0)
        atomicOr(&g_error, error);

    // Rows of slots and positions, kRows at a time, in wide stores where the arrays allow it.
    const int64_t row_end = min(tokens0 + tile_tokens, q.tokens);
    const bool wide_stores = ((reinterpret_cast<uintptr_t>(q.slots) | reinterpret_cast<uintptr_t>(q.positions)) & 15u) == 0;
    for (int64_t row0 = tokens0 / kRows * kRows + thread * kRows; row0 < row_end; row0 += threads * kRows) {
        const int64_t from = max(row0, tokens0);
        int s = owner(tokens_at, n, first_step, static_cast<int>(from - tokens0)), page = -1, id = -1;
        long long slot[kRows];
        float position[kRows];
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const int64_t row = row0 + i;
            slot[i] = -1;
            position[i] = -1.0f;
            if (row < from || row >= row_end)
                continue;
            const int x = static_cast<int>(row - tokens0);
            while (s + 1 < n && tokens_at[s + 1] <= x) {
                ++s;
                page = -1;
            }
            const int pos = held[s] + (x - tokens_at[s]);
            if (pos >> shift != page) {
                page = pos >> shift;
                id = page < first[s] ? begun[s] : page_of(pages0 + pages_at[s] + (page - first[s]));
            }
            slot[i] = id < 0 ? -1 : (static_cast<int64_t>(id) << shift) + (pos & ((1 << shift) - 1));
            position[i] = static_cast<float>(pos);
        }
        if (wide_stores && row0 >= tokens0 && row0 + kRows <= row_end) {
            if (q.slots != nullptr) {
                *reinterpret_cast<longlong2 *>(q.slots + row0) = make_longlong2(slot[0], slot[1]);
                *reinterpret_cast<longlong2 *>(q.slots + row0 + 2) = make_longlong2(slot[2], slot[3]);
            }
            if (q.positions != nullptr)
                *reinterpret_cast<float4 *>(q.positions + row0) = make_float4(position[0], position[1], position[2], position[3]);
            continue;
        }
#pragma unroll
        for (int i = 0; i < kRows; ++i)
            if (row0 + i >= from && row0 + i < row_end) {
                if (q.slots != nullptr)
                    q.slots[row0 + i] = slot[i];
                if (q.positions != nullptr)
                    q.positions[row0 + i] = position[i];
            }
    }
    // Rows past the last token, by all.
    const int64_t wide = threads * gridDim.y;
    for (int64_t row = tokens_all + blockIdx.y * threads + thread; row < q.tokens; row += wide) {
        if (q.slots != nullptr)
            q.slots[row] = -1;
        if (q.positions != nullptr)
            q.positions[row] = -1.0f;
    }
}

}  // namespace

cudaError_t launch_kv_tables(const h3fp4_kv_requests &q, cudaStream_t st)
{
    const int shift = q.page_size == 16 ? 4 : q.page_size == 32 ? 5 : q.page_size == 64 ? 6 : 7;
    const int tiles = std::max(1, (q.batch + kTile - 1) / kTile);
    // CTAs of a tile: one for each kThreads * kRows = 2,048 of its rows, until the SMs have two each.
    const int64_t rows = q.slots != nullptr || q.positions != nullptr ? q.tokens : 0;
    const int64_t wanted = (rows / tiles + kThreads * kRows - 1) / (kThreads * kRows), most = std::max(1, 2 * sm_count() / tiles);
    const dim3 grid(static_cast<unsigned>(std::clamp<int64_t>(wanted, 1, most)), static_cast<unsigned>(tiles));
    tables_kernel<<<grid, kThreads, 0, st>>>(q, shift);
    return cudaGetLastError();
}

cudaError_t read_kv_tables_error(uint32_t *code)
{
    uint32_t v = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_error, sizeof(v));
    if (e != cudaSuccess)
        return e;
    const uint32_t zero = 0;
    e = cudaMemcpyToSymbol(g_error, &zero, sizeof(zero));
    *code = v;
    return e;
}

}  // namespace h3fp4
