// The end of a step of drafted tokens (qa_tree_accept): the path of drafted
// rows that the model agrees with, and its key and value rows moved, in every
// layer, to the positions right behind the cache.
//
//   path[0] = 0;  path[j + 1] = the first c with parents[c] = path[j] and
//   draft[c] = target[path[j]];  slot n_past + j takes slot n_past + path[j]
//
// One CTA a request and pool, no two of which overlap.  Every CTA walks its
// request's tree by itself (a ballot a step over at most 64 rows held two a
// lane), which is cheaper than a launch, or a wait, between the walk and the
// moves.  A thread owns 16 bytes of a row and goes up the path: path[j] >= j,
// and it rises, so that a slot is read before, or in the same batch of loads
// as, it is written, and no thread waits for another.
//
// What bounds it is latency: boundaries, then tokens and parents, then page
// ids, then rows: 3.3 us for 64 requests in four layers, 2.4 us for one, as
// nodes of a graph.  With the four layers' appends before it 26.2 and 14.2 us
// replayed, and 33.0 and 19.6 called one by one, where five calls on the host
// bound the small one.
#include <cuda_runtime.h>
#include <stdint.h>

#include "qa_internal.h"

namespace qa {
namespace {

__device__ unsigned int g_status;

constexpr int kThreads = 128;  // 8 KV heads of 128 dims, 8 dims a thread
constexpr int kBatch = 8;      // rows in flight a thread

struct AcceptArgs {
    const int32_t *draft, *target, *parents, *cu, *past, *page_table;
    int32_t *n_accepted, *path, *next_token;
    int rows, max_rows, max_pages, num_pages, row_chunks, early;  // row_chunks: 16-byte pieces of a row
    int n_pools;
    uint4 *pools[2 * kAcceptMaxLayers];
};

__global__ void __launch_bounds__(kThreads) tree_accept_kernel(const __grid_constant__ AcceptArgs a) {
    constexpr unsigned kAll = 0xffffffffu;
    __shared__ int s_path[kTreeMaxRows], s_count;
    __shared__ long long s_from[kTreeMaxRows], s_to[kTreeMaxRows];  // the rows' numbers in a pool, -1: not moved
    const int lane = threadIdx.x & 31, b = blockIdx.x, pool = blockIdx.y;
    if (!a.early) asm volatile("griddepcontrol.wait;" ::: "memory");
    if (threadIdx.x < 32) {
        const int first = a.cu[b], end = a.cu[b + 1];
        const long long past = a.past[b], cap = (long long)a.max_pages * 16;
        const bool segment = first >= 0 && end >= first && end <= a.rows;
        const int n = segment ? end - first : 0;
        const bool fits = n <= a.max_rows && past >= 0 && past + n <= cap;
        if (lane == 0 && pool == 0 && !(segment && fits))
            atomicOr(&g_status, segment ? QA_DEVICE_BAD_LENGTH : QA_DEVICE_BAD_SEGMENTS);
        const int rows = fits ? n : 0;
        int parent[2], draft[2], target[2];
        for (int x = 0; x < 2; ++x) {
            const int i = lane + 32 * x;
            parent[x] = -1;
            if (i < rows) {
                parent[x] = a.parents ? a.parents[first + i] : i - 1;
                if (parent[x] < -1 || parent[x] >= i) {
                    atomicOr(&g_status, QA_DEVICE_BAD_TREE);
                    parent[x] = -1;
                }
            }
        }
        if (a.early) asm volatile("griddepcontrol.wait;" ::: "memory");
        for (int x = 0; x < 2; ++x) {
            const int i = lane + 32 * x;
            draft[x] = i < rows ? a.draft[first + i] : 0;
            target[x] = i < rows ? a.target[first + i] : 0;
        }
        int count = 0, answer = -1;
        for (int node = rows > 0 ? 0 : -1; node >= 0;) {
            if (lane == 0) s_path[count] = node;
            ++count;
            const int low = __shfl_sync(kAll, target[0], node & 31), high = __shfl_sync(kAll, target[1], node & 31);
            answer = node < 32 ? low : high;
            const unsigned m0 = __ballot_sync(kAll, parent[0] == node && draft[0] == answer);
            const unsigned m1 = __ballot_sync(kAll, parent[1] == node && draft[1] == answer);
            node = m0 ? __ffs(m0) - 1 : m1 ? 31 + __ffs(m1) : -1;  // beyond node: a parent comes before its rows
        }
        __syncwarp();
        const int32_t *table = a.page_table + (size_t)b * a.max_pages;
        for (int j = lane; j < count && a.n_pools > 0; j += 32) {
            const int i = s_path[j];
            long long from = -1, to = -1;
            if (i != j) {
                const int p = (int)(past + i), q = (int)(past + j);
                const int from_page = table[p >> 4], to_page = table[q >> 4];
                if ((unsigned)from_page < (unsigned)a.num_pages && (unsigned)to_page < (unsigned)a.num_pages)
                    from = (long long)from_page * 16 + (p & 15), to = (long long)to_page * 16 + (q & 15);
                else
                    atomicOr(&g_status, QA_DEVICE_BAD_PAGE);
            }
            s_from[j] = from, s_to[j] = to;
        }
        if (pool == 0) {
            if (lane == 0) a.n_accepted[b] = count, a.next_token[b] = answer;
            for (int j = lane; j < a.max_rows; j += 32) a.path[(size_t)b * a.max_rows + j] = j < count ? s_path[j] : -1;
        }
        if (lane == 0) s_count = count;
    } else if (a.early) {
        asm volatile("griddepcontrol.wait;" ::: "memory");
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    __syncthreads();
    if ((int)threadIdx.x >= a.row_chunks || pool >= a.n_pools) return;
    uint4 *rows = a.pools[pool] + threadIdx.x;
    const int count = s_count;
    for (int j = 0; j < count; j += kBatch) {
        uint4 x[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k)
            if (j + k < count && s_from[j + k] >= 0) x[k] = rows[s_from[j + k] * a.row_chunks];
#pragma unroll
        for (int k = 0; k < kBatch; ++k)
            if (j + k < count && s_from[j + k] >= 0) rows[s_to[j + k] * a.row_chunks] = x[k];
    }
}

}  // namespace

cudaError_t launch_tree_accept(const TreeAccept &x, const qa_attn_params &p, cudaStream_t stream) {
    AcceptArgs a = {};
    a.draft = x.draft;
    a.target = x.target;
    a.parents = x.parents;
    a.cu = x.cu_seqlens;
    a.past = x.n_past;
    a.page_table = x.page_table;
    a.n_accepted = x.n_accepted;
    a.path = x.path;
    a.next_token = x.next_token;
    a.rows = x.rows;
    a.max_rows = x.max_rows;
    a.max_pages = p.max_pages_per_seq;
    a.num_pages = p.num_pages;
    a.row_chunks = p.n_kv_heads * 16;
    a.early = (p.abi_version >= 2 && p.stable_metadata >= 1) ? 1 : 0;
    a.n_pools = x.n_pools;
    for (int i = 0; i < x.n_pools; ++i) a.pools[i] = static_cast<uint4 *>(x.pools[i]);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)x.batch, (unsigned)(a.n_pools > 0 ? a.n_pools : 1));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, tree_accept_kernel, a);
}

unsigned int status_read_clear_tree_accept(cudaStream_t stream, cudaError_t *err) {
    unsigned int v = 0, zero = 0;
    cudaError_t e = cudaMemcpyFromSymbolAsync(&v, g_status, sizeof v, 0, cudaMemcpyDeviceToHost, stream);
    if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
    if (e == cudaSuccess && v) e = cudaMemcpyToSymbolAsync(g_status, &zero, sizeof zero, 0, cudaMemcpyHostToDevice, stream);
    if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
    if (err) *err = e;
    return v;
}

}  // namespace qa
