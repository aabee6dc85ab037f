// C-ABI layer of drafted rows over the paged cache and of cross attention:
// argument validation, status codes and dispatch to the kernel launchers.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>
#include <functional>

#include "api_checks.h"
#include "qa.h"
#include "qa_internal.h"

namespace {

using namespace qa::checks;

constexpr int kMaxRows = 1 << 30;
constexpr int kMaxPoolPages = (1 << 27) - 1;  // token slots are coordinates of 31 bits
constexpr int kMaxSeqPages = (1 << 27) - 8;   // positions and the ends of their tiles of 128 are counted in 31 bits
constexpr long long kMaxTiles = 1LL << 30;    // a call's key tiles are numbered in 32 bits

// What every call with packed rows, their requests and pages has.
qa_status check_rows(const char *fn, int batch, int most_requests, int rows, const int32_t *cu, const int32_t *past,
                     const int32_t *parents, const int32_t *page_table, const qa_attn_params *p) {
    qa_status st = qa::check_params(p, fn);
    if (st != QA_STATUS_OK) return st;
    if ((st = qa::check_gqa_params(p, fn)) != QA_STATUS_OK) return st;
    if (batch < 1 || batch > most_requests)
        return reject(QA_STATUS_INVALID_PARAMS, "%s: batch %d outside [1, %d]", fn, batch, most_requests);
    if (rows < 0 || rows > kMaxRows) return reject(QA_STATUS_INVALID_PARAMS, "%s: total_rows %d outside [0, 2^30]", fn, rows);
    if (!cu || !page_table) return invalid(fn, "NULL tensor pointer");
    if (!aligned(cu, 4) || !aligned(past, 4) || !aligned(parents, 4) || !aligned(page_table, 4))
        return invalid(fn, "int32 arrays must be 4-byte aligned");
    return QA_STATUS_OK;
}

// Shared by qa_tree_attn and qa_cross_attn.
qa_status attn_entry(const char *fn, const qa::RowsAttn &x, const qa_attn_params *p) {
    qa_status st = check_rows(fn, x.batch, qa::kRowsMaxBatch, x.rows, x.cu_seqlens, x.past, x.parents, x.page_table, p);
    if (st != QA_STATUS_OK) return st;
    if (x.max_rows < 1 || (x.tree && x.max_rows > qa::kTreeMaxRows))
        return x.tree ? reject(QA_STATUS_INVALID_PARAMS, "%s: max_rows %d outside [1, %d]", fn, x.max_rows, qa::kTreeMaxRows)
                      : reject(QA_STATUS_INVALID_PARAMS, "%s: max_rows %d < 1", fn, x.max_rows);
    if (!x.past || !x.k_pages || !x.v_pages || (x.rows > 0 && (!x.q || !x.out))) return invalid(fn, "NULL tensor pointer");
    if (!aligned(x.q, 16) || !aligned(x.out, 16) || !aligned(x.k_pages, 16) || !aligned(x.v_pages, 16))
        return invalid(fn, "tensors must be 16-byte aligned");
    if ((st = check_stride(fn, "ldq", x.ldq, (long long)p->n_q_heads * p->head_dim)) != QA_STATUS_OK) return st;
    if (p->num_pages > kMaxPoolPages)
        return reject(QA_STATUS_INVALID_PARAMS, "%s: num_pages %d above %d", fn, p->num_pages, kMaxPoolPages);
    if (p->max_pages_per_seq > kMaxSeqPages)
        return reject(QA_STATUS_INVALID_PARAMS, "%s: max_pages_per_seq %d above %d", fn, p->max_pages_per_seq, kMaxSeqPages);
    // rows of a request in blocks of at least 64
    const long long tiles = (long long)x.batch * p->max_pages_per_seq, blocks = ((long long)x.max_rows + 63) / 64;
    if (tiles > kMaxTiles || tiles * blocks > kMaxTiles)
        return reject(QA_STATUS_INVALID_PARAMS, "%s: batch * max_pages_per_seq * (max_rows / 64, rounded up) above %lld", fn,
                      kMaxTiles);
    if (x.rows == 0) return QA_STATUS_OK;
    const size_t need = qa::rows_attn_workspace_bytes(x.max_rows, p->n_q_heads, p->n_kv_heads);
    if (!need) return reject(QA_STATUS_LAUNCH_FAILED, "%s: no CUDA device", fn);
    if (!p->workspace || p->workspace_bytes < need || !aligned(p->workspace, 256))
        return reject(QA_STATUS_INVALID_PARAMS, "%s: workspace must be >= %zu bytes and 256-byte aligned (got %zu)", fn, need,
                      p->workspace_bytes);
    const float scale = p->scale > 0.f ? p->scale : 1.0f / sqrtf((float)p->head_dim);
    cudaStream_t stream = static_cast<cudaStream_t>(p->stream);
    st = launched(qa::launch_rows_attn(x, *p, scale, stream), fn);
    if (st != QA_STATUS_OK || !p->debug_checks) return st;
    cudaError_t e;
    const unsigned int bits = qa::status_read_clear_rows_attn(stream, &e);
    return qa::report_device_status(bits, e, fn);
}

}  // namespace

QA_API qa_status qa_append_rows(const void *q, long long ldq, const void *k, long long ldk, const void *v, long long ldv,
                                const int32_t *cu_seqlens, const int32_t *n_past, const int32_t *parents, int batch,
                                int total_rows, const int32_t *page_table, void *k_pages, void *v_pages, void *q_out,
                                long long ldq_out, const qa_rope *rope, const qa_attn_params *p) {
    const char *fn = "qa_append_rows";
    qa::set_last_error("");
    qa_status st = check_rows(fn, batch, qa::kDecodeMaxBatch, total_rows, cu_seqlens, n_past, parents, page_table, p);
    if (st != QA_STATUS_OK) return st;
    if (!k_pages || !v_pages) return invalid(fn, "NULL tensor pointer");
    if (rope && (st = check_rope(fn, rope, p->head_dim, false, false)) != QA_STATUS_OK) return st;
    const long long wq = (long long)p->n_q_heads * p->head_dim, wk = (long long)p->n_kv_heads * p->head_dim;
    if ((st = check_stride(fn, "ldk", ldk, wk)) != QA_STATUS_OK || (st = check_stride(fn, "ldv", ldv, wk)) != QA_STATUS_OK) return st;
    if (q && ((st = check_stride(fn, "ldq", ldq, wq)) != QA_STATUS_OK ||
              (st = check_stride(fn, "ldq_out", ldq_out, wq)) != QA_STATUS_OK))
        return st;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(k_pages, 16) || !aligned(v_pages, 16) ||
        !aligned(q ? q_out : nullptr, 16))
        return invalid(fn, "tensors must be 16-byte aligned");
    if (total_rows == 0) return QA_STATUS_OK;  // empty tensors have no address
    if (!k || !v || (q && !q_out)) return invalid(fn, "NULL tensor pointer");
    if (q && q_out == q && (ldq ? ldq : wq) != (ldq_out ? ldq_out : wq)) return invalid(fn, "q_out is q with another row stride");
    cudaStream_t stream = static_cast<cudaStream_t>(p->stream);
    const qa::AppendRows x{q, k, v, ldq, ldk, ldv, cu_seqlens, n_past, parents, page_table, batch, total_rows,
                           k_pages, v_pages, q_out, ldq_out, rope};
    st = launched(qa::launch_append_rows(x, *p, stream), fn);
    if (st != QA_STATUS_OK || !p->debug_checks) return st;
    cudaError_t e;
    const unsigned int bits = qa::status_read_clear_append_rows(stream, &e);
    return qa::report_device_status(bits, e, fn);
}

QA_API size_t qa_rows_attn_workspace_size(int max_rows, const qa_attn_params *p) {
    const char *fn = "qa_rows_attn_workspace_size";
    qa::set_last_error("");
    if (qa::check_params(p, fn) != QA_STATUS_OK || qa::check_gqa_params(p, fn) != QA_STATUS_OK) return 0;
    if (max_rows < 1) {
        reject(QA_STATUS_INVALID_PARAMS, "%s: max_rows %d < 1", fn, max_rows);
        return 0;
    }
    const size_t n = qa::rows_attn_workspace_bytes(max_rows, p->n_q_heads, p->n_kv_heads);
    if (!n) reject(QA_STATUS_LAUNCH_FAILED, "%s: no CUDA device", fn);
    return n;
}

QA_API qa_status qa_tree_attn(const void *q, long long ldq, const int32_t *cu_seqlens, const int32_t *n_past,
                              const int32_t *parents, int batch, int total_rows, int max_rows, const int32_t *page_table,
                              const void *k_pages, const void *v_pages, void *out, const qa_attn_params *p) {
    qa::set_last_error("");
    return attn_entry("qa_tree_attn", {q, ldq, cu_seqlens, n_past, parents, page_table, batch, total_rows, max_rows, k_pages,
                                       v_pages, out, true}, p);
}

QA_API qa_status qa_cross_attn(const void *q, long long ldq, const int32_t *cu_seqlens, const int32_t *seq_lens, int batch,
                               int total_rows, int max_rows, const int32_t *page_table, const void *k_pages,
                               const void *v_pages, void *out, const qa_attn_params *p) {
    qa::set_last_error("");
    return attn_entry("qa_cross_attn", {q, ldq, cu_seqlens, seq_lens, nullptr, page_table, batch, total_rows, max_rows, k_pages,
                                        v_pages, out, false}, p);
}

QA_API qa_status qa_tree_accept(const int32_t *draft, const int32_t *target, const int32_t *parents,
                                const int32_t *cu_seqlens, const int32_t *n_past, int batch, int total_rows, int max_rows,
                                const int32_t *page_table, int n_layers, void *const *k_pages, void *const *v_pages,
                                int32_t *n_accepted, int32_t *path, int32_t *next_token, const qa_attn_params *p) {
    const char *fn = "qa_tree_accept";
    qa::set_last_error("");
    qa_status st = check_rows(fn, batch, qa::kDecodeMaxBatch, total_rows, cu_seqlens, n_past, parents, page_table, p);
    if (st != QA_STATUS_OK) return st;
    if (max_rows < 1 || max_rows > qa::kTreeMaxRows)
        return reject(QA_STATUS_INVALID_PARAMS, "%s: max_rows %d outside [1, %d]", fn, max_rows, qa::kTreeMaxRows);
    if (n_layers < 0 || n_layers > qa::kAcceptMaxLayers)
        return reject(QA_STATUS_INVALID_PARAMS, "%s: n_layers %d outside [0, %d]", fn, n_layers, qa::kAcceptMaxLayers);
    if (!n_past || (total_rows > 0 && (!draft || !target)) || !n_accepted || !path || !next_token ||
        (n_layers > 0 && (!k_pages || !v_pages)))
        return invalid(fn, "NULL tensor pointer");
    if (!aligned(draft, 4) || !aligned(target, 4) || !aligned(n_accepted, 4) || !aligned(path, 4) || !aligned(next_token, 4))
        return invalid(fn, "int32 arrays must be 4-byte aligned");
    for (int i = 0; i < n_layers; ++i) {
        if (!k_pages[i] || !v_pages[i]) return invalid(fn, "NULL tensor pointer");
        if (!aligned(k_pages[i], 16) || !aligned(v_pages[i], 16)) return invalid(fn, "tensors must be 16-byte aligned");
    }
    // Each pool once, in the order of their addresses: two CTAs that move a pool's rows in place would read one another's.
    void *pools[2 * qa::kAcceptMaxLayers];
    for (int i = 0; i < n_layers; ++i) pools[2 * i] = k_pages[i], pools[2 * i + 1] = v_pages[i];
    std::sort(pools, pools + 2 * n_layers, std::less<void *>());
    const int n_pools = (int)(std::unique(pools, pools + 2 * n_layers) - pools);
    const uintptr_t bytes = (uintptr_t)p->num_pages * p->page_size * p->n_kv_heads * p->head_dim * sizeof(uint16_t);
    for (int i = 1; i < n_pools; ++i)
        if (reinterpret_cast<uintptr_t>(pools[i]) - reinterpret_cast<uintptr_t>(pools[i - 1]) < bytes)
            return invalid(fn, "two pools overlap without being the same");
    cudaStream_t stream = static_cast<cudaStream_t>(p->stream);
    const qa::TreeAccept x{draft, target, parents, cu_seqlens, n_past, page_table, batch, total_rows, max_rows, pools,
                           n_pools, n_accepted, path, next_token};
    st = launched(qa::launch_tree_accept(x, *p, stream), fn);
    if (st != QA_STATUS_OK || !p->debug_checks) return st;
    cudaError_t e;
    const unsigned int bits = qa::status_read_clear_tree_accept(stream, &e);
    return qa::report_device_status(bits, e, fn);
}
