// C-ABI layer of rotary positions and the 4-bit cache: argument validation,
// status codes and dispatch to the kernel launchers.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include "api_checks.h"
#include "qa.h"
#include "qa_internal.h"

namespace {

using namespace qa::checks;

constexpr int kHeadBytes = 1280;
constexpr long long kMaxPages = 1LL << 30;

// Shared by the page write and read.
qa_status check_pages(const char *fn, const void *k, const void *v, const int32_t *cu, const int32_t *n_past, int batch,
                      int total, const int32_t *page_table, const void *k_pages, const void *v_pages,
                      const qa_attn_params *p) {
    qa_status st = qa::check_params(p, fn);
    if (st != QA_STATUS_OK) return st;
    if ((st = qa::check_gqa_params(p, fn)) != QA_STATUS_OK) return st;
    if (batch < 1 || batch > qa::kDecodeMaxBatch)
        return reject(QA_STATUS_INVALID_PARAMS, "%s: batch %d outside [1, %d]", fn, batch, qa::kDecodeMaxBatch);
    if (total < 0) return reject(QA_STATUS_INVALID_PARAMS, "%s: total_tokens %d < 0", fn, total);
    if ((total > 0 && (!k || !v)) || !cu || !page_table || !k_pages || !v_pages) return invalid(fn, "NULL tensor pointer");
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(k_pages, 16) || !aligned(v_pages, 16) || !aligned(cu, 4) ||
        !aligned(n_past, 4) || !aligned(page_table, 4))
        return invalid(fn, "tensors must be 16-byte aligned (int32 arrays 4-byte)");
    return QA_STATUS_OK;
}

// Shared by qa_kvq_decode_attn and qa_kvq_decode_step (app != nullptr).
qa_status decode_entry(const char *fn, const void *q, long long ldq, const void *k_pages, const void *v_pages,
                       const int32_t *page_table, const int32_t *seq_lens, int batch, void *out, const qa_attn_params *p,
                       const qa::KvqAppend *app) {
    const qa_status ok = qa::check_decode_call(fn, q, k_pages, v_pages, page_table, seq_lens, batch, out, p);
    if (ok != QA_STATUS_OK) return ok;
    if ((long long)batch * p->max_pages_per_seq > kMaxPages)  // a call's pages are numbered in 32 bits
        return reject(QA_STATUS_INVALID_PARAMS, "%s: batch * max_pages_per_seq %lld above %lld", fn,
                      (long long)batch * p->max_pages_per_seq, kMaxPages);
    const int ctas = qa::current_decode_ctas();
    if (ctas <= 0) return reject(QA_STATUS_LAUNCH_FAILED, "%s: no CUDA device", fn);
    const size_t need = qa::kvq_decode_workspace_bytes(batch, p->n_q_heads, p->n_kv_heads, ctas);
    if (!p->workspace || p->workspace_bytes < need || !aligned(p->workspace, 256))
        return reject(QA_STATUS_INVALID_PARAMS, "%s: workspace must be >= %zu bytes and 256-byte aligned (got %zu)", fn, need,
                      p->workspace_bytes);
    const float scale = p->scale > 0.f ? p->scale : 1.0f / sqrtf((float)p->head_dim);
    cudaStream_t stream = static_cast<cudaStream_t>(p->stream);
    qa_status st = launched(qa::launch_kvq_decode(q, ldq, const_cast<void *>(k_pages), const_cast<void *>(v_pages), page_table,
                                                  seq_lens, batch, out, *p, scale, ctas, stream, app),
                            fn);
    if (st != QA_STATUS_OK || !p->debug_checks) return st;
    cudaError_t e;
    const unsigned int bits = qa::status_read_clear_kvq_decode(stream, &e);
    return qa::report_device_status(bits, e, fn);
}

}  // namespace

QA_API int qa_rope_axes(const int *sections, int n_axes, int interleaved, int head_dim, uint8_t *pair_axis) {
    const char *fn = "qa_rope_axes";
    qa::set_last_error("");
    if (!sections || !pair_axis) return invalid(fn, "NULL pointer"), -1;
    if (n_axes < 1 || n_axes > kMaxAxes)
        return reject(QA_STATUS_INVALID_PARAMS, "%s: n_axes %d outside [1, %d]", fn, n_axes, kMaxAxes), -1;
    if (head_dim != 64 && head_dim != 128)
        return reject(QA_STATUS_INVALID_PARAMS, "%s: head_dim %d unsupported (64 or 128)", fn, head_dim), -1;
    const int half = head_dim / 2;
    long long sum = 0;
    for (int a = 0; a < n_axes; ++a) {
        if (sections[a] < 0) return reject(QA_STATUS_INVALID_PARAMS, "%s: sections[%d] = %d < 0", fn, a, sections[a]), -1;
        sum += sections[a];
    }
    if (sum != half)
        return reject(QA_STATUS_INVALID_PARAMS, "%s: sections add up to %lld, not head_dim / 2 = %d", fn, sum, half), -1;
    uint8_t got[64];
    int count[kMaxAxes] = {0};
    if (interleaved) {
        for (int i = 0; i < half; ++i) {
            const int a = i % n_axes;
            got[i] = (uint8_t)(i < n_axes * sections[a] ? a : 0);
            ++count[got[i]];
        }
        for (int a = 0; a < n_axes; ++a)
            if (count[a] != sections[a])
                return reject(QA_STATUS_INVALID_PARAMS, "%s: sections cannot be interleaved (axis %d gets %d of %d pairs)", fn, a,
                              count[a], sections[a]), -1;
    } else {
        int i = 0;
        for (int a = 0; a < n_axes; ++a)
            for (int c = 0; c < sections[a]; ++c) got[i++] = (uint8_t)a;
    }
    memcpy(pair_axis, got, half);
    return 0;
}

QA_API qa_status qa_rope_rows(const void *q, long long ldq, const void *k, long long ldk, int rows, void *q_out,
                              long long ldq_out, void *k_out, long long ldk_out, const qa_rope *rope,
                              const qa_attn_params *p) {
    const char *fn = "qa_rope_rows";
    qa::set_last_error("");
    qa_status st = qa::check_params(p, fn);
    if (st != QA_STATUS_OK) return st;
    if (p->head_dim != 64 && p->head_dim != 128)
        return reject(QA_STATUS_INVALID_PARAMS, "%s: head_dim %d unsupported (64 or 128)", fn, p->head_dim);
    if (p->n_q_heads < 1 || p->n_q_heads > 1024 || (k && (p->n_kv_heads < 1 || p->n_kv_heads > 1024)))
        return reject(QA_STATUS_INVALID_PARAMS, "%s: head counts (%d, %d) outside [1, 1024]", fn, p->n_q_heads, p->n_kv_heads);
    if (rows < 0 || rows > 1 << 30) return reject(QA_STATUS_INVALID_PARAMS, "%s: rows %d outside [0, 2^30]", fn, rows);
    if (rows == 0) return QA_STATUS_OK;  // empty tensors have no address
    if (!q || !q_out || (k && !k_out)) return invalid(fn, "NULL tensor pointer");
    if ((st = check_rope(fn, rope, p->head_dim, false, true)) != QA_STATUS_OK) return st;
    const long long wq = (long long)p->n_q_heads * p->head_dim, wk = (long long)p->n_kv_heads * p->head_dim;
    if ((st = check_stride(fn, "ldq", ldq, wq)) != QA_STATUS_OK || (st = check_stride(fn, "ldq_out", ldq_out, wq)) != QA_STATUS_OK)
        return st;
    if (k && ((st = check_stride(fn, "ldk", ldk, wk)) != QA_STATUS_OK ||
              (st = check_stride(fn, "ldk_out", ldk_out, wk)) != QA_STATUS_OK))
        return st;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(q_out, 16) || !aligned(k ? k_out : nullptr, 16))
        return invalid(fn, "tensors must be 16-byte aligned");
    if (q_out == q && (ldq ? ldq : wq) != (ldq_out ? ldq_out : wq)) return invalid(fn, "q_out is q with another row stride");
    if (k && k_out == k && (ldk ? ldk : wk) != (ldk_out ? ldk_out : wk))
        return invalid(fn, "k_out is k with another row stride");
    cudaStream_t stream = static_cast<cudaStream_t>(p->stream);
    st = launched(qa::launch_rope_rows(q, ldq, k, ldk, rows, q_out, ldq_out, k_out, ldk_out, *rope, *p, stream), fn);
    if (st != QA_STATUS_OK || !p->debug_checks) return st;
    cudaError_t e;
    const unsigned int bits = qa::status_read_clear_rope(stream, &e);
    return qa::report_device_status(bits, e, fn);
}

QA_API size_t qa_kvq_page_bytes(const qa_attn_params *p) {
    const char *fn = "qa_kvq_page_bytes";
    qa::set_last_error("");
    if (qa::check_params(p, fn) != QA_STATUS_OK) return 0;
    if (p->head_dim != 128 || p->page_size != 16 || p->n_kv_heads < 1 || p->n_kv_heads > 8) {
        invalid(fn, "head_dim 128, page_size 16 and n_kv_heads in [1, 8] required");
        return 0;
    }
    return (size_t)p->n_kv_heads * kHeadBytes;
}

QA_API qa_status qa_kvq_write(const void *k, long long ldk, const void *v, long long ldv, const int32_t *cu_seqlens,
                              const int32_t *n_past, int batch, int total_tokens, const int32_t *page_table, void *k_pages,
                              void *v_pages, const qa_attn_params *p) {
    const char *fn = "qa_kvq_write";
    qa::set_last_error("");
    qa_status st = check_pages(fn, k, v, cu_seqlens, n_past, batch, total_tokens, page_table, k_pages, v_pages, p);
    if (st != QA_STATUS_OK) return st;
    const long long width = (long long)p->n_kv_heads * p->head_dim;
    if ((st = check_stride(fn, "ldk", ldk, width)) != QA_STATUS_OK || (st = check_stride(fn, "ldv", ldv, width)) != QA_STATUS_OK)
        return st;
    cudaStream_t stream = static_cast<cudaStream_t>(p->stream);
    st = launched(qa::launch_kvq_write(k, ldk, v, ldv, cu_seqlens, n_past, batch, total_tokens, page_table, k_pages, v_pages,
                                       *p, stream),
                  fn);
    if (st != QA_STATUS_OK || !p->debug_checks) return st;
    cudaError_t e;
    const unsigned int bits = qa::status_read_clear_kvq_pages(stream, &e);
    return qa::report_device_status(bits, e, fn);
}

QA_API qa_status qa_kvq_read(const void *k_pages, const void *v_pages, const int32_t *page_table, const int32_t *cu_seqlens,
                             const int32_t *n_past, int batch, int total_tokens, void *k_out, void *v_out,
                             const qa_attn_params *p) {
    const char *fn = "qa_kvq_read";
    qa::set_last_error("");
    qa_status st = check_pages(fn, k_out, v_out, cu_seqlens, n_past, batch, total_tokens, page_table, k_pages, v_pages, p);
    if (st != QA_STATUS_OK) return st;
    cudaStream_t stream = static_cast<cudaStream_t>(p->stream);
    st = launched(qa::launch_kvq_read(k_pages, v_pages, page_table, cu_seqlens, n_past, batch, total_tokens, k_out, v_out, *p,
                                      stream),
                  fn);
    if (st != QA_STATUS_OK || !p->debug_checks) return st;
    cudaError_t e;
    const unsigned int bits = qa::status_read_clear_kvq_pages(stream, &e);
    return qa::report_device_status(bits, e, fn);
}

QA_API size_t qa_kvq_decode_workspace_size(int batch, int max_seq_len, const qa_attn_params *p) {
    const char *fn = "qa_kvq_decode_workspace_size";
    qa::set_last_error("");
    if (qa::check_params(p, fn) != QA_STATUS_OK || qa::check_gqa_params(p, fn) != QA_STATUS_OK) return 0;
    if (batch < 1 || batch > qa::kDecodeMaxBatch) {
        reject(QA_STATUS_INVALID_PARAMS, "%s: batch %d outside [1, %d]", fn, batch, qa::kDecodeMaxBatch);
        return 0;
    }
    if (max_seq_len < 0 || (long long)max_seq_len > (long long)p->max_pages_per_seq * p->page_size) {
        reject(QA_STATUS_INVALID_PARAMS, "%s: max_seq_len %d outside [0, max_pages_per_seq * page_size]", fn, max_seq_len);
        return 0;
    }
    const int ctas = qa::current_decode_ctas();
    if (ctas <= 0) {
        reject(QA_STATUS_LAUNCH_FAILED, "%s: no CUDA device", fn);
        return 0;
    }
    return qa::kvq_decode_workspace_bytes(batch, p->n_q_heads, p->n_kv_heads, ctas);
}

QA_API qa_status qa_kvq_decode_attn(const void *q, const void *k_pages, const void *v_pages, const int32_t *page_table,
                                    const int32_t *seq_lens, int batch, void *out, const qa_attn_params *p) {
    qa::set_last_error("");
    return decode_entry("qa_kvq_decode_attn", q, 0, k_pages, v_pages, page_table, seq_lens, batch, out, p, nullptr);
}

QA_API qa_status qa_kvq_decode_step(const void *q, long long ldq, const void *k, const void *v, long long ldkv,
                                    const qa_rope *rope, void *k_pages, void *v_pages, const int32_t *page_table,
                                    const int32_t *seq_lens, int batch, void *out, const qa_attn_params *p) {
    const char *fn = "qa_kvq_decode_step";
    qa::set_last_error("");
    qa_status st = qa::check_params(p, fn);
    if (st != QA_STATUS_OK) return st;
    if ((st = qa::check_gqa_params(p, fn)) != QA_STATUS_OK) return st;
    if ((st = check_rope(fn, rope, p->head_dim, true, false)) != QA_STATUS_OK) return st;
    if (!rope->positions && (long long)p->max_pages_per_seq * p->page_size > (1 << 18))
        return reject(QA_STATUS_INVALID_PARAMS, "%s: positions up to %d supported (max_pages_per_seq * page_size = %lld)", fn,
                      1 << 18, (long long)p->max_pages_per_seq * p->page_size);
    if (!k || !v) return invalid(fn, "NULL tensor pointer");
    if (!aligned(k, 16) || !aligned(v, 16)) return invalid(fn, "k and v must be 16-byte aligned");
    if ((st = check_stride(fn, "ldq", ldq, (long long)p->n_q_heads * p->head_dim)) != QA_STATUS_OK ||
        (st = check_stride(fn, "ldkv", ldkv, (long long)p->n_kv_heads * p->head_dim)) != QA_STATUS_OK)
        return st;
    const qa::KvqAppend app{k, v, ldkv, rope};
    return decode_entry(fn, q, ldq, k_pages, v_pages, page_table, seq_lens, batch, out, p, &app);
}
