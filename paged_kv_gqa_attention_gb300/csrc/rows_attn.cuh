// What the two kernels of qa_tree_attn and qa_cross_attn share: a call's
// arguments, how its key tiles are cut into workers, and the partial results
// that one worker leaves for the merge.
//
// Work split.  A job is a request's block of query rows (up to `rows_a_block`
// of them); its key tiles run over the request's positions.  All jobs' tiles
// form one list, requests in order and a request's blocks in order, with a few
// places before a job's tiles for what it costs beside them; worker w of n
// takes the places [w per, (w + 1) per), per = ceil(total / n).
// A job inside one worker is finished by it.  Of a job that spans several,
// each leaves fp32 (max, sum, accumulator) rows in a slot of its own, 2 w for
// the first job of its range and 2 w + 1 for one that begins inside it and
// goes on behind it; and the worker that has the job's first tile describes
// it in its `Split`, for the merge kernel behind (merge_rows_kernel).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "qa_internal.h"
#include "waits.cuh"

namespace qa {

// A job that spans several workers: rows [0, rows) (a query row's `group`
// heads in turn) of every KV head, in the first worker's slot and in the even
// slots of the `count - 1` workers behind it.
struct Split {
    int count, first_slot, out_row, rows;
};

struct RowsArgs {
    const uint16_t *q, *v_pages;
    uint16_t *out;
    long long ldq;
    const int32_t *cu, *past, *parents, *page_table;
    float *acc;     // [slots][hkv][block rows][128]
    float *ml;      // [slots][hkv][block rows][2]: running max (log2 units) and sum
    Split *splits;  // [workers]
    int batch, rows, max_rows, hq, hkv, group, max_pages, num_pages;
    int block_rows;  // rows of a slot: query rows times group
    int workers;
    int tree, early;
    float scale_log2;
};

// A request's rows and keys; keys 0 where it has nothing to attend to.
struct Request {
    int first, rows, past, keys;
    bool valid;  // its rows are its own: they may be written
};

__device__ __forceinline__ Request request_of(const RowsArgs &a, int first, int end, int past, unsigned int *report) {
    Request r = {first, 0, 0, 0, first >= 0 && end >= first && end <= a.rows};
    if (!r.valid) {
        if (report) atomicOr(report, QA_DEVICE_BAD_SEGMENTS);
        return r;
    }
    r.rows = end - first;
    const long long keys = (long long)past + (a.tree ? r.rows : 0);
    if (r.rows > a.max_rows || past < 0 || keys > (long long)a.max_pages * 16) {
        if (report) atomicOr(report, QA_DEVICE_BAD_LENGTH);
        return r;
    }
    r.past = past;
    r.keys = r.rows > 0 ? (int)keys : 0;
    return r;
}
__device__ __forceinline__ Request request_of(const RowsArgs &a, int b, unsigned int *report) {
    return request_of(a, a.cu[b], a.cu[b + 1], a.past[b], report);
}

// A request with nothing to attend to has zero rows.
__device__ __forceinline__ void zero_rows(const RowsArgs &a, const Request &r, int thread, int threads) {
    if (!r.valid || r.keys > 0) return;
    uint4 *dst = reinterpret_cast<uint4 *>(a.out + (size_t)r.first * a.hq * 128);
    const long long n = (long long)r.rows * a.hq * 16;
    for (long long i = thread; i < n; i += threads) dst[i] = make_uint4(0u, 0u, 0u, 0u);
}

// Row i's parent in its request's tree, checked.
__device__ __forceinline__ int parent_of(const RowsArgs &a, int first, int i, unsigned int *report) {
    if (!a.parents) return i - 1;
    const int p = a.parents[first + i];
    if (p >= -1 && p < i) return p;
    atomicOr(report, QA_DEVICE_BAD_TREE);
    return -1;
}

// A bf16 pair's elements that are not finite become 0.
__device__ __forceinline__ uint32_t finite_or_zero(uint32_t w) {
    if ((w & 0x7f80u) == 0x7f80u) w &= 0xffff0000u;
    if ((w & 0x7f800000u) == 0x7f800000u) w &= 0x0000ffffu;
    return w;
}
// The elements that are not finite, the others 0.
__device__ __forceinline__ uint32_t not_finite(uint32_t w) { return w ^ finite_or_zero(w); }

cudaError_t launch_rows_tiles(const RowsArgs &a, const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv,
                              cudaStream_t stream);
unsigned int status_read_clear_rows_tiles(cudaStream_t stream, cudaError_t *err);
int rows_tiles_workers(int hkv);

}  // namespace qa
