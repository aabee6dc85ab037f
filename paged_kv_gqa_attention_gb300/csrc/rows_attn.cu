// Attention of packed rows over paged states (qa_tree_attn, qa_cross_attn):
// the kernel for few rows a request, the merge of both kernels' split jobs,
// and the launch.  The kernel for many rows is rows_tiles.cu.
//
//   out[t][h] = softmax_j(q[t][h] . K_r[j] scale) V_r[j]
//
// over the request's n_past positions and the row's own ancestors in the tree
// behind them (tree), or over all its states (cross).
//
// Few rows (rows x group up to 16).  Bound by HBM: every key and value is
// read once, for all rows of its request and both query heads of its KV head.
// As in the single-token decode a persistent grid cuts the list of all pages
// into equal ranges (rows_attn.cuh) and a producer warp streams whole pages,
// all KV heads of 16 tokens, through a ring in shared memory.  The pages come
// as boxes of a tensor map that puts the heads outermost and swizzles the
// rows of 64 dims, so that 8 tokens of one head are read by one ldmatrix
// without a bank conflict.  One consumer warp a KV head: its rows (a query
// row's heads in turn) are the M of mma.sync m16n8k16, so that S stays in
// registers as the A operand of P V.  A tcgen05 tile would be 128 rows for
// these 16, and its S would have to come back from TMEM for the softmax;
// the tensor pipe is not what bounds.  64 requests of 4 to 8 rows over 2000 to
// 16000 positions (16 heads on 8): 345 us, 6.8 TB/s; 1 request of 8 over 257:
// 9.4 us, of which the pages are 0.2: a launch, lengths, page ids and a page one
// after another (5.5 us), the end of the grid and the merge.
//
// P enters P V as two bf16 terms (p truncated, and the rest rounded): about
// 16 bits of each probability, with fp32 statistics.  The running max of a
// row moves only when a page exceeds it by 2^8 (log2 units 8), so that the
// accumulator is seldom rescaled; the result does not depend on the
// reference.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "async.cuh"
#include "rows_attn.cuh"
#include "tc.cuh"
#include "tmap.h"

namespace qa {
namespace {

__device__ unsigned int g_status;

constexpr int kPage = 16;
constexpr int kMaxStages = 8;
constexpr float kSlack = 8.f;
constexpr int kMergeThreads = 512;  // of all CTAs of the merge on an SM
constexpr int kManyParts = 8;       // partials above which a CTA merges a row together
constexpr int kFewEach = 5, kMaxWorkers = 32 * 20;  // workers of a lane of the merge, and all

// Bytes of a stage: K and V of one page, each two halves of 64 dims.
__host__ __device__ constexpr uint32_t half_bytes(int hkv) { return (uint32_t)hkv * kPage * 128; }
__host__ __device__ constexpr uint32_t stage_bytes(int hkv) { return 4 * half_bytes(hkv); }

// CTAs an SM that few KV heads leave room for, and the ring's stages.
constexpr int ctas_per_sm(int hkv) { return hkv >= 5 ? 1 : hkv >= 3 ? 2 : 4; }
constexpr int stages_of(int hkv) {
    const int n = (int)(216u * 1024u / ctas_per_sm(hkv) / stage_bytes(hkv));
    return n < kMaxStages ? n : kMaxStages;
}

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Places of the list that a request takes before its pages, for its queries
// and its partial result.  With 0, 1, 2, 3 places: 32 requests of 8 rows over
// 200 to 2000 positions 38.3, 38.3, 36.6, 36.2 us, 16 over 100 to 500 18.0,
// 15.9, 15.9, 14.7, 5 of 1 to 4 over 13 to 390 7.3, 7.4, 7.6, 7.9, 64 of 4 to 8
// over 2000 to 16000 345, 347, 344, 349 (16 heads on 8; the third 8 on 8).
constexpr int kSwitch = 2;

// prefix[b] = places of the requests before b, by one warp.
__device__ __forceinline__ void count_pages(const RowsArgs &a, int *prefix, unsigned int *report) {
    const int lane = threadIdx.x & 31;
    int carry = 0;
    if (lane == 0) prefix[0] = 0;
    for (int base = 0; base < a.batch; base += 32) {
        const int b = base + lane;
        int v = 0;
        if (b < a.batch) {
            v = (request_of(a, b, report).keys + kPage - 1) / kPage;
            if (v > 0) v += kSwitch;
        }
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += u;
        }
        if (b < a.batch) prefix[b + 1] = carry + v;
        carry += __shfl_sync(0xffffffffu, v, 31);
    }
}

// First request whose places reach past place x.
__device__ __forceinline__ int request_at(const int *prefix, int batch, int x) {
    int l = 0, r = batch - 1;
    while (l < r) {
        const int mid = (l + r) >> 1;
        if (prefix[mid + 1] > x) r = mid; else l = mid + 1;
    }
    return l;
}

__device__ __forceinline__ void grid_wait() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

__global__ void __launch_bounds__(288, 1)
    few_rows_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
                    const __grid_constant__ RowsArgs a, int stages) {
    constexpr unsigned kAll = 0xffffffffu;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw), ring = (raw + 1023u) & ~1023u;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, hkv = a.hkv;
    const uint32_t half = half_bytes(hkv), stage_size = stage_bytes(hkv);
    const uint32_t full_k = ring + stages * stage_size, full_v = full_k + 8 * kMaxStages, empty = full_v + 8 * kMaxStages;
    int *page_ok = reinterpret_cast<int *>(smem_raw + (empty + 8 * kMaxStages - raw));
    const Waits wait{page_ok + kMaxStages, &g_status, kWaitLimitNs};
    int *prefix = page_ok + kMaxStages + 1;
    const int worker = blockIdx.x;
    if (warp == hkv && lane == 0) {
        tc::prefetch_tmap(&tk);
        tc::prefetch_tmap(&tv);
    }
    if (!a.early) grid_wait();
    if (warp == 0) {
        count_pages(a, prefix, worker == 0 ? &g_status : nullptr);
        if (lane == 0) {
            *wait.abort = 0;
            for (int s = 0; s < stages; ++s) {
                mbar_init(full_k + 8 * s, 1);
                mbar_init(full_v + 8 * s, 1);
                mbar_init(empty + 8 * s, hkv);
            }
            fence_mbar_init();
        }
    }
    __syncthreads();
    const int total = prefix[a.batch], per = (total + a.workers - 1) / a.workers;
    const int lo = (int)min(worker * (long long)per, (long long)total), hi = min(lo + per, total);
    const int b0 = lo < hi ? request_at(prefix, a.batch, lo) : 0, b_last = lo < hi ? request_at(prefix, a.batch, hi - 1) : -1;
    int first_ids = -1;
    if (warp == hkv && lo < hi) {
        const int p0 = prefix[b0] + kSwitch, j = max(lo - p0, 0) + lane;
        if (j < min(hi, prefix[b0 + 1]) - p0) first_ids = a.page_table[(size_t)b0 * a.max_pages + j];
    }
    if (a.early) grid_wait();
    for (int b = worker; b < a.batch; b += a.workers)
        if (prefix[b + 1] == prefix[b]) zero_rows(a, request_of(a, b, nullptr), threadIdx.x, blockDim.x);

    if (warp == hkv) {
        // the producer: lanes fetch page ids, lane 0 issues the copies
        if (lane == 0) {
            Split s = {0, 0, 0, 0};
            const int p0 = lo < hi ? prefix[b_last] + kSwitch : hi;
            if (p0 >= lo && p0 < hi && prefix[b_last + 1] > hi) {
                const Request r = request_of(a, b_last, nullptr);
                s.count = (prefix[b_last + 1] - 1) / per - worker + 1;
                s.first_slot = 2 * worker + (prefix[b_last] > lo);
                s.out_row = r.first;
                s.rows = r.rows * a.group;
            }
            a.splits[worker] = s;
        }
        int stage = 0, phase = 0, asked = 0;  // asked: pages whose stages were filled
        for (int b = b0; b <= b_last; ++b) {
            const int p0 = prefix[b] + kSwitch, p1 = prefix[b + 1];
            const int j0 = max(lo, p0) - p0, j1 = min(hi, p1) - p0;
            if (j0 >= j1) continue;
            const int32_t *row = a.page_table + (size_t)b * a.max_pages;
            for (int jb = j0; jb < j1; jb += 32) {
                const int mine = b == b0 && jb == j0 ? first_ids : jb + lane < j1 ? row[jb + lane] : -1;
                for (int j = jb; j < min(jb + 32, j1); ++j) {
                    const int id = __shfl_sync(kAll, mine, j - jb);
                    if (lane == 0) wait(empty + 8 * stage, phase ^ 1);
                    if (lane == 0 && !*wait.abort) {  // else the stage may still be read
                        ++asked;
                        const bool ok = id >= 0 && id < a.num_pages;
                        page_ok[stage] = ok;
                        if (ok) {
                            const uint32_t k = ring + stage * stage_size, v = k + 2 * half;
                            mbar_arrive_expect_tx(full_k + 8 * stage, 2 * half);
                            tc::tma_load_3d(k, &tk, 0, id * kPage, 0, full_k + 8 * stage);
                            tc::tma_load_3d(k + half, &tk, 64, id * kPage, 0, full_k + 8 * stage);
                            mbar_arrive_expect_tx(full_v + 8 * stage, 2 * half);
                            tc::tma_load_3d(v, &tv, 0, id * kPage, 0, full_v + 8 * stage);
                            tc::tma_load_3d(v + half, &tv, 64, id * kPage, 0, full_v + 8 * stage);
                        } else {
                            atomicOr(&g_status, QA_DEVICE_BAD_PAGE);
                            mbar_arrive(full_k + 8 * stage);
                            mbar_arrive(full_v + 8 * stage);
                        }
                    }
                    if (++stage == stages) stage = 0, phase ^= 1;
                }
            }
        }
        named_barrier(1, blockDim.x);
        if (lane == 0 && *wait.abort)  // a wait ran out: what is still under way writes shared memory
            for (int i = max(0, asked - stages); i < asked; ++i) {
                mbar_wait(full_k + 8 * (i % stages), i / stages & 1, &g_status);
                mbar_wait(full_v + 8 * (i % stages), i / stages & 1, &g_status);
            }
        return;
    }

    const int G = a.group, quad = lane >> 2, pair = 2 * (lane & 3), head = warp;
    // a lane's rows of ldmatrix: K, 8 keys by 8 dims each (keys 0..7, two chunks; keys 8..15); V, transposed, the other way round
    const uint32_t at_k = head * 2048 + ((lane >> 4) * 8 + (lane & 7)) * 128, chunk_k = (lane >> 3) & 1;
    const uint32_t at_v = head * 2048 + (((lane >> 3) & 1) * 8 + (lane & 7)) * 128, chunk_v = lane >> 4;
    int stage = 0, phase = 0;
    for (int b = b0; b <= b_last; ++b) {
        const int p0 = prefix[b] + kSwitch, p1 = prefix[b + 1];
        const int j0 = max(lo, p0) - p0, j1 = min(hi, p1) - p0;
        if (j0 >= j1) continue;
        const Request r = request_of(a, b, nullptr);
        const int rows = r.rows * G;
        uint32_t qf[8][4];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int row = quad + 8 * e;
            const bool live = row < rows;
            const uint16_t *src = a.q + (r.first + (row >> (G - 1))) * a.ldq + (head * G + (row & (G - 1))) * 128 + pair;
#pragma unroll
            for (int kk = 0; kk < 8; ++kk) {
                qf[kk][e] = live ? *reinterpret_cast<const uint32_t *>(src + 16 * kk) : 0u;
                qf[kk][e + 2] = live ? *reinterpret_cast<const uint32_t *>(src + 16 * kk + 8) : 0u;
            }
        }
        // the rows that each of the lane's two rows sees among the drafted ones (bit j: row j); reach doubles every round
        uint32_t seen[2] = {0, 0};
        if (a.tree && j1 * kPage > r.past) {
            int up = lane < r.rows ? parent_of(a, r.first, lane, &g_status) : -1;
            uint32_t mine = a.parents ? 1u << lane : 0xffffffffu >> (31 - lane);
            if (a.parents)
                for (int n = 0; n < 4; ++n) {
                    const uint32_t theirs = __shfl_sync(kAll, mine, up & 31);
                    const int next = __shfl_sync(kAll, up, up & 31);
                    if (up >= 0) mine |= theirs, up = next;
                }
#pragma unroll
            for (int e = 0; e < 2; ++e) seen[e] = __shfl_sync(kAll, mine, (quad + 8 * e) >> (G - 1));
        }
        float o[16][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
        bool odd = false;  // a drafted value that is not finite was met
#pragma unroll
        for (int n = 0; n < 16; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
        for (int j = j0; j < j1; ++j) {
            const uint32_t k = ring + stage * stage_size, v = k + 2 * half;
            wait(full_k + 8 * stage, phase);
            const bool ok = page_ok[stage];
            bool wrote = false;
            if (ok) {
                float s[2][4];
#pragma unroll
                for (int n = 0; n < 2; ++n) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
#pragma unroll
                for (int kk = 0; kk < 8; ++kk) {
                    uint32_t f[4];
                    ldmatrix4(f, k + (kk >> 2) * half + at_k + (((2 * (kk & 3) + chunk_k) ^ (lane & 7)) << 4));
                    mma16816(s[0], qf[kk], f[0], f[1]);
                    mma16816(s[1], qf[kk], f[2], f[3]);
                }
                const int behind = r.past - j * kPage;  // keys of this page that every row sees
                if (behind < kPage) {
#pragma unroll
                    for (int n = 0; n < 2; ++n)
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            const int t = n * 8 + pair + (x & 1), d = t - behind;
                            if (d >= 0 && !(a.tree && d < r.rows && (seen[x >> 1] >> d & 1))) s[n][x] = -INFINITY;
                        }
                }
                uint32_t hi_p[4], lo_p[4];
                float alpha[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float mx = fmaxf(fmaxf(s[0][2 * e], s[0][2 * e + 1]), fmaxf(s[1][2 * e], s[1][2 * e + 1]));
                    mx = fmaxf(mx, __shfl_xor_sync(kAll, mx, 1));
                    mx = fmaxf(mx, __shfl_xor_sync(kAll, mx, 2)) * a.scale_log2;
                    const float next = mx > m[e] + kSlack ? mx : m[e];
                    alpha[e] = next == m[e] ? 1.f : exp2_approx(m[e] - next);
                    m[e] = next;
                    const float ref = next == -INFINITY ? 0.f : next;
#pragma unroll
                    for (int n = 0; n < 2; ++n)
#pragma unroll
                        for (int x = 2 * e; x < 2 * e + 2; ++x) s[n][x] = exp2_approx(fmaf(s[n][x], a.scale_log2, -ref));
                    l[e] = l[e] * alpha[e] + ((s[0][2 * e] + s[0][2 * e + 1]) + (s[1][2 * e] + s[1][2 * e + 1]));
                }
                if (__any_sync(kAll, alpha[0] != 1.f || alpha[1] != 1.f)) {
#pragma unroll
                    for (int n = 0; n < 16; ++n) {
                        o[n][0] *= alpha[0], o[n][1] *= alpha[0];
                        o[n][2] *= alpha[1], o[n][3] *= alpha[1];
                    }
                }
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float x = s[n][2 * e], y = s[n][2 * e + 1];
                        const uint32_t w = __byte_perm(__float_as_uint(x), __float_as_uint(y), 0x7632);
                        hi_p[2 * n + e] = w;
                        lo_p[2 * n + e] = pack_bf16x2(x - bf16lo(w), y - bf16hi(w));
                    }
                wait(full_v + 8 * stage, phase);
                if (behind < kPage) {
                    // Slots that hold no key are zeroed, and of drafted values what is not finite, so that a probability
                    // of 0 meets nothing that it would not cancel; the rows that see such a value get it at the end.
                    const int n_keys = r.keys - j * kPage, from = max(behind, 0) * 16 + lane;
                    const auto chunk = [&](int c) { return v + (c >> 3 & 1) * half + head * 2048 + (c >> 4) * 128 + (c & 7) * 16; };
                    bool here = false;
                    for (int c = from; c < min(n_keys, kPage) * 16; c += 32) {
                        const uint4 x = lds128(chunk(c));
                        here |= not_finite(x.x) | not_finite(x.y) | not_finite(x.z) | not_finite(x.w);
                    }
                    here = __any_sync(kAll, here);
                    odd |= here;
                    for (int c = here ? from : max(n_keys, 0) * 16 + lane; c < kPage * 16; c += 32) {
                        uint4 x = make_uint4(0u, 0u, 0u, 0u);
                        if (c >> 4 < n_keys) {
                            x = lds128(chunk(c));
                            x = make_uint4(finite_or_zero(x.x), finite_or_zero(x.y), finite_or_zero(x.z), finite_or_zero(x.w));
                        }
                        tc::st_shared_v4(chunk(c), x.x, x.y, x.z, x.w);
                    }
                    wrote = true;
                    __syncwarp();
                }
#pragma unroll
                for (int c = 0; c < 16; c += 2) {
                    uint32_t f[4];
                    ldmatrix4_trans(f, v + (c >> 3) * half + at_v + ((((c & 7) + chunk_v) ^ (lane & 7)) << 4));
                    mma16816(o[c], hi_p, f[0], f[1]);
                    mma16816(o[c + 1], hi_p, f[2], f[3]);
                    mma16816(o[c], lo_p, f[0], f[1]);
                    mma16816(o[c + 1], lo_p, f[2], f[3]);
                }
            } else {
                wait(full_v + 8 * stage, phase);
            }
            if (wrote) tc::fence_proxy_async_smem();  // before the next copy into these bytes
            __syncwarp();
            if (lane == 0) mbar_arrive(empty + 8 * stage);
            if (++stage == stages) stage = 0, phase ^= 1;
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            l[e] += __shfl_xor_sync(kAll, l[e], 1);
            l[e] += __shfl_xor_sync(kAll, l[e], 2);
        }
        if (odd) {
            const int32_t *row = a.page_table + (size_t)b * a.max_pages;
            for (int pos = max(r.past, j0 * kPage); pos < min(r.keys, j1 * kPage); ++pos) {
                const int id = row[pos >> 4];
                if (id < 0 || id >= a.num_pages) continue;
                const uint16_t *src = a.v_pages + (((size_t)id * kPage + (pos & 15)) * hkv + head) * 128 + pair;
#pragma unroll
                for (int n = 0; n < 16; ++n) {
                    const uint32_t w = not_finite(*reinterpret_cast<const uint32_t *>(src + 8 * n));
#pragma unroll
                    for (int x = 0; x < 4; ++x)
                        if (seen[x >> 1] >> (pos - r.past) & 1) o[n][x] += x & 1 ? bf16hi(w) : bf16lo(w);
                }
            }
        }
        const bool whole = lo <= p0 && p1 <= hi;
        const int slot = 2 * worker + (prefix[b] > lo);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int row = quad + 8 * e;
            if (row >= rows) continue;
            if (whole) {
                const float inv = l[e] > 0.f ? 1.f / l[e] : l[e];
                uint16_t *dst = a.out + ((size_t)(r.first + (row >> (G - 1))) * a.hq + head * G + (row & (G - 1))) * 128 + pair;
#pragma unroll
                for (int n = 0; n < 16; ++n)
                    *reinterpret_cast<uint32_t *>(dst + 8 * n) = pack_bf16x2(o[n][2 * e] * inv, o[n][2 * e + 1] * inv);
            } else {
                const size_t at = ((size_t)slot * hkv + head) * a.block_rows + row;
                float *dst = a.acc + at * 128 + pair;
#pragma unroll
                for (int n = 0; n < 16; ++n) *reinterpret_cast<float2 *>(dst + 8 * n) = make_float2(o[n][2 * e], o[n][2 * e + 1]);
                if (pair == 0) *reinterpret_cast<float2 *>(a.ml + 2 * at) = make_float2(m[e], l[e]);
            }
        }
    }
    named_barrier(1, blockDim.x);
}

// A running merge of partials: the lane's four dims of one row.  The maxima
// pass over NaN, so that a worker whose scores of a row were all NaN leaves
// -inf beside a sum of NaN, as one that saw no key leaves it beside zeros:
// equal maxima, -inf too, have the weight 1, and every sum is taken.
struct Merge {
    float m = -INFINITY, sum = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    __device__ void add(float2 ml, float4 v) {
        const float next = fmaxf(m, ml.x);
        const float old = m == next ? 1.f : exp2_approx(m - next), now = ml.x == next ? 1.f : exp2_approx(ml.x - next);
        sum = sum * old + ml.y * now;
        acc.x = acc.x * old + v.x * now, acc.y = acc.y * old + v.y * now;
        acc.z = acc.z * old + v.z * now, acc.w = acc.w * old + v.w * now;
        m = next;
    }
};

// item / rows for fewer than 2^12 of each: half a row more keeps the quotient
// 2^-13 from a whole number, the approximate division is within 2^-21 of it.
__device__ __forceinline__ int head_of(const Split &s, int item) { return (int)__fdividef((float)item + 0.5f, (float)s.rows); }

// Merges row `item` (a head's rows in turn) of worker w's split over the
// partials first, first + by, .., in this order, four loads in flight.  Two
// rows of three, or three CTAs an SM, were no faster: 32 requests of eight
// drafted rows 40.1 and 38.2 us in all against 38.3.
__device__ __forceinline__ Merge merge_item(const RowsArgs &a, const Split &s, int w, int item, int first, int by) {
    constexpr int kFlight = 4;
    const int lane = threadIdx.x & 31;
    const int head = head_of(s, item);
    const size_t row = (size_t)head * a.block_rows + (item - head * s.rows);
    Merge g;
    for (int i = first; i < s.count; i += kFlight * by) {
        float2 ml[kFlight];
        float4 v[kFlight];
#pragma unroll
        for (int x = 0; x < kFlight; ++x)
            if (i + x * by < s.count) {
                const size_t slot = i + x * by == 0 ? s.first_slot : 2 * (w + i + x * by), at = slot * a.hkv * a.block_rows + row;
                ml[x] = __ldcg(reinterpret_cast<const float2 *>(a.ml) + at);
                v[x] = __ldcg(reinterpret_cast<const float4 *>(a.acc) + at * 32 + lane);
            }
#pragma unroll
        for (int x = 0; x < kFlight; ++x)
            if (i + x * by < s.count) g.add(ml[x], v[x]);
    }
    return g;
}

__device__ __forceinline__ void store_item(const RowsArgs &a, const Split &s, int item, const Merge &g) {
    const int head = head_of(s, item), row = item - head * s.rows, by = a.group - 1;  // group is 1 or 2
    const float inv = g.sum > 0.f ? 1.f / g.sum : g.sum;
    uint16_t *dst = a.out + ((size_t)(s.out_row + (row >> by)) * a.hq + head * a.group + (row & by)) * 128;
    reinterpret_cast<uint2 *>(dst)[threadIdx.x & 31] =
        make_uint2(pack_bf16x2(g.acc.x * inv, g.acc.y * inv), pack_bf16x2(g.acc.z * inv, g.acc.w * inv));
}

// A row of many partials by a CTA, whose warps take them in turn.
template <int THREADS>
__device__ __forceinline__ void merge_by_cta(const RowsArgs &a, const Split &s, int w, int item) {
    constexpr int kWarps = THREADS / 32;
    __shared__ float4 s_acc[kWarps][32];
    __shared__ float2 s_ml[kWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const Merge g = merge_item(a, s, w, item, warp, kWarps);
    s_acc[warp][lane] = g.acc;
    if (lane == 0) s_ml[warp] = make_float2(g.m, g.sum);
    __syncthreads();
    if (warp == 0) {
        Merge all;
        for (int x = 0; x < kWarps; ++x) all.add(s_ml[x], s_acc[x][lane]);
        store_item(a, s, item, all);
    }
    __syncthreads();
}

// The merge of both kernels' splits: every warp sums up the steps that all
// splits take, EACH workers a lane, and the CTAs take them in turn.
//
// CTAs of 128 threads find room beside the kernel for few rows, and wait there
// for its end; of 256, a row of very many partials takes fewer rounds.  128 and
// 256 threads, 8 rows a request, 16 heads on 8: 32 requests of 1100 positions
// 34.2 and 35.9 us, 16 of 300 13.2 and 15.3, 4 of 500 11.2 and 12.1, 1 of 257
// 9.7 and 9.4, 1 of 4000 14.3 and 12.1; 2 heads on 1: 64 of 1100 19.6 and 20.8,
// 1 of 4000 20.8 and 16.3.  Behind the kernel for many rows, which has few
// workers: 1 request of 64 rows over 8000 17.4 and 19.0.
template <int EACH, int THREADS>
__global__ void __launch_bounds__(THREADS, kMergeThreads / THREADS) merge_rows_kernel(const __grid_constant__ RowsArgs a) {
    constexpr unsigned kAll = 0xffffffffu;
    constexpr int kWarps = THREADS / 32;
    grid_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int steps[EACH], mine = 0;
#pragma unroll
    for (int x = 0; x < EACH; ++x) {
        const int w = lane * EACH + x;
        steps[x] = 0;
        if (w < a.workers) {
            const Split s = a.splits[w];
            const int n = s.rows * a.hkv;
            steps[x] = s.count == 0 ? 0 : s.count <= kManyParts ? (n + kWarps - 1) / kWarps : n;
        }
        mine += steps[x];
    }
    int before = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(kAll, before, o);
        if (lane >= o) before += u;
    }
    const int total = __shfl_sync(kAll, before, 31);
    before -= mine;
    for (int step = blockIdx.x; step < total; step += gridDim.x) {
        // the last lane that starts at or before the step, and which of its workers has it
        const int l = 31 - __clz(__ballot_sync(kAll, before <= step));
        int w = lane * EACH, begin = before, at = before;
#pragma unroll
        for (int x = 0; x < EACH; ++x) {
            if (steps[x] > 0 && at <= step) w = lane * EACH + x, begin = at;
            at += steps[x];
        }
        w = __shfl_sync(kAll, w, l), begin = __shfl_sync(kAll, begin, l);
        const Split s = a.splits[w];
        if (s.count > kManyParts) {
            merge_by_cta<THREADS>(a, s, w, step - begin);
        } else {
            const int item = (step - begin) * kWarps + warp;
            if (item < s.rows * a.hkv) store_item(a, s, item, merge_item(a, s, w, item, 0, 1));
        }
    }
}

// Three warps wait eight times each on barriers that nothing ever completes:
// one limit in all, not eight (qa_check_bounded_wait).
constexpr int kCheckThreads = 96, kCheckBars = 8;
__global__ void shared_waits_check_kernel(unsigned long long limit_ns) {
    __shared__ __align__(8) unsigned long long bars[kCheckBars];
    __shared__ int abort;
    const uint32_t b = smem_u32(bars);
    if (threadIdx.x == 0) {
        abort = 0;
        for (int i = 0; i < kCheckBars; ++i) mbar_init(b + 8 * i, 1);
        fence_mbar_init();
    }
    __syncthreads();
    const Waits wait{&abort, &g_status, limit_ns};
    for (int i = 0; i < kCheckBars; ++i) wait(b + 8 * i, 0);
}

struct Plan {
    bool few;
    int workers, block_rows;
    size_t acc, ml, splits, total;
};

// Rows times group up to which the rows of a request are few: one m16 block.
// With two blocks (32 rows, 32 requests of 200..2000 positions) mma.sync took
// 45.3 us against 42.8 of rows_tiles.cu, with eight (128 rows, 24 requests of
// 500..8000) 322 us against 102: 48 products a page, head and block at a
// measured 2048 multiply-adds in 4.7 clocks an SM are slower than HBM from two
// blocks on.
constexpr int kFewRows = 16;

int sm_count() {
    int device = 0, sms = 0;
    if (cudaGetDevice(&device) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device) != cudaSuccess)
        return 0;
    return sms;
}

bool plan_of(int max_rows, int hq, int hkv, Plan *p) {
    const int group = hq / hkv, sms = sm_count();
    if (sms <= 0) return false;
    *p = {};
    p->few = (long long)max_rows * group <= kFewRows;
    p->workers = p->few ? sms * ctas_per_sm(hkv) : rows_tiles_workers(hkv);
    p->block_rows = p->few ? 16 : 128;
    if (p->workers > kMaxWorkers) p->workers = kMaxWorkers;
    const size_t rows = (size_t)2 * p->workers * hkv * p->block_rows;
    // Behind the region that the decodes of either cache have their arrival counters in, which have to be zero between
    // calls: so one workspace may serve all of them in turn.
    p->splits = (size_t)kDecodeMaxBatch * 8 * sizeof(int32_t);
    p->ml = p->splits + ((sizeof(Split) * p->workers + 255) & ~(size_t)255);
    p->acc = p->ml + ((rows * 2 * sizeof(float) + 255) & ~(size_t)255);
    p->total = p->acc + rows * 128 * sizeof(float);
    return true;
}

// Pools as {dims, token slots, KV heads}: a box is one page's 64 dims of all
// heads, the rows of 16 tokens of a head together.
bool make_pool_tmap(CUtensorMap *map, const void *base, int hkv, long long slots) {
    PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
    if (!enc) return false;
    cuuint64_t dims[3] = {128, (cuuint64_t)slots, (cuuint64_t)hkv};
    cuuint64_t strides[2] = {(cuuint64_t)hkv * 256, 256};
    cuuint32_t box[3] = {64, 16, (cuuint32_t)hkv}, estr[3] = {1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Pools as {64 dims, 8 tokens, halves of the dims, groups of 8 tokens, KV
// heads}: a box is one page of a head, its groups one after another, of each
// the first 64 dims and then the others.
bool make_head_tmap(CUtensorMap *map, const void *base, int hkv, long long slots) {
    PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
    if (!enc) return false;
    const cuuint64_t row = (cuuint64_t)hkv * 256;
    cuuint64_t dims[5] = {64, 8, 2, (cuuint64_t)slots / 8, (cuuint64_t)hkv};
    cuuint64_t strides[4] = {row, 128, 8 * row, 256};
    cuuint32_t box[5] = {64, 8, 2, 2, 1}, estr[5] = {1, 1, 1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<void *>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Packed query rows as {dims, heads, rows}: a box is 64 dims of a KV head's
// `group` heads in 128 / group rows.
bool make_query_tmap(CUtensorMap *map, const void *base, int hq, long long rows, long long ld, int group) {
    PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
    if (!enc) return false;
    cuuint64_t dims[3] = {128, (cuuint64_t)hq, (cuuint64_t)rows};
    cuuint64_t strides[2] = {256, (cuuint64_t)ld * 2};
    cuuint32_t box[3] = {64, (cuuint32_t)group, (cuuint32_t)(128 / group)}, estr[3] = {1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

// Enough for calls of max_rows or fewer, whichever kernel they take.
size_t rows_attn_workspace_bytes(int max_rows, int n_q_heads, int n_kv_heads) {
    const int group = n_q_heads / n_kv_heads;
    size_t most = 0;
    for (int n : {kFewRows / group, max_rows}) {
        Plan p;
        if (!plan_of(n < max_rows ? n : max_rows, n_q_heads, n_kv_heads, &p)) return 0;
        if (p.total > most) most = p.total;
    }
    return most;
}

cudaError_t launch_rows_attn(const RowsAttn &x, const qa_attn_params &p, float scale, cudaStream_t stream) {
    Plan plan;
    if (!plan_of(x.max_rows, p.n_q_heads, p.n_kv_heads, &plan)) return cudaErrorInvalidDevice;
    RowsArgs a = {};
    uint8_t *ws = static_cast<uint8_t *>(p.workspace);
    a.q = static_cast<const uint16_t *>(x.q);
    a.v_pages = static_cast<const uint16_t *>(x.v_pages);
    a.out = static_cast<uint16_t *>(x.out);
    a.ldq = x.ldq ? x.ldq : (long long)p.n_q_heads * 128;
    a.cu = x.cu_seqlens;
    a.past = x.past;
    a.parents = x.parents;
    a.page_table = x.page_table;
    a.acc = reinterpret_cast<float *>(ws + plan.acc);
    a.ml = reinterpret_cast<float *>(ws + plan.ml);
    a.splits = reinterpret_cast<Split *>(ws + plan.splits);
    a.batch = x.batch;
    a.rows = x.rows;
    a.max_rows = x.max_rows;
    a.hq = p.n_q_heads;
    a.hkv = p.n_kv_heads;
    a.group = p.n_q_heads / p.n_kv_heads;
    a.max_pages = p.max_pages_per_seq;
    a.num_pages = p.num_pages;
    a.block_rows = plan.block_rows;
    a.workers = plan.workers;
    a.tree = x.tree;
    a.early = (p.abi_version >= 2 && p.stable_metadata >= 1) ? 1 : 0;
    a.scale_log2 = scale * kLog2e;
    CUtensorMap tk, tv;
    const long long slots = (long long)p.num_pages * kPage;
    const auto make = plan.few ? make_pool_tmap : make_head_tmap;
    if (!make(&tk, x.k_pages, a.hkv, slots) || !make(&tv, x.v_pages, a.hkv, slots)) return cudaErrorInvalidValue;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t e;
    if (plan.few) {
        const int stages = stages_of(a.hkv);
        cfg.gridDim = dim3((unsigned)plan.workers);
        cfg.blockDim = dim3((a.hkv + 1) * 32);
        cfg.dynamicSmemBytes = 1024 + stages * stage_bytes(a.hkv) + 3 * 8 * kMaxStages + 4 * (kMaxStages + 1) + 4 * (x.batch + 1);
        // the most of any call, so that host threads' calls cannot lower one another's
        e = cudaFuncSetAttribute(few_rows_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
        if (e != cudaSuccess) return e;
        e = cudaLaunchKernelEx(&cfg, few_rows_kernel, tk, tv, a, stages);
    } else {
        CUtensorMap tq;
        if (!make_query_tmap(&tq, x.q, a.hq, x.rows, a.ldq, a.group)) return cudaErrorInvalidValue;
        e = launch_rows_tiles(a, tq, tk, tv, stream);
    }
    if (e != cudaSuccess) return e;
    const int threads = plan.few && plan.workers > 16 * x.batch ? 256 : 128;  // workers of a request on average: many partials a row, or not
    const bool small = plan.workers <= 32 * kFewEach;
    constexpr int kEach = kMaxWorkers / 32;
    const auto merge = threads == 256 ? (small ? merge_rows_kernel<kFewEach, 256> : merge_rows_kernel<kEach, 256>)
                                      : (small ? merge_rows_kernel<kFewEach, 128> : merge_rows_kernel<kEach, 128>);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = 0;
    cfg.gridDim = dim3((unsigned)(kMergeThreads / threads * sm_count()));
    return cudaLaunchKernelEx(&cfg, merge, a);
}

cudaError_t launch_shared_waits_check(unsigned int limit_us, cudaStream_t stream) {
    shared_waits_check_kernel<<<1, kCheckThreads, 0, stream>>>((unsigned long long)limit_us * 1000ull);
    return cudaGetLastError();
}

unsigned int status_read_clear_rows_attn(cudaStream_t stream, cudaError_t *err) {
    unsigned int v = 0, zero = 0;
    cudaError_t e = cudaMemcpyFromSymbolAsync(&v, g_status, sizeof v, 0, cudaMemcpyDeviceToHost, stream);
    if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
    if (e == cudaSuccess && v) e = cudaMemcpyToSymbolAsync(g_status, &zero, sizeof zero, 0, cudaMemcpyHostToDevice, stream);
    if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
    if (e != cudaSuccess) {
        if (err) *err = e;
        return v;
    }
    return v | status_read_clear_rows_tiles(stream, err);
}

}  // namespace qa
