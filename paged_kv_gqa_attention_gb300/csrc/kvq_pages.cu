// Writing packed K/V rows into 4-bit pages (qa_kvq_write) and reading them
// back (qa_kvq_read).
//
// One warp takes one KV head of one page: its 16 tokens x 128 dims of K, of
// V, or (reading) of both.  Lane 4 r + c owns exactly the bytes of the page
// that it owns as a tensor-core fragment in decode (kvq.cuh): of K, tokens r
// and r + 8, the 8 dims [8c, 8c + 8) of each group; of V, tokens 2c, 2c + 1
// (+ 8), the 4 dims [4r, 4r + 4) of each group.  So a group of K is spread
// over the 4 lanes of equal r and one of V over the 8 of equal c, and every
// code a lane makes goes into its own words.
//
// Both move 512 bytes of rows and 160 of pages a token and KV head.  35032
// rows of 8 heads (188 MB) are written in 38.4 us, 4.9 TB/s, 72 % of the copy
// rate.  Nothing is full (640 instructions a warp of K or V, issue slots 58 %,
// ALU 48 %, DRAM 60 %): a CTA of one page begins its chain from cu_seqlens to
// the rows with nothing in flight.  56691 rows (305 MB) are read back in 48.7
// us, 6.26 TB/s, 92 %; few rows wait on the loop's loads, each behind the
// stores before it (16 requests of 53..430 4.96 us).  Warps that walk over pages
// with the next rows on their way into shared memory were slower (written and
// read back 77..81 us against 72.7): fewer fit, and it is warps that cover the
// chains of the quantiser.
#include <cuda_runtime.h>
#include <stdint.h>

#include "kvq.cuh"
#include "qa_internal.h"

namespace qa {
namespace {

__device__ unsigned int g_status;

struct PagesArgs {
    const uint16_t *k_in, *v_in;  // write: packed rows
    uint16_t *k_out, *v_out;      // read: packed rows
    long long ldk, ldv;
    const int32_t *cu, *n_past, *page_table;
    uint8_t *k_pages, *v_pages;
    int batch, total, hkv, max_pages, num_pages, early;
};

// What a CTA works on: slots [t0, t1) of a page, whose slot t holds packed
// row `row0 + t` (row0 may be negative: only rows of [t0, t1) exist).
struct Job {
    int t0, t1;
    long long row0;
    size_t entry;  // of the page table
};

// The job of page id `id`; false when there is none.  Warp-collective.
__device__ __forceinline__ bool find_job(const PagesArgs &a, int id, Job &j, bool report) {
    const int lane = threadIdx.x & 31;
    // the last request with S(r) <= id: of the last 32 candidates each lane reads all there is to know of one, so that
    // a small batch costs one round trip to memory (larger ones one more for each factor of 32)
    int lo = 0, n = a.batch;  // the answer is in [lo, lo + n), or there is none
    while (n > 32) {
        const int step = (n + 31) / 32;
        const int r = lo + lane * step;
        const bool le = lane * step < n && a.cu[r] / 16 + 2 * r <= id;
        const unsigned votes = __ballot_sync(0xffffffffu, le);
        const int last = votes ? 31 - __clz(votes) : 0;
        n = min(step, n - last * step);
        lo += last * step;
    }
    const int mine = min(lo + lane, lo + n - 1);
    const int c0_own = a.cu[mine], c1_own = a.cu[mine + 1], past_own = a.n_past ? a.n_past[mine] : 0;
    const unsigned votes = __ballot_sync(0xffffffffu, lane < n && c0_own / 16 + 2 * mine <= id);
    const int from = votes ? 31 - __clz(votes) : 0;
    const int r = lo + from;
    const int c0 = __shfl_sync(0xffffffffu, c0_own, from), c1 = __shfl_sync(0xffffffffu, c1_own, from);
    const int past = __shfl_sync(0xffffffffu, past_own, from);
    if (c0 < 0 || c1 > a.total || c1 < c0) {
        if (report) atomicOr(&g_status, QA_DEVICE_BAD_SEGMENTS);
        return false;
    }
    const long long cap = (long long)a.max_pages * kKvqTokens;
    if (past < 0 || past > cap) {
        if (report) atomicOr(&g_status, QA_DEVICE_BAD_LENGTH);
        return false;
    }
    long long end = (long long)past + (c1 - c0);
    if (end > cap) {
        if (report) atomicOr(&g_status, QA_DEVICE_BAD_LENGTH);
        end = cap;
    }
    const int k = id - (c0 / 16 + 2 * r);
    if (k < 0) return false;
    const long long pg = (long long)past / kKvqTokens + k;
    const long long p0 = pg * kKvqTokens;
    if (p0 >= end) return false;
    j.t0 = (int)max(0LL, past - p0);  // t1 where there are no rows
    j.t1 = (int)min((long long)kKvqTokens, end - p0);
    j.row0 = c0 + p0 - past;
    j.entry = (size_t)r * a.max_pages + pg;
    return true;
}

// Whether a job's page is one.
__device__ __forceinline__ bool page_ok(const PagesArgs &a, int page) {
    if (page >= 0 && page < a.num_pages) return true;
    if (threadIdx.x == 0) atomicOr(&g_status, QA_DEVICE_BAD_PAGE);
    return false;
}

// The CTA's job, found by its first warp.
__device__ __forceinline__ bool cta_job(const PagesArgs &a, Job &j) {
    __shared__ Job shared;
    if (threadIdx.x < 32) {
        Job own = {0, 0, 0, 0};
        find_job(a, blockIdx.x, own, threadIdx.x == 0);
        if (threadIdx.x == 0) shared = own;
    }
    __syncthreads();
    j = shared;
    return j.t1 > j.t0;
}

// cu_seqlens as a whole, checked once a call.
__device__ __forceinline__ void check_segments(const PagesArgs &a) {
    if (blockIdx.x != 0) return;
    bool bad = threadIdx.x == 0 && (a.cu[0] != 0 || a.cu[a.batch] != a.total);
    for (int r = threadIdx.x; r < a.batch; r += blockDim.x) bad |= a.cu[r] > a.cu[r + 1];
    if (bad) atomicOr(&g_status, QA_DEVICE_BAD_SEGMENTS);
}

__device__ __forceinline__ void wait_dependency() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {  // of bf16 pairs; NaN stays
    uint32_t d;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
// (maximum, minus minimum) of the two halves of maxima and of minima: a range that max2 alone reduces further.
__device__ __forceinline__ uint32_t range_of(uint32_t mx, uint32_t mn) {
    return max2(__byte_perm(mx, mn, 0x5410) ^ 0x80000000u, __byte_perm(mx, mn, 0x7632) ^ 0x80000000u);
}
__device__ __forceinline__ KvqGroup group_of(uint32_t range) {
    return kvq_group(bf16lo(range >> 16 ^ 0x8000u), bf16lo(range));
}

// One step of a reduction over lanes that shares the results out: of 2 N
// ranges, lanes with the bit `o` clear go on with the first N, the others
// with the last N.
template <int N>
__device__ __forceinline__ void reduce_half(uint32_t *x, int lane, int o) {
    const bool upper = lane & o;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const uint32_t got = __shfl_xor_sync(0xffffffffu, upper ? x[i] : x[i + N], o);
        x[i] = max2(upper ? x[i + N] : x[i], got);
    }
}

// Codes of 2 N values in the low 8 N bits: rint((x - m) r) by adding
// 1.5 * 2^23 (kvq_code), whose bits, 0x4b400000 + n, a multiply-add chain
// shifts together; what the constants add up to is taken off in advance.
template <int N>
__device__ __forceinline__ uint32_t codes_of(const uint32_t (&w)[N], float m, float r) {
    constexpr uint32_t kOffset = 0x4b400000u * (N == 4 ? 0x11111111u : 0x1111u);
    uint32_t code = 0;
#pragma unroll
    for (int i = N - 1; i >= 0; --i) {
        // the product is rounded by itself: the sums are not packed, or the two would be joined
        const float2 d = fmul2(fsub2(make_float2(bf16lo(w[i]), bf16hi(w[i])), make_float2(m, m)), make_float2(r, r));
        code = code * 16u + __float_as_uint(__fadd_rn(d.y, 12582912.0f));
        code = code * 16u + __float_as_uint(__fadd_rn(d.x, 12582912.0f));
    }
    return code - kOffset;
}

// The K rows of a job: tokens r and r + 8, dims [32 g + 8 c, + 8) of each
// group.  Slots without a row read a neighbour's, and write nothing.  The
// reduction over a group's lanes ends with each lane holding two groups of
// one token, whose parameters it computes, writes, and leaves in `params`
// (m and 1 / s of two groups, by token and group pair) for the others.
__device__ __forceinline__ void write_k(const PagesArgs &a, const Job &j, int h, int lane, float4 *params) {
    const int r = lane >> 2, c = lane & 3;
    const auto in = [&](int t) { return t >= j.t0 && t < j.t1; };
    const uint16_t *row = a.k_in + j.row0 * a.ldk + h * kKvqDim + 8 * c;
    const int id = a.page_table[j.entry];  // on its way together with the rows
    uint4 k[2][4];
#pragma unroll
    for (int y = 0; y < 2; ++y) {
        const uint16_t *p = row + (long long)min(max(r + 8 * y, j.t0), j.t1 - 1) * a.ldk;
#pragma unroll
        for (int g = 0; g < 4; ++g) k[y][g] = *reinterpret_cast<const uint4 *>(p + 32 * g);
    }
    if (!page_ok(a, id)) return;
    uint8_t *page = a.k_pages + ((size_t)id * a.hkv + h) * kKvqHeadBytes;
    uint32_t range[8];
#pragma unroll
    for (int y = 0; y < 2; ++y)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            const uint4 w = k[y][g];
            range[4 * y + g] = range_of(max2(max2(w.x, w.y), max2(w.z, w.w)), min2(min2(w.x, w.y), min2(w.z, w.w)));
        }
    reduce_half<4>(range, lane, 1);  // token r + 8 (c & 1)
    reduce_half<2>(range, lane, 2);  // groups 2 (c >> 1), + 1
    const KvqGroup ga = group_of(range[0]), gb = group_of(range[1]);
    const int own = r + 8 * (c & 1);
    if (in(own)) *reinterpret_cast<uint2 *>(page + kvq_param_offset(own, 2 * (c >> 1))) = make_uint2(ga.sm, gb.sm);
    params[2 * own + (c >> 1)] = make_float4(ga.m, ga.r, gb.m, gb.r);
    const bool nan = __any_sync(0xffffffffu, isnan(ga.r) || isnan(gb.r));
    __syncwarp();
#pragma unroll
    for (int y = 0; y < 2; ++y) {
        const int t = r + 8 * y;
        uint32_t code[4];
#pragma unroll
        for (int g = 0; g < 4; g += 2) {
            const float4 p = params[2 * t + g / 2];
            const uint32_t w0[4] = {k[y][g].x, k[y][g].y, k[y][g].z, k[y][g].w};
            const uint32_t w1[4] = {k[y][g + 1].x, k[y][g + 1].y, k[y][g + 1].z, k[y][g + 1].w};
            code[g] = codes_of<4>(w0, p.x, p.y);
            code[g + 1] = codes_of<4>(w1, p.z, p.w);
            if (nan) code[g] = isnan(p.y) ? 0u : code[g], code[g + 1] = isnan(p.w) ? 0u : code[g + 1];
        }
        if (in(t)) *reinterpret_cast<uint4 *>(page + t * 64 + c * 16) = make_uint4(code[0], code[1], code[2], code[3]);
    }
}

// The V rows of a job: tokens 8 u + 2 c + e, dims [32 g + 4 r, + 4).
__device__ __forceinline__ void write_v(const PagesArgs &a, const Job &j, int h, int lane, float4 *params) {
    const int r = lane >> 2, c = lane & 3;
    const auto in = [&](int t) { return t >= j.t0 && t < j.t1; };
    const uint16_t *row = a.v_in + j.row0 * a.ldv + h * kKvqDim + 4 * r;
    const int id = a.page_table[j.entry];
    uint2 v[4][4];  // [2 u + e][g]
#pragma unroll
    for (int y = 0; y < 4; ++y) {
        const uint16_t *p = row + (long long)min(max(8 * (y >> 1) + 2 * c + (y & 1), j.t0), j.t1 - 1) * a.ldv;
#pragma unroll
        for (int g = 0; g < 4; ++g) v[y][g] = *reinterpret_cast<const uint2 *>(p + 32 * g);
    }
    if (!page_ok(a, id)) return;
    uint8_t *page = a.v_pages + ((size_t)id * a.hkv + h) * kKvqHeadBytes;
    uint32_t range[16];  // [e][u][g], so that each step halves it
#pragma unroll
    for (int y = 0; y < 4; ++y)
#pragma unroll
        for (int g = 0; g < 4; ++g) range[8 * (y & 1) + 4 * (y >> 1) + g] = range_of(max2(v[y][g].x, v[y][g].y), min2(v[y][g].x, v[y][g].y));
    reduce_half<8>(range, lane, 4);
    reduce_half<4>(range, lane, 8);
    reduce_half<2>(range, lane, 16);
    const KvqGroup ga = group_of(range[0]), gb = group_of(range[1]);
    const int own = 8 * (r >> 1 & 1) + 2 * c + (r & 1);
    if (in(own)) *reinterpret_cast<uint2 *>(page + kvq_param_offset(own, 2 * (r >> 2))) = make_uint2(ga.sm, gb.sm);
    params[2 * own + (r >> 2)] = make_float4(ga.m, ga.r, gb.m, gb.r);
    const bool nan = __any_sync(0xffffffffu, isnan(ga.r) || isnan(gb.r));
    __syncwarp();
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        uint32_t code[2][4];
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int g = 0; g < 4; g += 2) {
                const float4 p = params[2 * (8 * u + 2 * c + e) + g / 2];
                const uint32_t w0[2] = {v[2 * u + e][g].x, v[2 * u + e][g].y}, w1[2] = {v[2 * u + e][g + 1].x, v[2 * u + e][g + 1].y};
                code[e][g] = codes_of<2>(w0, p.x, p.y);
                code[e][g + 1] = codes_of<2>(w1, p.z, p.w);
                if (nan) code[e][g] = isnan(p.y) ? 0u : code[e][g], code[e][g + 1] = isnan(p.w) ? 0u : code[e][g + 1];
            }
        uint8_t *dst = page + u * 512 + lane * 16;
        const int t = 8 * u + 2 * c;
        if (in(t) && in(t + 1)) {
            *reinterpret_cast<uint4 *>(dst) = make_uint4(__byte_perm(code[0][0], code[1][0], 0x5410), __byte_perm(code[0][1], code[1][1], 0x5410),
                                                         __byte_perm(code[0][2], code[1][2], 0x5410), __byte_perm(code[0][3], code[1][3], 0x5410));
        } else {  // the neighbour's codes stay as they are
#pragma unroll
            for (int e = 0; e < 2; ++e)
                if (in(t + e))
#pragma unroll
                    for (int g = 0; g < 4; ++g) *reinterpret_cast<uint16_t *>(dst + g * 4 + e * 2) = (uint16_t)code[e][g];
        }
    }
}

// blockIdx.y 0 writes K, 1 writes V: with half the rows a warp holds, twice
// the warps fit, and their loads cover one another's arithmetic.
__global__ void __launch_bounds__(256, 4) kvq_write_kernel(const __grid_constant__ PagesArgs a) {
    __shared__ float4 params[8][32];
    if (!a.early) wait_dependency();
    const int h = threadIdx.x >> 5, lane = threadIdx.x & 31;
    Job j;
    const bool work = cta_job(a, j);
    if (blockIdx.y == 0) check_segments(a);
    if (a.early) wait_dependency();
    if (!work) return;
    if (blockIdx.y == 0) write_k(a, j, h, lane, params[h]);
    else write_v(a, j, h, lane, params[h]);
}

// The value of code n of a group.
__device__ __forceinline__ float kvq_value(uint32_t n, float s, float m) { return fmaf(s, (float)n, m); }

__global__ void __launch_bounds__(256) kvq_read_kernel(const __grid_constant__ PagesArgs a) {
    if (!a.early) wait_dependency();
    const int h = threadIdx.x >> 5, lane = threadIdx.x & 31;
    Job j;
    const bool work = cta_job(a, j);
    check_segments(a);
    if (a.early) wait_dependency();
    if (!work) return;
    const int id = a.page_table[j.entry];
    if (!page_ok(a, id)) return;
    const int r = lane >> 2, c = lane & 3;
    const uint8_t *kp = a.k_pages + ((size_t)id * a.hkv + h) * kKvqHeadBytes;
    const uint8_t *vp = a.v_pages + ((size_t)id * a.hkv + h) * kKvqHeadBytes;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        const int t = r + 8 * half;
        if (t < j.t0 || t >= j.t1) continue;
        const uint4 w4 = *reinterpret_cast<const uint4 *>(kp + t * 64 + c * 16);
        const uint4 p4 = *reinterpret_cast<const uint4 *>(kp + kvq_param_offset(t, 0));
        const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w}, p[4] = {p4.x, p4.y, p4.z, p4.w};
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            const float s = bf16lo(p[g]), m = bf16hi(p[g]);
            uint32_t o[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                o[i] = pack_bf16x2(kvq_value((w[g] >> (8 * i)) & 15u, s, m), kvq_value((w[g] >> (8 * i + 4)) & 15u, s, m));
            *reinterpret_cast<uint4 *>(a.k_out + ((j.row0 + t) * a.hkv + h) * kKvqDim + 32 * g + 8 * c) =
                make_uint4(o[0], o[1], o[2], o[3]);
        }
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        const uint4 w4 = *reinterpret_cast<const uint4 *>(vp + u * 512 + lane * 16);
        const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int t = 8 * u + 2 * c + e;
            if (t < j.t0 || t >= j.t1) continue;
            const uint4 p4 = *reinterpret_cast<const uint4 *>(vp + kvq_param_offset(t, 0));
            const uint32_t p[4] = {p4.x, p4.y, p4.z, p4.w};
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const float s = bf16lo(p[g]), m = bf16hi(p[g]);
                const uint32_t n = w[g] >> (16 * e);
                *reinterpret_cast<uint2 *>(a.v_out + ((j.row0 + t) * a.hkv + h) * kKvqDim + 32 * g + 4 * r) =
                    make_uint2(pack_bf16x2(kvq_value(n & 15u, s, m), kvq_value((n >> 4) & 15u, s, m)),
                               pack_bf16x2(kvq_value((n >> 8) & 15u, s, m), kvq_value((n >> 12) & 15u, s, m)));
            }
        }
    }
}

cudaError_t launch_pages(const PagesArgs &a, bool write, cudaStream_t stream) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.total / kKvqTokens + 2 * a.batch), write ? 2u : 1u);
    cfg.blockDim = dim3((unsigned)(a.hkv * 32));
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, write ? kvq_write_kernel : kvq_read_kernel, a);
}

PagesArgs pages_args(const int32_t *cu, const int32_t *n_past, int batch, int total, const int32_t *page_table,
                     const qa_attn_params &p) {
    PagesArgs a = {};
    a.cu = cu;
    a.n_past = n_past;
    a.page_table = page_table;
    a.batch = batch;
    a.total = total;
    a.hkv = p.n_kv_heads;
    a.max_pages = p.max_pages_per_seq;
    a.num_pages = p.num_pages;
    a.early = (p.abi_version >= 2 && p.stable_metadata >= 1) ? 1 : 0;
    return a;
}

}  // namespace

cudaError_t launch_kvq_write(const void *k, long long ldk, const void *v, long long ldv, const int32_t *cu_seqlens,
                             const int32_t *n_past, int batch, int total_tokens, const int32_t *page_table,
                             void *k_pages, void *v_pages, const qa_attn_params &p, cudaStream_t stream) {
    PagesArgs a = pages_args(cu_seqlens, n_past, batch, total_tokens, page_table, p);
    a.k_in = static_cast<const uint16_t *>(k);
    a.v_in = static_cast<const uint16_t *>(v);
    a.ldk = ldk ? ldk : (long long)p.n_kv_heads * kKvqDim;
    a.ldv = ldv ? ldv : (long long)p.n_kv_heads * kKvqDim;
    a.k_pages = static_cast<uint8_t *>(k_pages);
    a.v_pages = static_cast<uint8_t *>(v_pages);
    return launch_pages(a, true, stream);
}

cudaError_t launch_kvq_read(const void *k_pages, const void *v_pages, const int32_t *page_table,
                            const int32_t *cu_seqlens, const int32_t *n_past, int batch, int total_tokens, void *k_out,
                            void *v_out, const qa_attn_params &p, cudaStream_t stream) {
    PagesArgs a = pages_args(cu_seqlens, n_past, batch, total_tokens, page_table, p);
    a.k_out = static_cast<uint16_t *>(k_out);
    a.v_out = static_cast<uint16_t *>(v_out);
    a.k_pages = const_cast<uint8_t *>(static_cast<const uint8_t *>(k_pages));
    a.v_pages = const_cast<uint8_t *>(static_cast<const uint8_t *>(v_pages));
    return launch_pages(a, false, stream);
}

unsigned int status_read_clear_kvq_pages(cudaStream_t stream, cudaError_t *err) {
    unsigned int v = 0, zero = 0;
    cudaError_t e = cudaMemcpyFromSymbolAsync(&v, g_status, sizeof v, 0, cudaMemcpyDeviceToHost, stream);
    if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
    if (e == cudaSuccess && v) e = cudaMemcpyToSymbolAsync(g_status, &zero, sizeof zero, 0, cudaMemcpyHostToDevice, stream);
    if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
    if (err) *err = e;
    return v;
}

}  // namespace qa
