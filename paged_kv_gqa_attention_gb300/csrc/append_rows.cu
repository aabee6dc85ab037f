// Rows normed, rotated and written to the pages of the bf16 cache
// (qa_append_rows): drafted trees, prompt chunks, or an encoder's states as
// they are.
//
//   y = x / sqrt(mean x^2 + eps) * gain;  a_i = position theta^(-2i/128)
//   z_i = y_i cos a_i - y_{i+64} sin a_i,  z_{i+64} = y_i sin a_i + y_{i+64} cos a_i
//
// for q and k; v, and without a rotation all three, bit for bit.  A warp takes
// a row, or a share of its heads where rows are few, four heads a pass: 8
// lanes a head, a lane dims [8 l, 8 l + 8) and their partners 64 further.  The
// passes of its rows come through a ring of its own in shared memory (16-byte
// asynchronous copies, each lane its own bytes).  Where a row goes and what it
// is turned by is found once a row and a row ahead, because it is a chain of
// dependent loads: the request by a search over the boundaries, its cached
// length, the page, and the row's depth in the tree.
//
// Bound by HBM where rows are many: 17600 rows of 16 + 8 + 8 heads in a fused
// projection, three axes: 50 us, 5.9 TB/s, 88 % of a copy; 65000 rows of 8 + 8
// heads, bit for bit: 80 us, 6.6 TB/s, 98 %.  Where they are few, by that chain.
#include <cuda_runtime.h>
#include <stdint.h>
#include <string.h>

#include "async.cuh"
#include "common.cuh"
#include "qa_internal.h"
#include "rotary.cuh"

namespace qa {
namespace {

__device__ unsigned int g_status;

constexpr int kD = 128, kHalf = 64;
constexpr int kThreads = 128, kWarps = kThreads / 32;
constexpr int kStages = 4;
constexpr int kPassBytes = 1024;
constexpr int kMaxPos = 1 << 18;  // sincos_turns's range
constexpr int kCtasPerSm = 5;
// A row is shared by so many warps that there are about this many of them.
// Rows of 16 + 8 + 8 heads in a fused projection, trees, by 1 / 2 / 4 / 8
// warps a row: 8 rows 5.5 / 3.9 / 3.2 / 2.8 us, 256 rows 5.6 / 4.0 / 3.5 / 3.6,
// 1024 rows 6.5 / 6.0 / 6.8 / 7.9, 2112 rows 8.4 / 10.0 / 11.0 / 14, 17600 rows
// (three axes) 47.5 / 53 / 58 / 76.
constexpr int kShareRows = 2048;
// CTAs a grid has for each SM at most: 5 / 10 / 20 for 17600 rows 50.3 / 49.7 /
// 47.5 us, for 64000 rows of 8 + 8 heads as they are 87.7 / 82.3 / 79.5.
constexpr int kMostPerSm = 20;

struct AppendArgs {
    const uint16_t *q, *k, *v;
    uint16_t *q_out, *k_pages, *v_pages;
    long long ldq, ldk, ldv, ldq_out;
    const int32_t *cu, *past, *parents, *page_table, *positions;
    const float *q_gain, *k_gain;
    int rows, batch, hq, hkv, heads, turned;  // heads: hq + 2 hkv; turned: those before it are rotated
    int max_pages, num_pages, n_axes, early;
    float eps;
    uint8_t pair_axis[kHalf];
    float freq_hi[kHalf], freq_lo[kHalf];
};

// Where a row goes, and what it is turned by.
struct Place {
    int pos;       // lane x: the position on axis x
    long long at;  // the row's number in the pools, -1: no place in them
    bool live;     // the row belongs to a request
};

// A warp's search for row t's request, the last one that begins at or before
// it (32 boundaries a round, `probe` the first round's), then its place and,
// without explicit positions, its depth in the tree.  The parents of the 64
// rows up to t come with two loads a lane; a walk that leaves these goes on in
// memory, a load a step.
__device__ __forceinline__ Place place_of(const AppendArgs &a, long long t, int probe) {
    constexpr unsigned kAll = 0xffffffffu;
    const int lane = threadIdx.x & 31;
    Place p = {0, -1, false};
    if (t >= a.rows) return p;
    const int row = (int)t;
    if (a.positions && lane < a.n_axes) p.pos = a.positions[(size_t)lane * a.rows + row];
    int r = 0;
    for (int n = a.batch, at = probe;;) {
        const int step = (n + 31) / 32;
        const unsigned before = __ballot_sync(kAll, lane * step < n && at <= row);
        if (before == 0) return p;
        const int k = 31 - __clz(before);
        r += k * step;
        n = min(step, n - k * step);
        if (step == 1) break;
        const int next = (n + 31) / 32;
        at = lane * next < n ? a.cu[r + lane * next] : 0;
    }
    const int first = a.cu[r], end = a.cu[r + 1];
    const long long past = a.past ? a.past[r] : 0, cap = (long long)a.max_pages * 16;
    if (first < 0 || end > a.rows || row >= end) return p;
    const int i = row - first, base = max(0, i - 63);
    const bool climb = !a.positions && a.turned && a.parents;
    const int low = climb && base + lane <= i ? a.parents[first + base + lane] : -1;
    const int high = climb && base + 32 + lane <= i ? a.parents[first + base + 32 + lane] : -1;
    if (past < 0 || past > cap) {
        if (lane == 0) atomicOr(&g_status, QA_DEVICE_BAD_LENGTH);
        return p;
    }
    p.live = true;
    const long long at = past + i;
    if (at < cap) {
        const int page = a.page_table[(size_t)r * a.max_pages + (int)(at >> 4)];
        if (page >= 0 && page < a.num_pages) p.at = (long long)page * 16 + (at & 15);
        else if (lane == 0) atomicOr(&g_status, QA_DEVICE_BAD_PAGE);
    } else if (lane == 0) {
        atomicOr(&g_status, QA_DEVICE_BAD_LENGTH);
    }
    if (!a.positions && a.turned) {
        int depth = i;
        if (a.parents) {
            const auto checked = [&](int up, int node) {
                if (up >= -1 && up < node) return up;
                atomicOr(&g_status, QA_DEVICE_BAD_TREE);
                return -1;
            };
            const int up_low = checked(low, max(base + lane, 0)), up_high = checked(high, base + 32 + lane);
            // numbered from `base`, 64 where the walk leaves the rows at hand: a shuffle a step
            const uint32_t both = (uint32_t)(up_low >= base ? up_low - base : 64) | (uint32_t)(up_high >= base ? up_high - base : 64) << 8;
            int at = i - base;
            for (depth = 0;; ++depth) {
                const uint32_t w = __shfl_sync(kAll, both, at & 31), up = at < 32 ? w & 0xffu : w >> 8;
                if (up == 64) break;
                at = (int)up;
            }
            const int x = __shfl_sync(kAll, up_low, at & 31), y = __shfl_sync(kAll, up_high, at & 31);
            for (int node = at < 32 ? x : y; node >= 0; ++depth) node = checked(a.parents[first + node], node);
        }
        const long long pos = past + depth;
        p.pos = lane == 0 ? (pos < kMaxPos ? (int)pos : kMaxPos) : 0;
    }
    return p;
}

template <bool NORM>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) append_rows_kernel(const __grid_constant__ AppendArgs a) {
    constexpr unsigned kAll = 0xffffffffu;
    __shared__ __align__(16) uint8_t smem[kWarps * kStages * kPassBytes];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, l = lane & 7, sub = lane >> 3;
    const uint32_t ring = smem_u32(smem) + warp * (kStages * kPassBytes) + 16 * lane;
    const int passes = (a.heads + 3) >> 2;
    const int p0 = passes * (int)blockIdx.y / (int)gridDim.y, p1 = passes * ((int)blockIdx.y + 1) / (int)gridDim.y;
    const int stride = gridDim.x * kWarps;
    int t = blockIdx.x * kWarps + warp;

    // of the lane's 8 pairs 8 l + j, j = 2 sub + y
    float f_hi[2], f_lo[2];
    int axis[2];
    const float *hi = a.freq_hi, *lo = a.freq_lo;
    const uint8_t *pair_axis = a.pair_axis;
    asm("" : "+l"(hi), "+l"(lo), "+l"(pair_axis));  // generic addresses: the lanes' loads go together
#pragma unroll
    for (int y = 0; y < 2; ++y) {
        const int i = 8 * l + 2 * sub + y;
        f_hi[y] = hi[i], f_lo[y] = lo[i], axis[y] = pair_axis[i];
    }
    const auto fetch = [&](long long row, int pass, int stage) {  // a pass's copies, or nothing past the last: a group either way
        const int h = 4 * pass + sub;
        if (row < a.rows && h < a.heads) {
            const uint16_t *src = h < a.hq ? a.q + row * a.ldq + h * kD
                                  : h < a.hq + a.hkv ? a.k + row * a.ldk + (h - a.hq) * kD
                                                     : a.v + row * a.ldv + (h - a.hq - a.hkv) * kD;
            copy16(ring + stage * kPassBytes, src + 8 * l);
            copy16(ring + stage * kPassBytes + 512, src + 8 * l + kHalf);
        }
        copy_commit();
    };
    const auto wait = [] {
        asm volatile("griddepcontrol.wait;" ::: "memory");
        asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    };
    if (!a.early) wait();
    const int step = (a.batch + 31) / 32;
    const int probe = lane * step < a.batch ? a.cu[lane * step] : 0;
    Place next;
    if (a.early) next = place_of(a, t, probe), wait();
    long long tf = t;  // the row and pass whose copies go out next
    int pf = p0;
    const auto ahead = [&](int stage) {
        fetch(tf, pf, stage);
        if (++pf == p1) pf = p0, tf += stride;
    };
#pragma unroll
    for (int n = 0; n < kStages; ++n) ahead(n);
    if (!a.early) next = place_of(a, t, probe);
    if (blockIdx.x == 0 && blockIdx.y == 0 && warp == 0) {
        bool wrong = false;
        for (int r = lane; r < a.batch; r += 32) wrong |= a.cu[r] < 0 || a.cu[r] > a.cu[r + 1] || a.cu[r + 1] > a.rows;
        if (__any_sync(kAll, wrong) && lane == 0) atomicOr(&g_status, QA_DEVICE_BAD_SEGMENTS);
    }
    int stage = 0;
    for (; t < a.rows; t += stride) {
        const Place here = next;
        next = place_of(a, (long long)t + stride, probe);
        bool bad = __any_sync(kAll, here.pos < 0 || here.pos >= kMaxPos);
        if (bad && here.live && lane == 0) atomicOr(&g_status, QA_DEVICE_BAD_POSITION);
        bad |= !here.live;
        float2 c[4], s[4];
        if (4 * p0 < a.turned) {
            float c_own[2], s_own[2];
#pragma unroll
            for (int y = 0; y < 2; ++y) sincos_turns(__shfl_sync(kAll, here.pos, axis[y]), f_hi[y], f_lo[y], &s_own[y], &c_own[y]);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float cj = __shfl_sync(kAll, c_own[j & 1], j / 2 * 8 + l), sj = __shfl_sync(kAll, s_own[j & 1], j / 2 * 8 + l);
                if (j & 1) c[j / 2].y = cj, s[j / 2].y = sj; else c[j / 2].x = cj, s[j / 2].x = sj;
            }
        }
        for (int pass = p0; pass < p1; ++pass) {
            const int h = 4 * pass + sub;
            copy_wait<kStages - 1>();
            const uint4 w0 = lds128(ring + stage * kPassBytes), w1 = lds128(ring + stage * kPassBytes + 512);
            ahead(stage);
            stage = (stage + 1) % kStages;
            uint32_t z[4] = {w0.x, w0.y, w0.z, w0.w}, u[4] = {w1.x, w1.y, w1.z, w1.w};
            if (4 * pass < a.turned) {  // some of the pass's heads are rotated
                const float *gain = (h < a.hq ? a.q_gain : a.k_gain) + 8 * l;
                float2 x[4], y[4], s2 = make_float2(0.f, 0.f);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    x[i] = make_float2(bf16lo(z[i]), bf16hi(z[i]));
                    y[i] = make_float2(bf16lo(u[i]), bf16hi(u[i]));
                    if (NORM) s2 = ffma2(x[i], x[i], ffma2(y[i], y[i], s2));
                }
                float r = 1.f;
                if (NORM) {
                    float ss = s2.x + s2.y;
#pragma unroll
                    for (int o = 4; o > 0; o >>= 1) ss += __shfl_xor_sync(kAll, ss, o);
                    r = rsqrtf(fmaf(ss, 1.0f / kD, a.eps));
                }
                const float2 rr = make_float2(r, r);
                if (h < a.turned) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if (NORM) {
                            x[i] = fmul2(x[i], fmul2(rr, __ldg(reinterpret_cast<const float2 *>(gain) + i)));
                            y[i] = fmul2(y[i], fmul2(rr, __ldg(reinterpret_cast<const float2 *>(gain + kHalf) + i)));
                        }
                        const float2 first = fsub2(fmul2(x[i], c[i]), fmul2(y[i], s[i])), second = ffma2(x[i], s[i], fmul2(y[i], c[i]));
                        z[i] = pack_bf16x2(first.x, first.y);
                        u[i] = pack_bf16x2(second.x, second.y);
                    }
                }
            }
            if (h < a.heads && !bad && (h < a.hq || here.at >= 0)) {
                uint16_t *dst = h < a.hq ? a.q_out + (long long)t * a.ldq_out + h * kD
                                : h < a.hq + a.hkv ? a.k_pages + (here.at * a.hkv + (h - a.hq)) * kD
                                                   : a.v_pages + (here.at * a.hkv + (h - a.hq - a.hkv)) * kD;
                *reinterpret_cast<uint4 *>(dst + 8 * l) = make_uint4(z[0], z[1], z[2], z[3]);
                *reinterpret_cast<uint4 *>(dst + 8 * l + kHalf) = make_uint4(u[0], u[1], u[2], u[3]);
            }
        }
    }
}

}  // namespace

cudaError_t launch_append_rows(const AppendRows &x, const qa_attn_params &p, cudaStream_t stream) {
    AppendArgs a = {};
    const long long wq = (long long)p.n_q_heads * kD, wk = (long long)p.n_kv_heads * kD;
    a.q = static_cast<const uint16_t *>(x.q);
    a.k = static_cast<const uint16_t *>(x.k);
    a.v = static_cast<const uint16_t *>(x.v);
    a.q_out = static_cast<uint16_t *>(x.q_out);
    a.k_pages = static_cast<uint16_t *>(x.k_pages);
    a.v_pages = static_cast<uint16_t *>(x.v_pages);
    a.ldq = x.ldq ? x.ldq : wq;
    a.ldk = x.ldk ? x.ldk : wk;
    a.ldv = x.ldv ? x.ldv : wk;
    a.ldq_out = x.ldq_out ? x.ldq_out : wq;
    a.cu = x.cu_seqlens;
    a.past = x.n_past;
    a.parents = x.parents;
    a.page_table = x.page_table;
    a.rows = x.rows;
    a.batch = x.batch;
    a.hq = x.q ? p.n_q_heads : 0;
    a.hkv = p.n_kv_heads;
    a.heads = a.hq + 2 * a.hkv;
    a.turned = x.rope ? a.hq + a.hkv : 0;
    a.max_pages = p.max_pages_per_seq;
    a.num_pages = p.num_pages;
    a.early = (p.abi_version >= 2 && p.stable_metadata >= 1) ? 1 : 0;
    a.n_axes = 1;
    if (x.rope) {
        a.q_gain = x.rope->q_gain;
        a.k_gain = x.rope->k_gain;
        a.positions = x.rope->positions;
        a.n_axes = x.rope->n_axes;
        a.eps = x.rope->rms_eps;
        if (x.rope->pair_axis) memcpy(a.pair_axis, x.rope->pair_axis, kHalf);
        rope_frequencies(x.rope->theta, kD, a.freq_hi, a.freq_lo);
    }
    int device = 0, sms = 0;
    if (cudaGetDevice(&device) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device) != cudaSuccess || sms <= 0)
        return cudaErrorInvalidDevice;
    const int passes = (a.heads + 3) / 4;
    int shares = kShareRows / x.rows;
    shares = shares < 1 ? 1 : shares > passes ? passes : shares;
    const int ctas = (x.rows + kWarps - 1) / kWarps, most = (sms * kMostPerSm + shares - 1) / shares;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(ctas < most ? ctas : most), (unsigned)shares);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, a.q_gain ? append_rows_kernel<true> : append_rows_kernel<false>, a);
}

unsigned int status_read_clear_append_rows(cudaStream_t stream, cudaError_t *err) {
    unsigned int v = 0, zero = 0;
    cudaError_t e = cudaMemcpyFromSymbolAsync(&v, g_status, sizeof v, 0, cudaMemcpyDeviceToHost, stream);
    if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
    if (e == cudaSuccess && v) e = cudaMemcpyToSymbolAsync(g_status, &zero, sizeof zero, 0, cudaMemcpyHostToDevice, stream);
    if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
    if (err) *err = e;
    return v;
}

}  // namespace qa
