// Per-head QK-norm and rotary positions with up to four axes over packed
// query and key rows (qa_rope_rows).
//
//   y = x / sqrt(mean x^2 + eps) * gain;  a_i = positions[axis(i)][t] theta^(-2i/D)
//   z_i = y_i cos a_i - y_{i+D/2} sin a_i,  z_{i+D/2} = y_i sin a_i + y_{i+D/2} cos a_i
//
// Every warp works by itself.  An item is one row and PASSES x 512 / D of its
// heads: D/16 lanes share a head, a lane holds dims [8l, 8l + 8) and their
// partners D/2 further.  A warp has kStages items in flight in its part of
// shared memory (16-byte asynchronous copies, each lane its own bytes, so
// nothing waits on other lanes), and computes each of a row's D/2 angles once
// and exchanges them by shuffles.  Frequencies are read once a warp, and as
// memory: the constant bank serves one address at a time, and read so for
// every row it was what bounded.
//
// Bound by HBM: 16111 rows of 16 + 8 heads of 128 in fused rows (198 MB) take
// 32.2 us, 6.15 TB/s, 91 % of the copy rate; 4095 rows of 28 heads of 64 (out
// of L2 in part) 4.3 us; 32 rows 1.6 us, a launch.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include <type_traits>

#include "async.cuh"
#include "common.cuh"
#include "qa_internal.h"
#include "rotary.cuh"

namespace qa {
namespace {

__device__ unsigned int g_status;

constexpr int kMaxHalf = 64;
// Head vectors up to which an item is one pass, which gives few rows more
// warps; beyond, two passes share their row's angles.  Rows of 24 heads of
// 128, one pass against two: 32 rows 1.56 and 1.71 us, 100 rows 1.71 and 1.72,
// 300 rows 2.05 and 1.89, 1000 rows 3.85 and 2.76, 16111 rows 37.3 and 32.3
// (three 33.5, six 35.2).
constexpr int kFewHeads = 4096;
constexpr int kThreads = 128;
constexpr int kStages = 2;
// CTAs a grid has for each SM at most.  Five are resident at two passes with a
// norm (96 registers), so such a grid comes in two waves; rows of 24 heads of
// 128, 5 / 8 / 10 / 15 / 20: 3000 rows 5.8 / 6.5 / 6.3 / 6.2 / 6.2 us, 8000 rows
// 16.9 / 16.3 / 15.2 / 15.7 / 16.4, 16111 rows 36.0 / 32.5 / 32.3 / 31.7 / 31.5.
constexpr int kCtasPerSm = 10;
constexpr int kMaxPos = 1 << 18;  // sincos_turns's range

struct RopeArgs {
    const uint16_t *q, *k;
    uint16_t *q_out, *k_out;
    long long ldq, ldk, ldq_out, ldk_out;
    const float *q_gain, *k_gain;
    const int32_t *positions;
    int rows, hq, heads, n_axes;  // heads: hq + hkv (hq alone without k)
    int early;
    float eps;
    uint8_t pair_axis[kMaxHalf];
    float freq_hi[kMaxHalf], freq_lo[kMaxHalf];
};

template <int D, int PASSES, bool NORM>
__global__ void __launch_bounds__(kThreads) rope_rows_kernel(const __grid_constant__ RopeArgs a) {
    constexpr int HALF = D / 2;
    constexpr int LANES = D / 16;        // lanes of a head
    constexpr int HEADS = 32 / LANES;    // of a pass
    constexpr int OWN = HALF / 32;       // angles of a lane
    constexpr int STAGE = PASSES * 1024;
    extern __shared__ __align__(16) uint8_t smem[];
    const int lane = threadIdx.x & 31, l = lane % LANES, sub = lane / LANES;
    const uint32_t ring = smem_u32(smem) + (threadIdx.x >> 5) * (kStages * STAGE) + 16 * lane;
    const int h0 = blockIdx.y * (HEADS * PASSES) + sub;  // the lane's head of the first pass
    const int stride = gridDim.x * (kThreads / 32);
    int t = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);

    float f_hi[OWN], f_lo[OWN];
    int axis[OWN];
    const float *hi = a.freq_hi, *lo = a.freq_lo;
    const uint8_t *pair_axis = a.pair_axis;
    asm("" : "+l"(hi), "+l"(lo), "+l"(pair_axis));  // generic addresses: the lanes' loads go together
#pragma unroll
    for (int y = 0; y < OWN; ++y) {  // of the lane's 8 pairs 8 l + j, j = OWN sub + y
        const int i = 8 * l + OWN * sub + y;
        f_hi[y] = hi[i], f_lo[y] = lo[i], axis[y] = pair_axis[i];
    }
    // where the lane's head of pass p lies in a row: its first pass's place as a query or as a key, p HEADS D further
    const int at_q = h0 * D + 8 * l, at_k = (h0 - a.hq) * D + 8 * l;
    auto fetch = [&](long long row, int stage) {  // a row's copies, or nothing past the last: a group either way
        if (row < a.rows) {
            const uint16_t *q = a.q + row * a.ldq + at_q, *k = a.k + row * a.ldk + at_k;
#pragma unroll
            for (int p = 0; p < PASSES; ++p) {
                const int h = h0 + p * HEADS;
                if (h < a.heads) {
                    const uint16_t *src = (h < a.hq ? q : k) + p * (HEADS * D);
                    copy16(ring + stage * STAGE + p * 1024, src);
                    copy16(ring + stage * STAGE + p * 1024 + 512, src + HALF);
                }
            }
        }
        copy_commit();
    };
    auto position = [&](long long row) -> int {  // lane x: the row's position on axis x
        return row < a.rows && lane < a.n_axes ? a.positions[(size_t)lane * a.rows + row] : 0;
    };
    const auto wait = [] {
        asm volatile("griddepcontrol.wait;" ::: "memory");
        asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    };
    if (!a.early) wait();
    int pos_next = position(t);
    if (a.early) wait();
#pragma unroll
    for (int n = 0; n < kStages; ++n) fetch(t + (long long)n * stride, n);
    int stage = 0;
    for (; t < a.rows; t += stride) {
        const int pos = pos_next;
        pos_next = position((long long)t + stride);
        const bool bad = __any_sync(0xffffffffu, pos < 0 || pos >= kMaxPos);
        if (bad && lane == 0) atomicOr(&g_status, QA_DEVICE_BAD_POSITION);
        float c_own[OWN], s_own[OWN];
        float2 c[4], s[4];
#pragma unroll
        for (int y = 0; y < OWN; ++y)
            sincos_turns(__shfl_sync(0xffffffffu, pos, axis[y]), f_hi[y], f_lo[y], &s_own[y], &c_own[y]);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float cj = __shfl_sync(0xffffffffu, c_own[j % OWN], j / OWN * LANES + l);
            const float sj = __shfl_sync(0xffffffffu, s_own[j % OWN], j / OWN * LANES + l);
            if (j & 1) c[j / 2].y = cj, s[j / 2].y = sj; else c[j / 2].x = cj, s[j / 2].x = sj;
        }
        // z = xc x - ys y, u = xs x + yc y, times 1 / rms: the gains of query heads, then of key heads, are in the factors
        float2 xc[4], xs[4], yc[4], ys[4];
        auto factors = [&](bool is_q) {
            const float *gain = (is_q ? a.q_gain : a.k_gain) + 8 * l;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float2 g0 = make_float2(1.f, 1.f), g1 = g0;
                if (NORM) g0 = __ldg(reinterpret_cast<const float2 *>(gain) + i), g1 = __ldg(reinterpret_cast<const float2 *>(gain + HALF) + i);
                xc[i] = fmul2(c[i], g0), xs[i] = fmul2(s[i], g0), yc[i] = fmul2(c[i], g1);
                ys[i] = fmul2(s[i], make_float2(-g1.x, -g1.y));
            }
        };
        factors(h0 < a.hq);
        uint16_t *q_out = a.q_out + (long long)t * a.ldq_out + at_q, *k_out = a.k_out + (long long)t * a.ldk_out + at_k;
        copy_wait<kStages - 1>();
#pragma unroll
        for (int p = 0; p < PASSES; ++p) {
            const int h = h0 + p * HEADS;
            if (NORM && p > 0) {
                const bool turned = h >= a.hq && h - HEADS < a.hq;  // the lane's first key head
                if (__any_sync(0xffffffffu, turned)) {
                    if (turned) factors(false);
                }
            }
            const uint4 w0 = lds128(ring + stage * STAGE + p * 1024), w1 = lds128(ring + stage * STAGE + p * 1024 + 512);
            const uint32_t wx[4] = {w0.x, w0.y, w0.z, w0.w}, wy[4] = {w1.x, w1.y, w1.z, w1.w};
            float2 x[4], y[4];
            float2 s2 = make_float2(0.f, 0.f);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[i] = make_float2(bf16lo(wx[i]), bf16hi(wx[i]));
                y[i] = make_float2(bf16lo(wy[i]), bf16hi(wy[i]));
                if (NORM) s2 = ffma2(x[i], x[i], ffma2(y[i], y[i], s2));
            }
            float r = 1.f;
            if (NORM) {
                float ss = s2.x + s2.y;
#pragma unroll
                for (int o = LANES / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
                r = rsqrtf(fmaf(ss, 1.0f / D, a.eps));
            }
            const float2 rr = make_float2(r, r);
            uint32_t z[4], u[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float2 lo = ffma2(x[i], xc[i], fmul2(y[i], ys[i])), hi = ffma2(x[i], xs[i], fmul2(y[i], yc[i]));
                if (NORM) lo = fmul2(lo, rr), hi = fmul2(hi, rr);
                z[i] = pack_bf16x2(lo.x, lo.y);
                u[i] = pack_bf16x2(hi.x, hi.y);
            }
            if (h < a.heads && !bad) {
                uint16_t *dst = (h < a.hq ? q_out : k_out) + p * (HEADS * D);
                *reinterpret_cast<uint4 *>(dst) = make_uint4(z[0], z[1], z[2], z[3]);
                *reinterpret_cast<uint4 *>(dst + HALF) = make_uint4(u[0], u[1], u[2], u[3]);
            }
        }
        fetch((long long)t + (long long)kStages * stride, stage);
        stage = stage + 1 == kStages ? 0 : stage + 1;
    }
}

}  // namespace

void rope_frequencies(float theta, int head_dim, float *hi, float *lo) {
    // one entry of the last theta and head_dim: a decode step of many layers
    // computes its 64 powers once a thread
    thread_local float t_theta = 0.f, t_hi[kMaxHalf], t_lo[kMaxHalf];
    thread_local int t_dim = 0;
    const int half = head_dim / 2;
    if (theta != t_theta || head_dim != t_dim) {
        for (int i = 0; i < half; ++i) {
            const double f = pow((double)theta, -2.0 * i / head_dim) / 6.283185307179586476925286766559;
            t_hi[i] = (float)f;
            t_lo[i] = (float)(f - (double)t_hi[i]);
        }
        t_theta = theta;
        t_dim = head_dim;
    }
    memcpy(hi, t_hi, half * sizeof(float));
    memcpy(lo, t_lo, half * sizeof(float));
}

cudaError_t launch_rope_rows(const void *q, long long ldq, const void *k, long long ldk, int rows, void *q_out,
                             long long ldq_out, void *k_out, long long ldk_out, const qa_rope &rope,
                             const qa_attn_params &p, cudaStream_t stream) {
    RopeArgs a = {};
    const long long wq = (long long)p.n_q_heads * p.head_dim, wk = (long long)p.n_kv_heads * p.head_dim;
    a.q = static_cast<const uint16_t *>(q);
    a.k = static_cast<const uint16_t *>(k);
    a.q_out = static_cast<uint16_t *>(q_out);
    a.k_out = static_cast<uint16_t *>(k_out);
    a.ldq = ldq ? ldq : wq;
    a.ldk = ldk ? ldk : wk;
    a.ldq_out = ldq_out ? ldq_out : wq;
    a.ldk_out = ldk_out ? ldk_out : wk;
    a.q_gain = rope.q_gain;
    a.k_gain = rope.k_gain;
    a.positions = rope.positions;
    a.rows = rows;
    a.hq = p.n_q_heads;
    a.heads = p.n_q_heads + (k ? p.n_kv_heads : 0);
    a.n_axes = rope.n_axes;
    a.early = (p.abi_version >= 2 && p.stable_metadata >= 1) ? 1 : 0;
    a.eps = rope.rms_eps;
    if (rope.pair_axis) memcpy(a.pair_axis, rope.pair_axis, p.head_dim / 2);
    rope_frequencies(rope.theta, p.head_dim, a.freq_hi, a.freq_lo);

    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const bool wide = p.head_dim == 128, norm = rope.q_gain != nullptr;
    int device = 0, sms = 0;
    if (cudaGetDevice(&device) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device) != cudaSuccess || sms <= 0)
        return cudaErrorInvalidDevice;
    const auto pick = [&](auto n) {
        constexpr int N = decltype(n)::value;
        const int heads_an_item = 512 / p.head_dim * N, chunks = (a.heads + heads_an_item - 1) / heads_an_item;
        const int ctas = (rows + kThreads / 32 - 1) / (kThreads / 32), most = (sms * kCtasPerSm + chunks - 1) / chunks;
        cfg.gridDim = dim3((unsigned)(ctas < most ? ctas : most), (unsigned)chunks);
        cfg.dynamicSmemBytes = (kThreads / 32) * kStages * N * 1024;
        return norm ? cudaLaunchKernelEx(&cfg, wide ? rope_rows_kernel<128, N, true> : rope_rows_kernel<64, N, true>, a)
                    : cudaLaunchKernelEx(&cfg, wide ? rope_rows_kernel<128, N, false> : rope_rows_kernel<64, N, false>, a);
    };
    if ((long long)rows * a.heads <= kFewHeads) return pick(std::integral_constant<int, 1>());
    return pick(std::integral_constant<int, 2>());
}

unsigned int status_read_clear_rope(cudaStream_t stream, cudaError_t *err) {
    unsigned int v = 0, zero = 0;
    cudaError_t e = cudaMemcpyFromSymbolAsync(&v, g_status, sizeof v, 0, cudaMemcpyDeviceToHost, stream);
    if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
    if (e == cudaSuccess && v) e = cudaMemcpyToSymbolAsync(g_status, &zero, sizeof zero, 0, cudaMemcpyHostToDevice, stream);
    if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
    if (err) *err = e;
    return v;
}

}  // namespace qa
