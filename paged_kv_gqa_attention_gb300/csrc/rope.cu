// Per-head QK-norm and rotary positions with up to four axes over packed
// query and key rows (qa_rope_rows).
//
//   y = x / sqrt(mean x^2 + eps) * gain;  a_i = positions[axis(i)][t] theta^(-2i/D)
//   z_i = y_i cos a_i - y_{i+D/2} sin a_i,  z_{i+D/2} = y_i sin a_i + y_{i+D/2} cos a_i
//
// A CTA takes kRows rows.  Its threads first compute the rows' D/2 angles
// once into shared memory (every head of a row turns by the same angles),
// then D/8 lanes share a head: a lane holds dims [4l, 4l + 4) and their
// partners D/2 further, two 8-byte loads and stores.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include "common.cuh"
#include "qa_internal.h"

namespace qa {
namespace {

__device__ unsigned int g_status;

constexpr int kMaxHalf = 64;
constexpr int kMaxPos = 1 << 18;  // sincos_pos_freq's range

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

template <int D, int ROWS, int THREADS>
__global__ void __launch_bounds__(THREADS) rope_rows_kernel(const __grid_constant__ RopeArgs a) {
    constexpr int HALF = D / 2;
    constexpr int LANES = D / 8;  // lanes of a head
    __shared__ float2 turn[ROWS][HALF];  // cos, sin
    __shared__ int row_ok[ROWS];
    if (!a.early) asm volatile("griddepcontrol.wait;" ::: "memory");
    const int r0 = blockIdx.x * ROWS;
    const int n_rows = min(ROWS, a.rows - r0);
    if (threadIdx.x < (unsigned)n_rows) {
        int ok = 1;
        for (int x = 0; x < a.n_axes; ++x) {
            const int pos = a.positions[(size_t)x * a.rows + r0 + threadIdx.x];
            ok &= pos >= 0 && pos < kMaxPos;
        }
        if (!ok) atomicOr(&g_status, QA_DEVICE_BAD_POSITION);
        row_ok[threadIdx.x] = ok;
    }
    for (int u = threadIdx.x; u < n_rows * HALF; u += THREADS) {
        const int row = u / HALF, i = u % HALF;
        const int pos = a.positions[(size_t)a.pair_axis[i] * a.rows + r0 + row];
        float s, c;
        sincos_pos_freq(pos, a.freq_hi[i], a.freq_lo[i], &s, &c);
        turn[row][i] = make_float2(c, s);
    }
    __syncthreads();
    if (a.early) asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    const int l = threadIdx.x % LANES;
    for (int h = threadIdx.x / LANES; h < a.heads; h += THREADS / LANES) {
        const bool is_q = h < a.hq;
        const float *gain = is_q ? a.q_gain : a.k_gain;
        float4 g0 = make_float4(1.f, 1.f, 1.f, 1.f), g1 = g0;
        if (gain) {
            g0 = *reinterpret_cast<const float4 *>(gain + 4 * l);
            g1 = *reinterpret_cast<const float4 *>(gain + HALF + 4 * l);
        }
        for (int row = 0; row < n_rows; ++row) {
            const long long t = r0 + row;
            const int hh = is_q ? h : h - a.hq;
            const uint16_t *src = (is_q ? a.q + t * a.ldq : a.k + t * a.ldk) + hh * D + 4 * l;
            uint16_t *dst = (is_q ? a.q_out + t * a.ldq_out : a.k_out + t * a.ldk_out) + hh * D + 4 * l;
            const uint2 w0 = *reinterpret_cast<const uint2 *>(src), w1 = *reinterpret_cast<const uint2 *>(src + HALF);
            float x[4] = {bf16lo(w0.x), bf16hi(w0.x), bf16lo(w0.y), bf16hi(w0.y)};
            float y[4] = {bf16lo(w1.x), bf16hi(w1.x), bf16lo(w1.y), bf16hi(w1.y)};
            if (gain) {
                float ss = 0.f;
#pragma unroll
                for (int c = 0; c < 4; ++c) ss += x[c] * x[c] + y[c] * y[c];
                const unsigned mask = LANES == 32 ? 0xffffffffu : ((1u << LANES) - 1u) << (threadIdx.x % 32 / LANES * LANES);
#pragma unroll
                for (int o = LANES / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(mask, ss, o);
                const float r = 1.0f / sqrtf(ss * (1.0f / D) + a.eps);
                x[0] *= r * g0.x, x[1] *= r * g0.y, x[2] *= r * g0.z, x[3] *= r * g0.w;
                y[0] *= r * g1.x, y[1] *= r * g1.y, y[2] *= r * g1.z, y[3] *= r * g1.w;
            }
            if (!row_ok[row]) continue;
            float z[4], u[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const float2 cs = turn[row][4 * l + c];
                z[c] = x[c] * cs.x - y[c] * cs.y;
                u[c] = x[c] * cs.y + y[c] * cs.x;
            }
            *reinterpret_cast<uint2 *>(dst) = make_uint2(pack_bf16x2(z[0], z[1]), pack_bf16x2(z[2], z[3]));
            *reinterpret_cast<uint2 *>(dst + HALF) = make_uint2(pack_bf16x2(u[0], u[1]), pack_bf16x2(u[2], u[3]));
        }
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
            const double f = pow((double)theta, -2.0 * i / head_dim);
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

    constexpr int kThreads = 384, kRowsPerCta = 4;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((rows + kRowsPerCta - 1) / kRowsPerCta));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    auto kernel = p.head_dim == 128 ? rope_rows_kernel<128, kRowsPerCta, kThreads> : rope_rows_kernel<64, kRowsPerCta, kThreads>;
    return cudaLaunchKernelEx(&cfg, kernel, a);
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
