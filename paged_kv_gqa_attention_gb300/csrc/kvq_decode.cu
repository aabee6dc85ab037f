// Paged GQA decode over a 4-bit KV pool (qa_kvq_decode_attn), and the decode
// step that norms, rotates, quantises and appends the new token first
// (qa_kvq_decode_step).
//
//   score_j = scale sum_g (m_jg sum_{d in g} q_d + s_jg sum_{d in g} q_d n_jd)
//   out = sum_j p_j (m_j + s_j n_j) / sum_j p_j,  p = exp(score - max)
//
// One warp takes one request's KV head and its query heads.  Lane l holds
// dims [4l, 4l + 4); running maximum, sum and outputs are fp32.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include "kvq.cuh"
#include "qa_internal.h"

namespace qa {
namespace {

__device__ unsigned int g_status;

constexpr int kD = kKvqDim;
constexpr int kPS = kKvqTokens;
constexpr int kMaxRopePos = 1 << 18;

struct KvqArgs {
    const uint16_t *q;
    uint8_t *k_pages, *v_pages;
    const int32_t *page_table, *seq_lens;
    uint16_t *out;
    long long ldq, ldkv;
    int batch, hkv, max_pages, num_pages;
    float scale_log2;
    // step only
    const uint16_t *k_new, *v_new;
    const float *q_gain, *k_gain;
    const int32_t *positions;  // [n_axes][batch], or nullptr: seq_lens - 1
    int n_axes;
    float eps;
    uint8_t pair_axis[kD / 2];
    float freq_hi[kD / 2], freq_lo[kD / 2];
};

// Norm and rotation of a head vector over a warp; lane l holds dims
// [4l, 4l + 4), whose rotation partners are on lane l ^ 16.  Rounded to bf16.
__device__ __forceinline__ uint2 norm_rope(uint2 w, const float *gain, float eps, const float *cs, const float *sn, int lane) {
    const float x[4] = {bf16lo(w.x), bf16hi(w.x), bf16lo(w.y), bf16hi(w.y)};
    const float ss = warp_sum(x[0] * x[0] + x[1] * x[1] + x[2] * x[2] + x[3] * x[3]);
    const float r = 1.0f / sqrtf(ss * (1.0f / kD) + eps);
    const float4 g = *reinterpret_cast<const float4 *>(gain + 4 * lane);
    const float y[4] = {x[0] * r * g.x, x[1] * r * g.y, x[2] * r * g.z, x[3] * r * g.w};
    float z[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        const float p = __shfl_xor_sync(0xffffffffu, y[c], 16);
        z[c] = lane < 16 ? y[c] * cs[c] - p * sn[c] : p * sn[c] + y[c] * cs[c];
    }
    return make_uint2(pack_bf16x2(z[0], z[1]), pack_bf16x2(z[2], z[3]));
}

// Quantises a row over a warp (lane l: dims [4l, 4l + 4)): the lane's four
// codes (16 bits) and its group's parameters.
__device__ __forceinline__ uint32_t quantise_row(uint2 w, int lane, uint32_t &sm) {
    const float x[4] = {bf16lo(w.x), bf16hi(w.x), bf16lo(w.y), bf16hi(w.y)};
    float lo = x[0], hi = x[0];
    bool bad = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        lo = fminf(lo, x[i]);
        hi = fmaxf(hi, x[i]);
        bad |= isnan(x[i]);
    }
    if (bad) hi = CUDART_INF_F;
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) {
        lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
        hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    }
    const KvqGroup g = kvq_group(lo, hi);
    sm = g.sm;
    uint32_t word = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) word |= kvq_code(x[i], g) << (4 * i);
    return word;
}

template <int GROUP, bool APPEND>
__global__ void __launch_bounds__(32) kvq_decode_kernel(const __grid_constant__ KvqArgs a) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int b = blockIdx.x / a.hkv, g = blockIdx.x % a.hkv, lane = threadIdx.x;
    int len = a.seq_lens[b];
    if (len < (APPEND ? 1 : 0) || len > a.max_pages * kPS) {
        if (lane == 0) atomicOr(&g_status, QA_DEVICE_BAD_LENGTH);
        len = 0;
    }
    float cs[4], sn[4];
    if (APPEND && len > 0) {
        bool ok = true;
        for (int x = 0; x < a.n_axes; ++x) {
            const int pos = a.positions ? a.positions[(size_t)x * a.batch + b] : len - 1;
            ok &= pos >= 0 && pos < kMaxRopePos;
        }
        if (!ok) {
            if (lane == 0) atomicOr(&g_status, QA_DEVICE_BAD_POSITION);
            len = 0;
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const int i = 4 * (lane & 15) + c;
            const int pos = a.positions ? a.positions[(size_t)a.pair_axis[i] * a.batch + b] : len - 1;
            sincos_pos_freq(pos, a.freq_hi[i], a.freq_lo[i], &sn[c], &cs[c]);
        }
    }
    const int32_t *row = a.page_table + (size_t)b * a.max_pages;
    if (APPEND && len > 0) {
        const int t = (len - 1) % kPS, page = row[(len - 1) / kPS];
        const size_t o = b * a.ldkv + g * kD + 4 * lane;
        const uint2 kw = norm_rope(*reinterpret_cast<const uint2 *>(a.k_new + o), a.k_gain, a.eps, cs, sn, lane);
        uint32_t ksm, vsm;
        const uint32_t kc = quantise_row(kw, lane, ksm);
        const uint32_t vc = quantise_row(*reinterpret_cast<const uint2 *>(a.v_new + o), lane, vsm);
        if (page >= 0 && page < a.num_pages) {
            uint8_t *kp = a.k_pages + ((size_t)page * a.hkv + g) * kKvqHeadBytes;
            uint8_t *vp = a.v_pages + ((size_t)page * a.hkv + g) * kKvqHeadBytes;
            *reinterpret_cast<uint16_t *>(kp + kvq_k_quad_offset(t, lane)) = (uint16_t)kc;
            *reinterpret_cast<uint16_t *>(vp + kvq_v_quad_offset(t, lane)) = (uint16_t)vc;
            if ((lane & 7) == 0) {
                *reinterpret_cast<uint32_t *>(kp + kvq_param_offset(t, lane >> 3)) = ksm;
                *reinterpret_cast<uint32_t *>(vp + kvq_param_offset(t, lane >> 3)) = vsm;
            }
        }
        __syncwarp();
    }
    float q[GROUP][4], acc[GROUP][4], m[GROUP], l[GROUP];
#pragma unroll
    for (int i = 0; i < GROUP; ++i) {
        uint2 w = *reinterpret_cast<const uint2 *>(a.q + b * a.ldq + (g * GROUP + i) * kD + 4 * lane);
        if (APPEND && len > 0) w = norm_rope(w, a.q_gain, a.eps, cs, sn, lane);
        q[i][0] = bf16lo(w.x) * a.scale_log2, q[i][1] = bf16hi(w.x) * a.scale_log2;
        q[i][2] = bf16lo(w.y) * a.scale_log2, q[i][3] = bf16hi(w.y) * a.scale_log2;
        acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
        m[i] = -INFINITY, l[i] = 0.f;
    }
    for (int j = 0; j < len; ++j) {
        const int page = row[j / kPS], t = j % kPS;
        if (page < 0 || page >= a.num_pages) {
            if (lane == 0) atomicOr(&g_status, QA_DEVICE_BAD_PAGE);
            continue;
        }
        const uint8_t *kp = a.k_pages + ((size_t)page * a.hkv + g) * kKvqHeadBytes;
        const uint8_t *vp = a.v_pages + ((size_t)page * a.hkv + g) * kKvqHeadBytes;
        const uint32_t kc = *reinterpret_cast<const uint16_t *>(kp + kvq_k_quad_offset(t, lane));
        const uint32_t vc = *reinterpret_cast<const uint16_t *>(vp + kvq_v_quad_offset(t, lane));
        const uint32_t ksm = *reinterpret_cast<const uint32_t *>(kp + kvq_param_offset(t, lane >> 3));
        const uint32_t vsm = *reinterpret_cast<const uint32_t *>(vp + kvq_param_offset(t, lane >> 3));
        float k[4], v[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            k[c] = fmaf(bf16lo(ksm), (float)((kc >> (4 * c)) & 15u), bf16hi(ksm));
            v[c] = fmaf(bf16lo(vsm), (float)((vc >> (4 * c)) & 15u), bf16hi(vsm));
        }
#pragma unroll
        for (int i = 0; i < GROUP; ++i) {
            const float s = warp_sum(q[i][0] * k[0] + q[i][1] * k[1] + q[i][2] * k[2] + q[i][3] * k[3]);
            const float m_new = fmaxf(m[i], s);
            const float alpha = exp2_approx(m[i] - m_new), p = exp2_approx(s - m_new);
            m[i] = m_new;
            l[i] = l[i] * alpha + p;
#pragma unroll
            for (int c = 0; c < 4; ++c) acc[i][c] = acc[i][c] * alpha + p * v[c];
        }
    }
#pragma unroll
    for (int i = 0; i < GROUP; ++i) {
        const float inv = l[i] > 0.f ? 1.f / l[i] : (l[i] == 0.f ? 0.f : l[i]);
        *reinterpret_cast<uint2 *>(a.out + ((size_t)b * a.hkv * GROUP + g * GROUP + i) * kD + 4 * lane) =
            make_uint2(pack_bf16x2(acc[i][0] * inv, acc[i][1] * inv), pack_bf16x2(acc[i][2] * inv, acc[i][3] * inv));
    }
}

}  // namespace

size_t kvq_decode_workspace_bytes(int batch, int n_q_heads, int ctas) {
    (void)batch, (void)n_q_heads, (void)ctas;
    return 256;
}

cudaError_t launch_kvq_decode(const void *q, long long ldq, void *k_pages, void *v_pages, const int32_t *page_table,
                              const int32_t *seq_lens, int batch, void *out, const qa_attn_params &p, float scale,
                              int ctas, cudaStream_t stream, const KvqAppend *app) {
    (void)ctas;
    KvqArgs a = {};
    const int group = p.n_q_heads / p.n_kv_heads;
    a.q = static_cast<const uint16_t *>(q);
    a.ldq = ldq ? ldq : (long long)p.n_q_heads * kD;
    a.k_pages = static_cast<uint8_t *>(k_pages);
    a.v_pages = static_cast<uint8_t *>(v_pages);
    a.page_table = page_table;
    a.seq_lens = seq_lens;
    a.out = static_cast<uint16_t *>(out);
    a.batch = batch;
    a.hkv = p.n_kv_heads;
    a.max_pages = p.max_pages_per_seq;
    a.num_pages = p.num_pages;
    a.scale_log2 = scale * kLog2e;
    if (app) {
        const qa_rope &rope = *app->rope;
        a.k_new = static_cast<const uint16_t *>(app->k_new);
        a.v_new = static_cast<const uint16_t *>(app->v_new);
        a.ldkv = app->ldkv ? app->ldkv : (long long)p.n_kv_heads * kD;
        a.q_gain = rope.q_gain;
        a.k_gain = rope.k_gain;
        a.positions = rope.positions;
        a.n_axes = rope.n_axes;
        a.eps = rope.rms_eps;
        if (rope.pair_axis) memcpy(a.pair_axis, rope.pair_axis, kD / 2);
        rope_frequencies(rope.theta, kD, a.freq_hi, a.freq_lo);
    }
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(batch * p.n_kv_heads));
    cfg.blockDim = dim3(32);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    auto kernel = app ? (group == 2 ? kvq_decode_kernel<2, true> : kvq_decode_kernel<1, true>)
                      : (group == 2 ? kvq_decode_kernel<2, false> : kvq_decode_kernel<1, false>);
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

unsigned int status_read_clear_kvq_decode(cudaStream_t stream, cudaError_t *err) {
    unsigned int v = 0, zero = 0;
    cudaError_t e = cudaMemcpyFromSymbolAsync(&v, g_status, sizeof v, 0, cudaMemcpyDeviceToHost, stream);
    if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
    if (e == cudaSuccess && v) e = cudaMemcpyToSymbolAsync(g_status, &zero, sizeof zero, 0, cudaMemcpyHostToDevice, stream);
    if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
    if (err) *err = e;
    return v;
}

}  // namespace qa
