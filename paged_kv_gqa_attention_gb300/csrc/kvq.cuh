// The 4-bit KV page format, and the arithmetic of its groups (qa.h,
// qa_kvq_page_bytes, has the format in words).
//
// Why this order of the bytes: decode multiplies the codes on the tensor
// cores with mma.m16n8k16, whose A fragment gives lane 4 r + c rows r and
// r + 8 and, in each 32-bit register, two neighbouring k.  K is the A of
// scores (rows tokens, k dims), V^T the A of outputs (rows dims, k tokens).
// The codes lie so that each lane's share of a page is whole 16-byte words,
// neighbouring lanes read neighbouring words, and the two halves of a
// 32-bit word are one register's two k: masking one nibble of both halves
// gives the register, a pair of fp16 subnormals, without a shuffle.
#pragma once

#include <float.h>
#include <math_constants.h>

#include "common.cuh"

namespace qa {

constexpr int kKvqTokens = 16;      // tokens of a page
constexpr int kKvqDim = 128;
constexpr int kKvqGroups = 4;       // groups of 32 dims in a head vector
constexpr int kKvqCodeBytes = 1024; // of one head in a page
constexpr int kKvqHeadBytes = 1280; // codes and parameters

// Byte offsets inside a head's part of a page.
__host__ __device__ constexpr int kvq_k_quad_offset(int t, int quad) {  // 4 dims from 4 quad on: 2 bytes
    return t * 64 + (quad % 8 / 2) * 16 + (quad / 8) * 4 + (quad & 1) * 2;
}
__host__ __device__ constexpr int kvq_v_quad_offset(int t, int quad) {
    return (t / 8) * 512 + (quad % 8) * 64 + (t % 8 / 2) * 16 + (quad / 8) * 4 + (t & 1) * 2;
}
__host__ __device__ constexpr int kvq_param_offset(int t, int g) { return kKvqCodeBytes + t * 16 + g * 4; }

// A group's parameters: s (bf16 bits, low half) and m (high half), and the
// fp32 factor that turns x - m into codes.
struct KvqGroup {
    uint32_t sm;
    float m, r;
};

// Parameters of a group with minimum lo and maximum hi (bf16 values; NaN if
// the group holds one).  d / 15: one step of Newton's residual correction
// (P. W. Markstein, "Computation of elementary functions on the IBM RISC
// System/6000 processor", 1990) rounds it correctly for the d that give a
// normal s.
__device__ __forceinline__ KvqGroup kvq_group(float lo, float hi) {
    KvqGroup g;
    const float d = __fsub_rn(hi, lo);
    constexpr float kInv15 = 1.0f / 15.0f;
    const float q0 = __fmul_rn(d, kInv15);
    const float q1 = __fmaf_rn(__fmaf_rn(-15.0f, q0, d), kInv15, q0);
    uint32_t s = pack_bf16x2(q1, 0.f) & 0xffffu;
    float sf = bf16lo(s);
    if (!(sf >= FLT_MIN)) s = 0, sf = 0.f;
    g.sm = s | (__float_as_uint(lo) & 0xffff0000u);
    g.m = lo;
    g.r = sf > 0.f ? __frcp_rn(sf) : 0.f;
    if (!(d <= FLT_MAX)) {  // an infinity or NaN: the whole group is NaN, codes 0
        g.sm = 0x7fc07fc0u;
        g.m = 0.f;
        g.r = CUDART_NAN_F;
    }
    return g;
}

// Code of x in its group: rint((x - m) r) by adding 1.5 * 2^23, whose ulp is
// 1, so the sum's low bits are the rounded value (at most 15: s is within
// 2^-9 of range / 15).  A group of NaN has codes 0.
__device__ __forceinline__ uint32_t kvq_code(float x, const KvqGroup &g) {
    const float y = __fadd_rn(__fmul_rn(__fsub_rn(x, g.m), g.r), 12582912.0f);
    return isnan(g.r) ? 0u : (__float_as_uint(y) & 15u);
}

}  // namespace qa
