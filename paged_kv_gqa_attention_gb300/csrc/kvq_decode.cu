// Paged GQA decode over a 4-bit KV pool (qa_kvq_decode_attn), and the decode
// step that norms, rotates, quantises and appends the new token first
// (qa_kvq_decode_step).
//
//   score_j = scale sum_g (m_jg sum_{d in g} q_d + s_jg sum_{d in g} q_d n_jd)
//   out = sum_j p_j (m_j + s_j n_j) / sum_j p_j,  p = exp(score - max)
//
// What bounds it: for long contexts HBM, 160 bytes a token and KV head (80 of K,
// 80 of V); below that the latency of a page's chain at 16 warps an SM
// (about 245 instructions a page and head, issue slots 50 % full, ALU 48 %,
// tensor pipe 26 %).  64 requests of 2000..16000 tokens (651 MB) take 100..105
// us, 6.2..6.5 TB/s, 91..96 % of the copy rate; 32 of 200..2000 (48 MB) 14.2
// us, of which 7 are the bytes: the rest is the launch, the first pages' round
// trip and the merging of split requests.  A step of 128 requests of 100..4000
// tokens takes 61 us, 4 more than its attention.
//
// Work split.  The pages of all requests form one flat list (request-major),
// cut into contiguous ranges (Split), one a worker.  A worker is one warp for
// each KV head, and a CTA of 8 warps holds 8 / Hkv workers, two CTAs an SM.
// Every warp streams the part of its own head (1280 contiguous bytes of a K
// page and of a V page) through its own ring of shared memory with 16-byte
// asynchronous copies, five a lane and page, so the warps of a CTA never
// meet after the prologue: there is no producer warp to feed, no barrier to
// poll and none to release a stage (651 MB: a producer warp with bulk copies
// into a ring shared by the heads 110 us, bulk copies by each warp 115 us,
// these, with arithmetic in pairs, 103 us: successive steps, not one change).
//
// A request that lies in one worker's range is finished there.  Otherwise
// each worker writes an fp32 partial (maximum, sum, outputs) to slot v + b
// (worker v, request b: unique, since both ranges are ordered) and counts
// itself in the arrival counter of (request, KV head); the warp that arrives
// last merges the partials and resets the counter, so nothing waits on
// another CTA.  Many partials are merged in two levels.
//
// Arithmetic of one page and KV head (16 tokens, mma.m16n8k16 on fp16, fp32
// sums).  A masked nibble of both halves of a code word is a pair of fp16
// subnormals, n 2^-24 or 16 n 2^-24: the codes are multiplied as they lie,
// exactly and without an offset to take back (a word of 8 codes costs one
// shift and four ANDs; as 128 + n in bf16 it cost seven, the ALU pipe was the
// busiest, and 136 times the sums had to cancel).  q is scaled by a power of
// two to a maximum below 2^15, where bf16's 8 bits are exact in fp16 down to
// 2^-22 of the largest.  The 8 columns are (group g, query head h): B of the
// scores holds head h's dims of group g and zeros elsewhere, so one product
// gives sum_{d in g} q_d n_jd for each group apart, to which its s and m are
// applied in fp32.  B of the outputs holds p_jh s_jg, rounded to fp16 (2^-11
// of itself), and the columns of a dim's own group are kept; sum p m is kept
// in fp32 beside it.  fp16's range: p is taken against a reference maximum
// that is moved when a p passes 2^4, and p s of a group and head is
// brought to 2^11 by a factor that is moved when a product passes 65000, or
// with the reference, so it is a normal number down to 2^-25 of the largest
// p s, and rounded to 2^-36 of that below.  The factor follows the products,
// not s alone: a token of little weight may have values of any size, and one
// of all the weight values of none.  Most pages move neither, which leaves
// the reductions over tokens out.
//
// Two pages go through together: their chains of products, shuffles and
// exponentials cover one another, on 4 warps a scheduler.
#include <cuda_runtime.h>
#include <limits.h>
#include <math.h>
#include <stdint.h>
#include <string.h>
#include <algorithm>
#include <type_traits>

#include "async.cuh"
#include "kvq.cuh"
#include "qa_internal.h"
#include "rotary.cuh"

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
    float *part_acc, *group_acc;    // [slots][Hq][D]
    float *part_ml, *group_ml;      // [slots][Hq][2]
    int *arrivals;                  // kCounters words, zero between calls
    int batch, hkv, max_pages, num_pages;
    int group_from;  // workers_to_group
    float scale_log2;
    int early, early_pools;  // stable_metadata >= 1, >= 2
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
__device__ __forceinline__ uint2 norm_rope(uint2 w, float4 g, float eps, const float (&cs)[4], const float (&sn)[4], int lane) {
    const float x[4] = {bf16lo(w.x), bf16hi(w.x), bf16lo(w.y), bf16hi(w.y)};
    const float ss = warp_sum(x[0] * x[0] + x[1] * x[1] + x[2] * x[2] + x[3] * x[3]);
    const float r = rsqrtf(fmaf(ss, 1.0f / kD, eps));
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

constexpr int kMaxHkv = 8;
constexpr int kWarps = 8;             // of a CTA
constexpr int kCtasPerSm = 2;
constexpr int kMaxStages = 5;         // pages in a warp's ring
// A stage: K codes, V codes, K parameters, V parameters, so that lane l copies
// 16 bytes at 16 l of each 512.
constexpr int kStageBytes = 2 * kKvqHeadBytes;
constexpr int kAlignedBatch = 256;    // requests up to which a split may follow their boundaries: one a thread
// Pages of a worker on average up to which it may.  Requests of 200..2000
// tokens, even split and this one: 16 of them (4 pages) 12.8 and 11.4 us, 32
// (7) 16.4 and 13.6, 64 (14) 21.0 and 19.5, 80 (18) 23.2 and 22.0, 96 (22) 27.7
// and 27.1, 128 (28) 34.7 and 36.1, 200 (45) 47.5 and 48.2.
constexpr int kAlignedPages = 24;
constexpr int kMinPages = 3;          // of a worker (one request of 257 tokens: 1 page 7.3 us, 2 6.4, 3 6.2, 4 6.8)
constexpr int kMergeMost = 8;         // partials merged in one round of loads, workers of a group (10 and 12 spill)
constexpr int kAtV = kKvqCodeBytes, kAtKp = 2 * kKvqCodeBytes, kAtVp = kAtKp + kKvqHeadBytes - kKvqCodeBytes;
constexpr float kRefSlack = 16.f;     // p above which the reference is moved
constexpr float kProductAim = 2048.f;   // p s times its factor: the largest when the factor was set,
constexpr float kProductMost = 65000.f; // and what moves it (fp16 ends at 65504)

constexpr int kFullRings = 2048;      // requests up to which rings have all their stages

// Workers of a CTA.
__host__ __device__ constexpr int workers_of(int hkv) { return kWarps / hkv; }

struct SmemLayout {
    uint32_t stages, off_scan, off_new, off_freq, off_pieces, off_prefix, total;
};

// Two CTAs share an SM's 227 KB; the prefix sums of a large batch cost one
// stage of every ring.
__host__ __device__ constexpr SmemLayout smem_layout(int batch) {
    SmemLayout s = {};
    s.stages = batch <= kFullRings ? kMaxStages : kMaxStages - 1;
    uint32_t o = s.stages * kStageBytes * kWarps;
    s.off_scan = o;  // warp sums of the prefix scan
    o += kWarps * 4;
    s.off_new = o;  // the step's new row of each warp: codes and parameters
    o += kWarps * 32 * 8;
    s.off_freq = o;  // rotation frequencies (hi, lo) and axes of the 64 pairs
    o += kD / 2 * 8 + kD / 2;
    s.off_pieces = o;  // workers of the requests before each, where a split follows them
    o += (kAlignedBatch + 1) * 4;
    s.off_prefix = o;
    o += (batch + 1) * 4;
    s.total = (o + 15) & ~15u;
    return s;
}

constexpr uint32_t kMostSmem = std::max(smem_layout(kFullRings).total, smem_layout(kDecodeMaxBatch).total);

// Workspace: arrival counters in a region of fixed size, zero between calls,
// then the partials of workers and of groups.  The region is the one that the
// bf16 decode has its counters in, so that calls of both may share a
// workspace: neither's partials lie on the other's counters.  A request's
// counters (one a KV head) are counted from the region's start, those of
// groups of workers from its end.
constexpr int kCounters = kDecodeMaxBatch * kMaxHkv;
struct WorkspaceLayout {
    size_t arrivals, acc, ml, group_acc, group_ml, total;
};

__host__ __device__ inline WorkspaceLayout workspace_layout(int batch, int hq, int workers) {
    const size_t slots = (size_t)workers + (size_t)batch;
    const size_t group_slots = (size_t)workers / kMergeMost + 1 + (size_t)batch;
    const auto up = [](size_t x) { return (x + 255) & ~(size_t)255; };
    WorkspaceLayout w;
    w.arrivals = 0;
    w.acc = up((size_t)kCounters * sizeof(int));
    w.ml = w.acc + up(slots * hq * kD * sizeof(float));
    w.group_acc = w.ml + up(slots * hq * 2 * sizeof(float));
    w.group_ml = w.group_acc + up(group_slots * hq * kD * sizeof(float));
    w.total = w.group_ml + up(group_slots * hq * 2 * sizeof(float));
    return w;
}

// Place, from the region's end, of the counter of group q of a request that is
// merged by groups, q0 its first one, for KV head g.  Such a request has more
// than 16 workers, so at most one begins in a group, and at most one comes
// from the group before.
__device__ __forceinline__ int group_counter(int q, int q0, int g, int hkv) { return (2 * q + (q == q0)) * hkv + g + 1; }
// Workers from which a request is merged by groups: where their counters have
// room behind those of the requests, which with 8 KV heads and 304 workers is
// up to 4018 requests, with fewer heads always.
inline int workers_to_group(int batch, int workers, int hkv) {
    return (batch + 2 * (workers / kMergeMost + 1)) * hkv <= kCounters ? 2 * kMergeMost + 1 : INT_MAX;
}

// How the flat page list is cut into one range a worker, none empty.
//
// Evenly: worker v has pages [total v / nv, total (v + 1) / nv), and a CTA
// has neighbouring workers, so CTAs differ by one page at most.  With fewer
// than kMinPages for every worker there are as many workers as have that
// many, on half the CTAs (the first ones of a grid lie on different SMs): a
// worker more would save less than its partial costs to merge.
//
// By requests (pieces): where there are few pages a worker, each request gets
// workers of its own, one for up to `most` pages, if that takes no more than
// there are: a worker with the end of one request and the start of another
// pays twice for beginning and for settling, about 2 us (32 requests of
// 200..2000 tokens 16.4 -> 13.6 us, 4 of 500 9.4 -> 7.3 us), which a few
// pages' imbalance costs less than.
struct Split {
    int total, nv;
    bool half;          // on the first half of the CTAs
    const int *pieces;  // prefix sums of the requests' workers, or nullptr: evenly
    __device__ __forceinline__ int worker(int cta, int ctas, int e, int s) const {
        return !half ? cta * s + e : e * (ctas / kCtasPerSm) + (cta < ctas / kCtasPerSm ? cta : ctas * s);
    }
    // 64-bit divisions cost ten times 32-bit ones, which serve up to 2^19 pages (nv is below 2^13)
    __device__ __forceinline__ int lo(int v) const {
        if (v >= nv) return total;
        return total < 1 << 19 ? (int)((uint32_t)total * (uint32_t)v / (uint32_t)nv) : (int)((long long)total * v / nv);
    }
    __device__ __forceinline__ int of_page(int x) const {
        return total < 1 << 19 ? (int)(((uint32_t)(x + 1) * (uint32_t)nv - 1u) / (uint32_t)total)
                               : (int)((((long long)x + 1) * nv - 1) / total);
    }
};

// Pages request b contributes; invalid lengths and positions contribute none
// (and are reported once, by CTA 0).
template <bool APPEND>
__device__ __forceinline__ int pages_of(const KvqArgs &a, int b, bool report) {
    const int len = a.seq_lens[b];
    if (len < (APPEND ? 1 : 0) || len > a.max_pages * kPS) {
        if (report) atomicOr(&g_status, QA_DEVICE_BAD_LENGTH);
        return 0;
    }
    if (APPEND && a.positions) {
        bool ok = true;
        for (int x = 0; x < a.n_axes; ++x) {
            const int pos = a.positions[(size_t)x * a.batch + b];
            ok &= pos >= 0 && pos < kMaxRopePos;
        }
        if (!ok) {
            if (report) atomicOr(&g_status, QA_DEVICE_BAD_POSITION);
            return 0;
        }
    }
    return (len + kPS - 1) / kPS;
}

// First request b whose pages reach past page x (prefix[b + 1] > x).
__device__ __forceinline__ int request_of(const int *prefix, int batch, int x) {
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

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The same from zero.
__device__ __forceinline__ void mma16816_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                               uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// 8 x 8 transpose of 16-bit values over the warp: lane 4 i + j gives and gets
// row i, columns 2j and 2j + 1.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// fp16 pair of nibble I of both halves of a code word: n 2^-24 (I even) or
// 16 n 2^-24 (I odd).
template <int I>
__device__ __forceinline__ uint32_t code_pair(uint32_t w) {
    return (I < 2 ? w : w >> 8) & (I & 1 ? 0x00f000f0u : 0x000f000fu);
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    uint32_t d;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}

// The power of two 2^e (e in [-126, 127]).
__device__ __forceinline__ float pow2i(int e) { return __int_as_float((e + 127) << 23); }
__device__ __forceinline__ int exponent_of(float x) { return (__float_as_int(x) >> 23 & 255) - 127; }

// Merges the partials at slots [s0, s0 + n) of both heads of KV head g: the
// lane's dims, maximum and sum.  A round loads kMergeMost partials at once;
// lane 16 i + u holds the maximum and sum of the round's partial u of head i.
template <int GROUP>
__device__ __forceinline__ void merge(const float *acc, const float *ml, size_t s0, int n, int hq, int g, int lane,
                                      float (&z)[GROUP][4], float (&m)[GROUP], float (&ls)[GROUP]) {
    static_assert(kMergeMost <= 16, "a head's partials of a round lie on 16 lanes");
#pragma unroll
    for (int i = 0; i < GROUP; ++i) z[i][0] = z[i][1] = z[i][2] = z[i][3] = 0.f;
    float m_own = -INFINITY, l_own = 0.f;  // of this lane's head: maximum (of both lanes' halves alike), sum over its partials
    for (int w0 = 0; w0 < n; w0 += kMergeMost) {
        const int cnt = min(kMergeMost, n - w0);
        const int hi = GROUP == 2 ? lane >> 4 : 0, u_own = lane & 15;
        float2 mine = make_float2(-INFINITY, 0.f);
        if (u_own < cnt) mine = __ldcg(reinterpret_cast<const float2 *>(ml + ((s0 + w0 + u_own) * hq + g * GROUP + hi) * 2));
        float4 pv[GROUP][kMergeMost];
#pragma unroll
        for (int u = 0; u < kMergeMost; ++u)
#pragma unroll
            for (int i = 0; i < GROUP; ++i)
                pv[i][u] = __ldcg(reinterpret_cast<const float4 *>(acc + ((s0 + w0 + min(u, cnt - 1)) * hq + g * GROUP + i) * kD + 4 * lane));
        float mb = fmaxf(m_own, mine.x);
#pragma unroll
        for (int o = 1; o < 16; o <<= 1) mb = fmaxf(mb, __shfl_xor_sync(0xffffffffu, mb, o));
        const float at = mb == -INFINITY ? 0.f : mb;  // nothing attended so far: weights 2^-inf
        const float alpha = exp2_approx(m_own - at);
        const float w_own = u_own < cnt ? exp2_approx(mine.x - at) : 0.f;
        l_own = fmaf(w_own, mine.y, l_own * alpha);
        m_own = mb;
#pragma unroll
        for (int i = 0; i < GROUP; ++i) {
            const float al = __shfl_sync(0xffffffffu, alpha, 16 * i);
#pragma unroll
            for (int k = 0; k < 4; ++k) z[i][k] *= al;
#pragma unroll
            for (int u = 0; u < kMergeMost; ++u) {
                const float w = __shfl_sync(0xffffffffu, w_own, 16 * i + u);
                if (u < cnt) {
                    z[i][0] = fmaf(w, pv[i][u].x, z[i][0]);
                    z[i][1] = fmaf(w, pv[i][u].y, z[i][1]);
                    z[i][2] = fmaf(w, pv[i][u].z, z[i][2]);
                    z[i][3] = fmaf(w, pv[i][u].w, z[i][3]);
                }
            }
        }
    }
#pragma unroll
    for (int o = 1; o < 16; o <<= 1) l_own += __shfl_xor_sync(0xffffffffu, l_own, o);
#pragma unroll
    for (int i = 0; i < GROUP; ++i) {
        m[i] = __shfl_sync(0xffffffffu, m_own, 16 * i);
        ls[i] = __shfl_sync(0xffffffffu, l_own, 16 * i);
    }
}

template <int GROUP>
__device__ __forceinline__ void write_partial(float *acc, float *ml, size_t slot, int hq, int g, int lane, const float (&z)[GROUP][4],
                                              const float (&m)[GROUP], const float (&l)[GROUP]) {
#pragma unroll
    for (int i = 0; i < GROUP; ++i) {
        const size_t row = slot * hq + g * GROUP + i;
        *reinterpret_cast<float4 *>(acc + row * kD + 4 * lane) = make_float4(z[i][0], z[i][1], z[i][2], z[i][3]);
        if (lane == 0) *reinterpret_cast<float2 *>(ml + row * 2) = make_float2(m[i], l[i]);
    }
}

// Lane 4 r + c holds dims [32 c + 4 r, + 4) of an output row.
template <int GROUP>
__device__ __forceinline__ void write_out(uint16_t *out, int hq, int b, int g, int lane, const float (&z)[GROUP][4],
                                          const float (&l)[GROUP]) {
#pragma unroll
    for (int i = 0; i < GROUP; ++i) {
        const float inv = l[i] == 0.f ? 0.f : 1.f / l[i];
        *reinterpret_cast<uint2 *>(out + ((size_t)b * hq + g * GROUP + i) * kD + 32 * (lane & 3) + 4 * (lane >> 2)) =
            make_uint2(pack_bf16x2(z[i][0] * inv, z[i][1] * inv), pack_bf16x2(z[i][2] * inv, z[i][3] * inv));
    }
}

// Counts this warp in after all its writes, and tells (every lane) whether it
// was the last of `others` + 1.  Lane 0's fences order the partials before
// the count and, in the last one, the reads after it.
__device__ __forceinline__ bool last_in(int *counter, int others, int lane) {
    __syncwarp();
    int before = 0;
    if (lane == 0) {
        asm volatile("fence.acq_rel.gpu;" ::: "memory");
        asm volatile("atom.add.relaxed.gpu.s32 %0, [%1], 1;" : "=r"(before) : "l"(counter) : "memory");
        if (before == others) asm volatile("fence.acq_rel.gpu;" ::: "memory");
    }
    __syncwarp();
    return __shfl_sync(0xffffffffu, before, 0) == others;
}

template <int GROUP, bool APPEND>
__global__ void __launch_bounds__(kWarps * 32, kCtasPerSm) kvq_decode_kernel(const __grid_constant__ KvqArgs a) {
    extern __shared__ __align__(128) uint8_t smem[];
    const SmemLayout L = smem_layout(a.batch);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int S = workers_of(a.hkv);
    const int hq = a.hkv * GROUP;
    const int n_stages = (int)L.stages;
    int *prefix = reinterpret_cast<int *>(smem + L.off_prefix);
    int *scan = reinterpret_cast<int *>(smem + L.off_scan);
    uint8_t *ring = smem + warp * n_stages * kStageBytes;
    const uint32_t ring_base = smem_u32(ring), ring_end = ring_base + n_stages * kStageBytes;

    if (!a.early) grid_wait();
    if (threadIdx.x == 0) prefix[0] = 0;
    float2 *freq = reinterpret_cast<float2 *>(smem + L.off_freq);
    uint2 *new_row = reinterpret_cast<uint2 *>(smem + L.off_new) + 32 * warp;
    uint8_t *axis = smem + L.off_freq + kD / 2 * 8;
    if (APPEND && threadIdx.x < kD / 2) {
        const float *f_hi = a.freq_hi, *f_lo = a.freq_lo;
        const uint8_t *pair_axis = a.pair_axis;
        asm("" : "+l"(f_hi), "+l"(f_lo), "+l"(pair_axis));  // as memory: the constant bank serves one address at a time
        freq[threadIdx.x] = make_float2(f_hi[threadIdx.x], f_lo[threadIdx.x]);
        axis[threadIdx.x] = pair_axis[threadIdx.x];
    }
    // sums over the CTA's threads before this one, and of all; every thread calls it
    auto scan_block = [&](int own, int &sum) -> int {
        int v = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += u;
        }
        if (lane == 31) scan[warp] = v;
        __syncthreads();
        int before = v - own;
        sum = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const int x = scan[w];
            before += w < warp ? x : 0;
            sum += x;
        }
        __syncthreads();
        return before;
    };
    // prefix sums of the page counts, one request a thread
    int total = 0, own_pages = 0;
    for (int base = 0; base < a.batch; base += kWarps * 32) {
        const int b = base + threadIdx.x;
        own_pages = b < a.batch ? pages_of<APPEND>(a, b, blockIdx.x == 0) : 0;
        int sum;
        const int before = total + scan_block(own_pages, sum);
        if (b < a.batch) prefix[b + 1] = before + own_pages;
        total += sum;
    }
    Split split;
    {
        const int most_workers = gridDim.x * S;
        split.total = total;
        split.half = total < most_workers * kMinPages;
        split.nv = split.half ? most_workers / kCtasPerSm : most_workers;
        split.pieces = nullptr;
        if (a.batch <= kAlignedBatch && total > 0 && total < most_workers * kAlignedPages) {
            // the smallest of four sizes that serves, from the even one to a quarter above; two sums a word
            int most = max(kMinPages, (total + split.nv - 1) / split.nv), chosen = 0, sum;
            for (int k = 0; k < 4 && !chosen; k += 2) {
                const int m0 = most + (most * k + 11) / 12, m1 = most + (most * (k + 1) + 11) / 12;
                scan_block((own_pages + m0 - 1) / m0 | (own_pages + m1 - 1) / m1 << 16, sum);
                chosen = (sum & 0xffff) <= split.nv ? m0 : sum >> 16 <= split.nv ? m1 : 0;
            }
            if (chosen) {
                int *pieces = reinterpret_cast<int *>(smem + L.off_pieces);
                const int own = (own_pages + chosen - 1) / chosen, before = scan_block(own, split.nv);
                if (threadIdx.x == 0) pieces[0] = 0;
                if ((int)threadIdx.x < a.batch) pieces[threadIdx.x + 1] = before + own;
                split.pieces = pieces;
            }
        }
        if (!split.pieces && split.half) split.nv = min(split.nv, max(1, total / kMinPages));
        if (split.nv > total) split.nv = total;
        __syncthreads();
    }

    // this warp: KV head g of worker v, pages [lo, hi) of the flat list
    const int g = warp % a.hkv, e = warp / a.hkv;
    const int v = split.worker(blockIdx.x, gridDim.x, e, S);
    const bool working = e < S && v < split.nv;
    int lo = 0, hi = 0, b = 0;  // b: the request of page lo
    if (working) {
        if (split.pieces) {
            b = request_of(split.pieces, a.batch, v);
            const int i = v - split.pieces[b], n = split.pieces[b + 1] - split.pieces[b], p0 = prefix[b], pages = prefix[b + 1] - p0;
            lo = p0 + (int)((uint32_t)pages * i / n), hi = p0 + (int)((uint32_t)pages * (i + 1) / n);
        } else {
            lo = split.lo(v), hi = split.lo(v + 1);
            b = request_of(prefix, a.batch, lo);
        }
    }
    // page ids, 32 at a time, one a lane: bad ones are -1.  Windows overlap by two, so that a pair of pages lies in one.
    bool any_bad = false;
    auto find = [&](int x) -> int {
        int page = -1;
        bool bad = false;
        if (x < hi) {
            const int b = request_of(prefix, a.batch, x);
            page = a.page_table[(size_t)b * a.max_pages + (x - prefix[b])];
            if (page < 0 || page >= a.num_pages) {
                atomicOr(&g_status, QA_DEVICE_BAD_PAGE);
                page = -1;
                bad = true;
            }
        }
        any_bad |= __any_sync(0xffffffffu, bad);
        return page;
    };
    int ids = find(lo + lane), ids_next = -1;
    int to_issue = hi - lo, in_window = 0;  // pages to copy yet, and the next one's place among the ids
    const uint64_t policy = policy_evict_first();
    const size_t head_at = (size_t)g * kKvqHeadBytes + 16 * lane;
    const uint8_t *k_src = a.k_pages + head_at, *v_src = a.v_pages + head_at;
    const uint8_t *p_src = (lane < 16 ? a.k_pages : a.v_pages - 256) + kKvqCodeBytes + head_at;
    const uint32_t page_stride = (uint32_t)a.hkv * kKvqHeadBytes;
    auto issue = [&](auto np, const uint32_t *stage) {  // the next NP pages, or nothing after the last: groups either way
        constexpr int NP = decltype(np)::value;
#pragma unroll
        for (int y = 0; y < NP; ++y) {
            if (y < to_issue) {
                const int page = __shfl_sync(0xffffffffu, ids, in_window + y);
                if (page >= 0) {
                    const size_t off = (size_t)(uint32_t)page * page_stride;
                    const uint32_t dst = stage[y] + 16 * lane;
                    copy16(dst, k_src + off, policy);
                    copy16(dst + 512, k_src + off + 512, policy);
                    copy16(dst + kAtV, v_src + off, policy);
                    copy16(dst + kAtV + 512, v_src + off + 512, policy);
                    copy16(dst + kAtKp, p_src + off, policy);
                }
            }
            copy_commit();
        }
        to_issue -= NP, in_window += NP;
        if (in_window >= 30) {
            ids = ids_next, in_window -= 30;
        } else if (in_window >= 16 && in_window < 16 + NP) {
            ids_next = find(hi - to_issue - in_window + 30 + lane);
        }
    };

    // The first request's length, and (step) the angles that its position gives: metadata, read before the wait too.
    int seq_len = lo < hi ? a.seq_lens[b] : 0;
    float cs[4], sn[4];
    auto angles = [&]() {  // of pairs 4 (l mod 16) + u: each of two lanes takes half of them
        int pos_own = seq_len - 1;
        if (a.positions) pos_own = lane < a.n_axes ? a.positions[(size_t)lane * a.batch + b] : 0;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int i = 4 * (lane & 15) + (lane >> 4) * 2 + u;
            const int pos = a.positions ? __shfl_sync(0xffffffffu, pos_own, axis[i]) : pos_own;
            float s1, c1;
            sincos_turns(pos, freq[i].x, freq[i].y, &s1, &c1);
            const float s2 = __shfl_xor_sync(0xffffffffu, s1, 16), c2 = __shfl_xor_sync(0xffffffffu, c1, 16);
            sn[u] = lane < 16 ? s1 : s2, sn[2 + u] = lane < 16 ? s2 : s1;
            cs[u] = lane < 16 ? c1 : c2, cs[2 + u] = lane < 16 ? c2 : c1;
        }
    };
    // With the pools vouched for (early_pools) the rings fill before the wait.
    if (a.early && !a.early_pools) grid_wait();
#pragma unroll 1
    for (int s = 0; s < n_stages; ++s) {
        const uint32_t stage[1] = {ring_base + s * kStageBytes};
        issue(std::integral_constant<int, 1>(), stage);
    }
    if (APPEND && lo < hi) angles();
    if (a.early && a.early_pools) grid_wait();

    if (blockIdx.x == 0) {  // zero rows of requests with nothing to attend over
        const int chunks = hq * kD * 2 / 16;
        for (int b = warp; b < a.batch; b += kWarps) {
            if (prefix[b + 1] != prefix[b]) continue;
            uint4 *dst = reinterpret_cast<uint4 *>(a.out + (size_t)b * hq * kD);
            for (int c = lane; c < chunks; c += 32) dst[c] = make_uint4(0u, 0u, 0u, 0u);
        }
    }
    if (lo >= hi) return;
    const int r = lane >> 2, c = lane & 3;

    // A split request's partial: written, counted in, and merged with the others where this warp is the last.  A request
    // over more workers than two rounds of loads take is merged by groups of neighbouring workers first, each by the
    // last of its group.  The first of a worker's two split requests is settled before its other pages: left to the
    // end, one warp merged both, which the whole grid waited for.
    auto settle = [&](int b, const float (&acc)[GROUP][4], const float (&ref)[GROUP], const float (&sum)[GROUP]) {
        write_partial<GROUP>(a.part_acc, a.part_ml, (size_t)v + b, hq, g, lane, acc, ref, sum);
        const int v0 = split.pieces ? split.pieces[b] : split.of_page(prefix[b]);
        const int v1 = split.pieces ? split.pieces[b + 1] - 1 : split.of_page(prefix[b + 1] - 1);
        int *counter = a.arrivals + b * a.hkv + g;
        float z[GROUP][4], m[GROUP], l[GROUP];
        if (v1 - v0 + 1 >= a.group_from) {
            const int q = v / kMergeMost, q0 = v0 / kMergeMost, q1 = v1 / kMergeMost;
            const int a0 = max(v0, q * kMergeMost), a1 = min(v1, q * kMergeMost + kMergeMost - 1);
            int *group = a.arrivals + kCounters - group_counter(q, q0, g, a.hkv);
            if (!last_in(group, a1 - a0, lane)) return;
            merge<GROUP>(a.part_acc, a.part_ml, (size_t)a0 + b, a1 - a0 + 1, hq, g, lane, z, m, l);
            if (lane == 0) *group = 0;
            write_partial<GROUP>(a.group_acc, a.group_ml, (size_t)q + b, hq, g, lane, z, m, l);
            if (!last_in(counter, q1 - q0, lane)) return;
            merge<GROUP>(a.group_acc, a.group_ml, (size_t)q0 + b, q1 - q0 + 1, hq, g, lane, z, m, l);
        } else {
            if (!last_in(counter, v1 - v0, lane)) return;
            merge<GROUP>(a.part_acc, a.part_ml, (size_t)v0 + b, v1 - v0 + 1, hq, g, lane, z, m, l);
        }
        write_out<GROUP>(a.out, hq, b, g, lane, z, l);
        if (lane == 0) *counter = 0;
    };
    uint32_t at = ring_base;    // stage of the next page

    for (int x = lo; x < hi;) {
        const int p0 = prefix[b], p1 = prefix[b + 1];
        const int j0 = x - p0, j1 = min(hi, p1) - p0;
        uint2 qw[GROUP], kw = make_uint2(0u, 0u), vw = kw;
#pragma unroll
        for (int i = 0; i < GROUP; ++i)
            qw[i] = *reinterpret_cast<const uint2 *>(a.q + b * a.ldq + (g * GROUP + i) * kD + 4 * lane);
        const bool has_new = APPEND && j1 == p1 - p0;
        if (APPEND) {
            const float4 gq = *reinterpret_cast<const float4 *>(a.q_gain + 4 * lane);
            float4 gk;
            if (has_new) {
                const size_t o = b * a.ldkv + g * kD + 4 * lane;
                kw = *reinterpret_cast<const uint2 *>(a.k_new + o);
                vw = *reinterpret_cast<const uint2 *>(a.v_new + o);
                gk = *reinterpret_cast<const float4 *>(a.k_gain + 4 * lane);
            }
            if (x != lo) angles();
#pragma unroll
            for (int i = 0; i < GROUP; ++i) qw[i] = norm_rope(qw[i], gq, a.eps, cs, sn, lane);
            if (has_new) {
                uint32_t k_sm, v_sm;
                const uint32_t k_codes = quantise_row(norm_rope(kw, gk, a.eps, cs, sn, lane), lane, k_sm);
                const uint32_t v_codes = quantise_row(vw, lane, v_sm);
                new_row[lane] = make_uint2(k_codes | v_codes << 16, lane & 1 ? v_sm : k_sm);  // parameters of K on even lanes
            }
        }
        // the next request: its q on its way to L2 (in registers a segment ahead it cost spills), its length read
        int b_next = b + 1, len_next = 0;
        if (p1 < hi) {
            while (prefix[b_next + 1] == prefix[b_next]) ++b_next;
            len_next = a.seq_lens[b_next];
            const uint8_t *q_row = reinterpret_cast<const uint8_t *>(a.q + b_next * a.ldq + g * GROUP * kD);
            if (lane < GROUP * 2) prefetch_l2(q_row + 128 * lane);
        }
        // B of the scores: lane (n, c), n = (group n / 2, head n % 2), holds head n % 2's dims [32 g + 8 c, + 8) of its
        // own group, as the pairs (j, j + 4) that the code words hold, a 16th of the pairs whose codes come 16-fold
        uint32_t bq[16];
        float2 qsum = make_float2(0.f, 0.f);  // softmax scale times the sum of the heads' q over group c
        float2 qback = qsum;                  // softmax scale times 2^24 / q's scale
        {
            float w[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
            const int src = 8 * (r >> 1) + 2 * c;
#pragma unroll
            for (int i = 0; i < GROUP; ++i) {
                const float x[4] = {bf16lo(qw[i].x), bf16hi(qw[i].x), bf16lo(qw[i].y), bf16hi(qw[i].y)};
                float m = fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3])));
                float s = (x[0] + x[1]) + (x[2] + x[3]);
#pragma unroll
                for (int o = 1; o < 8; o <<= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
                const int k = max(min(14 - exponent_of(m), 126), -100);  // 126: q is zero or nearly; -100: it is past 2^114
                const float up = pow2i(k), back = pow2i(24 - k) * a.scale_log2;
                s = __shfl_sync(0xffffffffu, s, 8 * c) * a.scale_log2;
                if (i == 0) qsum.x = s, qback.x = back; else qsum.y = s, qback.y = back;
#pragma unroll
                for (int d = 0; d < 4; ++d) {
                    const float y0 = __shfl_sync(0xffffffffu, x[d] * up, src), y1 = __shfl_sync(0xffffffffu, x[d] * up, src + 1);
                    if ((r & 1) == i) w[d] = y0, w[4 + d] = y1;
                }
            }
            const uint32_t pr[4] = {pack_f16x2(w[0], w[4]), pack_f16x2(w[1] * 0.0625f, w[5] * 0.0625f), pack_f16x2(w[2], w[6]),
                                    pack_f16x2(w[3] * 0.0625f, w[7] * 0.0625f)};
#pragma unroll
            for (int k2 = 0; k2 < 16; ++k2) bq[k2] = (k2 >> 2) == (r >> 1) ? pr[k2 & 3] : 0u;
        }
        // outputs, and of both heads (x, y): the reference (log2), sum of p and sum of p m over this lane's tokens
        float o[8][4];
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
        float2 ref = make_float2(-INFINITY, -INFINITY), l = make_float2(0.f, 0.f), corr = make_float2(0.f, 0.f);
        float2 up = make_float2(INFINITY, GROUP == 2 ? INFINITY : 0.f);  // factor of p s: the first page sets it

        // NP neighbouring pages at once: their chains of products, shuffles and exponentials are independent
        auto pages = [&](auto np, int j) {
            constexpr int NP = decltype(np)::value;
            if (n_stages == kMaxStages) copy_wait<kMaxStages - NP>(); else copy_wait<kMaxStages - 1 - NP>();
            __syncwarp();
            uint32_t ks[NP], vp0[NP], vp1[NP];
#pragma unroll
            for (int y = 0; y < NP; ++y) {
                ks[y] = at;
                at = at + kStageBytes == ring_end ? ring_base : at + kStageBytes;
            }
            const int left = seq_len - j * kPS;  // tokens from the first of these pages on
            if (has_new && j + NP == j1) {
                // the new token's row, in the stage and in the pools
                const int t = left - 1 - (NP - 1) * kPS, page = a.page_table[(size_t)b * a.max_pages + j1 - 1];
                const uint32_t new_codes = new_row[lane].x, new_sm = new_row[lane].y;
                if (page >= 0 && page < a.num_pages) {
                    uint8_t *stage = ring + (ks[NP - 1] - ring_base);
                    const size_t off = ((size_t)page * a.hkv + g) * kKvqHeadBytes;
                    *reinterpret_cast<uint16_t *>(stage + kvq_k_quad_offset(t, lane)) = (uint16_t)new_codes;
                    *reinterpret_cast<uint16_t *>(stage + kAtV + kvq_v_quad_offset(t, lane)) = (uint16_t)(new_codes >> 16);
                    *reinterpret_cast<uint16_t *>(a.k_pages + off + kvq_k_quad_offset(t, lane)) = (uint16_t)new_codes;
                    *reinterpret_cast<uint16_t *>(a.v_pages + off + kvq_v_quad_offset(t, lane)) = (uint16_t)(new_codes >> 16);
                    if ((lane & 6) == 0) {  // two lanes of each group
                        const int p = kvq_param_offset(t, lane >> 3);
                        *reinterpret_cast<uint32_t *>(stage + (lane & 1 ? kAtVp : kAtKp) - kKvqCodeBytes + p) = new_sm;
                        *reinterpret_cast<uint32_t *>((lane & 1 ? a.v_pages : a.k_pages) + off + p) = new_sm;
                    }
                    __syncwarp();
                }
            }
            // scores: A rows are tokens r and r + 8
            float d[NP][4];
            float2 sc[NP][2];
            uint32_t kp0[NP], kp1[NP];
#pragma unroll
            for (int y = 0; y < NP; ++y) {
                const uint4 k0 = lds128(ks[y] + 16 * lane), k1 = lds128(ks[y] + 512 + 16 * lane);
                kp0[y] = lds32(ks[y] + kAtKp + 4 * lane), kp1[y] = lds32(ks[y] + kAtKp + 128 + 4 * lane);
                vp0[y] = lds32(ks[y] + kAtVp + 4 * lane), vp1[y] = lds32(ks[y] + kAtVp + 128 + 4 * lane);
                const uint32_t w0[4] = {k0.x, k0.y, k0.z, k0.w}, w1[4] = {k1.x, k1.y, k1.z, k1.w};
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    if (u == 0)
                        mma16816_first(d[y], code_pair<0>(w0[u]), code_pair<0>(w1[u]), code_pair<1>(w0[u]), code_pair<1>(w1[u]), bq[0], bq[1]);
                    else
                        mma16816(d[y], code_pair<0>(w0[u]), code_pair<0>(w1[u]), code_pair<1>(w0[u]), code_pair<1>(w1[u]), bq[4 * u],
                                 bq[4 * u + 1]);
                    mma16816(d[y], code_pair<2>(w0[u]), code_pair<2>(w1[u]), code_pair<3>(w0[u]), code_pair<3>(w1[u]),
                             bq[4 * u + 2], bq[4 * u + 3]);
                }
            }
            // s and m of (token, group c), then the sum over groups (the 4 lanes of a token)
#pragma unroll
            for (int y = 0; y < NP; ++y) {
                const float s0 = bf16lo(kp0[y]), m0 = bf16hi(kp0[y]), s1 = bf16lo(kp1[y]), m1 = bf16hi(kp1[y]);
                sc[y][0] = ffma2(fmul2(make_float2(d[y][0], d[y][1]), qback), make_float2(s0, s0), fmul2(make_float2(m0, m0), qsum));
                sc[y][1] = ffma2(fmul2(make_float2(d[y][2], d[y][3]), qback), make_float2(s1, s1), fmul2(make_float2(m1, m1), qsum));
            }
#pragma unroll
            for (int z = 1; z < 4; z <<= 1)
#pragma unroll
                for (int y = 0; y < NP; ++y)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        float2 w = make_float2(__shfl_xor_sync(0xffffffffu, sc[y][h].x, z), 0.f);
                        if (GROUP == 2) w.y = __shfl_xor_sync(0xffffffffu, sc[y][h].y, z);
                        sc[y][h] = fadd2(sc[y][h], w);
                    }
            bool none = false;
            if (left < NP * kPS || any_bad) {  // slots past the length, and bad pages, may hold anything
                int tokens = 0;
#pragma unroll
                for (int y = 0; y < NP; ++y) {
                    int nt = min(kPS, left - y * kPS);
                    if (any_bad) {
                        const int page = a.page_table[(size_t)b * a.max_pages + j + y];
                        if (page < 0 || page >= a.num_pages) nt = 0;
                    }
                    if (r >= nt) sc[y][0] = make_float2(-INFINITY, -INFINITY), vp0[y] = 0u;
                    if (r + 8 >= nt) sc[y][1] = make_float2(-INFINITY, -INFINITY), vp1[y] = 0u;
                    tokens += nt;
                }
                none = tokens == 0;  // there may be no reference yet
            }
            // p of the tokens, and p s of (token, group c) times its factor, for both heads; sums of p and p m
            float2 p[NP][2], ps[NP][2], l_next, corr_next;
            auto weigh = [&]() {
                l_next = l, corr_next = corr;
#pragma unroll
                for (int y = 0; y < NP; ++y)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t sm = h ? vp1[y] : vp0[y];
                        const float s = bf16lo(sm), m = bf16hi(sm);
                        const float2 e = fsub2(sc[y][h], ref);
                        p[y][h] = make_float2(exp2_approx(e.x), GROUP == 2 ? exp2_approx(e.y) : 0.f);
                        l_next = fadd2(l_next, p[y][h]);
                        corr_next = ffma2(p[y][h], make_float2(m, m), corr_next);
                        ps[y][h] = fmul2(fmul2(p[y][h], make_float2(s, s)), up);
                    }
            };
            if (!none) {
                bool move = j == j0;  // the first pages set the references
                if (!move) {
                    weigh();
                    float p_max = 0.f, ps_max = 0.f;
#pragma unroll
                    for (int y = 0; y < NP; ++y)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            p_max = GROUP == 2 ? fmax3(p_max, p[y][h].x, p[y][h].y) : fmaxf(p_max, p[y][h].x);
                            ps_max = GROUP == 2 ? fmax3(ps_max, fabsf(ps[y][h].x), fabsf(ps[y][h].y)) : fmaxf(ps_max, fabsf(ps[y][h].x));
                        }
                    move = __any_sync(0xffffffffu, p_max > kRefSlack || ps_max > kProductMost);
                }
                if (move) {  // the references, to the maxima so far
                    float m[GROUP], w[GROUP];  // largest score, and score with log2 s on it (p s in units of any reference)
#pragma unroll
                    for (int i = 0; i < GROUP; ++i) m[i] = w[i] = -INFINITY;
#pragma unroll
                    for (int y = 0; y < NP; ++y) {
                        const float s0 = __log2f(fabsf(bf16lo(vp0[y]))), s1 = __log2f(fabsf(bf16lo(vp1[y])));
#pragma unroll
                        for (int i = 0; i < GROUP; ++i) {
                            const float a0 = i == 0 ? sc[y][0].x : sc[y][0].y, a1 = i == 0 ? sc[y][1].x : sc[y][1].y;
                            m[i] = fmax3(m[i], a0, a1);
                            w[i] = fmax3(w[i], a0 + s0, a1 + s1);
                        }
                    }
#pragma unroll
                    for (int z = 4; z < 32; z <<= 1)
#pragma unroll
                        for (int i = 0; i < GROUP; ++i) {
                            m[i] = fmaxf(m[i], __shfl_xor_sync(0xffffffffu, m[i], z));
                            w[i] = fmaxf(w[i], __shfl_xor_sync(0xffffffffu, w[i], z));
                        }
                    float alpha[2] = {1.f, 1.f};
#pragma unroll
                    for (int i = 0; i < GROUP; ++i) {
                        float &rf = i == 0 ? ref.x : ref.y, &li = i == 0 ? l.x : l.y, &ci = i == 0 ? corr.x : corr.y;
                        float &ui = i == 0 ? up.x : up.y;
                        float f = 1.f;
                        if (m[i] > rf) {
                            f = exp2_approx(rf - m[i]);
                            rf = m[i];
                            li *= f;
                            ci *= f;
                        }
                        // the largest p s of these tokens, or what the factor stood for, in units of the new reference;
                        // within bounds where the factor and its inverse are normal numbers
                        const float before = __fdividef(f, ui);  // 0 the first time
                        const float t = fmaxf(exp2_approx(w[i] - rf), kProductAim * before);
                        ui = __fdividef(kProductAim, fminf(fmaxf(t, kProductAim / 0x1p126f), 0x1p126f));
                        alpha[i] = ui * before;
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i) o[i][0] *= alpha[0], o[i][1] *= alpha[1], o[i][2] *= alpha[0], o[i][3] *= alpha[1];
                    weigh();
                }
                l = l_next, corr = corr_next;
#pragma unroll
                for (int y = 0; y < NP; ++y) {
                    // p s rounded to fp16, transposed into B
                    const uint32_t b0 = transpose8x8(pack_f16x2(ps[y][0].x, ps[y][0].y)), b1 = transpose8x8(pack_f16x2(ps[y][1].x, ps[y][1].y));
                    const uint4 v0 = lds128(ks[y] + kAtV + 16 * lane), v1 = lds128(ks[y] + kAtV + 512 + 16 * lane);
                    const uint32_t x0[4] = {v0.x, v0.y, v0.z, v0.w}, x1[4] = {v1.x, v1.y, v1.z, v1.w};
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        mma16816(o[2 * u], code_pair<0>(x0[u]), code_pair<1>(x0[u]), code_pair<0>(x1[u]), code_pair<1>(x1[u]), b0, b1);
                        mma16816(o[2 * u + 1], code_pair<2>(x0[u]), code_pair<3>(x0[u]), code_pair<2>(x1[u]), code_pair<3>(x1[u]), b0,
                                 b1);
                    }
                }
            }
            __syncwarp();
            issue(np, ks);  // into the stages that these pages leave
        };
        int j = j0;
        for (; j + 2 <= j1; j += 2) pages(std::integral_constant<int, 2>(), j);
        if (j < j1) pages(std::integral_constant<int, 1>(), j);

        // sums over the tokens (lanes of equal c); the lane keeps dims [32 c + 4 r, + 4) of both heads
        float acc[GROUP][4], l_sum[GROUP], ref_of[GROUP];
        const float2 back = make_float2(1.f / up.x, 1.f / up.y);  // 0 where nothing was attended
#pragma unroll
        for (int i = 0; i < GROUP; ++i) {
            float ls = i == 0 ? l.x : l.y, cr = i == 0 ? corr.x : corr.y;
#pragma unroll
            for (int z = 4; z < 32; z <<= 1) {
                ls += __shfl_xor_sync(0xffffffffu, ls, z);
                cr += __shfl_xor_sync(0xffffffffu, cr, z);
            }
            l_sum[i] = ls;
            ref_of[i] = i == 0 ? ref.x : ref.y;
#pragma unroll
            for (int d = 0; d < 4; ++d) {
                const int k = (d & 1) * 2 + i, t = d >> 1;
                const float lo2 = c & 1 ? o[2 + t][k] : o[t][k], hi2 = c & 1 ? o[6 + t][k] : o[4 + t][k];
                acc[i][d] = fmaf((c & 2 ? hi2 : lo2) * (d & 1 ? 1048576.f : 16777216.f), i == 0 ? back.x : back.y, cr);
            }
        }
        if (j0 == 0 && j1 == p1 - p0) {
            write_out<GROUP>(a.out, hq, b, g, lane, acc, l_sum);
        } else {
            settle(b, acc, ref_of, l_sum);
        }
        x = p0 + j1;
        b = b_next;
        seq_len = len_next;
    }
}

}  // namespace

size_t kvq_decode_workspace_bytes(int batch, int n_q_heads, int n_kv_heads, int ctas) {
    return workspace_layout(batch, n_q_heads, ctas * kCtasPerSm * workers_of(n_kv_heads)).total;
}

cudaError_t launch_kvq_decode(const void *q, long long ldq, void *k_pages, void *v_pages, const int32_t *page_table,
                              const int32_t *seq_lens, int batch, void *out, const qa_attn_params &p, float scale,
                              int ctas, cudaStream_t stream, const KvqAppend *app) {
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
    a.early = (p.abi_version >= 2 && p.stable_metadata >= 1) ? 1 : 0;
    a.early_pools = (p.abi_version >= 2 && p.stable_metadata >= 2) ? 1 : 0;
    const int workers = ctas * kCtasPerSm * workers_of(p.n_kv_heads);
    a.group_from = workers_to_group(batch, workers, p.n_kv_heads);
    const WorkspaceLayout w = workspace_layout(batch, p.n_q_heads, workers);
    uint8_t *ws = static_cast<uint8_t *>(p.workspace);
    a.part_acc = reinterpret_cast<float *>(ws + w.acc);
    a.part_ml = reinterpret_cast<float *>(ws + w.ml);
    a.group_acc = reinterpret_cast<float *>(ws + w.group_acc);
    a.group_ml = reinterpret_cast<float *>(ws + w.group_ml);
    a.arrivals = reinterpret_cast<int *>(ws + w.arrivals);
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
    cfg.gridDim = dim3((unsigned)(ctas * kCtasPerSm));
    cfg.blockDim = dim3(kWarps * 32);
    cfg.dynamicSmemBytes = smem_layout(batch).total;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    auto kernel = app ? (group == 2 ? kvq_decode_kernel<2, true> : kvq_decode_kernel<1, true>)
                      : (group == 2 ? kvq_decode_kernel<2, false> : kvq_decode_kernel<1, false>);
    // the most of any batch, not this call's: another thread's call of another batch may set it before the launch
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMostSmem);
    if (e != cudaSuccess) return e;
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
