// Attention of packed rows over paged states on the tensor cores, for many
// rows a request (rows_attn.cu says what is computed and when it is taken).
//
// A job is 128 rows, 128 / group query rows with the heads of one KV head in
// turn, over its request's keys, 64 at a time.  Two CTAs an SM, a group of
// hkv CTAs a worker: the group's CTAs take the same key tiles of each KV head,
// so that whole token rows are asked of HBM at about the same time.
//
//   warp 4     producer: Q once a job, then K and V of each tile, page by
//              page (boxes of 16 tokens by 64 dims), two slots each
//   warp 5     issues S = Q K^T (M 128, N 64) into one of two buffers in TMEM
//              and O += P V (N 128), P from TMEM.  S of the next tile is
//              issued before P V of this one, so the tensor core has work
//              while the softmax has it
//   warps 0-3  softmax, a row a thread: the row's 64 scores in registers, the
//              lazy running max (log2 slack 8: O is rescaled only when it
//              moves), P written over its scores as two bf16 terms of 16
//              columns each for every 32 keys; then the epilogue
//
// Two terms of P make P V two products: 16 bits of each probability, as in
// the prefill kernels.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "rows_attn.cuh"
#include "tc.cuh"

namespace qa {
namespace {

__device__ unsigned int g_status;

constexpr int kPage = 16;
constexpr int kTile = 64;
constexpr int kThreads = 192;
constexpr float kSlack = 8.f;
constexpr uint32_t kHalf = kTile * 128;            // 64 dims of a tile's rows
constexpr uint32_t kSlot = 2 * kHalf;              // K or V of a tile
constexpr uint32_t kQ = 0;                         // two halves of 128 rows
constexpr uint32_t kK = kQ + 2 * tc::kSubTileBytes;
constexpr uint32_t kV = kK + 2 * kSlot;
constexpr uint32_t kBar = kV + 2 * kSlot;
enum : uint32_t { kQFull, kQEmpty, kKFull, kKEmpty = kKFull + 2, kVFull = kKEmpty + 2, kVEmpty = kVFull + 2,
                  kSFull = kVEmpty + 2, kPFull = kSFull + 2, kDone = kPFull + 2, kOFull, kOFree, kBars };
constexpr uint32_t kTmem = kBar + 8 * kBars, kAbort = kTmem + 4, kPrefix = kAbort + 4;
constexpr uint32_t kColO = 128;  // TMEM: S / P in [0, 64) and [64, 128), O in [128, 256)

// The tiles of one job that are the worker's: the walk of every role.
struct Walk {
    const RowsArgs &a;
    const int *prefix;
    int at, hi, b;
    int block, t0, t1;  // the segment: rows block, tiles [t0, t1) of `tiles`
    int tiles;
    Request r;
    __device__ Walk(const RowsArgs &args, const int *p, int lo, int end) : a(args), prefix(p), at(lo), hi(end), b(-1) {
        t0 = t1 = 0;
    }
    __device__ bool next() {
        at += t1 - t0;
        if (at >= hi) return false;
        if (b < 0) b = request_at(prefix, a.batch, at), load();
        else if (at >= prefix[b + 1]) {
            do ++b; while (prefix[b + 1] == prefix[b]);
            load();
        }
        const int x = at - prefix[b];
        block = x / tiles;
        t0 = x - block * tiles;
        t1 = min(tiles, t0 + hi - at);
        return true;
    }
    __device__ void load() {
        r = request_of(a, b, nullptr);
        tiles = (r.keys + kTile - 1) / kTile;
    }
};

// Waits that give up: one that runs out ends every later one that would block.
struct Waits {
    volatile int *abort;
    __device__ __forceinline__ void operator()(uint32_t bar, uint32_t parity) const {
        if (mbar_try_wait(bar, parity)) return;
        const unsigned long long t0 = globaltimer_ns();
        while (!mbar_try_wait(bar, parity)) {
            if (*abort) return;
            if (globaltimer_ns() - t0 > kWaitLimitNs) {
                atomicOr(&g_status, QA_DEVICE_TIMEOUT);
                *abort = 1;
                return;
            }
        }
    }
};

__device__ __forceinline__ bool any_of_rows(bool x) {  // the 128 threads that own rows
    uint32_t r;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.or.pred q, 1, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
                 : "=r"(r)
                 : "r"((uint32_t)x)
                 : "memory");
    return r != 0;
}

__device__ __forceinline__ void store32(float *dst, const float *v) {  // 32-byte aligned
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(dst), "r"(__float_as_uint(v[0])),
                 "r"(__float_as_uint(v[1])), "r"(__float_as_uint(v[2])), "r"(__float_as_uint(v[3])), "r"(__float_as_uint(v[4])),
                 "r"(__float_as_uint(v[5])), "r"(__float_as_uint(v[6])), "r"(__float_as_uint(v[7]))
                 : "memory");
}

// The rows that row i sees among the drafted ones (bit j: row j), by a warp
// for all 64 rows, two a lane: reach doubles every round.
__device__ __forceinline__ void ancestors(const RowsArgs &a, const Request &r, uint64_t (&seen)[2]) {
    constexpr unsigned kAll = 0xffffffffu;
    const int lane = threadIdx.x & 31;
    int up[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        const int i = lane + 32 * x;
        if (!a.parents) {
            seen[x] = ~0ull >> (63 - i);
            continue;
        }
        up[x] = i < r.rows ? parent_of(a, r.first, i, &g_status) : -1;
        seen[x] = 1ull << i;
    }
    if (!a.parents) return;
    for (int n = 0; n < 6; ++n) {
        uint64_t theirs[2];
        int next[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const uint64_t s0 = __shfl_sync(kAll, seen[0], up[x] & 31), s1 = __shfl_sync(kAll, seen[1], up[x] & 31);
            const int u0 = __shfl_sync(kAll, up[0], up[x] & 31), u1 = __shfl_sync(kAll, up[1], up[x] & 31);
            theirs[x] = up[x] < 32 ? s0 : s1, next[x] = up[x] < 32 ? u0 : u1;
        }
#pragma unroll
        for (int x = 0; x < 2; ++x)
            if (up[x] >= 0) seen[x] |= theirs[x], up[x] = next[x];
    }
}

__global__ void __launch_bounds__(kThreads, 2)
    rows_tiles_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                      const __grid_constant__ CUtensorMap tv, const __grid_constant__ RowsArgs a) {
    constexpr unsigned kAll = 0xffffffffu;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw), sb = (raw + 1023u) & ~1023u;
    uint8_t *smem = smem_raw + (sb - raw);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int head = blockIdx.x % a.hkv, worker = blockIdx.x / a.hkv;
    const int rows_a_block = 128 / a.group;
    int *prefix = reinterpret_cast<int *>(smem + kPrefix);
    const Waits wait{reinterpret_cast<volatile int *>(smem + kAbort)};
    const auto bar = [&](uint32_t i) { return sb + kBar + 8 * i; };
    const auto grid_wait = [] {
        asm volatile("griddepcontrol.wait;" ::: "memory");
        asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    };
    if (!a.early) grid_wait();
    if (warp == 0) {
        count_tiles<kTile>(a, prefix, rows_a_block, blockIdx.x == 0 ? &g_status : nullptr);
    } else if (warp == 4) {
        if (lane == 0) {
            for (uint32_t i = 0; i < kBars; ++i) {
                const bool rows = i == kOFree || i == kPFull || i == kPFull + 1;  // an arrival of each of four warps
                mbar_init(bar(i), rows ? 4 : 1);
            }
            *wait.abort = 0;
            fence_mbar_init();
            tc::prefetch_tmap(&tq);
            tc::prefetch_tmap(&tk);
            tc::prefetch_tmap(&tv);
        }
    } else if (warp == 5) {
        tc::tmem_alloc(sb + kTmem, 256);
    }
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(smem + kTmem);
    const int total = prefix[a.batch], per = (total + a.workers - 1) / a.workers;
    const int lo = (int)min(worker * (long long)per, (long long)total), hi = min(lo + per, total);
    if (a.early) grid_wait();
    if (head == 0) zero_rows(a, prefix, worker, threadIdx.x, kThreads);
    Walk w(a, prefix, lo, hi);

    if (warp == 4) {
        if (head == 0 && lane == 0) {
            Split s = {0, 0, 0, 0};
            if (lo < hi) {
                const int b = request_at(prefix, a.batch, hi - 1);
                const Request r = request_of(a, b, nullptr);
                const int tiles = (r.keys + kTile - 1) / kTile, block = (hi - 1 - prefix[b]) / tiles;
                const int p0 = prefix[b] + block * tiles, p1 = p0 + tiles;  // the job that holds the last tile
                if (p0 >= lo && p1 > hi) {
                    s.count = (p1 - 1) / per - worker + 1;
                    s.first_slot = 2 * worker + (p0 > lo);
                    s.out_row = r.first + block * rows_a_block;
                    s.rows = min(rows_a_block, r.rows - block * rows_a_block) * a.group;
                }
            }
            a.splits[worker] = s;
        }
        __syncwarp();
        // K of a tile goes out before V of the tile before it (which waits for an earlier P V)
        const int p = lane >> 1, sd = lane & 1;
        int n = 0, job = 0, id_before = -1;
        const auto load = [&](const CUtensorMap *map, uint32_t slots, uint32_t full, uint32_t empty, int i, int id) {
            const int slot = i & 1;
            wait(bar(empty + slot), ((i >> 1) & 1) ^ 1);
            const unsigned boxes = __ballot_sync(kAll, id >= 0);
            if (lane == 0) mbar_arrive_expect_tx(bar(full + slot), __popc(boxes) * kPage * 128);
            __syncwarp();
            if (id >= 0) tc::tma_load_3d(sb + slots + slot * kSlot + sd * kHalf + p * kPage * 128, map, sd * 64, id * kPage, head, bar(full + slot));
        };
        while (w.next()) {
            const int32_t *row = a.page_table + (size_t)w.b * a.max_pages;
            const int pages = (w.r.keys + kPage - 1) / kPage;
            if (n > 0) load(&tv, kV, kVFull, kVEmpty, n - 1, id_before);
            wait(bar(kQEmpty), (job & 1) ^ 1);
            if (lane == 0) {
                mbar_arrive_expect_tx(bar(kQFull), 2 * tc::kSubTileBytes);
                for (int i = 0; i < 2; ++i)
                    tc::tma_load_3d(sb + kQ + i * tc::kSubTileBytes, &tq, i * 64, head * a.group, w.r.first + w.block * rows_a_block, bar(kQFull));
            }
            __syncwarp();
            ++job;
            int ids = -1, chunk = -1;
            for (int t = w.t0; t < w.t1; ++t, ++n) {
                if (t >> 3 != chunk) {  // 32 page ids at a time
                    chunk = t >> 3;
                    ids = chunk * 32 + lane < pages ? row[chunk * 32 + lane] : -1;
                    const bool bad = chunk * 32 + lane < pages && (ids < 0 || ids >= a.num_pages);
                    if (bad) {
                        const int tile = chunk * 8 + (lane >> 2);
                        if (tile >= w.t0 && tile < w.t1) atomicOr(&g_status, QA_DEVICE_BAD_PAGE);
                        ids = -1;
                    }
                }
                int id = __shfl_sync(kAll, ids, (4 * t + (p & 3)) & 31);
                if (lane >= 8) id = -1;
                load(&tk, kK, kKFull, kKEmpty, n, id);
                if (t > w.t0) load(&tv, kV, kVFull, kVEmpty, n - 1, id_before);
                id_before = id;
            }
        }
        if (n > 0) load(&tv, kV, kVFull, kVEmpty, n - 1, id_before);
    } else if (warp == 5) {
        if (lane == 0) {
            constexpr uint32_t idesc_s = tc::idesc_bf16(128, kTile, false), idesc_o = tc::idesc_bf16(128, 128, true);
            int n = 0, job = 0;
            // S of tile i takes the buffer that P V of tile i - 2 has read.  Within a job that is the newest P V but one;
            // at a job's first tile P V of tile i - 1 is out already, and is waited for: a parity names two phases.
            const auto issue_s = [&](int i, bool first) {
                wait(bar(kKFull + (i & 1)), (i >> 1) & 1);
                if (i >= 2 || (first && i >= 1)) wait(bar(kDone), (first ? i + 1 : i) & 1);
                tc::fence_after();
                const uint32_t k = sb + kK + (i & 1) * kSlot;
#pragma unroll
                for (int kk = 0; kk < 8; ++kk)
                    tc::mma_bf16(tmem + (i & 1) * kTile, tc::sw128_desc(sb + kQ + (kk >> 2) * tc::kSubTileBytes + (kk & 3) * 32),
                                 tc::sw128_desc(k + (kk >> 2) * kHalf + (kk & 3) * 32), idesc_s, kk > 0);
                tc::mma_commit(bar(kSFull + (i & 1)));
                tc::mma_commit(bar(kKEmpty + (i & 1)));
            };
            while (w.next()) {
                wait(bar(kQFull), job & 1);
                issue_s(n, true);
                for (int t = w.t0; t < w.t1; ++t, ++n) {
                    if (t + 1 < w.t1) issue_s(n + 1, false);
                    else tc::mma_commit(bar(kQEmpty));
                    wait(bar(kPFull + (n & 1)), (n >> 1) & 1);
                    wait(bar(kVFull + (n & 1)), (n >> 1) & 1);
                    if (t == w.t0 && job > 0) wait(bar(kOFree), (job - 1) & 1);
                    tc::fence_after();
                    const uint32_t p = tmem + (n & 1) * kTile, v = sb + kV + (n & 1) * kSlot;
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) {
                        const uint32_t hi_p = p + (kk >> 1) * 32 + (kk & 1) * 8;
                        const uint64_t vdesc = tc::sw128_desc_mn(v + kk * 2048, kHalf);
                        tc::mma_bf16_ts(tmem + kColO, hi_p, vdesc, idesc_o, t > w.t0 || kk > 0);
                        tc::mma_bf16_ts(tmem + kColO, hi_p + 16, vdesc, idesc_o, 1u);
                    }
                    tc::mma_commit(bar(kVEmpty + (n & 1)));
                    tc::mma_commit(bar(kDone));
                }
                // the job's own barrier: a row's thread may be two P V ahead here, more than kDone's parity tells apart
                tc::mma_commit(bar(kOFull));
                ++job;
            }
        }
    } else {
        const int row = threadIdx.x;
        const uint32_t lanes = (uint32_t)(warp * 32) << 16, t_o = tmem + kColO + lanes;
        int n = 0, job = 0;
        while (w.next()) {
            const Request &r = w.r;
            const int32_t *table = a.page_table + (size_t)w.b * a.max_pages;
            const int pages = (r.keys + kPage - 1) / kPage;
            const bool drafted = a.tree && w.t1 * kTile > r.past;
            uint64_t seen = 0;
            if (drafted) {
                uint64_t all[2];
                ancestors(a, r, all);
                const int node = row / a.group;
                const uint64_t s0 = __shfl_sync(kAll, all[0], node & 31), s1 = __shfl_sync(kAll, all[1], node & 31);
                seen = node >= r.rows ? 0 : node < 32 ? s0 : s1;
            }
            const auto ids_ok = [&](int t) -> uint32_t {  // which of tile t's four pages can be read
                const int page = 4 * t + (lane & 3), id = t < w.t1 && page < pages ? table[page] : 0;
                return __ballot_sync(kAll, id >= 0 && id < a.num_pages) & 15u;
            };
            float m = -INFINITY, l = 0.f;
            bool odd = false;
            uint32_t next_ok = ids_ok(w.t0);
            for (int t = w.t0; t < w.t1; ++t, ++n) {
                const uint32_t ok = next_ok, s = tmem + (n & 1) * kTile + lanes;
                next_ok = ids_ok(t + 1);
                wait(bar(kSFull + (n & 1)), (n >> 1) & 1);
                __syncwarp();
                tc::fence_after();
                uint32_t sc[2][32];
                tc::tmem_ld32_issue(s, sc[0]);
                tc::tmem_ld32_issue(s + 32, sc[1]);
                tc::tmem_ld32_wait(sc[0]);
                tc::tmem_ld32_wait(sc[1]);
                const int behind = r.past - t * kTile;  // keys of this tile that every row sees
                const bool masked = behind < kTile || ok != 15u;
                if (masked) {
                    uint64_t vis = behind >= kTile ? ~0ull : behind > 0 ? ~(~0ull << behind) : 0ull;
                    if (behind < kTile && behind > -kTile) vis |= behind >= 0 ? seen << behind : seen >> -behind;
#pragma unroll
                    for (int p = 0; p < 4; ++p)
                        if (!(ok >> p & 1)) vis &= ~(0xffffull << 16 * p);
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const uint32_t v = (uint32_t)(vis >> 32 * c);
#pragma unroll
                        for (int j = 0; j < 32; ++j) sc[c][j] = v >> j & 1 ? sc[c][j] : __float_as_uint(-INFINITY);
                    }
                }
                float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int c = 0; c < 2; ++c)
#pragma unroll
                    for (int j = 0; j < 32; j += 2)
                        mx4[(j >> 1) & 3] = fmax3(mx4[(j >> 1) & 3], __uint_as_float(sc[c][j]), __uint_as_float(sc[c][j + 1]));
                const float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3])) * a.scale_log2;
                const float next = mx > m + kSlack ? mx : m;
                const float alpha = next == m ? 1.f : exp2_approx(m - next);
                m = next;
                const float ref = next == -INFINITY ? 0.f : next;
                if (t > w.t0 && __any_sync(kAll, alpha != 1.f)) {
                    wait(bar(kDone), (n - 1) & 1);  // P V of the tile before has written O
                    __syncwarp();
                    tc::fence_after();
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        float o[32];
                        tc::tmem_ld32(t_o + c * 32, o);
#pragma unroll
                        for (int j = 0; j < 32; ++j) o[j] *= alpha;
                        tc::tmem_st32(t_o + c * 32, o);
                    }
                }
                const float2 scale2 = make_float2(a.scale_log2, a.scale_log2), ref2 = make_float2(-ref, -ref);
                float2 sum[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    uint32_t ph[16], pl[16];
#pragma unroll
                    for (int j = 0; j < 32; j += 2) {
                        const float2 x = ffma2(make_float2(__uint_as_float(sc[c][j]), __uint_as_float(sc[c][j + 1])), scale2, ref2);
                        const float2 p = make_float2(exp2_approx(x.x), exp2_approx(x.y));
                        sum[(j >> 1) & 3] = fadd2(sum[(j >> 1) & 3], p);
                        const uint32_t b0 = __float_as_uint(p.x), b1 = __float_as_uint(p.y);
                        ph[j >> 1] = __byte_perm(b0, b1, 0x7632);
                        const float2 rest = fsub2(p, make_float2(__uint_as_float(b0 & 0xffff0000u), __uint_as_float(b1 & 0xffff0000u)));
                        pl[j >> 1] = pack_bf16x2(rest.x, rest.y);
                    }
                    tc::tmem_st16(s + c * 32, ph);
                    tc::tmem_st16(s + c * 32 + 16, pl);
                }
                const float2 both = fadd2(fadd2(sum[0], sum[1]), fadd2(sum[2], sum[3]));
                l = l * alpha + (both.x + both.y);
                if (masked) {
                    // Slots that hold no key (or were not loaded) are zeroed, and of drafted values what is not finite, so
                    // that a probability of 0 meets nothing that it would not cancel; rows that see such a value get it at
                    // the end.  Two threads a key.
                    wait(bar(kVFull + (n & 1)), (n >> 1) & 1);
                    const int key = row >> 1, pos = t * kTile + key;
                    uint8_t *v = smem + kV + (n & 1) * kSlot + (row & 1) * kHalf + key * 128;
                    const bool live = pos < r.keys && (ok >> (key >> 4) & 1);
                    if (!live || pos >= r.past) {
#pragma unroll
                        for (int c = 0; c < 8; ++c) {
                            uint4 *at = reinterpret_cast<uint4 *>(v) + c;
                            uint4 z = make_uint4(0u, 0u, 0u, 0u);
                            if (live) {
                                const uint4 x = *at;
                                z = make_uint4(finite_or_zero(x.x), finite_or_zero(x.y), finite_or_zero(x.z), finite_or_zero(x.w));
                                if (z.x == x.x && z.y == x.y && z.z == x.z && z.w == x.w) continue;
                                odd = true;
                            }
                            *at = z;
                        }
                    }
                    tc::fence_proxy_async_smem();
                    __syncwarp();
                }
                tc::tmem_wait_st();
                tc::fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(kPFull + (n & 1)));
            }
            const bool any_odd = drafted && any_of_rows(odd);
            wait(bar(kOFull), job & 1);
            ++job;
            __syncwarp();
            tc::fence_after();
            const bool whole = w.t0 == 0 && w.t1 == w.tiles;
            const int left = (r.rows - w.block * rows_a_block) * a.group;  // rows from this block's first on
            const int slot = 2 * worker + (w.at > lo);
            const size_t part = ((size_t)slot * a.hkv + head) * 128 + row;
            const float inv = l > 0.f ? 1.f / l : l;
            uint16_t *dst = a.out + ((size_t)(r.first + w.block * rows_a_block + row / a.group) * a.hq + head * a.group + row % a.group) * 128;
            const bool wide = (reinterpret_cast<uintptr_t>(a.out) & 31) == 0;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                float o[32];
                tc::tmem_ld32(t_o + c * 32, o);
                if (any_odd) {
                    for (int pos = max(r.past, w.t0 * kTile); pos < min(r.keys, w.t1 * kTile); ++pos) {
                        const int id = table[pos >> 4];
                        if (id < 0 || id >= a.num_pages || !(seen >> (pos - r.past) & 1)) continue;
                        const uint32_t *v = reinterpret_cast<const uint32_t *>(a.v_pages + (((size_t)id * kPage + (pos & 15)) * a.hkv + head) * 128 + c * 32);
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            const uint32_t x = not_finite(v[j]);
                            o[2 * j] += bf16lo(x), o[2 * j + 1] += bf16hi(x);
                        }
                    }
                }
                if (row < left) {
                    if (whole) {
                        uint32_t y[16];
#pragma unroll
                        for (int j = 0; j < 16; ++j) y[j] = pack_bf16x2(o[2 * j] * inv, o[2 * j + 1] * inv);
                        if (wide) {
                            store32(reinterpret_cast<float *>(dst + c * 32), reinterpret_cast<const float *>(y));
                            store32(reinterpret_cast<float *>(dst + c * 32 + 16), reinterpret_cast<const float *>(y + 8));
                        } else {
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                *reinterpret_cast<uint4 *>(dst + c * 32 + 8 * j) = make_uint4(y[4 * j], y[4 * j + 1], y[4 * j + 2], y[4 * j + 3]);
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < 4; ++j) store32(a.acc + part * 128 + c * 32 + 8 * j, o + 8 * j);
                    }
                }
                __syncwarp();
            }
            if (!whole && row < left) *reinterpret_cast<float2 *>(a.ml + 2 * part) = make_float2(m, l);
            tc::fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(kOFree));
        }
    }
    __syncthreads();
    if (warp == 5) {
        tc::fence_after();
        tc::tmem_dealloc(tmem, 256);
    }
}

}  // namespace

int rows_tiles_workers(int hkv) {
    int device = 0, sms = 0;
    if (cudaGetDevice(&device) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device) != cudaSuccess)
        return 0;
    return 2 * sms / hkv;
}

cudaError_t launch_rows_tiles(const RowsArgs &a, const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv,
                              cudaStream_t stream) {
    const uint32_t bytes = 1024 + kPrefix + 4 * (a.batch + 1);
    // the most of any call, so that host threads' calls cannot lower one another's
    cudaError_t e = cudaFuncSetAttribute(rows_tiles_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)(1024 + kPrefix + 4 * (kRowsMaxBatch + 1)));
    if (e != cudaSuccess) return e;
    e = cudaFuncSetAttribute(rows_tiles_kernel, cudaFuncAttributePreferredSharedMemoryCarveout, (int)cudaSharedmemCarveoutMaxShared);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.workers * a.hkv));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = bytes;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, rows_tiles_kernel, tq, tk, tv, a);
}

unsigned int status_read_clear_rows_tiles(cudaStream_t stream, cudaError_t *err) {
    unsigned int v = 0, zero = 0;
    cudaError_t e = cudaMemcpyFromSymbolAsync(&v, g_status, sizeof v, 0, cudaMemcpyDeviceToHost, stream);
    if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
    if (e == cudaSuccess && v) e = cudaMemcpyToSymbolAsync(g_status, &zero, sizeof zero, 0, cudaMemcpyHostToDevice, stream);
    if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
    if (err) *err = e;
    return v;
}

}  // namespace qa
