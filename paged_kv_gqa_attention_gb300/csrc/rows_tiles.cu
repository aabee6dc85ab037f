// Attention of packed rows over paged states on the tensor cores, for many
// rows a request (rows_attn.cu says what is computed and when it is taken).
//
// A job is 128 rows, 128 / group query rows with the heads of one KV head in
// turn, over its request's keys, 128 at a time.  One CTA an SM, a group of
// hkv CTAs a worker: the group's CTAs take the same key tiles of each KV head,
// so that whole token rows are asked of HBM at about the same time.
//
//   warp 16    producer: Q once a job (two buffers), K and V of each tile,
//              page by page, into one ring of five slots in the order they
//              are used.  A page's 16 tokens of a head are one box, of 8 keys
//              by 64 dims four times: as two boxes of 16 keys by 64 dims the
//              copies came at 25 bytes a clock (80 clocks a box), which was
//              what bounded
//   warp 17    issues S = Q K^T (M 128, N 128) into one of three buffers in
//              TMEM, up to two tiles ahead, into the next job too
//   warp 18    issues O += P V (N 128), P from TMEM; one thread for both
//              products was slower, 1.98 us a tile against 1.30
//   warp 19    the scout: a job ahead, whether any of its pages is bad, and
//              which drafted rows each row sees
//   warps 0-15 softmax, a row a thread: a warpgroup has 32 of each tile's keys.
//              32 scores in registers, a lazy running max (log2 slack 8: O is
//              rescaled only when it moves), P written over its scores as two
//              bf16 terms of 16 columns each.  A row's four parts share its
//              reference: a barrier a tile says whether any row's moves, and
//              only then do they exchange maxima.  So one O serves all, which
//              leaves TMEM for the third buffer of S
//
// Two terms of P make P V two products: 16 bits of each probability, as in
// the prefill kernels.
//
// What bounds.  One request of 4000 rows over 15600 states that stay in L2 (16
// heads on 8): 530 us, 1.3 us a tile, 1.43 PFLOP/s with both terms of P, 76 %
// of the measured peak.  The tensor core needs 514 clocks for S and 1028 for
// P V of a tile (measured: 64.2 an instruction; N = 64 would take 48), shared
// memory as many; P waits for the products, not they for it.  Not faster were
// two teams of softmax warps with two buffers of S and an O each (1.47 us a
// tile), two blocks of rows for each tile's K and V (1.38), pairs of workers on
// two blocks of a request, which halve what is read from HBM (8 requests of 448
// rows over 8000 states 313 us against 265; an odd block idles a worker).
// 24 requests of 33 to 64 rows over 500 to 8000 positions: 89 us, 5.2 TB/s,
// floor 68.6 us by their bytes.  32 requests of 9 to 16 rows over 200 to 2000:
// 36.7 us, floor 21.8: jobs are a few tiles long, and each costs 2 to 4 us
// beside them (the last tile waits for V, then O is given back); four parts or
// two of 64 keys there: 44.0 and 45.1 us before that.  8 requests of 100 to 448
// rows over 2000 to 15600 states: 224 us, where K and V are read again for each
// 64 rows, 1.33 GB at 6.4 TB/s.  (Calls repeated on one set of inputs; where
// these change from call to call 90.5, 37.4 and 231 us.)  Putting a job's end
// off until the next one's first P is there costs registers in the loop: 45.5
// us for the second of these calls, against 39.4 at the time.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "rows_attn.cuh"
#include "tc.cuh"

namespace qa {
namespace {

__device__ unsigned int g_status;

constexpr int kPage = 16;
constexpr int kTile = 128;
constexpr int kParts = 4;               // of a tile's keys, each a warpgroup's
constexpr int kKeys = kTile / kParts;   // of a thread
constexpr int kRows = kParts * 128;     // threads that own rows
constexpr int kProducer = kParts * 4, kIssueS = kProducer + 1, kIssueO = kIssueS + 1, kScout = kIssueO + 1;  // warps
constexpr int kThreads = (kScout + 1) * 32;
constexpr int kSlots = 5;
constexpr int kBufs = 3;
constexpr float kSlack = 8.f;
// The scout waits while its warps work through a whole job: this much longer
// for each of its tiles, 1.3 us when all is well.  (Every other wait is for a
// tile's time at most, and ends this one too if it runs out.)
constexpr unsigned long long kScoutTileNs = 20000;
constexpr uint32_t kQBytes = 2 * tc::kSubTileBytes;  // two halves of 64 dims of 128 rows; K and V of a tile too
constexpr uint32_t kAtom = 1024, kGroup = 2 * kAtom;    // of K and V: 8 keys' first 64 dims, then their others
constexpr uint32_t kRing = 2 * kQBytes;
constexpr uint32_t kBar = kRing + kSlots * kQBytes;
enum : uint32_t { kQFull, kQEmpty = kQFull + 2, kFull = kQEmpty + 2, kSFull = kFull + kSlots,
                  kPFull = kSFull + kBufs, kDone = kPFull + kBufs, kOFull = kDone + kBufs,
                  kInfoFull, kInfoFree, kDrained, kBars };
constexpr uint32_t kTmem = kBar + 8 * kBars, kAbort = kTmem + 4, kStart = kAbort + 4, kStats = kStart + 32;
// What the scout finds of a job.
struct Info {
    uint64_t seen[64];  // the drafted rows that a row sees (bit j: row j)
    int bad;            // a page of the job's tiles cannot be read
};
constexpr uint32_t kInfo = kStats + kParts * 128 * 4, kSmem = kInfo + sizeof(Info);  // kStats: [part][row]
static_assert(kSmem <= 227 * 1024, "shared memory");
constexpr uint32_t kColO = kBufs * kTile;  // TMEM: three buffers of S / P, then O

// The list of a call's places, of which every worker gets as many: a job's
// tiles, and kSwitch places before them for what a job costs beside its tiles.
// With 0, 1, 2, 3, 5 places: 64 requests of 32 rows over 550 positions 59.7,
// 55.8, 51.9, 51.2, 50.5 us; 32 of 9 to 16 over 200 to 2000 43.4, 40.5, 40.0,
// 39.5, 40.0; one of 4000 over 15600 531, 534, 538, 538, 537.
constexpr int kSwitch = 3;

// The places of a call, and the request of the worker's first one, by one warp.
struct Start {
    int total, b, base;   // base: the places before request b
    int first, end, past; // request b's numbers
    int per;              // places a worker
};
__device__ __forceinline__ int block_shift(const RowsArgs &a) { return 8 - a.group; }  // a block is 128 / group rows, group 1 or 2
__device__ __forceinline__ int places_of(int tiles, int rows, int shift) {
    return tiles == 0 ? 0 : (tiles + kSwitch) * ((rows + (1 << shift) - 1) >> shift);
}
__device__ __forceinline__ int places_of(const RowsArgs &a, const Request &r) {
    return places_of((r.keys + kTile - 1) / kTile, r.rows, block_shift(a));
}
__device__ __forceinline__ Start find_start(const RowsArgs &a, int worker, unsigned int *report) {
    constexpr unsigned kAll = 0xffffffffu;
    const int lane = threadIdx.x & 31;
    int sum = 0, first = 0;  // first: of the first 32 requests
    for (int b = lane; b < a.batch; b += 32) {
        const int v = places_of(a, request_of(a, b, report));
        if (b < 32) first = v;
        sum += v;
    }
    Start s = {__reduce_add_sync(kAll, sum), 0, 0, 0, 0, 0, 0};
    s.per = (s.total + a.workers - 1) / a.workers;
    const long long lo = (long long)worker * s.per;
    if (lo >= s.total) return s;
    for (int begin = 0, carry = 0; begin < a.batch; begin += 32) {
        const int b = begin + lane;
        const int v = begin == 0 ? first : b < a.batch ? places_of(a, request_of(a, b, nullptr)) : 0;
        int up_to = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(kAll, up_to, o);
            if (lane >= o) up_to += u;
        }
        const unsigned past = __ballot_sync(kAll, carry + up_to > lo);
        if (past) {
            const int l = __ffs(past) - 1;
            s.b = begin + l;
            s.base = carry + __shfl_sync(kAll, up_to - v, l);
            s.first = a.cu[s.b], s.end = a.cu[s.b + 1], s.past = a.past[s.b];
            return s;
        }
        carry += __shfl_sync(kAll, up_to, 31);
    }
    return s;
}

// The jobs of a worker, one after another: the walk of every role.
struct Walk {
    const RowsArgs &a;
    int at, hi, b, base;
    int block, t0, t1;  // the segment: rows block, tiles [t0, t1) of `tiles`
    int tiles;
    int first, end;     // the places of the job's tile 0, and behind the segment
    Request r;
    int first_next, end_next, past_next;  // of request b + 1
    __device__ Walk(const RowsArgs &args, const Start &s, int lo, int end)
        : a(args), at(lo), hi(end), b(s.b), base(s.base), end(lo) {
        if (lo >= end) return;
        first_next = s.first, end_next = s.end, past_next = s.past;
        load();
    }
    __device__ bool next() {
        do {
            at = end;
            if (at >= hi) return false;
            for (int n = mine(); at >= base + n; n = mine()) base += n, ++b, load();
            const int job = tiles + kSwitch, x = at - base;
            block = x < job ? 0 : x / job;
            first = base + block * job + kSwitch;
            end = min(first + tiles, hi);
            t0 = max(at - first, 0);
            t1 = end - first;
        } while (t0 >= t1);
        return true;
    }
    __device__ int mine() const { return places_of(tiles, r.rows, block_shift(a)); }
    __device__ void load() {  // the request whose numbers are here, and asks for the next one's
        r = request_of(a, first_next, end_next, past_next, nullptr);
        tiles = (r.keys + kTile - 1) / kTile;
        if (b + 1 < a.batch) first_next = end_next, end_next = a.cu[b + 2], past_next = a.past[b + 1];
    }
};

// The ring's pieces are, of each job, K 0, K 1, V 0, K 2, V 1, .., V of the
// last tile: the places of a tile's among the job's.
__device__ __forceinline__ int k_piece(int tile) { return tile == 0 ? 0 : 2 * tile - 1; }
__device__ __forceinline__ int v_piece(int tile, int tiles) { return tile + 1 < tiles ? 2 * tile + 2 : 2 * tile + 1; }

__device__ __forceinline__ bool any_of_rows(bool x) {  // the threads that own rows
    uint32_t r;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.or.pred q, 1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
                 : "=r"(r)
                 : "r"((uint32_t)x), "n"(kRows)
                 : "memory");
    return r != 0;
}

// One lane of a whole warp, in a form that lets the products' operands be
// kept in uniform registers.
__device__ __forceinline__ bool elected() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}
template <class T>
__device__ __forceinline__ T same_in_warp(T x) {
    return __shfl_sync(0xffffffffu, x, 0);
}

__device__ __forceinline__ void store32(float *dst, const float *v) {  // 32-byte aligned
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(dst), "r"(__float_as_uint(v[0])),
                 "r"(__float_as_uint(v[1])), "r"(__float_as_uint(v[2])), "r"(__float_as_uint(v[3])), "r"(__float_as_uint(v[4])),
                 "r"(__float_as_uint(v[5])), "r"(__float_as_uint(v[6])), "r"(__float_as_uint(v[7]))
                 : "memory");
}

// The rows that row i sees among the drafted ones (bit j: row j), by a warp
// for all 64 rows, two a lane: reach doubles every round.
__device__ __forceinline__ void ancestors(const RowsArgs &a, int (&up)[2], uint64_t (&seen)[2]) {
    constexpr unsigned kAll = 0xffffffffu;
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int x = 0; x < 2; ++x) seen[x] = a.parents ? 1ull << (lane + 32 * x) : ~0ull >> (63 - lane - 32 * x);
    if (!a.parents) return;
    while (__any_sync(kAll, up[0] >= 0 || up[1] >= 0)) {
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

__global__ void __launch_bounds__(kThreads, 1)
    rows_tiles_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                      const __grid_constant__ CUtensorMap tv, const __grid_constant__ RowsArgs a) {
    constexpr unsigned kAll = 0xffffffffu;
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t sb = smem_u32(smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int head = blockIdx.x % a.hkv, worker = blockIdx.x / a.hkv;
    const int rows_a_block = 1 << block_shift(a), by = a.group - 1;  // a tile's row i is query row i >> by, head i & by
    const Waits wait{reinterpret_cast<volatile int *>(smem + kAbort), &g_status, kWaitLimitNs};
    const auto bar = [&](uint32_t i) { return sb + kBar + 8 * i; };
    const auto grid_wait = [] {
        asm volatile("griddepcontrol.wait;" ::: "memory");
        asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    };
    if (warp == kProducer && lane == 0) {
        tc::prefetch_tmap(&tq);
        tc::prefetch_tmap(&tk);
        tc::prefetch_tmap(&tv);
    }
    if (!a.early) grid_wait();
    if (warp == 0) {
        const Start s = find_start(a, worker, blockIdx.x == 0 ? &g_status : nullptr);
        if (lane == 0) *reinterpret_cast<Start *>(smem + kStart) = s;
    } else if (warp == kProducer && lane == 0) {
        for (uint32_t i = 0; i < kBars; ++i)
            mbar_init(bar(i), (i >= kPFull && i < kPFull + kBufs) || i == kInfoFree ? kParts * 4 : i == kDrained ? 2 : 1);
        *wait.abort = 0;
        fence_mbar_init();
    }
    // TMEM only once the kernel before has ended: one that starts its successors before it allocates could wait for
    // columns that this one holds while it waits for that kernel
    if (a.early) grid_wait();
    if (warp == kIssueS) tc::tmem_alloc(sb + kTmem, 512);
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(smem + kTmem);
    const Start start = *reinterpret_cast<const Start *>(smem + kStart);
    const int total = start.total, per = start.per;
    const int lo = (int)min(worker * (long long)per, (long long)total), hi = min(lo + per, total);
    if (head == 0)
        for (int b = worker; b < a.batch; b += a.workers) zero_rows(a, request_of(a, b, nullptr), threadIdx.x, kThreads);
    Walk w(a, start, lo, hi);
    int pieces = 0, jobs = 0;  // whose copies the producer has asked for

    if (warp == kProducer) {
        const int p = lane & 7;
        int slot = 0, job = 0, tile = 0;
        int ends[kSlots];  // of the last pieces, newest first: the barrier that says that its slot is free, and its parity
#pragma unroll
        for (int i = 0; i < kSlots; ++i) ends[i] = -1;
        Split split = {0, 0, 0, 0};
        const auto load = [&](const CUtensorMap *map, int id, uint32_t end, int of) {
            if (ends[kSlots - 1] >= 0) wait(bar(ends[kSlots - 1] >> 1), ends[kSlots - 1] & 1);
#pragma unroll
            for (int i = kSlots - 1; i > 0; --i) ends[i] = ends[i - 1];
            ends[0] = 2 * (end + of % kBufs) + (of / kBufs & 1);
            if (__any_sync(kAll, *wait.abort)) return;  // the slot may still be read
            ++pieces;
            const unsigned boxes = __ballot_sync(kAll, id >= 0);
            if (lane == 0) mbar_arrive_expect_tx(bar(kFull + slot), __popc(boxes) * 2 * kGroup);
            __syncwarp();
            if (id >= 0) tc::tma_load_5d(sb + kRing + slot * kQBytes + p * 2 * kGroup, map, 0, 0, 0, 2 * id, head, bar(kFull + slot));
            if (++slot == kSlots) slot = 0;
        };
        // a job's numbers; the next job's are taken, and its first page ids asked for, before this one's copies go out
        struct Job {
            const int32_t *row;
            int pages, t0, t1, q_row;
        };
        const auto page_ids = [&](const Job &j, int chunk) { return chunk * 32 + lane < j.pages ? j.row[chunk * 32 + lane] : -1; };
        Job next = {};
        int next_ids = -1;
        const auto take = [&] {
            if (!w.next()) return false;
            next = {a.page_table + (size_t)w.b * a.max_pages, (w.r.keys + kPage - 1) / kPage, w.t0, w.t1, w.r.first + w.block * rows_a_block};
            next_ids = page_ids(next, w.t0 >> 2);
            const int last = w.first + w.tiles - 1;  // the place of the job's last tile
            if (w.t0 == 0 && last >= hi) {
                split.count = last / per - worker + 1;
                split.first_slot = 2 * worker + (w.at > lo);
                split.out_row = next.q_row;
                split.rows = min(rows_a_block, w.r.rows - w.block * rows_a_block) * a.group;
            }
            return true;
        };
        for (bool more = take(); more; ++job) {
            const Job j = next;
            int ids = -1, ids_next = next_ids, id_before = -1;
            more = take();
            wait(bar(kQEmpty + (job & 1)), ((job >> 1) & 1) ^ 1);
            if (__any_sync(kAll, *wait.abort)) break;
            ++jobs;
            if (lane == 0) {
                mbar_arrive_expect_tx(bar(kQFull + (job & 1)), kQBytes);
                for (int i = 0; i < 2; ++i)
                    tc::tma_load_3d(sb + (job & 1) * kQBytes + i * tc::kSubTileBytes, &tq, i * 64, head * a.group, j.q_row,
                                    bar(kQFull + (job & 1)));
            }
            __syncwarp();
            for (int t = j.t0; t < j.t1; ++t) {
                if (t == j.t0 || (t & 3) == 0) {  // 32 page ids at a time, the next ones on their way
                    const int chunk = t >> 2;
                    ids = ids_next;
                    ids_next = page_ids(j, chunk + 1);
                    if (chunk * 32 + lane < j.pages && (ids < 0 || ids >= a.num_pages)) {
                        const int tile = chunk * 4 + (lane >> 3);
                        if (tile >= j.t0 && tile < j.t1) atomicOr(&g_status, QA_DEVICE_BAD_PAGE);
                        ids = -1;
                    }
                }
                int id = __shfl_sync(kAll, ids, (8 * t + p) & 31);
                if (lane >= 8) id = -1;
                load(&tk, id, kSFull, tile);
                if (t > j.t0) load(&tv, id_before, kDone, tile - 1);
                id_before = id;
                ++tile;
            }
            load(&tv, id_before, kDone, tile - 1);
        }
        if (head == 0 && lane == 0) a.splits[worker] = split;
    } else if (warp == kIssueS) {
        constexpr uint32_t idesc_s = tc::idesc_bf16(128, kTile, false);
        int n = 0, job = 0, buf = 0, phase = 0;
        while (w.next()) {
            const uint32_t q = sb + (job & 1) * kQBytes;
            wait(bar(kQFull + (job & 1)), (job >> 1) & 1);
            for (int t = w.t0; t < w.t1; ++t, ++n) {
                const int piece = 2 * (n - (t - w.t0)) + k_piece(t - w.t0), slot = piece % kSlots;
                wait(bar(kFull + slot), piece / kSlots & 1);
                if (n >= kBufs) wait(bar(kDone + buf), phase ^ 1);  // P V of tile n - 3 has read this buffer
                __syncwarp();
                tc::fence_after();
                const uint64_t qd = same_in_warp(tc::sw128_desc(q)), kd = same_in_warp(tc::sw128_desc(sb + kRing + slot * kQBytes, kGroup, 0));
                const uint32_t d = same_in_warp(tmem + buf * kTile);
                if (elected()) {
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk)
                        tc::mma_bf16(d, qd + ((kk >> 2) * tc::kSubTileBytes + (kk & 3) * 32) / 16, kd + ((kk >> 2) * kAtom + (kk & 3) * 32) / 16, idesc_s, kk > 0);
                    tc::mma_commit(bar(kSFull + buf));
                    if (t + 1 == w.t1) tc::mma_commit(bar(kQEmpty + (job & 1)));
                }
                __syncwarp();
                if (++buf == kBufs) buf = 0, phase ^= 1;
            }
            ++job;
        }
    } else if (warp == kIssueO) {
        constexpr uint32_t idesc_o = tc::idesc_bf16(128, 128, true);
        int n = 0, buf = 0, phase = 0;
        while (w.next()) {
            for (int t = w.t0; t < w.t1; ++t, ++n) {
                const int piece = 2 * (n - (t - w.t0)) + v_piece(t - w.t0, w.t1 - w.t0), slot = piece % kSlots;
                wait(bar(kFull + slot), piece / kSlots & 1);
                wait(bar(kPFull + buf), phase);
                __syncwarp();
                tc::fence_after();
                const uint64_t vd = same_in_warp(tc::sw128_desc(sb + kRing + slot * kQBytes, kGroup, kAtom));
                const uint32_t p = same_in_warp(tmem + buf * kTile), o = same_in_warp(tmem + kColO);
                if (elected()) {
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk) {
                        const uint32_t hi_p = p + (kk >> 1) * 32 + (kk & 1) * 8;
                        tc::mma_bf16_ts(o, hi_p, vd + kk * 2 * kGroup / 16, idesc_o, t > w.t0 || kk > 0);
                        tc::mma_bf16_ts(o, hi_p + 16, vd + kk * 2 * kGroup / 16, idesc_o, 1u);
                    }
                    tc::mma_commit(bar(kDone + buf));
                    if (t + 1 == w.t1) tc::mma_commit(bar(kOFull));
                }
                __syncwarp();
                if (++buf == kBufs) buf = 0, phase ^= 1;
            }
        }
    } else if (warp == kScout) {
        Info &info = *reinterpret_cast<Info *>(smem + kInfo);
        unsigned tiles_before = 0, tiles_last = 0;  // of the job before the last one, which the warps are at, and of the last
        for (int job = 0; w.next(); ++job) {
            const int32_t *table = a.page_table + (size_t)w.b * a.max_pages;
            const int end = min(w.t1 * (kTile / kPage), (w.r.keys + kPage - 1) / kPage);
            bool bad = false;
            for (int j = w.t0 * (kTile / kPage) + lane; j < end; j += 8 * 32) {
                int id[8];
#pragma unroll
                for (int x = 0; x < 8; ++x) id[x] = j + 32 * x < end ? table[j + 32 * x] : 0;
#pragma unroll
                for (int x = 0; x < 8; ++x) bad |= id[x] < 0 || id[x] >= a.num_pages;
            }
            bad = __any_sync(kAll, bad);
            uint64_t seen[2] = {0, 0};
            if (a.tree && w.t1 * kTile > w.r.past) {
                int up[2];
#pragma unroll
                for (int y = 0; y < 2; ++y) up[y] = lane + 32 * y < w.r.rows ? parent_of(a, w.r.first, lane + 32 * y, &g_status) : -1;
                ancestors(a, up, seen);
            }
            wait(bar(kInfoFree), (job & 1) ^ 1, tiles_before * kScoutTileNs);
            tiles_before = tiles_last, tiles_last = w.t1 - w.t0;
            info.seen[lane] = seen[0], info.seen[lane + 32] = seen[1];
            if (lane == 0) info.bad = bad;
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(kInfoFull));
        }
    } else {
        const int h = warp >> 2, row = threadIdx.x & 127;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21, t_o = tmem + kColO + h * kKeys + lanes;  // of O, the part's share of the dims
        float *stats = reinterpret_cast<float *>(smem + kStats) + row;  // [part][row]
        int n = 0, job = 0, buf = 0, phase = 0;
        for (bool more = w.next(); more; ++job) {
            const Request r = w.r;
            const int t0 = w.t0, t1 = w.t1;
            const int32_t *table = a.page_table + (size_t)w.b * a.max_pages;
            const bool drafted = a.tree && t1 * kTile > r.past;
            const Info &info = *reinterpret_cast<const Info *>(smem + kInfo);
            wait(bar(kInfoFull), job & 1);
            const bool holes = info.bad;  // then each tile looks which of its pages are there
            const uint64_t seen = drafted && (row >> by) < r.rows ? info.seen[row >> by] : 0;
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(kInfoFree));
            constexpr int kPages = kKeys / kPage;
            const auto pages_of = [&](int t) -> uint32_t {  // which of the part's pages can be read
                const int page = 8 * t + kPages * h + lane % kPages, id = page * kPage < r.keys ? table[page] : 0;
                return __ballot_sync(kAll, id >= 0 && id < a.num_pages) & ((1u << kPages) - 1);
            };
            float m = -INFINITY, l = 0.f;
            bool odd = false, agreed = false;
            for (int t = t0; t < t1; ++t, ++n) {
                const uint32_t ok = holes ? pages_of(t) : (1u << kPages) - 1;
                const uint32_t s = tmem + buf * kTile + h * kKeys + lanes;
                wait(bar(kSFull + buf), phase);
                __syncwarp();
                tc::fence_after();
                uint32_t sc[kKeys / 32][32];
#pragma unroll
                for (int c = 0; c < kKeys / 32; ++c) tc::tmem_ld32_issue(s + 32 * c, sc[c]);
#pragma unroll
                for (int c = 0; c < kKeys / 32; ++c) tc::tmem_ld32_wait(sc[c]);
                const int key0 = t * kTile + h * kKeys, behind = r.past - key0;  // keys of this part that every row sees
                const bool masked = behind < kKeys || ok != (1u << kPages) - 1;
                if (masked) {
                    uint64_t vis = behind >= 64 ? ~0ull : behind > 0 ? ~(~0ull << behind) : 0ull;
                    if (behind < 64 && behind > -64) vis |= behind >= 0 ? seen << behind : seen >> -behind;
#pragma unroll
                    for (int p = 0; p < kPages; ++p)
                        if (!(ok >> p & 1)) vis &= ~(0xffffull << 16 * p);
#pragma unroll
                    for (int c = 0; c < kKeys / 32; ++c) {
                        const uint32_t v = (uint32_t)(vis >> 32 * c);
#pragma unroll
                        for (int j = 0; j < 32; ++j) sc[c][j] = v >> j & 1 ? sc[c][j] : __float_as_uint(-INFINITY);
                    }
                }
                float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int c = 0; c < kKeys / 32; ++c)
#pragma unroll
                    for (int j = 0; j < 32; j += 2)
                        mx4[(j >> 1) & 3] = fmax3(mx4[(j >> 1) & 3], __uint_as_float(sc[c][j]), __uint_as_float(sc[c][j + 1]));
                const float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3])) * a.scale_log2;
                // one reference a row, for all parts: where a row's moves, they agree on the largest maximum
                float alpha = 1.f;
                agreed = any_of_rows(mx > m + kSlack);
                if (agreed) {
                    stats[h * 128] = mx;
                    named_barrier(1, kRows);
                    float top = stats[0];
#pragma unroll
                    for (int x = 1; x < kParts; ++x) top = fmaxf(top, stats[x * 128]);
                    const float next = top > m + kSlack ? top : m;
                    alpha = next == m ? 1.f : exp2_approx(m - next);
                    m = next;
                    if (t > t0 && __any_sync(kAll, alpha != 1.f)) {
                        // P V of the tile before has written O, of which each part scales its share of the dims
                        wait(bar(kDone + (buf == 0 ? kBufs - 1 : buf - 1)), buf == 0 ? phase ^ 1 : phase);
                        __syncwarp();
                        tc::fence_after();
#pragma unroll
                        for (int c = 0; c < kKeys / 32; ++c) {
                            float o[32];
                            tc::tmem_ld32(t_o + c * 32, o);
#pragma unroll
                            for (int j = 0; j < 32; ++j) o[j] *= alpha;
                            tc::tmem_st32(t_o + c * 32, o);
                        }
                    }
                }
                const float ref = m == -INFINITY ? 0.f : m;
                const float2 scale2 = make_float2(a.scale_log2, a.scale_log2), ref2 = make_float2(-ref, -ref);
                float2 sum[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                for (int c = 0; c < kKeys / 16; ++c) {
                    uint32_t ph[8], pl[8];
#pragma unroll
                    for (int jj = 0; jj < 16; jj += 2) {
                        const int j = (c & 1) * 16 + jj;
                        const float2 x = ffma2(make_float2(__uint_as_float(sc[c / 2][j]), __uint_as_float(sc[c / 2][j + 1])), scale2, ref2);
                        const float2 p = make_float2(exp2_approx(x.x), exp2_approx(x.y));
                        sum[(j >> 1) & 3] = fadd2(sum[(j >> 1) & 3], p);
                        const uint32_t b0 = __float_as_uint(p.x), b1 = __float_as_uint(p.y);
                        ph[jj >> 1] = __byte_perm(b0, b1, 0x7632);
                        const float2 rest = fsub2(p, make_float2(__uint_as_float(b0 & 0xffff0000u), __uint_as_float(b1 & 0xffff0000u)));
                        pl[jj >> 1] = pack_bf16x2(rest.x, rest.y);
                    }
                    tc::tmem_st8(s + (c >> 1) * 32 + (c & 1) * 8, ph);
                    tc::tmem_st8(s + (c >> 1) * 32 + 16 + (c & 1) * 8, pl);
                }
                const float2 both = fadd2(fadd2(sum[0], sum[1]), fadd2(sum[2], sum[3]));
                l = l * alpha + (both.x + both.y);
                if (masked) {
                    // Slots that hold no key (or were not loaded) are zeroed, and of drafted values what is not finite, so
                    // that a probability of 0 meets nothing that it would not cancel; rows that see such a value get it at
                    // the end.
                    const int piece = 2 * (n - (t - t0)) + v_piece(t - t0, t1 - t0), v_slot = piece % kSlots;
                    wait(bar(kFull + v_slot), piece / kSlots & 1);
                    constexpr int kEach = 128 / kKeys, kChunks = 16 / kEach;  // threads of a key, 16-byte pieces of a thread
                    const int key = row / kEach, piece0 = row % kEach * kChunks, pos = key0 + key;
                    uint8_t *v = smem + kRing + v_slot * kQBytes + (kKeys / 8 * h + (key >> 3)) * kGroup + (piece0 >> 3) * kAtom + (key & 7) * 128;
                    const bool live = pos < r.keys && (ok >> (key >> 4) & 1);
                    if (!live || pos >= r.past) {
#pragma unroll
                        for (int c = 0; c < kChunks; ++c) {  // keys begin at pieces of their own: fewer bank conflicts
                            uint4 *at = reinterpret_cast<uint4 *>(v) + (piece0 & 7) + (c + key) % kChunks;
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
                if (lane == 0) mbar_arrive(bar(kPFull + buf));
                if (++buf == kBufs) buf = 0, phase ^= 1;
            }
            if (agreed) named_barrier(1, kRows);  // the last tile's maxima have been read
            stats[h * 128] = l;
            const bool any_odd = any_of_rows(odd);  // all parts' sums are there too
            float sum = 0.f;
#pragma unroll
            for (int x = 0; x < kParts; ++x) sum += stats[x * 128];
            // each part's warps give their share of the dims
            const bool whole = t0 == 0 && t1 == w.tiles;
            const int left = (r.rows - w.block * rows_a_block) * a.group;  // rows from this block's first on
            const int q_row = r.first + w.block * rows_a_block, slot = 2 * worker + (w.at > lo);
            more = w.next();  // while the last P V runs
            wait(bar(kOFull), job & 1);
            __syncwarp();
            tc::fence_after();
            const size_t part = ((size_t)slot * a.hkv + head) * 128 + row;
            const float inv = !whole ? 1.f : sum > 0.f ? 1.f / sum : sum;
            uint16_t *dst = a.out + ((size_t)(q_row + (row >> by)) * a.hq + head * a.group + (row & by)) * 128;
            const bool wide = (reinterpret_cast<uintptr_t>(a.out) & 31) == 0;
#pragma unroll
            for (int c = 0; c < kKeys / 32; ++c) {
                const int dim = h * kKeys + c * 32;
                float o[32];
                tc::tmem_ld32(t_o + c * 32, o);
#pragma unroll
                for (int j = 0; j < 32; ++j) o[j] *= inv;
                if (any_odd) {
                    for (int pos = max(r.past, t0 * kTile); pos < min(r.keys, t1 * kTile); ++pos) {
                        const int id = table[pos >> 4];
                        if (id < 0 || id >= a.num_pages || !(seen >> (pos - r.past) & 1)) continue;
                        const uint32_t *v = reinterpret_cast<const uint32_t *>(a.v_pages + (((size_t)id * kPage + (pos & 15)) * a.hkv + head) * 128 + dim);
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
                        for (int j = 0; j < 16; ++j) y[j] = pack_bf16x2(o[2 * j], o[2 * j + 1]);
                        if (wide) {
                            store32(reinterpret_cast<float *>(dst + dim), reinterpret_cast<const float *>(y));
                            store32(reinterpret_cast<float *>(dst + dim + 16), reinterpret_cast<const float *>(y + 8));
                        } else {
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                *reinterpret_cast<uint4 *>(dst + dim + 8 * j) = make_uint4(y[4 * j], y[4 * j + 1], y[4 * j + 2], y[4 * j + 3]);
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < 4; ++j) store32(a.acc + part * 128 + dim + 8 * j, o + 8 * j);
                    }
                }
                __syncwarp();
            }
            if (!whole && h == 0 && row < left) *reinterpret_cast<float2 *>(a.ml + 2 * part) = make_float2(m, sum);
            tc::fence_before();  // before the next job's P is handed over
        }
    }
    __syncthreads();
    if (*wait.abort) {  // a wait ran out: what is still under way writes shared memory and TMEM
        if (warp == kProducer && lane == 0) {
            for (int i = max(0, pieces - kSlots); i < pieces; ++i) mbar_wait(bar(kFull + i % kSlots), i / kSlots & 1, &g_status);
            for (int i = max(0, jobs - 2); i < jobs; ++i) mbar_wait(bar(kQFull + (i & 1)), i >> 1 & 1, &g_status);
        } else if ((warp == kIssueS || warp == kIssueO) && elected()) {
            tc::mma_commit(bar(kDrained));
            mbar_wait(bar(kDrained), 0, &g_status);
        }
        __syncthreads();
    }
    if (warp == kIssueS) {
        tc::fence_after();
        tc::tmem_dealloc(tmem, 512);
    }
}

}  // namespace

int rows_tiles_workers(int hkv) {
    int device = 0, sms = 0;
    if (cudaGetDevice(&device) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device) != cudaSuccess)
        return 0;
    return sms / hkv;
}

cudaError_t launch_rows_tiles(const RowsArgs &a, const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv,
                              cudaStream_t stream) {
    cudaError_t e = cudaFuncSetAttribute(rows_tiles_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.workers * a.hkv));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmem;
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
