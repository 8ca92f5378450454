// paged_attention_prefill_weights: the softmax weights that a chunk's queries, or its
// last `window` ones, give to each of the row's tokens, added to the tokens' running
// sums, on the 5th-generation tensor cores (tcgen05, scores in tensor memory).
//
// Mathematics.  For one KV head, flat row f of a row's used queries is query f / group and head
// f % group of the group.  With s[f][t] the base-2 scores, a token t gets
//   sum over f that see it of 2^(s[f][t] - e[f]),   e[f] = log2 sum_t 2^s[f][t],
// and e[f] is known only after f's last token: the scores are computed twice, each time
// in the orientation in which the sum runs along a thread's registers.
//   1. S = Q K^T, a flat row a thread: its reference maximum and its sum;
//   2. e, from the pieces that a row's keys were cut into;
//   3. S^T = K Q^T, a token a thread: the sum over the flat rows;
//   4. the tokens' pieces added to the running sums.
//
// Work of 1 and 3.  A job is a 128 x 128 product of one query block, as many whole queries of
// a group as 128 rows hold, and one tile of 128 tokens, some of which the block sees.  A
// unit is a query block (1) or a token tile (3) of one row and KV head and walks the jobs
// that it takes part in; all jobs of all units in order are cut into one contiguous
// range per block, one block an SM.  A unit inside one range is done by one block; the others
// leave pieces, which are brought together in order.
//
// Warp roles (each walks the same jobs):
//   warps 0-15  sums, in four groups of four that take every fourth job, each from a buffer
//               of 128 columns of its own: a row of the product a thread, 32 scores at a time;
//   warp 16     copies: the unit's fixed tile (two buffers), the others through a ring of
//               four (three), by TMA; K as one box of 16 to 128 tokens of a page each, its pool
//               rows found through the block table;
//   warp 17     products: one thread issues eight tcgen05.mma a job;
//   warps 18-21 (E4M3 pools) widen K's codes, exactly, into the operand tiles.
// The copying and the issuing warp run alone, so what an instruction of theirs takes, some five
// clocks, is in every job: their loops keep slots and parities as running values and find
// pool rows a batch at a time (with divisions and a look-up a job: 0.72 us a job).
//
// What bounds it.  Four rows of 3900 to 4096, every query (12 heads over 2): 240 us, 117 a pass
// for 165 jobs an SM, 0.71 us or 1,180 clocks a job.  No unit is full: 16,384 exponentials take the
// special-function unit 512 clocks (32 a clock, measured; 40 to 42% busy), the products the tensor pipe 490
// (41 to 43%), L2 gives 28% of its rate and 48 to 52% of the issue slots are used.  What is left are the roles'
// chains: without the sums both passes take 183 us, 0.55 a job for copies, barriers and products, and a
// group's wait, loads from tensor memory and sums do not hide behind them fully.
// Eight chunks of 512 over 300 to 2100 (32 heads over 8): 123 us.  The last 32 queries of 16 rows of 600
// to 4500, E4M3: 35 us, of which 9 are four launches with nothing to do, 13 the eight or nine
// jobs an SM of each pass, and the rest each pass's first copy, product and sum and its
// end, which nothing hides.
//
// Every wait is bounded: a block that gives up flags the error, tells its other warps to stop,
// and lets its copies and products in flight finish before it frees tensor memory.
//
// What is not seen (later tokens, table entries out of range) is left out of sums and maxima by
// selection, whatever its scores are, and so are in 3 the rows behind a query block's queries (1 gives
// them sums that nothing uses).
#include <limits.h>
#include <math.h>

#include <atomic>

#include "fp8_codec.cuh"
#include "pkv_internal.cuh"
#include "tcgen05.cuh"

namespace pkv {
namespace prompt {
using namespace tc;

constexpr int kTile = 128;
constexpr int kGroups = 4, kSumWarps = 4 * kGroups;
constexpr int kCopyWarp = kSumWarps, kMmaWarp = kSumWarps + 1, kConvWarp = kSumWarps + 2, kConvWarps = 4;
constexpr int kFixed = 2;   // a unit's fixed tiles
constexpr int kRaw = 2;     // tiles of codes
constexpr int kBufs = kGroups;  // products in tensor memory, a group's each
constexpr int kComb = 2;    // units whose sums the groups bring together
constexpr int kAhead = 12;  // jobs whose -e are kept: see the assertion
constexpr int kMaxRows = 1024;
constexpr uint32_t kHalf = kTile * 128;      // 128 rows x 64 dims
constexpr uint32_t kOperand = 2 * kHalf;
constexpr uint32_t kCodes = kTile * 128;     // 128 tokens of codes
constexpr uint32_t kTmemCols = 512;
constexpr int kCertain = 112;                // columns that are not asked whether a query has them
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kMove = 16.f;                // a score this far above the reference moves it

template <bool kFp8>
__host__ __device__ constexpr int threads() { return (kConvWarp + (kFp8 ? kConvWarps : 0)) * 32; }

struct Params {
    float* weights;
    const float* k_scale;
    const int32_t* tables;
    const int32_t* seq_lens;
    const int32_t* q_start;
    int64_t stride;
    int rows, total, hk, group, bs, mbpr, nb, limit, window;
    int nq;            // queries of a block
    int kbox;          // tokens of a copy of K
    int grid;
    int most_units;    // query blocks that the workspace has room for
    float scale_log2;
    // workspace
    int* head;         // [0]: query blocks, [1]: 1, or 0 where nothing may be done
    int* tile_pre;     // [rows + 1]: token tiles of the rows before
    int2* block_info;  // [query block]: first block that has a piece of it, pieces
    int2* tile_info;   // [token tile]
    float2* ml;        // [block + query block][128]: maxima and sums of the pieces
    float* neg_lse;    // [query block][128]: -e
    float* sums;       // [block + token tile][128]
    int32_t* dev_err;
    int last[4];       // (kHook) jobs of a block that copies, products, widening and sums do before they give up
};

// The block whose range of the W jobs holds job j (block c's starts at c W / n).
__device__ __forceinline__ int owner_of(int j, int W, int n) { return (int)((((int64_t)j + 1) * n - 1) / W); }

// Rows as the walk needs them, in shared memory.
struct Rows {
    const int *len, *used, *end;  // tokens, queries that count, the index behind the last query
    const int* units;             // units of the rows before
    const int* blocks;            // query blocks of the rows before
    int nq;
    __device__ __forceinline__ int query_blocks(int r) const { return (used[r] + nq - 1) / nq; }
    __device__ __forceinline__ int tiles(int r) const { return used[r] ? (len[r] + kTile - 1) / kTile : 0; }
    // Token tiles that query block m sees; the first query block that sees tile k.
    __device__ __forceinline__ int seen(int r, int m) const {
        return (len[r] - used[r] + min(used[r], (m + 1) * nq) - 1) / kTile + 1;
    }
    __device__ __forceinline__ int first(int r, int k) const {
        const int i = k * kTile - (len[r] - used[r]);
        return i > 0 ? i / nq : 0;
    }
};

// A place in the jobs: the unit x (query block, or token tile where kSums) of row r and KV head
// k, and the other tile s of [s0, n) that the unit walks.
template <bool kSums>
struct Walk {
    int r, k, x, s, s0, n, left;
    __device__ __forceinline__ void enter(const Rows& w) {
        if (kSums) {
            s0 = w.first(r, x);
            n = w.query_blocks(r);
        } else {
            s0 = 0;
            n = w.seen(r, x);
        }
        s = s0;
    }
    // On to the next job; true where that is another unit's.
    __device__ __forceinline__ bool next(const Rows& w, int hk) {
        --left;
        if (++s < n) return false;
        if (left <= 0) return true;
        if (++x == (kSums ? w.tiles(r) : w.query_blocks(r))) {
            x = 0;
            if (++k == hk) {
                k = 0;
                do ++r; while (w.used[r] == 0);
            }
        }
        enter(w);
        return true;
    }
    __device__ __forceinline__ int block() const { return kSums ? s : x; }
    __device__ __forceinline__ int tile() const { return kSums ? x : s; }
    __device__ __forceinline__ int unit(const Rows& w) const {
        return w.units[r] + k * (kSums ? w.tiles(r) : w.query_blocks(r)) + x;
    }
};

// Shared memory, from a 1024-byte boundary on.
template <bool kFp8>
struct Smem {
    static constexpr int kRing = kFp8 ? 3 : 4;  // streamed tiles
    static constexpr uint32_t fixed = 0;
    static constexpr uint32_t ring = fixed + kFixed * kOperand;
    static constexpr uint32_t raw = ring + kRing * kOperand;
    // 1: groups' maxima and sums [kComb][kGroups - 1][128] float2; 3: -e [kAhead][128], then the
    // groups' sums
    static constexpr uint32_t lse = raw + (kFp8 ? kRaw * kCodes : 0);
    static constexpr uint32_t comb = lse + kAhead * kTile * 4;
    static constexpr uint32_t bars = comb + kComb * (kGroups - 1) * kTile * 4;
    static_assert(kComb * (kGroups - 1) * 4 <= kAhead * 4, "the groups' sums fit");
    // -e of job j + kAhead are copied once the products of job j + kAhead - kRing are done, which were
    // issued after the group of job j had read job j + kBufs, and so was done with job j.
    static_assert(kAhead - kRing >= 2 * kBufs, "what the sums still need is not overwritten");
    static constexpr uint32_t misc = bars + 64 * 8;                      // tmem address, start [8], stop, warp sums
    static constexpr uint32_t bad = misc + 256;                          // [16] 16-token groups of K not to be seen
    static constexpr uint32_t rows = bad + 64;                           // 6 x [rows + 1] ints
    __host__ __device__ static constexpr uint32_t total(int n) { return rows + 6 * ((uint32_t)n + 1) * 4 + 1024; }
};
static_assert(Smem<true>::total(kMaxRows) <= 232448 && Smem<false>::total(kMaxRows) <= 232448, "shared memory per block");

__device__ __forceinline__ void sts16(uint32_t addr, uint4 v) {
    asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
                 : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
    return v;
}
__device__ __forceinline__ uint32_t low_bits(int n) { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1; }

// Inclusive prefix over the warp's lanes, held at `most`.
__device__ __forceinline__ int scan_most(int v, int most) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v = min(v, most - t) + t;  // both below most: no overflow
    }
    return v;
}

// kHook: for tests, a role that gives up.
template <bool kFp8, bool kSums, bool kHook>
__global__ void __launch_bounds__(threads<kFp8>(), 1)
    tile_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap qmap,
                const __grid_constant__ Params p) {
    using S = Smem<kFp8>;
    constexpr int kThreads = threads<kFp8>(), kWarps = kThreads / 32, kMost = 1 << 30, kRing = S::kRing;
    extern __shared__ unsigned char smem_raw[];
    unsigned char* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    const uint32_t sbase = smem_u32(smem);
    const uint32_t bar_ffull = sbase + S::bars;             // [kFixed] the unit's tile is there
    const uint32_t bar_ffree = bar_ffull + 8 * kFixed;      // [kFixed] its products are done
    const uint32_t bar_rfull = bar_ffree + 8 * kFixed;      // [kRing]
    const uint32_t bar_rfree = bar_rfull + 8 * kRing;       // [kRing]
    const uint32_t bar_wfull = bar_rfree + 8 * kRing;       // [kRaw] codes are there
    const uint32_t bar_wfree = bar_wfull + 8 * kRaw;        // [kRaw] and are widened
    const uint32_t bar_lse = bar_wfree + 8 * kRaw;          // [kAhead] a job's -e are there
    const uint32_t bar_done = bar_lse + 8 * kAhead;         // [kBufs] products are done
    const uint32_t bar_read = bar_done + 8 * kBufs;         // [kBufs] and are read
    const uint32_t bar_comb = bar_read + 8 * kBufs;         // [kComb] the other groups' sums of a unit are there
    const uint32_t bar_took = bar_comb + 8 * kComb;         // [kComb] and are taken
    const uint32_t bar_fin = bar_took + 8 * kComb;          // the last products are done
    volatile int* misc = reinterpret_cast<volatile int*>(smem + S::misc);
    const volatile int* stop = misc + 16;
    volatile int* bad = reinterpret_cast<volatile int*>(smem + S::bad);
    int* sm_rows = reinterpret_cast<int*>(smem + S::rows);
    const int rows = p.rows, hk = p.hk, nq = p.nq;
    int *sm_len = sm_rows, *sm_used = sm_len + rows + 1, *sm_end = sm_used + rows + 1, *sm_jobs = sm_end + rows + 1;
    int *sm_blocks = sm_jobs + rows + 1, *sm_tiles = sm_blocks + rows + 1;
    Rows w;
    w.len = sm_len;
    w.used = sm_used;
    w.end = sm_end;
    w.units = kSums ? sm_tiles : sm_blocks;
    w.blocks = sm_blocks;
    w.nq = nq;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (tid == 0) {
        for (int i = 0; i < kFixed; ++i) {
            mbar_init(bar_ffull + 8 * i, kFp8 && kSums ? kConvWarps : 1);
            mbar_init(bar_ffree + 8 * i, 1);
        }
        for (int i = 0; i < kRing; ++i) {
            mbar_init(bar_rfull + 8 * i, kFp8 && !kSums ? kConvWarps : 1);
            mbar_init(bar_rfree + 8 * i, 1);
        }
        for (int i = 0; i < kRaw; ++i) {
            mbar_init(bar_wfull + 8 * i, 1);
            mbar_init(bar_wfree + 8 * i, kConvWarps);
        }
        for (int i = 0; i < kAhead; ++i) mbar_init(bar_lse + 8 * i, 1);
        for (int i = 0; i < kComb; ++i) {
            mbar_init(bar_comb + 8 * i, kSumWarps - 4);
            mbar_init(bar_took + 8 * i, 4);
        }
        for (int i = 0; i < kBufs; ++i) {
            mbar_init(bar_done + 8 * i, 2);  // the products, and the thread that issued them
            mbar_init(bar_read + 8 * i, 4);
        }
        mbar_init(bar_fin, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        misc[16] = 0;
    }
    if (warp == kCopyWarp && lane < 2)
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(lane ? &qmap : &kmap)) : "memory");
    if (warp == kMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(sbase + S::misc),
                     "r"(kTmemCols));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    // Rows of the query operands that no copy writes hold zeros.
    for (int i = tid; i < (kSums ? kRing : kFixed) * 2 * (kTile - nq * p.group) * 8; i += kThreads) {
        const int per = (kTile - nq * p.group) * 8, half = i / per, c = i - half * per;
        sts16(sbase + (kSums ? S::ring : S::fixed) + half * kHalf + nq * p.group * 128 + c * 16, make_uint4(0, 0, 0, 0));
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    griddep_wait();

    // ---- the rows: lengths, then jobs, query blocks and token tiles and their prefixes ----
    for (int r = tid; r < rows; r += kThreads) {
        const int q0 = p.q_start[r], q1 = p.q_start[r + 1], C = q1 - q0, L = p.seq_lens[r];
        const bool wrong = q0 < 0 || q1 < q0 || q1 > p.total || L < C || L > p.limit;
        if (wrong && blockIdx.x == 0 && !kSums) flag_error(p.dev_err, PKV_DEV_ERR_SEQ_LEN);
        sm_len[r] = wrong ? 0 : L;
        sm_used[r] = wrong ? 0 : min(C, p.window);
        sm_end[r] = q1;
    }
    __syncthreads();
    for (int r = warp; r < rows; r += kWarps) {  // a warp a row: the jobs of its query blocks
        const int nm = w.query_blocks(r);
        int sum = 0;
        for (int m = lane; m < nm; m += 32) sum += w.seen(r, m);
        sum = __reduce_add_sync(0xffffffffu, sum);
        if (lane == 0) {
            sm_jobs[r] = (int)min((int64_t)kMost, (int64_t)sum * hk);
            sm_blocks[r] = (int)min((int64_t)kMost, (int64_t)nm * hk);
            sm_tiles[r] = (int)min((int64_t)kMost, (int64_t)w.tiles(r) * hk);
        }
    }
    __syncthreads();
    if (warp < 3) {  // exclusive prefixes in place, a warp an array
        int* a = warp == 0 ? sm_jobs : warp == 1 ? sm_blocks : sm_tiles;
        int run = 0;
        for (int r0 = 0; r0 < rows; r0 += 32) {
            const int v = r0 + lane < rows ? a[r0 + lane] : 0;
            const int incl = scan_most(v, kMost), last = __shfl_sync(0xffffffffu, incl, 31);
            if (r0 + lane < rows) a[r0 + lane] = min(incl - v, kMost - run) + run;
            run = min(last, kMost - run) + run;
        }
        if (lane == 0) a[rows] = run;
    }
    __syncthreads();
    // Rows that overlap may have more blocks than there is room for: nothing is done.
    const bool fits = sm_blocks[rows] <= p.most_units && sm_jobs[rows] < kMost && sm_tiles[rows] < kMost;
    if (blockIdx.x == 0 && !kSums) {
        if (tid == 0) {
            if (!fits) flag_error(p.dev_err, PKV_DEV_ERR_SEQ_LEN);
            p.head[0] = fits ? sm_blocks[rows] : 0;
            p.head[1] = fits;
        }
        for (int r = tid; r <= rows; r += kThreads) p.tile_pre[r] = sm_tiles[r];
    }
    const int W = fits ? sm_jobs[rows] : 0, grid = min(W, p.grid), cta = blockIdx.x;
    const bool idle = cta >= grid;
    const int j0 = idle ? 0 : (int)((int64_t)W * cta / grid), j1 = idle ? 0 : (int)((int64_t)W * (cta + 1) / grid);
    if (!idle && warp == 0) {
        // the unit that job j0 is in
        int lo = 0, hi = rows - 1;
        while (lo < hi) {  // the last row whose jobs start at or before j0
            const int mid = (lo + hi + 1) >> 1;
            if (sm_jobs[mid] <= j0) lo = mid; else hi = mid - 1;
        }
        const int r = lo, per_head = (sm_jobs[r + 1] - sm_jobs[r]) / hk, k = (j0 - sm_jobs[r]) / per_head;
        const int off = j0 - sm_jobs[r] - k * per_head, units = kSums ? w.tiles(r) : w.query_blocks(r);
        int run = 0, x = 0, before = 0;
        for (int x0 = 0; x0 < units; x0 += 32) {
            const int y = x0 + lane;
            const int v = y < units ? (kSums ? w.query_blocks(r) - w.first(r, y) : w.seen(r, y)) : 0;
            const int incl = scan_most(v, kMost);
            const unsigned over = __ballot_sync(0xffffffffu, run + incl > off);
            if (over) {
                const int l = __ffs(over) - 1;
                x = x0 + l;
                before = run + __shfl_sync(0xffffffffu, incl - v, l);
                break;
            }
            run += __shfl_sync(0xffffffffu, incl, 31);
        }
        if (lane == 0) {
            misc[4] = r;
            misc[5] = k;
            misc[6] = x;
            misc[7] = off - before;  // jobs of the unit before j0
            if (kHook) misc[8] = j1 - j0;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<uint32_t*>(smem + S::misc);
    auto give_up = [&] {
        misc[16] = 1;
        flag_error(p.dev_err, PKV_DEV_ERR_TIMEOUT);
    };
    Walk<kSums> at;
    if (!idle) {
        at.r = misc[4];
        at.k = misc[5];
        at.x = misc[6];
        at.enter(w);
        at.s += misc[7];
    }
    at.left = j1 - j0;
    auto cut = [&](int role) { return kHook && misc[8] > p.last[role]; };  // it gives up before its last job

    if (idle) {
        // nothing to do but the release below
    } else if (warp == kCopyWarp) {
        // ============================ copies ============================
        bool ok = true;
        Walk<kSums> c = at;
        if (kHook) c.left = min(c.left, p.last[0]);
        // A ring's next slot, the parity of the wait for it to be free (from the second lap on), fills.
        struct Ring {
            int s = 0, fills = 0;
            uint32_t ph = 1;
            __device__ __forceinline__ void next(int n) {
                ++fills;
                if (++s == n) {
                    s = 0;
                    ph ^= 1;
                }
            }
        };
        Ring fix, str, raw, neg;
        // Lane l knows box l % boxes of tile l / boxes of a batch of 32 / boxes tiles.
        const int boxes = kTile / p.kbox, batch = 32 / boxes, my_tile = lane / boxes, my_box = lane - my_tile * boxes;
        const uint32_t box_bytes = (uint32_t)p.kbox * 128;
        const int my_off = my_tile * kTile + my_box * p.kbox;
        auto fetch = [&](int r, int tile) {  // its table entry in the batch from `tile` on
            const int t = tile * kTile + my_off;
            return t < w.len[r] ? p.tables[(int64_t)r * p.mbpr + t / p.bs] : 0;
        };
        int row = -1;        // the box's pool row (-1: none)
        uint32_t lost = 0;   // its 16-token groups that are not to be seen
        auto resolve = [&](int r, int tile, int pb) {
            const int t = tile * kTile + my_off;
            row = -1;
            lost = 0;
            if (t < w.len[r]) {
                if (pb >= 0 && pb < p.nb) {
                    row = pb * p.bs + t % p.bs;
                } else {
                    flag_error(p.dev_err, PKV_DEV_ERR_BLOCK_ID);
                    lost = ((1u << (p.kbox / 16)) - 1) << (my_box * (p.kbox / 16));
                }
            }
        };
        // Tile j of the batch to the next slot of its ring.
        auto copy_k = [&](int j, int k, int note) {
            Ring& ring = kFp8 ? raw : kSums ? fix : str;
            const int n = kFp8 ? kRaw : kSums ? kFixed : kRing;
            const uint32_t full = (kFp8 ? bar_wfull : kSums ? bar_ffull : bar_rfull) + 8 * ring.s;
            const uint32_t free = (kFp8 ? bar_wfree : kSums ? bar_ffree : bar_rfree) + 8 * ring.s;
            const uint32_t dst = sbase + (kFp8 ? S::raw : kSums ? S::fixed : S::ring) + ring.s * (kFp8 ? kCodes : kOperand);
            if (ring.fills >= n && !mbar_waitw(free, ring.ph, stop)) return false;
            const bool mine = my_tile == j;
            const uint32_t some = __ballot_sync(0xffffffffu, mine && row >= 0);
            const uint32_t gone = __reduce_or_sync(0xffffffffu, mine ? lost : 0u);
            if (lane == 0) {
                bad[note & 15] = (int)gone;
                mbar_arrive_expect_tx(full, __popc(some) * box_bytes * (kFp8 ? 1 : 2));
            }
            __syncwarp();
            if (mine && row >= 0) {
                tma_load_3d(dst + my_box * box_bytes, &kmap, 0, k, row, full);
                if (!kFp8) tma_load_3d(dst + kHalf + my_box * box_bytes, &kmap, 64, k, row, full);
            }
            ring.next(n);
            return true;
        };
        const uint32_t q_bytes = (uint32_t)(nq * p.group) * 256u;
        int units = 0, jobs = 0;
        int pb_next = fetch(c.r, c.tile());
        while (c.left > 0 && ok) {
            const int end = min(c.n, c.s + c.left), pb = pb_next;
            Walk<kSums> nx = c;  // the next piece, whose first batch is looked up meanwhile
            nx.left -= end - c.s - 1;
            nx.s = end - 1;
            nx.next(w, hk);
            if (nx.left > 0) pb_next = fetch(nx.r, nx.tile());
            resolve(c.r, c.tile(), pb);
            int q = w.end[c.r] - w.used[c.r] + c.block() * nq;
            if (kSums) {
                // the fixed token tile, then the query blocks and their -e by one lane
                if (!(ok = copy_k(0, c.k, units))) break;
                if (lane == 0) {
                    const float* e = p.neg_lse + (int64_t)(w.blocks[c.r] + c.k * w.query_blocks(c.r) + c.s) * kTile;
#pragma unroll 1
                    for (int o = c.s; o < end; ++o) {
                        if (str.fills >= kRing && !(ok = mbar_wait1(bar_rfree + 8 * str.s, str.ph, stop))) break;
                        const uint32_t full = bar_rfull + 8 * str.s, dst = sbase + S::ring + str.s * kOperand;
                        mbar_arrive_expect_tx(full, q_bytes);
                        tma_load_3d(dst, &qmap, 0, c.k * p.group, q, full);
                        tma_load_3d(dst + kHalf, &qmap, 64, c.k * p.group, q, full);
                        mbar_arrive_expect_tx(bar_lse + 8 * neg.s, kTile * 4);
                        bulk_load(sbase + S::lse + neg.s * kTile * 4, e, kTile * 4, bar_lse + 8 * neg.s);
                        q += nq;
                        e += kTile;
                        str.next(kRing);
                        neg.next(kAhead);
                    }
                }
                ok = __shfl_sync(0xffffffffu, ok, 0);
            } else {
                // the fixed query block, then the token tiles, a batch's rows at a time
                if (fix.fills >= kFixed && !(ok = mbar_waitw(bar_ffree + 8 * fix.s, fix.ph, stop))) break;
                if (lane == 0) {
                    const uint32_t full = bar_ffull + 8 * fix.s, dst = sbase + S::fixed + fix.s * kOperand;
                    mbar_arrive_expect_tx(full, q_bytes);
                    tma_load_3d(dst, &qmap, 0, c.k * p.group, q, full);
                    tma_load_3d(dst + kHalf, &qmap, 64, c.k * p.group, q, full);
                }
                fix.next(kFixed);
                int pb2 = c.s + batch < end ? fetch(c.r, c.s + batch) : 0, j = 0;
#pragma unroll 1
                for (int o = c.s; o < end; ++o, ++j, ++jobs) {
                    if (j == batch) {
                        j = 0;
                        resolve(c.r, o, pb2);
                        pb2 = o + batch < end ? fetch(c.r, o + batch) : 0;
                    }
                    if (!(ok = copy_k(j, c.k, jobs))) break;
                }
            }
            ++units;
            c = nx;
        }
        if (lane == 0) {
            if (!ok || cut(0)) give_up();
            // every copy has landed before the block exits
            auto drain = [&](uint32_t bar, int n, int count) {
                for (int i = max(0, n - count); i < n; ++i) mbar_drain1(bar + 8 * (i % count), (uint32_t)(i / count) & 1);
            };
            drain(bar_ffull, fix.fills, kFixed);
            drain(bar_rfull, str.fills, kRing);
            drain(bar_wfull, raw.fills, kRaw);
            drain(bar_lse, neg.fills, kAhead);
        }
        __syncwarp();
    } else if (warp == kMmaWarp) {
        // ============================ products ============================
        if (lane == 0) {
            const uint32_t id = idesc(kTile, kTile, 0);
            const uint64_t a0 = sdesc(sbase + S::fixed, 16, 1024), b0 = sdesc(sbase + S::ring, 16, 1024);
            bool ok = true;
            int f = 0, s = 0, b = 0;
            uint32_t fph = 0, sph = 0, bph = 1;
            Walk<kSums> c = at;
            if (kHook) c.left = min(c.left, p.last[1]);
            while (c.left > 0 && ok) {
                const int end = min(c.n, c.s + c.left);
                if (!(ok = mbar_wait1(bar_ffull + 8 * f, fph, stop))) break;
                const uint64_t da = a0 + (uint64_t)(f * (kOperand >> 4));
#pragma unroll 1
                for (int o = c.s; o < end; ++o) {
                    if (!(ok = mbar_wait1(bar_rfull + 8 * s, sph, stop))) break;
                    // (a fresh barrier counts the phase before its first as complete)
                    if (!(ok = mbar_wait1(bar_read + 8 * b, bph, stop))) break;
                    tc_fence_after();
                    const uint64_t db = b0 + (uint64_t)(s * (kOperand >> 4));
#pragma unroll
                    for (int ks = 0; ks < 8; ++ks) {
                        const uint32_t off = ((ks >> 2) * kHalf + (ks & 3) * 32) >> 4;
                        umma_ss(tmem + b * kTile, da + off, db + off, id, ks > 0);
                    }
                    mbar_arrive(bar_done + 8 * b);  // (what this thread has seen, the sums see too)
                    umma_commit(bar_done + 8 * b);
                    umma_commit(bar_rfree + 8 * s);
                    if (++s == kRing) {
                        s = 0;
                        sph ^= 1;
                    }
                    if (++b == kBufs) {
                        b = 0;
                        bph ^= 1;
                    }
                }
                if (!ok) break;
                umma_commit(bar_ffree + 8 * f);
                if (++f == kFixed) {
                    f = 0;
                    fph ^= 1;
                }
                c.left -= end - c.s - 1;
                c.s = end - 1;
                c.next(w, hk);
            }
            if (!ok || cut(1)) give_up();
            umma_commit(bar_fin);
            if (!mbar_drain1(bar_fin, 0)) flag_error(p.dev_err, PKV_DEV_ERR_TIMEOUT);
        }
        __syncwarp();
    } else if (kFp8 && warp >= kConvWarp) {
        // ============================ widening ============================
        bool ok = true, fresh = true;
        int units = 0, jobs = 0, codes = 0;
        Walk<kSums> c = at;
        if (kHook) c.left = min(c.left, p.last[2]);
        const int row = tid - kConvWarp * 32;  // a token a thread
        while (c.left > 0 && ok) {
            if (!kSums || fresh) {
                const int n = kSums ? units : jobs, count = kSums ? kFixed : kRing, to = n % count, from = codes % kRaw;
                const uint32_t full = (kSums ? bar_ffull : bar_rfull) + 8 * to;
                const uint32_t free = (kSums ? bar_ffree : bar_rfree) + 8 * to;
                if (!(ok = mbar_waitw(bar_wfull + 8 * from, (uint32_t)(codes / kRaw) & 1, stop))) break;
                if (n >= count && !(ok = mbar_waitw(free, (uint32_t)(n / count - 1) & 1, stop))) break;
                const uint32_t src = sbase + S::raw + from * kCodes + row * 128;
                const uint32_t dst = sbase + (kSums ? S::fixed : S::ring) + to * kOperand + row * 128;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const uint4 x = lds16(src + ((i ^ (row & 7)) << 4));
                    const uint32_t o = dst + (i >> 2) * kHalf;
                    sts16(o + (((2 * i & 7) ^ (row & 7)) << 4), widen8(make_uint2(x.x, x.y)));
                    sts16(o + (((2 * i + 1 & 7) ^ (row & 7)) << 4), widen8(make_uint2(x.z, x.w)));
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(full);
                    mbar_arrive(bar_wfree + 8 * from);
                }
                ++codes;
            }
            if (fresh) ++units;
            ++jobs;
            fresh = c.next(w, hk);
        }
        if ((!ok || cut(2)) && lane == 0) give_up();
    } else if (warp < kSumWarps) {
        // ============================ sums ============================
        const int i = (warp & 3) * 32 + lane, grp = warp >> 2;  // row of the product; group
        const uint32_t from_tmem = tmem + ((uint32_t)((warp & 3) * 32) << 16) + grp * kTile;
        bool ok = true;
        int units = 0, jobs = 0;
        Walk<kSums> c = at;
        if (kHook) c.left = min(c.left, p.last[3]);
        const int group = p.group;
        const int my_q = i / group, columns = nq * group;
        // The 32 columns of chunk ch, all of which count but, of flat rows, those that no query has.
        auto add_plain = [&](int ch, float& ref, float& acc, float sl2, uint64_t sl, const float4* lse) {
            uint32_t v[32];
            tmem_ld32(from_tmem + 32 * ch, v);
            float base = 0.f;
            if (!kSums) {
                float a, z, top;  // the largest score, in base 2
                if (sl2 >= 0.f) {
                    a = z = -INFINITY;
#pragma unroll
                    for (int x = 0; x < 32; x += 4) {
                        a = fmaxf(fmaxf(__uint_as_float(v[x]), __uint_as_float(v[x + 1])), a);
                        z = fmaxf(fmaxf(__uint_as_float(v[x + 2]), __uint_as_float(v[x + 3])), z);
                    }
                    top = fmaxf(a, z) * sl2;
                } else {
                    a = z = INFINITY;
#pragma unroll
                    for (int x = 0; x < 32; x += 4) {
                        a = fminf(fminf(__uint_as_float(v[x]), __uint_as_float(v[x + 1])), a);
                        z = fminf(fminf(__uint_as_float(v[x + 2]), __uint_as_float(v[x + 3])), z);
                    }
                    top = fminf(a, z) * sl2;
                }
                if (top > ref + kMove) {  // (from -inf any score is)
                    acc *= ref == -INFINITY ? 1.f : fast_exp2(ref - top);
                    ref = top;
                }
                base = ref == -INFINITY ? 0.f : -ref;
            }
            uint64_t s0 = f32x2(0.f, 0.f), s1 = s0;
#pragma unroll
            for (int x = 0; x < 32; x += 4) {
                float4 y = make_float4(base, base, base, base);
                if (kSums) y = lse[ch * 8 + x / 4];
                float a, b, d, f;
                f32x2_split(fma_f32x2(f32x2(__uint_as_float(v[x]), __uint_as_float(v[x + 1])), sl, f32x2(y.x, y.y)), a, b);
                f32x2_split(fma_f32x2(f32x2(__uint_as_float(v[x + 2]), __uint_as_float(v[x + 3])), sl, f32x2(y.z, y.w)), d, f);
                if (kSums && x >= kCertain - 96) {  // zeros times a key that is no number
                    const int from = 32 * ch + x;
                    a = from < columns ? a : -INFINITY;
                    b = from + 1 < columns ? b : -INFINITY;
                    d = from + 2 < columns ? d : -INFINITY;
                    f = from + 3 < columns ? f : -INFINITY;
                }
                s0 = add_f32x2(s0, f32x2(fast_exp2(a), fast_exp2(b)));
                s1 = add_f32x2(s1, f32x2(fast_exp2(d), fast_exp2(f)));
            }
            float a, b;
            f32x2_split(add_f32x2(s0, s1), a, b);
            acc += a + b;
        };
        // The same of the columns in `seen`.
        auto add_seen = [&](int ch, uint32_t seen, float& ref, float& acc, float sl2, const float4* lse) {
            uint32_t v[32];
            tmem_ld32(from_tmem + 32 * ch, v);
            if (!__any_sync(0xffffffffu, seen != 0)) return;
            float base = 0.f;
            if (!kSums) {
                float top = -INFINITY;
#pragma unroll
                for (int x = 0; x < 32; ++x)
                    if (seen >> x & 1) top = fmaxf(top, __uint_as_float(v[x]) * sl2);
                if (top > ref + kMove) {
                    acc *= ref == -INFINITY ? 1.f : fast_exp2(ref - top);
                    ref = top;
                }
                base = ref == -INFINITY ? 0.f : -ref;
            }
            float s = 0.f;
#pragma unroll
            for (int x = 0; x < 32; ++x) {
                const float y = kSums ? reinterpret_cast<const float*>(lse)[32 * ch + x] : base;
                if (seen >> x & 1) s += fast_exp2(fmaf(__uint_as_float(v[x]), sl2, y));
            }
            acc += s;
        };
        auto let_go = [&] {  // the scores are read
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar_read + 8 * grp);
        };
        uint32_t turn = 0;  // parity of this group's next buffer
        // jobs of this block, in units: c stands at the first one not yet walked
        while (c.left > 0 && ok) {
            const int from = c.s, job0 = jobs;  // the piece's first job
            const float sl2 = kFp8 ? p.scale_log2 * p.k_scale[c.k] : p.scale_log2;
            const uint64_t sl = f32x2(sl2, sl2);
            // Positions: query q of the row's used ones sees tokens up to p0 + q.
            const int used = w.used[c.r], p0 = w.len[c.r] - used, end = min(c.n, c.s + c.left);
            float ref = -INFINITY, acc = 0.f;  // what exponents are taken from; the row's sum
            const int skip = (grp - job0) & (kGroups - 1);
            jobs += end - c.s;
#pragma unroll 1
            for (int o = c.s + skip, job = job0 + skip; o < end; o += kGroups, job += kGroups, turn ^= 1) {
                const int e = kSums ? job % kAhead : 0;
                if (!(ok = mbar_waitw(bar_done + 8 * grp, turn, stop))) break;
                if (kSums && !(ok = mbar_waitw(bar_lse + 8 * e, (uint32_t)(job / kAhead) & 1, stop))) break;
                tc_fence_after();
                const uint32_t hidden = (uint32_t)bad[(kSums ? units : job) & 15];
                const int q0 = (kSums ? o : c.x) * nq, t0 = (kSums ? c.x : o) * kTile;
                const int here = min(nq, used - q0);  // queries of the block
                const float4* lse = reinterpret_cast<const float4*>(smem + S::lse + e * kTile * 4);
                // (1: what rows behind the queries get is not used)
                if (t0 + kTile - 1 <= p0 + q0 && !hidden && (!kSums || (here == nq && columns >= kCertain))) {
#pragma unroll 1
                    for (int ch = 0; ch < 4; ++ch) {
                        add_plain(ch, ref, acc, sl2, sl, lse);
                    }
                } else {
                    // columns lo .. hi - 1 count
                    int lo = 0, hi = kTile;
                    if (!kSums) {
                        hi = p0 + q0 + my_q - t0 + 1;  // row i: query; column: token
                    } else {
                        lo = max(0, t0 + i - p0 - q0) * group;  // row i: token; column: flat row
                        hi = hidden >> (i >> 4) & 1 ? 0 : here * group;
                    }
#pragma unroll 1
                    for (int ch = 0; ch < 4; ++ch) {
                        uint32_t seen = low_bits(hi - 32 * ch) & ~low_bits(lo - 32 * ch);
                        if (!kSums && hidden) {
                            if (hidden >> (2 * ch) & 1) seen &= 0xffff0000u;
                            if (hidden >> (2 * ch + 1) & 1) seen &= 0x0000ffffu;
                        }
                        if (__all_sync(0xffffffffu, seen == ~0u))
                            add_plain(ch, ref, acc, sl2, sl, lse);
                        else
                            add_seen(ch, seen, ref, acc, sl2, lse);
                    }
                }
                let_go();
            }
            if (!ok) break;
            // ---- the block's piece of the unit: the groups' sums ----
            const int slot = units % kComb, lap = units / kComb;
            float* one = reinterpret_cast<float*>(smem + S::comb) + slot * (kGroups - 1) * kTile + i;
            float2* two = reinterpret_cast<float2*>(smem + S::lse) + slot * (kGroups - 1) * kTile + i;
            if (grp > 0) {
                if (lap > 0 && !(ok = mbar_waitw(bar_took + 8 * slot, (uint32_t)(lap - 1) & 1, stop))) break;
                if (kSums)
                    one[(grp - 1) * kTile] = acc;
                else
                    two[(grp - 1) * kTile] = make_float2(ref, acc);
                __syncwarp();
                if (lane == 0) mbar_arrive(bar_comb + 8 * slot);
            } else {
                if (!(ok = mbar_waitw(bar_comb + 8 * slot, (uint32_t)lap & 1, stop))) break;
                const int unit = c.unit(w);
                const int64_t rec = (int64_t)cta + unit;
                if (kSums) {
#pragma unroll
                    for (int g = 0; g < kGroups - 1; ++g) acc += one[g * kTile];
                    p.sums[rec * kTile + i] = acc;
                } else {
                    float M = ref;
#pragma unroll
                    for (int g = 0; g < kGroups - 1; ++g) M = fmaxf(M, two[g * kTile].x);
                    const float z = M == -INFINITY ? 0.f : M;
                    acc *= fast_exp2(ref - z);
#pragma unroll
                    for (int g = 0; g < kGroups - 1; ++g) acc += two[g * kTile].y * fast_exp2(two[g * kTile].x - z);
                    p.ml[rec * kTile + i] = make_float2(M, acc);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(bar_took + 8 * slot);
                if (i == 0 && from == c.s0)  // this block has the unit's first job: who has its last
                    (kSums ? p.tile_info : p.block_info)[unit] =
                        make_int2(cta, owner_of(j0 + job0 + c.n - c.s0 - 1, W, grid) - cta + 1);
            }
            ++units;
            c.left -= end - c.s - 1;  // to the piece's last job
            c.s = end - 1;
            c.next(w, hk);
        }
        if ((!ok || cut(3)) && lane == 0) give_up();
    }

    // ---- release tensor memory ----
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols));
    }
}

// 2: a query block's -e from its pieces, in order; -inf for rows that no query has or that see nothing.
__global__ void __launch_bounds__(kTile) lse_kernel(const __grid_constant__ Params p) {
    const int unit = (int)blockIdx.x, i = (int)threadIdx.x;
    griddep_wait();
    if (unit >= p.head[0]) return;
    const int2 at = p.block_info[unit];
    float M = -INFINITY, L = 0.f;
    // (a call that timed out may have left anything there)
    if (i < p.nq * p.group && at.x >= 0 && at.x < p.grid && at.y > 0 && at.y <= p.grid - at.x) {
        const float2* ml = p.ml + ((int64_t)at.x + unit) * kTile + i;
#pragma unroll 4
        for (int c = 0; c < at.y; ++c) {
            const float2 y = ml[(int64_t)c * kTile];
            const float N = fmaxf(M, y.x), g = N == -INFINITY ? 0.f : N;
            L = L * fast_exp2(M - g) + y.y * fast_exp2(y.x - g);
            M = N;
        }
    }
    p.neg_lse[(int64_t)unit * kTile + i] = L == 0.f ? -INFINITY : -((M == -INFINITY ? 0.f : M) + log2f(L));
}

// 4: a token's sum over its pieces, in order, added to the running sum; the chunk's own tokens
// start from zero.
constexpr int kEndThreads = 256;
__global__ void __launch_bounds__(kEndThreads) add_kernel(const __grid_constant__ Params p) {
    const int k = (int)blockIdx.x, r = (int)blockIdx.y, t = (int)(blockIdx.z * kEndThreads + threadIdx.x);
    griddep_wait();
    if (!p.head[1]) return;
    const int tiles = (p.tile_pre[r + 1] - p.tile_pre[r]) / p.hk;  // 0 for rows without queries
    const int L = p.seq_lens[r], C = p.q_start[r + 1] - p.q_start[r], tile = t / kTile;
    if (tile >= tiles || t >= L) return;
    const int unit = p.tile_pre[r] + k * tiles + tile;
    float* w = p.weights + ((int64_t)r * p.hk + k) * p.stride + t;
    const float was = t < L - C ? *w : 0.f;
    const int2 at = p.tile_info[unit];
    float sum = 0.f;
    if (at.x >= 0 && at.x < p.grid && at.y > 0 && at.y <= p.grid - at.x) {
        const float* s = p.sums + ((int64_t)at.x + unit) * kTile + t % kTile;
#pragma unroll 4
        for (int c = 0; c < at.y; ++c) sum += s[(int64_t)c * kTile];
    }
    *w = was + sum;
}

// For tests (pkv_debug_set_weights_hooks); 0 in normal use.
std::atomic<int> g_hook_role{0}, g_hook_jobs{0};

struct Layout {
    size_t tile_pre, block_info, tile_info, ml, neg_lse, sums, bytes;
    int64_t blocks, tiles;
    int nq;
};
// Query blocks of rows whose chunks do not overlap.
static int64_t most_blocks(int rows, int total, int kv_heads, int nq, int window) {
    const int64_t all = (int64_t)total / nq + rows, some = (int64_t)rows * (((int64_t)window + nq - 1) / nq);
    return (all < some ? all : some) * kv_heads;
}
static Layout layout(int rows, int total, int kv_heads, int group, int max_seq_len, int window, int sms) {
    Layout l;
    l.nq = kTile / group;
    l.blocks = most_blocks(rows, total, kv_heads, l.nq, window);
    l.tiles = (int64_t)rows * kv_heads * (((int64_t)max_seq_len + kTile - 1) / kTile);
    size_t at = 256;
    auto take = [&](size_t bytes) {
        const size_t here = at;
        at += align_up(bytes, 256);
        return here;
    };
    l.tile_pre = take(((size_t)rows + 1) * 4);
    l.block_info = take((size_t)l.blocks * 8);
    l.tile_info = take((size_t)l.tiles * 8);
    l.ml = take((size_t)(l.blocks + sms) * kTile * 8);
    l.neg_lse = take((size_t)l.blocks * kTile * 4);
    l.sums = take((size_t)(l.tiles + sms) * kTile * 4);
    l.bytes = at;
    return l;
}
static bool supported(int rows, int total, int q_heads, int kv_heads, int head_dim, int max_seq_len, int block_size,
                      int window) {
    if (head_dim != kHeadDim || block_size % 16 || rows > kMaxRows || q_heads / kv_heads > kTile ||
        max_seq_len > (1 << 23) || kv_heads > 65535)
        return false;
    const int nq = kTile / (q_heads / kv_heads);
    const int64_t tiles = ((int64_t)max_seq_len + kTile - 1) / kTile;
    const int64_t blocks = most_blocks(rows, total, kv_heads, nq, window);
    return blocks < (int64_t(1) << 30) && (tiles == 0 || blocks < (int64_t(1) << 30) / tiles) &&
           (int64_t)rows * kv_heads * tiles < (int64_t(1) << 30);
}

}  // namespace prompt
}  // namespace pkv

extern "C" size_t paged_attention_prefill_weights_workspace_size(int rows, int total_q, int q_heads, int kv_heads,
                                                                 int head_dim, int max_seq_len, int block_size,
                                                                 int window) {
    using namespace pkv::prompt;
    if (rows <= 0 || total_q < 0 || q_heads <= 0 || kv_heads <= 0 || head_dim <= 0 || q_heads % kv_heads ||
        max_seq_len < 0 || block_size <= 0 || window < 1 ||
        !supported(rows, total_q, q_heads, kv_heads, head_dim, max_seq_len, block_size, window))
        return 0;
    const int sms = pkv::device_sms();  // on a machine without a GPU, as for one of 256 SMs
    return layout(rows, total_q, kv_heads, q_heads / kv_heads, max_seq_len, window, sms > 0 ? sms : 256).bytes;
}

extern "C" int paged_attention_prefill_weights(float* weights, const void* q, const void* k_pool, const float* k_scale,
                                               const int32_t* block_tables, const int32_t* seq_lens,
                                               const int32_t* q_start, int rows, int total_q, int q_heads,
                                               int kv_heads, int head_dim, int block_size, float scale, int window,
                                               int max_blocks_per_row, int num_blocks, int max_seq_len,
                                               int64_t weights_stride, void* workspace, size_t workspace_bytes,
                                               int32_t* dev_err, cudaStream_t stream) {
    using namespace pkv;
    using namespace pkv::prompt;
    if (q_heads <= 0 || kv_heads <= 0 || head_dim <= 0 || q_heads % kv_heads) return PKV_ERR_INVALID_ARG;
    if (rows < 0 || total_q < 0 || block_size <= 0 || max_blocks_per_row <= 0 || num_blocks <= 0 || max_seq_len < 0 ||
        !isfinite(scale) || window < 1 || weights_stride < max_seq_len)
        return PKV_ERR_INVALID_ARG;
    if ((int64_t)max_seq_len > (int64_t)max_blocks_per_row * block_size) return PKV_ERR_INVALID_ARG;
    if (!supported(rows, total_q, q_heads, kv_heads, head_dim, max_seq_len, block_size, window) ||
        weights_stride > (int64_t(1) << 40) || (int64_t)num_blocks * block_size >= (int64_t(1) << 31))
        return PKV_ERR_UNSUPPORTED;
    if (rows == 0 || total_q == 0) return PKV_OK;
    if (!weights || !q || !k_pool || !block_tables || !seq_lens || !q_start) return PKV_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k_pool)) return PKV_ERR_INVALID_ARG;
    const int sms = device_sms();
    if (sms <= 0) return PKV_ERR_CUDA;
    const int group = q_heads / kv_heads;
    const Layout l = layout(rows, total_q, kv_heads, group, max_seq_len, window, sms);
    if (!workspace || workspace_bytes < l.bytes || (reinterpret_cast<uintptr_t>(workspace) & 255))
        return PKV_ERR_WORKSPACE;
    const size_t wide = (size_t)rows * kv_heads * weights_stride * 4, tall = (size_t)total_q * q_heads * head_dim * 2;
    if (overlap(weights, wide, q, tall) || overlap(weights, wide, workspace, l.bytes) ||
        overlap(q, tall, workspace, l.bytes))
        return PKV_ERR_INVALID_ARG;

    unsigned char* ws = static_cast<unsigned char*>(workspace);
    Params p{};
    p.weights = weights;
    p.k_scale = k_scale;
    p.tables = block_tables;
    p.seq_lens = seq_lens;
    p.q_start = q_start;
    p.stride = weights_stride;
    p.rows = rows;
    p.total = total_q;
    p.hk = kv_heads;
    p.group = group;
    p.bs = block_size;
    p.mbpr = max_blocks_per_row;
    p.nb = num_blocks;
    p.limit = max_seq_len;
    p.window = window;
    p.nq = l.nq;
    p.kbox = 16;
    while (p.kbox < kTile && block_size % (2 * p.kbox) == 0) p.kbox *= 2;
    p.grid = sms;
    p.most_units = (int)l.blocks;
    p.scale_log2 = scale * kLog2e;
    p.head = reinterpret_cast<int*>(ws);
    p.tile_pre = reinterpret_cast<int*>(ws + l.tile_pre);
    p.block_info = reinterpret_cast<int2*>(ws + l.block_info);
    p.tile_info = reinterpret_cast<int2*>(ws + l.tile_info);
    p.ml = reinterpret_cast<float2*>(ws + l.ml);
    p.neg_lse = reinterpret_cast<float*>(ws + l.neg_lse);
    p.sums = reinterpret_cast<float*>(ws + l.sums);
    p.dev_err = dev_err;
    const int hook = g_hook_jobs.load(std::memory_order_relaxed);
    for (int& jobs : p.last) jobs = INT_MAX;
    if (hook) p.last[g_hook_role.load(std::memory_order_relaxed)] = hook - 1;
    if (l.blocks == 0 || max_seq_len == 0) return PKV_OK;

    CUtensorMap kmap, qmap;
    const int elt = k_scale ? 1 : 2;
    const int64_t kdims[3] = {head_dim, kv_heads, (int64_t)num_blocks * block_size};
    const int64_t kstrides[2] = {(int64_t)head_dim * elt, (int64_t)kv_heads * head_dim * elt};
    const int kb[3] = {128 / elt, 1, p.kbox};
    int st = tiled_map_3d(k_pool, k_scale ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, kdims,
                          kstrides, kb, &kmap);
    if (st != PKV_OK) return st;
    const int64_t qdims[3] = {head_dim, q_heads, total_q};
    const int64_t qstrides[2] = {(int64_t)head_dim * 2, (int64_t)q_heads * head_dim * 2};
    const int qb[3] = {64, group, p.nq};
    if ((st = tiled_map_3d(q, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, qdims, qstrides, qb, &qmap)) != PKV_OK) return st;
    auto* first = hook      ? (k_scale ? tile_kernel<true, false, true> : tile_kernel<false, false, true>)
                  : k_scale ? tile_kernel<true, false, false>
                            : tile_kernel<false, false, false>;
    auto* second = hook      ? (k_scale ? tile_kernel<true, true, true> : tile_kernel<false, true, true>)
                   : k_scale ? tile_kernel<true, true, false>
                             : tile_kernel<false, true, false>;
    const int most = (int)(k_scale ? Smem<true>::total(kMaxRows) : Smem<false>::total(kMaxRows));
    const size_t smem = k_scale ? Smem<true>::total(rows) : Smem<false>::total(rows);
    const unsigned block = (unsigned)(k_scale ? threads<true>() : threads<false>());
    if (cudaFuncSetAttribute(first, cudaFuncAttributeMaxDynamicSharedMemorySize, most) != cudaSuccess ||
        cudaFuncSetAttribute(second, cudaFuncAttributeMaxDynamicSharedMemorySize, most) != cudaSuccess) {
        cudaGetLastError();
        return PKV_ERR_CUDA;
    }
    if ((st = launch_early(first, (unsigned)p.grid, block, smem, stream, kmap, qmap, p)) != PKV_OK) return st;
    if ((st = launch_early(lse_kernel, (unsigned)l.blocks, kTile, 0, stream, p)) != PKV_OK) return st;
    if ((st = launch_early(second, (unsigned)p.grid, block, smem, stream, kmap, qmap, p)) != PKV_OK) return st;
    const unsigned z = (unsigned)((max_seq_len + kEndThreads - 1) / kEndThreads);
    return launch_early(add_kernel, dim3((unsigned)kv_heads, (unsigned)rows, z), kEndThreads, 0, stream, p);
}

namespace pkv {
namespace weights {
extern std::atomic<int> g_hook_granule;  // decode_weights.cu
}
}  // namespace pkv

extern "C" int pkv_debug_set_weights_hooks(int granule, int role, int jobs) {
    if (granule < 0 || role < 0 || role > 3 || jobs < 0) return PKV_ERR_INVALID_ARG;
    pkv::weights::g_hook_granule.store(granule, std::memory_order_relaxed);
    pkv::prompt::g_hook_role.store(role, std::memory_order_relaxed);
    pkv::prompt::g_hook_jobs.store(jobs, std::memory_order_relaxed);
    return PKV_OK;
}
