// paged_kv_evict: of each list (layer, row, KV head) the tokens of lowest weight
// leave the cache and the others move together, every layer at once.
//
// Mathematics.  A list of L tokens keeps n = min(L, budget): those that are
// protected (the row's first `sinks` positions and last `recent`), then the ones of
// the largest weight, the lowest slot first where weights are equal.  Weights become 32-bit
// keys whose unsigned order is the weights' order, and the n-th largest key is found
// digit by digit, 10 bits at a time from the first bit in which the keys differ: a
// histogram of the digit over the keys that share the digits so far, summed from the
// top, gives the next digit and how many keys lie above it; the search ends where
// the keys that share the digits all stay.  Nothing is sorted: tokens that stay and lie
// below n stay where they are, and the j-th slot below n that loses its token takes the
// j-th token that stays from n on.  Sources lie at n or past it and destinations below
// it, so the moves have no order among themselves, and there are as few as can be: the
// tokens that leave, not the tokens that stay.
//
// Work.  A short list has a small block, a long one a larger block or, where there are few, a
// cluster of them; every block holds its share of the keys in shared memory, and a cluster's blocks add up their
// histograms and counts through distributed shared memory.  Four neighbouring tokens
// are a lane's, 128 a warp's, at once.  The moves are dealt to the warps 32 at a time:
// a lane finds one move's slots through the table and moves its weight and
// position, then the warp moves the keys and values, several vectors in flight a lane.
//
// What bounds it.  The choice is a chain: load, differing bits, one to four histograms, the
// equal keys, the slots.  1792 lists of 1025 tokens, of which one leaves each (14.7 MB of weights
// and positions): 17.4 us, all but 1.5 the choice; all blocks are resident at once, 12 an SM, and
// issue in 66% of the cycles, 6,700 warp instructions a list (64 threads a block, 20 an SM: 23.3).
// 896 lists of 1900 to 2304, E4M3: 23.0 us, 15 of them the choice.  32 lists of 30,000 to 32,768 down
// to 4096: 39.2 us, 18.4 the choice (three cluster barriers a histogram) and 21 the
// moves, 117 MB in pieces of 256 bytes, 5.4 TB/s.
#include "pkv_internal.cuh"
#include "ptx.cuh"

namespace pkv {
namespace evict {

// Threads of a list's blocks, and blocks an SM: of lists of up to kSmall tokens, up to kShort, and long ones.
constexpr int kSmallThreads = 128, kSmallBlocks = 12, kSmall = 2048;
constexpr int kShortThreads = 256, kShortBlocks = 5, kShort = 4096;
constexpr int kLongThreads = 512, kLongBlocks = 2;
constexpr int kChunk = 4096;       // tokens of a long list's block, while its cluster may still grow
constexpr int kMostBlocks = 8;     // of a cluster (the portable limit)
constexpr int kMostChunk = 24576;  // tokens of a block, at most: 6 bytes of shared memory each
constexpr int kDigit = 10, kBins = 1 << kDigit;
constexpr int kBatch = 4;          // vectors in flight a lane
constexpr uint32_t kSafe = 0xffffffffu, kNan = 0xfffffffeu;

struct Params {
    uint4* k_pool;
    uint4* v_pool;
    const int32_t* tables;
    const int32_t* seq_lens;
    const float* weights;
    const int32_t* token_pos;
    const int32_t* tracked;   // null: nothing is recorded
    const int32_t* next_pos;  // null: the slots are the positions
    float* weights_out;
    int32_t* pos_out;
    int32_t* new_lens;
    int64_t stride;
    int rows, hk, vecs;  // vecs: 16-byte vectors of a head
    int bs, mbpr, nb, limit, budget, sinks, recent;
    int blocks;  // of a cluster
    int cap;     // tokens of a block, rounded up to whole rounds of its warps
    int in_place;
    int vec4;    // the lists' entries may be read and written four at a time
    int32_t* dev_err;
};

// The order of the floats as unsigned numbers; both zeros are one key, and NaN lies above infinity.
__device__ __forceinline__ uint32_t key_of(float w) {
    if (w != w) return kNan;
    const uint32_t u = __float_as_uint(w + 0.f);  // -0 + 0 = 0
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ uint32_t block_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
// Every thread of the cluster has arrived, and what each wrote before is seen by all.
__device__ __forceinline__ void cluster_sync() {
    __syncwarp();  // the aligned form wants the whole warp together
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The word at shared address `addr` of block `rank` of the cluster.
__device__ __forceinline__ uint32_t peer_word(uint32_t addr, int rank) {
    uint32_t a, v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(rank));
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    return v;
}

__device__ __forceinline__ uint32_t peer_half(uint32_t addr, int rank) {
    uint32_t a;
    uint16_t v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(rank));
    asm volatile("ld.shared::cluster.u16 %0, [%1];" : "=h"(v) : "r"(a) : "memory");
    return v;
}

// Sum over the lanes before this one.
__device__ __forceinline__ uint32_t lanes_before(uint32_t v) {
    const int lane = threadIdx.x & 31;
    uint32_t incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t t = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += t;
    }
    return incl - v;
}

// The slot of a row's token in the pools, or -1 for a bad table entry.
__device__ __forceinline__ int slot_of(const Params& p, const int32_t* row, int t) {
    const int lb = t / p.bs, pb = row[lb];
    return pb < 0 || pb >= p.nb ? -1 : pb * p.bs + (t - lb * p.bs);
}

// A list's place and lengths, as every thread of its blocks has them.
struct List {
    int r, h, layer, L, n, trk, end;
    bool choose;  // some of its tokens leave
    bool ask;     // and positions matter for which
    int last;     // the first position that is protected as a recent one
    int64_t base;
    __device__ __forceinline__ List(const Params& p, int head) {
        h = head;
        r = (int)blockIdx.y;
        layer = (int)blockIdx.z;
        L = p.seq_lens[r];
        n = min(L, p.budget);
        trk = p.tracked ? max(0, min(p.tracked[r], L)) : 0;
        end = p.next_pos ? p.next_pos[r] : L;  // the next token's position
        base = (((int64_t)layer * p.rows + r) * p.hk + h) * p.stride;
        choose = L > n;
        ask = choose && (p.sinks > 0 || p.recent > 0);
        last = end - p.recent;
    }
    // Reports for its row, by one thread of one list; false where the row is skipped.
    __device__ __forceinline__ bool good(const Params& p, bool reports) const {
        const bool bad = L < 0 || L > p.limit;
        if (reports && layer == 0 && h == 0) {
            if (bad)
                flag_error(p.dev_err, PKV_DEV_ERR_SEQ_LEN);
            else if (p.new_lens)
                p.new_lens[r] = n;
        }
        return !bad;
    }
    // The keys of tokens t .. t + 3 below `to` (0 for the others); what stays below n is copied
    // where the outputs lie elsewhere.
    __device__ __forceinline__ uint4 load(const Params& p, int t, int to) const {
        float w[4] = {0.f, 0.f, 0.f, 0.f};
        int pos[4] = {0, 0, 0, 0};
        const bool told = t < trk && t < to && (ask || (t < n && !p.in_place));  // positions are read
        if (p.vec4) {
            if (t < to) *reinterpret_cast<float4*>(w) = *reinterpret_cast<const float4*>(p.weights + base + t);
            if (told) *reinterpret_cast<int4*>(pos) = *reinterpret_cast<const int4*>(p.token_pos + base + t);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (t + j < to) w[j] = p.weights[base + t + j];
                if (told && t + j < trk) pos[j] = p.token_pos[base + t + j];
            }
        }
        uint32_t key[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (t + j >= trk) pos[j] = end - L + t + j;
            key[j] = t + j >= to ? 0u : ask && (pos[j] < p.sinks || pos[j] >= last) ? kSafe : key_of(w[j]);
        }
        if (p.vec4 && !p.in_place && t + 4 <= min(to, n)) {
            *reinterpret_cast<float4*>(p.weights_out + base + t) = *reinterpret_cast<const float4*>(w);
            *reinterpret_cast<int4*>(p.pos_out + base + t) = *reinterpret_cast<const int4*>(pos);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (t + j < min(to, n) && (!p.in_place || t + j >= trk)) {
                    p.pos_out[base + t + j] = pos[j];
                    if (!p.in_place) p.weights_out[base + t + j] = w[j];
                }
        }
        return make_uint4(key[0], key[1], key[2], key[3]);
    }
};

// The list's moves, 32 at a time to a warp, warps `first`, `first` + `step`, ...:
// entry(j, false) is the j-th slot that loses its token, entry(j, true) the token that
// takes it.  A lane finds one move's slots and moves its weight and position; then
// the warp moves the vectors, g lanes a token, kBatch of them in flight a lane.
template <class F>
__device__ __forceinline__ void move_tokens(const Params& p, const List& l, int moves, int first, int step, F&& entry) {
    const int lane = threadIdx.x & 31;
    const int32_t* row = p.tables + (int64_t)l.r * p.mbpr;
    const int64_t layer0 = (int64_t)l.layer * p.nb * p.bs;
    int g = 32;
    while (g >= 4 * p.vecs) g >>= 1;
    const int sub = lane / g, c0 = lane % g, at_once = 32 / g;
#pragma unroll 1
    for (int j0 = first * 32; j0 < moves; j0 += step * 32) {
        const int j = j0 + lane;
        int src = -1, dst = -1;
        if (j < moves) {
            const int to = entry(j, false), from = entry(j, true);
            src = slot_of(p, row, from);
            dst = slot_of(p, row, to);
            p.weights_out[l.base + to] = p.weights[l.base + from];
            p.pos_out[l.base + to] = from < l.trk ? p.token_pos[l.base + from] : l.end - l.L + from;
            if (src < 0 || dst < 0) {
                flag_error(p.dev_err, PKV_DEV_ERR_BLOCK_ID);
                src = -1;
            }
        }
        const int got = min(32, moves - j0);
#pragma unroll 1
        for (int i0 = 0; i0 < got; i0 += kBatch * at_once) {
#pragma unroll 1
            for (int cc = 0; cc < 2 * p.vecs; cc += g) {
                const int c = cc + c0;
                const bool is_v = c >= p.vecs;
                uint4* pool = is_v ? p.v_pool : p.k_pool;
                const int col = is_v ? c - p.vecs : c;
                uint4 x[kBatch];
                int64_t to[kBatch];
#pragma unroll
                for (int k = 0; k < kBatch; ++k) {
                    const int i = i0 + k * at_once + sub;
                    const int s = __shfl_sync(0xffffffffu, src, i & 31), d = __shfl_sync(0xffffffffu, dst, i & 31);
                    to[k] = -1;
                    if (i < got && s >= 0 && c < 2 * p.vecs) {
                        to[k] = ((layer0 + d) * p.hk + l.h) * p.vecs + col;
                        x[k] = pool[((layer0 + s) * p.hk + l.h) * p.vecs + col];
                    }
                }
#pragma unroll
                for (int k = 0; k < kBatch; ++k)
                    if (to[k] >= 0) pool[to[k]] = x[k];
            }
        }
    }
}

// kThreads a block, kBlocks blocks an SM; kCluster: p.blocks blocks a list.
template <int kThreads, int kBlocks, bool kCluster>
__global__ void __launch_bounds__(kThreads, kBlocks) evict_kernel(const __grid_constant__ Params p) {
    constexpr int kWarps = kThreads / 32, kPer = kBins / kThreads;
    constexpr int kRounds = (kThreads == kLongThreads ? kMostChunk : kShort) / (4 * kThreads);  // of 128 tokens a warp, at most
    extern __shared__ uint4 dyn[];
    uint32_t* keys = reinterpret_cast<uint32_t*>(dyn);             // [cap]
    uint16_t* list = reinterpret_cast<uint16_t*>(keys + p.cap);    // [cap]: holes from the front, fillers from the back
    __shared__ __align__(16) uint32_t hist[kBins];
    __shared__ __align__(16) uint32_t all[kCluster ? kBins : 4];   // the cluster's
    // A row of the warps' sums a use (0: protected, then bins; 1: equal keys; 2: holes | fillers << 16): where
    // exactly the protected stay, nothing but this keeps one use's reads from the next one's writes.
    __shared__ uint32_t sums[3][kWarps], ors[kWarps], ands[kWarps];
    __shared__ uint32_t found[3];   // digit (in the end the key), keys above it, keys in it
    __shared__ uint32_t few[32];    // keys that share the digits, when they are few
    __shared__ uint32_t mine[4];    // this block's: or (or the number of `few`), and, protected; equal keys, then holes | fillers << 16
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = kCluster ? (int)block_rank() : 0, blocks = kCluster ? p.blocks : 1;
    for (int i = tid; i < kBins / 4; i += kThreads) reinterpret_cast<uint4*>(hist)[i] = make_uint4(0, 0, 0, 0);
    if (tid == 0) mine[0] = 0;
    ptx::griddep_wait();
    const List l(p, kCluster ? (int)blockIdx.x / blocks : (int)blockIdx.x);
    if (!l.good(p, rank == 0 && tid == 0)) return;
    const int per = ((l.L + blocks - 1) / blocks + 3) & ~3;       // tokens of a block
    const int b0 = min(l.L, rank * per), cnt = min(l.L - b0, per);
    // Rounds of 128 tokens, this warp's next to each other (1025 tokens, four warps: 3, 2, 2, 2).
    const int all_rounds = (cnt + 127) / 128, extra = all_rounds % kWarps;
    const int rounds = all_rounds / kWarps + (warp < extra);
    const int w0 = (all_rounds / kWarps * warp + min(warp, extra)) * 128 + 4 * lane;  // this lane's first token, from b0 on

    // ---- keys; the bits in which they differ; how many are protected ----
    uint32_t any = 0, every = ~0u, safe = 0;
#pragma unroll 4
    for (int i = 0; i < rounds; ++i) {
        const int x = w0 + 128 * i;
        const uint4 k = l.load(p, b0 + x, b0 + cnt);
        *reinterpret_cast<uint4*>(keys + x) = k;
        const uint32_t ks[4] = {k.x, k.y, k.z, k.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const bool guarded = ks[j] == kSafe;
            safe += guarded;
            any |= guarded ? 0u : ks[j];
            every &= ks[j] == 0u ? ~0u : ks[j];  // the protected have every bit
        }
    }
    if (!l.choose) return;
    any = __reduce_or_sync(0xffffffffu, any);
    every = __reduce_and_sync(0xffffffffu, every);
    safe = __reduce_add_sync(0xffffffffu, safe);
    if (lane == 0) {
        ors[warp] = any;
        ands[warp] = every;
        sums[0][warp] = safe;
    }
    __syncthreads();
    safe = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        any |= ors[w];
        every &= ands[w];
        safe += sums[0][w];
    }
    if (kCluster) {
        if (tid == 0) {
            mine[0] = any;
            mine[1] = every;
            mine[2] = safe;
        }
        cluster_sync();
        // lane c asks block c
        const bool there = lane < blocks;
        const uint32_t a = there ? peer_word(ptx::smem_u32(mine), lane) : 0u;
        const uint32_t b = there ? peer_word(ptx::smem_u32(mine + 1), lane) : ~0u;
        const uint32_t c = there ? peer_word(ptx::smem_u32(mine + 2), lane) : 0u;
        any = __reduce_or_sync(0xffffffffu, a);
        every = __reduce_and_sync(0xffffffffu, b);
        safe = __reduce_add_sync(0xffffffffu, c);
    }

    // ---- the last key that stays: its digits from bit `shift` on are `prefix`, and of the
    // `equal` keys that share them the `need` of the lowest slots stay ----
    const uint32_t n = (uint32_t)l.n;
    const bool full = safe > n;  // more are protected than may stay (positions named twice)
    const uint32_t differ = any & ~every;
    int shift = full || safe == n ? 0 : 32 - __clz(differ);
    uint32_t prefix = full || safe == n ? kSafe : shift < 32 ? every >> shift : 0u;
    uint32_t need = full ? n : n - safe, equal = full ? safe : need ? (uint32_t)l.L - safe : 0u;
    // The first and the last key that share the digits; no key of a missing token and no
    // protected one but where those are chosen from.
    uint32_t lo, hi;
    auto bounds = [&] {
        lo = shift < 32 ? prefix << shift : 0u;
        hi = shift < 32 ? lo | ((1u << shift) - 1) : ~0u;
        if (!full && hi == kSafe) --hi;
        if (lo == 0) lo = 1;
    };
    bounds();
#pragma unroll 1
    while (need < equal && shift > 0) {
        const int above = shift;
        shift = max(0, above - kDigit);
        const uint32_t mask = (1u << (above - shift)) - 1;
#pragma unroll 2
        for (int i = 0; i < rounds; ++i) {
            const uint4 k = *reinterpret_cast<const uint4*>(keys + w0 + 128 * i);
            const uint32_t ks[4] = {k.x, k.y, k.z, k.w};
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (ks[j] - lo <= hi - lo) atomicAdd(&hist[ks[j] >> shift & mask], 1u);
        }
        if (kCluster) {
            cluster_sync();
            // each block adds up its slice of the bins, then takes the other blocks' slices
            const int slice = kBins / blocks;
            for (int i = tid; i < slice; i += kThreads) {
                const int b = rank * slice + i;
                uint32_t x[kMostBlocks], t = 0;  // (asked for together)
#pragma unroll
                for (int c = 0; c < kMostBlocks; ++c) x[c] = c < blocks ? peer_word(ptx::smem_u32(hist + b), c) : 0u;
#pragma unroll
                for (int c = 0; c < kMostBlocks; ++c) t += x[c];
                all[b] = t;
            }
            cluster_sync();
            uint32_t x[kPer];
#pragma unroll
            for (int j = 0; j < kPer; ++j) {
                const int b = tid + j * kThreads;
                x[j] = peer_word(ptx::smem_u32(all + b), b / slice);
            }
#pragma unroll
            for (int j = 0; j < kPer; ++j) {
                const int b = tid + j * kThreads;
                if (b / slice != rank) all[b] = x[j];
                hist[b] = 0;
            }
            cluster_sync();
        } else {
            __syncthreads();
        }
        // thread i: kPer bins, the first thread the highest ones
        uint32_t c[kPer], sum = 0;
        uint32_t* bins = (kCluster ? all : hist) + kBins - kPer * (tid + 1);
#pragma unroll
        for (int j = 0; j < kPer; ++j) sum += c[j] = bins[j];
        if (!kCluster) {
#pragma unroll
            for (int j = 0; j < kPer; ++j) bins[j] = 0;
        }
        uint32_t over = lanes_before(sum);
        if (lane == 31) sums[0][warp] = over + sum;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kWarps; ++w) over += w < warp ? sums[0][w] : 0u;
        if (over < need && need <= over + sum) {
#pragma unroll
            for (int j = kPer - 1; j >= 0; --j) {
                if (over < need && need <= over + c[j]) {
                    found[0] = (uint32_t)(kBins - kPer * (tid + 1) + j);
                    found[1] = over;
                    found[2] = c[j];
                }
                over += c[j];
            }
        }
        __syncthreads();
        prefix = above == 32 ? found[0] : prefix << (above - shift) | found[0];
        need -= found[1];
        equal = found[2];
        bounds();
        if (!kCluster && equal <= 32 && need < equal && shift > 0) {
            // few share the digits: a warp ranks them
#pragma unroll 2
            for (int i = 0; i < rounds; ++i) {
                const uint4 k = *reinterpret_cast<const uint4*>(keys + w0 + 128 * i);
                const uint32_t ks[4] = {k.x, k.y, k.z, k.w};
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (ks[j] - lo <= hi - lo) few[atomicAdd(&mine[0], 1u)] = ks[j];
            }
            __syncthreads();
            if (warp == 0) {
                const uint32_t k = lane < (int)equal ? few[lane] : 0u;
                uint32_t larger = 0, like = 0;
                for (int j = 0; j < (int)equal; ++j) {
                    const uint32_t x = __shfl_sync(0xffffffffu, k, j);
                    larger += x > k;
                    like += x == k;
                }
                if (k && larger < need && need <= larger + like) {  // lanes of one key write the same
                    found[0] = k;
                    found[1] = larger;
                    found[2] = like;
                }
            }
            __syncthreads();
            shift = 0;
            prefix = found[0];
            need -= found[1];
            equal = found[2];
            bounds();
        }
    }

    // ---- which of the equal keys stay: the first `left` from this warp's first on ----
    uint32_t left = ~0u;
    if (need < equal) {
        uint32_t eq = 0;
#pragma unroll 2
        for (int i = 0; i < rounds; ++i) {
            const uint4 k = *reinterpret_cast<const uint4*>(keys + w0 + 128 * i);
            eq += (k.x - lo <= hi - lo) + (k.y - lo <= hi - lo) + (k.z - lo <= hi - lo) + (k.w - lo <= hi - lo);
        }
        eq = __reduce_add_sync(0xffffffffu, eq);
        if (lane == 0) sums[1][warp] = eq;
        __syncthreads();
        uint32_t before = 0, total = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            before += w < warp ? sums[1][w] : 0u;
            total += sums[1][w];
        }
        if (kCluster) {
            if (tid == 0) mine[3] = total;
            cluster_sync();
            before += __reduce_add_sync(0xffffffffu, lane < rank ? peer_word(ptx::smem_u32(mine + 3), lane) : 0u);
            cluster_sync();  // mine[3] is written again below
        }
        left = before < need ? need - before : 0u;
    }
    // ---- this lane's tokens that move or make room: four bits a round ----
    uint64_t flags = 0;
    uint32_t count = 0;  // holes | fillers << 16
    const uint32_t least = left == ~0u ? lo : hi + 1;  // this key and all above stay (0: none is above)
    const int border = min(l.n, b0 + cnt) - b0;        // slots below it lose what does not stay
#pragma unroll 2
    for (int i = 0; i < rounds; ++i) {
        const int x = w0 + 128 * i;
        const uint4 k = *reinterpret_cast<const uint4*>(keys + x);
        const uint32_t ks[4] = {k.x, k.y, k.z, k.w};
        uint32_t stay = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) stay |= ks[j] >= least && least ? 1u << j : 0u;
        if (left != ~0u) {
            uint32_t tie = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) tie |= ks[j] - lo <= hi - lo ? 1u << j : 0u;
            if (__any_sync(0xffffffffu, tie != 0)) {
                const uint32_t here = __popc(tie), before = lanes_before(here);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if ((tie >> j & 1) && before + __popc(tie & ((1u << j) - 1)) < left) stay |= 1u << j;
                left -= min(left, __shfl_sync(0xffffffffu, before + here, 31));
            }
        }
        const int below = min(4, max(0, border - x));
        const uint32_t low = (1u << below) - 1, hole = low & ~stay, fill = stay & ~low;
        flags |= (uint64_t)(hole | fill) << (4 * i);
        count += __popc(hole) | __popc(fill) << 16;
    }
    static_assert(4 * kRounds <= 64, "a lane's flags fit");
    const uint32_t sum = __reduce_add_sync(0xffffffffu, count);
    if (lane == 0) sums[2][warp] = sum;
    __syncthreads();
    uint32_t at = 0, total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        at += w < warp ? sums[2][w] : 0u;
        total += sums[2][w];
    }
#pragma unroll 1
    for (int i = 0; i < rounds; ++i) {
        const uint32_t f = (uint32_t)(flags >> (4 * i)) & 15u;
        if (!__any_sync(0xffffffffu, f != 0)) continue;
        const int x = w0 + 128 * i;
        const uint32_t low = (1u << min(4, max(0, border - x))) - 1;
        const uint32_t c = __popc(f & low) | __popc(f & ~low) << 16, before = lanes_before(c);
        uint32_t ho = (at + before) & 0xffffu, fo = (at + before) >> 16;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (f >> j & 1) list[low >> j & 1 ? ho++ : p.cap - 1 - fo++] = (uint16_t)(x + j);
        at += __shfl_sync(0xffffffffu, before + c, 31);
    }

    // ---- the moves, dealt to the warps of all blocks ----
    if (!kCluster) {
        __syncthreads();
        move_tokens(p, l, (int)(total & 0xffffu), warp, kWarps,
                    [&](int j, bool filler) { return (int)list[filler ? p.cap - 1 - j : j]; });
        return;
    }
    if (tid == 0) mine[3] = total;
    cluster_sync();
    uint32_t part[kMostBlocks];  // holes | fillers << 16 of each block
    int moves = 0;
#pragma unroll
    for (int c = 0; c < kMostBlocks; ++c) {
        part[c] = c < blocks ? peer_word(ptx::smem_u32(mine + 3), c) : 0u;
        moves += part[c] & 0xffffu;
    }
    move_tokens(p, l, moves, rank * kWarps + warp, blocks * kWarps, [&](int j, bool filler) {
        int c = 0;
#pragma unroll
        for (int k = 0; k < kMostBlocks - 1; ++k) {
            const int x = (int)(filler ? part[k] >> 16 : part[k] & 0xffffu);
            if (c == k && j >= x) {
                j -= x;
                ++c;
            }
        }
        return c * per + (int)peer_half(ptx::smem_u32(list + (filler ? p.cap - 1 - j : j)), c);
    });
    cluster_sync();  // the other blocks read this one's lists
}

}  // namespace evict
}  // namespace pkv

extern "C" int paged_kv_evict(void* k_pool, void* v_pool, const int32_t* block_tables, const int32_t* seq_lens,
                              const float* weights, const int32_t* token_pos, const int32_t* tracked,
                              const int32_t* next_pos, float* weights_out, int32_t* token_pos_out,
                              int32_t* new_seq_lens, int layers, int rows, int kv_heads, int head_dim,
                              int elt_bytes, int block_size, int max_blocks_per_row, int num_blocks,
                              int max_seq_len, int64_t weights_stride, int budget, int sinks, int recent,
                              int32_t* dev_err, cudaStream_t stream) {
    using namespace pkv;
    using namespace pkv::evict;
    if (layers < 0 || rows < 0 || kv_heads <= 0 || head_dim <= 0 || block_size <= 0 || max_blocks_per_row <= 0 ||
        num_blocks <= 0 || max_seq_len < 0 || (elt_bytes != 1 && elt_bytes != 2) || weights_stride < max_seq_len)
        return PKV_ERR_INVALID_ARG;
    if (budget < 1 || sinks < 0 || recent < 0 || (int64_t)sinks + recent > budget) return PKV_ERR_INVALID_ARG;
    if ((int64_t)max_seq_len > (int64_t)max_blocks_per_row * block_size) return PKV_ERR_INVALID_ARG;
    if ((int64_t)head_dim * elt_bytes % 16) return PKV_ERR_UNSUPPORTED;
    const int64_t vecs = (int64_t)head_dim * elt_bytes / 16;
    if (vecs > (1 << 16) || max_seq_len > kMostBlocks * kMostChunk ||
        (int64_t)num_blocks * block_size >= (int64_t(1) << 31))
        return PKV_ERR_UNSUPPORTED;
    if (layers == 0 || rows == 0) return PKV_OK;
    if (!k_pool || !v_pool || !block_tables || !seq_lens || !weights || !token_pos || !weights_out ||
        !token_pos_out)
        return PKV_ERR_INVALID_ARG;
    if (!aligned16(k_pool) || !aligned16(v_pool)) return PKV_ERR_INVALID_ARG;
    const int64_t lists = (int64_t)layers * rows * kv_heads;
    if (rows > 65535 || layers > 65535 || kv_heads > 0x7fffffff / kMostBlocks ||
        weights_stride > (int64_t(1) << 40) / lists)
        return PKV_ERR_UNSUPPORTED;
    // In place both or neither; apart from that no output lies over an input or another output.
    const bool in_place = weights_out == weights;
    if (in_place != (token_pos_out == token_pos)) return PKV_ERR_INVALID_ARG;
    const size_t wide = (size_t)lists * weights_stride * 4, n = (size_t)rows * 4;
    struct Span {
        const void* at;
        size_t bytes;
    };
    // (a pool of more bytes than there are addresses reaches to the last one)
    const double slots = (double)layers * num_blocks * block_size, pool_bytes = slots * kv_heads * (double)(vecs * 16);
    auto pool = [&](const void* at) {
        const size_t rest = ~reinterpret_cast<uintptr_t>(at);
        return Span{at, pool_bytes < 1e18 && (size_t)pool_bytes < rest ? (size_t)pool_bytes : rest};
    };
    const Span outs[] = {{weights_out, wide}, {token_pos_out, wide}, {new_seq_lens, n}};
    const Span ins[] = {{weights, wide}, {token_pos, wide}, {seq_lens, n},  {block_tables, n * max_blocks_per_row},
                        {tracked, n},    {next_pos, n},     pool(k_pool),   pool(v_pool), {dev_err, 4}};
    for (int o = 0; o < 3; ++o) {
        if (!outs[o].at) continue;
        for (int i = 0; i < 9; ++i) {
            if (!ins[i].at || (in_place && o == i && o < 2)) continue;
            if (overlap(outs[o].at, outs[o].bytes, ins[i].at, ins[i].bytes)) return PKV_ERR_INVALID_ARG;
        }
        for (int q = 0; q < o; ++q)
            if (overlap(outs[o].at, outs[o].bytes, outs[q].at, outs[q].bytes)) return PKV_ERR_INVALID_ARG;
    }

    Params p{};
    p.k_pool = static_cast<uint4*>(k_pool);
    p.v_pool = static_cast<uint4*>(v_pool);
    p.tables = block_tables;
    p.seq_lens = seq_lens;
    p.weights = weights;
    p.token_pos = token_pos;
    p.tracked = tracked;
    p.next_pos = next_pos;
    p.weights_out = weights_out;
    p.pos_out = token_pos_out;
    p.new_lens = new_seq_lens;
    p.stride = weights_stride;
    p.rows = rows;
    p.hk = kv_heads;
    p.vecs = (int)vecs;
    p.bs = block_size;
    p.mbpr = max_blocks_per_row;
    p.nb = num_blocks;
    p.limit = max_seq_len;
    p.budget = budget;
    p.sinks = sinks;
    p.recent = recent;
    p.in_place = in_place;
    p.dev_err = dev_err;
    p.vec4 = weights_stride % 4 == 0 && aligned16(weights) && aligned16(token_pos) && aligned16(weights_out) &&
             aligned16(token_pos_out);
    // Many small lists want many blocks resident (1792 of 1025 tokens: 17.9 us with 128 threads, 24.6
    // with 256), larger ones more warps for their moves (896 of 1900 to 2304, E4M3: 28.3 and 23.2), and
    // clusters of large blocks do not pay at such lengths (the same 896: 86.9).  Long lists: a cluster of
    // blocks of up to kChunk tokens, as long as all blocks are resident at once.  32 lists of 16,384 to
    // 2048: two blocks 40.2 us, four 27.5, eight 32.4; 128 of them: two 61.6, four 72.3; 224: one 109.7, two
    // 113.7, four 124.3; 224 of 8192 to 1024: one 48.9, two 65.1, four 93.2; 32 of 8192: two 22.2, four 20.8.
    const bool is_small = max_seq_len <= kSmall, is_short = max_seq_len <= kShort;
    p.blocks = 1;
    const int sms = device_sms();
    if (sms <= 0) return PKV_ERR_CUDA;
    const int64_t resident = (int64_t)sms * kLongBlocks;
    while (!is_short && p.blocks < kMostBlocks) {
        const int chunk = (max_seq_len + p.blocks - 1) / p.blocks;
        if (chunk <= kMostChunk && (chunk <= kChunk || lists * 2 * p.blocks > resident)) break;
        p.blocks *= 2;
    }
    // whole rounds of a block's warps; a block's share is a multiple of four tokens
    const int threads = is_small ? kSmallThreads : is_short ? kShortThreads : kLongThreads, round = 4 * threads;
    p.cap = (((max_seq_len + p.blocks - 1) / p.blocks + 3) / 4 * 4 + round - 1) / round * round;
    const size_t smem = (size_t)p.cap * 6;
    const dim3 grid((unsigned)(kv_heads * p.blocks), (unsigned)rows, (unsigned)layers);
    if (is_small)
        return launch_early(evict_kernel<kSmallThreads, kSmallBlocks, false>, grid, threads, smem, stream, p);
    if (is_short)
        return launch_early(evict_kernel<kShortThreads, kShortBlocks, false>, grid, threads, smem, stream, p);
    auto* kernel = p.blocks > 1 ? evict_kernel<kLongThreads, kLongBlocks, true>
                                : evict_kernel<kLongThreads, kLongBlocks, false>;
    if (smem > 32768 &&
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostChunk * 6) != cudaSuccess) {
        cudaGetLastError();
        return PKV_ERR_CUDA;
    }
    return launch_early_clusters(kernel, grid, threads, smem, (unsigned)p.blocks, stream, p);
}
