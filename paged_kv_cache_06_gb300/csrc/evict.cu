// paged_kv_evict: of each list (layer, row, KV head) the tokens of lowest weight
// leave the cache and the others move together, every layer at once.
//
// Mathematics.  A list of L tokens keeps n = min(L, budget): those that are
// protected (the row's first `sinks` positions and last `recent`), then the ones of
// the largest weight, the lowest slot first where weights are equal.  Weights become 32-bit
// keys whose unsigned order is the weights' order (protected tokens take the
// largest key), and the n-th largest key is found digit by digit, 11 bits at a
// time from the top: a histogram of the digit over the keys that share the digits so
// far, summed from the top, gives the next digit and how many keys lie above it.
// Nothing is sorted: tokens that stay and lie below n stay where they are, and
// the j-th slot below n that loses its token takes the j-th token that stays from n on.
// Sources lie at n or past it and destinations below it, so the moves have
// no order among themselves, and there are as few as can be: the tokens that leave, not
// the tokens that stay.
//
// Work.  A cluster of thread blocks takes a list, one block where it has at most
// kChunk tokens; every block holds its share of the keys in shared memory, and the
// histograms and counts of the blocks are added up through distributed shared
// memory.  The cluster's moves are then dealt to its blocks evenly, 32 at a time to a
// warp: a lane finds one move's slots through the table and moves its weight and
// position, then the warp moves the keys and values, several moves' vectors in
// flight a lane.
#include "pkv_internal.cuh"
#include "ptx.cuh"

namespace pkv {
namespace evict {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kChunk = 4096;      // tokens of a block, while a cluster may still grow
constexpr int kMostBlocks = 8;    // of a cluster (the portable limit)
constexpr int kMostChunk = 24576;  // tokens of a block, at most: 8 bytes of shared memory each
constexpr int kBins = 2048;       // 11-bit digits
constexpr int kBatch = 4;         // vectors in flight a lane
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
    int cap;     // tokens of a block
    int in_place;
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
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The word at shared address `addr` of block `rank` of the cluster.
__device__ __forceinline__ uint32_t peer_word(uint32_t addr, int rank) {
    uint32_t a, v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(rank));
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    return v;
}

// Exclusive prefix over the block's threads, in thread order, and the total.
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t* warp_sums, uint32_t& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t t = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += t;
    }
    if (lane == 31) warp_sums[warp] = incl;
    __syncthreads();
    uint32_t w = lane < kWarps ? warp_sums[lane] : 0u;
#pragma unroll
    for (int o = 1; o < kWarps; o <<= 1) {
        const uint32_t t = __shfl_up_sync(0xffffffffu, w, o);
        if (lane >= o) w += t;
    }
    total = __shfl_sync(0xffffffffu, w, kWarps - 1);
    const uint32_t before = __shfl_sync(0xffffffffu, w, warp > 0 ? warp - 1 : 0);
    __syncthreads();  // the sums may be overwritten
    return incl - v + (warp > 0 ? before : 0u);
}

// The slot of a row's token in the pools, or -1 for a bad table entry.
__device__ __forceinline__ int slot_of(const Params& p, const int32_t* row, int t) {
    const int lb = t / p.bs, pb = row[lb];
    return pb < 0 || pb >= p.nb ? -1 : pb * p.bs + (t - lb * p.bs);
}

template <bool kCluster>
__global__ void __launch_bounds__(kThreads) evict_kernel(const __grid_constant__ Params p) {
    extern __shared__ uint32_t dyn[];
    uint32_t* keys = dyn;           // [cap]
    uint32_t* list = dyn + p.cap;   // [cap]: holes from the front, the tokens that fill them from the back
    __shared__ uint32_t hist[kBins], all[kCluster ? kBins : 1];
    __shared__ uint32_t warp_sums[kWarps];
    __shared__ uint32_t found[3];   // digit, keys above it, keys in it
    __shared__ uint32_t counts[2];  // this block's: equal keys; holes | fillers << 16
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = kCluster ? (int)block_rank() : 0, blocks = kCluster ? p.blocks : 1;
    const int li = (int)(blockIdx.x / (unsigned)blocks);  // (layer, row, head)
    const int h = li % p.hk, lr = li / p.hk, r = lr % p.rows, layer = lr / p.rows;
    const bool first = layer == 0 && h == 0 && rank == 0;  // reports for its row
    auto all_sync = [] {
        if (kCluster)
            cluster_sync();
        else
            __syncthreads();
    };

    ptx::griddep_wait();
    const int L = p.seq_lens[r];
    if (L < 0 || L > p.limit) {
        if (first && tid == 0) flag_error(p.dev_err, PKV_DEV_ERR_SEQ_LEN);
        return;
    }
    const int n = min(L, p.budget);
    if (first && tid == 0 && p.new_lens) p.new_lens[r] = n;
    const int trk = p.tracked ? max(0, min(p.tracked[r], L)) : 0;
    const int end = p.next_pos ? p.next_pos[r] : L;  // the next token's position
    const int64_t base = (int64_t)li * p.stride;
    const float* wts = p.weights + base;
    const int32_t* tps = p.token_pos + base;
    float* wts_out = p.weights_out + base;
    int32_t* pos_out = p.pos_out + base;
    const int per = (L + blocks - 1) / blocks, t0 = min(L, rank * per), cnt = min(L - t0, per);
    const bool choose = L > n;
    const bool ask = choose && (p.sinks > 0 || p.recent > 0);  // whether positions matter
    const int last = end - p.recent;                           // the first protected position

    // ---- keys; what stays below n is copied where the outputs lie elsewhere ----
#pragma unroll 4
    for (int i = tid; i < cnt; i += kThreads) {
        const int t = t0 + i;
        const float w = wts[t];
        const bool keep_out = t < n && (!p.in_place || t >= trk);
        int pos = end - L + t;
        if (t < trk && (ask || keep_out)) pos = tps[t];
        if (choose) keys[i] = ask && (pos < p.sinks || pos >= last) ? kSafe : key_of(w);
        if (keep_out) {
            pos_out[t] = pos;
            if (!p.in_place) wts_out[t] = w;
        }
    }
    if (!choose) return;

    // ---- the n-th largest key, digit by digit ----
    uint32_t prefix = 0, need = (uint32_t)n;  // of the keys that share the digits so far, `need` stay
    int shift = 32;
    uint32_t equal = (uint32_t)L;             // keys that share the digits
#pragma unroll 1
    for (int pass = 0; pass < 3 && need < equal; ++pass) {
        const int bits = pass < 2 ? 11 : 10, above = shift;
        shift -= bits;
        const uint32_t mask = (1u << bits) - 1;
        for (int i = tid; i < kBins; i += kThreads) hist[i] = 0;
        __syncthreads();
        for (int i = warp * 32; i < cnt; i += kThreads) {
            const uint32_t k = i + lane < cnt ? keys[i + lane] : 0u;
            const bool in = i + lane < cnt && (pass == 0 || k >> above == prefix);
            // the protected, which come in a row, are counted a warp at a time
            const unsigned safe = __ballot_sync(0xffffffffu, in && k == kSafe);
            if (safe && lane == 0) atomicAdd(&hist[mask], __popc(safe));
            if (in && k != kSafe) atomicAdd(&hist[k >> shift & mask], 1u);
        }
        all_sync();
        if (kCluster) {
            // each block adds up its slice of the bins, then takes the other blocks' slices
            const int slice = kBins / blocks;
            for (int i = tid; i < slice; i += kThreads) {
                const int b = rank * slice + i;
                uint32_t s = 0;
                for (int c = 0; c < blocks; ++c) s += peer_word(ptx::smem_u32(hist + b), c);
                all[b] = s;
            }
            cluster_sync();
            for (int b = tid; b < kBins; b += kThreads)
                if (b / slice != rank) all[b] = peer_word(ptx::smem_u32(all + b), b / slice);
            cluster_sync();
        }
        // thread i: four bins, the first thread the highest ones
        constexpr int kPer = kBins / kThreads;
        const uint32_t* h4 = (kCluster ? all : hist) + kBins - kPer * (tid + 1);
        uint32_t c[kPer], sum = 0, total;
#pragma unroll
        for (int j = 0; j < kPer; ++j) sum += c[j] = h4[j];
        uint32_t over = block_scan(sum, warp_sums, total);
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
        prefix = pass == 0 ? found[0] : prefix << bits | found[0];
        need -= found[1];
        equal = found[2];
    }
    // Keys above `prefix` stay; of those that share it the `need` of the lowest slots do.
    const int m = ((cnt + kThreads - 1) / kThreads) | 1;  // a thread's tokens; odd, so that banks differ
    const int a = min(cnt, tid * m), b = min(cnt, a + m);
    uint32_t left = ~0u;  // how many more of the equal keys stay, from this thread's first on
    if (need < equal) {
        uint32_t eq = 0, total;
        for (int i = a; i < b; ++i) eq += keys[i] >> shift == prefix;
        uint32_t before = block_scan(eq, warp_sums, total);
        if (kCluster) {
            if (tid == 0) counts[0] = total;
            cluster_sync();
            for (int c = 0; c < rank; ++c) before += peer_word(ptx::smem_u32(counts), c);
        }
        left = before < need ? need - before : 0u;
    }
    auto stays = [&](uint32_t k) {
        const uint32_t d = shift < 32 ? k >> shift : 0u;
        if (d != prefix) return d > prefix;
        if (left == 0) return false;
        --left;
        return true;
    };
    const uint32_t left0 = left;
    uint32_t mine = 0, total;
    for (int i = a; i < b; ++i) {
        const bool s = stays(keys[i]), low = t0 + i < n;
        mine += low ? !s : (uint32_t)s << 16;
    }
    left = left0;
    const uint32_t at = block_scan(mine, warp_sums, total);
    uint32_t ho = at & 0xffffu, fo = at >> 16;
    for (int i = a; i < b; ++i) {
        const bool s = stays(keys[i]), low = t0 + i < n;
        if (low && !s) list[ho++] = (uint32_t)(t0 + i);
        if (!low && s) list[p.cap - 1 - fo++] = (uint32_t)(t0 + i);
    }
    if (tid == 0) counts[1] = total;
    all_sync();

    // ---- the moves, dealt to the blocks evenly ----
    uint32_t sums[kMostBlocks];  // holes | fillers << 16 of each block
    int moves = 0;
#pragma unroll
    for (int c = 0; c < kMostBlocks; ++c) {
        sums[c] = 0;
        if (c < blocks) sums[c] = kCluster ? peer_word(ptx::smem_u32(counts + 1), c) : counts[1];
        moves += sums[c] & 0xffffu;
    }
    auto entry = [&](int j, bool filler) -> int {  // token of the j-th hole or filler
        if (!kCluster) return (int)list[filler ? p.cap - 1 - j : j];
        int c = 0;
#pragma unroll
        for (int k = 0; k < kMostBlocks - 1; ++k) {
            const int x = (int)(filler ? sums[k] >> 16 : sums[k] & 0xffffu);
            if (c == k && j >= x) {
                j -= x;
                ++c;
            }
        }
        return (int)peer_word(ptx::smem_u32(list + (filler ? p.cap - 1 - j : j)), c);
    };
    const int32_t* row = p.tables + (int64_t)r * p.mbpr;
    const int64_t layer0 = (int64_t)layer * p.nb * p.bs;
    int g = 32;  // lanes of a move
    while (g >= 4 * p.vecs) g >>= 1;
    const int sub = lane / g, c0 = lane % g;
    const int groups = (moves + 31) / 32;
#pragma unroll 1
    for (int w = rank * kWarps + warp; w < groups; w += blocks * kWarps) {
        const int j = w * 32 + lane;
        int src = -1, dst = -1;
        if (j < moves) {
            const int to = entry(j, false), from = entry(j, true);
            wts_out[to] = wts[from];
            pos_out[to] = from < trk ? tps[from] : end - L + from;
            src = slot_of(p, row, from);
            dst = slot_of(p, row, to);
            if (src < 0 || dst < 0) {
                flag_error(p.dev_err, PKV_DEV_ERR_BLOCK_ID);
                src = -1;
            }
        }
        const int got = min(32, moves - w * 32);
        for (int i0 = 0; i0 < got; i0 += kBatch * (32 / g)) {
            for (int cc = 0; cc < 2 * p.vecs; cc += g) {
                const int c = cc + c0;
                const bool is_v = c >= p.vecs;
                uint4* pool = is_v ? p.v_pool : p.k_pool;
                const int col = is_v ? c - p.vecs : c;
                uint4 x[kBatch];
                int64_t to[kBatch];
#pragma unroll
                for (int k = 0; k < kBatch; ++k) {
                    const int i = i0 + k * (32 / g) + sub;
                    const int s = __shfl_sync(0xffffffffu, src, i & 31), d = __shfl_sync(0xffffffffu, dst, i & 31);
                    to[k] = -1;
                    if (i < got && s >= 0 && c < 2 * p.vecs) {
                        to[k] = ((layer0 + d) * p.hk + h) * p.vecs + col;
                        x[k] = pool[((layer0 + s) * p.hk + h) * p.vecs + col];
                    }
                }
#pragma unroll
                for (int k = 0; k < kBatch; ++k)
                    if (to[k] >= 0) pool[to[k]] = x[k];
            }
        }
    }
    if (kCluster) cluster_sync();  // the other blocks read this one's lists
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
    if (lists > 0x7fffffff / kMostBlocks || weights_stride > (int64_t(1) << 40) / lists) return PKV_ERR_UNSUPPORTED;
    // In place both or neither; apart from that no output lies over an input or another output.
    const bool in_place = weights_out == weights;
    if (in_place != (token_pos_out == token_pos)) return PKV_ERR_INVALID_ARG;
    const size_t wide = (size_t)lists * weights_stride * 4, n = (size_t)rows * 4;
    struct Span {
        const void* at;
        size_t bytes;
    };
    const Span outs[] = {{weights_out, wide}, {token_pos_out, wide}, {new_seq_lens, n}};
    const Span ins[] = {{weights, wide},  {token_pos, wide}, {seq_lens, n}, {block_tables, n * max_blocks_per_row},
                        {tracked, n},     {next_pos, n}};
    for (int o = 0; o < 3; ++o) {
        if (!outs[o].at) continue;
        for (int i = 0; i < 6; ++i) {
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
    p.blocks = 1;
    while (p.blocks < kMostBlocks && (max_seq_len + p.blocks - 1) / p.blocks > kChunk) p.blocks *= 2;
    p.cap = (max_seq_len + p.blocks - 1) / p.blocks;
    const size_t smem = (size_t)p.cap * 8;
    auto* kernel = p.blocks > 1 ? evict_kernel<true> : evict_kernel<false>;
    if (smem > 24576 && cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostChunk * 8) !=
                            cudaSuccess) {
        cudaGetLastError();
        return PKV_ERR_CUDA;
    }
    return launch_early_clusters(kernel, (unsigned)(lists * p.blocks), kThreads, smem, (unsigned)p.blocks, stream, p);
}
