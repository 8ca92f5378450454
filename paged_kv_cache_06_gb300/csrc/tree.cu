// paged_attention_tree: attention of each row's drafted nodes over its cached
// tokens and the nodes that their mask lets them see, on the 5th-generation
// tensor cores (tcgen05, accumulators and probabilities in tensor memory).
//
// Mathematics.  The group = q_heads / kv_heads query heads of one KV head and
// all nodes of a row read the same keys, so they are the rows of one matrix
// product: flat row f stands for node f / group and head f % group of the
// group.  S = Q K^T, an online softmax in base 2 and 32 bits over tiles of 128
// tokens, O += P V; the mask only touches the tiles that hold nodes.
//
// Work.  A unit is 128 flat rows of one (row, KV head) and walks the row's
// tokens in 128-token tiles.  All units' 64-token granules, in (row, KV head,
// rows, token) order, are cut into equal contiguous ranges, one per block, one
// block per SM, whatever the mix of lengths (the host never reads them); a cut
// that falls within a few granules of a unit's border moves to it, which spares
// a partial result of 64 KB for a little imbalance.
//
// Units cut over P blocks.  Each piece stores its partial result (reference
// maxima, row sums, unnormalised output in 32 bits) and counts itself as
// arrived.  A block walks its range from the last unit to the first, so a piece
// that others continue is stored first, and merges last: its warps wait a
// little for the unit's other pieces and then claim jobs (some rows by eight
// dims), each merged over the pieces in order, so the result does not depend on
// who does it.  The block that arrives last waits for nobody and does whatever
// is unclaimed; the others give up after a while.  So no block's progress
// depends on another block running, and two calls can share the GPU.  The last
// warp to leave a unit sets its words back to zero.
//
// Warp roles (each walks the same segments):
//   warps 0-7   softmax: warps w and w + 4 share flat rows 32 (w % 4) .. (TMEM
//               lanes); half hf = w / 4 takes 64 of a tile's tokens and 64 of
//               the output's dims;
//   warp 8      queries (cp.async) and S issue;  warp 9  PV issue;
//   fp16 pools: warp 10 K tiles, warp 11 V halves, by TMA, one box of 16, 32 or
//               64 consecutive tokens of a page a copy;
//   FP8 pools:  warps 10-13 load the codes, widen them (exactly) to fp16 and
//               store them where a copy would have put them; the scales go into
//               the score scale and the normalisation.
// The rings (three K slots of 128 tokens, five V slots of 64) and the three S
// buffers are those of the prefill kernel, as are the bounded waits: a block
// that gives up flags the error, tells its other warps to stop, and lets its
// copies in flight land before it frees tensor memory.
//
// What is not seen.  Scores of tokens a flat row does not see become -inf
// before the maximum.  A weight of zero times an infinity or NaN in V would
// still reach the output, so in the tiles that hold nodes the softmax warps
// zero every element of a node's V that is no number (and the slots' rows past
// the last token); a node that does see such an element gets it added to its
// output afterwards.  Cached tokens are seen by every node of the row and need
// no such care.
#include <mutex>

#include "fp8_codec.cuh"
#include "pkv_internal.cuh"
#include "tcgen05.cuh"

namespace pkv {
namespace tree {
using namespace tc;

constexpr int kRows = 128;     // flat rows of a unit: TMEM lanes
constexpr int kTile = 128;     // tokens of a step
constexpr int kGranule = 64;   // tokens: the grain of the work split
constexpr int kKSlots = 3;     // K ring, 128 tokens a slot
constexpr int kVSlots = 5;     // V ring, 64 tokens a slot
constexpr int kSBufs = 3;      // S buffers in TMEM
constexpr int kSoftWarps = 8;
constexpr int kSIssue = 8, kPvIssue = 9, kLoad = 10;  // warp roles
constexpr int kConvWarps = 4;  // FP8: warps that load and widen
constexpr int kMaxRows = 1024;
constexpr int kMaxGrid = 192;  // blocks: one per SM, at most this many
constexpr int kMaxWords = 32;  // mask words: up to 1024 nodes a row
constexpr int kHeadInts = 32;  // ints between two units' words: arrived, next job, left
constexpr int kMinGranules = 4;  // of a block's range and of a moved cut
constexpr uint32_t kHalfQ = kRows * 128;      // 128 flat rows x 64 dims
constexpr uint32_t kKHalf = kTile * 128;      // 128 tokens x 64 dims
constexpr uint32_t kKSlot = 2 * kKHalf;
constexpr uint32_t kVHalf = 64 * 128;         // 64 tokens x 64 dims
constexpr uint32_t kVSlot = 2 * kVHalf;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColS = 0;    // S buffers [0, 128), [128, 256), [256, 384)
constexpr uint32_t kColO = 384;  // O [384, 512)
// A partial: m[128], l[128], then O as [32 groups of 4 dims][128 rows][4].
constexpr int kPartFloats = 2 * kRows + kRows * kHeadDim;
constexpr uint64_t kHelpNs = 100000;  // how long a block waits for a unit's other pieces
constexpr float kLog2e = 1.4426950408889634f;

template <bool kFp8>
__host__ __device__ constexpr int threads() { return (kLoad + (kFp8 ? kConvWarps : 2)) * 32; }

struct Params {
    const __half* q;
    __half* out;
    const void* k_pool;
    const void* v_pool;
    const float* k_scale;
    const float* v_scale;
    const int32_t* tables;
    const int32_t* seq_lens;
    const int32_t* q_start;
    const uint32_t* mask;
    int words;
    int rows, total, hq, hk, group, bs, mbpr, nb, limit;
    int box;       // tokens per copy
    float scale;
    int out_v8;    // out is 32-byte aligned: 32-byte stores
    float* part;   // [grid][2][kPartFloats]
    int* heads;    // [grid][kHeadInts], zero between calls: of the cut unit that starts in a block
    int32_t* dev_err;
};

struct Smem {
    static constexpr uint32_t q = 0;                               // Q lo, Q hi
    static constexpr uint32_t kring = q + 2 * kHalfQ;
    static constexpr uint32_t vring = kring + kKSlots * kKSlot;
    static constexpr uint32_t bars = vring + kVSlots * kVSlot;
    static constexpr uint32_t tmem = bars + 40 * 8;
    static constexpr uint32_t misc = tmem + 16;                    // first unit [8], abort flag at 7
    static constexpr uint32_t bad = misc + 32;                     // [8] tiles: 16-token groups not to be seen
    static constexpr uint32_t odd = bad + 32;                      // [2][kMaxWords] nodes whose V is no number
    static constexpr uint32_t xch = odd + 2 * kMaxWords * 4;       // row maxima [2][2][128], sums [2][128]
    static constexpr uint32_t rowc = xch + 6 * kRows * 4;          // per row: nodes
    static constexpr uint32_t rowp = rowc + kMaxRows * 4;          // per row: cached tokens
    static constexpr uint32_t rowq = rowp + kMaxRows * 4;          // per row: q_start
    // the scan's scratch lives in the K ring: it is read before the first copy is issued
    static constexpr uint32_t part = kring;
    static constexpr uint32_t pre = part + 1024 * 4;
    __host__ __device__ static constexpr uint32_t total() { return rowq + kMaxRows * 4 + 1024; }
};
static_assert(Smem::kring % 1024 == 0 && Smem::vring % 1024 == 0 && (Smem::q + kHalfQ) % 1024 == 0,
              "swizzled tiles need 1024-byte alignment");
static_assert(Smem::pre + (kMaxRows + 1) * 4 <= Smem::kring + kKSlots * kKSlot, "scan scratch fits the K ring");
static_assert(Smem::total() <= 232448, "shared memory per block");

// A unit: flat rows 128 t .. of KV head k of row r, its first granule U and its
// n granules.
struct Unit {
    int r, k, t, U, n;
};

// How the granules of all units are cut: raw cut c lies at floor(W c / G); one
// within `slack` granules of a border of the unit it falls in moves there.
struct Split {
    int W, G, slack;
    __device__ __forceinline__ int raw(int c) const { return (int)((int64_t)W * c / G); }
    __device__ __forceinline__ int moved(int x, const Unit& u) const {
        const int d0 = x - u.U, d1 = u.U + u.n - x;
        if (min(d0, d1) > slack) return x;
        return d0 <= d1 ? u.U : u.U + u.n;
    }
    // The pieces of unit u (1: whole) and the block that holds the first one.
    __device__ __forceinline__ int pieces(const Unit& u, int& first) const {
        const int64_t a = u.U + slack + 1, b = u.U + u.n - slack - 1;  // cuts that stay lie in a .. b
        const int lo = (int)((a * G + W - 1) / W), hi = (int)(((b + 1) * G + W - 1) / W) - 1;
        first = lo - 1;
        return a <= b && hi >= lo ? hi - lo + 2 : 1;
    }
};

// The units of a block's range [s0, s1), last to first; [e0, e1): the granules
// of the present unit that lie in it.
struct Walk : Unit {
    int s0, e, hk, group;
    const int* C;
    const int* P;
    __device__ __forceinline__ int g0() const { return max(s0 - U, 0); }
    __device__ __forceinline__ int g1() const { return min(e - U, n); }
    __device__ __forceinline__ int len() const { return P[r] + C[r]; }
    __device__ __forceinline__ int ta() const { return g0() * kGranule; }
    __device__ __forceinline__ int te() const { return min(g1() * kGranule, len()); }
    __device__ __forceinline__ int flat() const { return min(kRows, C[r] * group - t * kRows); }
    __device__ __forceinline__ bool prev() {
        if (U <= s0) return false;
        e = U;
        if (t > 0) {
            --t;
        } else {
            if (k > 0) {
                --k;
            } else {
                do --r; while (C[r] == 0);
                k = hk - 1;
            }
            t = (C[r] * group + kRows - 1) / kRows - 1;
            n = (len() + kGranule - 1) / kGranule;
        }
        U -= n;
        return true;
    }
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool valid) {
    const uint32_t bytes = valid ? 16u : 0u;  // nothing is read when it is not: zeros are written
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void sts16(uint32_t addr, uint4 v) {
    asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
                 : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
    return v;
}
// Nonzero bits 15 / 31: the word's low / high half is an infinity or NaN.
__device__ __forceinline__ uint32_t no_number(uint32_t w) { return ((w & 0x7c007c00u) + 0x04000400u) & 0x80008000u; }

// 64 mask bits of a node from node index j0 on (j0 > -64; bits of negative
// nodes, cached tokens, are set).
__device__ __forceinline__ uint64_t mask_bits(const uint32_t* row, int words, int j0) {
    const int w = max(j0, 0) >> 5;
    auto word = [&](int i) -> uint64_t { return i < words ? __ldg(row + i) : 0u; };
    if (j0 < 0) return ((word(0) | word(1) << 32) << -j0) | ((uint64_t(1) << -j0) - 1);
    const int sh = j0 & 31;
    const uint64_t lo = word(w) | word(w + 1) << 32;
    return sh ? (lo >> sh) | word(w + 2) << (64 - sh) : lo;
}
__device__ __forceinline__ uint64_t low_bits(int n) {
    return n <= 0 ? 0 : n >= 64 ? ~uint64_t(0) : (uint64_t(1) << n) - 1;
}

// A node's V that is no number reaches the rows that see it: the odd nodes'
// elements of dims d0 .. d0 + 63 are added to this thread's stored output
// (`orow`, fp16) or partial (`po`, dim group g at po[g * kRows]).
template <bool kFp8>
__device__ __noinline__ void add_odd(const Params& p, const uint32_t* odd, int r, int P, int C, int node, int g,
                                     int kvh, int d0, __half* orow, float4* po) {
    for (int w = 0; w < kMaxWords; ++w) {
        for (uint32_t bits = odd[w]; bits; bits &= bits - 1) {
            const int j = 32 * w + __ffs(bits) - 1;
            const bool sees = p.mask ? (p.mask[(int64_t)g * p.words + w] >> (j & 31)) & 1 : j <= node;
            if (j >= C || !sees) continue;
            const int t = P + j, pb = p.tables[(int64_t)r * p.mbpr + t / p.bs];
            if (pb < 0 || pb >= p.nb) continue;
            const int64_t at = (((int64_t)pb * p.bs + t % p.bs) * p.hk + kvh) * kHeadDim + d0;
            for (int d = 0; d < 64; ++d) {
                __half x;
                if (kFp8) {
                    uint32_t lo, hi;
                    widen4(static_cast<const uint8_t*>(p.v_pool)[at + d], lo, hi);
                    x = __ushort_as_half((unsigned short)(lo & 0xffffu));
                } else {
                    x = static_cast<const __half*>(p.v_pool)[at + d];
                }
                const float f = __half2float(x);
                if (isfinite(f)) continue;
                if (orow) orow[d] = __float2half_rn(__half2float(orow[d]) + f);
                if (po) reinterpret_cast<float*>(po + (d >> 2) * kRows)[d & 3] += f;
            }
        }
    }
}

// Merge the P pieces of a unit that starts in block `first`: jobs of eight dims
// by some rows, claimed by warps.
__device__ __forceinline__ void merge_unit(const Params& p, const Unit& u, int q0, int nq, int P, int first, bool last,
                                        float vs) {
    const int lane = threadIdx.x & 31;
    int* head = p.heads + (int64_t)first * kHeadInts;
    bool ready = last;
    if (!ready) {
        const uint64_t t0 = now_ns();
        for (;;) {
            int seen = 0;
            if (lane == 0) asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(seen) : "l"(head) : "memory");
            seen = __shfl_sync(0xffffffffu, seen, 0);
            if (seen >= P) {
                ready = true;
                break;
            }
            if (__shfl_sync(0xffffffffu, (int)(now_ns() - t0 > kHelpNs), 0)) break;
            __nanosleep(32);
        }
    }
    if (ready) {
        const int nrb = (nq + 31) / 32, rs = min(nrb, max(1, P / 2)), jobs = 16 * rs;
        for (;;) {
            int job = 0;
            if (lane == 0) job = atomicAdd(head + 1, 1);
            job = __shfl_sync(0xffffffffu, job, 0);
            if (job >= jobs) break;
            const int cc = job & 15;  // dims 8 cc ..
            for (int rb = job >> 4; rb < nrb; rb += rs) {
                const int i = rb * 32 + lane;
                if (i >= nq) continue;
                float M = -INFINITY, Lt = 0.f, acc[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) acc[e] = 0.f;
                for (int j0 = 0; j0 < P; j0 += 4) {
                    float mj[4], lj[4];
                    float4 x[4], y[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        mj[j] = -INFINITY;
                        if (j0 + j < P) {
                            const float* s = p.part + ((int64_t)(first + j0 + j) * 2 + (j0 + j == P - 1)) * kPartFloats;
                            mj[j] = __ldcg(s + i);
                            lj[j] = __ldcg(s + kRows + i);
                            const float4* o = reinterpret_cast<const float4*>(s + 2 * kRows) + 2 * cc * kRows + i;
                            x[j] = __ldcg(o);
                            y[j] = __ldcg(o + kRows);
                        }
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        if (j0 + j >= P || mj[j] == -INFINITY) continue;
                        const float mn = fmaxf(M, mj[j]);
                        const float a = M == -INFINITY ? 0.f : fast_exp2(M - mn), w = fast_exp2(mj[j] - mn);
                        M = mn;
                        Lt = Lt * a + w * lj[j];
                        const float o[8] = {x[j].x, x[j].y, x[j].z, x[j].w, y[j].x, y[j].y, y[j].z, y[j].w};
#pragma unroll
                        for (int e = 0; e < 8; ++e) acc[e] = acc[e] * a + w * o[e];
                    }
                }
                const float inv = Lt == 0.f ? 0.f : vs / Lt;
                const int f = u.t * kRows + i;
                uint4 o4;
                o4.x = pack_half2(acc[0] * inv, acc[1] * inv);
                o4.y = pack_half2(acc[2] * inv, acc[3] * inv);
                o4.z = pack_half2(acc[4] * inv, acc[5] * inv);
                o4.w = pack_half2(acc[6] * inv, acc[7] * inv);
                *reinterpret_cast<uint4*>(p.out + ((int64_t)(q0 + f / p.group) * p.hq + u.k * p.group + f % p.group) *
                                                      kHeadDim + cc * 8) = o4;
            }
        }
    }
    // the last of the unit's warps to leave re-arms its words for the next call
    __syncwarp();
    if (lane == 0) {
        __threadfence();
        if (atomicAdd(head + 2, 1) == P * kSoftWarps - 1) {
            head[0] = 0;
            head[1] = 0;
            head[2] = 0;
        }
    }
}

template <bool kFp8>
__global__ void __launch_bounds__(threads<kFp8>(), 1)
    tree_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                const __grid_constant__ Params p) {
    extern __shared__ unsigned char smem_raw[];
    unsigned char* smem = reinterpret_cast<unsigned char*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(smem);
    const uint32_t bar_kfull = sbase + Smem::bars;           // [K slots]
    const uint32_t bar_kempty = bar_kfull + kKSlots * 8;     // [K slots]
    const uint32_t bar_vfull = bar_kempty + kKSlots * 8;     // [V slots]
    const uint32_t bar_vempty = bar_vfull + kVSlots * 8;     // [V slots]
    const uint32_t bar_s = bar_vempty + kVSlots * 8;         // [3]: S buffer computed
    const uint32_t bar_p = bar_s + 8 * kSBufs;               // [3]: P of S buffer written
    const uint32_t bar_o = bar_p + 8 * kSBufs;               // [3]: PV product of buffer done
    const uint32_t bar_x = bar_o + 8 * kSBufs;               // [2]: both halves' row maxima of a tile written
    const uint32_t bar_l = bar_x + 16;                       // both halves' row sums written
    const uint32_t bar_qfree = bar_l + 8;                    // a segment's S products are done with its queries
    const uint32_t bar_odrained = bar_qfree + 8;             // the softmax warps have read a segment's O out
    const uint32_t bar_sfin = bar_odrained + 8;              // the S issuer's last products are complete
    const uint32_t bar_pfin = bar_sfin + 8;                  // the PV issuer's last products are complete
    const uint32_t bar_pub = bar_pfin + 8;                   // the softmax warps have written a partial
    uint32_t* sm_tmem = reinterpret_cast<uint32_t*>(smem + Smem::tmem);
    volatile int* sm_misc = reinterpret_cast<volatile int*>(smem + Smem::misc);
    const volatile int* abort = sm_misc + 7;
    volatile uint32_t* sm_bad = reinterpret_cast<volatile uint32_t*>(smem + Smem::bad);
    uint32_t* sm_odd = reinterpret_cast<uint32_t*>(smem + Smem::odd);
    int* sm_part = reinterpret_cast<int*>(smem + Smem::part);
    int* sm_pre = reinterpret_cast<int*>(smem + Smem::pre);
    int* sm_C = reinterpret_cast<int*>(smem + Smem::rowc);
    int* sm_P = reinterpret_cast<int*>(smem + Smem::rowp);
    int* sm_qs = reinterpret_cast<int*>(smem + Smem::rowq);

    constexpr int kThreads = threads<kFp8>();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rows = p.rows, group = p.group;

    // ---- per row: nodes, cached tokens, granules of all its units; their prefix ----
    const int per = (rows + kThreads - 1) / kThreads;
    int sum = 0;
    for (int i = 0; i < per; ++i) {
        const int r = tid * per + i;
        if (r < rows) {
            const int q0 = p.q_start[r], L = p.seq_lens[r];
            int C = p.q_start[r + 1] - q0;
            if (C < 0 || L < C || L > p.limit || q0 < 0 || q0 > p.total - C) {
                if (blockIdx.x == 0) flag_error(p.dev_err, PKV_DEV_ERR_SEQ_LEN);
                C = 0;
            } else if (p.mask && C > 32 * p.words) {
                if (blockIdx.x == 0) flag_error(p.dev_err, PKV_DEV_ERR_MASK);
                C = 0;
            }
            sm_C[r] = C;
            sm_P[r] = L - C;
            sm_qs[r] = q0;
            // below 2^31 in total (checked by the host)
            sm_pre[r] = C > 0 ? p.hk * ((C * group + kRows - 1) / kRows) * ((L + kGranule - 1) / kGranule) : 0;
            sum += sm_pre[r];
        }
    }
    sm_part[tid] = sum;
    if (tid < 2 * kMaxWords) sm_odd[tid] = 0;
    __syncthreads();
    if (warp == 0) {
        constexpr int kPer = (kThreads + 31) / 32;
        int v[kPer], acc = 0;
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            v[j] = sm_part[lane * kPer + j];
            acc += v[j];
        }
        int incl = acc;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int t = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += t;
        }
        int run = incl - acc;
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            sm_part[lane * kPer + j] = run;
            run += v[j];
        }
    }
    __syncthreads();
    {
        int run = sm_part[tid];
        for (int i = 0; i < per; ++i) {
            const int r = tid * per + i;
            if (r < rows) {
                const int c = sm_pre[r];
                sm_pre[r] = run;
                run += c;
            }
        }
        if (tid == kThreads - 1) sm_pre[rows] = run;
    }
    __syncthreads();

    // ---- this block's range ----
    Split sp;
    sp.W = sm_pre[rows];
    sp.G = min((int)gridDim.x, max(sp.W / kMinGranules, 1));
    sp.slack = max(kMinGranules, sp.W / sp.G / 16);
    const int cta = blockIdx.x;
    if (sp.W == 0 || cta >= sp.G) return;
    auto locate = [&](int x) -> Unit {  // the unit that holds granule x
        int lo = 0, hi = rows - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (sm_pre[mid] <= x) lo = mid; else hi = mid - 1;
        }
        Unit u;
        u.r = lo;
        u.n = (sm_P[lo] + sm_C[lo] + kGranule - 1) / kGranule;
        const int nt = (sm_C[lo] * group + kRows - 1) / kRows;
        const int i = (x - sm_pre[lo]) / u.n;
        u.k = i / nt;
        u.t = i - u.k * nt;
        u.U = sm_pre[lo] + i * u.n;
        return u;
    };
    // warp 0: the moved cuts on both sides and the unit before the upper one
    if (warp == 0) {
        const int x = sp.raw(cta + (lane & 1));
        const int cut = x < sp.W ? sp.moved(x, locate(x)) : sp.W;
        const int c0 = __shfl_sync(0xffffffffu, cut, 0), c1 = __shfl_sync(0xffffffffu, cut, 1);
        if (c0 < c1) {
            const Unit u = locate(c1 - 1);
            if (lane == 0) {
                sm_misc[0] = u.r;
                sm_misc[1] = u.k;
                sm_misc[2] = u.t;
                sm_misc[3] = u.U;
                sm_misc[4] = u.n;
            }
        }
        if (lane == 0) {
            sm_misc[5] = c0;
            sm_misc[6] = c1;
            sm_misc[7] = 0;  // abort
        }
    }

    // ---- barriers and tensor memory ----
    if (tid == 32) {
        const int fill = kFp8 ? kConvWarps : 1;
        for (int s = 0; s < kKSlots; ++s) {
            mbar_init(bar_kfull + 8 * s, fill);
            mbar_init(bar_kempty + 8 * s, 1);
        }
        for (int s = 0; s < kVSlots; ++s) {
            mbar_init(bar_vfull + 8 * s, fill);
            mbar_init(bar_vempty + 8 * s, 1);
        }
        mbar_init(bar_l, kSoftWarps);
        for (int b = 0; b < 2; ++b) mbar_init(bar_x + 8 * b, kSoftWarps);
        for (int b = 0; b < kSBufs; ++b) {
            mbar_init(bar_s + 8 * b, 1);
            mbar_init(bar_p + 8 * b, kSoftWarps);
            mbar_init(bar_o + 8 * b, 1);
        }
        mbar_init(bar_qfree, 1);
        mbar_init(bar_odrained, kSoftWarps);
        mbar_init(bar_sfin, 1);
        mbar_init(bar_pfin, 1);
        mbar_init(bar_pub, kSoftWarps);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 2) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(sbase + Smem::tmem),
                     "r"(kTmemCols));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *sm_tmem;
    auto raise_abort = [&]() { sm_misc[7] = 1; };

    Walk w;
    w.r = sm_misc[0];
    w.k = sm_misc[1];
    w.t = sm_misc[2];
    w.U = sm_misc[3];
    w.n = sm_misc[4];
    w.s0 = sm_misc[5];
    w.e = sm_misc[6];
    w.hk = p.hk;
    w.group = group;
    w.C = sm_C;
    w.P = sm_P;
    const bool any = w.s0 < w.e;  // both cuts may have moved to one border

    if (!any) {
        // nothing to do but to free the tensor memory below
    } else if (!kFp8 && warp >= kLoad) {
        // ============================== TMA ==============================
        // Warp kLoad streams K tiles, the next one V halves.  Table entries are
        // fetched a batch ahead: lane l handles box l % gpu of copy unit l / gpu
        // of a batch, so the table's latency is paid once a batch.
        const bool is_v = warp == kLoad + 1;
        const int nslots = is_v ? kVSlots : kKSlots;
        const int unit_tok = is_v ? 64 : kTile;
        const uint32_t full0 = is_v ? bar_vfull : bar_kfull;
        const uint32_t empty0 = is_v ? bar_vempty : bar_kempty;
        const uint32_t ring = sbase + (is_v ? Smem::vring : Smem::kring);
        const uint32_t slot_bytes = is_v ? kVSlot : kKSlot;
        const uint32_t half_bytes = is_v ? kVHalf : kKHalf;
        const CUtensorMap* map = is_v ? &vmap : &kmap;
        const int box = p.box;
        const int gpu = unit_tok / box, upb = 32 / gpu;
        const int my_j = lane / gpu, my_g = lane % gpu;
        const uint32_t box_bytes = (uint32_t)box * 128;
        const int nowhere = p.nb * p.bs;  // a row past the pool: a copy of zeros
        int s = 0, armed = 0;
        uint32_t ph = 0, fb = full0, eb = empty0, slot = ring;
        bool ok = true;
        do {
            const int ta = w.ta(), te = w.te();
            const int units = (te - ta + unit_tok - 1) / unit_tok;
            const int32_t* trow = p.tables + (int64_t)w.r * p.mbpr;
            auto fetch = [&](int ub) -> int {  // raw block id of this lane's box in the batch at unit ub
                const int tok = ta + (ub + my_j) * unit_tok + my_g * box;
                return tok < te ? __ldg(trow + tok / p.bs) : 0;
            };
            auto to_row = [&](int ub, int pb) -> int {  // its pool row, or -1 for no copy
                const int tok = ta + (ub + my_j) * unit_tok + my_g * box;
                if (tok >= te) return -1;
                if (pb < 0 || pb >= p.nb) {
                    if (!is_v) flag_error(p.dev_err, PKV_DEV_ERR_BLOCK_ID);
                    return nowhere;
                }
                return pb * p.bs + tok % p.bs;
            };
            int pb_next = fetch(0);
            int row = to_row(0, pb_next);
            pb_next = fetch(upb);
            int j = 0;
            for (int u = 0; u < units; ++u) {
                if (!mbar_waitw(eb, ph ^ 1, abort)) {
                    ok = false;
                    break;
                }
                const bool issue = my_j == j && row >= 0;
                const uint32_t nissue = __popc(__ballot_sync(0xffffffffu, issue));
                if (!is_v) {
                    // groups of 16 tokens whose table entry is out of range: read by the softmax
                    // warps at this tile, long before the word's next use eight tiles on
                    const uint32_t mine = issue && row == nowhere ? ((1u << (box / 16)) - 1) << (my_g * (box / 16)) : 0;
                    const uint32_t all = __reduce_or_sync(0xffffffffu, mine);
                    if (lane == 0) sm_bad[armed & 7] = all;
                }
                if (lane == 0) mbar_arrive_expect_tx(fb, nissue * 2 * box_bytes);
                __syncwarp();
                if (issue) {
                    const uint32_t st = slot + my_g * box_bytes;
                    tma_load_3d(st, map, 0, w.k, row, fb);
                    tma_load_3d(st + half_bytes, map, 64, w.k, row, fb);
                }
                ++armed;
                if (++j == upb) {
                    j = 0;
                    row = to_row(u + 1, pb_next);
                    pb_next = fetch(u + 1 + upb);
                }
                if (++s == nslots) {
                    s = 0;
                    ph ^= 1;
                    fb = full0;
                    eb = empty0;
                    slot = ring;
                } else {
                    fb += 8;
                    eb += 8;
                    slot += slot_bytes;
                }
            }
        } while (ok && w.prev());
        if (!ok && lane == 0) {
            raise_abort();
            flag_error(p.dev_err, PKV_DEV_ERR_TIMEOUT);
        }
        // every armed slot's copies have landed before the block exits
        for (int u = max(0, armed - nslots); u < armed; ++u)
            if (!mbar_drain1(full0 + 8 * (u % nslots), (uint32_t)(u / nslots) & 1) && lane == 0)
                flag_error(p.dev_err, PKV_DEV_ERR_TIMEOUT);
        __syncwarp();
    } else if (kFp8 && warp >= kLoad) {
        // ======================= FP8: load and widen =======================
        // Per tile, thread (warp c, lane l) takes 16 codes (l % 8) of token 4 c +
        // l / 8 of each of the tile's eight 16-token groups, K then V.  A tile's
        // V is loaded before its K is stored and the next tile's K before its V
        // is, and its table entries a tile earlier still.
        const int c = warp - kLoad, tok_in = 4 * c + (lane >> 3), col = lane & 7;
        const int tok_bytes = p.hk * kHeadDim;
        Walk nx = w;  // the walk, one tile ahead
        int nt0 = nx.ta();
        bool more = true;
        auto fetch = [&]() -> int {  // raw block id of group `lane` of the next tile
            const int tok = nt0 + 16 * lane;
            return more && lane < 8 && tok < nx.te() ? __ldg(p.tables + (int64_t)nx.r * p.mbpr + tok / p.bs) : 0;
        };
        int pb = fetch();
        int row = -1, te = 0, t0 = 0, kvh = 0;
        auto step = [&]() -> bool {  // the next tile becomes the present one
            if (!more) return false;
            t0 = nt0;
            te = nx.te();
            kvh = nx.k;
            const int tok = t0 + 16 * lane;
            row = -1;
            if (lane < 8 && tok < te) {
                if (pb < 0 || pb >= p.nb) {
                    row = -2;  // not to be seen
                    if (c == 0) flag_error(p.dev_err, PKV_DEV_ERR_BLOCK_ID);
                } else {
                    row = pb * p.bs + tok % p.bs;
                }
            }
            nt0 += kTile;
            if (nt0 >= te) {
                more = nx.prev();
                nt0 = nx.ta();
            }
            pb = fetch();
            return true;
        };
        auto load = [&](const void* pool, uint4 (&x)[8]) {
#pragma unroll
            for (int g = 0; g < 8; ++g) {
                const int base = __shfl_sync(0xffffffffu, row, g);
                const bool have = base >= 0 && t0 + 16 * g + tok_in < te;
                x[g] = have ? __ldg(reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(pool) +
                                                                   (int64_t)(base + tok_in) * tok_bytes +
                                                                   kvh * kHeadDim + col * 16))
                            : make_uint4(0, 0, 0, 0);
            }
        };
        auto store = [&](uint32_t lo, uint32_t half_bytes, int r0, const uint4& x) {
            // chunks 2 col and 2 col + 1 of 8 dims; the lanes of the upper dims store theirs the
            // other way round, so that eight lanes meet eight bank groups
            const uint4 a = widen8(make_uint2(x.x, x.y)), b = widen8(make_uint2(x.z, x.w));
            const int sw = col >> 2;
            const uint32_t at = lo + sw * half_bytes + r0 * 128;
            const int c0 = 2 * (col & 3) + sw, c1 = 2 * (col & 3) + 1 - sw;
            sts16(at + ((c0 ^ (r0 & 7)) << 4), sw ? b : a);
            sts16(at + ((c1 ^ (r0 & 7)) << 4), sw ? a : b);
        };
        int ks = 0, vs = 0, tile = 0;
        uint32_t kph = 0, vph = 0;
        bool ok = true;
        uint4 xk[8], xv[8];
        bool have = step();
        load(p.k_pool, xk);
        while (have) {
            load(p.v_pool, xv);
            const int n = te - t0;  // tokens of this tile that are this segment's (may exceed 128)
            const uint32_t gone = __ballot_sync(0xffffffffu, row == -2);
            // K
            if (!(ok = mbar_waitw(bar_kempty + 8 * ks, kph ^ 1, abort))) break;
            if (c == 0 && lane == 0) sm_bad[tile & 7] = gone;
            ++tile;
#pragma unroll
            for (int g = 0; g < 8; ++g)
                if (16 * g < n) store(sbase + Smem::kring + ks * kKSlot, kKHalf, 16 * g + tok_in, xk[g]);
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar_kfull + 8 * ks);
            if (++ks == kKSlots) {
                ks = 0;
                kph ^= 1;
            }
            have = step();
            if (have) load(p.k_pool, xk);
            // V, in halves
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (64 * h < n) {
                    if (!(ok = mbar_waitw(bar_vempty + 8 * vs, vph ^ 1, abort))) break;
#pragma unroll
                    for (int g = 0; g < 4; ++g)
                        if (64 * h + 16 * g < n)
                            store(sbase + Smem::vring + vs * kVSlot, kVHalf, 16 * g + tok_in, xv[4 * h + g]);
                    fence_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar_vfull + 8 * vs);
                    if (++vs == kVSlots) {
                        vs = 0;
                        vph ^= 1;
                    }
                }
            }
            if (!ok) break;
        }
        if (!ok && lane == 0) {
            raise_abort();
            flag_error(p.dev_err, PKV_DEV_ERR_TIMEOUT);
        }
        __syncwarp();
    } else if (warp == kSIssue) {
        // ====================== queries and S issue ======================
        // Per segment the warp brings the unit's 128 flat rows in (256 bytes a
        // row, swizzled; rows past the unit's are zeros) once the previous
        // segment's products no longer read the buffer.  Then its first lane
        // issues S_t = Q . K_t^T into S buffer t % 3, once K_t has landed and
        // PV_{t-3} has read P_{t-3} out of that buffer.
        const uint32_t id_s = idesc(kRows, kTile, 0);
        const uint64_t kd0 = sdesc(sbase + Smem::kring, 16, 1024);
        uint64_t kd = kd0;
        const uint64_t qd = sdesc(sbase + Smem::q, 16, 1024);
        uint32_t kf = bar_kfull, ke = bar_kempty, ph = 0;
        int s = 0, sb = 0, gt = 0, seg = 0;
        uint32_t sph = 0;  // use parity of S buffer sb
        bool ok = true;
        do {
            const int nq = w.flat(), q0 = sm_qs[w.r];
            int at[4];  // of rows lane, lane + 32, ..: (node, head) index, or -1
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int i = 32 * j + lane, f = w.t * kRows + i, node = f / group;
                at[j] = i < nq ? (q0 + node) * p.hq + w.k * group + (f - node * group) : -1;
            }
            if (seg > 0 && !(ok = mbar_waitw(bar_qfree, (uint32_t)(seg - 1) & 1, abort))) break;
            const int ch = lane & 15;
            const uint32_t dst0 = sbase + Smem::q + (ch >> 3) * kHalfQ;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
#pragma unroll 4
                for (int x = 0; x < 16; ++x) {
                    const int rr = 2 * x + (lane >> 4), i = 32 * j + rr;
                    const int a = __shfl_sync(0xffffffffu, at[j], rr);
                    cp_async16(dst0 + i * 128 + (((ch & 7) ^ (i & 7)) << 4), p.q + (int64_t)max(a, 0) * kHeadDim + ch * 8,
                               a >= 0);
                }
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
            fence_async_smem();
            __syncwarp();
            if (lane == 0) {
                const int te = w.te();
                for (int t0 = w.ta(); t0 < te; t0 += kTile, ++gt) {
                    if (!(ok = mbar_wait1(kf, ph, abort))) break;
                    if (gt >= kSBufs && !(ok = mbar_wait1(bar_o + 8 * sb, sph ^ 1, abort))) break;
                    tc_fence_after();
                    const uint32_t d = tmem + kColS + sb * kTile;
#pragma unroll
                    for (int ks = 0; ks < 8; ++ks) {
                        const uint32_t off = (uint32_t)((((ks >> 2) * kHalfQ) + (ks & 3) * 32) >> 4);
                        umma_ss(d, qd + off, kd + off, id_s, ks > 0);
                    }
                    umma_commit(bar_s + 8 * sb);
                    umma_commit(ke);  // K_t is no longer read
                    if (++sb == kSBufs) {
                        sb = 0;
                        sph ^= 1;
                    }
                    if (++s == kKSlots) {
                        s = 0;
                        ph ^= 1;
                        kd = kd0;
                        kf = bar_kfull;
                        ke = bar_kempty;
                    } else {
                        kd += kKSlot >> 4;
                        kf += 8;
                        ke += 8;
                    }
                }
                if (ok) umma_commit(bar_qfree);
            }
            ok = __shfl_sync(0xffffffffu, (int)ok, 0) != 0;
            ++seg;
        } while (ok && w.prev());
        if (lane == 0) {
            if (!ok) {
                raise_abort();
                flag_error(p.dev_err, PKV_DEV_ERR_TIMEOUT);
            }
            umma_commit(bar_sfin);
            if (!mbar_drain1(bar_sfin, 0)) flag_error(p.dev_err, PKV_DEV_ERR_TIMEOUT);
        }
        __syncwarp();
    } else if (warp == kPvIssue) {
        // ============================ PV issue ===========================
        // O += P_t . V_t once both V halves have landed and the softmax warps
        // have stored P_t (and seen to V's rows that need it); a segment's first
        // product starts O afresh, after the previous segment's O was read.
        // K-steps past the last token are skipped.
        if (lane == 0) {
            const uint32_t id_o = idesc(kRows, 128, 1);
            const uint64_t vd0 = sdesc(sbase + Smem::vring, kVHalf, 1024);
            int va = 0;        // V slot of a tile's first half
            uint32_t vph = 0;  // its fill parity
            int pb = 0;        // S buffer holding P_t
            uint32_t pph = 0;  // its use parity
            int seg = 0;
            bool ok = true;
            do {
                const int ta = w.ta(), te = w.te();
                for (int t0 = ta; t0 < te; t0 += kTile) {
                    int vb = va + 1;
                    uint32_t vphb = vph;
                    if (vb == kVSlots) {
                        vb = 0;
                        vphb ^= 1;
                    }
                    const bool two = te - t0 > 64;
                    const int nsteps = (min(kTile, te - t0) + 15) / 16;
                    if (!(ok = mbar_wait1(bar_vfull + 8 * va, vph, abort))) break;
                    if (two && !(ok = mbar_wait1(bar_vfull + 8 * vb, vphb, abort))) break;
                    if (!(ok = mbar_wait1(bar_p + 8 * pb, pph, abort))) break;
                    if (t0 == ta && seg > 0 && !(ok = mbar_wait1(bar_odrained, (uint32_t)(seg - 1) & 1, abort))) break;
                    tc_fence_after();
                    const uint32_t pa = tmem + kColS + pb * kTile;
                    const uint64_t da = vd0 + (uint64_t)(va * (kVSlot >> 4));
                    const uint64_t db = vd0 + (uint64_t)(vb * (kVSlot >> 4));
                    // tokens 64 e .. 64 e + 63 sit in columns 64 e .. 64 e + 31
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk) {
                        if (kk < nsteps)
                            umma_ts(tmem + kColO, pa + (kk >> 2) * 64 + (kk & 3) * 8,
                                    (kk < 4 ? da : db) + (uint64_t)((kk & 3) * 128), id_o,
                                    (t0 > ta || kk > 0) ? 1u : 0u);
                    }
                    umma_commit(bar_o + 8 * pb);
                    umma_commit(bar_vempty + 8 * va);
                    if (two) umma_commit(bar_vempty + 8 * vb);
                    va = two ? vb + 1 : vb;
                    vph = vphb;
                    if (va == kVSlots) {
                        va = 0;
                        vph ^= 1;
                    }
                    if (++pb == kSBufs) {
                        pb = 0;
                        pph ^= 1;
                    }
                }
                ++seg;
            } while (ok && w.prev());
            if (!ok) {
                raise_abort();
                flag_error(p.dev_err, PKV_DEV_ERR_TIMEOUT);
            }
            umma_commit(bar_pfin);
            if (!mbar_drain1(bar_pfin, 0)) flag_error(p.dev_err, PKV_DEV_ERR_TIMEOUT);
        }
        __syncwarp();
    } else {
        // ============================ softmax =============================
        const int quarter = warp & 3, hf = warp >> 2;
        const int i = quarter * 32 + lane;  // flat row of the unit, TMEM lane
        const uint32_t lane_base = (uint32_t)(quarter * 32) << 16;
        float* xmax = reinterpret_cast<float*>(smem + Smem::xch);  // [2][2][128]
        float* xsum = xmax + 4 * kRows;                            // [2][128]
        bool ok = true;
        int sb = 0, psb = 0;          // S buffer of this tile and of the previous one
        uint32_t sph = 0, psph = 0;   // their use parities
        int gt = 0, seg = 0;          // tiles and segments done by this block
        int va = 0;                   // V slot of the tile's first half
        uint32_t vph = 0;             // its fill parity
        // the cut units to merge in the end: the one that goes on behind this
        // block's range (stored first), the one that began before it
        Unit cut[2];
        int cutP[2] = {0, 0}, cutF[2] = {0, 0};
        bool cutL[2] = {false, false};
        uint32_t pubs = 0;
        do {
            const int r = w.r, C = sm_C[r], P = sm_P[r], nq = w.flat();
            const int f = w.t * kRows + min(i, nq - 1);  // rows past the unit's shadow its last one
            const int node = f / group, h = w.k * group + (f - node * group), g = sm_qs[r] + node;
            const uint32_t* mrow = p.mask ? p.mask + (int64_t)g * p.words : nullptr;
            const int ta = w.ta(), te = w.te();
            const float sc = p.scale * (kFp8 ? p.k_scale[w.k] : 1.f);
            // weights are powers of two: a scale of zero stands for the smallest one, so that
            // a masked score of -inf stays one
            const float scale_log2 = fmaxf(fabsf(sc) * kLog2e, 1e-37f);
            const bool flip = sc < 0.f;
            uint32_t* odd = sm_odd + (seg & 1) * kMaxWords;
            bool scanned = false;
            float m = -INFINITY, l = 0.f;
            for (int t0 = ta; t0 < te; t0 += kTile, ++gt) {
                // ---- what this thread's row sees of its 64 tokens ----
                const int base = t0 + hf * 64;
                const bool nodes = t0 + kTile > P;  // the tile holds nodes
                uint64_t vis = ~uint64_t(0);
                if (base + 63 >= P) {
                    const int rel = base - P;
                    vis = mrow ? mask_bits(mrow, p.words, rel) : low_bits(node - rel + 1);
                }
                vis &= low_bits(te - base);
                if (!(ok = mbar_waitw(bar_s + 8 * sb, sph, abort))) break;
                tc_fence_after();
                float s[64];
                {
                    uint32_t v0[32], v1[32];
                    tmem_ld64(tmem + lane_base + kColS + sb * kTile + hf * 64, v0, v1);
#pragma unroll
                    for (int c = 0; c < 32; ++c) {
                        s[c] = __uint_as_float(v0[c]);
                        s[32 + c] = __uint_as_float(v1[c]);
                    }
                }
                const uint32_t gone = (sm_bad[gt & 7] >> (4 * hf)) & 15u;
                if (flip) {
#pragma unroll
                    for (int c = 0; c < 64; ++c) s[c] = -s[c];
                }
                if (gone) {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if ((gone >> e) & 1) vis &= ~(uint64_t(0xffff) << (16 * e));
                }
                if (__any_sync(0xffffffffu, vis != ~uint64_t(0))) {
                    const uint32_t lo = (uint32_t)vis, hi = (uint32_t)(vis >> 32);
#pragma unroll
                    for (int c = 0; c < 64; ++c)
                        s[c] = ((c < 32 ? lo : hi) >> (c & 31)) & 1 ? s[c] : -INFINITY;
                }
                float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int c = 0; c < 64; ++c) mx4[c & 3] = fmaxf(mx4[c & 3], s[c]);
                const float pm = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3]));
                xmax[((gt & 1) * 2 + hf) * kRows + i] = pm;
                __syncwarp();
                if (lane == 0) mbar_arrive(bar_x + 8 * (gt & 1));
                if (!(ok = mbar_waitw(bar_x + 8 * (gt & 1), ((uint32_t)gt >> 1) & 1, abort))) break;
                // every softmax warp is past the previous segment: its odd nodes' words are free
                if (t0 == ta && tid < kMaxWords) sm_odd[((seg + 1) & 1) * kMaxWords + tid] = 0;
                const float mx = fmaxf(pm, xmax[((gt & 1) * 2 + (hf ^ 1)) * kRows + i]) * scale_log2;
                // Lazy rescaling: the reference maximum m only moves when a score
                // exceeds it by more than 2^8 (weights stay <= 256, exact enough in
                // fp16).  A row that sees nothing yet stays at m = -inf with zero weights.
                float alpha = 1.f;
                bool moved = false;
                if (mx > m + 8.f) {
                    alpha = fast_exp2(m - mx);  // 0 while m is -inf
                    m = mx;
                    moved = t0 > ta;
                }
                const float mneg = m == -INFINITY ? 0.f : -m;
                uint32_t pk[32];
                // scores in pairs: one packed FMA for the exponents, one packed add
                // for the row sums; P is rounded to fp16 for the product (2^-11 a weight)
                const uint64_t sc2 = f32x2(scale_log2, scale_log2), mn2 = f32x2(mneg, mneg);
                uint64_t rs2[2] = {f32x2(0.f, 0.f), f32x2(0.f, 0.f)};
#pragma unroll
                for (int c = 0; c < 32; ++c) {
                    float x0, x1;
                    f32x2_split(fma_f32x2(f32x2(s[2 * c], s[2 * c + 1]), sc2, mn2), x0, x1);
                    const float e0 = fast_exp2(x0);
                    const float e1 = fast_exp2(x1);
                    pk[c] = pack_half2(e0, e1);
                    rs2[c & 1] = add_f32x2(rs2[c & 1], f32x2(e0, e1));
                }
                float r0, r1, r2, r3;
                f32x2_split(rs2[0], r0, r1);
                f32x2_split(rs2[1], r2, r3);
                l = l * alpha + ((r0 + r1) + (r2 + r3));
                // O is rescaled only after the previous PV product is complete.
                if (__any_sync(0xffffffffu, moved)) {
                    if (!(ok = mbar_waitw(bar_o + 8 * psb, psph, abort))) break;
                    tc_fence_after();
#pragma unroll 1
                    for (int c0 = 0; c0 < 64; c0 += 32) {
                        uint32_t v[32];
                        tmem_ld32(tmem + lane_base + kColO + hf * 64 + c0, v);
#pragma unroll
                        for (int c = 0; c < 32; ++c) v[c] = __float_as_uint(__uint_as_float(v[c]) * alpha);
                        tmem_st32(tmem + lane_base + kColO + hf * 64 + c0, v);
                    }
                }
                // P over the first 32 of this half's own 64 S columns (already read)
                tmem_st32(tmem + lane_base + kColS + sb * kTile + hf * 64, pk);
                // ---- V of a tile that holds nodes: zero what is no number (and rows
                // past the last token, up to the last k-step's end) ----
                int vb = va + 1;
                uint32_t vphb = vph;
                if (vb == kVSlots) {
                    vb = 0;
                    vphb ^= 1;
                }
                const bool two = te - t0 > 64;
                if (nodes) {
                    scanned = true;
                    if (!(ok = mbar_waitw(bar_vfull + 8 * va, vph, abort))) break;
                    if (two && !(ok = mbar_waitw(bar_vfull + 8 * vb, vphb, abort))) break;
                    const int vrows = min(kTile, te - t0), row = tid & 127, up = tid >> 7;  // up: dims 64 ..
                    const uint32_t at = sbase + Smem::vring + (row >= 64 ? vb : va) * kVSlot + up * kVHalf + (row & 63) * 128;
                    if (row < vrows && t0 + row >= P) {
                        uint32_t any_odd = 0;
#pragma unroll
                        for (int c = 0; c < 8; ++c) {
                            const uint4 x = lds16(at + (((c + row) & 7) << 4));
                            any_odd |= no_number(x.x) | no_number(x.y) | no_number(x.z) | no_number(x.w);
                        }
                        if (any_odd) {
                            for (int c = 0; c < 8; ++c) {
                                uint4 x = lds16(at + (c << 4));
                                uint32_t* e = reinterpret_cast<uint32_t*>(&x);
                                for (int d = 0; d < 4; ++d) {
                                    const uint32_t o = no_number(e[d]);
                                    if (o & 0x8000u) e[d] &= 0xffff0000u;
                                    if (o & 0x80000000u) e[d] &= 0x0000ffffu;
                                }
                                sts16(at + (c << 4), x);
                            }
                            const int j = t0 + row - P;
                            atomicOr(&odd[j >> 5], 1u << (j & 31));
                        }
                    } else if (row >= vrows && row < (vrows + 15) / 16 * 16) {
#pragma unroll
                        for (int c = 0; c < 8; ++c) sts16(at + (((c + row) & 7) << 4), make_uint4(0, 0, 0, 0));
                    }
                    fence_async_smem();
                }
                va = two ? vb + 1 : vb;
                vph = vphb;
                if (va == kVSlots) {
                    va = 0;
                    vph ^= 1;
                }
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar_p + 8 * sb);
                psb = sb;
                psph = sph;
                if (++sb == kSBufs) {
                    sb = 0;
                    sph ^= 1;
                }
            }
            if (!ok) break;
            // ---- end of the segment: wait for its last PV product, add the two
            // halves' row sums ----
            if (!(ok = mbar_waitw(bar_o + 8 * psb, psph, abort))) break;
            xsum[hf * kRows + i] = l;
            __syncwarp();
            if (lane == 0) mbar_arrive(bar_l);
            if (!(ok = mbar_waitw(bar_l, (uint32_t)seg & 1, abort))) break;
            tc_fence_after();
            const float L = l + xsum[(hf ^ 1) * kRows + i];
            bool any_odd = false;
            if (scanned) any_odd = __any_sync(0xffffffffu, odd[lane] != 0);
            uint32_t v[32], v2[32];
            tmem_ld64(tmem + lane_base + kColO + hf * 64, v, v2);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar_odrained);  // O is free for the next segment
            const bool mine = i < nq;
            if (w.g0() == 0 && w.g1() == w.n) {
                // ---- a whole unit: normalise and store ----
                const float vsc = kFp8 ? p.v_scale[w.k] : 1.f;
                const float inv = L == 0.f ? 0.f : __fdividef(vsc, L);
                __half* orow = p.out + ((int64_t)g * p.hq + h) * kHeadDim + hf * 64;
                if (mine && p.out_v8) {
#pragma unroll
                    for (int c = 0; c < 64; c += 16) {
                        const uint32_t* u = c < 32 ? v + c : v2 + (c - 32);
                        uint32_t w8[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            w8[e] = pack_half2(__uint_as_float(u[2 * e]) * inv, __uint_as_float(u[2 * e + 1]) * inv);
                        st_v8(orow + c, w8);
                    }
                } else if (mine) {
#pragma unroll
                    for (int c = 0; c < 64; c += 8) {
                        const uint32_t* u = c < 32 ? v + c : v2 + (c - 32);
                        uint4 q4;
                        q4.x = pack_half2(__uint_as_float(u[0]) * inv, __uint_as_float(u[1]) * inv);
                        q4.y = pack_half2(__uint_as_float(u[2]) * inv, __uint_as_float(u[3]) * inv);
                        q4.z = pack_half2(__uint_as_float(u[4]) * inv, __uint_as_float(u[5]) * inv);
                        q4.w = pack_half2(__uint_as_float(u[6]) * inv, __uint_as_float(u[7]) * inv);
                        *reinterpret_cast<uint4*>(orow + c) = q4;
                    }
                }
                if (mine && any_odd) add_odd<kFp8>(p, odd, r, P, C, node, g, w.k, hf * 64, orow, nullptr);
            } else {
                // ---- a piece: store the partial and count it ----
                const bool ends = w.g1() == w.n;
                float* slot = p.part + ((int64_t)cta * 2 + ends) * kPartFloats;
                if (hf == 0) {
                    __stcg(slot + i, m);
                    __stcg(slot + kRows + i, L);
                }
                float4* po = reinterpret_cast<float4*>(slot + 2 * kRows) + hf * 16 * kRows + i;
                if (mine) {
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const uint32_t* u = e < 8 ? v + 4 * e : v2 + 4 * (e - 8);
                        __stcg(po + e * kRows, make_float4(__uint_as_float(u[0]), __uint_as_float(u[1]),
                                                           __uint_as_float(u[2]), __uint_as_float(u[3])));
                    }
                    if (any_odd) add_odd<kFp8>(p, odd, r, P, C, node, g, w.k, hf * 64, nullptr, po);
                }
                __threadfence();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar_pub);
                const int x = cutP[0] ? 1 : 0;
                cut[x] = w;
                cutP[x] = sp.pieces(w, cutF[x]);
                if (warp == 0) {
                    // every softmax warp's stores are ordered before this count
                    if (!(ok = mbar_waitw(bar_pub, pubs & 1, abort))) break;
                    int old = 0;
                    if (lane == 0) {
                        __threadfence();
                        old = atomicAdd(p.heads + (int64_t)cutF[x] * kHeadInts, 1);
                        __threadfence();
                    }
                    cutL[x] = __shfl_sync(0xffffffffu, old, 0) == cutP[x] - 1;
                }
                ++pubs;
            }
            ++seg;
        } while (w.prev());
        if (!ok && lane == 0) {
            raise_abort();
            flag_error(p.dev_err, PKV_DEV_ERR_TIMEOUT);
        }
        if (ok) {
#pragma unroll 1
            for (int x = 0; x < 2; ++x) {
                if (!cutP[x]) break;
                const Unit& u = cut[x];
                const int nq = min(kRows, sm_C[u.r] * group - u.t * kRows);
                merge_unit(p, u, sm_qs[u.r], nq, cutP[x], cutF[x], cutL[x], kFp8 ? p.v_scale[u.k] : 1.f);
            }
        }
    }

    // ---- release tensor memory ----
    tc_fence_before();
    __syncthreads();
    if (warp == 2) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols));
    }
}

size_t head_bytes() { return align_up((size_t)kMaxGrid * kHeadInts * sizeof(int), 256); }
size_t workspace_bytes() { return head_bytes() + (size_t)kMaxGrid * 2 * kPartFloats * sizeof(float); }

// Once per device: the SM count, and the kernels' shared-memory size.
struct Device {
    std::once_flag once;
    int status = PKV_OK, blocks = 0;
};

int device_blocks(int* blocks) {
    static Device devices[64];
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess) return PKV_ERR_CUDA;
    if (dev < 0 || dev >= 64) return PKV_ERR_UNSUPPORTED;
    Device& d = devices[dev];
    std::call_once(d.once, [&] {
        int sms = 0;
        if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms <= 0 ||
            cudaFuncSetAttribute(tree_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, Smem::total()) !=
                cudaSuccess ||
            cudaFuncSetAttribute(tree_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, Smem::total()) !=
                cudaSuccess) {
            d.status = PKV_ERR_CUDA;
            return;
        }
        d.blocks = sms < kMaxGrid ? sms : kMaxGrid;
    });
    *blocks = d.blocks;
    return d.status;
}

template <bool kFp8>
int launch(const Params& prm, const CUtensorMap& km, const CUtensorMap& vm, int blocks, cudaStream_t stream) {
    tree_kernel<kFp8><<<blocks, threads<kFp8>(), Smem::total(), stream>>>(km, vm, prm);
    return launch_status();
}

}  // namespace tree
}  // namespace pkv

extern "C" size_t paged_attention_tree_workspace_size(int rows, int total_q, int q_heads, int kv_heads,
                                                      int head_dim, int block_size) {
    if (rows < 0 || total_q < 0 || q_heads <= 0 || kv_heads <= 0 || q_heads % kv_heads || head_dim <= 0 ||
        block_size <= 0)
        return 0;
    return pkv::tree::workspace_bytes();
}

extern "C" int paged_attention_tree(void* out, const void* q, const void* k_pool, const void* v_pool,
                                    const float* k_scale, const float* v_scale,
                                    const int32_t* block_tables, const int32_t* seq_lens,
                                    const int32_t* q_start, const uint32_t* mask, int mask_words, int rows,
                                    int total_q, int q_heads, int kv_heads, int head_dim, int block_size,
                                    float scale, int max_blocks_per_row, int num_blocks, int max_seq_len,
                                    void* workspace, size_t workspace_bytes, int32_t* dev_err,
                                    cudaStream_t stream) {
    using namespace pkv;
    using namespace pkv::tree;
    if (rows < 0 || total_q < 0 || q_heads <= 0 || kv_heads <= 0 || q_heads % kv_heads || head_dim <= 0 ||
        block_size <= 0 || max_blocks_per_row <= 0 || num_blocks <= 0 || max_seq_len < 0 || !isfinite(scale))
        return PKV_ERR_INVALID_ARG;
    if ((int64_t)max_seq_len > (int64_t)max_blocks_per_row * block_size) return PKV_ERR_INVALID_ARG;
    if ((k_scale == nullptr) != (v_scale == nullptr) || (mask && mask_words <= 0)) return PKV_ERR_INVALID_ARG;
    if (head_dim != kHeadDim || block_size % 16 || rows > kMaxRows || q_heads > 65535 ||
        (mask && mask_words > kMaxWords))
        return PKV_ERR_UNSUPPORTED;
    const int group = q_heads / kv_heads;
    // all units' granules, every (token, head) index and every pool row stay below 2^31
    const int64_t granules = (int64_t)kv_heads * (((int64_t)total_q * group) / kRows + rows) *
                             (((int64_t)max_seq_len + kGranule - 1) / kGranule);
    const int64_t pool_rows = (int64_t)num_blocks * block_size;
    if (granules >= (int64_t(1) << 31) || pool_rows >= (int64_t(1) << 31) - kTile ||
        (int64_t)total_q * q_heads >= (int64_t(1) << 31))
        return PKV_ERR_UNSUPPORTED;
    if (rows == 0 || total_q == 0) return PKV_OK;
    if (!out || !q || !k_pool || !v_pool || !block_tables || !seq_lens || !q_start) return PKV_ERR_INVALID_ARG;
    if (!aligned16(out) || !aligned16(q) || !aligned16(k_pool) || !aligned16(v_pool)) return PKV_ERR_INVALID_ARG;
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255) || workspace_bytes < tree::workspace_bytes())
        return PKV_ERR_WORKSPACE;

    int blocks = 0, st = device_blocks(&blocks);
    if (st != PKV_OK) return st;
    Params prm{};
    prm.q = static_cast<const __half*>(q);
    prm.out = static_cast<__half*>(out);
    prm.k_pool = k_pool;
    prm.v_pool = v_pool;
    prm.k_scale = k_scale;
    prm.v_scale = v_scale;
    prm.tables = block_tables;
    prm.seq_lens = seq_lens;
    prm.q_start = q_start;
    prm.mask = mask;
    prm.words = mask_words;
    prm.rows = rows;
    prm.total = total_q;
    prm.hq = q_heads;
    prm.hk = kv_heads;
    prm.group = group;
    prm.bs = block_size;
    prm.mbpr = max_blocks_per_row;
    prm.nb = num_blocks;
    prm.limit = max_seq_len;
    prm.scale = scale;
    prm.out_v8 = (reinterpret_cast<uintptr_t>(out) & 31) == 0;
    prm.heads = static_cast<int*>(workspace);
    prm.part = reinterpret_cast<float*>(static_cast<unsigned char*>(workspace) + head_bytes());
    prm.dev_err = dev_err;
    prm.box = 16;  // the largest power of two that divides a page, at most a granule
    while (prm.box < kGranule && block_size % (2 * prm.box) == 0) prm.box *= 2;
    CUtensorMap km{}, vm{};
    if (k_scale) return launch<true>(prm, km, vm, blocks, stream);
    const int64_t dims[3] = {kHeadDim, kv_heads, pool_rows};
    const int64_t strides[2] = {kHeadDim * 2, (int64_t)kv_heads * kHeadDim * 2};
    const int box[3] = {64, 1, prm.box};
    if ((st = encode_map_3d(k_pool, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, dims, strides, box, &km)) != PKV_OK) return st;
    if ((st = encode_map_3d(v_pool, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, dims, strides, box, &vm)) != PKV_OK) return st;
    return launch<false>(prm, km, vm, blocks, stream);
}
