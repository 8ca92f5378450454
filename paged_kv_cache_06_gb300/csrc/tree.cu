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
// Work.  A unit is 128 flat rows (an M block) of one (row, KV head) and walks the
// row's tokens in 128-token tiles; a job is one tile.  The units' 64-token
// granules, in (row, KV head, M block, token) order, are cut into equal
// contiguous ranges, one per thread block, one block per SM, whatever the mix of
// lengths (the host never reads them); a cut that falls within a few granules
// of a unit's border moves to it, which spares a partial result of 64 KB for a
// little imbalance.  Rows of several M blocks: M block m belongs to plane
// m % planes, the blocks are shared out over the planes by their work, and each
// plane is a sequence of its own.  Planes of equal work get as many blocks each and
// are walked in step, so the M blocks of a row read its cache at the same time,
// from DRAM once: in one sequence, 64 rows of 4096 tokens and 64 nodes (three M
// blocks) took three times the traffic, and with 51, 51 and 50 blocks, which drift
// apart, 110 us instead of 104.
//
// Units cut over P blocks.  A block walks its range from the last unit to the
// first, so a piece that others continue comes first.  It stores its partial
// result (reference maxima, row sums, unnormalised output in 32 bits).  Of two
// pieces the second folds the first's partial into its own result when it is
// done: the block before, which as a rule started earlier, stored it long ago.  Of more
// pieces each stores its partial and counts itself, and in the end each block
// waits for its cut units' other pieces and merges its share of each (some rows
// by some dims), over the pieces in order, so the result does not depend on
// time.  A block that has waited kHelpNs goes on: it gives its share up, and the block that
// arrives last, which waits for nobody, does what was given up; or, the second of two, it
// stores its piece, and whichever of the two stores last merges both, by the same
// operations.  So no block's progress depends on another one running, and two
// calls can share the GPU.  The counts return to zero by themselves (a wrapping
// increment on arrival and one on departure; a pair's by the block that uses both pieces).
//
// Warp roles (each walks the same segments, a unit's part in the block's range):
//   warps 0-7   softmax, in two groups of four that take alternate jobs: one
//               flat row a thread (TMEM lane), its 128 scores in two halves.
//               Both groups share the accumulator; a job's reference maximum
//               goes to the other group as soon as it is known, before the
//               exponentials;
//   warp 8      queries (cp.async) and S issue;  warp 9  PV issue;
//   warps 10/11 K / V by TMA, one box of 16, 32 or 64 tokens of a page a copy;
//               fp16 pools straight into the operand rings;
//   warps 12-15 (FP8 pools) widen the codes, exactly, from rings of their own
//               into the operand rings; the scales go into the score scale and
//               the normalisation.
// A job's two products take 1024 clocks, its 128 x 128 exponentials 512 (32 a clock
// and SM, measured); one group for all jobs also waits, loads and stores in
// turn, 2000 clocks a job.  A wait and its commits cost an issuing warp some 150
// clocks that nothing hides, so tiles of 64 tokens ran at half the rate.
//
// What bounds it (12 query heads over 2 unless said; times in a graph of calls over four
// sets of inputs).  64 rows of 4096, 64 nodes: 102.5 us, 998 TFLOP/s, 52% of cuBLAS's
// rate (108 us a call on fresh inputs); a job every 0.95 us.  Tensor memory
// holds three S buffers, and each is busy for 2.5 us: P is written 1.0 us after S is
// there, its product issued 0.7 later and done in 0.3, the next S issued and done in
// 0.45.  (A third fewer bytes from L2 changed nothing.)  4 rows of 32768, 5 to 16
// nodes: 35.1 us; the copies run at DRAM's rate for 22 of them, 6 are the start and 5
// the merge of 19 pieces.  32 rows of 1024, 25 nodes, E4M3: 21.3 us, nine tiles a block
// at 1.1 us, paced by the widening (0.55 us a granule for a pool's two warps) with
// 224 KB a tile through shared memory (0.9 us).  4 rows of 0 to 200: 8.4 us, one
// dependent chain.
// Every wait is bounded: a block that gives up flags the error, tells its other
// warps to stop, and lets its copies and products in flight finish before it
// frees tensor memory.
//
// What is not seen.  Scores of tokens a flat row does not see become -inf
// before the maximum.  A weight of zero times an infinity or NaN in V would
// still reach the output, so in the tiles that hold nodes the softmax warps
// zero every element of a node's V that is no number (and the slots' rows past
// the last token); a node that does see such an element gets it added to its
// output afterwards.  Cached tokens are seen by every node of the row and need
// no such care.
#include <atomic>
#include <mutex>

#include "fp8_codec.cuh"
#include "pkv_internal.cuh"
#include "tcgen05.cuh"
#include "tree_split.cuh"

namespace pkv {
namespace tree {
using namespace tc;

constexpr int kTile = 128;     // tokens of a tile
constexpr int kSoftWarps = 8;
constexpr int kSIssue = 8, kPvIssue = 9, kLoad = 10, kConv = 12;  // warp roles
constexpr int kConvWarps = 4;
constexpr int kMaxRows = 1024;
constexpr int kMaxGrid = 192;  // blocks: one per SM, at most this many
constexpr int kMaxWords = 32;  // mask words: up to 1024 nodes a row
constexpr int kHeadInts = 32;  // ints between two units' words: count, then given-up blocks' bits
constexpr uint32_t kHalfQ = kRows * 128;   // 128 flat rows x 64 dims
constexpr uint32_t kQBlock = 2 * kHalfQ;
constexpr uint32_t kKHalf = kTile * 128;   // 128 tokens x 64 dims
constexpr uint32_t kKSlot = 2 * kKHalf;    // a K tile: dims lo, hi
constexpr uint32_t kVHalf = kGrain * 128;  // 64 tokens x 64 dims
constexpr uint32_t kVSlot = 2 * kVHalf;    // half a V tile: dims lo, hi
constexpr uint32_t kRaw = kGrain * 128;    // a granule of codes
constexpr uint32_t kTmemCols = 512;
// A partial of one M block: m[128], l[128], then O as [32 groups of 4 dims][128 rows][4].
constexpr int kPartFloats = 2 * kRows + kRows * kHeadDim;
constexpr uint32_t kHelpNs = 100000;  // how long a block waits for a unit's other pieces
constexpr float kLog2e = 1.4426950408889634f;
// A row's reference lies 7 below its maximum at the time, which then weighs 2^7, and moves
// when a score passes it by more than 15: weights up to 2^15 are fp16 numbers, and the
// smallest normal one is 2^-21 of the first maximum's (with the reference at the
// maximum: 2^-14, and weights below 2^-25 were lost to the output while the row's sum
// kept them).  The reference is what every difference is taken from, so its own rounding
// is in all of them alike.
constexpr float kWeightLog2 = 7.f, kMoveLog2 = 15.f;
constexpr int kSBufs = 3;        // S buffers of 128 columns
constexpr uint32_t kColS = 128;  // above the accumulator's 128 columns

template <bool kFp8>
__host__ __device__ constexpr int threads() { return (kConv + (kFp8 ? kConvWarps : 0)) * 32; }

// n / d for 0 <= n < 2^31 and d >= 2: with 2^(l - 1) < d <= 2^l and m = ceil(2^(31 + l) / d),
// n m / 2^(31 + l) is above n / d by less than 1 / d.
struct By {
    uint32_t m;
    int shift;
    void set(int d) {
        int l = 1;
        while ((1ll << l) < d) ++l;
        m = (uint32_t)(((1ull << (31 + l)) + d - 1) / d);
        shift = l - 1;
    }
    __device__ __forceinline__ int operator()(int n) const { return (int)(__umulhi((uint32_t)n, m) >> shift); }
};

struct Params {
    const __half* q;
    __half* out;
    const void* v_pool;
    const float* k_scale;
    const float* v_scale;
    const int32_t* tables;
    const int32_t* seq_lens;
    const int32_t* q_start;
    const uint32_t* mask;
    int words;
    int rows, total, hq, hk, group, bs, mbpr, nb, limit;
    Planes planes;
    int box;       // log2 of the tokens per copy
    By by_bs;      // block_size
    float scale;
    float* part;   // [grid][2][kPartFloats]
    int* heads;    // [grid][kHeadInts], zero between calls: of the cut unit that starts in a block
    uint32_t help_ns;  // kHelpNs, but for tests
    uint32_t stop;     // for tests: blocks that fold give up once the copy is issued
    uint32_t linger_ns;  // for tests: how long warp 0 stays behind at each segment's end
    int32_t* dev_err;
};

// Shared memory.
template <bool kFp8>
struct Smem {
    static constexpr int kslots = kFp8 ? 2 : 3;  // tiles
    static constexpr int vslots = kFp8 ? 4 : 5;  // granules (4 at least: see the wait for V's tiles that hold nodes)
    static constexpr int raws = kFp8 ? 3 : 0;    // granules of codes, of K and of V
    static constexpr uint32_t q = 0;
    static constexpr uint32_t kring = q + kQBlock;
    static constexpr uint32_t vring = kring + kslots * kKSlot;
    static constexpr uint32_t kraw = vring + vslots * kVSlot;
    static constexpr uint32_t vraw = kraw + raws * kRaw;
    static constexpr uint32_t bars = vraw + raws * kRaw;
    static constexpr uint32_t tmem = bars + 64 * 8;
    // last unit [6], range [2], abort, odd V; then of each of two cut units what this block took
    // over of it [6], the verdict, its pieces, the first block, the count, and r, k, t
    static constexpr uint32_t misc = tmem + 16;
    static constexpr uint32_t bad = misc + 192;                    // [32] granules: 16-token groups not to be seen
    static constexpr uint32_t ref = bad + 128;                     // [2] jobs' reference maxima [128]
    static constexpr uint32_t sum = ref + 2 * kRows * 4;           // of a segment and the one before: [2 groups] last references, row sums [128]
    static constexpr uint32_t rowc = sum + 8 * kRows * 4;          // per row: nodes
    static constexpr uint32_t rowp = rowc + kMaxRows * 4;          // per row: cached tokens
    // the scan's scratch lives in the K ring: it is read before the first copy is issued
    static constexpr uint32_t part = kring;
    static constexpr uint32_t total = rowp + kMaxRows * 4 + 1024;
    static_assert(kring % 1024 == 0 && vring % 1024 == 0 && kraw % 1024 == 0, "swizzled tiles need 1024-byte alignment");
    static_assert(total <= 232448, "shared memory per block");
    static_assert(kslots * kKSlot + vslots * kVSlot >= kPartFloats * 4, "a partial fits the rings");
    static_assert(vslots >= 4, "two tiles before this one, a slot of it was filled for the last time");
    static_assert(2 * (kslots + vslots + 2 * raws) + 3 * kSBufs + 16 <= 64, "barriers");
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool valid) {
    const uint32_t bytes = valid ? 16u : 0u;  // nothing is read when it is not: zeros are written
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(addr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}
// Columns c .. c + 15 of this warp's 32 lanes, and the wait.
__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
        : "r"(addr)
        : "memory");
}
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void sts16(uint32_t addr, uint4 v) {
    asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
                 : "memory");
}
__device__ __forceinline__ uint2 lds8(uint32_t addr) {
    uint2 v;
    asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
    return v;
}
__device__ __forceinline__ uint4 lds16(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
    return v;
}
// Nonzero bits 15 / 31: the word's low / high half is an infinity or NaN.
__device__ __forceinline__ uint32_t no_number(uint32_t w) { return ((w & 0x7c007c00u) + 0x04000400u) & 0x80008000u; }

// The waits of tcgen05.cuh with everything but the first try out of line: the
// roles' loops share the instruction cache, which they would not fit.
__device__ __noinline__ bool waitw_slow(uint32_t bar, uint32_t parity, const volatile int* abort) {
    return mbar_waitw(bar, parity, abort);
}
__device__ __forceinline__ bool waitw(uint32_t bar, uint32_t parity, const volatile int* abort) {
    return __all_sync(0xffffffffu, mbar_try_wait_sleep(bar, parity)) || waitw_slow(bar, parity, abort);
}
// Lanes 0 to 3 (and the others with lane 3) each name a barrier: one look at all
// of them together, for the latency of one, and where that does not do, one
// wait after the other.  (Waits that sleep take one address for the warp.)
__device__ __noinline__ bool wait4_slow(uint32_t bar, uint32_t parity, const volatile int* abort) {
    bool ok = true;
#pragma unroll 1
    for (int i = 0; ok && i < 4; ++i)
        ok = mbar_waitw(__shfl_sync(0xffffffffu, bar, i), __shfl_sync(0xffffffffu, parity, i), abort);
    return ok;
}
__device__ __forceinline__ bool wait4(uint32_t bar, uint32_t parity, const volatile int* abort) {
    uint32_t there;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(there)
        : "r"(bar), "r"(parity)
        : "memory");
    return __all_sync(0xffffffffu, there) || wait4_slow(bar, parity, abort);
}
__device__ __noinline__ bool drain1(uint32_t bar, uint32_t parity) { return mbar_drain1(bar, parity); }

// A ring's slot and fill parity, advanced a slot at a time.
template <int kSlots>
struct Ring {
    int s = 0;
    uint32_t ph = 0;
    __device__ __forceinline__ void next() {
        if (++s == kSlots) {
            s = 0;
            ph ^= 1;
        }
    }
};

// 32 mask bits of a node from node index j0 on (j0 > -32; bits of negative
// nodes, cached tokens, are set).
__device__ __forceinline__ uint32_t mask_bits(const uint32_t* row, int words, int j0) {
    auto word = [&](int i) -> uint32_t { return i < words ? row[i] : 0u; };
    if (j0 < 0) return (word(0) << -j0) | ((1u << -j0) - 1);
    return __funnelshift_r(word(j0 >> 5), word((j0 >> 5) + 1), j0 & 31);
}
__device__ __forceinline__ uint32_t low_bits(int n) { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1; }

// A node's V that is no number reaches the rows that see it: such elements of
// dims d0 .. d0 + 63 of nodes j0 .. j1 - 1 are added to this thread's stored
// output (`orow`, fp16) or partial (`po`, dim group e at po[e * kRows]).
template <bool kFp8>
__device__ __noinline__ void add_odd(const Params& p, int r, int P, int j0, int j1, int node, int g, int kvh, int d0,
                                     __half* orow, float4* po) {
#pragma unroll 1
    for (int j = j0; j < j1; ++j) {
        const bool sees = p.mask ? (p.mask[(int64_t)g * p.words + (j >> 5)] >> (j & 31)) & 1 : j <= node;
        if (!sees) continue;
        const int t = P + j, pb = p.tables[(int64_t)r * p.mbpr + t / p.bs];
        if (pb < 0 || pb >= p.nb) continue;
        const int64_t at = (((int64_t)pb * p.bs + t % p.bs) * p.hk + kvh) * kHeadDim + d0;
#pragma unroll 1
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

// A share of merging a unit cut over P blocks, the first of them `first`: (32
// flat rows) x (4 dims) a warp's turn, turn w of all blocks' warps together, every
// 8 P-th; eight pieces' loads are in flight together (ten: 2% slower for a unit of 16
// pieces, 1% faster for one of 19; sixteen spill).  `dry`: one turn without its store (see its
// call).
constexpr int kMergeAtOnce = 8;
__device__ __noinline__ void merge_share(const Params& p, int k, int f0, int q0, int nq, int P, int first, int piece,
                                         float vs, bool dry) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int jobs = (nq + 31) / 32 * 32;
#pragma unroll 1
    for (int job = piece * kSoftWarps + warp; job < jobs; job += P * kSoftWarps) {
        const int cc = job & 31, i = (job & ~31) + lane;  // dims 4 cc .. of flat row i of the unit
        if (i >= nq) continue;
        float M = -INFINITY, Lt = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
        for (int j0 = 0; j0 < P; j0 += kMergeAtOnce) {
            // (no branch between the loads: past the last piece it is read again and left out)
            float mj[kMergeAtOnce], lj[kMergeAtOnce];
            float4 x[kMergeAtOnce];
#pragma unroll
            for (int j = 0; j < kMergeAtOnce; ++j) {
                const int jj = min(j0 + j, P - 1);
                const float* s = p.part + ((int64_t)(first + jj) * 2 + (jj == P - 1)) * kPartFloats;
                mj[j] = __ldcg(s + i);
                lj[j] = __ldcg(s + kRows + i);
                x[j] = __ldcg(reinterpret_cast<const float4*>(s + 2 * kRows) + cc * kRows + i);
            }
#pragma unroll
            for (int j = 0; j < kMergeAtOnce; ++j) {
                // (a piece that the row sees nothing of; one of NaN scores alone has that reference
                // too, and a sum that is NaN)
                if (j0 + j >= P || (mj[j] == -INFINITY && lj[j] == 0.f)) continue;
                const float mn = fmaxf(M, mj[j]);
                const float a = M == -INFINITY ? 0.f : fast_exp2(M - mn), w = fast_exp2(mj[j] - mn);
                M = mn;
                Lt = Lt * a + w * lj[j];
                acc.x = acc.x * a + w * x[j].x;
                acc.y = acc.y * a + w * x[j].y;
                acc.z = acc.z * a + w * x[j].z;
                acc.w = acc.w * a + w * x[j].w;
            }
        }
        if (dry) return;
        const float inv = Lt == 0.f ? 0.f : __fdividef(vs, Lt);
        const int f = f0 + i, node = div_of(f, p.group);
        *reinterpret_cast<uint2*>(p.out + ((int64_t)(q0 + node) * p.hq + k * p.group + (f - node * p.group)) * kHeadDim + 4 * cc) =
            make_uint2(pack_half2(acc.x * inv, acc.y * inv), pack_half2(acc.z * inv, acc.w * inv));
    }
}

// The weights of the two pieces of a unit, `a` the first's, and the normalisation in them:
// one order of operations for the fold and for the merge of a pair, so that the
// result is the same whichever was done.
__device__ __forceinline__ void pair_weights(float ma, float la, float mb, float lb, float vs, float& a, float& b) {
    const float M = fmaxf(ma, mb);
    a = ma == -INFINITY ? 0.f : fast_exp2(ma - M);
    b = mb == -INFINITY ? 0.f : fast_exp2(mb - M);
    const float L = __fmaf_rn(lb, b, __fmul_rn(la, a));
    const float inv = L == 0.f ? 0.f : __fdividef(vs, L);
    a *= inv;
    b *= inv;
}
__device__ __forceinline__ float pair_sum(float x, float a, float y, float b) { return __fmaf_rn(x, a, __fmul_rn(y, b)); }

// The merge of a unit cut in two, whose second block did not wait for the first: all of it,
// by the eight softmax warps of whichever block stored its piece last.
__device__ __noinline__ void merge_pair(const Params& p, int k, int f0, int q0, int nq, int first, float vs) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const float* s = p.part + (int64_t)first * 2 * kPartFloats;  // the second piece: of the next block, its slot 1
    const float* z = s + 3 * kPartFloats;
#pragma unroll 1
    for (int job = warp; job < (nq + 31) / 32 * 32; job += kSoftWarps) {
        const int cc = job & 31, i = (job & ~31) + lane;
        if (i >= nq) continue;
        float a, b;
        pair_weights(__ldcg(s + i), __ldcg(s + kRows + i), __ldcg(z + i), __ldcg(z + kRows + i), vs, a, b);
        const float4 x = __ldcg(reinterpret_cast<const float4*>(s + 2 * kRows) + cc * kRows + i);
        const float4 y = __ldcg(reinterpret_cast<const float4*>(z + 2 * kRows) + cc * kRows + i);
        const int f = f0 + i, node = div_of(f, p.group);
        *reinterpret_cast<uint2*>(p.out + ((int64_t)(q0 + node) * p.hq + k * p.group + (f - node * p.group)) * kHeadDim + 4 * cc) =
            make_uint2(pack_half2(pair_sum(x.x, a, y.x, b), pair_sum(x.y, a, y.y, b)),
                       pack_half2(pair_sum(x.z, a, y.z, b), pair_sum(x.w, a, y.w, b)));
    }
}

// A wrapping increment: the word goes back to zero after 2 P of them.
__device__ __forceinline__ int count_up(int* word, int P) {
    unsigned old;
    asm volatile("atom.acq_rel.gpu.global.inc.u32 %0, [%1], %2;" : "=r"(old) : "l"(word), "r"(2 * P - 1) : "memory");
    return (int)old;
}

// Of two pieces, the first (0) or the second (1), whose block did not wait, is stored: nonzero
// when the other one was stored before, and its block leaves the merge to this one.
__device__ __forceinline__ int count_pair(int* word, int piece) {
    int old;
    asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], %2;" : "=r"(old) : "l"(word), "r"(1 + piece) : "memory");
    return old;
}

__device__ __noinline__ void linger(uint32_t ns) {
    const uint64_t from = now_ns();
    while (now_ns() - from < ns) __nanosleep(100);
}

// One thread of each of a cut unit's blocks, after its own piece was counted as
// the n-th: waits for the others and says whether the block merges its share.
// `head`: the count, then a bit for each piece whose block gave up.  A block
// that gives up sets its bit and then looks at the count once more; the last
// one to arrive counts and then looks at the bits: one of the two sees the
// other, and whoever takes the bit away does the share (the last block gets the
// pieces it took in `taken`).  Every block, or the last one in its place, counts
// a second time, which brings the word back to zero.
__device__ __forceinline__ bool gather(int* head, int P, int piece, int n, uint32_t help_ns, volatile int* taken) {
    const bool last = n == P;
    const uint64_t t0 = now_ns();
    while (n < P) {
        if (now_ns() - t0 > help_ns) {
            int* word = head + 1 + (piece >> 5);
            const int bit = 1 << (piece & 31);
            atomicOr(word, bit);
            __threadfence();
            asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(n) : "l"(head) : "memory");
            if (n < P || !(atomicAnd(word, ~bit) & bit)) return false;
            break;
        }
        __nanosleep(20);
        asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(n) : "l"(head) : "memory");
    }
    count_up(head, P);
    if (last) {
        __threadfence();
        for (int i = 0; i < (P + 31) / 32; ++i) {
            if (!*reinterpret_cast<volatile int*>(head + 1 + i)) continue;
            const int bits = atomicExch(head + 1 + i, 0);
            taken[i] = bits;
            taken[13] = 1;
            for (int k = __popc(bits); k > 0; --k) count_up(head, P);
        }
    }
    return true;
}

template <bool kFp8>
__global__ void __launch_bounds__(threads<kFp8>(), 1)
    tree_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                const __grid_constant__ Params p) {
    using S = Smem<kFp8>;
    constexpr int kUnitCost = unit_cost<kFp8>();
    using Walk = tree::Walk<kUnitCost>;
    extern __shared__ unsigned char smem_raw[];
    unsigned char* smem = reinterpret_cast<unsigned char*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(smem);
    const uint32_t bar_kfull = sbase + S::bars;                // [K slots]
    const uint32_t bar_kempty = bar_kfull + S::kslots * 8;
    const uint32_t bar_vfull = bar_kempty + S::kslots * 8;     // [V slots]
    const uint32_t bar_vempty = bar_vfull + S::vslots * 8;
    const uint32_t bar_krfull = bar_vempty + S::vslots * 8;    // [raw slots] of K codes
    const uint32_t bar_krempty = bar_krfull + S::raws * 8;
    const uint32_t bar_vrfull = bar_krempty + S::raws * 8;     // [raw slots] of V codes
    const uint32_t bar_vrempty = bar_vrfull + S::raws * 8;
    const uint32_t bar_s = bar_vrempty + S::raws * 8;          // [S buffers]: computed
    const uint32_t bar_p = bar_s + 8 * kSBufs;                 // [S buffers]: P written
    const uint32_t bar_o = bar_p + 8 * kSBufs;                 // [S buffers]: P's product done
    const uint32_t bar_m = bar_o + 8 * kSBufs;                 // [8 softmax warps]: a job's references known
    const uint32_t bar_l = bar_m + 8 * kSoftWarps;             // both groups' row sums of a segment written
    const uint32_t bar_qfree = bar_l + 8;                      // a segment's S products are done with its queries
    const uint32_t bar_fin = bar_qfree + 8;                    // a segment's last PV product is done
    const uint32_t bar_odrained = bar_fin + 8;                 // the softmax warps have read a segment's O out
    const uint32_t bar_sfin = bar_odrained + 8;                // the S issuer's last products are complete
    const uint32_t bar_pfin = bar_sfin + 8;                    // the PV issuer's last products are complete
    const uint32_t bar_pub = bar_pfin + 8;                     // the softmax warps have written a partial
    const uint32_t bar_go = bar_pub + 8;                       // a cut unit's pieces are all there (or given up)
    uint32_t* sm_tmem = reinterpret_cast<uint32_t*>(smem + S::tmem);
    volatile int* sm_misc = reinterpret_cast<volatile int*>(smem + S::misc);
    const volatile int* abort = sm_misc + 8;
    volatile uint32_t* sm_bad = reinterpret_cast<volatile uint32_t*>(smem + S::bad);
    int* sm_part = reinterpret_cast<int*>(smem + S::part);
    int* sm_C = reinterpret_cast<int*>(smem + S::rowc);
    int* sm_P = reinterpret_cast<int*>(smem + S::rowp);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rows = p.rows, group = p.group;

    // ---- barriers, tensor memory, descriptors ----
    if (tid == kPvIssue * 32) {
        const int fill = kFp8 ? kConvWarps / 2 : 1;
        for (int s = 0; s < S::kslots; ++s) {
            mbar_init(bar_kfull + 8 * s, fill);
            mbar_init(bar_kempty + 8 * s, 1);
        }
        for (int s = 0; s < S::vslots; ++s) {
            mbar_init(bar_vfull + 8 * s, fill);
            mbar_init(bar_vempty + 8 * s, 1);
        }
        for (int s = 0; s < S::raws; ++s) {
            mbar_init(bar_krfull + 8 * s, 1);
            mbar_init(bar_krempty + 8 * s, kConvWarps / 2);
            mbar_init(bar_vrfull + 8 * s, 1);
            mbar_init(bar_vrempty + 8 * s, kConvWarps / 2);
        }
        for (int b = 0; b < kSBufs; ++b) {
            mbar_init(bar_s + 8 * b, 1);
            mbar_init(bar_p + 8 * b, kSoftWarps / 2);
            mbar_init(bar_o + 8 * b, 1);
        }
        for (int b = 0; b < kSoftWarps; ++b) mbar_init(bar_m + 8 * b, 1);
        mbar_init(bar_l, kSoftWarps);
        mbar_init(bar_qfree, 1);
        mbar_init(bar_fin, 1);
        mbar_init(bar_odrained, kSoftWarps);
        mbar_init(bar_sfin, 1);
        mbar_init(bar_pfin, 1);
        mbar_init(bar_pub, kSoftWarps);
        mbar_init(bar_go, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kLoad && lane < 2)
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(lane ? &vmap : &kmap)) : "memory");
    if (warp == kSIssue) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(sbase + S::tmem),
                     "r"(kTmemCols));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }

    ptx::griddep_wait();  // what came before in the stream is complete

    // ---- per row: nodes, cached tokens, its units' length in each plane; the planes'
    // prefixes.  Two halves of the block do the same, six warps each: one for
    // the range's lower cut, one for the upper.  One warp's dependent instructions
    // take some five clocks each, so what counts here is their number ----
    constexpr int kHalfWarps = 6;
    const int side = warp >= kHalfWarps, hw = warp - side * kHalfWarps;  // further warps only wait
    const int per = (rows + kHalfWarps * 32 - 1) / (kHalfWarps * 32), r0 = (hw * 32 + lane) * per;
    const Planes planes = p.planes;
    int sum[kPlanes] = {0, 0, 0, 0}, incl[kPlanes];
    if (hw < kHalfWarps) {
#pragma unroll 1
        for (int r = r0; r < min(r0 + per, rows); ++r) {
            const int q0 = p.q_start[r], L = p.seq_lens[r];
            int C = p.q_start[r + 1] - q0;
            if (C < 0 || L < C || L > p.limit || q0 < 0 || q0 > p.total - C) {
                if (blockIdx.x == 0) flag_error(p.dev_err, PKV_DEV_ERR_SEQ_LEN);
                C = 0;
            } else if (p.mask && C > 32 * p.words) {
                if (blockIdx.x == 0) flag_error(p.dev_err, PKV_DEV_ERR_MASK);
                C = 0;
            }
            if (side == 0) {
                sm_C[r] = C;
                sm_P[r] = L - C;
            }
            // a unit's length (all units' together stay below kTooMuch, checked by the host for starts
            // that rise)
            const int len = C > 0 ? p.hk * ((L + kGrain - 1) / kGrain + kUnitCost) : 0;
            sum[0] = add_work(sum[0], len * planes.blocks(C * group, 0));
            if (planes.n > 1) {
#pragma unroll
                for (int x = 1; x < kPlanes; ++x)
                    if (x < planes.n) sum[x] = add_work(sum[x], len * planes.blocks(C * group, x));
            }
        }
        auto scan = [&](int x) {
            incl[x] = sum[x];
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int t = __shfl_up_sync(0xffffffffu, incl[x], o);
                if (lane >= o) incl[x] = add_work(incl[x], t);
            }
            if (lane == 31) sm_part[(x * 2 + side) * 8 + hw] = incl[x];
        };
        scan(0);
        if (planes.n > 1) {
#pragma unroll
            for (int x = 1; x < kPlanes; ++x)
                if (x < planes.n) scan(x);
        }
    }
    if (tid < 48) sm_misc[tid] = 0;
    __syncthreads();

    // ---- this block's plane, the plane's blocks, and its range: the thread whose
    // row a cut falls in moves the cut ----
    int plane = 0, base_block = 0, run = 0, mine = 0;
    Split<kUnitCost> sp;
    sp.W = 0;
    {
        // of this half's warps: the work before this one and the whole plane's
        auto plane_of = [&](int x, int& before) -> int {
            int v = lane < kHalfWarps ? sm_part[(x * 2 + side) * 8 + lane] : 0;
#pragma unroll
            for (int o = 1; o < 8; o <<= 1) {
                const int t = __shfl_up_sync(0xffffffffu, v, o);
                if (lane >= o) v = add_work(v, t);
            }
            before = __shfl_sync(0xffffffffu, v, max(hw - 1, 0));
            if (hw == 0) before = 0;
            return __shfl_sync(0xffffffffu, v, kHalfWarps - 1);
        };
        int before;
        int W = plane_of(0, before);
        int from = 0, to = (int)gridDim.x;
        if (planes.n > 1) {
            int Wi[kPlanes], bf[kPlanes];
            Wi[0] = W;
            bf[0] = before;
            bool fits = W < kTooMuch;
#pragma unroll
            for (int x = 1; x < kPlanes; ++x) {
                Wi[x] = bf[x] = 0;
                if (x < planes.n) Wi[x] = plane_of(x, bf[x]);
                fits = fits && Wi[x] < kTooMuch;
            }
            if (!fits) {  // (rows of one M block each always fit)
                if (blockIdx.x == 0 && tid == 0) flag_error(p.dev_err, PKV_DEV_ERR_SEQ_LEN);
#pragma unroll
                for (int x = 0; x < kPlanes; ++x) Wi[x] = 0;
            }
            const Share s = share_of(Wi, planes, (int)gridDim.x, (int)blockIdx.x);
            plane = s.plane;
            W = s.W;
            from = s.from;
            to = s.to;
#pragma unroll
            for (int x = 0; x < kPlanes; ++x)
                if (x == plane) before = bf[x];
        }
        if (W > 0) {
            base_block = from;
            int i = incl[0], m = sum[0];
            if (planes.n > 1) {
#pragma unroll
                for (int x = 1; x < kPlanes; ++x)
                    if (x == plane) {
                        i = incl[x];
                        m = sum[x];
                    }
            }
            run = before + i - m;
            mine = hw < kHalfWarps ? m : 0;
            sp.set(W, to - from, unit_slack<kFp8>());
        }
    }
    const int cta = (int)blockIdx.x - base_block;
    if (sp.W > 0 && cta < sp.G) {
        // the lower cut lies in [run, run + mine) of one thread of the first half, the upper one
        // in (run, run + mine] of one of the second
        const int x = sp.raw(cta + side), in = x - side;
        if (in >= run && in < run + mine) {
            Walk u;
            u.hk = p.hk;
            u.group = group;
            u.plane = plane;
            u.planes = planes;
            u.C = sm_C;
            u.P = sm_P;
            u.r = r0;
            const int cut = place_cut(u, sp, x, side, run);
            if (side == 0) {
                sm_misc[6] = cut;
            } else {
                sm_misc[0] = u.r;
                sm_misc[1] = u.k;
                sm_misc[2] = u.t;
                sm_misc[3] = u.U;
                sm_misc[4] = u.n;
                sm_misc[7] = cut;
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *sm_tmem;
    auto raise_abort = [&]() { sm_misc[8] = 1; };

    Walk w;
    w.r = sm_misc[0];
    w.k = sm_misc[1];
    w.t = sm_misc[2];
    w.U = sm_misc[3];
    w.n = sm_misc[4];
    w.s0 = sm_misc[6];
    w.e = sm_misc[7];
    w.hk = p.hk;
    w.group = group;
    w.plane = plane;
    w.planes = planes;
    w.C = sm_C;
    w.P = sm_P;

    // A unit's flat rows (256 bytes a row, swizzled; rows past the last are zeros), by one warp.
    auto load_queries = [&](const Walk& u) {
        const int F = u.flat(), q0 = p.q_start[u.r], ch = lane & 15;
        const uint32_t dst0 = sbase + S::q + (ch >> 3) * kHalfQ;
#pragma unroll 1
        for (int j = 0; j < kRows; j += 32) {
            // of flat row j + lane: (node, head) index, or -1
            const int f = u.f0() + j + lane, node = div_of(f, group);
            const int at = f < F ? (q0 + node) * p.hq + u.k * group + (f - node * group) : -1;
#pragma unroll 4
            for (int x = 0; x < 16; ++x) {
                const int rr = 2 * x + (lane >> 4);
                const int a = __shfl_sync(0xffffffffu, at, rr);
                cp_async16(dst0 + (j + rr) * 128 + (((ch & 7) ^ (rr & 7)) << 4),
                           p.q + (int64_t)max(a, 0) * kHeadDim + ch * 8, a >= 0);
            }
        }
    };

    if (w.s0 >= w.e) {
        // no work, or both cuts moved to one border: nothing but to free the tensor memory below
    } else if (warp == kLoad || warp == kLoad + 1) {
        // ============================== TMA ==============================
        // K tiles or V granules (FP8: granules of codes).  Table entries are
        // fetched a batch ahead: lane l handles box l % gpu of copy unit l / gpu
        // of a batch, so the table's latency is paid once a batch.
        const bool is_v = warp == kLoad + 1;
        const int nslots = kFp8 ? S::raws : is_v ? S::vslots : S::kslots;
        const int unit_tok = kFp8 || is_v ? kGrain : kTile;
        const uint32_t full0 = kFp8 ? (is_v ? bar_vrfull : bar_krfull) : (is_v ? bar_vfull : bar_kfull);
        const uint32_t empty0 = kFp8 ? (is_v ? bar_vrempty : bar_krempty) : (is_v ? bar_vempty : bar_kempty);
        const uint32_t ring = sbase + (kFp8 ? (is_v ? S::vraw : S::kraw) : (is_v ? S::vring : S::kring));
        const uint32_t slot_bytes = kFp8 ? kRaw : is_v ? kVSlot : kKSlot;
        const uint32_t half_bytes = slot_bytes / 2;
        const CUtensorMap* map = is_v ? &vmap : &kmap;
        const int box = 1 << p.box;
        const int per_unit = (kFp8 || is_v ? kGrainLog : kGrainLog + 1) - p.box, upb = 32 >> per_unit;  // log2 boxes a unit
        const int my_j = lane >> per_unit, my_g = lane & ((1 << per_unit) - 1);
        const uint32_t box_bytes = (uint32_t)box * 128;
        const int nowhere = p.nb * p.bs;  // a row past the pool: a copy of zeros
        int s = 0, armed = 0, grain = 0;
        uint32_t ph = 0, fb = full0, eb = empty0, slot = ring;
        bool ok = true;
        do {
            const int ta = w.ta(), te = w.te();
            const int units = (te - ta + unit_tok - 1) / unit_tok;
            const int32_t* trow = p.tables + (int64_t)w.r * p.mbpr;
            auto fetch = [&](int ub) -> int {  // raw block id of this lane's box in the batch at copy unit ub
                const int tok = ta + (ub + my_j) * unit_tok + my_g * box;
                return tok < te ? trow[p.by_bs(tok)] : 0;
            };
            auto to_row = [&](int ub, int pb) -> int {  // its pool row, or -1 for no copy
                const int tok = ta + (ub + my_j) * unit_tok + my_g * box;
                if (tok >= te) return -1;
                if (pb < 0 || pb >= p.nb) {
                    if (!is_v) flag_error(p.dev_err, PKV_DEV_ERR_BLOCK_ID);
                    return nowhere;
                }
                return pb * p.bs + tok - p.by_bs(tok) * p.bs;
            };
            int pb = fetch(0), row = -1, j = 0;
#pragma unroll 1
            for (int u = 0; u < units; ++u) {
                if (j == 0) {
                    row = to_row(u, pb);
                    pb = fetch(u + upb);
                }
                if (!waitw(eb, ph ^ 1, abort)) {
                    ok = false;
                    break;
                }
                const bool issue = my_j == j && row >= 0;
                const uint32_t nissue = __popc(__ballot_sync(0xffffffffu, issue));
                if (!is_v) {
                    // groups of 16 tokens whose table entry is out of range: read by the softmax
                    // warps at this tile, before the word's next use 32 granules on (the rings
                    // and S buffers hold fewer between the two)
                    const uint32_t mine = issue && row == nowhere ? ((1u << (box / 16)) - 1) << (my_g * (box / 16)) : 0;
                    const uint32_t all = __reduce_or_sync(0xffffffffu, mine);
                    const bool two = !kFp8 && te - ta - u * kTile > kGrain;
                    if (lane < 1 + two) sm_bad[(grain + lane) & 31] = all >> (4 * lane);
                    __syncwarp();  // lane 1's word too is written before lane 0 arrives
                    grain += 1 + two;
                }
                if (lane == 0) mbar_arrive_expect_tx(fb, nissue * (kFp8 ? 1 : 2) * box_bytes);
                __syncwarp();
                if (issue) {
                    const uint32_t st = slot + my_g * box_bytes;
                    tma_load_3d(st, map, 0, w.k, row, fb);
                    if (!kFp8) tma_load_3d(st + half_bytes, map, 64, w.k, row, fb);
                }
                ++armed;
                if (++j == upb) j = 0;
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
#pragma unroll 1
        for (int u = max(0, armed - nslots); u < armed; ++u)
            if (!drain1(full0 + 8 * (u % nslots), (uint32_t)(u / nslots) & 1) && lane == 0)
                flag_error(p.dev_err, PKV_DEV_ERR_TIMEOUT);
        __syncwarp();
    } else if (kFp8 && warp >= kConv) {
        // ========================= FP8: widening =========================
        // Two warps for K and two for V, so that neither waits for the other's slots (in one
        // sequence the next tile's K came after this tile's V, whose slots are free only after
        // the product two tiles before).  Thread (warp c, lane l) widens 8 codes (chunk l % 16) of
        // tokens 32 c + l / 16 + 2 i of a granule: eight lanes write one row's 128 bytes of one
        // half, so all banks at once.  Rows past the last token hold whatever the slot held:
        // never seen.
        const int c = (warp - kConv) & 1, col = lane & 15;
        const bool is_v = warp - kConv >= 2;
        uint32_t from[4], to[4];  // rows i and i + 4 have the same swizzle
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = 32 * c + (lane >> 4) + 2 * i;
            from[i] = sbase + (is_v ? S::vraw : S::kraw) + r * 128 + (((col >> 1) ^ (r & 7)) << 4) + (col & 1) * 8;
            to[i] = sbase + (is_v ? S::vring + (col >> 3) * kVHalf : S::kring + (col >> 3) * kKHalf) + r * 128 +
                    (((col & 7) ^ (r & 7)) << 4);
        }
        const uint32_t rfull0 = is_v ? bar_vrfull : bar_krfull, rempty0 = is_v ? bar_vrempty : bar_krempty;
        const uint32_t full0 = is_v ? bar_vfull : bar_kfull, empty0 = is_v ? bar_vempty : bar_kempty;
        Ring<S::raws ? S::raws : 1> raw;
        int slot = 0;  // of the operand ring
        uint32_t slot_ph = 0;
        bool ok = true;
        do {
            const int g1 = w.g1();
#pragma unroll 1
            for (int g = w.g0(), h = 0; g < g1; ++g) {
                // h: the granule of its tile; a tile's K is one slot, its V a slot a granule
                if (!(ok = wait4(lane == 0 ? empty0 + 8 * slot : rfull0 + 8 * raw.s, lane == 0 ? slot_ph ^ 1 : raw.ph,
                                 abort)))
                    break;
                const uint32_t src = raw.s * kRaw, dst = is_v ? slot * kVSlot : slot * kKSlot + h * (kGrain * 128);
#pragma unroll 1
                for (int b = 0; b < 4096; b += 2048) {
                    uint2 x[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) x[i] = lds8(src + b + from[i & 3] + (i >> 2) * 1024);
#pragma unroll
                    for (int i = 0; i < 8; ++i) sts16(dst + b + to[i & 3] + (i >> 2) * 1024, widen8(x[i]));
                }
                fence_async_smem();
                __syncwarp();
                const bool full = is_v || h || g + 1 == g1;
                if (lane == 0) {
                    mbar_arrive(rempty0 + 8 * raw.s);
                    if (full) mbar_arrive(full0 + 8 * slot);
                }
                raw.next();
                h = is_v ? 0 : h ^ 1;
                if (full && ++slot == (is_v ? S::vslots : S::kslots)) {
                    slot = 0;
                    slot_ph ^= 1;
                }
            }
        } while (ok && w.prev());
        if (!ok && lane == 0) {
            raise_abort();
            flag_error(p.dev_err, PKV_DEV_ERR_TIMEOUT);
        }
        __syncwarp();
    } else if (warp == kSIssue) {
        // ====================== queries and S issue ======================
        // Per segment the warp brings the unit's flat rows in once the previous
        // segment's products no longer read the buffer.  Then job after job: S = Q . K^T
        // into the next S buffer, once the tile has landed and the P that the
        // buffer held has been used.  The warp stays together and one lane
        // issues: with the loop in one lane's branch the warp ran split from the
        // second segment on, and its query loads took 11 us instead of 1.6.
        const uint32_t id_s = idesc(kRows, kTile, 0);
        const uint64_t kd0 = sdesc(sbase + S::kring, 16, 1024);
        const uint64_t qd0 = sdesc(sbase + S::q, 16, 1024);
        Ring<S::kslots> k;
        Ring<kSBufs> b;
        int seg = 0;
        bool ok = true;
        do {
            // (parities of a phase before the first: such a wait passes at once)
            if (!(ok = waitw(bar_qfree, (uint32_t)(seg + 1) & 1, abort))) break;
            load_queries(w);
            asm volatile("cp.async.wait_all;" ::: "memory");
            fence_async_smem();
            __syncwarp();
            const int te = w.te();
#pragma unroll 1
            for (int t0 = w.ta(); ok && t0 < te; t0 += kTile) {
                if (!(ok = wait4(lane ? bar_o + 8 * b.s : bar_kfull + 8 * k.s, lane ? b.ph ^ 1 : k.ph, abort))) break;
                tc_fence_after();
                if (lane == 0) {
                    const uint64_t kd = kd0 + (uint64_t)(k.s * (kKSlot >> 4));
                    const uint32_t d = tmem + kColS + b.s * 128;
#pragma unroll
                    for (int ks = 0; ks < 8; ++ks) {
                        const uint64_t off = (uint64_t)(((ks >> 2) * kHalfQ + (ks & 3) * 32) >> 4);
                        umma_ss(d, qd0 + off, kd + off, id_s, ks > 0);
                    }
                    umma_commit(bar_s + 8 * b.s);
                    umma_commit(bar_kempty + 8 * k.s);  // the tile is no longer read
                }
                __syncwarp();
                b.next();
                k.next();
            }
            if (ok && lane == 0) umma_commit(bar_qfree);
            __syncwarp();
            ++seg;
        } while (ok && w.prev());
        if (lane == 0) {
            if (!ok) {
                raise_abort();
                flag_error(p.dev_err, PKV_DEV_ERR_TIMEOUT);
            }
            umma_commit(bar_sfin);
            if (!drain1(bar_sfin, 0)) flag_error(p.dev_err, PKV_DEV_ERR_TIMEOUT);
        }
        __syncwarp();
    } else if (warp == kPvIssue) {
        // ============================ PV issue ===========================
        // Job after job: O of its stream += P . V once V's tile has landed and
        // the softmax warps have stored P (and seen to V's rows that need it); a
        // segment's first products start the accumulators afresh, after the
        // previous segment's were read out.  K-steps past the last token are
        // skipped.
        const uint32_t id_o = idesc(kRows, 128, 1);
        // Merging comes last, when whole blocks wait for it, and would fetch its code from L2 first.
        // This warp has nothing to do before the first P, so it runs a turn of it now, which
        // leaves the code in the SM's cache: 1.0 us of 19 over ragged rows, 1.3 of 36 over four
        // rows of 32768.
        if (lane == 0) merge_share(p, 0, 0, 0, 1, 1, (int)blockIdx.x, 0, 1.f, true);
        __syncwarp();
        const uint64_t vd0 = sdesc(sbase + S::vring, kVHalf, 1024);
        Ring<S::vslots> v;
        Ring<kSBufs> b;
        int seg = 0;
        bool ok = true;
        do {
            const int ta = w.ta(), te = w.te();
#pragma unroll 1
            for (int t0 = ta; ok && t0 < te; t0 += kTile) {
                const int nsteps = (min(kTile, te - t0) + 15) / 16;
                const bool two = te - t0 > kGrain;
                // lane 0: V's first half; lane 1: its second; lane 2: the accumulator read out (a
                // segment's first product); the others: P
                uint32_t wbar = bar_p + 8 * b.s, wph = b.ph;
                const int va = v.s;
                if (lane == 0) wbar = bar_vfull + 8 * v.s, wph = v.ph;
                v.next();
                const int vb = v.s;
                if (two) {
                    if (lane == 1) wbar = bar_vfull + 8 * v.s, wph = v.ph;
                    v.next();
                }
                if (lane == 2 && t0 == ta) wbar = bar_odrained, wph = (uint32_t)(seg + 1) & 1;
                if (!(ok = wait4(wbar, wph, abort))) break;
                const uint64_t da = vd0 + (uint64_t)(va * (kVSlot >> 4)), db = vd0 + (uint64_t)(vb * (kVSlot >> 4));
                tc_fence_after();
                if (lane == 0) {
                    // tokens 64 e .. 64 e + 63 sit in columns 64 e .. 64 e + 31
                    const uint32_t pa = tmem + kColS + b.s * 128;
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk)
                        if (kk < nsteps)
                            umma_ts(tmem, pa + (kk >> 2) * 64 + (kk & 3) * 8, (kk < 4 ? da : db) + (uint64_t)((kk & 3) * 128),
                                    id_o, (t0 > ta || kk > 0) ? 1u : 0u);
                    umma_commit(bar_o + 8 * b.s);
                    umma_commit(bar_vempty + 8 * va);
                    if (two) umma_commit(bar_vempty + 8 * vb);
                    if (t0 + kTile >= te) umma_commit(bar_fin);
                }
                __syncwarp();
                b.next();
            }
            ++seg;
        } while (ok && w.prev());
        if (lane == 0) {
            if (!ok) {
                raise_abort();
                flag_error(p.dev_err, PKV_DEV_ERR_TIMEOUT);
            }
            umma_commit(bar_pfin);
            if (!drain1(bar_pfin, 0)) flag_error(p.dev_err, PKV_DEV_ERR_TIMEOUT);
        }
        __syncwarp();
    } else if (warp < kSoftWarps) {
        // ============================ softmax =============================
        const int quarter = warp & 3, wg = warp >> 2;
        const int i = quarter * 32 + lane;  // flat row of the M block, TMEM lane
        const uint32_t lane_base = (uint32_t)(quarter * 32) << 16;
        float* sm_ref = reinterpret_cast<float*>(smem + S::ref);  // [2][128]: of even and odd jobs
        bool ok = true;
        int job = 0, seg = 0;          // jobs and segments done by this block
        int grain = 0;                 // granules
        Ring<S::vslots> v;
        Ring<kSBufs> b;
        // The cut units' pieces that this block stores: the one that goes on behind its range
        // (stored first), the one that began before it.
        auto record = [&](int x) { return sm_misc + 16 + 16 * x; };
        int stored = 0, counted = 0, gos = 0;  // pieces, and uses of bar_go
        // Count the piece stored last.  Not at once: the release waits for its stores, and warp 0
        // with it, so it comes at the end of the next segment, when they are long done (before
        // a fold, lest blocks wait for each other in a row), or in the end.
        auto count_piece = [&]() -> bool {
            if (counted == stored) return true;
            ++counted;
            if (warp != 0) return true;
            if (!waitw(bar_pub, counted - 1, abort)) return false;
            if (lane == 0) {
                volatile int* c = record(counted - 1);
                int* word = p.heads + (int64_t)c[8] * kHeadInts;
                c[9] = c[7] == 2 ? count_pair(word, (int)blockIdx.x - c[8]) : count_up(word, c[7]) + 1;
            }
            return true;
        };
        do {
            const int r = w.r, P = sm_P[r], F = w.flat(), q0 = p.q_start[r];
            const int ta = w.ta(), te = w.te();
            // (loaded here, first used when scores are there)
            const float k_sc = kFp8 ? p.k_scale[w.k] : 1.f, v_sc = kFp8 ? p.v_scale[w.k] : 1.f;
            const bool whole = w.whole();
            // this group's last reference and its sum of the row's weights
            float ref = -INFINITY, l = 0.f;
#pragma unroll 1
            for (int t0 = ta; ok && t0 < te; t0 += kTile) {
                const bool nodes = t0 + kTile > P;  // the tile holds nodes
                const bool two = te - t0 > kGrain;
                const int va = v.s;
                const uint32_t va_ph = v.ph;
                v.next();
                const int vb = v.s;
                const uint32_t vb_ph = v.ph;
                if (two) v.next();
                if ((job & 1) == wg) {
                    // what this thread's flat row sees of a tile that holds nodes, 32 tokens a word
                    uint32_t vis[4];
                    if (nodes) {
                        const int node = div_of(min(w.f0() + i, F - 1), group);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int rel = t0 + 32 * e - P;
                            vis[e] = rel <= -32 ? ~0u
                                     : p.mask   ? mask_bits(p.mask + (int64_t)(q0 + node) * p.words, p.words, rel)
                                                : low_bits(node - rel + 1);
                        }
                    }
                    if (!(ok = waitw(bar_s + 8 * b.s, b.ph, abort))) break;
                    tc_fence_after();
                    // weights are powers of two: a scale of zero stands for the smallest one, so that
                    // a masked score of -inf stays one (and one that is NaN stays NaN)
                    const float sc = p.scale * k_sc, sc_log2 = fabsf(sc) * kLog2e;
                    const float scale_log2 = sc_log2 < 1e-37f ? 1e-37f : sc_log2;
                    const bool flip = sc < 0.f;
                    const uint32_t scol = tmem + lane_base + kColS + b.s * 128;
                    const uint32_t gone = sm_bad[grain & 31] | (two ? sm_bad[(grain + 1) & 31] << 4 : 0u);
                    if (nodes || !two || gone || flip) {
                        // ---- tokens that this thread's flat row does not see: their scores become
                        // -inf (and all are negated where the scale is negative) ----
                        const uint32_t sign = flip ? 0x80000000u : 0u;
#pragma unroll 1
                        for (int e = 0; e < 4; ++e) {
                            uint32_t see = low_bits(te - t0 - 32 * e);
                            if (nodes) {
                                see &= vis[0];
                                vis[0] = vis[1];
                                vis[1] = vis[2];
                                vis[2] = vis[3];
                            }
                            if ((gone >> (2 * e)) & 1) see &= 0xffff0000u;
                            if ((gone >> (2 * e)) & 2) see &= 0x0000ffffu;
                            uint32_t x[32];
                            tmem_ld32(scol + 32 * e, x);
#pragma unroll
                            for (int c = 0; c < 32; ++c) x[c] = (see >> c) & 1 ? x[c] ^ sign : 0xff800000u;
                            tmem_st32(scol + 32 * e, x);
                        }
                        tmem_st_wait();
                    }
                    // (FP8: 128 registers a thread, so half as many scores at once)
                    constexpr int kAtOnce = kFp8 ? 32 : 64, kParts = 128 / kAtOnce;
                    float s[kAtOnce];
                    auto load = [&](int e) {
                        uint32_t v0[32];
                        if constexpr (kAtOnce == 64) {
                            uint32_t v1[32];
                            tmem_ld64(scol + e * 64, v0, v1);
#pragma unroll
                            for (int c = 0; c < 32; ++c) s[32 + c] = __uint_as_float(v1[c]);
                        } else {
                            tmem_ld32(scol + e * 32, v0);
                        }
#pragma unroll
                        for (int c = 0; c < 32; ++c) s[c] = __uint_as_float(v0[c]);
                    };
                    // the row's maximum, part by part; part 0, the last, stays in registers
                    float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
                    for (int e = kParts - 1; e >= 0; --e) {
                        load(e);
#pragma unroll
                        for (int c = 0; c < kAtOnce; ++c) mx4[c & 3] = fmaxf(mx4[c & 3], s[c]);
                    }
                    const float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3]));
                    // The reference so far comes from the job before, the other group's.  Lazy
                    // rescaling: it only moves when a weight would pass 2^15, by the very difference
                    // that is the weight's exponent (a sum rounds by 8 and more where scores
                    // pass 2^26).  A row that sees nothing yet stays at -inf with zero weights.
                    float now = -INFINITY, alpha = 1.f;
                    bool moved = false;
                    if (t0 > ta) {
                        if (!(ok = waitw(bar_m + 8 * ((wg ^ 1) * 4 + quarter), ((uint32_t)(job - 1) >> 1) & 1, abort))) break;
                        now = sm_ref[((job - 1) & 1) * kRows + i];
                    }
                    if (__fmaf_rn(mx, scale_log2, -now) > kMoveLog2) {
                        const float to = __fmaf_rn(mx, scale_log2, -kWeightLog2);
                        alpha = fast_exp2(now - to);  // 0 while it is -inf
                        now = to;
                        moved = t0 > ta;
                    }
                    sm_ref[(job & 1) * kRows + i] = now;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar_m + 8 * (wg * 4 + quarter));
                    l *= ref == now ? 1.f : fast_exp2(ref - now);  // 0 while ref is -inf
                    ref = now;
                    const float mneg = now == -INFINITY ? 0.f : -now;
                    // scores in pairs: one packed FMA for the exponents, one packed add for the
                    // row sums; P is rounded to fp16 for the product (2^-11 a weight; see kWeightLog2)
                    // and goes over the first 32 of each half's own 64 S columns, of parts already read
                    const uint64_t sc2 = f32x2(scale_log2, scale_log2), mn2 = f32x2(mneg, mneg);
                    uint64_t rs2[2] = {f32x2(0.f, 0.f), f32x2(0.f, 0.f)};
#pragma unroll 1
                    for (int e = 0; e < kParts; ++e) {
                        if (e > 0) load(e);
                        uint32_t pk[kAtOnce / 2];
#pragma unroll
                        for (int c = 0; c < kAtOnce / 2; ++c) {
                            float x0, x1;
                            f32x2_split(fma_f32x2(f32x2(s[2 * c], s[2 * c + 1]), sc2, mn2), x0, x1);
                            const float e0 = fast_exp2(x0);
                            const float e1 = fast_exp2(x1);
                            pk[c] = pack_half2(e0, e1);
                            rs2[c & 1] = add_f32x2(rs2[c & 1], f32x2(e0, e1));
                        }
                        if constexpr (kAtOnce == 64)
                            tmem_st32(scol + e * 64, pk);
                        else
                            tmem_st16(scol + (e >> 1) * 64 + (e & 1) * 16, pk);
                    }
                    float r0, r1, r2, r3;
                    f32x2_split(rs2[0], r0, r1);
                    f32x2_split(rs2[1], r2, r3);
                    l += (r0 + r1) + (r2 + r3);
                    // O is rescaled only after the product before is complete
                    if (__any_sync(0xffffffffu, moved)) {
                        if (!(ok = waitw(bar_o + 8 * ((job - 1) % kSBufs), (uint32_t)((job - 1) / kSBufs) & 1, abort))) break;
                        tc_fence_after();
#pragma unroll 1
                        for (int c0 = 0; c0 < 128; c0 += 32) {
                            uint32_t x[32];
                            tmem_ld32(tmem + lane_base + c0, x);
#pragma unroll
                            for (int c = 0; c < 32; ++c) x[c] = __float_as_uint(__uint_as_float(x[c]) * alpha);
                            tmem_st32(tmem + lane_base + c0, x);
                        }
                    }
                    // ---- V of a tile that holds nodes: zero what is no number (and rows past
                    // the last token, up to the last k-step's end) ----
                    if (nodes) {
                        // the product two jobs before first: then the slots' fills before are used, and a
                        // wait for this fill's parity means this fill (vslots >= 4)
                        if (!(ok = waitw(bar_o + 8 * ((job + 1) % kSBufs), (uint32_t)((job + 1) / kSBufs + 1) & 1, abort)))
                            break;
                        if (!(ok = waitw(bar_vfull + 8 * va, va_ph, abort))) break;
                        if (two && !(ok = waitw(bar_vfull + 8 * vb, vb_ph, abort))) break;
                        const int vrows = min(kTile, te - t0);
                        const uint32_t at = sbase + S::vring + (i >= kGrain ? vb : va) * kVSlot + (i & 63) * 128;
                        if (i < vrows && t0 + i >= P) {
                            uint32_t any_odd = 0;
#pragma unroll 4
                            for (int c = 0; c < 16; ++c) {
                                const uint4 x = lds16(at + (c >> 3) * kVHalf + (((c + i) & 7) << 4));
                                any_odd |= no_number(x.x) | no_number(x.y) | no_number(x.z) | no_number(x.w);
                            }
                            if (any_odd) {
#pragma unroll 1
                                for (int c = 0; c < 16; ++c) {
                                    const uint32_t a = at + (c >> 3) * kVHalf + ((c & 7) << 4);
                                    uint4 x = lds16(a);
                                    uint32_t* e = reinterpret_cast<uint32_t*>(&x);
                                    for (int d = 0; d < 4; ++d) {
                                        const uint32_t o = no_number(e[d]);
                                        if (o & 0x8000u) e[d] &= 0xffff0000u;
                                        if (o & 0x80000000u) e[d] &= 0x0000ffffu;
                                    }
                                    sts16(a, x);
                                }
                                sm_misc[9] = 1;
                            }
                        } else if (i >= vrows && i < (vrows + 15) / 16 * 16) {
#pragma unroll 4
                            for (int c = 0; c < 16; ++c)
                                sts16(at + (c >> 3) * kVHalf + (((c + i) & 7) << 4), make_uint4(0, 0, 0, 0));
                        }
                        fence_async_smem();
                    }
                    tmem_st_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar_p + 8 * b.s);
                }
                ++job;
                b.next();
                grain += 1 + two;
            }
            if (!ok) break;
            // ---- end of the segment: its last PV product (which every job's P came
            // before), the two groups' sums ----
            // (in two buffers: one is written again only after the segment between has ended for
            // all warps, when all have read it.  A warp without a job in the next segment is at its end
            // at once, while warp 0 may still count a piece of this one.)
            float* sm_sum = reinterpret_cast<float*>(smem + S::sum) + (seg & 1) * 4 * kRows;  // [2 groups][last reference, sum][128]
            sm_sum[wg * 2 * kRows + i] = ref;
            sm_sum[(wg * 2 + 1) * kRows + i] = l;
            __syncwarp();
            if (lane == 0) mbar_arrive(bar_l);
            int first = 0;
            const int np = whole ? 1 : sp.pieces(w, first);
            first += base_block;
            if (!(ok = waitw(bar_l, (uint32_t)seg & 1, abort))) break;
            if (!(ok = waitw(bar_fin, (uint32_t)seg & 1, abort))) break;
            tc_fence_after();
            if (p.linger_ns && warp == 0) linger(p.linger_ns);
            const bool ends = w.g1() == w.n;
            // the second of two pieces: wait for the first's partial, which its block stores
            // before anything else
            bool fold = np == 2 && ends;
            if (!(ok = count_piece())) break;
            if (fold) {
                // this is the block's last segment and its products are done: the K and V rings are
                // idle and take the partial
                if (tid == 0) {
                    int* word = p.heads + (int64_t)first * kHeadInts;
                    const uint64_t from = now_ns();
                    int there;
                    for (;;) {
                        asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(there) : "l"(word) : "memory");
                        if (there || now_ns() - from > p.help_ns) break;
                        __nanosleep(20);
                    }
                    sm_misc[10] = there;
                    if (there) {
                        *word = 0;
                        asm volatile("fence.proxy.async.global;" ::: "memory");
                        mbar_arrive_expect_tx(bar_go, (uint32_t)kPartFloats * 4u);
                        bulk_load(sbase + S::kring, p.part + (int64_t)first * 2 * kPartFloats, (uint32_t)kPartFloats * 4u, bar_go);
                    } else {
                        mbar_arrive(bar_go);
                    }
                }
                ok = waitw(bar_go, gos & 1, abort);
                fold = sm_misc[10] != 0;  // or else this piece is stored, and whichever block stores last merges
                if (p.stop && fold) ok = false;
                // the copy that this warp has issued lands before the block may exit
                if (!ok && warp == 0 && fold) drain1(bar_go, gos & 1);
                if (!ok) break;
                ++gos;
            }
            // some node's V, of this segment or another, was no number
            const bool any_odd = sm_misc[9] != 0;
            const int j0 = max(ta - P, 0), j1 = te - P;  // the segment's nodes
            // this group's half of the dims
            {
                const int f = min(w.f0() + i, F - 1), node = div_of(f, group), h = w.k * group + (f - node * group);
                const bool mine = w.f0() + i < F;
                const float M0 = sm_sum[i], M1 = sm_sum[2 * kRows + i];
                const float M = fmaxf(M0, M1);
                float a0 = 1.f, a2 = 0.f;
                const float Lr = (M0 == M ? sm_sum[kRows + i] : sm_sum[kRows + i] * fast_exp2(M0 - M)) +
                           (M1 == M ? sm_sum[3 * kRows + i] : sm_sum[3 * kRows + i] * fast_exp2(M1 - M));
                const float* before = reinterpret_cast<const float*>(smem + S::kring);  // fold: the first piece's
                const bool out = whole || fold;
                if (fold)
                    pair_weights(before[i], before[kRows + i], M, Lr, v_sc, a2, a0);
                else if (whole)
                    a0 = Lr == 0.f ? 0.f : __fdividef(v_sc, Lr);
                __half* orow = p.out + ((int64_t)(q0 + node) * p.hq + h) * kHeadDim + wg * 64;
                float* slot = p.part + ((int64_t)blockIdx.x * 2 + ends) * kPartFloats;
                if (!out && wg == 0) {
                    __stcg(slot + i, M);
                    __stcg(slot + kRows + i, Lr);
                }
                float4* po = reinterpret_cast<float4*>(slot + 2 * kRows) + wg * 16 * kRows + i;
                const float4* pb = reinterpret_cast<const float4*>(before + 2 * kRows) + wg * 16 * kRows + i;
                // sixteen dims at a time, rolled: this code runs once a segment, and fetching
                // it costs more than running it
#pragma unroll 1
                for (int c = 0; c < 64; c += 16) {
                    uint32_t x[16];
                    tmem_ld16(tmem + lane_base + wg * 64 + c, x);
                    float o[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) o[e] = __uint_as_float(x[e]) * a0;
                    if (fold) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float4 y = pb[(c / 4 + e) * kRows];
                            o[4 * e] = __fmaf_rn(y.x, a2, o[4 * e]);
                            o[4 * e + 1] = __fmaf_rn(y.y, a2, o[4 * e + 1]);
                            o[4 * e + 2] = __fmaf_rn(y.z, a2, o[4 * e + 2]);
                            o[4 * e + 3] = __fmaf_rn(y.w, a2, o[4 * e + 3]);
                        }
                    }
                    if (out && mine) {
                        uint32_t u8[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) u8[e] = pack_half2(o[2 * e], o[2 * e + 1]);
                        *reinterpret_cast<uint4*>(orow + c) = make_uint4(u8[0], u8[1], u8[2], u8[3]);
                        *reinterpret_cast<uint4*>(orow + c + 8) = make_uint4(u8[4], u8[5], u8[6], u8[7]);
                    } else if (mine) {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            __stcg(po + (c / 4 + e) * kRows, make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]));
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar_odrained);  // O is free for the next segment
                if (mine && any_odd)
                    add_odd<kFp8>(p, r, P, j0, j1, node, q0 + node, w.k, wg * 64, out ? orow : nullptr, out ? nullptr : po);
            }
            if (!whole && !fold) {
                if (tid == 0) {
                    volatile int* c = record(stored);
                    c[7] = np;
                    c[8] = first;
                    c[10] = w.r;
                    c[11] = w.k;
                    c[12] = w.t;
                }
                ++stored;
                __syncwarp();
                if (lane == 0) mbar_arrive(bar_pub);
            }
            ++seg;
        } while (w.prev());
        if (ok) ok = count_piece();
        // Only the merges are left: a kernel launched to start early (launch_early, PKV_FLAG_PDL) may
        // be set up.  At the start of the kernel, 0.2 us more of 23 and 0.9 of 38; never, 0.3 of 8.6.
        if (tid == 0) ptx::griddep_launch();
        // ---- the cut units ----
#pragma unroll 1
        for (int x = 0; ok && x < stored; ++x) {
            // (thread 0 wrote the record; the others read it after the wait)
            volatile int* c = record(x);
            if (tid == 0) {
                if (c[7] == 2) {
                    c[6] = c[9];  // the pair's other piece came first: the merge is this block's
                    if (c[9]) p.heads[(int64_t)c[8] * kHeadInts] = 0;
                } else {
                    c[6] = gather(p.heads + (int64_t)c[8] * kHeadInts, c[7], (int)blockIdx.x - c[8], c[9],
                                  p.help_ns, c);
                }
                mbar_arrive(bar_go);
            }
            if (!(ok = waitw(bar_go, gos & 1, abort))) break;
            ++gos;
            const int np = c[7], first = c[8], r = c[10], k = c[11], t = c[12];
            if (np == 2 && !c[6]) continue;
            const float vsc = kFp8 ? p.v_scale[k] : 1.f;
            const int f0 = (plane + planes.n * t) * kRows, nq = min(kRows, sm_C[r] * group - f0);
            if (np == 2) {
                merge_pair(p, k, f0, p.q_start[r], nq, first, vsc);
                continue;
            }
#pragma unroll 1
            for (int y = -1; y < (c[13] ? np : 0); ++y) {
                if (y < 0 ? !c[6] : !((c[y >> 5] >> (y & 31)) & 1)) continue;
                merge_share(p, k, f0, p.q_start[r], nq, np, first, y < 0 ? (int)blockIdx.x - first : y,
                                  vsc, false);
            }
        }
        if (!ok && lane == 0) {
            raise_abort();
            flag_error(p.dev_err, PKV_DEV_ERR_TIMEOUT);
        }
    }

    // ---- release tensor memory ----
    tc_fence_before();
    __syncthreads();
    if (warp == kSIssue) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols));
    }
}

size_t head_bytes() { return align_up((size_t)kMaxGrid * kHeadInts * sizeof(int), 256); }
size_t workspace_bytes() { return head_bytes() + (size_t)kMaxGrid * 2 * kPartFloats * sizeof(float); }

template <bool kFp8>
bool prepare_kernel() {
    return cudaFuncSetAttribute(tree_kernel<kFp8>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                Smem<kFp8>::total) == cudaSuccess;
}

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
            !prepare_kernel<false>() || !prepare_kernel<true>()) {
            d.status = PKV_ERR_CUDA;
            return;
        }
        d.blocks = sms < kMaxGrid ? sms : kMaxGrid;
    });
    *blocks = d.blocks;
    return d.status;
}

// For tests (pkv_debug_set_tree_hooks); 0 in normal use.
std::atomic<uint32_t> g_hook_help_ns{0}, g_hook_stop{0}, g_hook_linger_ns{0};

template <bool kFp8>
int launch(const Params& prm, const CUtensorMap& km, const CUtensorMap& vm, int blocks, cudaStream_t stream) {
    return launch_early(tree_kernel<kFp8>, blocks, threads<kFp8>(), Smem<kFp8>::total, stream, km, vm, prm);
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
    // the units' sequence, every (token, head) index and every pool row stay below 2^31
    const int64_t tiles = (int64_t)kv_heads * (((int64_t)total_q * group) / kRows + rows) *
                          (((int64_t)max_seq_len + kGrain - 1) / kGrain + unit_cost<true>());
    const int64_t pool_rows = (int64_t)num_blocks * block_size;
    if (tiles >= kTooMuch || pool_rows >= (int64_t(1) << 31) - kTile ||
        (int64_t)total_q * q_heads >= (int64_t(1) << 31))
        return PKV_ERR_UNSUPPORTED;
    if (rows == 0 || total_q == 0) return PKV_OK;
    if (!out || !q || !k_pool || !v_pool || !block_tables || !seq_lens || !q_start) return PKV_ERR_INVALID_ARG;
    if (!aligned16(out) || !aligned16(q) || !aligned16(k_pool) || !aligned16(v_pool)) return PKV_ERR_INVALID_ARG;
    const size_t bytes = (size_t)total_q * q_heads * head_dim * 2;
    if (overlap(out, bytes, q, bytes)) return PKV_ERR_INVALID_ARG;  // other blocks still read the queries
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255) ||
        workspace_bytes < tree::workspace_bytes())
        return PKV_ERR_WORKSPACE;

    int blocks = 0, st = device_blocks(&blocks);
    if (st != PKV_OK) return st;
    Params prm{};
    prm.q = static_cast<const __half*>(q);
    prm.out = static_cast<__half*>(out);
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
    prm.heads = static_cast<int*>(workspace);
    prm.part = reinterpret_cast<float*>(static_cast<unsigned char*>(workspace) + head_bytes());
    prm.dev_err = dev_err;
    const uint32_t help_ns = g_hook_help_ns.load(std::memory_order_relaxed);
    prm.help_ns = help_ns ? help_ns : kHelpNs;
    prm.stop = g_hook_stop.load(std::memory_order_relaxed);
    prm.linger_ns = g_hook_linger_ns.load(std::memory_order_relaxed);
    prm.box = 4;  // the largest power of two that divides a page, at most a granule
    while ((1 << prm.box) < kGrain && block_size % (2 << prm.box) == 0) ++prm.box;
    prm.by_bs.set(block_size);
    const bool fp8 = k_scale != nullptr;
    const int elt = fp8 ? 1 : 2;
    const int64_t dims[3] = {kHeadDim, kv_heads, pool_rows};
    const int64_t strides[2] = {kHeadDim * elt, (int64_t)kv_heads * kHeadDim * elt};
    const int box[3] = {fp8 ? kHeadDim : 64, 1, 1 << prm.box};
    const CUtensorMapDataType type = fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    CUtensorMap km, vm;
    if ((st = encode_map_3d(k_pool, type, dims, strides, box, &km)) != PKV_OK) return st;
    if ((st = encode_map_3d(v_pool, type, dims, strides, box, &vm)) != PKV_OK) return st;
    int64_t nodes = total_q < max_seq_len ? total_q : max_seq_len;  // the most a row can have
    if (mask && nodes > 32 * (int64_t)mask_words) nodes = 32 * (int64_t)mask_words;
    prm.planes = Planes::of(nodes, group);
    return fp8 ? launch<true>(prm, km, vm, blocks, stream) : launch<false>(prm, km, vm, blocks, stream);
}

extern "C" int pkv_debug_set_tree_hooks(unsigned help_ns, int stop_folds, unsigned linger_ns) {
    if (linger_ns > 1000000) return PKV_ERR_INVALID_ARG;
    pkv::tree::g_hook_help_ns.store(help_ns, std::memory_order_relaxed);
    pkv::tree::g_hook_stop.store(stop_folds != 0, std::memory_order_relaxed);
    pkv::tree::g_hook_linger_ns.store(linger_ns, std::memory_order_relaxed);
    return PKV_OK;
}
