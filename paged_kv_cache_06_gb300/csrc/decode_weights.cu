// paged_attention_decode_weights: decode attention that also adds to each cached
// token's running sum the softmax weight it got, over the heads of its group.
//
// Mathematics.  With s_h[t] the base-2 scores of query head h, m_h their maximum and
// l_h = sum_t 2^(s_h[t] - m_h), token t got sum_h 2^(s_h[t] - m_h) / l_h.  m_h and l_h
// are known only when the last of the row's tokens has been seen, by which time its keys
// are gone; so the first kernel writes its scores as it goes (4 bytes a head and token, 24
// for six heads, where their keys and values take 512, or 256 as E4M3 codes), and a second,
// which merges the parts of the output anyway, turns them into weights.
//
// Work.  Each unit, one KV head of a row, has its tokens in 16-token granules; all granules
// of all units, in (row, head, token) order, are cut into equal contiguous ranges, one for
// each of up to three blocks an SM.  A block's four warps take its granules in turn, each through
// a ring of its own that it fills by tiled copies, one box of 16 tokens and 64 dims (128
// codes) each; 192 KB an SM are on their way.  A granule costs a warp
//   S^T[16 tok][8 heads] = K Q^T, then O^T[128][8] += V^T P^T, P as the sum of two fp16 numbers,
// with the grouped heads as the products' eight columns (E4M3 codes are widened in registers,
// exactly, with the dims in an order that lets a lane read 16 bytes of a row at a time).  The
// reference that exponents are taken from moves only when a score passes it by kMove: as a rule a
// granule costs neither an exchange between lanes nor a rescaling.  Where a unit ends, and where
// the range does, the warps' states are brought together in shared memory and leave as the
// block's piece of the unit.
// The second kernel: each block finds its unit's maxima and sums over the pieces, and
// finishes a quarter of the unit's output or 1024 tokens' weights, in the same order every time.
// Short rows take one launch instead: a block a unit, or a cluster of up to eight, each with
// a contiguous share of its granules; the scores stay in shared memory, the blocks tell
// each other their maxima and sums and the parts of the output that another of them finishes
// through distributed shared memory, and each turns its own scores into weights.
//
// What bounds it.  Few rows: one dependent chain (32 rows of 1024, E4M3, in L2 8.7 us; stage by stage 1.7 for
// the launch and the length, 1.9 for the copies, 1.7 for four granules a warp, 1.3 and 2.3 for bringing the
// block's and the cluster's parts together).  Long rows: 4 of 32768, 31.3 us; the first kernel
// takes 25 of them, 5.3 TB/s, and the second, with its launch, 6.
#include <math.h>

#include <atomic>

#include "fp8_codec.cuh"
#include "pkv_internal.cuh"
#include "tcgen05.cuh"

namespace pkv {
namespace weights {
using namespace ptx;
using tc::mbar_drain1;
using tc::mbar_waitw;

constexpr int kGranule = 16;
constexpr int kWarps = 4, kThreads = kWarps * 32;
constexpr int kBlocks = 3;           // resident per SM
constexpr int kRing = 16 << 10;      // bytes of a warp's ring
constexpr int kMaxRows = 1024;
// A head's reference lies 7 (in powers of two) below the largest score at the time and moves when a score passes
// it by more than 15: weights stay below 2^15, fp16 numbers, and those down to 2^-21 of the largest are normal ones.
// (With the reference at the largest, weights below 2^-25 of it were in the row's sum and not in its output.)
// The output's products take a weight as two fp16 numbers, the rounded weight and what the rounding left, good to
// 2^-22 of it or 2^-32 of the largest; the sums and the weights handed out keep 32 bits.  The first number alone put
// the output off by 2.4e-4 to 2.9e-4 where its own rounding is 2.1e-4, for 0.1 to 0.2 us less in 10.5, 8.6 and 31.2.
constexpr float kLift = 7.f, kMove = 15.f;
constexpr int kClusterBlocks = 8;    // of a cluster, at most (the portable limit)
constexpr int kClusterTokens = 4096; // of a row that a cluster takes, at most
constexpr int kOrdered = 96;         // rows that may be ordered so that clusters take the long ones first
constexpr int kFewLong = 2048;       // rows longer than this are taken for few
constexpr int kShare = 64;           // granules of its block, at most
constexpr size_t kClusterDynamic = 1024 + kWarps * kRing + kShare * kGranule * kMaxGroup * sizeof(float);  // at most
constexpr size_t kSmShared = 228 << 10;                        // bytes of an SM's shared memory
constexpr size_t kClusterStatic = 5376, kAttendStatic = 640;   // of a block's, beside what it is launched with, at most
constexpr int kEndThreads = 256;     // of the second kernel: a warp a head
constexpr int kEndTokens = 4;        // a thread
constexpr int kTile = kEndThreads * kEndTokens;
constexpr int kOutBlocks = 4;        // of the second kernel for a unit's output
constexpr int kLeast = 8;            // granules of a range
constexpr int kAhead = 4;            // pieces of an output that a thread asks for at once
static_assert(kMaxGroup * kHeadDim / 4 <= kOutBlocks * kEndThreads, "a thread a group of four dims");
constexpr float kLog2e = 1.4426950408889634f;
static_assert(kEndThreads / 32 == kMaxGroup, "a warp a head");

struct Params {
    __half* out;
    float* weights;
    const __half* q;
    const float* k_scale;
    const float* v_scale;
    const int32_t* tables;
    const int32_t* seq_lens;
    int64_t stride;
    int rows, hq, hk, group, bs, mbpr, nb, limit;
    int tokens;        // of a row, at most: whole granules
    int pairs;         // of heads whose scores are kept
    int grid;          // blocks of the first kernel
    int blocks;        // of a cluster
    int slots;         // of a cluster's warps' rings
    int ordered;       // clusters take the long rows first
    float scale_log2;
    int* pre;          // [rows + 1]: granules of the rows before
    float* part;       // [block + unit][group][128]: the block's piece of the unit, unnormalised
    float2* ml;        // [block + unit][kMaxGroup]: its references and sums
    float* scores;     // [unit][tokens][2 * pairs]
    int32_t* dev_err;
    int give_up;       // (kHook) the granule of each block whose wait runs out at once
};

// The block whose range of the W granules holds granule g (block c's starts at c W / n): the
// largest c with c W <= (g + 1) n - 1 = x.  The quotient of floats is off by less than one.
__device__ __forceinline__ int owner_of(int g, int W, int n) {
    const int64_t x = (int64_t)(g + 1) * n - 1;
    int c = (int)__fdividef((float)x, (float)W);
    if ((int64_t)(c + 1) * W <= x) ++c;
    if ((int64_t)c * W > x) --c;
    return c;
}

// Ranges that W granules are cut into: one a block, but kLeast granules in each where there are few, since
// every piece is read again by all that merge it (one row of 8192, 2 KV heads: 14.5 us with 1, 11.2 with
// 4, 9.3 with 8, 9.0 with 16; 8 rows of 1 to 1024 and one of 8192: 14.2, 13.1, 11.4 and 13.6).
__device__ __forceinline__ int ranges_of(int W, int grid) { return min((W + kLeast - 1) / kLeast, grid); }

// A granule in shared memory, as the tiled copies lay it: boxes of 16 rows of 128 bytes, the
// 16-byte chunk c of row r at c ^ (r & 7).  fp16: keys' dims 0 .. 63, 64 .. 127, then the
// values'; codes: the keys, then the values.
constexpr int kBox = 16 * 128;
template <bool kFp8>
constexpr int granule_bytes = kFp8 ? 2 * kBox : 4 * kBox;

// Lane (g, t) = 4 g + t holds of the queries what the products' B operand wants: head g's dims
// in the order that the keys are read in.  Columns past the group repeat its last head.
template <bool kFp8>
__device__ __forceinline__ void load_q(uint32_t (&qb)[16], const __half* q0, int group, int lane) {
    const int h = min(lane >> 2, group - 1), t = lane & 3;
    if (kFp8) {  // codes 32 t .. 32 t + 31: chunks 2 t and 2 t + 1 of a row
        const uint4* row = reinterpret_cast<const uint4*>(q0 + h * kHeadDim + 32 * t);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint4 v = row[i];
            qb[4 * i] = v.x;
            qb[4 * i + 1] = v.y;
            qb[4 * i + 2] = v.z;
            qb[4 * i + 3] = v.w;
        }
    } else {
        const uint32_t* row = reinterpret_cast<const uint32_t*>(q0 + h * kHeadDim) + t;
#pragma unroll
        for (int ks = 0; ks < 8; ++ks) {
            qb[2 * ks] = row[8 * ks];
            qb[2 * ks + 1] = row[8 * ks + 4];
        }
    }
}
__device__ __forceinline__ uint32_t word(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

// S^T of a granule: token g (s[0], s[1]: heads 2 t, 2 t + 1) and g + 8 (s[2], s[3]).
template <bool kFp8>
__device__ __forceinline__ void scores_of(float (&s)[4], const unsigned char* data, uint32_t at,
                                          const uint32_t (&qb)[16], int lane) {
    float c0[4] = {0.f, 0.f, 0.f, 0.f}, c1[4] = {0.f, 0.f, 0.f, 0.f};
    if (kFp8) {
        const int g = lane >> 2, t = lane & 3;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const unsigned char* a = data + g * 128 + ((2 * t + j) ^ g) * 16;  // (g + 8) & 7 == g
            const uint4 x = *reinterpret_cast<const uint4*>(a), y = *reinterpret_cast<const uint4*>(a + 8 * 128);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t a0, a1, a2, a3;
                widen4(word(x, i), a0, a2);
                widen4(word(y, i), a1, a3);
                mma16816(i & 1 ? c1 : c0, a0, a1, a2, a3, qb[2 * (4 * j + i)], qb[2 * (4 * j + i) + 1]);
            }
        }
    } else {
        const int row = lane & 15;
#pragma unroll
        for (int ks = 0; ks < 8; ++ks) {
            const int chunk = (ks & 3) * 2 + (lane >> 4);
            uint32_t a0, a1, a2, a3;
            ldsm_x4(at + (ks >> 2) * kBox + row * 128 + ((chunk ^ (row & 7)) << 4), a0, a1, a2, a3);
            mma16816(ks & 1 ? c1 : c0, a0, a1, a2, a3, qb[2 * ks], qb[2 * ks + 1]);
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) s[i] = c0[i] + c1[i];
}
// Both halves, infinities as the largest finite number of their sign.
__device__ __forceinline__ uint32_t finite2(uint32_t x) {
    uint32_t y;
    asm("min.xorsign.abs.f16x2 %0, %1, %2;" : "=r"(y) : "r"(x), "r"(0x7bff7bffu));
    return y;
}
// O^T += V^T P^T; tile mt's rows g and g + 8 are the dims 16 mt + g and 16 mt + 8 + g, or, of
// codes, 16 g + 2 mt and 16 g + 2 mt + 1.
// P: pb, and qb, what rounding left of it, of any sign: it is multiplied by values that are finite, so that an infinite
// one stays what pb makes of it.  The values of tokens from `valid` on are taken for zeros (their slots may hold
// anything).
template <bool kFp8>
__device__ __forceinline__ void add_values(float (&o)[8][4], const unsigned char* data, uint32_t at, uint32_t pb0,
                                           uint32_t pb1, uint32_t qb0, uint32_t qb1, int valid, int lane) {
    const int t = lane & 3;
    if (kFp8) {
        const int g = lane >> 2;
        uint4 x[4];  // chunk g of tokens 2 t, 2 t + 1, 2 t + 8, 2 t + 9
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int row = 2 * t + (j & 1) + 8 * (j >> 1);
            x[j] = *reinterpret_cast<const uint4*>(data + kBox + row * 128 + ((g ^ (row & 7)) << 4));
            if (row >= valid) x[j] = make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int mt = 0; mt < 8; mt += 2) {  // two tiles: a tile's products follow each other at a distance
            uint32_t a[2][4];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint32_t sel = i ? 0x7362u : 0x5140u;
                widen4(__byte_perm(word(x[0], mt >> 1), word(x[1], mt >> 1), sel), a[i][0], a[i][1]);
                widen4(__byte_perm(word(x[2], mt >> 1), word(x[3], mt >> 1), sel), a[i][2], a[i][3]);
                mma16816(o[mt + i], a[i][0], a[i][1], a[i][2], a[i][3], pb0, pb1);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) mma16816(o[mt + i], a[i][0], a[i][1], a[i][2], a[i][3], qb0, qb1);
        }
    } else {
        const int row = (lane & 7) + (lane >> 4) * 8;
        const uint32_t lo = (2 * t < valid ? 0xffffu : 0u) | (2 * t + 1 < valid ? 0xffff0000u : 0u);
        const uint32_t hi = (2 * t + 8 < valid ? 0xffffu : 0u) | (2 * t + 9 < valid ? 0xffff0000u : 0u);
#pragma unroll
        for (int mt = 0; mt < 8; mt += 2) {
            uint32_t a[2][4];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int chunk = ((mt + i) & 3) * 2 + ((lane >> 3) & 1);
                ldsm_x4_t(at + (2 + (mt >> 2)) * kBox + row * 128 + ((chunk ^ (row & 7)) << 4), a[i][0], a[i][1],
                          a[i][2], a[i][3]);
                a[i][0] &= lo;
                a[i][1] &= lo;
                a[i][2] &= hi;
                a[i][3] &= hi;
                mma16816(o[mt + i], a[i][0], a[i][1], a[i][2], a[i][3], pb0, pb1);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i)
                mma16816(o[mt + i], finite2(a[i][0]), finite2(a[i][1]), finite2(a[i][2]), finite2(a[i][3]), qb0, qb1);
        }
    }
}
// A warp's running state: heads 2 t, 2 t + 1 of lane (g, t); the sums are a lane's own until reduced.
struct State {
    float m0, m1, l0, l1, o[8][4];
    __device__ __forceinline__ void reset() {
        m0 = m1 = -INFINITY;
        l0 = l1 = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    }
    __device__ __forceinline__ void reduce() {
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) {
            l0 += __shfl_xor_sync(0xffffffffu, l0, off);
            l1 += __shfl_xor_sync(0xffffffffu, l1, off);
        }
    }
};
// One granule of `valid` tokens; its scores to `to` (this lane's heads of token g, `pairs` a token).
template <bool kFp8>
__device__ __forceinline__ void attend(State& st, const unsigned char* data, uint32_t at, int valid,
                                       const uint32_t (&qb)[16], float sl2, float2* to, int pairs, int lane) {
    const int gq = lane >> 2;
    float s[4];
    scores_of<kFp8>(s, data, at, qb, lane);
#pragma unroll
    for (int j = 0; j < 4; ++j) s[j] = gq + 8 * (j >> 1) < valid ? s[j] * sl2 : -INFINITY;
    if ((lane & 3) < pairs) {
        to[0] = make_float2(s[0], s[1]);
        to[8 * pairs] = make_float2(s[2], s[3]);
    }
    const float x0 = fmaxf(s[0], s[2]), x1 = fmaxf(s[1], s[3]);
    if (__any_sync(0xffffffffu, x0 > st.m0 + kMove || x1 > st.m1 + kMove)) {
        float n0 = fmaxf(st.m0, x0 - kLift), n1 = fmaxf(st.m1, x1 - kLift);
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) {
            n0 = fmaxf(n0, __shfl_xor_sync(0xffffffffu, n0, off));
            n1 = fmaxf(n1, __shfl_xor_sync(0xffffffffu, n1, off));
        }
        // (a head that has seen nothing stays at -inf, with a state of zeros)
        const float f0 = n0 == -INFINITY ? 1.f : fast_exp2(st.m0 - n0);
        const float f1 = n1 == -INFINITY ? 1.f : fast_exp2(st.m1 - n1);
        st.m0 = n0;
        st.m1 = n1;
        st.l0 *= f0;
        st.l1 *= f1;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            st.o[i][0] *= f0;
            st.o[i][1] *= f1;
            st.o[i][2] *= f0;
            st.o[i][3] *= f1;
        }
    }
    const float u0 = st.m0 == -INFINITY ? 0.f : st.m0, u1 = st.m1 == -INFINITY ? 0.f : st.m1;
    const float p0 = fast_exp2(s[0] - u0), p1 = fast_exp2(s[1] - u1);
    const float p2 = fast_exp2(s[2] - u0), p3 = fast_exp2(s[3] - u1);
    // the sums take the weights in 32 bits: the weights handed out are divided by them too
    st.l0 += p0 + p2;
    st.l1 += p1 + p3;
    const __half2 h0 = __floats2half2_rn(p0, p1), h1 = __floats2half2_rn(p2, p3);
    const float2 f0 = __half22float2(h0), f1 = __half22float2(h1);
    add_values<kFp8>(st.o, data, at, movmatrix_t(*reinterpret_cast<const uint32_t*>(&h0)),
                     movmatrix_t(*reinterpret_cast<const uint32_t*>(&h1)), movmatrix_t(pack_half2(p0 - f0.x, p1 - f0.y)),
                     movmatrix_t(pack_half2(p2 - f1.x, p3 - f1.y)), valid, lane);
}

// Place d of a half's 64 dims of head h in a warp's state; pairs of heads lie on other banks.
__device__ __forceinline__ int state_at(int h, int d) { return h * 64 + (d ^ (((h >> 1) & 3) << 3)); }

// kHook: for tests, a wait that runs out at once.
template <bool kFp8, bool kHook>
__global__ void __launch_bounds__(kThreads, kBlocks)
    attend_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                  const __grid_constant__ Params p) {
    constexpr int kBytes = granule_bytes<kFp8>, kSlots = kRing / kBytes;
    // from 1024-byte alignment on: rings, the warps' states [warp][group][64], rows + 1 prefixes
    extern __shared__ unsigned char raw[];
    unsigned char* smem = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
    float* part = reinterpret_cast<float*>(smem + kWarps * kRing);
    int* pre = reinterpret_cast<int*>(part + kWarps * p.group * 64);
    __shared__ __align__(8) uint64_t bars[kWarps][kSlots];  // granule there
    __shared__ int2 asked[kWarps][kSlots];                   // its first token, and tokens (0: none is seen)
    __shared__ float2 part_ml[kWarps][kMaxGroup];
    __shared__ int warp_sums[kWarps];
    __shared__ int stop;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int gq = lane >> 2, tq = lane & 3;
    if (tid < kWarps * kSlots) {
        mbar_init(smem_u32(&bars[0][0] + tid), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (tid == 0) {
        stop = 0;
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&kmap)) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&vmap)) : "memory");
    }
    griddep_wait();

    // ---- the rows' granules ----
    auto length = [&](int r) {
        const int L = p.seq_lens[r];
        return L < 0 ? 0 : L > p.limit ? p.limit : L;
    };
    int run = 0;
    for (int r0 = 0; r0 < p.rows; r0 += kThreads) {
        const int r = r0 + tid;
        int c = 0;
        if (r < p.rows) {
            const int L = p.seq_lens[r], used = L < 0 ? 0 : L > p.limit ? p.limit : L;
            if (blockIdx.x == 0 && L != used) flag_error(p.dev_err, PKV_DEV_ERR_SEQ_LEN);
            c = (used + kGranule - 1) / kGranule * p.hk;
        }
        int incl = c;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int t = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += t;
        }
        if (lane == 31) warp_sums[warp] = incl;
        __syncthreads();
        int before = run;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp) before += warp_sums[w];
            run += warp_sums[w];
        }
        if (r < p.rows) pre[r] = before + incl - c;
        if (r == p.rows - 1) pre[p.rows] = before + incl;
        __syncthreads();
    }
    if (blockIdx.x == 0)  // for the second kernel
        for (int r = tid; r <= p.rows; r += kThreads) p.pre[r] = pre[r];
    const int W = run, n = ranges_of(W, p.grid);
    if ((int)blockIdx.x >= n) return;
    const int g0 = (int)((int64_t)W * blockIdx.x / n), all = (int)((int64_t)W * (blockIdx.x + 1) / n) - g0;
    // The row that granule g is in.
    auto row_of = [&](int g) {
        int lo = 0, hi = p.rows - 1;
        while (lo < hi) {  // the last row whose granules start at or before g
            const int mid = (lo + hi + 1) >> 1;
            if (pre[mid] <= g) lo = mid; else hi = mid - 1;
        }
        return lo;
    };
    const volatile int* stopped = &stop;
    unsigned char* ring = smem + warp * kRing;
    const uint32_t ring_at = smem_u32(ring);

    // ---- copies: this warp's granules warp, warp + kWarps, ... of the range ----
    // Lane j knows granule batch + j * kWarps: its KV head, first token, that token's pool row (-1:
    // none) and how many tokens there are.
    int batch = warp, kvh_j = 0, tok_j = 0, row_j = -1, valid_j = 0;
    auto look_up = [&] {
        const int x = batch + lane * kWarps;
        row_j = -1;
        valid_j = 0;
        if (x >= all) return;
        const int r = row_of(g0 + x), off = g0 + x - pre[r], count = (pre[r + 1] - pre[r]) / p.hk;
        kvh_j = off / count;
        tok_j = (off - kvh_j * count) * kGranule;
        const int lb = tok_j / p.bs, pb = p.tables[(int64_t)r * p.mbpr + lb], L = length(r);
        if (pb < 0 || pb >= p.nb) {
            flag_error(p.dev_err, PKV_DEV_ERR_BLOCK_ID);
        } else {
            row_j = pb * p.bs + (tok_j - lb * p.bs);
            valid_j = min(kGranule, L - tok_j);
        }
    };
    look_up();
    int ask_x = warp, ask_slot = 0;
    auto ask = [&] {  // the next granule into the next slot, which has been read
        if (ask_x >= all) return;
        if (ask_x >= batch + 32 * kWarps) {
            batch += 32 * kWarps;
            look_up();
        }
        if (lane == (ask_x - batch) / kWarps) {
            const uint32_t to = ring_at + ask_slot * kBytes, full = smem_u32(&bars[warp][ask_slot]);
            asked[warp][ask_slot] = make_int2(tok_j, valid_j);
            mbar_arrive_expect_tx(full, row_j < 0 ? 0u : (uint32_t)kBytes);
            if (row_j >= 0) {
                tma_load_3d(to, &kmap, 0, kvh_j, row_j, full);
                if (!kFp8) tma_load_3d(to + kBox, &kmap, 64, kvh_j, row_j, full);
                tma_load_3d(to + kBytes / 2, &vmap, 0, kvh_j, row_j, full);
                if (!kFp8) tma_load_3d(to + kBytes / 2 + kBox, &vmap, 64, kvh_j, row_j, full);
            }
        }
        __syncwarp();
        ask_x += kWarps;
        if (++ask_slot == kSlots) ask_slot = 0;
    };
#pragma unroll 1
    for (int i = 0; i < kSlots; ++i) ask();

    // ============================ attention ============================
    State st;
    uint32_t qb[16];
    int slot = 0;
    uint32_t parity = 0;
    bool ok = true;
    int x = warp;  // this warp's next granule, from g0 on
#pragma unroll 1
    for (int from = 0; from < all;) {
        // ---- the piece that starts at granule `from`: its unit, and its end ----
        const int r = row_of(g0 + from), count = (pre[r + 1] - pre[r]) / p.hk, row0 = pre[r] - g0;
        const int kvh = (from - row0) / count, unit = r * p.hk + kvh;
        const int end = min(all, row0 + (kvh + 1) * count);
        st.reset();
        const bool some = x < end;
        if (some) load_q<kFp8>(qb, p.q + ((int64_t)r * p.hq + kvh * p.group) * kHeadDim, p.group, lane);
        const float sl2 = kFp8 ? p.scale_log2 * p.k_scale[kvh] : p.scale_log2;
#pragma unroll 1
        for (; x < end && ok; x += kWarps) {
            if ((kHook && x == p.give_up) || !mbar_waitw(smem_u32(&bars[warp][slot]), parity, stopped)) {
                // gives up: what it has asked for lands before the block exits; the barriers below are
                // for all
                ok = false;
                if (lane == 0) {
                    stop = 1;
                    flag_error(p.dev_err, PKV_DEV_ERR_TIMEOUT);
                    for (int y = x; y < ask_x; y += kWarps) {
                        const int turn = y / kWarps;
                        mbar_drain1(smem_u32(&bars[warp][turn % kSlots]), (uint32_t)(turn / kSlots) & 1);
                    }
                }
                __syncwarp();
                break;
            }
            const unsigned char* data = ring + slot * kBytes;
            const uint32_t at = ring_at + slot * kBytes;
            const int2 what = asked[warp][slot];
            float2* to = reinterpret_cast<float2*>(p.scores) +
                         ((int64_t)unit * p.tokens + what.x + gq) * p.pairs + tq;
            attend<kFp8>(st, data, at, what.y, qb, sl2, to, p.pairs, lane);
            __syncwarp();  // the slot is read before its next copy is asked for
            if (++slot == kSlots) {
                slot = 0;
                parity ^= 1;
            }
            ask();
        }
        // ---- the block's piece: the warps' states brought together ----
        st.reduce();
        if (lane < 4) {
            part_ml[warp][2 * lane] = make_float2(st.m0, st.l0);
            part_ml[warp][2 * lane + 1] = make_float2(st.m1, st.l1);
        }
        // half of the dims at a time: tiles 4 half .. 4 half + 3
        const int64_t rec = (int64_t)blockIdx.x + unit;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            if (half) __syncthreads();  // the first half is read
            float* to = part + warp * p.group * 64;
#pragma unroll
            for (int mt = 0; mt < 4; ++mt) {
                const float (&v)[4] = st.o[4 * half + mt];
                const int d = kFp8 ? 8 * gq + 2 * mt : 16 * mt + gq, e = kFp8 ? d + 1 : d + 8;
                if (2 * tq < p.group) {
                    to[state_at(2 * tq, d)] = v[0];
                    to[state_at(2 * tq, e)] = v[2];
                }
                if (2 * tq + 1 < p.group) {
                    to[state_at(2 * tq + 1, d)] = v[1];
                    to[state_at(2 * tq + 1, e)] = v[3];
                }
            }
            __syncthreads();
            for (int i = tid; i < p.group * 16; i += kWarps * 32) {
                const int h = i / 16, d = i % 16 * 4;
                float M = -INFINITY, Lt = 0.f;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) M = fmaxf(M, part_ml[w][h].x);
                const float u = M == -INFINITY ? 0.f : M;
                float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    const float f = fast_exp2(part_ml[w][h].x - u);
                    const float4 z = *reinterpret_cast<const float4*>(part + w * p.group * 64 + state_at(h, d));
                    Lt += f * part_ml[w][h].y;
                    y.x += f * z.x;
                    y.y += f * z.y;
                    y.z += f * z.z;
                    y.w += f * z.w;
                }
                const int dim = kFp8 ? 16 * (d / 8) + 8 * half + d % 8 : 64 * half + d;
                *reinterpret_cast<float4*>(p.part + (rec * p.group + h) * kHeadDim + dim) = y;
                if (d == 0 && half == 0) p.ml[rec * kMaxGroup + h] = make_float2(M, Lt);
            }
        }
        from = end;
        if (from < all) __syncthreads();  // the states are read before the next piece's are written
    }
}

// The unit's pieces, and head h's maximum and sum over them by warp h, in end_ml.
struct Merge {
    int unit, c0, pieces;
    const float2* ml;
    __device__ __forceinline__ Merge(const Params& p, int r, int kvh, int before, int after, int W) {
        unit = r * p.hk + kvh;
        const int count = (after - before) / p.hk, ga = before + kvh * count, n = ranges_of(W, p.grid);
        c0 = owner_of(ga, W, n);
        pieces = owner_of(ga + count - 1, W, n) - c0 + 1;
        ml = p.ml + (int64_t)(c0 + unit) * kMaxGroup;
    }
    __device__ __forceinline__ void totals(const Params& p, float2* end_ml) const {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        if (warp < p.group) {
            float M = -INFINITY, Lt = 0.f;
#pragma unroll 2
            for (int c = lane; c < pieces; c += 32) {
                const float2 y = ml[c * kMaxGroup + warp];
                const float N = fmaxf(M, y.x), u = N == -INFINITY ? 0.f : N;
                Lt = Lt * fast_exp2(M - u) + y.y * fast_exp2(y.x - u);
                M = N;
            }
            float N = M;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) N = fmaxf(N, __shfl_xor_sync(0xffffffffu, N, o));
            N = N == -INFINITY ? 0.f : N;
            Lt *= fast_exp2(M - N);
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) Lt += __shfl_xor_sync(0xffffffffu, Lt, o);
            // where nothing is visible there is no weight
            if (lane == 0) end_ml[warp] = make_float2(N, Lt == 0.f ? 0.f : __fdividef(1.f, Lt));
        }
        __syncthreads();
    }
};

// kPairs pairs of heads; the last may be a half.  blockIdx.z below kOutBlocks: a share of the
// unit's output; above: 1024 tokens' weights.
template <int kPairs>
__global__ void __launch_bounds__(kEndThreads) merge_kernel(const __grid_constant__ Params p) {
    __shared__ float2 end_ml[kMaxGroup];  // the unit's maxima and reciprocal sums
    const int tid = threadIdx.x;
    const int r = (int)blockIdx.y, z = (int)blockIdx.z;
    griddep_wait();
    const int L = min(max(p.seq_lens[r], 0), p.limit);
    const int before = p.pre[r], after = p.pre[r + 1], W = p.pre[p.rows];
    if (z < kOutBlocks) {
        // ---- groups of four dims z, z + kOutBlocks, ..., `slices` lanes each ----
        const int kvh = (int)blockIdx.x;
        __half* ob = p.out + ((int64_t)r * p.hq + kvh * p.group) * kHeadDim;
        const int groups = p.group * (kHeadDim / 4), here = (groups - z + kOutBlocks - 1) / kOutBlocks;
        if (L == 0) {
            if (tid < here) *reinterpret_cast<uint2*>(ob + 4 * (z + tid * kOutBlocks)) = make_uint2(0, 0);
            return;
        }
        const Merge m(p, r, kvh, before, after, W);
        int slices = 1;
        while (slices < 32 && slices < m.pieces && 2 * slices * here <= kEndThreads) slices *= 2;
        const int s = tid & (slices - 1), j = tid / slices, i = z + min(j, here - 1) * kOutBlocks, h = i / (kHeadDim / 4);
        const float* part = p.part + ((int64_t)(m.c0 + m.unit) * p.group * (kHeadDim / 4) + i) * 4;
        const int step = p.group * kHeadDim;
        // the first pieces are asked for before the maxima are known
        float4 x[kAhead];
        float xm[kAhead];
        auto ask = [&](int c) {
#pragma unroll
            for (int a = 0; a < kAhead; ++a, c += slices) {
                x[a] = make_float4(0.f, 0.f, 0.f, 0.f);
                xm[a] = -INFINITY;
                if (c < m.pieces) {
                    x[a] = *reinterpret_cast<const float4*>(part + (int64_t)c * step);
                    xm[a] = m.ml[c * kMaxGroup + h].x;
                }
            }
        };
        ask(s);
        m.totals(p, end_ml);
        const float u = end_ml[h].x;
        float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
        for (int c = 0;;) {
#pragma unroll
            for (int a = 0; a < kAhead; ++a) {
                const float f = fast_exp2(xm[a] - u);
                y.x += f * x[a].x;
                y.y += f * x[a].y;
                y.z += f * x[a].z;
                y.w += f * x[a].w;
            }
            c += kAhead * slices;
            if (c >= m.pieces) break;  // the same for all lanes
            ask(c + s);
        }
        for (int o = slices >> 1; o > 0; o >>= 1) {
            y.x += __shfl_xor_sync(0xffffffffu, y.x, o);
            y.y += __shfl_xor_sync(0xffffffffu, y.y, o);
            y.z += __shfl_xor_sync(0xffffffffu, y.z, o);
            y.w += __shfl_xor_sync(0xffffffffu, y.w, o);
        }
        if (j < here && s == 0) {
            const float f = end_ml[h].y * (p.v_scale ? p.v_scale[kvh] : 1.f);
            *reinterpret_cast<uint2*>(ob + 4 * i) =
                make_uint2(pack_half2(y.x * f, y.y * f), pack_half2(y.z * f, y.w * f));
        }
        return;
    }
    // ---- tokens' weights ----
    const int first = (z - kOutBlocks) * kTile;
    if (first >= L) return;
    const Merge m(p, r, (int)blockIdx.x, before, after, W);
    const float2* sc = reinterpret_cast<const float2*>(p.scores) + (int64_t)m.unit * p.tokens * kPairs;
    float* wts = p.weights + (int64_t)m.unit * p.stride;
    float2 x[kEndTokens][kPairs];
    float was[kEndTokens];
#pragma unroll
    for (int i = 0; i < kEndTokens; ++i) {
        const int t = first + i * kEndThreads + tid;
        was[i] = t < L - 1 ? wts[t] : 0.f;  // the step's own token starts from zero
#pragma unroll
        for (int k = 0; k < kPairs; ++k) x[i][k] = t < L ? sc[(int64_t)t * kPairs + k] : make_float2(0.f, 0.f);
    }
    m.totals(p, end_ml);
    float mx[2 * kPairs], inv[2 * kPairs];
#pragma unroll
    for (int h = 0; h < 2 * kPairs; ++h) {
        mx[h] = h < p.group ? end_ml[h].x : 0.f;
        inv[h] = h < p.group ? end_ml[h].y : 0.f;
    }
#pragma unroll
    for (int i = 0; i < kEndTokens; ++i) {
        const int t = first + i * kEndThreads + tid;
        if (t >= L) continue;
        float sum = 0.f;
#pragma unroll
        for (int k = 0; k < kPairs; ++k) {
            sum += fast_exp2(x[i][k].x - mx[2 * k]) * inv[2 * k];
            if (2 * k + 1 < p.group) sum += fast_exp2(x[i][k].y - mx[2 * k + 1]) * inv[2 * k + 1];
        }
        wts[t] = was[i] + sum;
    }
}

// ---------------------------------------------------------------------------
// Short rows: a block or a cluster of them a unit, one launch.

__device__ __forceinline__ uint32_t block_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_arrive() {
    __syncwarp();  // the aligned form wants the whole warp together
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
    __syncwarp();
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t peer(uint32_t addr, int rank) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(rank));
    return a;
}
__device__ __forceinline__ void tell(uint32_t addr, float2 v) {
    asm volatile("st.shared::cluster.v2.f32 [%0], {%1,%2};" ::"r"(addr), "f"(v.x), "f"(v.y) : "memory");
}
__device__ __forceinline__ void tell(uint32_t addr, float4 v) {
    asm volatile("st.shared::cluster.v4.f32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w)
                 : "memory");
}

template <bool kFp8, bool kHook>
__global__ void __launch_bounds__(kThreads, 4)
    cluster_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                   const __grid_constant__ Params p) {
    constexpr int kBytes = granule_bytes<kFp8>, kMostSlots = kRing / kBytes, kDims = kHeadDim / 4;
    const int slots = p.slots, ring_bytes = slots * kBytes;
    // from 1024-byte alignment on: rings, then the block's scores [granules][16][2 * pairs]
    extern __shared__ unsigned char raw[];
    unsigned char* smem = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
    float2* scores = reinterpret_cast<float2*>(smem + kWarps * ring_bytes);
    __shared__ __align__(8) uint64_t bars[kWarps][kMostSlots];  // granule there
    __shared__ int asked[kWarps][kMostSlots];                    // its tokens (0: none is seen)
    __shared__ float2 part_ml[kWarps][kMaxGroup];
    // What the blocks tell each other: this block's share of the output, group of four dims i = rank +
    // active * j from block c at [j * active + c]; every block's maxima and sums.
    __shared__ __align__(16) float4 told[kMaxGroup * kDims + kClusterBlocks];
    __shared__ float2 all_ml[kClusterBlocks][kMaxGroup];
    __shared__ float2 end_ml[kMaxGroup];                      // the unit's maxima and reciprocal sums
    __shared__ int stop;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int gq = lane >> 2, tq = lane & 3;
    const int rank = (int)block_rank(), kvh = (int)blockIdx.x / p.blocks;
    int r = (int)blockIdx.y;
    if (tid < kWarps * kMostSlots) {
        mbar_init(smem_u32(&bars[0][0] + tid), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (tid == 0) {
        stop = 0;
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&kmap)) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&vmap)) : "memory");
    }
    griddep_wait();
    int L = 0;
    if (p.ordered) {
        // rows of more than a quarter of the limit come first, then the others; every warp finds the r-th by itself
        int len[kOrdered / 32], places = 0, before = 0;
        uint32_t tall[kOrdered / 32];
#pragma unroll
        for (int c = 0; c < kOrdered / 32; ++c) len[c] = 32 * c + lane < p.rows ? p.seq_lens[32 * c + lane] : 0;
#pragma unroll
        for (int c = 0; c < kOrdered / 32; ++c) {
            tall[c] = __ballot_sync(0xffffffffu, len[c] > p.limit / 4);
            places += __popc(tall[c]);
        }
        const int want = r;
#pragma unroll
        for (int c = 0; c < kOrdered / 32; ++c) {
            const int row = 32 * c + lane, taller = before + __popc(tall[c] & ((1u << lane) - 1));
            const int place = tall[c] >> lane & 1 ? taller : places + row - taller;
            const uint32_t it = __ballot_sync(0xffffffffu, place == want);
            if (it) {
                r = 32 * c + __ffs(it) - 1;
                L = __shfl_sync(0xffffffffu, len[c], __ffs(it) - 1);
            }
            before += __popc(tall[c]);
        }
    } else {
        L = p.seq_lens[r];
    }
    if (L < 0 || L > p.limit) {
        if (rank == 0 && kvh == 0 && tid == 0) flag_error(p.dev_err, PKV_DEV_ERR_SEQ_LEN);
        L = L < 0 ? 0 : p.limit;
    }
    const int n = (L + kGranule - 1) / kGranule;
    const int share = max(kWarps, (n + p.blocks - 1) / p.blocks);  // granules of a block
    const int g0 = rank * share, all = min(n, g0 + share) - g0;
    __half* ob = p.out + ((int64_t)r * p.hq + kvh * p.group) * kHeadDim;
    if (all <= 0) {  // nothing to do: the others neither wait for this block nor read its memory
        if (rank == 0)
            for (int i = tid; i < p.group * kHeadDim / 8; i += kThreads)
                reinterpret_cast<uint4*>(ob)[i] = make_uint4(0, 0, 0, 0);
        return;
    }
    const int active = (n + share - 1) / share;  // blocks that have something to do
    if (active > 1) cluster_arrive();            // this block may be told things
    __syncthreads();
    const volatile int* stopped = &stop;
    unsigned char* ring = smem + warp * ring_bytes;
    const uint32_t ring_at = smem_u32(ring);

    // ---- copies: this warp's granules warp, warp + kWarps, ... of the share ----
    const int32_t* row = p.tables + (int64_t)r * p.mbpr;
    int batch = warp, row_j = -1, valid_j = 0;  // lane j: granule batch + j * kWarps
    auto look_up = [&] {
        const int x = batch + lane * kWarps;
        row_j = -1;
        valid_j = 0;
        if (x >= all) return;
        const int t = (g0 + x) * kGranule, lb = t / p.bs, pb = row[lb];
        if (pb < 0 || pb >= p.nb) {
            flag_error(p.dev_err, PKV_DEV_ERR_BLOCK_ID);
        } else {
            row_j = pb * p.bs + (t - lb * p.bs);
            valid_j = min(kGranule, L - t);
        }
    };
    look_up();
    int ask_x = warp, ask_slot = 0;
    auto ask = [&] {  // the next granule into the next slot, which has been read
        if (ask_x >= all) return;
        if (ask_x >= batch + 32 * kWarps) {
            batch += 32 * kWarps;
            look_up();
        }
        if (lane == (ask_x - batch) / kWarps) {
            const uint32_t to = ring_at + ask_slot * kBytes, full = smem_u32(&bars[warp][ask_slot]);
            asked[warp][ask_slot] = valid_j;
            mbar_arrive_expect_tx(full, row_j < 0 ? 0u : (uint32_t)kBytes);
            if (row_j >= 0) {
                tma_load_3d(to, &kmap, 0, kvh, row_j, full);
                if (!kFp8) tma_load_3d(to + kBox, &kmap, 64, kvh, row_j, full);
                tma_load_3d(to + kBytes / 2, &vmap, 0, kvh, row_j, full);
                if (!kFp8) tma_load_3d(to + kBytes / 2 + kBox, &vmap, 64, kvh, row_j, full);
            }
        }
        __syncwarp();
        ask_x += kWarps;
        if (++ask_slot == slots) ask_slot = 0;
    };
#pragma unroll 1
    for (int i = 0; i < slots; ++i) ask();

    State st;
    st.reset();
    uint32_t qb[16];
    load_q<kFp8>(qb, p.q + ((int64_t)r * p.hq + kvh * p.group) * kHeadDim, p.group, lane);
    const float sl2 = kFp8 ? p.scale_log2 * p.k_scale[kvh] : p.scale_log2;
    const float vs = kFp8 ? p.v_scale[kvh] : 1.f;
    int slot = 0;
    uint32_t parity = 0;
#pragma unroll 1
    for (int x = warp; x < all; x += kWarps) {
        if ((kHook && x == p.give_up) || !mbar_waitw(smem_u32(&bars[warp][slot]), parity, stopped)) {
            // gives up: what it has asked for lands before the block exits; the barriers below are
            // for all
            if (lane == 0) {
                stop = 1;
                flag_error(p.dev_err, PKV_DEV_ERR_TIMEOUT);
                for (int y = x; y < ask_x; y += kWarps) {
                    const int turn = y / kWarps;
                    mbar_drain1(smem_u32(&bars[warp][turn % slots]), (uint32_t)(turn / slots) & 1);
                }
            }
            __syncwarp();
            break;
        }
        attend<kFp8>(st, ring + slot * kBytes, ring_at + slot * kBytes, asked[warp][slot], qb, sl2,
                     scores + (x * kGranule + gq) * p.pairs + tq, p.pairs, lane);
        __syncwarp();  // the slot is read before its next copy is asked for
        if (++slot == slots) {
            slot = 0;
            parity ^= 1;
        }
        ask();
    }

    // ---- the block's state: the warps' states over their rings, then brought together ----
    st.reduce();
    if (lane < 4) {
        part_ml[warp][2 * lane] = make_float2(st.m0, st.l0);
        part_ml[warp][2 * lane + 1] = make_float2(st.m1, st.l1);
    }
    auto place = [](int h, int d) { return h * kHeadDim + (d ^ (((h >> 1) & 3) << 3)); };
    float* mine = reinterpret_cast<float*>(ring);
#pragma unroll
    for (int mt = 0; mt < 8; ++mt) {
        const int d = kFp8 ? 16 * gq + 2 * mt : 16 * mt + gq, e = kFp8 ? d + 1 : d + 8;
        mine[place(2 * tq, d)] = st.o[mt][0];
        mine[place(2 * tq, e)] = st.o[mt][2];
        mine[place(2 * tq + 1, d)] = st.o[mt][1];
        mine[place(2 * tq + 1, e)] = st.o[mt][3];
    }
    if (active > 1) cluster_wait();
    __syncthreads();
    const uint32_t told_at = smem_u32(told), ml_at = smem_u32(all_ml[rank]);
#pragma unroll 1
    for (int i = tid; i < p.group * kDims; i += kThreads) {
        const int h = i / kDims, d = i % kDims * 4;
        float M = -INFINITY, Lt = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) M = fmaxf(M, part_ml[w][h].x);
        const float u = M == -INFINITY ? 0.f : M;
        float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float f = fast_exp2(part_ml[w][h].x - u);
            const float4 z = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(smem + w * ring_bytes) + place(h, d));
            Lt += f * part_ml[w][h].y;
            y.x += f * z.x;
            y.y += f * z.y;
            y.z += f * z.z;
            y.w += f * z.w;
        }
        const int j = i / active, c = i - j * active;
        if (active > 1)
            tell(peer(told_at + (j * active + rank) * 16, c), y);
        else
            told[i] = y;
        if (d == 0) {
            const float2 v = make_float2(M, Lt);
            if (active > 1)
                for (int x = 0; x < active; ++x) tell(peer(ml_at + h * 8, x), v);
            else
                all_ml[0][h] = v;
        }
    }
    if (active > 1) cluster_arrive();
    // the running sum that this thread adds to first is on its way meanwhile
    float* wts = p.weights + ((int64_t)r * p.hk + kvh) * p.stride;
    const int t0 = g0 * kGranule, t1 = min(L, t0 + all * kGranule);
    const float was = t0 + tid < min(t1, L - 1) ? wts[t0 + tid] : 0.f;
    if (active > 1)
        cluster_wait();  // nobody reads or writes another block's memory from here on
    else
        __syncthreads();

    // ---- the unit's maxima and sums ----
    if (tid < p.group) {
        float M = -INFINITY, Lt = 0.f;
        for (int c = 0; c < active; ++c) M = fmaxf(M, all_ml[c][tid].x);
        const float u = M == -INFINITY ? 0.f : M;
        for (int c = 0; c < active; ++c) Lt += fast_exp2(all_ml[c][tid].x - u) * all_ml[c][tid].y;
        end_ml[tid] = make_float2(u, Lt == 0.f ? 0.f : __fdividef(1.f, Lt));  // nothing visible: zeros
    }
    __syncthreads();

    // ---- this block's share of the output ----
#pragma unroll 1
    for (int j = tid; rank + active * j < p.group * kDims; j += kThreads) {
        const int i = rank + active * j, h = i / kDims, d = i % kDims * 4;
        const float u = end_ml[h].x, inv = end_ml[h].y * vs;
        float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int c = 0; c < active; ++c) {
            const float f = fast_exp2(all_ml[c][h].x - u);
            const float4 z = told[j * active + c];
            y.x += f * z.x;
            y.y += f * z.y;
            y.z += f * z.z;
            y.w += f * z.w;
        }
        *reinterpret_cast<uint2*>(ob + h * kHeadDim + d) =
            make_uint2(pack_half2(y.x * inv, y.y * inv), pack_half2(y.z * inv, y.w * inv));
    }

    // ---- its tokens' weights ----
#pragma unroll 1
    for (int t = t0 + tid; t < t1; t += kThreads) {
        const float2* s = scores + (t - t0) * p.pairs;
        const float before = t - t0 < kThreads ? was : t < L - 1 ? wts[t] : 0.f;  // the step's own token: zero
        float sum = 0.f;
#pragma unroll
        for (int k = 0; k < kMaxGroup / 2; ++k) {
            if (k >= p.pairs) break;
            const float2 x = s[k];
            sum += fast_exp2(x.x - end_ml[2 * k].x) * end_ml[2 * k].y;
            if (2 * k + 1 < p.group) sum += fast_exp2(x.y - end_ml[2 * k + 1].x) * end_ml[2 * k + 1].y;
        }
        wts[t] = before + sum;
    }
}

// ---------------------------------------------------------------------------
// Host side.

std::atomic<int> g_hook_granule{0};  // for tests (pkv_debug_set_weights_hooks); 0 in normal use

// Blocks of `dynamic` and `fixed` bytes of shared memory that an SM holds at once, up to `most` (their registers).
static int per_sm(size_t dynamic, size_t fixed, int most) {
    const int fit = (int)(kSmShared / (dynamic + fixed + 1024));  // (1 KB a block is the system's)
    return fit < 1 ? 1 : fit < most ? fit : most;
}
// Blocks of clusters of `blocks` that are resident at once.  Clusters fit into the device's groups of SMs, so fewer
// of the larger ones are (of 304 blocks, two an SM, 296 in fours and 288 in eights); the device is asked once for each
// number of blocks an SM.
template <class K>
static int64_t resident(K* kernel, bool fp8, int blocks, size_t smem, int sms) {
    static std::atomic<int> known[64][2][3][4];
    const int per = per_sm(smem, kClusterStatic, 4);
    int dev = 0;
    if (smem > kClusterDynamic || cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return (int64_t)sms * per;
    std::atomic<int>& slot = known[dev][fp8][blocks == 2 ? 0 : blocks == 4 ? 1 : 2][per - 1];
    int clusters = slot.load(std::memory_order_relaxed);
    if (clusters == 0) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)blocks);
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = smem;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = (unsigned)blocks;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        if (cudaOccupancyMaxActiveClusters(&clusters, kernel, &cfg) != cudaSuccess || clusters <= 0) {
            cudaGetLastError();
            return (int64_t)sms * per;
        }
        slot.store(clusters, std::memory_order_relaxed);
    }
    return (int64_t)clusters * blocks;
}

struct Layout {
    size_t ml, pre, scores, bytes;
    int tokens, pairs;
};
// Granules of rows that are all as long as may be.
static int64_t granules(int rows, int kv_heads, int max_seq_len) {
    return (int64_t)rows * kv_heads * (((int64_t)max_seq_len + kGranule - 1) / kGranule);
}
static bool supported(int rows, int q_heads, int kv_heads, int head_dim, int max_seq_len, int block_size) {
    return head_dim == kHeadDim && q_heads / kv_heads <= kMaxGroup && block_size % 16 == 0 && rows <= kMaxRows &&
           block_size <= 1024 && max_seq_len <= (1 << 24) && kv_heads <= 65536 &&
           granules(rows, kv_heads, max_seq_len) < (int64_t(1) << 31) - kMaxRows;
}
// Blocks of the first kernel, at most.
static int blocks_of(int sms) { return sms * kBlocks; }
// The current device's; on a machine without one, for as many SMs as any has.
static Layout layout(int rows, int q_heads, int kv_heads, int max_seq_len) {
    Layout l;
    const size_t units = (size_t)rows * kv_heads, group = (size_t)(q_heads / kv_heads);
    const int sms = device_sms();
    const size_t pieces = units + blocks_of(sms > 0 ? sms : 256);
    l.tokens = (int)align_up((size_t)max_seq_len, kGranule);
    l.pairs = (int)(group + 1) / 2;
    l.ml = align_up(pieces * group * kHeadDim * sizeof(float), 256);
    l.pre = l.ml + align_up(pieces * kMaxGroup * sizeof(float2), 256);
    l.scores = l.pre + align_up(((size_t)rows + 1) * sizeof(int), 256);
    l.bytes = l.scores + align_up(units * l.tokens * l.pairs * sizeof(float2), 256);
    return l;
}

}  // namespace weights
}  // namespace pkv

extern "C" size_t paged_attention_decode_weights_workspace_size(int rows, int q_heads, int kv_heads, int head_dim,
                                                                int max_seq_len, int block_size) {
    using namespace pkv::weights;
    if (rows <= 0 || q_heads <= 0 || kv_heads <= 0 || head_dim <= 0 || q_heads % kv_heads || max_seq_len < 0 ||
        block_size <= 0 || !supported(rows, q_heads, kv_heads, head_dim, max_seq_len, block_size))
        return 0;
    return layout(rows, q_heads, kv_heads, max_seq_len).bytes;
}

extern "C" int paged_attention_decode_weights(void* out, float* weights, const void* q, const void* k_pool,
                                              const void* v_pool, const float* k_scale, const float* v_scale,
                                              const int32_t* block_tables, const int32_t* seq_lens, int rows,
                                              int q_heads, int kv_heads, int head_dim, int block_size, float scale,
                                              int max_blocks_per_row, int num_blocks, int max_seq_len,
                                              int64_t weights_stride, void* workspace, size_t workspace_bytes,
                                              int32_t* dev_err, cudaStream_t stream) {
    using namespace pkv;
    using namespace pkv::weights;
    if (q_heads <= 0 || kv_heads <= 0 || head_dim <= 0 || q_heads % kv_heads) return PKV_ERR_INVALID_ARG;
    if (rows < 0 || block_size <= 0 || block_size > 1024 || max_blocks_per_row <= 0 || num_blocks <= 0 ||
        max_seq_len < 0 || !isfinite(scale) || weights_stride < max_seq_len)
        return PKV_ERR_INVALID_ARG;
    if ((int64_t)max_seq_len > (int64_t)max_blocks_per_row * block_size) return PKV_ERR_INVALID_ARG;
    if ((k_scale == nullptr) != (v_scale == nullptr)) return PKV_ERR_INVALID_ARG;
    if (!supported(rows, q_heads, kv_heads, head_dim, max_seq_len, block_size) ||
        weights_stride > (int64_t(1) << 40) || (int64_t)num_blocks * block_size >= (int64_t(1) << 31))
        return PKV_ERR_UNSUPPORTED;
    if (rows == 0) return PKV_OK;
    if (!out || !weights || !q || !k_pool || !v_pool || !block_tables || !seq_lens) return PKV_ERR_INVALID_ARG;
    if (!aligned16(out) || !aligned16(q) || !aligned16(k_pool) || !aligned16(v_pool)) return PKV_ERR_INVALID_ARG;
    const Layout l = layout(rows, q_heads, kv_heads, max_seq_len);
    if (!workspace || workspace_bytes < l.bytes || (reinterpret_cast<uintptr_t>(workspace) & 255))
        return PKV_ERR_WORKSPACE;
    const size_t wide = (size_t)rows * kv_heads * weights_stride * 4, tall = (size_t)rows * q_heads * head_dim * 2;
    if (overlap(weights, wide, out, tall) || overlap(weights, wide, q, tall) ||
        overlap(weights, wide, workspace, l.bytes) || overlap(out, tall, q, tall) ||
        overlap(out, tall, workspace, l.bytes))
        return PKV_ERR_INVALID_ARG;
    const int sms = device_sms();
    if (sms <= 0) return PKV_ERR_CUDA;

    unsigned char* ws = static_cast<unsigned char*>(workspace);
    Params p{};
    p.out = static_cast<__half*>(out);
    p.weights = weights;
    p.q = static_cast<const __half*>(q);
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    p.tables = block_tables;
    p.seq_lens = seq_lens;
    p.stride = weights_stride;
    p.rows = rows;
    p.hq = q_heads;
    p.hk = kv_heads;
    p.group = q_heads / kv_heads;
    p.bs = block_size;
    p.mbpr = max_blocks_per_row;
    p.nb = num_blocks;
    p.limit = max_seq_len;
    p.tokens = l.tokens;
    p.pairs = l.pairs;
    p.scale_log2 = scale * kLog2e;
    p.part = reinterpret_cast<float*>(ws);
    p.ml = reinterpret_cast<float2*>(ws + l.ml);
    p.pre = reinterpret_cast<int*>(ws + l.pre);
    p.scores = reinterpret_cast<float*>(ws + l.scores);
    p.dev_err = dev_err;
    p.give_up = g_hook_granule.load(std::memory_order_relaxed) - 1;
    const bool hook = p.give_up >= 0;
    const int elt = k_scale ? 1 : 2;
    const CUtensorMapDataType type = k_scale ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    const int64_t dims[3] = {head_dim, kv_heads, (int64_t)num_blocks * block_size};
    const int64_t strides[2] = {(int64_t)head_dim * elt, (int64_t)kv_heads * head_dim * elt};
    const int box[3] = {128 / elt, 1, kGranule};
    CUtensorMap kmap, vmap;
    int st = tiled_map_3d(k_pool, type, dims, strides, box, &kmap);
    if (st == PKV_OK) st = tiled_map_3d(v_pool, type, dims, strides, box, &vmap);
    if (st != PKV_OK) return st;
    // Short rows: a block a unit, or a cluster of up to eight, four granules a warp of the longest row, as many as
    // are resident at once by the shared memory they take (fp16: two an SM but for the shortest rows).  One launch
    // instead of two, and no wave that runs alone.  2 KV heads, pools that L2 does not hold, fp16, us, blocks a
    // unit 1 / 2 / 4 / 8 and the even cut; in brackets E4M3:
    //   32 rows of 1024  18.5 / 13.7 / 11.8 / 17.7, 15.8  (17.3 / 12.0 / 11.2 / 12.2, 14.8)
    //   48               19.5 / 15.7 / 19.7 / 19.9, 18.4  (17.5 / 14.6 / 19.0 / 19.7, 17.7)
    //   76               21.9 / 19.6 / 28.0 / 28.8, 23.9  (18.0 / 15.8 / 25.2 / 25.2, 20.1)
    //   128              28.7 / 33.3 / 39.9 / 45.0, 35.0  (21.8 / 27.9 / 36.7 / 38.5, 28.0)
    //   16 of 2048          - / 19.4 / 13.5 / 12.1, 15.5  (   - / 18.1 / 12.1 / 11.5, 14.6)
    //   64 of 2048          - / 29.6 / 33.2 / 41.5, 33.4  (   - / 22.8 / 28.0 / 39.3, 26.7)
    // More units than blocks fit take a block each all the same: 300 of 1024 61.1 and 70.2 (42.7 and 52.4), 200 48.9
    // and 49.8 (39.4 and 36.1), 400 of 256 28.3 and 40.7.  Blocks of more than 64 granules are the even cut's.
    // Rows longer than 2048 are taken for a few beside many short ones, whose blocks leave at once: eight blocks each,
    // where that makes no more than four an SM, and the long rows first where they are not all resident.  31 rows of
    // 16 to 512 and one of 4096, in any order: 10.6 to 11.4 us and the even cut 12.3 with the pools in L2, 13.2 and
    // 15.4 not (E4M3 12.3 and 13.3, 13.9 and 15.4; with the rows as they come 10.5 to 15.8 by where the long one is);
    // 32 of 16 to 4096, their logarithms even, 14.6 and 18.9; 8 of 4096 14.1 and 15.7; but 32 of 1 to 4096 23.4 and
    // 22.9, one of 4096 9.9 and 7.8, and 32 of them 34.6 and 31.4 (29.4 and 23.1).  With more units, or past 4096
    // tokens, such rows are the even cut's (64 of 4096: 54.8, in clusters of four 57.2; 96 of 16 to 600 and one of
    // 4000 18.1 and 29.4).
    if (max_seq_len <= kClusterTokens) {
        auto* kernel = hook      ? (k_scale ? cluster_kernel<true, true> : cluster_kernel<false, true>)
                       : k_scale ? cluster_kernel<true, false>
                                 : cluster_kernel<false, false>;
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kClusterDynamic) !=
            cudaSuccess) {
            cudaGetLastError();
            return PKV_ERR_CUDA;
        }
        const int n = l.tokens / kGranule;
        const int64_t units = (int64_t)rows * kv_heads;
        const int bytes = k_scale ? granule_bytes<true> : granule_bytes<false>, most_slots = kRing / bytes;
        int share = 0;
        size_t smem = 0;
        auto cut_into = [&](int blocks) {
            share = (n + blocks - 1) / blocks > kWarps ? (n + blocks - 1) / blocks : kWarps;
            p.slots = (share + kWarps - 1) / kWarps < most_slots ? (share + kWarps - 1) / kWarps : most_slots;
            p.blocks = blocks;
            smem = 1024 + (size_t)kWarps * p.slots * bytes + (size_t)share * kGranule * p.pairs * sizeof(float2);
        };
        cut_into(1);
        if (max_seq_len > kFewLong && units * kClusterBlocks <= 4 * (int64_t)sms && rows <= kOrdered) {
            cut_into(kClusterBlocks);
            p.ordered = units * kClusterBlocks > resident(kernel, k_scale != nullptr, kClusterBlocks, smem, sms);
        } else {
            while (p.blocks < kClusterBlocks && p.blocks * 4 * kWarps < n) {
                cut_into(2 * p.blocks);
                if (units * p.blocks <= resident(kernel, k_scale != nullptr, p.blocks, smem, sms)) continue;
                cut_into(p.blocks / 2);
                break;
            }
        }
        if (share <= kShare)
            return launch_early_clusters(kernel, dim3((unsigned)(kv_heads * p.blocks), (unsigned)rows), kThreads, smem,
                                         (unsigned)p.blocks, stream, kmap, vmap, p);
    }
    auto* attend = hook      ? (k_scale ? attend_kernel<true, true> : attend_kernel<false, true>)
                   : k_scale ? attend_kernel<true, false>
                             : attend_kernel<false, false>;
    const int state = 64 * (int)sizeof(float);  // of a head
    const size_t smem = 1024 + (size_t)kWarps * (kRing + p.group * state) + ((size_t)rows + 1) * sizeof(int);
    if (cudaFuncSetAttribute(attend, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             1024 + kWarps * (kRing + kMaxGroup * state) + (kMaxRows + 1) * (int)sizeof(int)) !=
        cudaSuccess) {
        cudaGetLastError();
        return PKV_ERR_CUDA;
    }
    // As many blocks as fill the device once: three an SM, but two where groups of eight heads and the prefixes of
    // some 400 rows take the shared memory (512 rows of 4160, one KV head, E4M3: 123.9 us; with three, of which the
    // last third ran alone, 142.8).
    const int wave = sms * per_sm(smem, kAttendStatic, kBlocks);
    const int64_t ranges = (granules(rows, kv_heads, max_seq_len) + kLeast - 1) / kLeast;
    p.grid = ranges < wave ? (ranges > 0 ? (int)ranges : 1) : wave;
    st = launch_early(attend, (unsigned)p.grid, kThreads, smem, stream, kmap, vmap, p);
    if (st != PKV_OK) return st;
    auto* merge = l.pairs == 1   ? merge_kernel<1>
                  : l.pairs == 2 ? merge_kernel<2>
                  : l.pairs == 3 ? merge_kernel<3>
                                 : merge_kernel<4>;
    const unsigned z = kOutBlocks + (unsigned)((max_seq_len + kTile - 1) / kTile);
    return launch_early(merge, dim3((unsigned)kv_heads, (unsigned)rows, z), kEndThreads, 0, stream, p);
}
