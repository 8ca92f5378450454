// paged_kv_rope_append: rotary positions on a step's queries and keys, and the
// step's keys and values written to their slots of the rows' blocks; and
// paged_kv_norm_rope_append: the same of queries and keys that are normalised
// first, head by head.
//
// Mathematics.  Pair i of a head's first rot_dim dims is turned by the angle
// position * f_i.  The frequencies come as 64-bit fixed-point fractions of a
// turn a token, F_i = f_i / (2 pi) * 2^64, so position * F_i modulo 2^64 IS the
// angle modulo a turn: one integer multiplication, with no rounding however far
// the position lies (a 32-bit float product is off by 6e-3 rad at position
// 100,000, a 64-bit one costs FP64 units that this GPU has few of).  Its top 32
// bits become a float in [-1/2, 1/2) turns, off by at most 2^-26, and sincospif
// gives the factors.  Products and sums are in 32 bits and each output is
// rounded once: to fp16, or for E4M3 pools straight from the 32-bit value
// (no fp16 rounding in between).
//
// Work.  A thread block takes some tokens.  A thread a token finds its row and pool
// slot; all make the block's table of factors, one pair a thread, shared by all heads;
// then each item is sixteen rotated dims of one head (two 16-byte vectors), eight passed-through
// dims, or eight dims of a value.  A thread's first item is loaded before the
// table is made, so the two latencies overlap.
//
// What bounds it: a small step is a launch and the chain q_start -> length -> table
// -> factors -> store (32 tokens, 12 + 2 heads of 128: 2.9 us); a large one the copy
// bandwidth, less the first 3 to 4 us in which every block looks up and makes its
// table (15,000 tokens: 24.8 us, 4.8 TB/s read and written, 71% of a plain copy's
// rate).  48 registers and five blocks an SM: with four, 25.3 us; with six, which
// spill, 27.2; two items in flight a thread, 25.2.  With norms 3.3 us and, for the 15,000
// tokens, 27.8 (4.3 TB/s, 63%): an item is a whole turn of loads, sums over lanes and
// stores, and three blocks an SM hold its 80 registers (four, which spill, 31.0 us, five 34.7).
#include <math.h>

#include "fp8_codec.cuh"
#include "pkv_internal.cuh"
#include "ptx.cuh"

namespace pkv {
namespace rope {

constexpr int kThreads = 256;
constexpr int kBlocks = 5;   // resident per SM
constexpr int kNormBlocks = 3;  // of the kernel with norms
constexpr int kTokens = 32;  // tokens per block, at most

// n / d for n < 2^16 and 1 <= d < 2^16, by one multiplication.
struct Div {
    uint32_t m, d;
    __device__ __forceinline__ int operator()(int n) const { return d == 1 ? n : (int)__umulhi((uint32_t)n, m); }
};

struct Params {
    __half* q_out;
    void* k_pool;
    void* v_pool;
    const float* k_scale;
    const float* v_scale;
    const int32_t* tables;
    const int32_t* seq_lens;
    const int32_t* q_start;
    const int32_t* rope_positions;
    const uint64_t* rates;
    const __half* q;
    const __half* k;
    const __half* v;
    int64_t q_stride, k_stride, v_stride;
    int rows, total, hq, hk, d, rot, bs, mbpr, nb, limit;
    float mscale;
    int32_t* dev_err;
    int n_pair, n_pass, n_val;  // items of a token
    Div per_head, pass_head, val_head, per_token;
    // norms
    const __half* q_weight;
    const __half* k_weight;
    float eps, inv_d;
    int lane_bits;  // log2 of a head's lanes, 16 dims each
};

// The row r whose chunk holds token g (q_start[r] <= g < q_start[r + 1]); -1 for a
// token behind the last row.
__device__ __forceinline__ int row_of(const int32_t* q_start, int rows, int g) {
    int lo = 0, n = rows + 1;  // entries lo .. lo + n - 1; q_start[lo] <= g
    while (n > 1) {
        const int m = (n + 3) >> 2;  // three entries at once
        int c = 0;
#pragma unroll
        for (int e = 1; e < 4; ++e) c += e * m < n && q_start[lo + e * m] <= g;
        lo += c * m;
        n = min(m, n - c * m);
    }
    return lo < rows ? lo : -1;
}

__device__ __forceinline__ void unpack8(const uint4& v, float (&x)[8]) {
    const __half2* h = reinterpret_cast<const __half2*>(&v);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(h[i]);
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
    uint4 v;
    __half2* h = reinterpret_cast<__half2*>(&v);
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
    return v;
}

// Whether a row of C nodes from q0 on and L tokens is skipped (and flagged).
__device__ __forceinline__ bool bad_row(int q0, int C, int L, int limit, int total) {
    return C < 0 || L < C || L > limit || q0 < 0 || q0 > total - C;
}

// Eight values to the pool: fp16, or E4M3 codes of the quotient by the scale.
template <bool kFp8>
__device__ __forceinline__ void store8(void* pool, int64_t at, const float (&x)[8], float scale) {
    if (kFp8) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = e4m3x2(__fdiv_rn(x[2 * i], scale), __fdiv_rn(x[2 * i + 1], scale));
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(pool) + at) =
            make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
    } else {
        *reinterpret_cast<uint4*>(static_cast<__half*>(pool) + at) = pack8(x);
    }
}

// The row, slot and rotary position of each of the block's tokens, a thread a token.
// Slot -2: the token is left alone; -1: only its keys and values are.
__device__ __forceinline__ void find_tokens(const Params& p, int g0, int nt, int* sm_slot, int* sm_pos) {
    const int tid = threadIdx.x;
    if (tid < nt) {
        const int t = tid;
        const int g = g0 + t;
        const int r = row_of(p.q_start, p.rows, g);
        int slot = -2, pos = 0;
        if (r >= 0) {
            const int q0 = p.q_start[r], C = p.q_start[r + 1] - q0, L = p.seq_lens[r];
            if (bad_row(q0, C, L, p.limit, p.total)) {
                flag_error(p.dev_err, PKV_DEV_ERR_SEQ_LEN);
            } else if (g >= q0 && g - q0 < C) {
                pos = L - C + (g - q0);
                const int lb = pos / p.bs;
                const int pb = lb < p.mbpr ? p.tables[(int64_t)r * p.mbpr + lb] : -1;
                slot = -1;
                if (pb < 0 || pb >= p.nb) {
                    flag_error(p.dev_err, lb < p.mbpr ? PKV_DEV_ERR_BLOCK_ID : PKV_DEV_ERR_POSITION);
                } else {
                    slot = pb * p.bs + pos % p.bs;  // below 2^31 (checked by the host)
                }
            }
        }
        sm_slot[t] = slot;
        sm_pos[t] = p.rope_positions ? p.rope_positions[g] : pos;
    } else if (blockIdx.x == 0 && p.dev_err) {
        // rows that no token leads to (without nodes, or past total) are looked at by the first
        // block's other threads meanwhile
        for (int r = tid - nt; r < p.rows; r += kThreads - nt)
            if (bad_row(p.q_start[r], p.q_start[r + 1] - p.q_start[r], p.seq_lens[r], p.limit, p.total))
                flag_error(p.dev_err, PKV_DEV_ERR_SEQ_LEN);
    }
}

// The factors of every token's pairs: pair 8 c + 2 k + e at [k][c][e].
__device__ __forceinline__ void make_factors(const Params& p, int nt, int half, int chunks, const int* sm_pos,
                                             float2* factors) {
    for (int x = threadIdx.x; x < nt * half; x += kThreads) {
        const int t = x / half, i = x - t * half;
        const uint64_t turns = (uint64_t)(int64_t)sm_pos[t] * p.rates[i];
        float s, c;
        sincospif((float)(int32_t)(turns >> 32) * 0x1p-31f, &s, &c);
        factors[t * half + (((i & 7) >> 1) * chunks + (i >> 3)) * 2 + (i & 1)] =
            make_float2(c * p.mscale, s * p.mscale);
    }
}

// A chunk's sixteen values (two vectors) turned in place, a pair by each of its eight factors.
template <bool kInterleaved>
__device__ __forceinline__ void turn16(const float4* f, int chunks, float (&a)[8], float (&b)[8]) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float4 cs = f[k * chunks];  // cos, sin of pairs 2k and 2k + 1
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int j = 2 * k + e;
            const float c = e ? cs.z : cs.x, s = e ? cs.w : cs.y;
            float& u = kInterleaved ? (j < 4 ? a[(2 * j) & 7] : b[(2 * j) & 7]) : a[j];
            float& w = kInterleaved ? (j < 4 ? a[(2 * j + 1) & 7] : b[(2 * j + 1) & 7]) : b[j];
            const float x = u * c - w * s, y = u * s + w * c;
            u = x;
            w = y;
        }
    }
}

// What a thread holds of an item between its loads and its stores.
struct Item {
    int kind;  // 0 rotated, 1 passed through, 2 value, -1 none
    int t, h, c;
    uint4 a, b;
};

template <bool kFp8, bool kInterleaved>
__global__ void __launch_bounds__(kThreads, kBlocks) rope_append_kernel(const __grid_constant__ Params p, int tokens) {
    extern __shared__ float2 factors[];  // [tokens][4][rot / 16][2]
    __shared__ int sm_slot[kTokens], sm_pos[kTokens];
    const int tid = threadIdx.x;
    const int g0 = blockIdx.x * tokens;
    const int nt = min(tokens, p.total - g0);
    const int half = p.rot / 2, chunks = p.rot / 16;
    const int items = p.n_pair + p.n_pass + p.n_val;

    auto load = [&](int x) {
        Item it;
        it.kind = -1;
        if (x >= nt * items) return it;
        it.t = p.per_token(x);
        int i = x - it.t * items;
        const int64_t g = g0 + it.t;
        if (i < p.n_pair) {
            it.kind = 0;
            it.h = p.per_head(i);
            it.c = i - it.h * chunks;
            const __half* src = it.h < p.hq ? p.q + g * p.q_stride + it.h * p.d
                                            : p.k + g * p.k_stride + (it.h - p.hq) * p.d;
            const int d0 = kInterleaved ? 16 * it.c : 8 * it.c;
            it.a = *reinterpret_cast<const uint4*>(src + d0);
            it.b = *reinterpret_cast<const uint4*>(src + d0 + (kInterleaved ? 8 : half));
        } else if ((i -= p.n_pair) < p.n_pass) {
            it.kind = 1;
            it.h = p.pass_head(i);
            it.c = p.rot + 8 * (i - it.h * ((p.d - p.rot) / 8));
            const __half* src = it.h < p.hq ? p.q + g * p.q_stride + it.h * p.d
                                            : p.k + g * p.k_stride + (it.h - p.hq) * p.d;
            it.a = *reinterpret_cast<const uint4*>(src + it.c);
        } else {
            i -= p.n_pass;
            it.kind = 2;
            it.h = p.val_head(i);
            it.c = 8 * (i - it.h * (p.d / 8));
            it.a = *reinterpret_cast<const uint4*>(p.v + g * p.v_stride + it.h * p.d + it.c);
        }
        return it;
    };
    ptx::griddep_wait();
    Item it = load(tid);

    find_tokens(p, g0, nt, sm_slot, sm_pos);
    __syncthreads();
    make_factors(p, nt, half, chunks, sm_pos, factors);
    __syncthreads();

    for (int x = tid; it.kind >= 0; ) {
        x += kThreads;
        const Item nx = load(x);
        const int slot = sm_slot[it.t];
        const bool is_q = it.kind < 2 && it.h < p.hq;
        if (slot >= 0 || (slot == -1 && is_q)) {
            const int64_t g = g0 + it.t;
            const int hk = it.kind == 2 ? it.h : it.h - p.hq;
            const int64_t at = is_q ? (g * p.hq + it.h) * p.d : ((int64_t)slot * p.hk + hk) * p.d;
            if (it.kind == 0) {
                float a[8], b[8];
                unpack8(it.a, a);
                unpack8(it.b, b);
                const float4* f = reinterpret_cast<const float4*>(factors + it.t * half) + it.c;
                turn16<kInterleaved>(f, chunks, a, b);
                const int d0 = kInterleaved ? 16 * it.c : 8 * it.c;
                const int d1 = d0 + (kInterleaved ? 8 : half);
                if (is_q) {
                    *reinterpret_cast<uint4*>(p.q_out + at + d0) = pack8(a);
                    *reinterpret_cast<uint4*>(p.q_out + at + d1) = pack8(b);
                } else {
                    const float sc = kFp8 ? p.k_scale[hk] : 1.f;
                    store8<kFp8>(p.k_pool, at + d0, a, sc);
                    store8<kFp8>(p.k_pool, at + d1, b, sc);
                }
            } else if (is_q) {
                *reinterpret_cast<uint4*>(p.q_out + at + it.c) = it.a;
            } else {
                void* pool = it.kind == 2 ? p.v_pool : p.k_pool;
                if (kFp8) {
                    *reinterpret_cast<uint2*>(static_cast<uint8_t*>(pool) + at + it.c) =
                        quantize8(it.a, (it.kind == 2 ? p.v_scale : p.k_scale)[hk]);
                } else {
                    *reinterpret_cast<uint4*>(static_cast<__half*>(pool) + at + it.c) = it.a;
                }
            }
        }
        it = nx;
    }
}

// The same with norms.  An item is sixteen dims of one head (two 16-byte vectors): the
// d / 16 lanes of a head, padded to a power of two, are neighbours in a warp, hold the
// whole head in registers and add up its squares by shuffles, so a head is read once and
// neither the mean nor the normalised head goes through memory.  A thread's items all
// have the same dims of a head, so it keeps its slices of the two weights in registers.
template <bool kFp8, bool kInterleaved>
__global__ void __launch_bounds__(kThreads, kNormBlocks)
    norm_rope_append_kernel(const __grid_constant__ Params p, int tokens) {
    extern __shared__ float2 factors[];
    __shared__ int sm_slot[kTokens], sm_pos[kTokens];
    const int tid = threadIdx.x;
    const int g0 = blockIdx.x * tokens;
    const int nt = min(tokens, p.total - g0);
    const int half = p.rot / 2, chunks = p.rot / 16;
    const int items = nt * p.per_token.d;
    const int c = tid & ((1 << p.lane_bits) - 1);
    const bool has = c < p.d / 16, turns = c < chunks;
    const int d0 = turns && !kInterleaved ? 8 * c : 16 * c;
    const int d1 = turns && !kInterleaved ? d0 + half : d0 + 8;

    struct Vectors {
        int t, h;
        uint4 a, b;
    };
    auto load = [&](int x) {
        Vectors v;
        v.a = v.b = make_uint4(0, 0, 0, 0);
        v.t = x < items ? p.per_token(x) : -1;
        v.h = 0;
        if (v.t >= 0 && has) {
            v.h = (x - v.t * (int)p.per_token.d) >> p.lane_bits;
            const int64_t g = g0 + v.t;
            const __half* src = v.h < p.hq          ? p.q + g * p.q_stride + v.h * p.d
                                : v.h < p.hq + p.hk ? p.k + g * p.k_stride + (v.h - p.hq) * p.d
                                                    : p.v + g * p.v_stride + (v.h - p.hq - p.hk) * p.d;
            const bool value = v.h >= p.hq + p.hk;  // nothing turns
            v.a = *reinterpret_cast<const uint4*>(src + (value ? 16 * c : d0));
            v.b = *reinterpret_cast<const uint4*>(src + (value ? 16 * c + 8 : d1));
        }
        return v;
    };
    ptx::griddep_wait();
    Vectors it = load(tid);
    uint4 wk[2], wq[2];
    wk[0] = wk[1] = wq[0] = wq[1] = make_uint4(0, 0, 0, 0);
    if (has) {
        wk[0] = *reinterpret_cast<const uint4*>(p.k_weight + d0);
        wk[1] = *reinterpret_cast<const uint4*>(p.k_weight + d1);
        if (p.hq) {
            wq[0] = *reinterpret_cast<const uint4*>(p.q_weight + d0);
            wq[1] = *reinterpret_cast<const uint4*>(p.q_weight + d1);
        }
    }
    find_tokens(p, g0, nt, sm_slot, sm_pos);
    __syncthreads();
    make_factors(p, nt, half, chunks, sm_pos, factors);
    __syncthreads();

    for (int x = tid; x - tid < items;) {  // the whole warp takes part in the sums
        x += kThreads;
        const Vectors nx = load(x);
        float a[8], b[8];
        unpack8(it.a, a);
        unpack8(it.b, b);
        float s0 = 0.f, s1 = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            s0 = fmaf(a[i], a[i], s0);
            s1 = fmaf(b[i], b[i], s1);
        }
        float ss = s0 + s1;
        for (int o = (1 << p.lane_bits) >> 1; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        const int slot = it.t >= 0 ? sm_slot[it.t] : -2;
        const bool is_q = it.h < p.hq, is_v = it.h >= p.hq + p.hk;
        if (has && (slot >= 0 || (slot == -1 && is_q))) {
            const int64_t g = g0 + it.t;
            if (is_v) {
                const int hk = it.h - p.hq - p.hk;
                const int64_t at = ((int64_t)slot * p.hk + hk) * p.d + 16 * c;
                if (kFp8) {
                    const float sc = p.v_scale[hk];
                    const uint2 lo = quantize8(it.a, sc), hi = quantize8(it.b, sc);
                    *reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.v_pool) + at) =
                        make_uint4(lo.x, lo.y, hi.x, hi.y);
                } else {
                    uint4* dst = reinterpret_cast<uint4*>(static_cast<__half*>(p.v_pool) + at);
                    dst[0] = it.a;
                    dst[1] = it.b;
                }
            } else {
                const float rs = rsqrtf(fmaf(ss, p.inv_d, p.eps));
                float wa[8], wb[8];
                unpack8(is_q ? wq[0] : wk[0], wa);
                unpack8(is_q ? wq[1] : wk[1], wb);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    a[i] = a[i] * rs * wa[i];
                    b[i] = b[i] * rs * wb[i];
                }
                if (turns) {
                    const float4* f = reinterpret_cast<const float4*>(factors + it.t * half) + c;
                    turn16<kInterleaved>(f, chunks, a, b);
                }
                const int hk = it.h - p.hq;
                const int64_t at = is_q ? (g * p.hq + it.h) * p.d : ((int64_t)slot * p.hk + hk) * p.d;
                if (is_q) {
                    *reinterpret_cast<uint4*>(p.q_out + at + d0) = pack8(a);
                    *reinterpret_cast<uint4*>(p.q_out + at + d1) = pack8(b);
                } else {
                    const float sc = kFp8 ? p.k_scale[hk] : 1.f;
                    store8<kFp8>(p.k_pool, at + d0, a, sc);
                    store8<kFp8>(p.k_pool, at + d1, b, sc);
                }
            }
        }
        it = nx;
    }
}

Div make_div(int d) { return Div{d > 1 ? (uint32_t)(0x100000000ull / d + 1) : 0u, (uint32_t)d}; }

}  // namespace rope
}  // namespace pkv

extern "C" int pkv_rope_frequencies(double* freqs, int rot_dim, double base, int scaling, double factor,
                                    double original_len, double low, double high) {
    constexpr double kTwoPi = 6.283185307179586476925286766559;
    if (!freqs || rot_dim <= 0 || rot_dim % 2 || !(base > 1.0) || !isfinite(base)) return PKV_ERR_INVALID_ARG;
    if (scaling < PKV_ROPE_SCALING_NONE || scaling > PKV_ROPE_SCALING_BY_PARTS) return PKV_ERR_INVALID_ARG;
    if (scaling != PKV_ROPE_SCALING_NONE && (!(factor >= 1.0) || !isfinite(factor))) return PKV_ERR_INVALID_ARG;
    if (scaling == PKV_ROPE_SCALING_BASE) {
        if (rot_dim <= 2) return PKV_ERR_INVALID_ARG;
        base *= pow(factor, (double)rot_dim / (rot_dim - 2));
        if (!isfinite(base)) return PKV_ERR_INVALID_ARG;
    }
    if (scaling == PKV_ROPE_SCALING_BY_PARTS &&
        (!(original_len > 0.0) || !isfinite(original_len) || !isfinite(low) || !(high > low) || !isfinite(high) ||
         !isfinite(high - low)))
        return PKV_ERR_INVALID_ARG;
    for (int i = 0; i < rot_dim / 2; ++i) {
        double f = pow(base, -2.0 * i / rot_dim);
        if (scaling == PKV_ROPE_SCALING_LINEAR) f /= factor;
        if (scaling == PKV_ROPE_SCALING_BY_PARTS) {
            double g = (original_len * f / kTwoPi - low) / (high - low);
            g = g < 0.0 ? 0.0 : g > 1.0 ? 1.0 : g;
            f = (1.0 - g) * f / factor + g * f;
        }
        freqs[i] = f;
    }
    return PKV_OK;
}

extern "C" int pkv_rope_rates(uint64_t* rates, const double* freqs, int n) {
    constexpr double kTwoPi = 6.283185307179586476925286766559;
    if (n < 0 || (n > 0 && (!rates || !freqs))) return PKV_ERR_INVALID_ARG;
    for (int i = 0; i < n; ++i)
        if (!isfinite(freqs[i])) return PKV_ERR_INVALID_ARG;
    for (int i = 0; i < n; ++i) {
        double turns = freqs[i] / kTwoPi;
        turns -= floor(turns);                          // whole turns change nothing
        const double scaled = ldexp(turns, 64);         // exact
        rates[i] = scaled >= 18446744073709551616.0 ? 0 : (uint64_t)scaled;
    }
    return PKV_OK;
}

namespace pkv {
namespace rope {

// Both entry points: with norms where `norm` is given.
struct Norm {
    const void *q_weight, *k_weight;
    float eps;
};
static int append(const Norm* norm, void* q_out, void* k_pool, void* v_pool, const float* k_scale,
                  const float* v_scale, const int32_t* block_tables, const int32_t* seq_lens, const int32_t* q_start,
                  const int32_t* rope_positions, const uint64_t* rates, const void* q, const void* k_new,
                  const void* v_new, int64_t q_stride, int64_t k_stride, int64_t v_stride, int rows, int total_q,
                  int q_heads, int kv_heads, int head_dim, int rot_dim, int layout, float mscale, int block_size,
                  int max_blocks_per_row, int num_blocks, int max_seq_len, int32_t* dev_err, cudaStream_t stream) {
    if (rows < 0 || total_q < 0 || q_heads < 0 || kv_heads <= 0 || head_dim <= 0 || rot_dim <= 0 ||
        rot_dim > head_dim || block_size <= 0 || max_blocks_per_row <= 0 || num_blocks <= 0 ||
        max_seq_len < 0 || !isfinite(mscale) ||
        (layout != PKV_ROPE_HALF && layout != PKV_ROPE_INTERLEAVED))
        return PKV_ERR_INVALID_ARG;
    if ((int64_t)max_seq_len > (int64_t)max_blocks_per_row * block_size) return PKV_ERR_INVALID_ARG;
    if ((k_scale == nullptr) != (v_scale == nullptr)) return PKV_ERR_INVALID_ARG;
    if (norm && (!(norm->eps >= 0.f) || !isfinite(norm->eps))) return PKV_ERR_INVALID_ARG;
    if (head_dim % 8 || rot_dim % 16) return PKV_ERR_UNSUPPORTED;
    if (norm && (head_dim % 16 || head_dim > 512)) return PKV_ERR_UNSUPPORTED;
    // the item index of a block stays below 2^16 and a slot below 2^31
    if (((int64_t)q_heads + 2 * kv_heads) * (head_dim / 8) * 4 >= 65536 || rot_dim > 1024 ||
        (int64_t)num_blocks * block_size >= (int64_t(1) << 31))
        return PKV_ERR_UNSUPPORTED;
    if (rows == 0 || total_q == 0) return PKV_OK;
    if (!k_pool || !v_pool || !block_tables || !seq_lens || !q_start || !rates || !k_new || !v_new)
        return PKV_ERR_INVALID_ARG;
    if (q_heads > 0 && (!q || !q_out)) return PKV_ERR_INVALID_ARG;
    if (norm && (!norm->k_weight || !aligned16(norm->k_weight) ||
                 (q_heads > 0 && (!norm->q_weight || !aligned16(norm->q_weight)))))
        return PKV_ERR_INVALID_ARG;
    const int64_t qd = (int64_t)q_heads * head_dim, kd = (int64_t)kv_heads * head_dim;
    if ((q_heads > 0 && (q_stride < qd || q_stride % 8)) || k_stride < kd || k_stride % 8 || v_stride < kd ||
        v_stride % 8)
        return PKV_ERR_INVALID_ARG;
    // in place only where each output lies exactly over its input
    if (q_heads > 0) {
        const size_t out = (size_t)total_q * qd * 2;
        auto over = [&](const void* x, int64_t stride, int64_t width) {
            return overlap(q_out, out, x, ((size_t)(total_q - 1) * stride + width) * 2);
        };
        if (q_out == q ? q_stride != qd : over(q, q_stride, qd)) return PKV_ERR_INVALID_ARG;
        if (over(k_new, k_stride, kd) || over(v_new, v_stride, kd)) return PKV_ERR_INVALID_ARG;
        if (norm && (overlap(q_out, out, norm->q_weight, head_dim * 2) ||
                     overlap(q_out, out, norm->k_weight, head_dim * 2)))
            return PKV_ERR_INVALID_ARG;
    }
    if (!aligned16(k_new) || !aligned16(v_new) || !aligned16(k_pool) || !aligned16(v_pool) ||
        (q_heads > 0 && (!aligned16(q) || !aligned16(q_out))) || (reinterpret_cast<uintptr_t>(rates) & 7))
        return PKV_ERR_INVALID_ARG;

    Params p{};
    p.q_out = static_cast<__half*>(q_out);
    p.k_pool = k_pool;
    p.v_pool = v_pool;
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    p.tables = block_tables;
    p.seq_lens = seq_lens;
    p.q_start = q_start;
    p.rope_positions = rope_positions;
    p.rates = rates;
    p.q = static_cast<const __half*>(q);
    p.k = static_cast<const __half*>(k_new);
    p.v = static_cast<const __half*>(v_new);
    p.q_stride = q_stride;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.rows = rows;
    p.total = total_q;
    p.hq = q_heads;
    p.hk = kv_heads;
    p.d = head_dim;
    p.rot = rot_dim;
    p.bs = block_size;
    p.mbpr = max_blocks_per_row;
    p.nb = num_blocks;
    p.limit = max_seq_len;
    p.mscale = mscale;
    p.dev_err = dev_err;
    const int chunks = rot_dim / 16, pass = (head_dim - rot_dim) / 8;
    p.n_pair = (q_heads + kv_heads) * chunks;
    p.n_pass = (q_heads + kv_heads) * pass;
    p.n_val = kv_heads * (head_dim / 8);
    p.per_head = make_div(chunks);
    p.pass_head = make_div(pass > 0 ? pass : 1);
    p.val_head = make_div(head_dim / 8);
    int items = p.n_pair + p.n_pass + p.n_val;
    if (norm) {
        p.q_weight = static_cast<const __half*>(norm->q_weight);
        p.k_weight = static_cast<const __half*>(norm->k_weight);
        p.eps = norm->eps;
        p.inv_d = 1.f / (float)head_dim;
        while ((16 << p.lane_bits) < head_dim) ++p.lane_bits;
        items = (q_heads + 2 * kv_heads) << p.lane_bits;
    }
    p.per_token = make_div(items);
    // As many tokens a block as fill the SMs once: small batches take a block a token, the
    // shortest path; large ones pay for the look-up and the table of factors once a block,
    // all blocks are resident together, and no last wave runs alone.  Measured: 32 tokens:
    // 2.9 us (a token a block); 640 tokens, half of each head rotated, E4M3: a token a
    // block 4.2 us, four 5.4; 15,000 tokens: 20 a block 24.8 us, 4 a block 26.7, 8 a block
    // 26.4, 16 a block 27.3 (one and a half waves).
    const int sms = device_sms();
    if (sms <= 0) return PKV_ERR_CUDA;
    const int wave = sms * (norm ? kNormBlocks : kBlocks);
    int tokens = total_q < wave ? 1 : (total_q + wave - 1) / wave;
    if (tokens > kTokens) tokens = kTokens;
    if (tokens > 65535 / items) tokens = 65535 / items;
    const int table = rot_dim / 2 * (int)sizeof(float2);  // at most 40 KB of factors a block
    if (tokens > 40960 / table) tokens = 40960 / table;
    const int grid = (total_q + tokens - 1) / tokens;
    const size_t smem = (size_t)tokens * table;
    const bool il = layout == PKV_ROPE_INTERLEAVED;
    if (norm) {
        auto* kernel = k_scale ? (il ? norm_rope_append_kernel<true, true> : norm_rope_append_kernel<true, false>)
                               : (il ? norm_rope_append_kernel<false, true> : norm_rope_append_kernel<false, false>);
        return launch_early(kernel, grid, kThreads, smem, stream, p, tokens);
    }
    auto* kernel = k_scale ? (il ? rope_append_kernel<true, true> : rope_append_kernel<true, false>)
                           : (il ? rope_append_kernel<false, true> : rope_append_kernel<false, false>);
    return launch_early(kernel, grid, kThreads, smem, stream, p, tokens);
}

}  // namespace rope
}  // namespace pkv

extern "C" int paged_kv_rope_append(void* q_out, void* k_pool, void* v_pool, const float* k_scale,
                                    const float* v_scale, const int32_t* block_tables,
                                    const int32_t* seq_lens, const int32_t* q_start,
                                    const int32_t* rope_positions, const uint64_t* rates, const void* q,
                                    const void* k_new, const void* v_new, int64_t q_stride,
                                    int64_t k_stride, int64_t v_stride, int rows, int total_q,
                                    int q_heads, int kv_heads, int head_dim, int rot_dim, int layout,
                                    float mscale, int block_size, int max_blocks_per_row, int num_blocks,
                                    int max_seq_len, int32_t* dev_err, cudaStream_t stream) {
    return pkv::rope::append(nullptr, q_out, k_pool, v_pool, k_scale, v_scale, block_tables, seq_lens, q_start,
                             rope_positions, rates, q, k_new, v_new, q_stride, k_stride, v_stride, rows, total_q,
                             q_heads, kv_heads, head_dim, rot_dim, layout, mscale, block_size, max_blocks_per_row,
                             num_blocks, max_seq_len, dev_err, stream);
}

extern "C" int paged_kv_norm_rope_append(void* q_out, void* k_pool, void* v_pool, const float* k_scale,
                                         const float* v_scale, const int32_t* block_tables,
                                         const int32_t* seq_lens, const int32_t* q_start,
                                         const int32_t* rope_positions, const uint64_t* rates, const void* q,
                                         const void* k_new, const void* v_new, const void* q_weight,
                                         const void* k_weight, float eps, int64_t q_stride, int64_t k_stride,
                                         int64_t v_stride, int rows, int total_q, int q_heads, int kv_heads,
                                         int head_dim, int rot_dim, int layout, float mscale, int block_size,
                                         int max_blocks_per_row, int num_blocks, int max_seq_len,
                                         int32_t* dev_err, cudaStream_t stream) {
    const pkv::rope::Norm norm{q_weight, k_weight, eps};
    return pkv::rope::append(&norm, q_out, k_pool, v_pool, k_scale, v_scale, block_tables, seq_lens, q_start,
                             rope_positions, rates, q, k_new, v_new, q_stride, k_stride, v_stride, rows, total_q,
                             q_heads, kv_heads, head_dim, rot_dim, layout, mscale, block_size, max_blocks_per_row,
                             num_blocks, max_seq_len, dev_err, stream);
}
