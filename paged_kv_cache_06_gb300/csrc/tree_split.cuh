// How paged_attention_tree's work is cut over its thread blocks: units, planes, cuts and
// the walk over a block's range.  Plain arithmetic, for the kernel and, compiled by a host
// compiler, for the tests that check it against the definition.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define PKV_HD __host__ __device__ __forceinline__
#define PKV_HD_CALL __host__ __device__ __noinline__
#else
#include <algorithm>
#include <cmath>
#define PKV_HD inline
#define PKV_HD_CALL inline
#endif

namespace pkv {
namespace tree {
#ifndef __CUDACC__
using std::max;
using std::min;
struct int4 {
    int x, y, z, w;
};
inline int4 make_int4(int x, int y, int z, int w) { return int4{x, y, z, w}; }
#endif

PKV_HD uint32_t mul_hi(uint32_t a, uint32_t b) {
#ifdef __CUDA_ARCH__
    return __umulhi(a, b);
#else
    return (uint32_t)((uint64_t)a * b >> 32);
#endif
}
PKV_HD float quotient(float a, float b) {
#ifdef __CUDA_ARCH__
    return __fdividef(a, b);
#else
    return a / b;
#endif
}
PKV_HD int nearest(float x) {
#ifdef __CUDA_ARCH__
    return __float2int_rn(x);
#else
    return (int)std::nearbyint(x);
#endif
}

constexpr int kRows = 128;     // flat rows of an M block: TMEM lanes
constexpr int kGrainLog = 6, kGrain = 1 << kGrainLog;  // tokens of a granule: the grain of the work split, and of V's slots
constexpr int kPlanes = 4;  // at most
// Granules that a unit's queries, first scores and output cost in time, and how near a
// unit's border a cut moves to it (farther than the cost, so that a cut that stays lies
// past it): a piece more costs its block a start, a partial and a merge, which is worth
// some imbalance.  Over FP8 pools a segment starts later and its products come slower.
// Measured, cost and slack: fp16, 32 rows of 16..512 and one of 4096, 8..24
// nodes: 2, 5: 19.0 us; 4, 4: 21.0; 3, 6: 20.6; 6, 12: 23.4; 90 drawn batches'
// geometric mean 15.3, 15.5, 15.1, 15.8.  FP8, 32 rows of 1024 and 25 nodes; 96 rows of
// 16..8192, chains of 3..7; 28 drawn batches: 6, 10: 20.7, 35.2, 15.8; 8, 12: 20.7, 35.4,
// 16.0; 8, 9: 23.4, 37.1, 15.7; 4, 6: 24.7, 35.9, 15.8.
template <bool kFp8>
constexpr PKV_HD int unit_cost() { return kFp8 ? 6 : 2; }
template <bool kFp8>
constexpr PKV_HD int unit_slack() { return kFp8 ? 10 : 5; }

// The planes: M block m of a row belongs to plane m % n; magic = 2^32 / n, rounded up.
struct Planes {
    int n;
    uint32_t magic;
    // A row's M blocks in a plane (a row has fewer than 2^28).
    PKV_HD int blocks(int flat, int plane) const {
        const int m = (flat + kRows - 1) / kRows - plane;
        return m <= 0 ? 0 : n == 1 ? m : (int)mul_hi((uint32_t)(m + n - 1), magic);
    }
    // For rows of up to `nodes` nodes.
    static Planes of(int64_t nodes, int group) {
        const int64_t m = (nodes * group + kRows - 1) / kRows;
        const int n = m < 1 ? 1 : m > kPlanes ? kPlanes : (int)m;
        return Planes{n, n > 1 ? (uint32_t)((0x100000000ull + n - 1) / n) : 0u};
    }
};

// a / b for 0 <= a < 2^31, 0 < b: a float quotient (off by 2^-21 of it at most,
// 1024), that of the remainder (off by one), and the last step.
PKV_HD int div_of(int a, int b) {
    const float rb = quotient(1.f, (float)b);
    int q = (int)((float)a * rb);
    q += nearest((float)(a - q * b) * rb);
    const int r = a - q * b;
    return r < 0 ? q - 1 : r >= b ? q + 1 : q;
}

// A unit: M block plane + planes t of KV head k of row r, its place U in the
// plane's sequence and its n granules; there it takes n + kUnitCost.
template <int kUnitCost>
struct Unit {
    int r, k, t, U, n;
    PKV_HD int end() const { return U + n + kUnitCost; }
};

PKV_HD_CALL int cut_at(int x, int W, int G, int quo, int rem);

// How a plane's sequence of units, W long, is cut over its G blocks: raw cut c lies at
// floor(W c / G); one within `slack` of a border of its unit moves there.
template <int kUnitCost>
struct Split {
    using Of = Unit<kUnitCost>;
    int W, G, slack, quo, rem;
    PKV_HD void set(int w, int blocks, int least) {
        W = w;
        G = min(blocks, max(w, 1));
        quo = div_of(W, G);
        rem = W - quo * G;
        slack = max(least, quo / 16);
    }
    PKV_HD int raw(int c) const { return quo * c + div_of(rem * c, G); }
    PKV_HD int moved(int x, const Of& u) const {
        const int d0 = x - u.U, d1 = u.end() - x;
        if (min(d0, d1) > slack) return x;
        return d0 <= d1 ? u.U : u.end();
    }
    // The pieces of unit u (1: whole) and the plane's block that holds the first one.
    PKV_HD int pieces(const Of& u, int& first) const {
        const int a = u.U + slack + 1, b = u.end() - slack;  // cuts that stay lie in [a, b)
        if (a >= b) return 1;
        const int lo = cut_at(a, W, G, quo, rem), hi = cut_at(b, W, G, quo, rem);
        first = lo - 1;
        return hi - lo + 1;
    }
};

// The first raw cut at x or behind it: the quotient's float estimate is off by
// one at most (there are at most kMaxGrid cuts).
PKV_HD_CALL int cut_at(int x, int W, int G, int quo, int rem) {
    int c = (int)quotient((float)x * (float)G, (float)W);
#pragma unroll 1
    while (c > 0 && quo * (c - 1) + div_of(rem * (c - 1), G) >= x) --c;
#pragma unroll 1
    while (quo * c + div_of(rem * c, G) < x) ++c;
    return c;
}

// The unit (r, k, t, n) before a unit; out of line, once for all the roles.
PKV_HD_CALL int4 unit_before(int4 u, int hk, int group, int plane, int n, uint32_t magic, const int* C,
                             const int* P) {
    const Planes planes{n, magic};
    if (u.z > 0) {
        --u.z;
        return u;
    }
    int nt = planes.blocks(C[u.x] * group, plane);
    if (u.y > 0) {
        --u.y;
    } else {
#pragma unroll 1
        do {
            --u.x;
            nt = planes.blocks(C[u.x] * group, plane);
        } while (nt == 0);
        u.y = hk - 1;
        u.w = (P[u.x] + C[u.x] + kGrain - 1) / kGrain;
    }
    u.z = nt - 1;
    return u;
}

// a + b, kept at 2^31 - 1: the work of rows whose starts fall, so that they overlap, may
// pass what the host has allowed for.
constexpr int kTooMuch = 0x7fffffff;
PKV_HD int add_work(int a, int b) { return (int)min((unsigned)a + (unsigned)b, (unsigned)kTooMuch); }

// The units of a block's range [s0, e), last to first.
template <int kUnitCost>
struct Walk : Unit<kUnitCost> {
    using Unit<kUnitCost>::r;
    using Unit<kUnitCost>::k;
    using Unit<kUnitCost>::t;
    using Unit<kUnitCost>::U;
    using Unit<kUnitCost>::n;
    using Unit<kUnitCost>::end;
    int s0, e, hk, group, plane;
    Planes planes;
    const int* C;
    const int* P;
    PKV_HD int g0() const { return max(s0 - U - kUnitCost, 0); }
    PKV_HD int g1() const { return min(e - U - kUnitCost, n); }
    PKV_HD bool whole() const { return s0 <= U && e >= end(); }
    PKV_HD int len() const { return P[r] + C[r]; }
    PKV_HD int flat() const { return C[r] * group; }
    PKV_HD int f0() const { return (plane + planes.n * t) * kRows; }  // first flat row
    // its tokens in the range: [ta, te)
    PKV_HD int ta() const { return g0() * kGrain; }
    PKV_HD int te() const { return min(g1() * kGrain, len()); }
    // step to the unit before
    PKV_HD void back() {
        const int4 v = unit_before(make_int4(r, k, t, n), hk, group, plane, planes.n, planes.magic, C, P);
        r = v.x;
        k = v.y;
        t = v.z;
        n = v.w;
        U -= n + kUnitCost;
    }
    PKV_HD bool prev() {
        if (U <= s0) return false;
        e = U;
        back();
        return true;
    }
};

// The blocks [from, to) of `grid` that share the plane of block `block`, and the plane's
// work W (0: the block has no plane).  Wi: the planes' work.
struct Share {
    int plane, W, from, to;
};
PKV_HD Share share_of(const int (&Wi)[kPlanes], const Planes& planes, int grid, int block) {
    // blocks in proportion to the planes' work, one at least where there is any
    float Wf[kPlanes], all = 0.f;
    int later = 0;  // planes with work that are still to come
#pragma unroll
    for (int x = 0; x < kPlanes; ++x) {
        all += Wf[x] = (float)Wi[x];
        later += Wi[x] > 0;
    }
    const float share = all > 0.f ? quotient((float)grid, all) : 0.f;
    // planes of equal work get as many blocks each, so that they stay in step
    bool even = true;
#pragma unroll
    for (int x = 1; x < kPlanes; ++x) even = even && (x >= planes.n || Wi[x] == Wi[0]);
    const int each = (int)((uint64_t)grid * planes.magic >> 32);
    float upto = 0.f;
    int next = 0;
    Share s{0, 0, 0, 0};
#pragma unroll
    for (int x = 0; x < kPlanes; ++x) {
        upto += Wf[x];
        later -= Wi[x] > 0;
        const int end = even ? next + (x < planes.n ? each : 0)
                             : min(max(nearest(upto * share), next + (Wi[x] > 0)), grid - later);
        if (block >= next && block < end) s = Share{x, Wi[x], next, end};
        next = end;
    }
    return s;
}

// The unit of a block's lower (side 0) or upper (side 1) cut at raw place x, in rows from u.r
// on, whose work starts at `run`; `u` ends as that unit, or as the one before the
// cut if an upper cut moved to its unit's start.  The cut's place.
template <int kUnitCost>
PKV_HD int place_cut(Walk<kUnitCost>& u, const Split<kUnitCost>& sp, int x, int side, int run) {
    const int in = x - side;
    int at = in - run, nt;
#pragma unroll 1
    for (;; ++u.r) {
        nt = u.planes.blocks(u.flat(), u.plane);
        u.n = (u.len() + kGrain - 1) / kGrain;
        const int here = u.hk * nt * (u.n + kUnitCost);
        if (at < here) break;
        at -= here;
    }
    const int i = div_of(at, u.n + kUnitCost);
    u.k = div_of(i, nt);
    u.t = i - u.k * nt;
    u.U = in - (at - i * (u.n + kUnitCost));
    const int cut = x < u.end() ? sp.moved(x, u) : x;
    if (side == 1 && cut == u.U && cut > 0) u.back();
    return cut;
}

}  // namespace tree
}  // namespace pkv
