// The kernel's work split (csrc/tree_split.cuh) walked on the host: every segment of
// every block, for test_tree_split.py.
#include "tree_split.cuh"

using namespace pkv::tree;

// One record a segment: block, plane, r, k, M block, g0, g1, n, whole, pieces, first block, s0, e.
constexpr int kRecord = 13;
constexpr int kLanes = 6 * 32;  // threads that scan the rows, a run of rows each

template <bool kFp8>
static long long walk(int rows, const int* C, const int* P, int group, int hk, long long most, int grid, int* out,
                      long long cap) {
    constexpr int kCost = unit_cost<kFp8>();
    const Planes planes = Planes::of(most, group);
    const int per = (rows + kLanes - 1) / kLanes;
    long long got = 0;
    int W[kPlanes] = {0, 0, 0, 0}, before[kPlanes][kLanes], mine[kPlanes][kLanes];
    for (int x = 0; x < planes.n; ++x)
        for (int l = 0; l < kLanes; ++l) {
            before[x][l] = W[x];
            mine[x][l] = 0;
            for (int r = l * per; r < min((l + 1) * per, rows); ++r) {
                const int len = C[r] > 0 ? hk * ((P[r] + C[r] + kGrain - 1) / kGrain + kCost) : 0;
                mine[x][l] = add_work(mine[x][l], len * planes.blocks(C[r] * group, x));
            }
            W[x] = add_work(W[x], mine[x][l]);
        }
    for (int x = 0; x < planes.n; ++x)
        if (W[x] == kTooMuch) return -1;
    for (int block = 0; block < grid; ++block) {
        Share s{0, W[0], 0, grid};
        if (planes.n > 1) s = share_of(W, planes, grid, block);
        if (s.W <= 0) continue;
        Split<kCost> sp;
        sp.set(s.W, s.to - s.from, unit_slack<kFp8>());
        const int cta = block - s.from;
        if (cta >= sp.G) continue;
        Walk<kCost> w{};
        int cuts[2];
        for (int side = 0; side < 2; ++side) {
            const int x = sp.raw(cta + side), in = x - side;
            int l = 0;
            while (!(in >= before[s.plane][l] && in < before[s.plane][l] + mine[s.plane][l])) ++l;
            w.hk = hk;
            w.group = group;
            w.plane = s.plane;
            w.planes = planes;
            w.C = C;
            w.P = P;
            w.r = l * per;
            cuts[side] = place_cut(w, sp, x, side, before[s.plane][l]);
        }
        w.s0 = cuts[0];
        w.e = cuts[1];
        if (w.s0 >= w.e) continue;
        do {
            int first = 0;
            const int np = w.whole() ? 1 : sp.pieces(w, first);
            if (got == cap) return -2;
            int* o = out + kRecord * got++;
            const int rec[kRecord] = {block, s.plane, w.r, w.k, w.f0() / kRows, w.g0(), w.g1(), w.n,
                                      w.whole(), np, first + s.from, w.s0, w.e};
            for (int i = 0; i < kRecord; ++i) o[i] = rec[i];
        } while (w.prev());
    }
    return got;
}

extern "C" long long split_walk(int fp8, int rows, const int* C, const int* P, int group, int hk, long long most,
                                int grid, int* out, long long cap) {
    return (fp8 ? walk<true> : walk<false>)(rows, C, P, group, hk, most, grid, out, cap);
}
extern "C" int split_div(int a, int b) { return div_of(a, b); }
