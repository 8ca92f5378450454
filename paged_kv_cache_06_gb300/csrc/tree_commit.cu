// paged_kv_tree_commit: the accepted path's keys and values move to the row's
// next positions, in every layer's pools, and the rows' new lengths come out.
//
// A path is strictly increasing, so path[j] >= j: step j reads slot P + path[j]
// and writes slot P + j.  A later step reads at P + path[j'] >= P + j' > P + j,
// never a slot that an earlier step has written, so a thread that takes its
// 16-byte column of every step in order, eight loads before eight stores, needs
// no copy on the side; columns do not touch each other.
//
// Work.  One warp per (layer, pool, row): its lanes find 32 steps' slots at a
// time (two table entries a step) and then move the tokens' columns.  Steps
// already in place (path[j] == j) move nothing.  The bytes are few (a thousand a
// token and layer at 2 KV heads), so the chain lengths -> path -> table ->
// load -> store bounds it, and all layers go in one launch: 32 rows, one layer,
// fp16: 2.6 us; 64 rows, 28 layers, E4M3 (3 MB moved): 3.7 us over lines that are in
// L2, 5.3 us over 60 sets that L2 does not hold (0.55 TB/s).  Eight loads in flight a
// lane cover a path of eight steps in one round.
#include "pkv_internal.cuh"
#include "ptx.cuh"

namespace pkv {
namespace commit {

constexpr int kWarps = 4;   // per block
constexpr int kBatch = 8;   // steps loaded before the first is stored

__global__ void __launch_bounds__(kWarps * 32) tree_commit_kernel(
    uint4* k_pool, uint4* v_pool, const int32_t* tables, const int32_t* seq_lens, const int32_t* q_start,
    const int32_t* path, const int32_t* path_lens, int32_t* new_lens,
    int layers, int rows, int max_path, int vecs, int bs, int mbpr, int nb, int limit, int32_t* dev_err) {
    const int lane = threadIdx.x & 31;
    const int64_t w = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (w >= (int64_t)layers * 2 * rows) return;
    ptx::griddep_wait();
    const int r = (int)(w % rows), lp = (int)(w / rows);
    const bool first = lp == 0;  // reports for its row
    const int n = path_lens[r], L = seq_lens[r], C = q_start[r + 1] - q_start[r];
    if (C < 0 || L < C || L > limit) {
        if (first && lane == 0) flag_error(dev_err, PKV_DEV_ERR_SEQ_LEN);
        return;
    }
    const int P = L - C;
    const int32_t* steps = path + (int64_t)r * max_path;
    // the whole path is checked before anything moves
    bool good = n >= 0 && n <= max_path && n <= C;
    for (int j = lane; good && j < n; j += 32) {
        const int x = steps[j];
        good = x >= 0 && x < C && (j == 0 || x > steps[j - 1]);
    }
    if (!__all_sync(0xffffffffu, good)) {
        if (first && lane == 0) flag_error(dev_err, PKV_DEV_ERR_POSITION);
        return;
    }
    if (first && new_lens && lane == 0) new_lens[r] = P + n;

    const int32_t* row = tables + (int64_t)r * mbpr;
    uint4* pool = ((lp & 1) ? v_pool : k_pool) + (int64_t)(lp >> 1) * nb * bs * vecs;
    for (int j0 = 0; j0 < n; j0 += 32) {
        // lane l: step j0 + l's source and destination slots, or -1 for none
        int src = -1, dst = -1;
        if (j0 + lane < n) {
            const int a = P + steps[j0 + lane], b = P + j0 + lane;
            if (a != b) {
                const int ba = row[a / bs], bb = row[b / bs];
                if (ba < 0 || ba >= nb || bb < 0 || bb >= nb) {
                    if (first) flag_error(dev_err, PKV_DEV_ERR_BLOCK_ID);
                } else {
                    src = ba * bs + a % bs;
                    dst = bb * bs + b % bs;
                }
            }
        }
        if (!__any_sync(0xffffffffu, src >= 0)) continue;
        const int m = min(32, n - j0);
        for (int c0 = 0; c0 < vecs; c0 += 32) {
            const int c = c0 + lane;
            for (int j = 0; j < m; j += kBatch) {
                uint4 x[kBatch];
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
                    const int s = __shfl_sync(0xffffffffu, src, (j + i) & 31);
                    if (j + i < m && s >= 0 && c < vecs) x[i] = pool[(int64_t)s * vecs + c];
                }
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
                    const int d = __shfl_sync(0xffffffffu, dst, (j + i) & 31);
                    if (j + i < m && d >= 0 && c < vecs) pool[(int64_t)d * vecs + c] = x[i];
                }
            }
        }
    }
}

}  // namespace commit
}  // namespace pkv

extern "C" int paged_kv_tree_commit(void* k_pool, void* v_pool, const int32_t* block_tables,
                                    const int32_t* seq_lens, const int32_t* q_start, const int32_t* path,
                                    const int32_t* path_lens, int32_t* new_seq_lens, int layers, int rows,
                                    int max_path, int kv_heads, int head_dim, int elt_bytes,
                                    int block_size, int max_blocks_per_row, int num_blocks,
                                    int max_seq_len, int32_t* dev_err, cudaStream_t stream) {
    using namespace pkv;
    using namespace pkv::commit;
    if (layers < 0 || rows < 0 || max_path < 0 || kv_heads <= 0 || head_dim <= 0 || block_size <= 0 ||
        max_blocks_per_row <= 0 || num_blocks <= 0 || max_seq_len < 0 || (elt_bytes != 1 && elt_bytes != 2))
        return PKV_ERR_INVALID_ARG;
    if ((int64_t)max_seq_len > (int64_t)max_blocks_per_row * block_size) return PKV_ERR_INVALID_ARG;
    if ((int64_t)head_dim * elt_bytes % 16) return PKV_ERR_UNSUPPORTED;
    const int64_t vecs = (int64_t)kv_heads * head_dim * elt_bytes / 16;
    if (vecs > (1 << 20) || (int64_t)num_blocks * block_size >= (int64_t(1) << 31)) return PKV_ERR_UNSUPPORTED;
    if (layers == 0 || rows == 0) return PKV_OK;
    if (!k_pool || !v_pool || !block_tables || !seq_lens || !q_start || !path_lens || (max_path > 0 && !path))
        return PKV_ERR_INVALID_ARG;
    if (!aligned16(k_pool) || !aligned16(v_pool)) return PKV_ERR_INVALID_ARG;
    // every layer's warps read these, so the new lengths lie elsewhere
    if (new_seq_lens) {
        const size_t n = (size_t)rows * 4;
        if (overlap(new_seq_lens, n, seq_lens, n) || overlap(new_seq_lens, n, q_start, n + 4) ||
            overlap(new_seq_lens, n, path_lens, n) || overlap(new_seq_lens, n, path, n * max_path) ||
            overlap(new_seq_lens, n, block_tables, n * max_blocks_per_row))
            return PKV_ERR_INVALID_ARG;
    }
    const int64_t warps = (int64_t)layers * 2 * rows;
    const int64_t blocks = (warps + kWarps - 1) / kWarps;
    if (blocks > 0x7fffffff) return PKV_ERR_UNSUPPORTED;
    return launch_early(tree_commit_kernel, (unsigned)blocks, kWarps * 32, 0, stream, static_cast<uint4*>(k_pool),
                        static_cast<uint4*>(v_pool), block_tables, seq_lens, q_start, path, path_lens, new_seq_lens,
                        layers, rows, max_path, (int)vecs, block_size, max_blocks_per_row, num_blocks, max_seq_len,
                        dev_err);
}
