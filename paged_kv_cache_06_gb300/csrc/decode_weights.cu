// paged_attention_decode_weights: decode attention that also adds to each cached
// token's running sum the softmax weight it got, over the heads of its group.
//
// Mathematics.  With s_h[t] the base-2 scores of query head h, m_h their maximum and
// l_h = sum_t 2^(s_h[t] - m_h), token t got sum_h 2^(s_h[t] - m_h) / l_h.  m_h and l_h
// are known only when the last of the row's tokens has been seen, by which time the keys
// are gone; so the decode kernel writes its scores as it goes (4 bytes a head and token, 24
// against the 512 bytes of keys and values that six heads read) and a second kernel,
// which starts early and waits for the first, turns them into weights.  Reading the keys
// again instead would cost 256 bytes a token.
//
// What bounds it: the decode kernel.  The second kernel reads the scores (from L2 as
// a rule) and reads and writes the sums, four tokens a thread.
#include <math.h>

#include "pkv_internal.cuh"
#include "ptx.cuh"

namespace pkv {
namespace weights {

constexpr int kThreads = 256;
constexpr int kTokens = 4;  // a thread

// Sum over a unit's heads (kPairs pairs of them; the last may be a half) of each token's weight.
template <int kPairs>
__global__ void __launch_bounds__(kThreads) add_weights_kernel(float* out, const float* scores, const float2* maxima,
                                                               const int32_t* seq_lens, int hk, int group,
                                                               int score_tokens, int64_t stride, int limit) {
    const int unit = (int)blockIdx.x, r = unit / hk;
    const int t0 = (int)blockIdx.y * (kThreads * kTokens) + (int)threadIdx.x;
    ptx::griddep_wait();
    const int L = min(max(seq_lens[r], 0), limit);
    if (t0 >= L) return;
    float m[2 * kPairs], inv[2 * kPairs];
#pragma unroll
    for (int h = 0; h < 2 * kPairs; ++h) {
        const float2 x = h < group ? maxima[(int64_t)unit * kMaxGroup + h] : make_float2(0.f, 0.f);
        m[h] = x.x;
        inv[h] = x.y;
    }
    const float2* s = reinterpret_cast<const float2*>(scores) + ((int64_t)unit * score_tokens) * kPairs;
    float* w = out + (int64_t)unit * stride;
    float2 x[kTokens][kPairs];
    float was[kTokens];
#pragma unroll
    for (int i = 0; i < kTokens; ++i) {
        const int t = t0 + i * kThreads;
        if (t >= L) continue;
#pragma unroll
        for (int k = 0; k < kPairs; ++k) x[i][k] = s[(int64_t)t * kPairs + k];
        was[i] = t < L - 1 ? w[t] : 0.f;  // the step's own token starts from zero
    }
#pragma unroll
    for (int i = 0; i < kTokens; ++i) {
        const int t = t0 + i * kThreads;
        if (t >= L) continue;
        float sum = 0.f;
#pragma unroll
        for (int k = 0; k < kPairs; ++k) {
            sum += ptx::fast_exp2(x[i][k].x - m[2 * k]) * inv[2 * k];
            if (2 * k + 1 < group) sum += ptx::fast_exp2(x[i][k].y - m[2 * k + 1]) * inv[2 * k + 1];
        }
        w[t] = was[i] + sum;
    }
}

struct Layout {
    size_t maxima, scores, bytes;
    int tokens, heads;
};
static Layout layout(int rows, int q_heads, int kv_heads, int max_seq_len) {
    Layout l;
    const size_t units = (size_t)rows * kv_heads;
    l.tokens = (int)align_up((size_t)max_seq_len, 16);
    l.heads = (q_heads / kv_heads + 1) / 2 * 2;
    l.maxima = align_up(tma_workspace_bytes(rows, q_heads, kv_heads, max_seq_len), 256);
    l.scores = l.maxima + align_up(units * kMaxGroup * sizeof(float2), 256);
    l.bytes = l.scores + align_up(units * l.tokens * l.heads * sizeof(float), 256);
    return l;
}

}  // namespace weights
}  // namespace pkv

extern "C" size_t paged_attention_decode_weights_workspace_size(int rows, int q_heads, int kv_heads, int head_dim,
                                                                int max_seq_len, int block_size) {
    using namespace pkv;
    if (rows <= 0 || q_heads <= 0 || kv_heads <= 0 || q_heads % kv_heads || max_seq_len < 0 ||
        max_seq_len > (1 << 30) || block_size <= 0 ||
        !tma_decode_supported(rows, q_heads, kv_heads, head_dim, block_size))
        return 0;
    return weights::layout(rows, q_heads, kv_heads, max_seq_len).bytes;
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
    if (!tma_decode_supported(rows, q_heads, kv_heads, head_dim, block_size) || (k_scale && kv_heads > 16) ||
        max_seq_len > (1 << 26) || weights_stride > (int64_t(1) << 40))
        return PKV_ERR_UNSUPPORTED;
    if (rows == 0) return PKV_OK;
    if (!out || !weights || !q || !k_pool || !v_pool || !block_tables || !seq_lens) return PKV_ERR_INVALID_ARG;
    if (!aligned16(out) || !aligned16(q) || !aligned16(k_pool) || !aligned16(v_pool)) return PKV_ERR_INVALID_ARG;
    const Layout l = layout(rows, q_heads, kv_heads, max_seq_len);
    if (!workspace || workspace_bytes < l.bytes || (reinterpret_cast<uintptr_t>(workspace) & 255))
        return PKV_ERR_WORKSPACE;
    const size_t wide = (size_t)rows * kv_heads * weights_stride * 4, tall = (size_t)rows * q_heads * head_dim * 2;
    if (overlap(weights, wide, out, tall) || overlap(weights, wide, q, tall) ||
        overlap(weights, wide, workspace, l.bytes))
        return PKV_ERR_INVALID_ARG;

    unsigned char* ws = static_cast<unsigned char*>(workspace);
    ScoreArgs sc;
    sc.scores = reinterpret_cast<float*>(ws + l.scores);
    sc.maxima = reinterpret_cast<float2*>(ws + l.maxima);
    sc.tokens = l.tokens;
    sc.heads = l.heads;
    const int st = tma_decode_launch(out, q, k_pool, v_pool, block_tables, seq_lens, rows, q_heads, kv_heads,
                                     block_size, scale, max_blocks_per_row, num_blocks, max_seq_len, 0, workspace,
                                     dev_err, stream, nullptr, false, k_scale, v_scale, nullptr, &sc);
    if (st != PKV_OK || max_seq_len == 0) return st;
    auto* kernel = l.heads == 2   ? add_weights_kernel<1>
                   : l.heads == 4 ? add_weights_kernel<2>
                   : l.heads == 6 ? add_weights_kernel<3>
                                  : add_weights_kernel<4>;
    const int tiles = (max_seq_len + kThreads * kTokens - 1) / (kThreads * kTokens);
    return launch_early(kernel, dim3((unsigned)(rows * kv_heads), (unsigned)tiles), kThreads, 0, stream, weights,
                        sc.scores, sc.maxima, seq_lens, kv_heads, q_heads / kv_heads, l.tokens, weights_stride,
                        max_seq_len);
}
