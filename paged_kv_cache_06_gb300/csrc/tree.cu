// paged_attention_tree: attention of each row's drafted nodes over its cached
// tokens and the nodes that their mask lets them see.
//
// One warp per (node, query head): four dims a lane, one token at a time, the
// running maximum and sum of the softmax in 32 bits.
#include "fp8_codec.cuh"
#include "pkv_internal.cuh"

namespace pkv {
namespace tree {

constexpr int kWarps = 4;
constexpr float kLog2e = 1.4426950408889634f;

template <bool kFp8>
__device__ __forceinline__ void load4(const void* pool, int64_t at, float (&x)[4]) {
    uint32_t lo, hi;
    if (kFp8) {
        widen4(*reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(pool) + at), lo, hi);
    } else {
        const uint2 v = *reinterpret_cast<const uint2*>(static_cast<const __half*>(pool) + at);
        lo = v.x;
        hi = v.y;
    }
    const float2 a = __half22float2(*reinterpret_cast<__half2*>(&lo));
    const float2 b = __half22float2(*reinterpret_cast<__half2*>(&hi));
    x[0] = a.x;
    x[1] = a.y;
    x[2] = b.x;
    x[3] = b.y;
}

template <bool kFp8>
__global__ void __launch_bounds__(kWarps * 32) tree_kernel(
    __half* out, const __half* q, const void* k_pool, const void* v_pool, const float* k_scale,
    const float* v_scale, const int32_t* tables, const int32_t* seq_lens, const int32_t* q_start,
    const uint32_t* mask, int words, int rows, int total, int hq, int hk, int bs, float scale, int mbpr, int nb,
    int limit, int32_t* dev_err) {
    const int lane = threadIdx.x & 31;
    const int64_t w = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    const int g = (int)(w / hq), h = (int)(w % hq);
    if (g >= total) return;
    int lo = 0, hi = rows;  // q_start[lo] <= g < q_start[hi]
    if (g >= q_start[rows] || g < q_start[0]) return;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (q_start[mid] <= g) lo = mid; else hi = mid;
    }
    const int r = lo, q0 = q_start[r], C = q_start[r + 1] - q0, L = seq_lens[r];
    const bool report = h == 0 && lane == 0;
    if (C < 0 || L < C || L > limit) {
        if (report) flag_error(dev_err, PKV_DEV_ERR_SEQ_LEN);
        return;
    }
    if (mask && C > 32 * words) {
        if (report) flag_error(dev_err, PKV_DEV_ERR_MASK);
        return;
    }
    const int i = g - q0, P = L - C, kvh = h / (hq / hk);
    const float ks = kFp8 ? k_scale[kvh] : 1.f, vs = kFp8 ? v_scale[kvh] : 1.f;
    const float sl = scale * ks * kLog2e;
    float x[4], o[4] = {0.f, 0.f, 0.f, 0.f}, m = -INFINITY, l = 0.f;
    load4<false>(q, ((int64_t)g * hq + h) * kHeadDim + lane * 4, x);
    for (int t = 0; t < L; ++t) {
        const int j = t - P;
        if (j >= 0 && !(mask ? (mask[(int64_t)g * words + (j >> 5)] >> (j & 31)) & 1 : j <= i)) continue;
        const int pb = tables[(int64_t)r * mbpr + t / bs];
        if (pb < 0 || pb >= nb) {
            if (report) flag_error(dev_err, PKV_DEV_ERR_BLOCK_ID);
            continue;
        }
        const int64_t at = (((int64_t)pb * bs + t % bs) * hk + kvh) * kHeadDim + lane * 4;
        float k[4], v[4];
        load4<kFp8>(k_pool, at, k);
        load4<kFp8>(v_pool, at, v);
        const float s = warp_sum(x[0] * k[0] + x[1] * k[1] + x[2] * k[2] + x[3] * k[3]) * sl;
        const float mn = fmaxf(m, s), a = exp2f(m - (mn == -INFINITY ? 0.f : mn));
        const float p = exp2f(s - (mn == -INFINITY ? 0.f : mn));
        m = mn;
        l = l * a + p;
#pragma unroll
        for (int d = 0; d < 4; ++d) o[d] = o[d] * a + p * v[d];
    }
    const float inv = l == 0.f ? 0.f : vs / l;
    __half2* dst = reinterpret_cast<__half2*>(out + ((int64_t)g * hq + h) * kHeadDim + lane * 4);
    dst[0] = __floats2half2_rn(o[0] * inv, o[1] * inv);
    dst[1] = __floats2half2_rn(o[2] * inv, o[3] * inv);
}

}  // namespace tree
}  // namespace pkv

extern "C" size_t paged_attention_tree_workspace_size(int rows, int total_q, int q_heads, int kv_heads,
                                                      int head_dim, int block_size) {
    if (rows < 0 || total_q < 0 || q_heads <= 0 || kv_heads <= 0 || q_heads % kv_heads || head_dim <= 0 ||
        block_size <= 0)
        return 0;
    return 256;
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
    if (rows < 0 || total_q < 0 || q_heads <= 0 || kv_heads <= 0 || q_heads % kv_heads || head_dim <= 0 ||
        block_size <= 0 || max_blocks_per_row <= 0 || num_blocks <= 0 || max_seq_len < 0 || !isfinite(scale))
        return PKV_ERR_INVALID_ARG;
    if ((int64_t)max_seq_len > (int64_t)max_blocks_per_row * block_size) return PKV_ERR_INVALID_ARG;
    if ((k_scale == nullptr) != (v_scale == nullptr) || (mask && mask_words <= 0)) return PKV_ERR_INVALID_ARG;
    if (head_dim != kHeadDim || block_size % 16 || rows > 1024 || q_heads > 65535 || (mask && mask_words > 32))
        return PKV_ERR_UNSUPPORTED;
    if (rows == 0 || total_q == 0) return PKV_OK;
    if (!out || !q || !k_pool || !v_pool || !block_tables || !seq_lens || !q_start) return PKV_ERR_INVALID_ARG;
    if (!aligned16(out) || !aligned16(q) || !aligned16(k_pool) || !aligned16(v_pool)) return PKV_ERR_INVALID_ARG;
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255) ||
        workspace_bytes < paged_attention_tree_workspace_size(rows, total_q, q_heads, kv_heads, head_dim, block_size))
        return PKV_ERR_WORKSPACE;
    const int64_t blocks = ((int64_t)total_q * q_heads + tree::kWarps - 1) / tree::kWarps;
    if (blocks > 0x7fffffff) return PKV_ERR_UNSUPPORTED;
    auto* f = k_scale ? tree::tree_kernel<true> : tree::tree_kernel<false>;
    f<<<(unsigned)blocks, tree::kWarps * 32, 0, stream>>>(
        static_cast<__half*>(out), static_cast<const __half*>(q), k_pool, v_pool, k_scale, v_scale, block_tables,
        seq_lens, q_start, mask, mask_words, rows, total_q, q_heads, kv_heads, block_size, scale,
        max_blocks_per_row, num_blocks, max_seq_len, dev_err);
    return launch_status();
}
