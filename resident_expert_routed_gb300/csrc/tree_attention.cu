// Attention of drafted tokens over the paged 8-bit key/value cache.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "common.cuh"

namespace {

struct AttnArgs {
    moe_kv_cache c;
    const __nv_bfloat16* q;
    int64_t q_token_stride, q_head_stride;
    int n_nodes, n_q_heads, group;               // group: query heads to a kv head
    const int32_t* table;
    int width, lanes, page_shift;
    const int32_t* kv_len;
    const int32_t* cu;
    int max_nodes;
    const int32_t* mask;
    int mask_words;
    float scale;
    __nv_bfloat16* out;
    float* lse;
    uint32_t* err;
};

MOE_DEV float2 e4m3x2_to_float2(uint32_t w) {
    return __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w & 0xFFFFu), __NV_E4M3)));
}

// One block per (node, query head): a thread scores one row of a tile of 128,
// the block joins the running maximum and sum, and a thread then adds up its
// columns of the output.
__global__ void __launch_bounds__(128) tree_attention(const AttnArgs a) {
    __shared__ float qs[256];
    __shared__ float ps[128];
    __shared__ int64_t rows[128];
    __shared__ float red[4];
    pdl_trigger();
    pdl_wait();
    const int node = blockIdx.x, qh = blockIdx.y, h = qh / a.group;
    const int D = a.c.head_dim, tid = threadIdx.x;
    int lo = 0, hi = a.lanes;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a.cu[mid] <= node) lo = mid; else hi = mid;
    }
    const int n = a.cu[lo + 1] - a.cu[lo], t = node - a.cu[lo];
    int len = a.kv_len[lo];
    if (n > a.max_nodes || len < n || ((int64_t)len + (1 << a.page_shift) - 1) >> a.page_shift > a.width) {
        if (tid == 0) record_error(a.err, MOE_DEV_BAD_PAGE);
        len = 0;
    }
    const int prefix = len - n;
    for (int d = tid; d < D; d += 128)
        qs[d] = __bfloat162float(a.q[node * a.q_token_stride + qh * a.q_head_stride + d]);
    const uint8_t* kc = static_cast<const uint8_t*>(a.c.k_codes);
    const uint8_t* vc = static_cast<const uint8_t*>(a.c.v_codes);
    float m = -INFINITY, l = 0.0f, acc[2] = {0.0f, 0.0f};
    for (int j0 = 0; j0 < len; j0 += 128) {
        __syncthreads();
        const int j = j0 + tid;
        float s = -INFINITY;
        int64_t row = 0;
        if (j < len) {
            int page = a.table[(int64_t)lo * a.width + (j >> a.page_shift)];
            if (page < 0 || page >= a.c.n_pages) {
                record_error(a.err, MOE_DEV_BAD_PAGE);
                page = 0;
            }
            row = (((int64_t)page * a.c.n_kv_heads + h) << a.page_shift) + (j & ((1 << a.page_shift) - 1));
            const int i = j - prefix;
            const bool sees = i < 0 || (a.mask ? (a.mask[(int64_t)node * a.mask_words + (i >> 5)] >> (i & 31)) & 1 : i <= t);
            if (sees) {
                float dot = 0.0f;
                for (int d = 0; d < D; d += 4) {
                    const uint32_t w = *reinterpret_cast<const uint32_t*>(kc + row * D + d);
                    const float2 x = e4m3x2_to_float2(w), y = e4m3x2_to_float2(w >> 16);
                    dot += x.x * qs[d] + x.y * qs[d + 1] + y.x * qs[d + 2] + y.y * qs[d + 3];
                }
                s = dot * e8m0_to_float(a.c.k_scales[row]) * a.scale;
            } else {
                row = -1;                                     // not seen: its values take no part
            }
        } else {
            row = -1;
        }
        rows[tid] = row;
        float mx = s;                                         // NaN scores pass by the maximum and reach the sum
        for (int off = 16; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, off));
        if ((tid & 31) == 0) red[tid >> 5] = mx;
        __syncthreads();
        const float mn = fmaxf(fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])), m);
        const float ref = mn == -INFINITY ? 0.0f : mn;
        const float alpha = expf(m - ref);
        const float p = row < 0 ? 0.0f : expf(s - ref);
        ps[tid] = p;
        m = mn;
        __syncthreads();
        float sum = 0.0f;
        for (int i = 0; i < 128; ++i) sum += ps[i];
        l = l * alpha + sum;
        for (int k = 0; k < 2; ++k) {
            const int d = tid + 128 * k;
            if (d >= D) break;
            float o = 0.0f;
            for (int i = 0; i < 128; ++i)
                if (rows[i] >= 0) {
                    const __half v = __half(__nv_cvt_fp8_to_halfraw(vc[rows[i] * D + d], __NV_E4M3));
                    o += ps[i] * __half2float(v) * e8m0_to_float(a.c.v_scales[rows[i]]);
                }
            acc[k] = acc[k] * alpha + o;
        }
    }
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    for (int k = 0; k < 2; ++k) {
        const int d = tid + 128 * k;
        if (d < D) a.out[((int64_t)node * a.n_q_heads + qh) * D + d] = __float2bfloat16_rn(acc[k] * inv);
    }
    if (a.lse && tid == 0) a.lse[(int64_t)node * a.n_q_heads + qh] = l == 0.0f ? -INFINITY : m + logf(l);
}

int log2_of(int p) { return 31 - __builtin_clz((unsigned)p); }

size_t attention_workspace() { return 256; }

}  // namespace

size_t moe_tree_attention_workspace_bytes(int n_nodes, int n_q_heads, int n_kv_heads, int head_dim, int lanes) {
    if (n_nodes < 1 || n_q_heads < 1 || n_kv_heads < 1 || head_dim < 1 || lanes < 1) return 0;
    return attention_workspace();
}

moe_status moe_tree_attention(const void* q, int64_t q_token_stride, int64_t q_head_stride, int n_nodes, int n_q_heads,
                              const moe_kv_cache* cache, const int32_t* page_table, int table_width, int lanes,
                              const int32_t* kv_len, const int32_t* cu_nodes, int max_nodes, const int32_t* tree_mask,
                              int mask_words, float scale, void* out, float* lse, void* workspace, size_t ws_bytes,
                              void* stream) {
    MOE_RANGE("moe_tree_attention");
    const moe_status cs = kv_cache_status(cache);
    if (cs != MOE_OK) return cs;
    if (n_nodes < 0) return MOE_EINVAL;
    if (n_nodes == 0) return MOE_OK;
    if (!q || !page_table || !kv_len || !cu_nodes || !out || !workspace) return MOE_EINVAL;
    if (((uintptr_t)q | (uintptr_t)out | (uintptr_t)workspace) & 15) return MOE_EINVAL;
    if (lanes < 1 || table_width < 1 || n_q_heads < 1 || max_nodes < 1 || n_q_heads % cache->n_kv_heads) return MOE_EINVAL;
    if (q_token_stride % 8 || q_head_stride % 8 || !(scale > 0.0f) || scale > 3.0e38f) return MOE_EINVAL;
    if (tree_mask && (mask_words < 1 || (int64_t)mask_words * 32 < max_nodes)) return MOE_EINVAL;
    if (lanes > 4096 || n_q_heads > 1024 || max_nodes > 65536 || mask_words > 2048) return MOE_EUNSUPPORTED;
    if (ws_bytes < moe_tree_attention_workspace_bytes(n_nodes, n_q_heads, cache->n_kv_heads, cache->head_dim, lanes)) return MOE_ENOMEM;
    uint32_t* err = moe_err_word();
    if (!err) return MOE_ECUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    AttnArgs a{};
    a.c = *cache;
    a.q = static_cast<const __nv_bfloat16*>(q);
    a.q_token_stride = q_token_stride;
    a.q_head_stride = q_head_stride;
    a.n_nodes = n_nodes;
    a.n_q_heads = n_q_heads;
    a.group = n_q_heads / cache->n_kv_heads;
    a.table = page_table;
    a.width = table_width;
    a.lanes = lanes;
    a.page_shift = log2_of(cache->page_size);
    a.kv_len = kv_len;
    a.cu = cu_nodes;
    a.max_nodes = max_nodes;
    a.mask = tree_mask;
    a.mask_words = mask_words;
    a.scale = scale;
    a.out = static_cast<__nv_bfloat16*>(out);
    a.lse = lse;
    a.err = err;
    moe_prof_begin(MK_ATTENTION, s);
    const cudaError_t e = moe_launch(tree_attention, dim3((unsigned)n_nodes, (unsigned)n_q_heads), dim3(128), 0, s, a);
    moe_prof_end(MK_ATTENTION, s);
    moe_count_launches(1);
    return e == cudaSuccess ? MOE_OK : MOE_ECUDA;
}
