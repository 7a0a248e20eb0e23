// Attention of a chunk of new tokens over the paged 8-bit key/value cache: a plain kernel.
//
// A block takes 32 rows (token, query head) of one lane and kv head, tiles of
// 32 cache rows come as fp32 into shared memory, and a running maximum and sum
// carry the softmax over them. All arithmetic is fp32 on the CUDA cores.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "common.cuh"

namespace {

struct ChunkArgs {
    moe_kv_cache c;
    const __nv_bfloat16* q;
    int64_t q_token, q_head;
    int n_tokens, n_q, group;
    const int32_t* table;
    int width, lanes, page_shift;
    const int32_t* kv_len;
    const int32_t* cu;
    float scale_log2;
    __nv_bfloat16* out;
    float* lse;
    uint32_t* err;
};

constexpr int ROWS = 32, TILE = 32, WARPS = 8;

template <int D>
__global__ void __launch_bounds__(WARPS * 32) chunk_attention(const ChunkArgs a) {
    extern __shared__ float sm[];
    float* Q = sm;                          // [ROWS][D]
    float* K = Q + ROWS * D;                // [TILE][D + 1]
    float* V = K + TILE * (D + 1);          // [TILE][D]
    __shared__ int place[4];
    pdl_trigger();
    pdl_wait();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, h = blockIdx.y, G = a.group;
    if (tid == 0) {                         // the lane whose rows this block has
        int u = blockIdx.x, b = 0;
        place[0] = -1;
        for (; b < a.lanes; ++b) {
            const int n0 = a.cu[b], n = a.cu[b + 1] - n0;
            if (n0 < 0 || n < 0 || n > a.n_tokens - n0) { if (h == 0) record_error(a.err, MOE_DEV_BAD_PAGE); continue; }
            const int units = (n * G + ROWS - 1) / ROWS;
            if (u < units) { place[0] = n0; place[1] = n; place[2] = u * ROWS; place[3] = b; break; }
            u -= units;
        }
    }
    __syncthreads();
    if (place[0] < 0) return;
    const int n0 = place[0], n = place[1], row0 = place[2], b = place[3];
    const int rows = min(ROWS, n * G - row0);
    int len = a.kv_len[b];
    bool refused = len < n || (((int64_t)len + (1 << a.page_shift) - 1) >> a.page_shift) > a.width;
    if (refused) { if (tid == 0) record_error(a.err, MOE_DEV_BAD_PAGE); len = 0; }
    const int prefix = len - n;
    for (int i = tid; i < rows * D; i += WARPS * 32) {
        const int r = i / D, d = i % D, t = (row0 + r) / G, g = (row0 + r) % G;
        Q[i] = __bfloat162float(a.q[(n0 + t) * a.q_token + (h * G + g) * a.q_head + d]) * a.scale_log2;
    }
    constexpr int V_ = D / 32, RW = ROWS / WARPS;
    float o[RW][V_] = {}, m[RW], l[RW];
    for (int r = 0; r < RW; ++r) { m[r] = -INFINITY; l[r] = 0.0f; }
    const int end = refused ? 0 : prefix + (row0 + rows - 1) / G + 1;
    for (int j0 = 0; j0 < end; j0 += TILE) {
        __syncthreads();
        for (int i = tid; i < TILE * D; i += WARPS * 32) {
            const int j = j0 + i / D, d = i % D;
            float kf = 0.0f, vf = 0.0f;
            if (j < end) {
                int page = a.table[(int64_t)b * a.width + (j >> a.page_shift)];
                if (page < 0 || page >= a.c.n_pages) { record_error(a.err, MOE_DEV_BAD_PAGE); page = 0; }
                const int64_t row = (((int64_t)page * a.c.n_kv_heads + h) << a.page_shift) + (j & ((1 << a.page_shift) - 1));
                auto value = [&](const void* codes, const uint8_t* scales) {
                    const uint32_t s = scales[row];
                    const __nv_fp8_storage_t code = static_cast<const uint8_t*>(codes)[row * D + d];
                    return __half2float(__half(__nv_cvt_fp8_to_halfraw(code, __NV_E4M3))) * e8m0_to_float(s);
                };
                kf = value(a.c.k_codes, a.c.k_scales);
                vf = value(a.c.v_codes, a.c.v_scales);
            }
            K[(i / D) * (D + 1) + d] = kf;
            V[i] = vf;
        }
        __syncthreads();
#pragma unroll
        for (int r = 0; r < RW; ++r) {
            const int row = warp * RW + r;
            if (row >= rows) continue;
            const int limit = prefix + (row0 + row) / G;         // the last row it sees
            float s = 0.0f;
            for (int d = 0; d < D; ++d) s = fmaf(Q[row * D + d], K[lane * (D + 1) + d], s);
            const bool sees = j0 + lane <= limit;
            if (!sees) s = -INFINITY;
            float top = s;
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, off));
            top = fmaxf(top, m[r]);
            const float base = top == -INFINITY ? 0.0f : top;
            const float p = exp2f(s - base), f = exp2f(m[r] - base);
            float sum = p;
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, off);
            l[r] = l[r] * f + sum;
            m[r] = top;
#pragma unroll
            for (int e = 0; e < V_; ++e) o[r][e] *= f;
            const int seen = min(TILE, limit + 1 - j0);
            for (int j = 0; j < seen; ++j) {
                const float pj = __shfl_sync(0xFFFFFFFFu, p, j);
#pragma unroll
                for (int e = 0; e < V_; ++e) o[r][e] = fmaf(pj, V[j * D + e * 32 + lane], o[r][e]);
            }
        }
    }
#pragma unroll
    for (int r = 0; r < RW; ++r) {
        const int row = warp * RW + r;
        if (row >= rows) continue;
        const int t = (row0 + row) / G, g = (row0 + row) % G;
        const int64_t at = (int64_t)(n0 + t) * a.n_q + h * G + g;
        for (int e = 0; e < V_; ++e) a.out[at * D + e * 32 + lane] = __float2bfloat16_rn(refused ? 0.0f : o[r][e] / l[r]);
        if (a.lse && lane == 0) a.lse[at] = refused ? -INFINITY : (m[r] + log2f(l[r])) * 0.69314718055994531f;
    }
}

template <int D>
cudaError_t launch(const ChunkArgs& a, cudaStream_t s) {
    const size_t smem = (size_t)(ROWS * D + TILE * (D + 1) + TILE * D) * sizeof(float);
    cudaError_t e = cudaFuncSetAttribute(chunk_attention<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    const int64_t units = (int64_t)a.n_tokens * a.group / ROWS + a.lanes;
    return moe_launch(chunk_attention<D>, dim3((unsigned)units, (unsigned)a.c.n_kv_heads), dim3(WARPS * 32), smem, s, a);
}

int log2_of(int p) { return 31 - __builtin_clz((unsigned)p); }

}  // namespace

size_t moe_chunk_attention_workspace_bytes(int n_tokens, int n_q_heads, int n_kv_heads, int head_dim, int lanes) {
    if (n_tokens < 1 || n_q_heads < 1 || n_kv_heads < 1 || head_dim < 1 || lanes < 1) return 0;
    return 16;
}

moe_status moe_chunk_attention(const void* q, int64_t q_token_stride, int64_t q_head_stride, int n_tokens, int n_q_heads,
                               const moe_kv_cache* cache, const int32_t* page_table, int table_width, int lanes,
                               const int32_t* kv_len, const int32_t* cu_tokens, float scale, void* out, float* lse,
                               void* workspace, size_t ws_bytes, void* stream) {
    MOE_RANGE("moe_chunk_attention");
    const moe_status cs = kv_cache_status(cache);
    if (cs != MOE_OK) return cs;
    if (n_tokens < 0) return MOE_EINVAL;
    if (n_tokens == 0) return MOE_OK;
    if (!q || !page_table || !kv_len || !cu_tokens || !out || !workspace) return MOE_EINVAL;
    if (((uintptr_t)q | (uintptr_t)out | (uintptr_t)workspace) & 15) return MOE_EINVAL;
    if (lanes < 1 || table_width < 1 || n_q_heads < 1 || n_q_heads % cache->n_kv_heads) return MOE_EINVAL;
    if (q_token_stride % 8 || q_head_stride % 8 || !(scale > 0.0f) || scale > 3.0e38f) return MOE_EINVAL;
    if (lanes > 4096 || n_q_heads > 1024 || n_q_heads / cache->n_kv_heads > 128 || n_tokens > (1 << 24)) return MOE_EUNSUPPORTED;
    if (ws_bytes < moe_chunk_attention_workspace_bytes(n_tokens, n_q_heads, cache->n_kv_heads, cache->head_dim, lanes)) return MOE_ENOMEM;
    uint32_t* err = moe_err_word();
    if (!err) return MOE_ECUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    ChunkArgs a{};
    a.c = *cache;
    a.q = static_cast<const __nv_bfloat16*>(q);
    a.q_token = q_token_stride;
    a.q_head = q_head_stride;
    a.n_tokens = n_tokens;
    a.n_q = n_q_heads;
    a.group = n_q_heads / cache->n_kv_heads;
    a.table = page_table;
    a.width = table_width;
    a.lanes = lanes;
    a.page_shift = log2_of(cache->page_size);
    a.kv_len = kv_len;
    a.cu = cu_tokens;
    a.scale_log2 = scale * 1.4426950408889634f;
    a.out = static_cast<__nv_bfloat16*>(out);
    a.lse = lse;
    a.err = err;
    moe_prof_begin(MK_CHUNK_ATTENTION, s);
    const cudaError_t e = cache->head_dim == 64 ? launch<64>(a, s) : cache->head_dim == 128 ? launch<128>(a, s) : launch<256>(a, s);
    moe_prof_end(MK_CHUNK_ATTENTION, s);
    moe_count_launches(1);
    return e == cudaSuccess ? MOE_OK : MOE_ECUDA;
}
