// The paged 8-bit key/value cache: writing, reading back, keeping an accepted path.
//
// Format (include/moe_resident.h): per (row, head) vector head_dim e4m3 codes
// and one e8m0 scale, 2^e with e the smallest exponent that keeps max|x| within
// 448 * 2^e. The three calls only move and convert bytes, so HBM bounds the
// large ones and the launch the small ones. A code is rounded once, to nearest
// (ties to even): scaling by a power of two is exact. Reading back multiplies
// by that power in fp32, which is exact too (but below the smallest normal
// fp16, and where a value of 2^127 and more leaves the type).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "common.cuh"

namespace {

constexpr int KV_THREADS = 256;

template <typename T> MOE_DEV float to_float(T v);
template <> MOE_DEV float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
template <> MOE_DEV float to_float(__half v) { return __half2float(v); }
template <> MOE_DEV float to_float(float v) { return v; }

template <typename T> MOE_DEV T from_float(float v);
template <> MOE_DEV __nv_bfloat16 from_float(float v) { return __float2bfloat16_rn(v); }
template <> MOE_DEV __half from_float(float v) { return __float2half_rn(v); }
template <> MOE_DEV float from_float(float v) { return v; }

// The scale exponent of a vector: the smallest e with amax <= 448 * 2^e =
// 1.75 * 2^(e + 8), clamped to [-100, 120]. With amax = m * 2^E, 1 <= m < 2:
// E - 8, and one more when m > 1.75.
MOE_DEV int kv_exponent(float amax) {
    if (amax == 0.0f) return 0;
    const int E = floor_log2_pos(amax);
    const bool over = E >= -126 && (__float_as_uint(amax) & 0x7FFFFFu) > 0x600000u;   // subnormals are clamped anyway
    const int e = E - 8 + (over ? 1 : 0);
    return e < -100 ? -100 : (e > 120 ? 120 : e);
}

struct KvSide {
    const void* src;
    int64_t token_stride, head_stride;     // elements
    uint8_t* codes;
    uint8_t* scales;
};

// moe_kv_write. D / 16 lanes share a vector: 16 elements a lane, one 16-byte
// store of codes, the maximum by shuffles within the group, so a vector is read
// once and stays in registers. blockIdx.y picks keys or values. Measured (calls back
// to back in a graph, so inputs partly from L2; 8 heads of 128, bf16): 8,192 rows 8.6 us
// (50.5 MB, 5.8 TB/s), two rows 1.5 us, a launch. Called from Python 20 and 15 us: the host.
template <typename T, int D>
__global__ void __launch_bounds__(KV_THREADS) kv_write(const KvSide k, const KvSide v, const int64_t* __restrict__ slots,
                                                       int n_tokens, int H, int page_shift, int64_t n_rows, uint32_t* err) {
    constexpr int LPV = D / 16;
    constexpr int PER_LOAD = 16 / sizeof(T), LOADS = 16 / PER_LOAD;
    pdl_trigger();
    const KvSide s = blockIdx.y ? v : k;
    const int64_t vec = ((int64_t)blockIdx.x * KV_THREADS + threadIdx.x) / LPV;
    const int part = threadIdx.x % LPV;
    pdl_wait();
    const bool inside = vec < (int64_t)n_tokens * H;
    const int t = inside ? (int)(vec / H) : 0, h = inside ? (int)(vec - (int64_t)t * H) : 0;
    const int64_t slot = inside ? slots[t] : -1;
    const bool on = slot >= 0 && slot < n_rows;
    float x[16];
    float amax = 0.0f;
    bool fine = true;
    if (on) {
        const uint4* p = reinterpret_cast<const uint4*>(static_cast<const T*>(s.src) + t * s.token_stride + h * s.head_stride + part * 16);
        uint4 raw[LOADS];
#pragma unroll
        for (int i = 0; i < LOADS; ++i) raw[i] = p[i];
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
            const T* e = reinterpret_cast<const T*>(&raw[i]);
#pragma unroll
            for (int j = 0; j < PER_LOAD; ++j) {
                const float f = to_float(e[j]);
                x[i * PER_LOAD + j] = f;
                amax = fmaxf(amax, fabsf(f));
                fine &= fabsf(f) <= 3.402823466e38f;      // false for infinities and NaN
            }
        }
    }
    // one value for the group: the bits of a non-negative float order as integers, a bad vector above all
    uint32_t key = fine ? __float_as_uint(amax) : 0x7FFFFFFFu;
#pragma unroll
    for (int off = LPV / 2; off > 0; off >>= 1) key = max(key, __shfl_xor_sync(0xFFFFFFFFu, key, off));
    if (!on) {
        if (inside && part == 0 && h == 0 && slot != -1) record_error(err, MOE_DEV_BAD_PAGE);
        return;
    }
    uint4 out = make_uint4(0u, 0u, 0u, 0u);
    uint32_t scale = 255u;
    if (key < 0x7F800000u) {
        const int e = kv_exponent(__uint_as_float(key));
        const float inv = exp2_int(-e);
        scale = (uint32_t)(e + 127);
        uint32_t* o = &out.x;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(x[4 * i] * inv, x[4 * i + 1] * inv), __NV_SATFINITE, __NV_E4M3);
            const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(x[4 * i + 2] * inv, x[4 * i + 3] * inv), __NV_SATFINITE, __NV_E4M3);
            o[i] = lo | (hi << 16);
        }
    } else if (part == 0) {
        record_error(err, MOE_DEV_NAN_KV);
    }
    const int64_t page = slot >> page_shift;
    const int64_t row = ((page * H + h) << page_shift) + (slot & ((1 << page_shift) - 1));
    *reinterpret_cast<uint4*>(s.codes + row * D + part * 16) = out;
    if (part == 0) s.scales[row] = (uint8_t)scale;
}

// moe_kv_read. A block takes a few rows; their places are looked up once (a
// binary search over the lanes' row counts) and then every thread converts
// 16-byte pieces of the output, neighbours next to each other, READ_UNROLL
// pieces under way (one: 8.4 us for 7.8; eight: no faster). What is written is not read again
// here, so it is stored as streaming. Measured (as above): 8,191 rows of one lane
// 7.8 us (50.5 MB, 6.5 TB/s); called from Python 11 us.
constexpr int READ_ROWS = 32, READ_UNROLL = 4;

template <typename T, int D>
__global__ void __launch_bounds__(KV_THREADS) kv_read(const moe_kv_cache c, const int32_t* __restrict__ table, int width,
                                                      int lanes, const int32_t* __restrict__ starts,
                                                      const int32_t* __restrict__ cu, int n_rows, int rows_per_block,
                                                      uint32_t by_heads, int page_shift, T* __restrict__ k_out, T* __restrict__ v_out,
                                                      uint32_t* err) {
    constexpr int EPC = 16 / sizeof(T), CPV = D / EPC;         // elements a piece, pieces a vector
    __shared__ int64_t base[READ_ROWS];                        // first cache row (head 0) of each of the block's rows
    pdl_trigger();
    pdl_wait();
    const int64_t r0 = (int64_t)blockIdx.x * rows_per_block;
    const int rows = n_rows - r0 < rows_per_block ? (int)(n_rows - r0) : rows_per_block;
    const int H = c.n_kv_heads;
    if ((int)threadIdx.x < rows) {
        const int r = (int)r0 + threadIdx.x;
        int lo = 0, hi = lanes;                                // the lane with cu[lane] <= r < cu[lane + 1]
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (cu[mid] <= r) lo = mid; else hi = mid;
        }
        const int64_t at = (int64_t)(starts ? starts[lo] : 0) + r - cu[lo];
        int64_t b = -1;
        if (at >= 0 && (at >> page_shift) < width) {
            const int page = table[(int64_t)lo * width + (at >> page_shift)];
            if (page >= 0 && page < c.n_pages) b = (((int64_t)page * H) << page_shift) + (at & ((1 << page_shift) - 1));
        }
        if (b < 0) record_error(err, MOE_DEV_BAD_PAGE);
        base[threadIdx.x] = b;
    }
    __syncthreads();
    const uint8_t* codes = static_cast<const uint8_t*>(blockIdx.y ? c.v_codes : c.k_codes);
    const uint8_t* scales = blockIdx.y ? c.v_scales : c.k_scales;
    T* out = (blockIdx.y ? v_out : k_out) + r0 * H * D;
    const int pieces = rows * H * CPV;
    for (int i0 = threadIdx.x; i0 < pieces; i0 += READ_UNROLL * KV_THREADS) {
        uint32_t w[READ_UNROLL][EPC / 4];
        uint32_t s[READ_UNROLL];
#pragma unroll
        for (int u = 0; u < READ_UNROLL; ++u) {                // all loads before the first use
            const int i = i0 + u * KV_THREADS;
            s[u] = 255u;
            if (i >= pieces) continue;
            const int vec = i / CPV, part = i % CPV;
            const int row = H == 1 ? vec : (int)__umulhi((uint32_t)vec, by_heads), h = vec - row * H;
            const int64_t b = base[row];
            if (b < 0) continue;
            const int64_t at = b + ((int64_t)h << page_shift);
            if constexpr (EPC == 8) {
                const uint2 q = *reinterpret_cast<const uint2*>(codes + at * D + part * 8);
                w[u][0] = q.x;
                w[u][1] = q.y;
            } else {
                w[u][0] = *reinterpret_cast<const uint32_t*>(codes + at * D + part * 4);
            }
            s[u] = scales[at];
        }
#pragma unroll
        for (int u = 0; u < READ_UNROLL; ++u) {
            const int i = i0 + u * KV_THREADS;
            if (i >= pieces) break;
            const float f = e8m0_to_float(s[u]);
            uint4 o;
            T* e = reinterpret_cast<T*>(&o);
#pragma unroll
            for (int q = 0; q < EPC / 2; ++q) {
                const uint32_t two = s[u] == 255u ? 0u : w[u][q / 2] >> (16 * (q & 1));
                const float2 p = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)two, __NV_E4M3)));
                e[2 * q] = from_float<T>(p.x * f);
                e[2 * q + 1] = from_float<T>(p.y * f);
            }
            __stcs(reinterpret_cast<uint4*>(out + (int64_t)i * EPC), o);
        }
    }
}

// moe_kv_keep. A block owns one (lane, head) of the keys or the values and
// takes the path in batches: all sources of a batch are read into registers,
// then, after a barrier, written. Since the path ascends from >= 0, path[i] >=
// i: the rows a batch writes are sources of this batch or of earlier ones
// only, all read by then. The launch and four dependent loads (count, path, page,
// codes) bound it: 2.9 us for one lane's 8 rows, 5.5 us for 64 lanes' paths.
constexpr int KEEP_BATCH = 64;

__global__ void __launch_bounds__(KV_THREADS) kv_keep(const moe_kv_cache c, const int32_t* __restrict__ table, int width,
                                                      const int32_t* __restrict__ prefix, const int32_t* __restrict__ path,
                                                      int path_width, const int32_t* __restrict__ n_keep, int page_shift,
                                                      uint32_t* err) {
    __shared__ int64_t src[KEEP_BATCH], dst[KEEP_BATCH];
    pdl_trigger();
    pdl_wait();
    const int lane = blockIdx.x / c.n_kv_heads, h = blockIdx.x % c.n_kv_heads;
    const int n = n_keep[lane];
    if (n <= 0) return;
    const int32_t* mine = path + (int64_t)lane * path_width;
    const int32_t* pages = table + (int64_t)lane * width;
    const int64_t first = prefix[lane];
    const int64_t mask = (1 << page_shift) - 1;
    auto row_of = [&](int64_t at) -> int64_t {                 // cache row of this head, or -1
        if (at < 0 || (at >> page_shift) >= width) return -1;
        const int page = pages[at >> page_shift];
        if (page < 0 || page >= c.n_pages) return -1;
        return (((int64_t)page * c.n_kv_heads + h) << page_shift) + (at & mask);
    };
    bool ok = n <= path_width;
    for (int i = threadIdx.x; ok && i < n; i += KV_THREADS) {
        const int p = mine[i];
        ok = p >= 0 && (i == 0 || p > mine[i - 1]) && row_of(first + p) >= 0 && row_of(first + i) >= 0;
    }
    if (__syncthreads_or(!ok)) {
        if (threadIdx.x == 0) record_error(err, MOE_DEV_BAD_PAGE);
        return;
    }
    uint8_t* codes = static_cast<uint8_t*>(blockIdx.y ? c.v_codes : c.k_codes);
    uint8_t* scales = blockIdx.y ? c.v_scales : c.k_scales;
    const int D = c.head_dim, parts = D / 16;
    constexpr int MOST = KEEP_BATCH * 16 / KV_THREADS;         // 16-byte pieces of a batch, a thread (head_dim 256)
    for (int i0 = 0; i0 < n; i0 += KEEP_BATCH) {
        const int m = n - i0 < KEEP_BATCH ? n - i0 : KEEP_BATCH;
        if ((int)threadIdx.x < m) {
            src[threadIdx.x] = row_of(first + mine[i0 + threadIdx.x]);
            dst[threadIdx.x] = row_of(first + i0 + threadIdx.x);
        }
        __syncthreads();
        uint4 v[MOST];
        uint8_t sc = 0;
#pragma unroll
        for (int q = 0; q < MOST; ++q) {
            const int i = threadIdx.x + q * KV_THREADS;
            if (i < m * parts) v[q] = *reinterpret_cast<const uint4*>(codes + src[i / parts] * D + (i % parts) * 16);
        }
        if ((int)threadIdx.x < m) sc = scales[src[threadIdx.x]];
        __syncthreads();
#pragma unroll
        for (int q = 0; q < MOST; ++q) {
            const int i = threadIdx.x + q * KV_THREADS;
            if (i < m * parts) *reinterpret_cast<uint4*>(codes + dst[i / parts] * D + (i % parts) * 16) = v[q];
        }
        if ((int)threadIdx.x < m) scales[dst[threadIdx.x]] = sc;
        __syncthreads();
    }
}

int log2_of(int p) { return 31 - __builtin_clz((unsigned)p); }

moe_status cuda_status(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ECUDA; }

template <typename T>
cudaError_t launch_write(const KvSide& k, const KvSide& v, const int64_t* slots, int n, const moe_kv_cache& c, uint32_t* err,
                         cudaStream_t s) {
    const int64_t lanes = (int64_t)n * c.n_kv_heads * (c.head_dim / 16);
    const dim3 grid((unsigned)((lanes + KV_THREADS - 1) / KV_THREADS), 2);
    const int shift = log2_of(c.page_size);
    const int64_t rows = (int64_t)c.n_pages * c.page_size;
    auto go = [&](auto kern) { return moe_launch(kern, grid, dim3(KV_THREADS), 0, s, k, v, slots, n, c.n_kv_heads, shift, rows, err); };
    return c.head_dim == 64 ? go(kv_write<T, 64>) : c.head_dim == 128 ? go(kv_write<T, 128>) : go(kv_write<T, 256>);
}

template <typename T>
cudaError_t launch_read(const moe_kv_cache& c, const int32_t* table, int width, int lanes, const int32_t* starts,
                        const int32_t* cu, int n_rows, void* k_out, void* v_out, uint32_t* err, cudaStream_t s) {
    const int per_row = c.n_kv_heads * c.head_dim / (16 / (int)sizeof(T));
    int rpb = 8 * KV_THREADS / per_row;                        // about eight pieces a thread (4 and 16: slower)
    rpb = rpb < 1 ? 1 : (rpb > READ_ROWS ? READ_ROWS : rpb);
    const dim3 grid((unsigned)((n_rows + rpb - 1) / rpb), 2);
    const int shift = log2_of(c.page_size);
    // ceil(2^32 / heads): a product's upper half divides by the heads (vectors of a block: below 2^15)
    const uint32_t by_heads = (uint32_t)((((uint64_t)1 << 32) + c.n_kv_heads - 1) / c.n_kv_heads);
    auto go = [&](auto kern) {
        return moe_launch(kern, grid, dim3(KV_THREADS), 0, s, c, table, width, lanes, starts, cu, n_rows, rpb, by_heads, shift,
                          static_cast<T*>(k_out), static_cast<T*>(v_out), err);
    };
    return c.head_dim == 64 ? go(kv_read<T, 64>) : c.head_dim == 128 ? go(kv_read<T, 128>) : go(kv_read<T, 256>);
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

}  // namespace

moe_status kv_cache_status(const moe_kv_cache* c) {
    if (!c || !c->k_codes || !c->v_codes || !c->k_scales || !c->v_scales) return MOE_EINVAL;
    if (!aligned16(c->k_codes) || !aligned16(c->v_codes) || !aligned16(c->k_scales) || !aligned16(c->v_scales)) return MOE_EINVAL;
    if (c->n_pages < 1 || c->n_kv_heads < 1 || c->page_size < 1 || (c->page_size & (c->page_size - 1))) return MOE_EINVAL;
    if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) return MOE_EUNSUPPORTED;
    if (c->page_size < 16 || c->page_size > 1024 || c->n_kv_heads > 1024) return MOE_EUNSUPPORTED;
    if ((int64_t)c->n_pages * c->n_kv_heads * c->page_size >= ((int64_t)1 << 31)) return MOE_EUNSUPPORTED;
    return MOE_OK;
}

moe_status moe_kv_write(const void* k, const void* v, int dtype, int64_t k_token_stride, int64_t k_head_stride,
                        int64_t v_token_stride, int64_t v_head_stride, const int64_t* slots, int T,
                        const moe_kv_cache* cache, void* stream) {
    MOE_RANGE("moe_kv_write");
    const moe_status cs = kv_cache_status(cache);
    if (cs != MOE_OK) return cs;
    if (T < 0 || dtype < MOE_BF16 || dtype > MOE_FP32) return MOE_EINVAL;
    if (T == 0) return MOE_OK;
    if (!k || !v || !slots || !aligned16(k) || !aligned16(v)) return MOE_EINVAL;
    const int per16 = dtype == MOE_FP32 ? 4 : 8;
    if (k_token_stride % per16 || k_head_stride % per16 || v_token_stride % per16 || v_head_stride % per16) return MOE_EINVAL;
    if ((int64_t)T * cache->n_kv_heads > ((int64_t)1 << 27)) return MOE_EUNSUPPORTED;
    uint32_t* err = moe_err_word();
    if (!err) return MOE_ECUDA;
    const KvSide ks{k, k_token_stride, k_head_stride, static_cast<uint8_t*>(cache->k_codes), cache->k_scales};
    const KvSide vs{v, v_token_stride, v_head_stride, static_cast<uint8_t*>(cache->v_codes), cache->v_scales};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    moe_prof_begin(MK_KV_WRITE, s);
    const cudaError_t e = dtype == MOE_BF16   ? launch_write<__nv_bfloat16>(ks, vs, slots, T, *cache, err, s)
                          : dtype == MOE_FP16 ? launch_write<__half>(ks, vs, slots, T, *cache, err, s)
                                              : launch_write<float>(ks, vs, slots, T, *cache, err, s);
    moe_prof_end(MK_KV_WRITE, s);
    moe_count_launches(1);
    return cuda_status(e);
}

moe_status moe_kv_read(const moe_kv_cache* cache, const int32_t* page_table, int table_width, int lanes,
                       const int32_t* starts, const int32_t* cu_rows, int n_rows, int dtype, void* k_out, void* v_out,
                       void* stream) {
    MOE_RANGE("moe_kv_read");
    const moe_status cs = kv_cache_status(cache);
    if (cs != MOE_OK) return cs;
    if (n_rows < 0 || dtype < MOE_BF16 || dtype > MOE_FP32) return MOE_EINVAL;
    if (n_rows == 0) return MOE_OK;
    if (!page_table || !cu_rows || !k_out || !v_out || !aligned16(k_out) || !aligned16(v_out)) return MOE_EINVAL;
    if (lanes < 1 || table_width < 1) return MOE_EINVAL;
    if (lanes > 65536 || (int64_t)n_rows * cache->n_kv_heads > ((int64_t)1 << 27)) return MOE_EUNSUPPORTED;
    uint32_t* err = moe_err_word();
    if (!err) return MOE_ECUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    moe_prof_begin(MK_KV_READ, s);
    cudaError_t e;
    if (dtype == MOE_BF16)
        e = launch_read<__nv_bfloat16>(*cache, page_table, table_width, lanes, starts, cu_rows, n_rows, k_out, v_out, err, s);
    else if (dtype == MOE_FP16)
        e = launch_read<__half>(*cache, page_table, table_width, lanes, starts, cu_rows, n_rows, k_out, v_out, err, s);
    else
        e = launch_read<float>(*cache, page_table, table_width, lanes, starts, cu_rows, n_rows, k_out, v_out, err, s);
    moe_prof_end(MK_KV_READ, s);
    moe_count_launches(1);
    return cuda_status(e);
}

moe_status moe_kv_keep(const moe_kv_cache* cache, const int32_t* page_table, int table_width, int lanes,
                       const int32_t* prefix, const int32_t* path, int path_width, const int32_t* n_keep,
                       void* stream) {
    MOE_RANGE("moe_kv_keep");
    const moe_status cs = kv_cache_status(cache);
    if (cs != MOE_OK) return cs;
    if (lanes < 0) return MOE_EINVAL;
    if (lanes == 0) return MOE_OK;
    if (!page_table || !prefix || !path || !n_keep || table_width < 1 || path_width < 1) return MOE_EINVAL;
    if (lanes > 65536 || path_width > 4096) return MOE_EUNSUPPORTED;
    uint32_t* err = moe_err_word();
    if (!err) return MOE_ECUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    moe_prof_begin(MK_KV_KEEP, s);
    const cudaError_t e = moe_launch(kv_keep, dim3((unsigned)(lanes * cache->n_kv_heads), 2), dim3(KV_THREADS), 0, s, *cache,
                                     page_table, table_width, prefix, path, path_width, n_keep, log2_of(cache->page_size), err);
    moe_prof_end(MK_KV_KEEP, s);
    moe_count_launches(1);
    return cuda_status(e);
}
