// Queries and keys of each head: root-mean-square norm, then the rotation by the token's position, in one pass.
//
//   y = x * w / sqrt(mean(x^2) + eps)                     (without weights: y = x)
//   (a, b) -> (a cos t - b sin t, b cos t + a sin t) * magnitude,   t = position * f_i,
// for the pairs of the first 2 n values of a head: (i, i + n), or (2 i, 2 i + 1) where they are interleaved; the others stay y.
//
// The frequencies come as whole numbers of 2^-64 turns a position: the product with the position, modulo 2^64, is the
// exact fraction of a turn, so a far position is as good as a near one and no 64-bit floating point is needed.
// All else is fp32, rounded once.
//
// HBM bounds the large calls: each value is read and written once. A lane holds eight whole pairs (so that no value has to be
// fetched from a neighbour), D / 16 lanes a vector; a warp takes a token's heads in turn, with the token's sines and cosines
// computed once (through shared memory: a pair's by one lane) and kept in registers. One vector more is under way a lane, in
// registers, of which 91 a thread leave 16.5 warps an SM (issue slots 49 %, DRAM 43 % as counted, part of it in L2): 8,192 tokens of
// 32 + 8 heads of 128, bf16, with norms take 36.1 us in a graph, 4.65 TB/s (without norms 33.0), in fp32, where a lane has twice the
// bytes under way, 4,096 tokens 31.2 us, 5.4 TB/s; two tokens take 2.1 us. More bytes under way in 16 bits, through shared
// memory, were not tried.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"

namespace {

constexpr int ROT_THREADS = 128;            // 64 / 128 / 256: 8,192 tokens 35.7 / 36.1 / 45.2 us, 512 3.9 / 3.9 / 5.8
// Warps an SM, before a warp takes more than one vector. 8 / 16 / 32 / 64: 512 tokens 5.0 / 3.9 / 5.6 / 5.6 us, 8,192 36.2 / 36.1 /
// 36.1 / 46.5, 833 of 25 heads of 64 2.9 / 3.3 / 3.3 / 3.3.
constexpr int WARPS = 16;

struct RotArgs {
    const void* q;
    const void* k;
    void* q_out;
    void* k_out;
    int64_t q_token, q_head, k_token, k_head, qo_token, qo_head, ko_token, ko_head;      // strides, elements
    int n_tokens, n_q, n_k;                 // heads
    const int32_t* positions;
    const int64_t* turns;
    int pairs;
    const float* q_weight;
    const float* k_weight;
    float eps, magnitude;
    int per_warp;                           // vectors that a warp's lanes take one after the other
    int groups;                             // warps to a token
};

template <typename T> struct Eight;         // eight values: as they lie in memory, and as fp32
template <> struct Eight<float> {
    struct Raw { float4 a, b; };
    static MOE_DEV Raw load(const void* p) { return Raw{static_cast<const float4*>(p)[0], static_cast<const float4*>(p)[1]}; }
    static MOE_DEV void expand(const Raw& r, float* x) {
        x[0] = r.a.x; x[1] = r.a.y; x[2] = r.a.z; x[3] = r.a.w; x[4] = r.b.x; x[5] = r.b.y; x[6] = r.b.z; x[7] = r.b.w;
    }
    static MOE_DEV void store(void* p, const float* x) {
        static_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
        static_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
    }
};
template <> struct Eight<__nv_bfloat16> {
    typedef uint4 Raw;
    static MOE_DEV Raw load(const void* p) { return *static_cast<const uint4*>(p); }
    static MOE_DEV void expand(const Raw& v, float* x) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
    static MOE_DEV void store(void* p, const float* x) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
        *static_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    }
};
template <> struct Eight<__half> {
    typedef uint4 Raw;
    static MOE_DEV Raw load(const void* p) { return *static_cast<const uint4*>(p); }
    static MOE_DEV void expand(const Raw& v, float* x) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
            x[2 * i] = f.x;
            x[2 * i + 1] = f.y;
        }
    }
    static MOE_DEV void store(void* p, const float* x) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __half2 h = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
        *static_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    }
};

template <typename T, int D, bool PAIRED>   // PAIRED: pairs side by side
__global__ void __launch_bounds__(ROT_THREADS) qk_rotate(const __grid_constant__ RotArgs a) {
    constexpr int LPV = D / 16, AT_ONCE = 32 / LPV;            // lanes to a vector, vectors that a warp holds
    __shared__ __align__(16) float2 turned[ROT_THREADS / 32][D / 2];
    pdl_trigger();
    const int lane = threadIdx.x & 31, part = lane % LPV, sub = lane / LPV;
    const int64_t warp = (int64_t)blockIdx.x * (ROT_THREADS / 32) + (threadIdx.x >> 5);
    pdl_wait();
    if (warp >= (int64_t)a.n_tokens * a.groups) return;
    const int t = (int)(warp / a.groups), group = (int)(warp - (int64_t)t * a.groups);
    // This lane's eight pairs, or sixteen of the values that are not turned: two pieces of eight, the first members of the
    // pairs and the second ones, or what lies side by side.
    const bool on = part < a.pairs / 8;
    const int at0 = PAIRED ? part * 16 : on ? part * 8 : part * 16;        // (half layout: 2 pairs + 16 (part - pairs / 8))
    const int at1 = PAIRED || !on ? at0 + 8 : a.pairs + at0;
    const int heads = a.n_q + a.n_k;
    const T* q = static_cast<const T*>(a.q) + t * a.q_token;
    const T* k = static_cast<const T*>(a.k) + t * a.k_token;
    T* qo = static_cast<T*>(a.q_out) + t * a.qo_token;
    T* ko = static_cast<T*>(a.k_out) + t * a.ko_token;
    const int h0 = group * a.per_warp * AT_ONCE + sub;
    typename Eight<T>::Raw next[2];                            // the next vector's values, under way (the first's beside the angles)
    auto load = [&](int i) {
        const int h = h0 + i * AT_ONCE;
        if (i >= a.per_warp || h >= heads) return;
        const T* from = h < a.n_q ? q + h * a.q_head : k + (h - a.n_q) * a.k_head;
        next[0] = Eight<T>::load(from + at0);
        next[1] = Eight<T>::load(from + at1);
    };
    load(0);
    // the token's cosines and sines, each once
    float2* mine = turned[threadIdx.x >> 5];
    const unsigned long long pos = a.pairs ? (unsigned long long)(long long)a.positions[t] : 0ull;
#pragma unroll 1
    for (int i = lane; i < a.pairs; i += 32) {
        // a signed fraction of half a turn: [-1, 1)
        const int turn = (int)((pos * (unsigned long long)a.turns[i]) >> 32);
        float sn, cs;
        sincospif((float)turn * 0x1p-31f, &sn, &cs);
        mine[i] = make_float2(cs * a.magnitude, sn * a.magnitude);
    }
    __syncwarp();
    float c[8], s[8];
    if (on) {
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            const float4 two = *reinterpret_cast<const float4*>(mine + part * 8 + i);
            c[i] = two.x; s[i] = two.y;
            c[i + 1] = two.z; s[i + 1] = two.w;
        }
    }
    int have = -1;                                             // whose weights w holds: 0 queries', 1 keys'
    float w[16];
#pragma unroll 1
    for (int i = 0; i < a.per_warp; ++i) {
        const int h = h0 + i * AT_ONCE, key = h >= a.n_q;
        float y[16];
        Eight<T>::expand(next[0], y);
        Eight<T>::expand(next[1], y + 8);
        load(i + 1);
        if (h >= heads) continue;                              // (whole vectors' lanes; nothing below needs the others)
        const float* weight = key ? a.k_weight : a.q_weight;
        if (weight) {
            if (key != have) {
                Eight<float>::expand(Eight<float>::load(weight + at0), w);
                Eight<float>::expand(Eight<float>::load(weight + at1), w + 8);
                have = key;
            }
            float even = 0.0f, odd = 0.0f;
#pragma unroll
            for (int e = 0; e < 16; e += 2) {
                even = fmaf(y[e], y[e], even);
                odd = fmaf(y[e + 1], y[e + 1], odd);
            }
            float sum = even + odd;
            constexpr uint32_t GROUP = (1u << LPV) - 1u;
#pragma unroll
            for (int o = LPV / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(GROUP << (lane - part), sum, o);
            const float r = rsqrtf(sum * (1.0f / D) + a.eps);
#pragma unroll
            for (int e = 0; e < 16; ++e) y[e] *= r * w[e];
        }
        if (on) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int m = PAIRED ? 2 * e : e, n = PAIRED ? 2 * e + 1 : e + 8;
                const float first = y[m], second = y[n];
                y[m] = first * c[e] - second * s[e];
                y[n] = second * c[e] + first * s[e];
            }
        }
        T* to = key ? ko + (h - a.n_q) * a.ko_head : qo + h * a.qo_head;
        Eight<T>::store(to + at0, y);
        Eight<T>::store(to + at1, y + 8);
    }
}

template <typename T, int D>
cudaError_t launch(RotArgs a, bool interleaved, cudaStream_t s) {
    constexpr int AT_ONCE = 32 / (D / 16);
    const int vectors = (a.n_q + a.n_k + AT_ONCE - 1) / AT_ONCE;        // a token's, in warps' loads
    // as many vectors a warp as leave WARPS warps an SM
    const int64_t warps = (int64_t)moe_sm_count() * WARPS;
    const int64_t per = (int64_t)a.n_tokens * vectors / warps;
    a.per_warp = (int)(per < 1 ? 1 : per > vectors ? vectors : per);
    a.groups = (vectors + a.per_warp - 1) / a.per_warp;
    const int64_t total = (int64_t)a.n_tokens * a.groups;
    const dim3 grid((unsigned)((total + ROT_THREADS / 32 - 1) / (ROT_THREADS / 32)));
    return interleaved ? moe_launch(qk_rotate<T, D, true>, grid, dim3(ROT_THREADS), 0, s, a)
                       : moe_launch(qk_rotate<T, D, false>, grid, dim3(ROT_THREADS), 0, s, a);
}
template <typename T>
cudaError_t launch_dim(const RotArgs& a, int D, bool interleaved, cudaStream_t s) {
    return D == 64 ? launch<T, 64>(a, interleaved, s) : D == 128 ? launch<T, 128>(a, interleaved, s) : launch<T, 256>(a, interleaved, s);
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

}  // namespace

moe_status moe_qk_rotate(const void* q, const void* k, int dtype, const int64_t* strides, int n_tokens, int n_q_heads, int n_k_heads,
                         int head_dim, const int32_t* positions, const int64_t* turns, int n_pairs, int interleaved, float magnitude,
                         const float* q_weight, const float* k_weight, float eps, void* q_out, void* k_out, void* stream) {
    MOE_RANGE("moe_qk_rotate");
    if (n_tokens < 0 || n_q_heads < 0 || n_k_heads < 0 || n_q_heads + n_k_heads < 1 || dtype < MOE_BF16 || dtype > MOE_FP32 || !strides) return MOE_EINVAL;
    if (head_dim != 64 && head_dim != 128 && head_dim != 256) return MOE_EUNSUPPORTED;
    if (n_pairs < 0 || 2 * (int64_t)n_pairs > head_dim || !(eps >= 0.0f) || eps > 3.0e38f || !(magnitude >= -3.0e38f && magnitude <= 3.0e38f)) return MOE_EINVAL;
    if (n_pairs % 8 || n_q_heads > 65536 || n_k_heads > 65536) return MOE_EUNSUPPORTED;
    if (n_tokens == 0) return MOE_OK;
    if ((n_q_heads && (!q || !q_out)) || (n_k_heads && (!k || !k_out)) || (n_pairs && (!positions || !turns))) return MOE_EINVAL;
    if (!aligned16(q) || !aligned16(k) || !aligned16(q_out) || !aligned16(k_out) || !aligned16(q_weight) || !aligned16(k_weight)) return MOE_EINVAL;
    const int per16 = dtype == MOE_FP32 ? 4 : 8;
    for (int i = 0; i < 8; ++i)
        if (strides[i] % per16) return MOE_EINVAL;
    if ((int64_t)n_tokens * (n_q_heads + n_k_heads) > ((int64_t)1 << 31)) return MOE_EUNSUPPORTED;
    RotArgs a{};
    a.q = q; a.k = k; a.q_out = q_out; a.k_out = k_out;
    a.q_token = strides[0]; a.q_head = strides[1]; a.k_token = strides[2]; a.k_head = strides[3];
    a.qo_token = strides[4]; a.qo_head = strides[5]; a.ko_token = strides[6]; a.ko_head = strides[7];
    a.n_tokens = n_tokens; a.n_q = n_q_heads; a.n_k = n_k_heads;
    a.positions = positions; a.turns = turns; a.pairs = n_pairs;
    a.q_weight = q_weight; a.k_weight = k_weight; a.eps = eps; a.magnitude = magnitude;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    moe_prof_begin(MK_QK_ROTATE, s);
    const cudaError_t e = dtype == MOE_BF16   ? launch_dim<__nv_bfloat16>(a, head_dim, interleaved != 0, s)
                          : dtype == MOE_FP16 ? launch_dim<__half>(a, head_dim, interleaved != 0, s)
                                              : launch_dim<float>(a, head_dim, interleaved != 0, s);
    moe_prof_end(MK_QK_ROTATE, s);
    moe_count_launches(1);
    return e == cudaSuccess ? MOE_OK : MOE_ECUDA;
}
