// Attention of drafted tokens over the paged 8-bit key/value cache.
//
// For the rows r = (node, query head) of one kv head and the cache rows j:
//   s[r,j] = scale log2(e) q_r . k_j        (k_j = codes * 2^ek_j)
//   out[r] = sum_j 2^s[r,j] v_j / sum_j 2^s[r,j]      (v_j = codes * 2^ev_j)
// over the j that r sees. Both products run on the tensor cores on the codes
// as they lie in the cache (tcgen05 kind::f8f6f4, fp32 accumulators in TMEM):
// no byte of the cache is converted or scaled outside the MMA, so TMA moves it
// from HBM to the operand buffers untouched.
//   - The other operand is split in two 8-bit parts. A bf16 query has 8
//     significant bits and e4m3 has 4: with its row scaled by a power of two to
//     128 <= max|q| < 256, hi = e4m3(q), lo = e4m3(q - hi) hold it exactly down
//     to 2^-9 of the row's maximum and within 2^-17 of the maximum below.
//   - A probability p is hi + lo too, with 8 significant bits as bf16 would
//     have: hi = e5m2(p), which is the upper byte of p in fp16 (rounded by an
//     integer add), lo = e4m3 of the rest.
//   - The scale of a key row multiplies its column of scores; the scale of a
//     value row is added to the exponent: s' = s + ev_j, p = 2^(s' - m + 8), so
//     values of any size keep their precision; the sum of weights gets p 2^-ev_j.
//   - m is a running reference, not each tile's maximum: it is the maximum of s'
//     when it is set, and stays until a score passes it by 2^3.5 (p would pass what lo can
//     hold); then it is set again and what has been added up is scaled down. Most tiles
//     so need no maximum at all: one compare, a vote, no reduction over the rows.
//     Weights below 2^-25 of the largest are dropped, the rest keep at least the 3 bits of
//     hi, which is unbiased.
//
// Orientation: cache rows are the MMA's M (128), tree rows its N (2R for S, R for
// O: hi and lo of the queries side by side; those of the probabilities
// accumulate), so a single token costs N = 16 and a wide tree 64, and nothing
// is padded to 128:
//   S^T[128 rows, 2R] = K[128, D] Q^T           O^T[D, R] += V^T[D, 128] P^T[128, R]
// A thread of a softmax group is a cache row: the rows' scales are its own
// registers, the sums of weights are kept per thread and added up once at the end.
//
// Two softmax groups of four warps. Up to R tree rows (R = 16, 32, 64; 32 at
// head_dim 256) they take the tiles of 128 cache rows in turn, each with an O of
// its own; above, PAIR, both take every tile, each for R of 2R tree rows, so that the
// cache is read once for twice the rows.
//
// Work: the (lane, kv head, tile of tree rows) units, each a run of cache
// tiles, are laid end to end and cut into equal parts, one per CTA. A unit that one
// CTA does whole is written at once; the others leave their parts (output, maximum, sum)
// in the workspace and tree_attention_join adds them up in order.
//
// Roles (512 threads):
//   warps 0-3, 4-7   softmax groups
//   warps 8-11       the next unit's queries (split and laid out), a finished unit's output
//   warp 12          TMA, one copy per page
//   warp 13          MMA issue, TMEM
//   warp 14          the rows' scales
// Waits are bounded as in the expert GEMMs.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <mutex>

#include <cudaTypedefs.h>

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
    float scale_log2;                            // scale * log2(e)
    __nv_bfloat16* out;
    float* lse;
    uint8_t* ws;
    uint32_t* err;
    uint64_t wait_ns;
};

struct AttnMaps {
    CUtensorMap k, v;                            // (head_dim, rows) bytes, box min(head_dim, 128) x min(page, 128) rows
};

constexpr int TILE = 128;                        // cache rows a tile
constexpr int ATTN_THREADS = 512;
constexpr int LANE_CACHE = 512;                  // lanes whose facts are kept in shared memory

// What the join needs, at the start of the workspace: the cut, and for each CTA the unit that its part begins in.
struct JoinHead {
    int64_t total;                               // tiles in all
    int32_t parts;                               // CTAs with work
    int32_t pad;
};
struct JoinUnit {
    int64_t first, end;                          // the unit's tiles in the whole run
    int32_t node0, rows, head, row0;             // first node of the lane, tree rows of the unit, kv head, first row in the lane
};
constexpr size_t JOIN_UNITS = 256;               // byte offset of JoinUnit[CTAs]

__host__ __device__ constexpr size_t part_floats(int RU, int D) { return (size_t)RU * (D + 2); }
__host__ __device__ inline size_t parts_offset(int ctas) { return (JOIN_UNITS + (size_t)ctas * sizeof(JoinUnit) + 255) / 256 * 256; }

template <int D, int R, bool PAIR>
struct Cfg {
    static constexpr int RU = PAIR ? 2 * R : R;               // tree rows of a unit
    static constexpr int ROWB = D >= 128 ? 128 : 64;          // bytes of an operand row: one swizzle atom
    static constexpr int PANELS = D / ROWB;
    static constexpr int PANEL = TILE * ROWB;
    static constexpr int SLOT = TILE * D;
    static constexpr int QROWS = 2 * RU;                      // hi and lo of each half's rows
    static constexpr int QBUFS = PAIR ? 1 : 2;                // PAIR: its 2R rows leave room for one
    static constexpr int QBUF = QROWS * D;
    static constexpr int PBUF = 2 * TILE * R;
    // ring of key and value tiles: what fits, 8 tiles of 16 KB at most (more measured no faster)
    static constexpr int NS = D == 64 ? 12 : D == 128 ? 8 : R == 16 ? 5 : PAIR ? 5 : 5;
    static constexpr int NSC = 4;                             // ring of scale tiles (128 key bytes, 128 value bytes)
    static constexpr int MB = D == 256 ? 2 : 1;               // M blocks of O^T
    static constexpr int OFF_RING = 0;
    static constexpr int OFF_P = OFF_RING + NS * SLOT;
    static constexpr int OFF_Q = OFF_P + 2 * PBUF;
    static constexpr int OFF_SC = OFF_Q + QBUFS * QBUF;
    static constexpr int OFF_F = OFF_SC + NSC * 256;          // floats from here
    static constexpr int F_O = 0;                             // [2 groups][R] 8 - m, as added to s'
    static constexpr int F_AL = F_O + 2 * R;                  // [2][R] scale-down of what has been added up
    static constexpr int F_WMAX = F_AL + 2 * R;               // [2][4 warps][R]
    static constexpr int F_QF = F_WMAX + 8 * R;               // [4][RU] 2^-a of the queries' rows
    static constexpr int F_L = F_QF + 4 * RU;                 // [2][4][R] sums at a part's end
    static constexpr int F_M = F_L + 8 * R;                   // [2][R] their references
    static constexpr int F_ST = F_M + 2 * R;                  // [4 warps][2][RU] factors of the output
    static constexpr int F_END = F_ST + 8 * RU;
    static constexpr int OFF_LANE = OFF_F + F_END * 4;        // int n0, n, len [LANE_CACHE]
    static constexpr int OFF_SCAN = OFF_LANE + 3 * LANE_CACHE * 4;
    static constexpr int OFF_BAR = OFF_SCAN + 32 * 8 + 64;
    // full, empty [NS]; scale full, empty [NSC]; sfull, pfull, pfree, vote, maxima, qfull, qfree, ofull, ofree [2]; lfull, lfree, drain
    static constexpr int N_BARS = 2 * NS + 2 * NSC + 18 + 3;
    static constexpr int OFF_MISC = (OFF_BAR + N_BARS * 8 + 15) / 16 * 16;     // tmem slot, abort flag, votes [2][2][4]
    static constexpr int SMEM = OFF_MISC + 16 + 64 + 1024;
    static constexpr int TMEM_O = 4 * R;                      // after S of both groups: O [group][unit parity][MB][R]
    static constexpr int TMEM_USED = 4 * R + 4 * R * MB;
    static constexpr int TMEM_COLS = TMEM_USED <= 128 ? 128 : TMEM_USED <= 256 ? 256 : 512;
    static_assert(TMEM_USED <= 512 && SMEM <= 227 * 1024, "TMEM, shared memory");
    static_assert(OFF_F % 16 == 0 && OFF_SCAN % 8 == 0 && OFF_BAR % 8 == 0 && OFF_MISC % 16 == 0, "alignment");
    static_assert(R == 16 || R == 32 || R == 64, "R");
};

constexpr float P_EXP = 8.0f;                    // p = 2^8 at the reference
constexpr float P_EXP_MAX = 11.5f;               // above it, lo = e4m3(p - hi) could pass 448

// ------------------------------------------------------------------ small device pieces

MOE_DEV float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
typedef unsigned long long f32x2;
MOE_DEV f32x2 pack2(float a, float b) {
    f32x2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
MOE_DEV float2 unpack2(f32x2 v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
MOE_DEV f32x2 add2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
MOE_DEV f32x2 mul2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
MOE_DEV f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
    f32x2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
// Maximum over the warp, in every lane (NaN inputs are passed over).
MOE_DEV float warp_max(float v) {
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}

MOE_DEV void tc_mma_f8(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}"
        ::"r"(d_tmem), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// kind::f8f6f4, e4m3 x e4m3 (or x e5m2) -> fp32; a_mn, b_mn: whether A and B lie with M and N (instead of K) contiguous.
__host__ __device__ constexpr uint32_t idesc_f8(int m, int n, int a_mn, int b_mn, int b_e5m2) {
    return (1u << 4) | ((uint32_t)b_e5m2 << 10) | ((uint32_t)a_mn << 15) | ((uint32_t)b_mn << 16) | ((uint32_t)(n >> 3) << 17) |
           ((uint32_t)(m >> 4) << 24);
}

// One lane of the (converged) warp.
MOE_DEV bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

MOE_DEV void tc_ld_x8(uint32_t taddr, uint32_t (&r)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
}

// Moves registers between the warpgroups of a block of 512 threads launched with 128 each: 2 x 184 + 80 + 64 = 4 x 128.
template <int N> MOE_DEV void regs_up() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N> MOE_DEV void regs_down() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

// Shared-memory matrix descriptor without its address: swizzle 2 = 128 B, 4 = 64 B, 6 = 32 B, 0 = none; `group` =
// bytes from one group of eight rows (of the strided axis) to the next. Every operand here is one
// atom wide on its contiguous axis, so the group stride is the only one in use: both offset fields hold it.
__host__ __device__ constexpr uint64_t desc_base(int swizzle, int group) {
    return ((uint64_t)(group >> 4) << 16) | ((uint64_t)(group >> 4) << 32) | ((uint64_t)1 << 46) | ((uint64_t)swizzle << 61);
}
MOE_DEV uint64_t desc_at(uint64_t base, uint32_t saddr) { return base + (uint64_t)(saddr >> 4); }   // below 256 KB: no carry

// A lane's facts. A lane that does not fit (see the header) has no rows, and its outputs become zeros.
struct Lane {
    int n0, n, len;
};
MOE_DEV Lane lane_facts(const AttnArgs& a, int b, bool* bad) {
    Lane l;
    l.n0 = a.cu[b];
    l.n = a.cu[b + 1] - l.n0;
    l.len = a.kv_len[b];
    *bad = false;
    if (l.n0 < 0 || l.n < 0 || l.n > a.n_nodes - l.n0) {      // row counts that would lead out of q and out
        *bad = true;
        l.n0 = l.n = l.len = 0;
    } else if (l.n > 0 && (l.n > a.max_nodes || l.len < l.n ||
                           (((int64_t)l.len + (1 << a.page_shift) - 1) >> a.page_shift) > a.width)) {
        *bad = true;
        l.len = 0;
    }
    return l;
}

// One CTA's way through its part of the run: the unit it is in and the tile within it.
template <int R>                                 // R: tree rows of a unit
struct Walk {
    int b, h, rt, t, tiles, nrt;
    Lane l;

    MOE_DEV void enter(const AttnArgs& a, const int* facts) {
        if (b < LANE_CACHE) {
            l.n0 = facts[b];
            l.n = facts[LANE_CACHE + b];
            l.len = facts[2 * LANE_CACHE + b];
        } else {
            bool bad;
            l = lane_facts(a, b, &bad);
        }
        tiles = l.len > 0 ? (l.len + TILE - 1) / TILE : 1;
        nrt = l.n > 0 ? (l.n * a.group + R - 1) / R : 1;
    }
    MOE_DEV void start(const AttnArgs& a, const int* facts, int lane, int64_t offset) {
        b = lane;
        enter(a, facts);
        const int u = (int)(offset / tiles);
        t = (int)(offset - (int64_t)u * tiles);
        h = u / nrt;
        rt = u - h * nrt;
    }
    // past n tiles, which do not lead out of the unit; more: whether tiles are left after them
    MOE_DEV void advance(const AttnArgs& a, const int* facts, int n, bool more) {
        t += n;
        if (t < tiles || !more) return;
        t = 0;
        if (++rt < nrt) return;
        rt = 0;
        if (++h < a.c.n_kv_heads) return;
        h = 0;
        do {
            ++b;
            enter(a, facts);
        } while (l.n == 0 && b + 1 < a.lanes);
    }
    MOE_DEV int rows(const AttnArgs& a) const {               // tree rows of this unit
        const int left = l.n * a.group - rt * R;
        return left < R ? left : R;
    }
};

template <int D, int R, bool PAIR>
__global__ void __launch_bounds__(ATTN_THREADS, 1) tree_attention(const __grid_constant__ AttnMaps maps, const AttnArgs a) {
    using C = Cfg<D, R, PAIR>;
    constexpr int RU = C::RU;
    constexpr int NS = C::NS, NSC = C::NSC;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
    uint64_t* empty = full + NS;
    uint64_t* scfull = empty + NS;
    uint64_t* scempty = scfull + NSC;
    uint64_t* sfull = scempty + NSC;             // [2 groups] S of a tile is ready
    uint64_t* pfull = sfull + 2;                 // [2] P is written (and S has been read)
    uint64_t* pfree = pfull + 2;                 // [2] P has been read (and added to O)
    uint64_t* vote = pfree + 2;                  // [2] the group's four warps have compared a tile's scores
    uint64_t* maxima = vote + 2;                 // [2] ... have written a tile's maxima
    uint64_t* qfull = maxima + 2;                // [QBUFS]
    uint64_t* qfree = qfull + 2;
    uint64_t* ofull = qfree + 2;                 // [2] O of a part is complete
    uint64_t* ofree = ofull + 2;                 // [2] ... and has been read
    uint64_t* lfull = ofree + 2;                 // the sums of a part are written
    uint64_t* lfree = lfull + 1;                 // ... and read
    uint64_t* drain = lfree + 1;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 4);
    volatile int* votes = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 16);       // [2 groups][2][4 warps]
    float* F = reinterpret_cast<float*>(smem + C::OFF_F);
    int* facts = reinterpret_cast<int*>(smem + C::OFF_LANE);
    unsigned long long* scratch = reinterpret_cast<unsigned long long*>(smem + C::OFF_SCAN);
    int64_t* begin_off = reinterpret_cast<int64_t*>(smem + C::OFF_SCAN + 256);       // where this CTA's part begins
    int* begin_lane = reinterpret_cast<int*>(smem + C::OFF_SCAN + 264);

    const int tid = threadIdx.x, warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0), lane = tid & 31;
    const int H = a.c.n_kv_heads, G = a.group;
    pdl_trigger();
    if (tid == 0) {
        for (int s = 0; s < NS; ++s) { mbar_init(&full[s], 1); mbar_init(&empty[s], 1); }
        for (int s = 0; s < NSC; ++s) { mbar_init(&scfull[s], 1); mbar_init(&scempty[s], PAIR ? 8 : 4); }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&sfull[s], 1); mbar_init(&pfull[s], 4); mbar_init(&pfree[s], 1); mbar_init(&vote[s], 4); mbar_init(&maxima[s], 4);
            mbar_init(&qfull[s], 4); mbar_init(&qfree[s], 1); mbar_init(&ofull[s], 1); mbar_init(&ofree[s], 4);
        }
        mbar_init(lfull, 8); mbar_init(lfree, 4); mbar_init(drain, 1);
        *abort_flag = 0;
        *begin_lane = 0;
        *begin_off = 0;
        fence_barrier_init();
        prefetch_tmap(&maps.k);
        prefetch_tmap(&maps.v);
    }
    if (warp == 13) { tmem_alloc(tmem_slot, C::TMEM_COLS); tmem_relinquish(); }
    pdl_wait();

    // ---------------------------------------------------------------- the cut
    auto work_of = [&](const Lane& l) -> unsigned long long {
        if (l.n == 0) return 0ull;
        const unsigned long long tiles = l.len > 0 ? (l.len + TILE - 1) / TILE : 1;
        return (unsigned long long)H * ((l.n * G + RU - 1) / RU) * tiles;
    };
    unsigned long long total = 0, mine = 0, incl = 0;
    for (int b0 = 0; b0 < a.lanes; b0 += ATTN_THREADS) {
        const int b = b0 + tid;
        Lane l{0, 0, 0};
        if (b < a.lanes) {
            bool bad;
            l = lane_facts(a, b, &bad);
            if (bad && blockIdx.x == 0) record_error(a.err, MOE_DEV_BAD_PAGE);
            if (b < LANE_CACHE) {
                facts[b] = l.n0;
                facts[LANE_CACHE + b] = l.n;
                facts[2 * LANE_CACHE + b] = l.len;
            }
        }
        mine = work_of(l);
        unsigned long long sum;
        incl = block_inclusive_scan_u64(mine, scratch, &sum) + total;
        total += sum;
    }
    const int parts = total < gridDim.x ? (int)total : (int)gridDim.x;
    const bool active = (int)blockIdx.x < parts;
    const int64_t first = active ? (int64_t)(total * blockIdx.x / parts) : 0;
    const int64_t count = active ? (int64_t)(total * (blockIdx.x + 1) / parts) - first : 0;
    if (active) {
        if (a.lanes <= ATTN_THREADS) {
            const unsigned long long excl = incl - mine;
            if ((unsigned long long)first >= excl && (unsigned long long)first < incl) {
                *begin_lane = tid;
                *begin_off = first - (int64_t)excl;
            }
        } else {
            unsigned long long before = 0;
            for (int b0 = 0; b0 < a.lanes; b0 += ATTN_THREADS) {
                const int b = b0 + tid;
                bool bad;
                mine = b < a.lanes ? work_of(lane_facts(a, b, &bad)) : 0ull;
                unsigned long long sum;
                incl = block_inclusive_scan_u64(mine, scratch, &sum) + before;
                const unsigned long long excl = incl - mine;
                if ((unsigned long long)first >= excl && (unsigned long long)first < incl) {
                    *begin_lane = b;
                    *begin_off = first - (int64_t)excl;
                }
                before += sum;
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    Walk<RU> w;
    w.start(a, facts, active ? *begin_lane : 0, active ? *begin_off : 0);
    if (tid == 0) {
        if (blockIdx.x == 0) *reinterpret_cast<JoinHead*>(a.ws) = JoinHead{(int64_t)total, parts, 0};
        if (active)
            reinterpret_cast<JoinUnit*>(a.ws + JOIN_UNITS)[blockIdx.x] =
                JoinUnit{first - w.t, first - w.t + w.tiles, w.l.n0, w.rows(a), w.h, w.rt * RU};
    }
    int64_t left = count;
    uint32_t issued = 0;                             // ring fills, by the producer

    if (warp < 8) {
        // ------------------------------------------------------------ softmax
        if constexpr (R == 64) regs_up<184>();
        const int g = warp >> 2, wl = warp & 3;      // group, warp in it
        const int j = tid & 127;                     // this thread's row of the tile
        const uint32_t trow = tmem + ((uint32_t)(wl * 32) << 16) + g * 2 * R;
        float* off = F + C::F_O + g * R;
        float* alpha = F + C::F_AL + g * R;
        float* wmax = F + C::F_WMAX + g * 4 * R;
        uint32_t i = 0, k = 0, sets = 0, polls = 0, piece = 0;       // tile of the CTA; of this group; references set; votes; part
        constexpr int RL = R > 32 ? 2 : 1;           // tree rows a lane keeps the reference of: lane, lane + 32
        bool ok = true;
        while (left > 0 && ok) {
            const int nt = left < w.tiles - w.t ? (int)left : w.tiles - w.t;
            f32x2 l2[R / 2];
            float M[RL];
#pragma unroll
            for (int r = 0; r < R / 2; ++r) l2[r] = 0ull;
#pragma unroll
            for (int r = 0; r < RL; ++r) M[r] = -INFINITY;
            const float* qf = F + C::F_QF + (piece & 3) * RU + (PAIR ? g * R : 0);
            const int prefix = w.l.len - w.l.n;
            const int row0 = w.rt * RU + (PAIR ? g * R : 0);         // this group's tree rows in the lane
            uint32_t ev_most = 0;                    // largest value scale seen so far
            bool set = true;                         // the reference is to be set (a part's first tile)
            for (int t = w.t; t < w.t + nt; ++t, ++i) {
                if (!PAIR && (int)(i & 1) != g) continue;
                const int j0 = t * TILE;
                const int valid = w.l.len - j0;      // rows of the tile that exist (can be <= 0 or > 128)
                const bool masked = j0 + TILE > prefix;
                // what this row is to each tree row
                uint64_t sees = ~0ull;
                if (masked) {
                    const int n = j0 + j - prefix;
                    if (j >= valid) {
                        sees = 0ull;
                    } else if (n >= 0) {
                        sees = 0ull;
                        const int end = w.l.n * G < row0 + R ? w.l.n * G : row0 + R;
                        for (int t1 = row0 / G; t1 * G < end; ++t1) {
                            const bool see = a.mask ? (a.mask[(int64_t)(w.l.n0 + t1) * a.mask_words + (n >> 5)] >> (n & 31)) & 1
                                                    : n <= t1;
                            if (!see) continue;
                            int lo = t1 * G - row0, hi = lo + G;
                            lo = lo < 0 ? 0 : lo;
                            hi = hi > R ? R : hi;
                            sees |= (hi == 64 ? ~0ull : (1ull << hi) - 1ull) & ~((1ull << lo) - 1ull);
                        }
                    }
                }
                const int sc = (int)(i % NSC);
                if (!warp_wait(&scfull[sc], (i / NSC) & 1, abort_flag, a.wait_ns)) { ok = false; break; }
                const uint8_t* scales = smem + C::OFF_SC + sc * 256;
                const uint32_t ks = scales[j], vs = scales[TILE + j];
                const uint32_t four = *reinterpret_cast<const uint32_t*>(scales + TILE + lane * 4);
                __syncwarp();
                if (lane == 0) mbar_arrive(&scempty[sc]);
                const uint32_t most = __vmaxu4(four, four >> 16), least = __vminu4(four, __byte_perm(four, 0, 0x1032));
                ev_most = max(ev_most, __reduce_max_sync(0xFFFFFFFFu, max(most & 255u, (most >> 8) & 255u)));
                // Value scales more than 2^104 apart: p could underflow in a row that matters to the sum of
                // weights, p 2^-ev; its weight then gets an exponential of its own.
                const bool wide = ev_most > __reduce_min_sync(0xFFFFFFFFu, min(least & 255u, (least >> 8) & 255u)) + 104u;
                const float cj = a.scale_log2 * e8m0_to_float(ks);
                const int evi = vs == 255u ? 0 : (int)vs - 127;
                const float ev = vs == 255u ? __uint_as_float(0x7FC00000u) : (float)evi;
                const f32x2 cj2 = pack2(cj, cj), ev2 = pack2(ev, ev);
                if (!warp_wait(&sfull[g], k & 1, abort_flag, a.wait_ns)) { ok = false; break; }
                tc_fence_after();
                // y = s' (+ off: the exponent of p); rows not seen are -inf
                f32x2 y[R / 2];
                auto scores = [&](bool with_off) {
#pragma unroll
                    for (int c0 = 0; c0 < R; c0 += 8) {
                        uint32_t hi[8], lo[8];
                        tc_ld_x8(trow + c0, hi);
                        tc_ld_x8(trow + R + c0, lo);
                        tc_wait_ld();
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const f32x2 f = *reinterpret_cast<const f32x2*>(qf + c0 + 2 * q);
                            const f32x2 o = *reinterpret_cast<const f32x2*>(off + c0 + 2 * q);
                            const f32x2 s = add2(pack2(__uint_as_float(hi[2 * q]), __uint_as_float(hi[2 * q + 1])),
                                                 pack2(__uint_as_float(lo[2 * q]), __uint_as_float(lo[2 * q + 1])));
                            y[c0 / 2 + q] = fma2(mul2(s, f), cj2, with_off ? add2(ev2, o) : ev2);
                        }
                    }
                    if (masked) {
#pragma unroll
                        for (int q = 0; q < R / 2; ++q) {
                            const float2 s = unpack2(y[q]);
                            y[q] = pack2((sees >> (2 * q)) & 1 ? s.x : -INFINITY, (sees >> (2 * q + 1)) & 1 ? s.y : -INFINITY);
                        }
                    }
                };
                auto set_reference = [&]() -> bool {
                    // the tile's maximum of s' in every tree row, over the group's 128 threads
                    float mine[RL];
#pragma unroll
                    for (int r = 0; r < RL; ++r) mine[r] = -INFINITY;
#pragma unroll
                    for (int q = 0; q < R / 2; ++q) {
                        const float2 s = unpack2(y[q]);
                        const float m0 = warp_max(s.x), m1 = warp_max(s.y);
                        if (lane == ((2 * q) & 31)) mine[q / 16] = m0;
                        if (lane == ((2 * q + 1) & 31)) mine[q / 16] = m1;
                    }
#pragma unroll
                    for (int r = 0; r < RL; ++r)
                        if (R >= 32 || lane < R) wmax[wl * R + r * 32 + lane] = mine[r];
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&maxima[g]);
                    if (!warp_wait(&maxima[g], sets & 1, abort_flag, a.wait_ns)) return false;
                    ++sets;
                    // every warp writes the same factors
#pragma unroll
                    for (int r = 0; r < RL; ++r) {
                        if (R < 32 && lane >= R) break;
                        const int row = r * 32 + lane;
                        const float m = fmaxf(fmaxf(wmax[row], wmax[R + row]), fmaxf(wmax[2 * R + row], wmax[3 * R + row]));
                        const float Mn = fmaxf(M[r], m);
                        // a row that has seen nothing: the first score it sees passes any limit
                        off[row] = Mn == -INFINITY ? 1e30f : P_EXP - Mn;
                        alpha[row] = M[r] == -INFINITY ? 0.0f : ex2(M[r] - Mn);
                        M[r] = Mn;
                    }
                    __syncwarp();
#pragma unroll
                    for (int q = 0; q < R / 2; ++q) {
                        y[q] = add2(y[q], *reinterpret_cast<const f32x2*>(off + 2 * q));
                        l2[q] = mul2(l2[q], *reinterpret_cast<const f32x2*>(alpha + 2 * q));
                    }
                    return true;
                };
                const bool first = set;
                scores(!first);
                if (first) {
                    if (!set_reference()) { ok = false; break; }
                    set = false;
                } else {
                    float top = -INFINITY;
#pragma unroll
                    for (int q = 0; q < R / 2; ++q) {
                        const float2 s = unpack2(y[q]);
                        top = fmaxf(top, fmaxf(s.x, s.y));
                    }
                    const bool over = __any_sync(0xFFFFFFFFu, top > P_EXP_MAX);
                    if (lane == 0) {
                        votes[g * 4 + wl] = over;
                        mbar_arrive(&vote[g]);
                    }
                }
                // P of this group's previous tile has been read, and its O added up
                if (k > 0 && !warp_wait(&pfree[g], (k - 1) & 1, abort_flag, a.wait_ns)) { ok = false; break; }
                uint8_t* P = smem + C::OFF_P + g * C::PBUF + j * R;
                auto write_p = [&]() {
                    const int swz = R == 64 ? (j >> 1) & 3 : R == 32 ? (j >> 2) & 1 : 0;
#pragma unroll
                    for (int c0 = 0; c0 < R; c0 += 16) {
                        uint32_t hi[4], lo[4];
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            uint32_t up[2];
                            __nv_fp8x2_storage_t l8[2];
#pragma unroll
                            for (int z = 0; z < 2; ++z) {
                                const float2 s = unpack2(y[c0 / 2 + 2 * q + z]);
                                const float p0 = ex2(s.x), p1 = ex2(s.y);
                                if (!wide) y[c0 / 2 + 2 * q + z] = pack2(p0, p1);
                                const __half2 ph = __floats2half2_rn(p0, p1);
                                // p rounded to the upper byte of its fp16 pattern (p <= 2900: no carry out of it; NaN
                                // stays in the rest), and the exact rest
                                up[z] = (*reinterpret_cast<const uint32_t*>(&ph) + 0x00800080u) & 0xFF00FF00u;
                                l8[z] = __nv_cvt_halfraw2_to_fp8x2(__hsub2(ph, *reinterpret_cast<const __half2*>(&up[z])),
                                                                   __NV_SATFINITE, __NV_E4M3);
                            }
                            hi[q] = __byte_perm(up[0], up[1], 0x7531);
                            lo[q] = (uint32_t)l8[0] | ((uint32_t)l8[1] << 16);
                        }
                        uint8_t* at = P + (((c0 / 16) ^ swz) << 4);
                        *reinterpret_cast<uint4*>(at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                        *reinterpret_cast<uint4*>(at + TILE * R) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                    }
                };
                write_p();
                if (!first) {
                    if (!warp_wait(&vote[g], polls & 1, abort_flag, a.wait_ns)) { ok = false; break; }
                    ++polls;
                    if (votes[g * 4] | votes[g * 4 + 1] | votes[g * 4 + 2] | votes[g * 4 + 3]) {
                        // a score has passed the limit: the reference is set again, and O scaled down to it
                        scores(false);
                        if (!set_reference()) { ok = false; break; }
                        tc_fence_after();
                        const uint32_t orow = tmem + ((uint32_t)(wl * 32) << 16) + C::TMEM_O + (g * 2 + (piece & 1)) * C::MB * R;
                        for (int c0 = 0; c0 < C::MB * R; c0 += 8) {
                            uint32_t o[8];
                            tc_ld_x8(orow + c0, o);
                            tc_wait_ld();
                            const float* al = alpha + c0 % R;
#pragma unroll
                            for (int q = 0; q < 8; ++q) o[q] = __float_as_uint(__uint_as_float(o[q]) * al[q]);
                            tc_st_x8(orow + c0, make_uint4(o[0], o[1], o[2], o[3]), make_uint4(o[4], o[5], o[6], o[7]));
                        }
                        tc_wait_st();
                        write_p();
                    }
                }
                if (wide) {
#pragma unroll
                    for (int q = 0; q < R / 2; ++q) {
                        const float2 s = unpack2(y[q]);
                        l2[q] = add2(l2[q], pack2(ex2(s.x - (float)evi), ex2(s.y - (float)evi)));
                    }
                } else {
                    const float wj = exp2_int(-evi);
                    const f32x2 wj2 = pack2(wj, wj);
#pragma unroll
                    for (int q = 0; q < R / 2; ++q) l2[q] = fma2(y[q], wj2, l2[q]);
                }
                if (valid < TILE && (!PAIR || g == 0)) {
                    // rows past the lane's end hold anything: their values are cleared, so that 0 * NaN does not arise
                    const uint32_t f = 2 * i + 1;
                    if (!warp_wait(&full[f % NS], (f / NS) & 1, abort_flag, a.wait_ns)) { ok = false; break; }
                    if (j >= valid)
#pragma unroll
                        for (int p = 0; p < C::PANELS; ++p)
#pragma unroll
                            for (int q = 0; q < C::ROWB / 16; ++q)
                                *reinterpret_cast<uint4*>(smem + C::OFF_RING + (f % NS) * C::SLOT + p * C::PANEL + j * C::ROWB + q * 16) =
                                    make_uint4(0u, 0u, 0u, 0u);
                }
                fence_proxy_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&pfull[g]);
                ++k;
            }
            if (!ok) break;
            // the part's sums over this group's rows
            if (piece > 0 && !warp_wait(lfree, (piece - 1) & 1, abort_flag, a.wait_ns)) break;
            float v[R];
#pragma unroll
            for (int r = 0; r < R / 2; ++r) {
                const float2 p = unpack2(l2[r]);
                v[2 * r] = p.x;
                v[2 * r + 1] = p.y;
            }
            // halve the rows while the lanes are paired: a lane ends with the sums of its R / 32 rows
            int n = R;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                if (n > 1) {
                    n /= 2;
#pragma unroll
                    for (int r = 0; r < R / 2; ++r) {
                        if (r >= n) break;
                        const bool up = lane & o;
                        const float keep = up ? v[r + n] : v[r], send = up ? v[r] : v[r + n];
                        v[r] = keep + __shfl_xor_sync(0xFFFFFFFFu, send, o);
                    }
                } else {
                    v[0] += __shfl_xor_sync(0xFFFFFFFFu, v[0], o);
                }
            }
            float* ls = F + C::F_L + (g * 4 + wl) * R;
            if (R == 64) { ls[2 * lane] = v[0]; ls[2 * lane + 1] = v[R > 32 ? 1 : 0]; }
            else if (R == 32) ls[lane] = v[0];
            else if ((lane & 1) == 0) ls[lane >> 1] = v[0];
            if (wl == 0)
#pragma unroll
                for (int r = 0; r < RL; ++r)
                    if (R >= 32 || lane < R) F[C::F_M + g * R + r * 32 + lane] = M[r];
            __syncwarp();
            if (lane == 0) mbar_arrive(lfull);
            left -= nt;
            w.advance(a, facts, nt, left > 0);
            ++piece;
        }
    } else if (warp < 12) {
        // ------------------------------------------------------------ queries and outputs
        if constexpr (R == 64) regs_down<80>();
        const int wl = warp & 3;
        // the queries of the next unit; all loads of a batch are under way before the first is used
        Walk<RU> wq = w;
        int64_t qleft = left;
        uint32_t qpiece = 0;
        auto convert = [&]() -> bool {
            constexpr int LPR = D / 8, RPW = 32 / LPR;                // lanes a row, rows a warp takes at once
            constexpr int ITER = RU / (4 * RPW) > 0 ? RU / (4 * RPW) : 1, BATCH = ITER < 8 ? ITER : 8;
            const int part = lane % LPR, sub = lane / LPR;
            const uint32_t qb = qpiece % C::QBUFS;
            const int rows = wq.rows(a), row0 = wq.rt * RU;
            uint8_t* Q = smem + C::OFF_Q + qb * C::QBUF;
            float* qf = F + C::F_QF + (qpiece & 3) * RU;
            for (int i0 = 0; i0 < ITER; i0 += BATCH) {
                uint4 raw[BATCH];
#pragma unroll
                for (int b = 0; b < BATCH; ++b) {
                    const int u = ((i0 + b) * 4 + wl) * RPW + sub;
                    raw[b] = make_uint4(0u, 0u, 0u, 0u);
                    if (u < rows) {
                        const int node = (row0 + u) / G, qh = wq.h * G + (row0 + u) - node * G;
                        raw[b] = *reinterpret_cast<const uint4*>(a.q + (wq.l.n0 + node) * a.q_token_stride + qh * a.q_head_stride + part * 8);
                    }
                }
                if (i0 == 0 && !warp_wait(&qfree[qb], ((qpiece / C::QBUFS) & 1) ^ 1, abort_flag, a.wait_ns)) return false;
#pragma unroll
                for (int b = 0; b < BATCH; ++b) {
                    const int u = ((i0 + b) * 4 + wl) * RPW + sub;
                    const uint32_t in[4] = {raw[b].x, raw[b].y, raw[b].z, raw[b].w};
                    uint32_t key = 0;                                 // max |x|: bit patterns order as integers
#pragma unroll
                    for (int e = 0; e < 4; ++e) key = max(key, max((in[e] << 16) & 0x7FFFFFFFu, in[e] & 0x7FFF0000u));
#pragma unroll
                    for (int o = LPR / 2; o > 0; o >>= 1) key = max(key, __shfl_xor_sync(0xFFFFFFFFu, key, o));
                    int up = key ? 7 - floor_log2_pos(__uint_as_float(key)) : 0;
                    up = up > 120 ? 120 : (up < -120 ? -120 : up);
                    const float gain = exp2_int(up);
                    uint32_t hi[2], lo[2];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float x0 = __uint_as_float(in[e] << 16) * gain, x1 = __uint_as_float(in[e] & 0xFFFF0000u) * gain;
                        const __nv_fp8x2_storage_t h8 = __nv_cvt_float2_to_fp8x2(make_float2(x0, x1), __NV_SATFINITE, __NV_E4M3);
                        const float2 hf = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(h8, __NV_E4M3)));
                        const __nv_fp8x2_storage_t l8 =
                            __nv_cvt_float2_to_fp8x2(make_float2(x0 - hf.x, x1 - hf.y), __NV_SATFINITE, __NV_E4M3);
                        if (e & 1) { hi[e / 2] |= (uint32_t)h8 << 16; lo[e / 2] |= (uint32_t)l8 << 16; }
                        else { hi[e / 2] = h8; lo[e / 2] = l8; }
                    }
                    if (u < RU) {
                        // a row that is not finite: its scores become NaN
                        if (part == 0) qf[u] = key >= 0x7F800000u ? __uint_as_float(0x7FC00000u) : exp2_int(-up);
                        const int byte = part * 8, panel = byte / C::ROWB, in_row = byte % C::ROWB;
                        auto place = [&](int row) {
                            const int swz = C::ROWB == 128 ? row & 7 : (row >> 1) & 3;
                            return Q + panel * C::QROWS * C::ROWB + row * C::ROWB + (((in_row >> 4) ^ swz) << 4) + (in_row & 15);
                        };
                        const int row = (u / R) * 2 * R + u % R;
                        *reinterpret_cast<uint2*>(place(row)) = make_uint2(hi[0], hi[1]);
                        *reinterpret_cast<uint2*>(place(row + R)) = make_uint2(lo[0], lo[1]);
                    }
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&qfull[qb]);
            const int nt = qleft < wq.tiles - wq.t ? (int)qleft : wq.tiles - wq.t;
            qleft -= nt;
            ++qpiece;
            wq.advance(a, facts, nt, qleft > 0);
            return true;
        };

        constexpr int RL = RU > 32 ? RU / 32 : 1;    // tree rows a lane looks after
        float* st = F + C::F_ST + wl * 2 * RU;
        const bool on = D >= 128 || lane < 16;       // M = 64 leaves 16 rows in each quarter of the lanes
        const int d0 = D >= 128 ? wl * 32 + lane : wl * 16 + (lane & 15);
        uint32_t i0 = 0, piece = 0;                  // the part's first tile
        if (left > 0) (void)convert();
        while (left > 0) {
            const int nt = left < w.tiles - w.t ? (int)left : w.tiles - w.t;
            if (qleft > 0 && !convert()) break;
            const uint32_t ob = piece & 1;
            if (!warp_wait(lfull, piece & 1, abort_flag, a.wait_ns) || !warp_wait(&ofull[ob], (piece >> 1) & 1, abort_flag, a.wait_ns)) break;
            tc_fence_after();
            const int rows = w.rows(a), row0 = w.rt * RU;
            const bool whole = nt == w.tiles;
            // a group without a tile in this part has no O
            const bool has0 = PAIR || nt > 1 || (i0 & 1) == 0, has1 = !PAIR && (nt > 1 || (i0 & 1) == 1);
            float* part = reinterpret_cast<float*>(a.ws + parts_offset(gridDim.x)) +
                          (size_t)(2 * blockIdx.x + (left == count ? 0 : 1)) * part_floats(RU, D);
#pragma unroll
            for (int r = 0; r < RL; ++r) {
                const int u = r * 32 + lane;
                if (u >= rows) break;
                const int g0 = PAIR ? u / R : 0, row = PAIR ? u % R : u;
                auto sum = [&](int g) {
                    const float* ls = F + C::F_L + g * 4 * R + row;
                    return (ls[0] + ls[R]) + (ls[2 * R] + ls[3 * R]);
                };
                float M = F[C::F_M + g0 * R + row], L = sum(g0), f0 = 1.0f, f1 = 0.0f;
                if (!PAIR) {
                    const float M0 = M, M1 = F[C::F_M + R + row];
                    M = fmaxf(M0, M1);
                    f0 = M0 == -INFINITY ? 0.0f : ex2(M0 - M);
                    f1 = M1 == -INFINITY ? 0.0f : ex2(M1 - M);
                    L = L * f0 + sum(1) * f1;                         // sums may be NaN
                }
                if (whole) {
                    // out = O / L; lse = ln 2 (M - 8 + log2 L): p carries 2^8
                    const float inv = L == 0.0f ? 0.0f : 1.0f / L;
                    f0 *= inv;
                    f1 *= inv;
                    if (wl == 0 && a.lse) {
                        const int node = (row0 + u) / G;
                        a.lse[(int64_t)(w.l.n0 + node) * a.n_q_heads + w.h * G + row0 + u - node * G] =
                            L == 0.0f ? -INFINITY : (M - P_EXP + log2f(L)) * 0.69314718055994531f;
                    }
                } else if (wl == 0) {
                    part[RU * D + u] = M;
                    part[RU * D + RU + u] = L;
                }
                st[u] = f0;
                st[RU + u] = f1;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(lfree);
            int node = row0 / G, sub = row0 - node * G;
            __nv_bfloat16* out = a.out + ((int64_t)(w.l.n0 + node) * a.n_q_heads + w.h * G + sub) * D + d0;
            const uint32_t orow = tmem + ((uint32_t)(wl * 32) << 16) + C::TMEM_O;
            for (int c0 = 0; c0 < rows; c0 += 8) {
                float x[C::MB][8];
#pragma unroll
                for (int m = 0; m < C::MB; ++m) {
                    const int c = PAIR ? c0 % R : c0, g0 = PAIR ? c0 / R : 0;
                    uint32_t o0[8], o1[8];
                    if (has0) tc_ld_x8(orow + ((g0 * 2 + ob) * C::MB + m) * R + c, o0);
                    if (has1) tc_ld_x8(orow + ((2 + ob) * C::MB + m) * R + c, o1);
                    tc_wait_ld();
#pragma unroll
                    for (int q = 0; q < 8; ++q) {
                        x[m][q] = has0 ? __uint_as_float(o0[q]) * st[c0 + q] : 0.0f;
                        if (has1) x[m][q] = fmaf(__uint_as_float(o1[q]), st[RU + c0 + q], x[m][q]);
                    }
                }
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    if (c0 + q >= rows) break;
#pragma unroll
                    for (int m = 0; m < C::MB; ++m) {
                        if (!on) continue;
                        if (whole) out[m * 128] = __float2bfloat16_rn(x[m][q]);
                        else part[(c0 + q) * D + m * 128 + d0] = x[m][q];
                    }
                    out += D;
                    if (++sub == G) { sub = 0; out += (int64_t)(a.n_q_heads - G) * D; }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&ofree[ob]);
            i0 += nt;
            left -= nt;
            w.advance(a, facts, nt, left > 0);
            ++piece;
        }
    } else {
        if constexpr (R == 64) regs_down<64>();
        const int P = 1 << a.page_shift;
        // the cache row of this unit's head at lane row `at` (its page's first one is at / P * P), -1 past the end
        auto row_of = [&](const Walk<RU>& x, int64_t at, bool tell) -> int {
            if (at >= x.l.len) return -1;
            int p = a.table[(int64_t)x.b * a.width + (at >> a.page_shift)];
            if (p < 0 || p >= a.c.n_pages) {
                if (tell) record_error(a.err, MOE_DEV_BAD_PAGE);
                p = 0;
            }
            return (p * H + x.h) * P + (int)(at & (P - 1));
        };
        if (warp == 12) {
            // -------------------------------------------------------- TMA: lane l copies the tile's l-th page (or 128 rows of it)
            const int rows_a_page = P < TILE ? P : TILE;
            auto place = [&]() { return lane * rows_a_page < TILE ? row_of(w, (int64_t)w.t * TILE + lane * rows_a_page, true) : -1; };
            int next = left > 0 ? place() : -1;
            bool ok = true;
            for (uint32_t i = 0; left > 0 && ok; ++i) {
                const int row = next;
                --left;
                if (left > 0) {                                       // the next tile's page, one tile ahead
                    w.advance(a, facts, 1, true);
                    next = place();
                }
                const uint32_t bytes = __popc(__ballot_sync(0xFFFFFFFFu, row >= 0)) * rows_a_page * D;
#pragma unroll
                for (int v = 0; v < 2; ++v) {
                    const uint32_t f = 2 * i + v, s = f % NS;
                    if (!warp_wait(&empty[s], ((f / NS) & 1) ^ 1, abort_flag, a.wait_ns)) { ok = false; break; }
                    if (lane == 0) mbar_arrive_expect_tx(&full[s], bytes);
                    ++issued;
                    __syncwarp();
                    if (row >= 0)
#pragma unroll
                        for (int p = 0; p < C::PANELS; ++p)
                            tma_load_2d(smem + C::OFF_RING + s * C::SLOT + p * C::PANEL + lane * rows_a_page * C::ROWB,
                                        v ? &maps.v : &maps.k, &full[s], p * 128, row);
                }
            }
        } else if (warp == 13) {
            // -------------------------------------------------------- MMA issue. The loop is uniform over the warp and one elected
            // lane issues, so that descriptors stay in uniform registers (39 clocks an MMA of N = 16 against 120
            // from a loop that one lane runs).
            constexpr uint64_t KD = desc_base(C::ROWB == 128 ? 2 : 4, 8 * C::ROWB);       // K, Q (along K) and V (along M): one atom, 8 rows
            constexpr uint64_t PD = desc_base(R == 64 ? 4 : R == 32 ? 6 : 0, 8 * R);
            constexpr uint32_t ID_S = idesc_f8(128, 2 * R, 0, 0, 0);
            constexpr uint32_t ID_HI = idesc_f8(D < 128 ? 64 : 128, R, 1, 1, 1), ID_LO = idesc_f8(D < 128 ? 64 : 128, R, 1, 1, 0);
            const uint32_t base = __shfl_sync(0xFFFFFFFFu, tmem, 0);
            const uint64_t ring = desc_at(KD, smem_u32(smem + C::OFF_RING));
            const uint64_t qd = desc_at(KD, smem_u32(smem + C::OFF_Q)), pd = desc_at(PD, smem_u32(smem + C::OFF_P));
            uint32_t i = 0, piece = 0;
            // the tile before: its part, its place in it, whether it ends it
            uint32_t pp = 0, pt = 0, plast = 0;
            bool ok = true;
            auto qk = [&](uint32_t s, uint32_t qb, uint32_t g, bool done, bool last) {
                const uint64_t kd = ring + (uint64_t)(s * (C::SLOT >> 4)), q = qd + (uint64_t)(qb * (C::QBUF >> 4) + (PAIR ? g * (2 * R * C::ROWB >> 4) : 0));
                if (elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < D / 32; ++kk) {
                        constexpr int STEPS = C::ROWB / 32;
                        tc_mma_f8(base + g * 2 * R, kd + (((kk / STEPS) * C::PANEL + (kk % STEPS) * 32) >> 4),
                                  q + (((kk / STEPS) * C::QROWS * C::ROWB + (kk % STEPS) * 32) >> 4), ID_S, kk ? 1u : 0u);
                    }
                    if (done) tc_commit(&empty[s]);
                    tc_commit(&sfull[g]);
                    if (done && last) tc_commit(&qfree[qb]);
                }
                __syncwarp();
            };
            auto pv = [&](uint32_t n, uint32_t g, bool done, bool ends) {                  // adds tile n to group g's O
                const uint32_t s = (2 * n + 1) % NS;
                const uint64_t vd = ring + (uint64_t)(s * (C::SLOT >> 4)), p = pd + (uint64_t)(g * (C::PBUF >> 4));
                const uint32_t fresh = PAIR ? pt == 0 : pt < 2;
                const uint32_t o = base + C::TMEM_O + (g * 2 + (pp & 1)) * C::MB * R;
                if (elect_one()) {
#pragma unroll
                    for (int m = 0; m < C::MB; ++m)
#pragma unroll
                        for (int kk = 0; kk < 8; ++kk)                 // four steps of 32 rows with hi, four with lo
                            tc_mma_f8(o + m * R, vd + ((m * C::PANEL + (kk & 3) * 32 * C::ROWB) >> 4),
                                      p + (((kk >> 2) * TILE * R + (kk & 3) * 32 * R) >> 4), kk < 4 ? ID_HI : ID_LO, kk ? 1u : fresh ^ 1u);
                    if (done) tc_commit(&empty[s]);
                    tc_commit(&pfree[g]);
                    if (ends) tc_commit(&ofull[pp & 1]);
                }
                __syncwarp();
            };
            auto wait = [&](uint64_t* bar, uint32_t parity) { return ok = warp_wait(bar, parity, abort_flag, a.wait_ns); };
            auto before_pv = [&](uint32_t n) {                         // the values, and room for the part's first O
                const uint32_t f = 2 * n + 1;
                return wait(&full[f % NS], (f / NS) & 1) && (pt > 0 || wait(&ofree[pp & 1], ((pp >> 1) & 1) ^ 1));
            };
            while (left > 0 && ok) {
                const int nt = __shfl_sync(0xFFFFFFFFu, left < w.tiles - w.t ? (int)left : w.tiles - w.t, 0);
                const uint32_t qb = piece % C::QBUFS;
                if (!wait(&qfull[qb], (piece / C::QBUFS) & 1)) break;
                for (int t = 0; t < nt; ++t, ++i) {
                    const uint32_t f = 2 * i, s = f % NS;
                    if (!wait(&full[s], (f / NS) & 1)) break;
                    if constexpr (PAIR) {
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            if (i > 0 && !wait(&pfull[h], (i - 1) & 1)) break;       // S of the tile before has been read
                            tc_fence_after();
                            qk(s, qb, h, h == 1, t == nt - 1);
                            if (i > 0) {
                                if (h == 0 && !before_pv(i - 1)) break;
                                tc_fence_after();
                                pv(i - 1, h, h == 1, h == 1 && plast);
                            }
                        }
                        if (!ok) break;
                    } else {
                        tc_fence_after();
                        qk(s, qb, i & 1, true, t == nt - 1);
                        if (i > 0) {                                   // also: S of tile i - 1 has been read before tile i + 1
                            if (!wait(&pfull[(i - 1) & 1], ((i - 1) >> 1) & 1) || !before_pv(i - 1)) break;
                            tc_fence_after();
                            pv(i - 1, (i - 1) & 1, true, plast);
                        }
                    }
                    pp = piece;
                    pt = t;
                    plast = t == nt - 1;
                }
                if (!ok) break;
                left -= nt;
                ++piece;
                w.advance(a, facts, nt, left > 0);
            }
            if (ok && i > 0) {
                if constexpr (PAIR) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        if (!wait(&pfull[h], (i - 1) & 1) || (h == 0 && !before_pv(i - 1))) break;
                        tc_fence_after();
                        pv(i - 1, h, h == 1, h == 1);
                    }
                } else if (wait(&pfull[(i - 1) & 1], ((i - 1) >> 1) & 1) && before_pv(i - 1)) {
                    tc_fence_after();
                    pv(i - 1, (i - 1) & 1, true, true);
                }
            }
        } else if (warp == 14) {
            // -------------------------------------------------------- scales: a lane takes four rows; pages are looked up two tiles
            // ahead and scales read one ahead
            auto place = [&]() { return row_of(w, (int64_t)w.t * TILE + lane * 4, false); };
            auto load = [&](int row, uint32_t& ks, uint32_t& vs) {
                ks = vs = 0x7F7F7F7Fu;
                if (row >= 0) {
                    ks = *reinterpret_cast<const uint32_t*>(a.c.k_scales + row);
                    vs = *reinterpret_cast<const uint32_t*>(a.c.v_scales + row);
                }
            };
            uint32_t ks = 0, vs = 0, ks1 = 0, vs1 = 0;
            int row1 = -1;
            if (left > 0) load(place(), ks, vs);
            if (left > 1) {
                w.advance(a, facts, 1, true);
                row1 = place();
            }
            for (uint32_t i = 0; left > 0; ++i) {
                if (left > 1) load(row1, ks1, vs1);
                if (left > 2) {
                    w.advance(a, facts, 1, true);
                    row1 = place();
                }
                const uint32_t sc = i % NSC;
                if (!warp_wait(&scempty[sc], ((i / NSC) & 1) ^ 1, abort_flag, a.wait_ns)) break;
                uint32_t* dst = reinterpret_cast<uint32_t*>(smem + C::OFF_SC + sc * 256);
                dst[lane] = ks;
                dst[32 + lane] = vs;
                __syncwarp();
                if (lane == 0) mbar_arrive(&scfull[sc]);
                ks = ks1;
                vs = vs1;
                --left;
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (*abort_flag) {                               // final after the barrier: nothing new is issued past it
        if (warp == 12 && lane == 0) drain_stage_fills(full, NS, issued);
        if (warp == 13 && elect_one()) tc_drain(drain);
        tc_fence_before();
        __syncthreads();
    }
    if (warp == 13) {
        tc_fence_after();
        tmem_dealloc(tmem, C::TMEM_COLS);
    }
    if (tid == 0 && *abort_flag) record_error(a.err, MOE_DEV_TIMEOUT);
}

// ------------------------------------------------------------------ join

// One warp per tree row of a unit that several CTAs share; blockIdx.x is the
// second of them (the first whose part begins inside the unit). The parts are
// added in the order of the cache rows, so the result does not depend on the order
// in which they were done.
constexpr int JOIN_WARPS = 8;

template <int D, int RU>
__global__ void __launch_bounds__(JOIN_WARPS * 32) tree_attention_join(const AttnArgs a, int ctas) {
    pdl_trigger();
    pdl_wait();
    const JoinHead head = *reinterpret_cast<const JoinHead*>(a.ws);
    const int c = blockIdx.x + 1;
    if (c >= head.parts) return;
    const JoinUnit u = reinterpret_cast<const JoinUnit*>(a.ws + JOIN_UNITS)[c];
    auto begin = [&](int k) { return (int64_t)((unsigned long long)head.total * k / head.parts); };
    if (begin(c) <= u.first || begin(c - 1) > u.first) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int r = blockIdx.y * JOIN_WARPS + warp;
    if (r >= u.rows) return;
    // the last CTA whose part begins before the unit's end: total k < end parts
    const int last = (int)(((unsigned long long)u.end * head.parts - 1) / head.total);
    const float* parts = reinterpret_cast<const float*>(a.ws + parts_offset(ctas));
    const int before = begin(c - 1) < u.first;       // that CTA comes to the unit from another one
    auto part = [&](int k) { return parts + (size_t)(2 * k + (k == c - 1 ? before : 0)) * part_floats(RU, D); };
    float M = -INFINITY;
    for (int k = c - 1 + lane; k <= last; k += 32) M = fmaxf(M, part(k)[RU * D + r]);
    M = warp_max(M);
    constexpr int V = D / 32;                        // columns a lane
    float acc[V] = {}, L = 0.0f;
#pragma unroll 4
    for (int k = c - 1; k <= last; ++k) {
        const float* p = part(k);
        const float m = p[RU * D + r];
        const float f = m == -INFINITY ? 0.0f : ex2(m - M);
        L += f * p[RU * D + RU + r];                   // NaN stays, also with a weight of zero
#pragma unroll
        for (int e = 0; e < V; ++e) acc[e] += f * p[r * D + e * 32 + lane];
    }
    const float inv = L == 0.0f ? 0.0f : 1.0f / L;
    const int tr = u.row0 + r, node = tr / a.group;
    const int64_t at = (int64_t)(u.node0 + node) * a.n_q_heads + u.head * a.group + tr - node * a.group;
#pragma unroll
    for (int e = 0; e < V; ++e) a.out[at * D + e * 32 + lane] = __float2bfloat16_rn(acc[e] * inv);
    if (a.lse && lane == 0) a.lse[at] = L == 0.0f ? -INFINITY : (M - P_EXP + log2f(L)) * 0.69314718055994531f;
}

// ------------------------------------------------------------------ host side

int log2_of(int p) { return 31 - __builtin_clz((unsigned)p); }

PFN_cuTensorMapEncodeTiled_v12000 encoder() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    });
    return fn;
}

cudaError_t codes_map(CUtensorMap* m, const void* base, const moe_kv_cache& c) {
    auto enc = encoder();
    if (!enc) return cudaErrorNotSupported;
    const cuuint64_t dims[2] = {(cuuint64_t)c.head_dim, (cuuint64_t)c.n_pages * c.n_kv_heads * c.page_size};
    const cuuint64_t strides[1] = {(cuuint64_t)c.head_dim};
    const cuuint32_t box[2] = {(cuuint32_t)(c.head_dim < 128 ? c.head_dim : 128), (cuuint32_t)(c.page_size < TILE ? c.page_size : TILE)};
    const cuuint32_t estr[2] = {1, 1};
    const CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
                           CU_TENSOR_MAP_INTERLEAVE_NONE, c.head_dim == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
                           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

constexpr int max_unit(int D) { return D == 256 ? 64 : 128; }        // RU: two halves of the widest R

template <int D, int R, bool PAIR>
cudaError_t launch(const AttnArgs& a, cudaStream_t s) {
    using C = Cfg<D, R, PAIR>;
    AttnMaps maps;
    cudaError_t e = codes_map(&maps.k, a.c.k_codes, a.c);
    if (e == cudaSuccess) e = codes_map(&maps.v, a.c.v_codes, a.c);
    if (e != cudaSuccess) return e;
    static bool attr_set[64] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev >= 0 && dev < 64 && !attr_set[dev]) {
        e = cudaFuncSetAttribute(tree_attention<D, R, PAIR>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
        if (e != cudaSuccess) return e;
        attr_set[dev] = true;
    }
    const int ctas = moe_sm_count();
    moe_prof_begin(MK_ATTENTION, s);
    e = moe_launch(tree_attention<D, R, PAIR>, dim3((unsigned)ctas), dim3(ATTN_THREADS), C::SMEM, s, maps, a);
    moe_prof_end(MK_ATTENTION, s);
    if (e != cudaSuccess || ctas < 2) return e;
    moe_prof_begin(MK_ATTENTION_JOIN, s);
    e = moe_launch(tree_attention_join<D, C::RU>, dim3((unsigned)(ctas - 1), C::RU / JOIN_WARPS), dim3(JOIN_WARPS * 32), 0, s, a, ctas);
    moe_prof_end(MK_ATTENTION_JOIN, s);
    return e;
}

// The tile of tree rows: the smallest that takes a lane's rows of one kv head at once.
template <int D>
cudaError_t launch_rows(const AttnArgs& a, cudaStream_t s) {
    const int64_t rows = (int64_t)(a.max_nodes < a.n_nodes ? a.max_nodes : a.n_nodes) * a.group;
    if (rows <= 16) return launch<D, 16, false>(a, s);
    if (rows <= 32) return launch<D, 32, false>(a, s);
    if constexpr (D == 256) {
        return launch<D, 32, true>(a, s);
    } else {
        if (rows <= 64) return launch<D, 64, false>(a, s);
        return launch<D, 64, true>(a, s);
    }
}

}  // namespace

size_t moe_tree_attention_workspace_bytes(int n_nodes, int n_q_heads, int n_kv_heads, int head_dim, int lanes) {
    if (n_nodes < 1 || n_q_heads < 1 || n_kv_heads < 1 || head_dim < 1 || lanes < 1) return 0;
    const int ctas = moe_sm_count();
    return parts_offset(ctas) + (size_t)2 * ctas * part_floats(max_unit(head_dim), head_dim) * sizeof(float);
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
    a.scale_log2 = scale * 1.4426950408889634f;
    a.out = static_cast<__nv_bfloat16*>(out);
    a.lse = lse;
    a.ws = static_cast<uint8_t*>(workspace);
    a.err = err;
    a.wait_ns = moe_wait_limit_ns();
    const cudaError_t e = cache->head_dim == 64    ? launch_rows<64>(a, s)
                          : cache->head_dim == 128 ? launch_rows<128>(a, s)
                                                   : launch_rows<256>(a, s);
    moe_count_launches(2);
    return e == cudaSuccess ? MOE_OK : MOE_ECUDA;
}
