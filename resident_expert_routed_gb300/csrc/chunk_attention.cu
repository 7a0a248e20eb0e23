// Attention of a chunk of new tokens over the paged 8-bit key/value cache.
//
// For the rows r = (token, query head) of one kv head and the cache rows j up to the token's own:
//   x[r,j] = scale log2(e) q_r . k_j        (k_j = codes * 2^ek_j)
//   out[r] = sum_j 2^x[r,j] v_j / sum_j 2^x[r,j]      (v_j = codes * 2^ev_j)
// The rows are the MMA's M (128 a tile), 128 cache rows its N, fp32 accumulators in TMEM:
//   S[128, 128] = Q hi K^T + Q lo K^T      kind::f8f6f4 on the cache's codes as TMA brings them; the queries in two e4m3 parts
//   O[128, D]  += P V                      kind::f16: P in bf16, from TMEM; V in bf16
//   - A bf16 query has 8 significant bits and e4m3 has 4: with its rows scaled by a power of two to at most 256, hi =
//     e4m3(q) and lo = e4m3(q - hi) hold it exactly down to 2^-9 of the maximum and within 2^-17 of the maximum below. Two
//     8-bit products cost what one of 16 bits costs, and no key is converted.
//   - A key row's scale is the factor of its column of scores: one fused multiply-add takes it and the reference.
//   - e4m3 codes times a power of two are exact in bf16, and bf16 has the exponents of fp32: weights and values
//     need no care about their range. Eight warps convert each tile of values once for the 256 rows that use it.
//   - m is a running reference, not each tile's maximum: it stays until a score passes it by 2^8 (p then up to 2^8, in
//     bf16 as good as below 1), and only then O and the sum are scaled down. A thread has a row to itself, so neither
//     maximum nor sum needs another thread.
// Scores, sums, O and the parts that the join adds up are fp32. Weights are rounded to bf16 for the second product, by at most
// 2^-8 of each (the sum takes them before), far less than a value's own 2^-4; lanes of few rows take what is left of them as a
// second part (FEW_ROWS), to 2^-16. The output is rounded once.
//
// A unit is a block of 256 rows (128 at head_dim 256, where O fills TMEM) of a lane and kv head, whole tokens with all their
// heads, so 256 / group tokens share each tile of the cache and the causal edge is as near as can be. Its tiles of cache
// rows come one after the other; the two tiles of 128 rows take turns: while one's softmax runs, the other's products do, and
// each works by halves of 64 cache rows: half's weights at work beside the other half's softmax, the next tile's scores of that
// half behind them. A unit of at most 128 rows (single tokens among them) has one row tile and two buffers of S, which the two
// groups of the softmax take in turn, each with an O of its own; the two are added up from TMEM at the end.
//
// Work: the units are laid end to end and cut into equal parts, one per CTA. A unit that one CTA does whole is written at
// once; the others leave parts (O, reference, sum) in the workspace, and chunk_attention_join adds them up in order.
//
// Roles, 20 warps: two softmax groups of four; two groups of four that convert pieces of values in turn and together prepare
// queries; one warp that walks the run and issues TMA; one of MMA issue for each buffer of S; one of scales, which also
// bounds all waits.
//
// What bounds it at head_dim 128: 128 cache rows take the two row tiles about 3,300 clocks, and shared memory is busy for nearly
// all of them: 336 KB of operands (2,690 clocks: the queries and keys once for each row tile and half 192 KB, values for each row
// tile 64, through the conversion 48, copies 32) and 512 reads of the columns' factors. The tensor cores work 2,050 of them, the
// softmax issues for 2,000 on each of the SM's four schedulers. 1,024 tokens over 65,536 rows (32 / 8 heads) take 778 us, 1,425
// TFLOP/s; over and over they draw 1.4 kW and the clock falls: 870 us. A prompt of 8,192 takes 461 us, 1,195 TFLOP/s: the edge,
// a unit's first tile, its queries and its output, some 9 us a unit, are what its 6.7 units a CTA pay. At head_dim 64 nothing is
// near its limit (issue slots 64 %, tensor cores 33 %, a prompt 365 us): softmax and issue wait for one another, and for short prompts
// one instruction fetch in six misses its cache. At 256 (990 us) the conversion serves 128 rows only, and the tensor cores are at 49 %.
// Single tokens over 8,192 rows, 64 lanes: 345 us, 3.2 TB/s, the conversion of a tile for the 4 rows that use it; issue slots 71 %,
// tensor cores 53 % (without the softmax of warps whose rows are nobody's 343). 300 tokens take 14.6 us in a table of as many rows, of which 3 to find the parts, 4 to bring and split the
// queries and 2 for a first tile's scores; in a table for 8,192 rows 23 us (SHORT_TILES).
// The instructions' cache is as scarce as anything: loops that are not unrolled, and code in one place, are faster in most places.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <climits>
#include <type_traits>

#include "attention.cuh"

namespace {

struct ChunkArgs {
    moe_kv_cache c;
    const __nv_bfloat16* q;
    int64_t q_token, q_head;
    int n_tokens, n_q, group, block;             // group: query heads to a kv head; block: tokens of a unit
    uint32_t by_group;                           // ceil(2^16 / group): divides a row of a unit by group
    const int32_t* table;
    int width, lanes, page_shift;
    const int32_t* kv_len;
    const int32_t* cu;
    int whole;                                   // units are not cut
    float scale_log2;
    __nv_bfloat16* out;
    float* lse;
    uint8_t* ws;
    uint32_t* err;
    uint64_t wait_ns;
};

struct ChunkMaps {
    CUtensorMap k, v;                            // (head_dim, rows) bytes; boxes: an operand panel of keys, whole rows of values
};

constexpr int TILE = 128;                        // cache rows a tile, and rows a row tile
// Units are not cut, and no parts joined, where the table has at most SHORT_TILES tiles (cut / whole: 40 prompts of 300 tokens
// 134 / 132 us, 9 of 600 87 / 83), or WHOLE_TILES and there are at most two full units an SM (a prompt of 1024 43 / 33, two
// 56 / 54, 200 single tokens over 1000 182 / 165; but three prompts 66 / 74, eight 134 / 144; a prompt of 2048 67 / 81). The host
// has the table's width and not the lanes' lengths, so a short prompt in a wide table is cut: 300 tokens 23 us for 14.6, 1024 35 for 28,
// 16 tokens 13.0 for 10.8, 40 prompts of 300 132 for 128 (back to back in a graph; tables of 8,192 and of 131,072 rows alike).
constexpr int SHORT_TILES = 5, WHOLE_TILES = 8;
// Lanes with at most so many rows (new tokens times query heads) have their weights in two bf16 parts. One part is as coarse as the
// output's own rounding, and over few rows that does not average out to less (error against 64 bits up to 1.55 times that of fp32
// rounded once, over 60 rows; 1.3 to 1.4 over many). By the lane, so that what a token gets does not depend on the others in the call.
// One / two parts: one token in 30 lanes, 2 heads of 64 over 10,476 rows 46 / 55 us; 64 lanes, 32 / 8 heads of 128 over 8,192 rows
// 310 / 345; 33 lanes, of which 22 take one token, 233 / 243; 8 tokens over 300 rows 14 / 14. That the second form is there costs the
// others too, in registers and instruction fetches (without it / with it: a prompt of 8,192 457 / 461, at head_dim 64 357 / 365, 24
// prompts of 1,024 there 151 / 160; at 256 980 / 990). Figures beside the other choices of this file were taken without it.
constexpr int FEW_ROWS = 1024;
constexpr float NEVER = -3.402823466e38f;        // the reference of a row that has seen nothing: below any finite score
constexpr float LIMIT = 8.0f;                    // log2 of the largest weight before the reference moves (4 or 16: no difference)

// The run's measure: a cache row of a unit with two row tiles, of one with one (200 single tokens beside three chunks of 500,
// 64 query heads, for 2 / 3 / 4: 642 / 615 / 759 us). A unit beside its rows: see Cfg.
constexpr int FULL_COST = 4, HALF_COST = 3;
constexpr int STAGGER = 20;                      // looks (0 / 20 / 64: a prompt at head_dim 64 367 / 359 / 368 us, 24 of 1,024 152 / 158 / 171)
constexpr int LEAST_PART = 2048;                 // of a part (half or twice as much: no difference)

struct Pos {                                     // a place in the run
    int lane, unit, tile, pad;
};
MOE_DEV bool same_unit(const Pos& a, const Pos& b) { return a.lane == b.lane && a.unit == b.unit; }
MOE_DEV bool before(const Pos& a, const Pos& b) {
    return a.lane != b.lane ? a.lane < b.lane : a.unit != b.unit ? a.unit < b.unit : a.tile < b.tile;
}

// A CTA's way through its part of the run: a unit, and its tiles [t0, t1) that are this CTA's. One warp walks and tells the
// others (six copies of the walk would crowd the softmax out of the instruction cache).
struct alignas(16) Part {
    int b, h, tok0, first;                       // lane, kv head, first token, its own row (as in Unit)
    int rows, nt, end, tiles;
    int t0, t1;                                  // t1 = 0: there are no more
    int two, pad;                                // whether its weights are in two parts (FEW_ROWS)
};

template <int D>
struct Cfg {
    static constexpr int NT = D <= 128 ? 2 : 1;               // row tiles of a unit
    static constexpr int ROWS = NT * TILE;
    static constexpr int THREADS = 640;
    // For 1536 / 2048 / 2560, us: head_dim 128, a prompt of 8192 tokens 480 / 456 / 459, 22 single tokens and 11 chunks over
    // prefixes 264 / 238 / 234; head_dim 64, a prompt 361 / 366 / 369; head_dim 256, 1033 / 1056 / 1074. (1024: 517, 388, 1115)
    static constexpr int UNIT_COST = D == 128 ? 2560 : 1536;
    static constexpr int ROWB = D >= 128 ? 128 : 64;          // bytes of an operand row of keys and queries: one swizzle atom
    static constexpr int PANELS = D / ROWB;
    static constexpr int KPANEL = TILE * ROWB, KSLOT = TILE * D;
    static constexpr int QPANEL = 2 * TILE * ROWB, QTILE = 2 * TILE * D;      // hi, then lo
    // Rings have even numbers of slots: see MMA issue, and the groups that convert, of which each takes every second piece. What
    // fits beside the queries: at head_dim 128 four slots of codes instead of six 480 us a prompt for 457, pieces of 32 rows 491; at
    // 64 eight key tiles 158 us for 24 prompts of 1,024, for 150, four pieces in bf16 367 a prompt for 359; at 256 pieces of 16 rows 1203
    // for 1025, three slots of codes for both groups together 1176.
    static constexpr int NK = D == 64 ? 4 : 2;                // ring of key tiles
    static constexpr int VR = D == 256 ? 32 : 64;             // values come in pieces of so many rows
    static constexpr int PIECES = TILE / VR;
    static constexpr int NR = D == 64 ? 8 : D == 128 ? 6 : 2; // ring of pieces as codes
    static constexpr int RSLOT = VR * D;
    static constexpr int NB = D == 64 ? 8 : 4;                // ring of pieces in bf16
    static constexpr int VPANEL = VR * 128, BSLOT = VR * D * 2;
    static constexpr int SA = 4, NSC = 2 * SA;                // tiles that scales are under way ahead; their ring:
    static constexpr int SC_BYTES = 3 * TILE * 2;             // key bytes, value bytes, the columns' factors (float)
    static constexpr int OFF_Q = 0;
    static constexpr int OFF_K = OFF_Q + NT * QTILE;
    static constexpr int OFF_R = OFF_K + NK * KSLOT;
    static constexpr int OFF_B = OFF_R + NR * RSLOT;
    static constexpr int OFF_SC = OFF_B + NB * BSLOT;
    static constexpr int OFF_SID = OFF_SC + NSC * SC_BYTES;   // page ids, [2 SA][32]
    // What the softmax reads of a part's queries: of four parts, as the next parts' queries may be ready before a part of one
    // tile is begun (its scores wait for those of two items before alone).
    static constexpr int QB = 4;
    static constexpr int OFF_QF = OFF_SID + 2 * SA * 128;     // [QB][ROWS] 2^-a of the queries' rows
    static constexpr int OFF_QU = OFF_QF + QB * ROWS * 4;     // [QB][2] 2^-a of a unit's rows; whether they differ instead
    static constexpr int OFF_QX = OFF_QU + QB * 8;            // [2][largest, smallest][8 warps]
    static constexpr int NPD = 4;                             // parts that are told ahead
    static constexpr int OFF_PD = OFF_QX + 128;
    static constexpr int OFF_ML = OFF_PD + NPD * (int)sizeof(Part);       // [2][TILE] references and sums that the groups tell one another
    static constexpr int OFF_ONE = OFF_ML + (NT == 2 ? 2 * TILE * 8 : 0);        // [32] 1
    static constexpr int OFF_BAR = OFF_ONE + 128;
    static constexpr int B_KFULL = OFF_BAR;                   // [NK] a tile of keys has arrived
    static constexpr int B_KEMPTY = B_KFULL + 8 * NK;         // [NK] ... has been used
    static constexpr int B_RFULL = B_KEMPTY + 8 * NK;         // [NR] a piece of values has arrived
    static constexpr int B_REMPTY = B_RFULL + 8 * NR;
    static constexpr int B_BFULL = B_REMPTY + 8 * NR;         // [NB] ... is there in bf16
    static constexpr int B_BEMPTY = B_BFULL + 8 * NB;
    static constexpr int B_SCFULL = B_BEMPTY + 8 * NB;        // [NSC] a tile's factors and value bytes are there
    static constexpr int B_SCEMPTY = B_SCFULL + 8 * NSC;
    static constexpr int B_SFULL = B_SCEMPTY + 8 * NSC;       // [2][2] half of S is ready
    static constexpr int B_PFULL = B_SFULL + 32;              // [2][2] half of P is written (that half of S has been read)
    static constexpr int B_OHALF = B_PFULL + 32;              // [2] the first half of P has been used
    static constexpr int B_ODONE = B_OHALF + 16;              // [2] both: a tile is added to O
    static constexpr int B_QFULL = B_ODONE + 16;              // [QB] the queries of a part are there
    static constexpr int B_QFREE = B_QFULL + 8 * QB;              // ... have been used
    static constexpr int B_QMAX = B_QFREE + 8;                // the eight warps have their maxima
    static constexpr int B_PDFULL = B_QMAX + 8;               // [NPD] a part is told
    static constexpr int B_PDEMPTY = B_PDFULL + 8 * NPD;      // [NPD] ... and read by the other nineteen warps
    static constexpr int B_MERGE = B_PDEMPTY + 8 * NPD;       // of a part with one row tile: both groups' O stands; it is read
    static constexpr int B_DONE = B_MERGE + 8;                // the block's last output is written
    static constexpr int B_DRAIN = B_DONE + 8;
    static constexpr int OFF_MISC = (B_DRAIN + 16 + 15) / 16 * 16;    // tmem slot, abort flag, progress [3] and one more, start, end
    static constexpr int SMEM = OFF_MISC + 32 + 32 + 1024;
    static constexpr int TMEM_O = 2 * TILE;                   // after S [2]
    static constexpr int SOFT_REGS = 152, CONV_REGS = 56, REST_REGS = 64;     // 2 x 152 + 2 x 56 + 64 = 5 x 96
    static_assert(OFF_B % 1024 == 0 && OFF_R % 128 == 0 && OFF_K % 1024 == 0 && BSLOT % 1024 == 0, "alignment");
    static_assert(OFF_BAR % 8 == 0 && OFF_QF % 16 == 0 && SMEM <= 227 * 1024, "shared memory");
    static_assert(2 * SOFT_REGS + 2 * CONV_REGS + REST_REGS <= 5 * 96, "registers");
    static constexpr size_t PART_FLOATS = (size_t)ROWS * (D + 2);     // O [D / 4][ROWS][4], references, sums
};
constexpr size_t parts_offset(int ctas) { return ((size_t)(ctas + 1) * sizeof(Pos) + 255) / 256 * 256; }

// ------------------------------------------------------------------ device pieces

MOE_DEV void tc_mma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
        ::"r"(d_tmem), "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// kind::f16, bf16 x bf16 -> fp32, B with N contiguous.
__host__ __device__ constexpr uint32_t idesc_bf16(int m, int n) {
    return (1u << 4) | (1u << 7) | (1u << 10) | (1u << 16) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}
MOE_DEV void tc_ld_x32(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {"
        "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
}
// What reads the registers of a tcgen05.ld under way: volatile, so that it stays behind the wait, which is too.
MOE_DEV f32x2 fma2_loaded(f32x2 a, f32x2 b, f32x2 c) {
    f32x2 r;
    asm volatile("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
MOE_DEV f32x2 mul2_loaded(f32x2 a, f32x2 b) {
    f32x2 r;
    asm volatile("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
MOE_DEV void tc_st_x32(uint32_t taddr, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {"
        "%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
        "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};"
        ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
          "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
          "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]),
          "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}
MOE_DEV uint32_t pack_bf16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// 32 bytes, a whole sector, of a thread.
MOE_DEV void store_32(void* to, uint32_t a, uint32_t b, uint32_t c, uint32_t d, uint32_t e, uint32_t f, uint32_t g, uint32_t h) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                 ::"l"(to), "r"(a), "r"(b), "r"(c), "r"(d), "r"(e), "r"(f), "r"(g), "r"(h) : "memory");
}
MOE_DEV void cp_async_16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
MOE_DEV uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
MOE_DEV void arrive_at_n(uint32_t bar, uint32_t n) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(n) : "memory");
}

// ------------------------------------------------------------------ lanes, units, the cut

// A lane that does not fit (see the header): no rows, and its outputs become zeros; so too, though not bad, one of no rows
// with tokens, as a plan refuses it. One whose tokens would lead out of q has none of them either.
struct Lane {
    int n0, n, len;
};
MOE_DEV Lane lane_facts(const ChunkArgs& a, int b, bool* bad) {
    Lane l;
    l.n0 = a.cu[b];
    l.n = a.cu[b + 1] - l.n0;
    l.len = a.kv_len[b];
    *bad = false;
    if (l.n0 < 0 || l.n < 0 || l.n > a.n_tokens - l.n0) {
        *bad = true;
        l.n0 = l.n = l.len = 0;
    } else if (l.n > 0 && l.len != 0 && (l.len < l.n || l.len > 1 << 30 || (((int64_t)l.len + (1 << a.page_shift) - 1) >> a.page_shift) > a.width)) {
        *bad = true;
        l.len = 0;
    }
    return l;
}

struct Unit {
    int b, h;                                    // lane, kv head
    int tok0;                                    // the unit's first token, in q
    int first;                                   // that token's own row in the lane; -2^30 where the lane is refused
    int rows, nt;                                // rows (token, head) of the unit; row tiles
    int end, tiles;                              // rows of the lane that it sees at all; tiles of them
    int units;                                   // of the lane
    int two;                                     // whether its weights are in two parts (FEW_ROWS)
};
template <int D>
MOE_DEV Unit unit_at(const ChunkArgs& a, int b, int u) {
    bool bad;
    const Lane l = lane_facts(a, b, &bad);
    Unit x;
    const int blocks = l.n > 0 ? (l.n + a.block - 1) / a.block : 1;
    x.b = b;
    x.h = u / blocks;
    const int rb = u - x.h * blocks, t0 = rb * a.block;
    const int tokens = min(a.block, l.n - t0);
    x.tok0 = l.n0 + t0;
    x.rows = tokens * a.group;
    x.nt = x.rows > TILE ? 2 : 1;
    x.first = l.len > 0 ? l.len - l.n + t0 : -(1 << 30);
    x.end = l.len > 0 ? x.first + tokens : 0;
    x.tiles = x.end > 0 ? (x.end + TILE - 1) / TILE : 1;
    x.units = a.c.n_kv_heads * blocks;
    x.two = (int64_t)l.n * a.n_q <= FEW_ROWS;
    return x;
}
template <int D>
MOE_DEV Part next_part(const ChunkArgs& a, const Pos& end, Pos& at, int& units) {      // units: of the lane; 0 before the first part
    for (;;) {
        if (units > 0 && ++at.unit >= units) {
            at.unit = 0;
            bool bad;
            do ++at.lane; while (at.lane < end.lane && lane_facts(a, at.lane, &bad).n == 0);
        }
        if (units > 0) at.tile = 0;
        if (!before(at, end)) return Part{};
        const Unit x = unit_at<D>(a, at.lane, at.unit);
        units = x.units;
        const int t1 = same_unit(at, end) ? min(end.tile, x.tiles) : x.tiles;
        if (t1 > at.tile) return Part{x.b, x.h, x.tok0, x.first, x.rows, x.nt, x.end, x.tiles, at.tile, t1, x.two, 0};
    }
}

// Costs of the units before block rb of a head with n tokens (rb full blocks; the last may be short).
struct LaneCost {
    long long base, step;                        // cost of block r: base + step (r + 1), but for the last
    long long last;                              // of the last block
    int blocks;
    MOE_DEV unsigned long long upto(int rb) const { return (unsigned long long)(base * rb + step * rb * (rb + 1) / 2); }
    MOE_DEV unsigned long long head() const { return blocks ? upto(blocks - 1) + (unsigned long long)last : 0ull; }
};
template <int D>
MOE_DEV LaneCost lane_cost(const ChunkArgs& a, const Lane& l) {
    LaneCost c{0, 0, 0, 0};
    if (l.n == 0) return c;
    c.blocks = (l.n + a.block - 1) / a.block;
    if (a.whole) {
        c.base = c.last = 1;
        return c;
    }
    const int left = (l.n - (c.blocks - 1) * a.block) * a.group;
    const int w = Cfg<D>::NT == 2 && left <= TILE ? HALF_COST : FULL_COST;
    c.base = c.last = Cfg<D>::UNIT_COST;
    if (l.len > 0) {
        c.base += (long long)FULL_COST * (l.len - l.n);
        c.step = (long long)FULL_COST * a.block;
        c.last += (long long)w * l.len;
    }
    return c;
}

// Every CTA adds up all lanes' costs and finds where its part begins and ends.
template <int D>
__device__ __noinline__ void cut_run(const ChunkArgs& a, unsigned long long* scratch, Pos* here) {
    const int tid = threadIdx.x, H = a.c.n_kv_heads;
    unsigned long long all = 0, at = 0, size = 0;
    Lane l{0, 0, 0};
    LaneCost c{0, 0, 0, 0};
    auto scan_lanes = [&](int b0, bool tell) {
        const int b = b0 + tid;
        l = Lane{0, 0, 0};
        if (b < a.lanes) {
            bool bad;
            l = lane_facts(a, b, &bad);
            if (bad && tell && blockIdx.x == 0) record_error(a.err, MOE_DEV_BAD_PAGE);
        }
        c = lane_cost<D>(a, l);
        size = (unsigned long long)H * c.head();
        unsigned long long x = size, y = 0, tx, ty;
        scan2(x, y, scratch, &tx, &ty);
        at = all + x - size;
        all += tx;
    };
    for (int b0 = 0; b0 < a.lanes; b0 += (int)blockDim.x) scan_lanes(b0, true);
    const unsigned long long total = all;
    unsigned long long most = a.whole ? total : total / LEAST_PART;
    if (most < 1) most = 1;
    const int parts = most < gridDim.x ? (int)most : (int)gridDim.x;
    const unsigned long long first = (int)blockIdx.x < parts ? (unsigned long long)part_begin(total, parts, blockIdx.x) : total;
    const unsigned long long next = (int)blockIdx.x < parts ? (unsigned long long)part_begin(total, parts, blockIdx.x + 1) : total;
    if (tid < 2) here[tid] = Pos{a.lanes, 0, 0, 0};
    auto locate = [&](int b0) {                  // by the thread whose lane it is in
        for (int z = 0; z < 2; ++z) {
            const unsigned long long x = z ? next : first;
            if (x < at || x >= at + size) continue;
            const unsigned long long off = x - at, head = c.head();
            const int h = (off | head) >> 32 ? (int)(off / head) : (int)((uint32_t)off / (uint32_t)head);
            const unsigned long long rest = off - h * head;
            int lo = 0, hi = c.blocks - 1;       // the last block that begins at or before rest
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (c.upto(mid) <= rest) lo = mid; else hi = mid - 1;
            }
            int tile = 0;
            const unsigned long long in = rest - c.upto(lo);
            if (!a.whole && in > Cfg<D>::UNIT_COST) {
                const int left = (l.n - lo * a.block) * a.group;
                const int w = Cfg<D>::NT == 2 && left <= TILE ? HALF_COST : FULL_COST;
                tile = (int)((uint32_t)((in - Cfg<D>::UNIT_COST) / TILE) / (uint32_t)w);
            }
            here[z] = Pos{b0 + tid, h * c.blocks + lo, tile, 0};
        }
    };
    __syncthreads();
    if (a.lanes <= (int)blockDim.x) {
        locate(0);
    } else {
        all = 0;
        for (int b0 = 0; b0 < a.lanes; b0 += (int)blockDim.x) {
            scan_lanes(b0, false);
            locate(b0);
        }
    }
    __syncthreads();
    if (tid == 0 && !a.whole) {
        Pos* to = reinterpret_cast<Pos*>(a.ws);
        to[blockIdx.x] = here[0];
        if (blockIdx.x == gridDim.x - 1) to[gridDim.x] = here[1];
    }
}

template <int D>
__global__ void __launch_bounds__(640, 1) chunk_attention(const __grid_constant__ ChunkMaps maps, const __grid_constant__ ChunkArgs a) {
    using C = Cfg<D>;
    constexpr int NK = C::NK, NR = C::NR, NB = C::NB, NSC = C::NSC, QB = C::QB, ROWS = C::ROWS;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    const uint32_t base = smem_u32(smem), stop = base + C::OFF_MISC + 4;
    auto bar = [&](int offset, uint32_t i = 0) { return base + offset + 8 * i; };
    auto bar_ptr = [&](int offset) { return reinterpret_cast<uint64_t*>(smem + offset); };
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 4);
    volatile uint32_t* progress = reinterpret_cast<volatile uint32_t*>(smem + C::OFF_MISC + 8);      // items of the two buffers; parts out
    Pos* ends = reinterpret_cast<Pos*>(smem + C::OFF_MISC + 32);

    const int tid = threadIdx.x, warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0), lane = tid & 31;
    const int G = a.group;
    pdl_trigger();
    if (tid == 0) {
        auto init = [&](int offset, int n, int arrivals) {
            for (int i = 0; i < n; ++i) mbar_init(bar_ptr(offset) + i, arrivals);
        };
        init(C::B_KFULL, NK, 1); init(C::B_KEMPTY, NK, 2); init(C::B_RFULL, NR, 1); init(C::B_REMPTY, NR, 4);
        init(C::B_BFULL, NB, 4); init(C::B_BEMPTY, NB, 2); init(C::B_SCFULL, NSC, 1); init(C::B_SCEMPTY, NSC, 16);
        init(C::B_SFULL, 4, 1); init(C::B_PFULL, 4, 4); init(C::B_OHALF, 2, 1); init(C::B_ODONE, 2, 1); init(C::B_QFULL, QB, 8); init(C::B_QFREE, 1, 2);
        init(C::B_QMAX, 1, 8); init(C::B_PDFULL, C::NPD, 1); init(C::B_PDEMPTY, C::NPD, 19); init(C::B_MERGE, 1, 8); init(C::B_DONE, 1, 8); init(C::B_DRAIN, 2, 1);
        *abort_flag = 0;
        progress[0] = progress[1] = progress[2] = 0;
        fence_barrier_init();
        prefetch_tmap(&maps.k);
        prefetch_tmap(&maps.v);
    }
    if (warp == 17) { tmem_alloc(tmem_slot, 512); tmem_relinquish(); }
    if (tid < 32) *reinterpret_cast<float*>(smem + C::OFF_ONE + tid * 4) = 1.0f;
    pdl_wait();
    cut_run<D>(a, reinterpret_cast<unsigned long long*>(smem + C::OFF_Q), ends);      // (the queries' room, not yet in use)
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    // The n-th part of this CTA, for a whole warp; false: there is none, or the block has been stopped.
    auto part_at = [&](uint32_t n, Part& p) -> bool {
        if (!warp_wait_at(bar(C::B_PDFULL, n % C::NPD), (n / C::NPD) & 1, stop)) return false;
        const int4* from = reinterpret_cast<const int4*>(smem + C::OFF_PD + (n % C::NPD) * sizeof(Part));
        *reinterpret_cast<int4*>(&p.b) = from[0];
        *reinterpret_cast<int4*>(&p.rows) = from[1];
        *reinterpret_cast<int4*>(&p.t0) = from[2];
        __syncwarp();
        if (lane == 0) arrive_at(bar(C::B_PDEMPTY, n % C::NPD));
        return p.t1 > 0;
    };
    uint32_t issued_k = 0, issued_r = 0;             // ring fills, by the producer

    if (warp < 8) {
        // ------------------------------------------------------------ softmax: a thread is a row
        regs_up<C::SOFT_REGS>();
        const int g = warp >> 2, wl = warp & 3, j = tid & 127;
        const uint32_t trow = tmem + ((uint32_t)(wl * 32) << 16);
        uint32_t items = 0, tiles = 0, piece = 0;    // of the CTA: items (tile, row tile), tiles, parts
        bool ok = true;
        Part x;
        while (ok && part_at(piece, x)) {
            const int t0 = x.t0, t1 = x.t1, nt = t1 - t0;
            {
                // (a group that has no rows here waits too: it may not run ahead of barriers whose phases it does not see)
                if (!warp_wait_at(bar(C::B_QFULL, piece % QB), (piece / QB) & 1, stop)) break;
                // Two row tiles: one a group. One: the groups take its tiles in turn, each with an O of its own, which are added up
                // at the end (at head_dim 256 there is room for one O: group 0 takes them all).
                const bool split = C::NT == 2 && x.nt == 1;
                if (split || g < x.nt) {
                    const uint32_t o_at = trow + C::TMEM_O + g * (C::NT == 2 ? D : 0);
                    const int tile_row = split ? 0 : g * TILE, row = tile_row + j;
                    const int u = row < x.rows ? row : x.rows - 1;
                    const int t = (int)((uint32_t)u * a.by_group >> 16);
                    const int limit = x.first + t;                   // the last cache row that this row sees
                    const int open = x.first + (int)((uint32_t)tile_row * a.by_group >> 16);         // that every row of the tile sees
                    const float2 unit = *reinterpret_cast<const float2*>(smem + C::OFF_QU + (piece % QB) * 8);
                    const bool rowwise = unit.y != 0.0f;
                    const float rf = rowwise ? *reinterpret_cast<const float*>(smem + C::OFF_QF + ((piece % QB) * ROWS + row) * 4) : 1.0f;
                    const f32x2 rf2 = pack2(rf, rf);
                    float m = NEVER, l = 0.0f;
                    bool fresh = true;               // nothing has been added to O
                    uint32_t item = 0;
                    auto weigh = [&](auto two) {
                        for (int i = split ? (int)((items ^ (uint32_t)g) & 1) : 0; i < nt; i += split ? 2 : 1) {
                            item = split ? items + i : items + i * x.nt + g;
                            const uint32_t buf = item & 1, sc = (tiles + i) % NSC;
                            const uint32_t s_at = trow + buf * TILE;
                            const int j0 = (t0 + i) * TILE;
                            const bool masked = j0 + TILE - 1 > open;
                            const int rel = limit - j0;                  // columns up to rel are seen
                            if (!warp_wait_at(bar(C::B_SCFULL, sc), ((tiles + i) / NSC) & 1, stop)) { ok = false; break; }
                            auto scores_at = [&](int h) {
                                if (!warp_wait_at(bar(C::B_SFULL, 2 * buf + h), (item >> 1) & 1, stop)) return ok = false;
                                tc_fence_after();
                                return true;
                            };
                            const uint4* kf = reinterpret_cast<const uint4*>(smem + C::OFF_SC + sc * C::SC_BYTES + 2 * TILE);
                            // Half a tile at a time: its weights are at work, and the next tile's scores of that half are made, beside the
                            // other half's softmax.
                            auto publish = [&](int h) {
                                tc_wait_st();
                                tc_fence_before();
                                __syncwarp();
                                if (lane == 0) arrive_at(bar(C::B_PFULL, 2 * buf + h));
                            };
                            // The reference moves to `most`, the largest score so far, and what has been added up with it.
                            auto refer = [&](float most, int h) {
                                const float mn = fmaxf(m, most);
                                const float alpha = ex2(m - mn);
                                l *= alpha;
                                m = mn;
                                if (fresh) return true;
                                const uint32_t before_it = item - C::NT;
                                if (h > 0 ? !warp_wait_at(bar(C::B_OHALF, buf), (item >> 1) & 1, stop)
                                          : !warp_wait_at(bar(C::B_ODONE, before_it & 1), (before_it >> 1) & 1, stop)) return ok = false;
                                tc_fence_after();
#pragma unroll 1
                                for (int c = 0; c < D / 16; ++c) {
                                    uint32_t o[16];
                                    tc_load(o_at + c * 16, o);
#pragma unroll
                                    for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                                    tc_st_x8(o_at + c * 16, make_uint4(o[0], o[1], o[2], o[3]), make_uint4(o[4], o[5], o[6], o[7]));
                                    tc_st_x8(o_at + c * 16 + 8, make_uint4(o[8], o[9], o[10], o[11]), make_uint4(o[12], o[13], o[14], o[15]));
                                }
                                tc_wait_st();
                                return true;
                            };
                            // 32 columns of scores to weights
                            f32x2 sum0, sum1;
                            float top0, top1;
                            auto weights = [&](auto plain, uint32_t (&s)[32], uint32_t* P, const uint4* k8, f32x2 f2, float m, int seen) {
                                const f32x2 m2 = pack2(-m, -m);
#pragma unroll
                                for (int e = 0; e < 16; ++e) {
                                    const uint4 kk = k8[e / 2];
                                    f32x2 y = pack2(__uint_as_float(s[2 * e]), __uint_as_float(s[2 * e + 1]));
                                    if constexpr (!plain) y = mul2_loaded(y, f2);
                                    y = fma2_loaded(y, e & 1 ? pack2(__uint_as_float(kk.z), __uint_as_float(kk.w)) : pack2(__uint_as_float(kk.x), __uint_as_float(kk.y)), m2);
                                    float2 v = unpack2(y);
                                    if constexpr (!plain) {
                                        if (2 * e > seen) v.x = -INFINITY;
                                        if (2 * e + 1 > seen) v.y = -INFINITY;
                                    }
                                    const float p0 = ex2(v.x), p1 = ex2(v.y);
                                    if (e & 1) {
                                        top1 = max3(top1, v.x, v.y);
                                        sum1 = add2(sum1, pack2(p0, p1));
                                    } else {
                                        top0 = max3(top0, v.x, v.y);
                                        sum0 = add2(sum0, pack2(p0, p1));
                                    }
                                    P[e] = pack_bf16(p0, p1);
                                }
                            };
                            auto clear = [&]() {
                                top0 = top1 = -INFINITY;
                                sum0 = sum1 = 0ull;
                            };
                            auto passes = [&]() { return __any_sync(0xFFFFFFFFu, fmaxf(top0, top1) > LIMIT); };
                            auto add_up = [&]() {
                                const float2 p = unpack2(add2(sum0, sum1));
                                l += p.x + p.y;
                            };
                            int h = 0;                   // the half that is to be done
                            if constexpr (two) {
                                // Weights in two parts, in one form: the scores in place of what the MMA left, their largest, then the weights, eight
                                // columns' first and second parts at a time (all at once would not fit the registers).
#pragma unroll 1
                                for (; h < 2; ++h) {
                                    const uint32_t sh = s_at + h * 64;
                                    const uint4* kh = kf + 16 * h;
                                    if (!scores_at(h)) break;
                                    uint32_t s[64];
                                    tc_ld_x32(sh, *reinterpret_cast<uint32_t (*)[32]>(s));
                                    tc_ld_x32(sh + 32, *reinterpret_cast<uint32_t (*)[32]>(s + 32));
                                    tc_wait_ld();
                                    clear();
#pragma unroll
                                    for (int e = 0; e < 32; ++e) {
                                        const uint4 kk = kh[e / 2];
                                        const f32x2 y = mul2_loaded(pack2(__uint_as_float(s[2 * e]), __uint_as_float(s[2 * e + 1])), rf2);
                                        const float2 v = unpack2(mul2(y, e & 1 ? pack2(__uint_as_float(kk.z), __uint_as_float(kk.w)) : pack2(__uint_as_float(kk.x), __uint_as_float(kk.y))));
                                        s[2 * e] = __float_as_uint(v.x);
                                        s[2 * e + 1] = __float_as_uint(v.y);
                                    }
                                    if (masked) {
                                        const int seen = rel - 64 * h;
#pragma unroll
                                        for (int e = 0; e < 64; ++e)
                                            if (e > seen) s[e] = 0xFF800000u;
                                    }
#pragma unroll
                                    for (int e = 0; e < 64; e += 4) {
                                        top0 = max3(top0, __uint_as_float(s[e]), __uint_as_float(s[e + 1]));
                                        top1 = max3(top1, __uint_as_float(s[e + 2]), __uint_as_float(s[e + 3]));
                                    }
                                    const float most = fmaxf(top0, top1);
                                    if ((fresh || __any_sync(0xFFFFFFFFu, most > m + LIMIT)) && !refer(most, h)) break;
                                    const f32x2 m2 = pack2(-m, -m);
#pragma unroll
                                    for (int e = 0; e < 64; e += 16) {
                                        uint32_t P[16];
#pragma unroll
                                        for (int z = 0; z < 8; ++z) {
                                            const float2 v = unpack2(add2(pack2(__uint_as_float(s[e + 2 * z]), __uint_as_float(s[e + 2 * z + 1])), m2));
                                            const float p0 = ex2(v.x), p1 = ex2(v.y);
                                            if (z & 1) sum1 = add2(sum1, pack2(p0, p1)); else sum0 = add2(sum0, pack2(p0, p1));
                                            P[z] = pack_bf16(p0, p1);
                                            P[8 + z] = pack_bf16(p0 - __uint_as_float(P[z] << 16), p1 - __uint_as_float(P[z] & 0xFFFF0000u));
                                        }
                                        tc_st_x8(sh + e / 2, make_uint4(P[0], P[1], P[2], P[3]), make_uint4(P[4], P[5], P[6], P[7]));
                                        tc_st_x8(sh + 32 + e / 2, make_uint4(P[8], P[9], P[10], P[11]), make_uint4(P[12], P[13], P[14], P[15]));
                                    }
                                    add_up();
                                    publish(h);
                                    fresh = false;
                                }
                            } else {
                                // Most tiles: no edge, no factor of the row's, the reference stays. (A form of its own: with branches within, the
                                // scores are copied from where the loads leave them, two moves a pair. A loop, though the second half's scores
                                // could come ahead: the instructions' cache is as scarce.)
                                if (!fresh && !masked && !rowwise)
#pragma unroll 1
                                    for (; h < 2; ++h) {
                                        if (!scores_at(h)) break;
                                        uint32_t sa[32], sb[32], P[32];
                                        tc_ld_x32(s_at + h * 64, sa);
                                        tc_ld_x32(s_at + h * 64 + 32, sb);
                                        tc_wait_ld();
                                        clear();
                                        weights(std::true_type{}, sa, P, kf + 16 * h, 0ull, m, 0);
                                        weights(std::true_type{}, sb, P + 16, kf + 16 * h + 8, 0ull, m, 0);
                                        if (passes()) break;
                                        add_up();
                                        tc_st_x32(s_at + 64 * h, P);
                                        publish(h);
                                    }
                                if (!ok) break;
#pragma unroll 1
                                for (; h < 2; ++h) {
                                    const int seen = masked ? rel - 64 * h : TILE;   // columns of this half up to here are seen
                                    const uint32_t sh = s_at + h * 64;
                                    const uint4* kh = kf + 16 * h;           // the factors of the columns' scores,
                                    int next8 = 8;
                                    f32x2 f2 = rf2;                          // and of the row's
                                    if (!scores_at(h)) break;
                                    uint32_t sa[32], sb[32], P[32];
                                    if (!fresh && __all_sync(0xFFFFFFFFu, seen < 0)) {       // behind the edge of all 32 rows
#pragma unroll
                                        for (int e = 0; e < 32; ++e) P[e] = 0u;
                                        tc_st_x32(sh, P);
                                        publish(h);
                                        continue;
                                    }
                                    tc_ld_x32(sh, sa);
                                    tc_ld_x32(sh + 32, sb);
                                    tc_wait_ld();
                                    bool move = fresh;
                                    for (bool moved = false;; moved = true) {
                                        if (move) {
                                            float most = -INFINITY;
                                            auto largest = [&](uint32_t (&s)[32], const uint4* k8, int seen) {
#pragma unroll
                                                for (int e = 0; e < 16; ++e) {
                                                    const uint4 kk = k8[e / 2];
                                                    const f32x2 y = mul2_loaded(pack2(__uint_as_float(s[2 * e]), __uint_as_float(s[2 * e + 1])), f2);
                                                    const float2 v = unpack2(mul2(y, e & 1 ? pack2(__uint_as_float(kk.z), __uint_as_float(kk.w)) : pack2(__uint_as_float(kk.x), __uint_as_float(kk.y))));
                                                    s[2 * e] = __float_as_uint(v.x);
                                                    s[2 * e + 1] = __float_as_uint(v.y);
                                                    most = max3(most, 2 * e <= seen ? v.x : -INFINITY, 2 * e + 1 <= seen ? v.y : -INFINITY);
                                                }
                                            };
                                            largest(sa, kh, seen);
                                            largest(sb, kh + 8, seen - 32);
                                            // They are rounded now, and their difference to the largest is exact: a fused one would leave the product's
                                            // last bits, which of scores past 2^31 alone make a weight infinite.
                                            kh = reinterpret_cast<const uint4*>(smem + C::OFF_ONE);
                                            next8 = 0;
                                            f2 = pack2(1.0f, 1.0f);
                                            if (!refer(most, h)) break;
                                        }
                                        clear();
                                        weights(std::false_type{}, sa, P, kh, f2, m, seen);
                                        weights(std::false_type{}, sb, P + 16, kh + next8, f2, m, seen - 32);
                                        tc_st_x32(sh, P);
                                        move = passes();
                                        if (moved || !move) {
                                            add_up();
                                            break;
                                        }
                                    }
                                    if (!ok) break;
                                    publish(h);
                                    fresh = false;
                                }
                            }
                            if (!ok) break;
                            if (lane == 0) arrive_at_n(bar(C::B_SCEMPTY, sc), x.nt == 2 ? 1 : 2);
                        }
                    };
                    if (__builtin_expect(x.two, 0)) weigh(std::true_type{}); else weigh(std::false_type{});
                    if (!ok) break;
                    // ---- the part's output
                    if (!fresh && !warp_wait_at(bar(C::B_ODONE, item & 1), (item >> 1) & 1, stop)) break;
                    tc_fence_after();
                    const bool live = row < x.rows, whole = t0 == 0 && t1 == x.tiles;
                    float f0 = fresh ? 0.0f : 1.0f, f1 = 0.0f;       // factors of this group's O and of the other's
                    if (split) {
                        // One row, two O: in the same lanes of TMEM, where each group reads both, of half the columns.
                        float2* ml = reinterpret_cast<float2*>(smem + C::OFF_ML);
                        ml[g * TILE + j] = make_float2(m, l);
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) arrive_at(bar(C::B_MERGE));
                        if (!warp_wait_at(bar(C::B_MERGE), 0, stop)) break;
                        tc_fence_after();
                        const float2 other = ml[(1 - g) * TILE + j];
                        const float mn = fmaxf(m, other.x);
                        if (m != NEVER || l != 0.0f) f0 = ex2(m - mn);
                        if (other.x != NEVER || other.y != 0.0f) f1 = ex2(other.x - mn);
                        const float mine = l * f0, theirs = other.y * f1;
                        l = mine + theirs;
                        m = mn;
                    }
                    float* part = nullptr;           // where this thread's row lies in a part, in the workspace
                    uint4* dst = nullptr;            // or in the output
                    if (whole) {
                        const int64_t to = (int64_t)(x.tok0 + t) * a.n_q + x.h * G + u - t * G;
                        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
                        if (a.lse && live && (!split || g == 0)) a.lse[to] = l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
                        f0 *= inv;
                        f1 *= inv;
                        dst = reinterpret_cast<uint4*>(a.out + to * D);
                    } else {
                        part = reinterpret_cast<float*>(a.ws + parts_offset(gridDim.x)) + (size_t)(2 * blockIdx.x + (t0 > 0 ? 0 : 1)) * C::PART_FLOATS;
                        if (live && (!split || g == 0)) {
                            part[ROWS * D + row] = m;
                            part[ROWS * D + ROWS + row] = l;
                        }
                    }
                    // (A factor of 0: nothing has been added up there. A row without a weight has zeros.)
                    const int cn = split ? D / 64 : D / 32, c0 = split ? g * cn : 0;
                    if (__any_sync(0xFFFFFFFFu, live))
#pragma unroll 1
                        for (int c = c0; c < c0 + cn; ++c) {
                            uint32_t o[32];
                            __syncwarp();
                            tc_load(o_at + c * 32, o);
                            float v[32];
#pragma unroll
                            for (int e = 0; e < 32; ++e) v[e] = f0 == 0.0f ? 0.0f : __uint_as_float(o[e]) * f0;
                            if (split) {
                                tc_load(trow + C::TMEM_O + (1 - g) * D + c * 32, o);
                                if (f1 != 0.0f)
#pragma unroll
                                    for (int e = 0; e < 32; ++e) v[e] = fmaf(__uint_as_float(o[e]), f1, v[e]);
                            }
                            if (live && whole) {
#pragma unroll
                                for (int e = 0; e < 32; e += 16)
                                    store_32(dst + c * 4 + e / 8, pack_bf16(v[e], v[e + 1]), pack_bf16(v[e + 2], v[e + 3]), pack_bf16(v[e + 4], v[e + 5]),
                                             pack_bf16(v[e + 6], v[e + 7]), pack_bf16(v[e + 8], v[e + 9]), pack_bf16(v[e + 10], v[e + 11]),
                                             pack_bf16(v[e + 12], v[e + 13]), pack_bf16(v[e + 14], v[e + 15]));
                            } else if (live) {
#pragma unroll
                                for (int e = 0; e < 8; ++e)
                                    *reinterpret_cast<float4*>(part + ((size_t)(c * 8 + e) * ROWS + row) * 4) = make_float4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
                            }
                        }
                    if (split) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) arrive_at(bar(C::B_MERGE));
                        if (!warp_wait_at(bar(C::B_MERGE), 1, stop)) break;
                        tc_fence_after();
                    }
                    tc_fence_before();
                    if (lane == 0 && wl == 0 && g == 0) progress[2] = piece + 1;
                }
                items += nt * x.nt;
                tiles += nt;
                ++piece;
            }
        }
        tc_wait_ld();
        __syncwarp();
        if (lane == 0) arrive_at(bar(C::B_DONE));
    } else if (warp < 16) {
        // ------------------------------------------------------------ queries in two parts; values in bf16
        regs_down<C::CONV_REGS>();
        const int wl = warp - 8, cg = wl >> 2, ct = tid & 127;       // of both groups; group
        // A unit's queries go through twice: for the largest size of each row (while the part before is at work, a few rows
        // with each piece of its values), then for the parts.
        constexpr int LPR = D / 8, RPW = 32 / LPR, STEP = 8 * RPW;            // lanes a row, rows a warp takes at once, all eight
        constexpr int BATCH = 4;                                              // loads under way
        const int part = lane % LPR, mine = wl * RPW + lane / LPR;
        auto place = [&](const Part& x, int u) {     // (rows past the unit's last are its last again, and their results nobody's)
            u = min(u, x.rows - 1);
            const int t = (int)((uint32_t)u * a.by_group >> 16);
            return reinterpret_cast<const uint4*>(a.q + (int64_t)(x.tok0 + t) * a.q_token + (int64_t)(x.h * G + u - t * G) * a.q_head + part * 8);
        };
        // A row's bf16 values take as many bytes as its two parts: they come asynchronously, all at once, to where the parts
        // will lie (an eighth of the segments to a lane), and the row's lanes then replace them.
        constexpr int SEG = C::ROWB / 16;            // lanes a segment
        auto row_at = [&](int u) { return C::OFF_Q + (u >> 7) * C::QTILE + (u & (TILE - 1)) * C::ROWB; };
        const int raw_at = part / SEG / 2 * C::QPANEL + (part / SEG & 1) * TILE * C::ROWB + part % SEG * 16;
        auto fetch = [&](const Part& x) {
#pragma unroll 1
            for (int u = mine; u < x.nt * TILE; u += STEP) cp_async_16(base + row_at(u) + raw_at, place(x, u));
            cp_async_commit();
            cp_async_wait<0>();
        };
        auto row_factors = [&](uint32_t n) { return reinterpret_cast<float*>(smem + C::OFF_QF) + (n % QB) * ROWS; };
        uint32_t most = 0, least = 0x7FFFu;          // sizes of the next part's rows, as bf16 bits
        auto sizes = [&](const uint4 (&raw)[BATCH], uint32_t n, int r0) {
            uint32_t* keys = reinterpret_cast<uint32_t*>(row_factors(n));
#pragma unroll
            for (int b = 0; b < BATCH; ++b) {
                auto abs2 = [](uint32_t v) {
                    v &= 0x7FFF7FFFu;
                    return *reinterpret_cast<const __nv_bfloat162*>(&v);
                };
                __nv_bfloat162 v = __hmax2_nan(__hmax2_nan(abs2(raw[b].x), abs2(raw[b].y)), __hmax2_nan(abs2(raw[b].z), abs2(raw[b].w)));
                v = __hmax2_nan(v, __lowhigh2highlow(v));
#pragma unroll
                for (int o = LPR / 2; o > 0; o >>= 1) v = __hmax2_nan(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
                const uint32_t key = *reinterpret_cast<const uint32_t*>(&v) & 0xFFFFu;
                if (part == 0) keys[(r0 + b) * STEP + mine] = key;
                most = max(most, key);
                if (key) least = min(least, key);
            }
        };
        auto prepare = [&](const Part& x, uint32_t n) -> bool {
            uint32_t* qx = reinterpret_cast<uint32_t*>(smem + C::OFF_QX) + (n & 1) * 16;
            most = __reduce_max_sync(0xFFFFFFFFu, most);
            least = __reduce_min_sync(0xFFFFFFFFu, least);
            if (lane == 0) {
                qx[wl] = most;
                qx[8 + wl] = least;
                arrive_at(bar(C::B_QMAX));
            }
            if (!warp_wait_at(bar(C::B_QMAX), n & 1, stop)) return false;
#pragma unroll
            for (int w = 0; w < 8; ++w) {
                most = max(most, qx[w]);
                least = min(least, qx[8 + w]);
            }
            // Rows within 2^4 of one another share one power of two, and the scores need no factor of their row's; the
            // smallest rows' low parts then end 2^-13 below their own maximum. (Subnormal rows count as 2^-126.)
            auto up_of = [](uint32_t k) {            // 2^up * maximum is in [128, 256)
                const int up = k ? 134 - (int)(k >> 7) : 0;
                return up > 120 ? 120 : (up < -120 ? -120 : up);
            };
            const int unit_up = up_of(most);
            const bool rowwise = most >= 0x7F80u || (least < most && up_of(least) - unit_up > 4);
            most = 0;
            least = 0x7FFFu;
            float* qf = row_factors(n);
            const uint32_t* keys = reinterpret_cast<const uint32_t*>(qf);
            if (wl == 0 && lane == 0)
                *reinterpret_cast<float2*>(smem + C::OFF_QU + (n % QB) * 8) = make_float2(rowwise ? 1.0f : exp2_int(-unit_up), rowwise ? 1.0f : 0.0f);
            const int rounds = x.nt * TILE / STEP;
            const int panel = part * 8 / C::ROWB, chunk = part * 8 % C::ROWB / 16;
            if (n > 0) {
                if (!warp_wait_at(bar(C::B_QFREE), (n - 1) & 1, stop)) return false;
                fetch(x);
            }
            // 1 / 2 / 4: a prompt of 8192 tokens 484 / 479 / 518 us, at head_dim 256 1060 / 1031 / 1049; 24 of 1024 at 64 158 / 167 / 175
            constexpr int AT_ONCE = D > 64 ? 2 : 1;
#pragma unroll 1
            for (int r = 0; r < rounds; r += AT_ONCE) {
                uint4 raw[AT_ONCE];
                uint32_t key[AT_ONCE];
#pragma unroll
                for (int z = 0; z < AT_ONCE; ++z) {
                    const int u = (r + z) * STEP + mine;
                    raw[z] = *reinterpret_cast<const uint4*>(smem + row_at(u) + raw_at);
                    key[z] = rowwise ? keys[u] : 0u;
                }
                __syncwarp();
#pragma unroll
                for (int z = 0; z < AT_ONCE; ++z) {
                    const int u = (r + z) * STEP + mine;
                    const int up = rowwise ? up_of(key[z]) : unit_up;
                    const float gain = exp2_int(up);
                    const f32x2 gain2 = pack2(gain, gain);
                    const uint32_t in[4] = {raw[z].x, raw[z].y, raw[z].z, raw[z].w};
                    uint32_t hi[4], lo[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        // a scaled bf16 value is exact in fp16 (down to 2^-16, far below what lo resolves)
                        const float2 v = unpack2(mul2(pack2(__uint_as_float(in[e] << 16), __uint_as_float(in[e] & 0xFFFF0000u)), gain2));
                        const __half2 vh = __floats2half2_rn(v.x, v.y);
                        hi[e] = __nv_cvt_halfraw2_to_fp8x2(vh, __NV_SATFINITE, __NV_E4M3);
                        const __half2 rest = __hsub2(vh, __half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)hi[e], __NV_E4M3)));
                        lo[e] = __nv_cvt_halfraw2_to_fp8x2(rest, __NV_SATFINITE, __NV_E4M3);
                    }
                    // a row that is not finite: its scores become NaN
                    if (rowwise && part == 0) qf[u] = key[z] >= 0x7F80u ? __uint_as_float(0x7FC00000u) : exp2_int(-up);
                    const int swz = C::ROWB == 128 ? u & 7 : (u >> 1) & 3;
                    uint8_t* to = smem + row_at(u) + panel * C::QPANEL + ((chunk ^ swz) << 4) + (part & 1) * 8;
                    *reinterpret_cast<uint2*>(to) = make_uint2(__byte_perm(hi[0], hi[1], 0x5410), __byte_perm(hi[2], hi[3], 0x5410));
                    *reinterpret_cast<uint2*>(to + TILE * C::ROWB) = make_uint2(__byte_perm(lo[0], lo[1], 0x5410), __byte_perm(lo[2], lo[3], 0x5410));
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) arrive_at(bar(C::B_QFULL, n % QB));
            return true;
        };
        // One piece of values (of the part's, the group's i-th): codes to bf16.
        constexpr int MINE = C::PIECES / 2;          // pieces of a tile that are this group's
        uint32_t tile = 0;                           // of the CTA
        auto convert = [&](const Part& x, int i) -> bool {
            const int pc = i % MINE * 2 + cg, t = x.t0 + i / MINE;
            const uint32_t pieces = tile * C::PIECES + pc, sc = tile % NSC, rs = pieces % NR, bs = pieces % NB;
            if (pc < 2 && !warp_wait_at(bar(C::B_SCFULL, sc), (tile / NSC) & 1, stop)) return false;
            if (!warp_wait_at(bar(C::B_RFULL, rs), (pieces / NR) & 1, stop)) return false;
            if (!warp_wait_at(bar(C::B_BEMPTY, bs), ((pieces / NB) & 1) ^ 1, stop)) return false;
            const uint8_t* bytes = smem + C::OFF_SC + sc * C::SC_BYTES + TILE + pc * C::VR;
            constexpr int EACH = C::VR * D / 16 / 128;                       // 16 codes at once, of a thread
            const int left = x.end - t * TILE - pc * C::VR;                  // rows that somebody sees; what lies behind is anything
            // One after the other: two or four at once cost more in instruction fetches than they save (1 / 2 / 4: a prompt of 8192 tokens
            // 457 / 459 / 468 us, 24 prompts of 1024 at head_dim 64 158 / 163 / 163). Not so at head_dim 256, where a tile of values serves
            // 128 rows alone: 1057 / 1074 / 988, 1024 tokens over 30,000 1125 / 1145 / 1053.
            constexpr int AT_ONCE = D == 256 ? 4 : 1;
#pragma unroll AT_ONCE
            for (int e = 0; e < EACH; ++e) {
                // Eight neighbours take four places of a row in one panel of 64 columns and four of the next row in the
                // next panel: all on different banks, where they read and where they write.
                const int i = e * 128 + ct;
                int row = i >> 2, panel = 0;
                if constexpr (D > 64) {
                    constexpr int HP = D / 128;
                    const int rest = i >> 4, odd = (i >> 2) & 1;
                    row = rest / HP * 2 + odd;
                    panel = rest % HP * 2 + (((i >> 3) & 1) ^ odd);
                }
                const uint4 raw = *reinterpret_cast<const uint4*>(smem + C::OFF_R + rs * C::RSLOT + row * D + panel * 64 + (i & 3) * 16);
                const uint32_t s = bytes[row];
                // e4m3's bits, moved to bf16's places, stand for the code times 2^-120
                uint32_t f = s <= 134u ? (s + 120u) << 7 : 0x7F00u;
                if (s == 0u || row >= left) f = 0u;
                f |= f << 16;
                const uint32_t in[4] = {raw.x, raw.y, raw.z, raw.w};
                uint32_t v[8];
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    // the upper bytes (sign, upper exponent bits) and the lower ones (last exponent bit, mantissa) of four values
                    const uint32_t hi = (in[w] & 0x80808080u) | ((in[w] >> 4) & 0x07070707u), lo = (in[w] & 0x0F0F0F0Fu) * 16u;
                    v[2 * w] = mul_bf16x2(__byte_perm(lo, hi, 0x5140), f);
                    v[2 * w + 1] = mul_bf16x2(__byte_perm(lo, hi, 0x7362), f);
                }
                if (s > 134u) {
                    const uint32_t f2 = ((s - 7u) << 7) * 0x10001u;
#pragma unroll
                    for (int w = 0; w < 8; ++w) v[w] = mul_bf16x2(v[w], f2);
                }
                uint8_t* to = smem + C::OFF_B + bs * C::BSLOT + panel * C::VPANEL + row * 128;
                const int q0 = (i & 3) * 2;
                *reinterpret_cast<uint4*>(to + ((q0 ^ (row & 7)) << 4)) = make_uint4(v[0], v[1], v[2], v[3]);
                *reinterpret_cast<uint4*>(to + (((q0 + 1) ^ (row & 7)) << 4)) = make_uint4(v[4], v[5], v[6], v[7]);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                arrive_at(bar(C::B_BFULL, bs));
                arrive_at(bar(C::B_REMPTY, rs));
                if (pc >= C::PIECES - 2) arrive_at(bar(C::B_SCEMPTY, sc));
            }
            if (pc >= C::PIECES - 2) ++tile;
            return true;
        };
        Part x{}, nx;
        bool ok = true, more = part_at(0, nx);
        if (more) fetch(nx);                         // (of the first part from where they will lie)
        for (uint32_t n = 0; ok; ++n) {              // the values of part n - 1 (none), with them the next queries' sizes; then these
            const int todo = (x.t1 - x.t0) * MINE, batches = more ? nx.nt * TILE / STEP / BATCH : 0;
#pragma unroll 1
            for (int i = 0; i < todo || i < batches; ++i) {
                uint4 raw[BATCH];
                if (i < batches)
#pragma unroll
                    for (int b = 0; b < BATCH; ++b) {
                        const int u = (i * BATCH + b) * STEP + mine;
                        raw[b] = *(n == 0 ? reinterpret_cast<const uint4*>(smem + row_at(u) + raw_at) : place(nx, u));
                    }
                if (i < todo && !convert(x, i)) { ok = false; break; }
                if (i < batches) sizes(raw, n, i * BATCH);
            }
            if (!ok || !more) break;
            x = nx;
            if (!prepare(x, n)) break;
            more = part_at(n + 1, nx);
        }
    } else {
        regs_down<C::REST_REGS>();
        const int P = 1 << a.page_shift;
        auto checked = [&](int page, bool tell) {
            if (page >= 0 && page < a.c.n_pages) return page;
            if (tell) record_error(a.err, MOE_DEV_BAD_PAGE);
            return 0;
        };
        if (warp == 16) {
            // -------------------------------------------------------- TMA: lane l < 8 looks up the page of the tile's rows 16 l ..
            const int rk = P < TILE ? P : TILE, rv = P < C::VR ? P : C::VR;          // rows a copy
            const Pos end = ends[1];
            Pos at = ends[0];
            int units = 0;
            bool ok = true;
            Part x{}, nx{};
            for (uint32_t n = 0; ok; ++n) {          // tells part n, then copies part n - 1: the next queries are looked at early
                if (n == 0 || x.t1 > 0) {
                    nx = next_part<D>(a, end, at, units);
                    if (!warp_wait_at(bar(C::B_PDEMPTY, n % C::NPD), ((n / C::NPD) & 1) ^ 1, stop)) break;
                    if (lane == 0) {
                        *reinterpret_cast<Part*>(smem + C::OFF_PD + (n % C::NPD) * sizeof(Part)) = nx;
                        arrive_at(bar(C::B_PDFULL, n % C::NPD));
                    }
                    __syncwarp();
                }
                if (n == 0) {
                    x = nx;
                    if (x.t1 == 0) break;
                    continue;
                }
                const int t0 = x.t0, t1 = x.t1, hp = x.h * P;
                const int32_t* table = a.table + (int64_t)x.b * a.width;
                auto look = [&](int t) {
                    const int j = t * TILE + lane * 16;
                    return lane < 8 && t < t1 && j < x.end ? table[j >> a.page_shift] : 0;
                };
                int id = look(t0);
                for (int t = t0; t < t1 && ok; ++t) {
                    const int next = look(t + 1);
                    const int j = t * TILE + lane * 16;
                    int row = 0;                     // this lane's first cache row
                    if (lane < 8 && j < x.end) row = checked(id, true) * a.c.n_kv_heads * P + hp + (j & (P - 1));
                    id = next;
                    {
                        const uint32_t s = issued_k % NK;
                        const int r = __shfl_sync(0xFFFFFFFFu, row, lane * rk / 16 & 31);
                        const bool some = lane * rk < TILE && t * TILE + lane * rk < x.end;
                        const uint32_t bytes = __popc(__ballot_sync(0xFFFFFFFFu, some)) * rk * D;
                        if (!warp_wait_at(bar(C::B_KEMPTY, s), ((issued_k / NK) & 1) ^ 1, stop)) { ok = false; break; }
                        if (lane == 0) arrive_expect_tx_at(bar(C::B_KFULL, s), bytes);
                        ++issued_k;
                        __syncwarp();
                        if (some)
#pragma unroll
                            for (int q = 0; q < C::PANELS; ++q)
                                tma_load_at(base + C::OFF_K + s * C::KSLOT + q * C::KPANEL + lane * rk * C::ROWB, &maps.k, bar(C::B_KFULL, s), q * 128, r);
                    }
#pragma unroll 1
                    for (int pc = 0; pc < C::PIECES; ++pc) {
                        const uint32_t s = issued_r % NR;
                        const int in = pc * C::VR + lane * rv;
                        const int first = __shfl_sync(0xFFFFFFFFu, row, in / 16 & 7);        // (a page of 1024 rows: the same one, further down)
                        const bool some = lane * rv < C::VR && t * TILE + in < x.end;
                        const uint32_t bytes = __popc(__ballot_sync(0xFFFFFFFFu, some)) * rv * D;
                        if (!warp_wait_at(bar(C::B_REMPTY, s), ((issued_r / NR) & 1) ^ 1, stop)) { ok = false; break; }
                        if (lane == 0) arrive_expect_tx_at(bar(C::B_RFULL, s), bytes);
                        ++issued_r;
                        __syncwarp();
                        if (some) tma_load_at(base + C::OFF_R + s * C::RSLOT + lane * rv * D, &maps.v, bar(C::B_RFULL, s), 0, first);
                    }
                }
                x = nx;
                if (x.t1 == 0) break;
            }
        } else if (warp < 19) {
            // -------------------------------------------------------- MMA issue: a warp for each buffer of S, which items (tile, row tile)
            // use in turn, half by half. (One warp for both has more to decide a step than the step's products take.) With one row
            // tile a warp sees every second tile only: the ring of keys has an even number of slots, so that the slot's fill before,
            // from whose parity the next one's differs, was its own too.
            constexpr uint64_t KD = desc_base(C::ROWB == 128 ? 2 : 4, 8 * C::ROWB, 8 * C::ROWB);
            constexpr uint64_t VD = desc_base(2, C::VPANEL, 1024);
            constexpr uint32_t ID_S = idesc_f8(TILE, C::NT == 2 ? TILE / 2 : TILE, 0, 0, 0), ID_PV = idesc_bf16(TILE, D);
            const uint32_t tm = __shfl_sync(0xFFFFFFFFu, tmem, 0);
            // A descriptor's lower word changes, its upper one is constant. Lower words go through a shuffle, which leaves them
            // in uniform registers: an MMA then costs its issue and no moves of its operands (four words each, 80 clocks).
            auto lower = [&](uint64_t kind, uint32_t at_byte) { return __shfl_sync(0xFFFFFFFFu, (uint32_t)kind + (at_byte >> 4), 0); };
            auto desc = [](uint64_t kind, uint32_t lo) {
                uint64_t d;
                asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(lo), "r"((uint32_t)(kind >> 32)));
                return d;
            };
            constexpr int PH = C::PIECES / 2;        // pieces of values of half a tile
            const int b = warp - 17;
            const uint32_t s_tm = __shfl_sync(0xFFFFFFFFu, tm + b * TILE, 0);        // this buffer's S
            uint32_t item = 0, tile = 0, piece = 0;  // of the CTA: the first item of the part, its first tile, part
            uint32_t mine = b;                       // this buffer's next item
            bool ok = true;
            Part x;
            for (; ok && part_at(piece, x); ++piece) {
                const int nt = __shfl_sync(0xFFFFFFFFu, x.nt, 0), tiles = __shfl_sync(0xFFFFFFFFu, x.t1 - x.t0, 0);
                const int two = __shfl_sync(0xFFFFFFFFu, x.two, 0);
                const uint32_t last = item + tiles * nt;
                if (mine < last && !warp_wait_at(bar(C::B_QFULL, piece % QB), (piece / QB) & 1, stop)) break;
                // This buffer's halves of the part in a row: half z's output, then the scores of half z + 2, which take its place in TMEM.
                const int halves = mine < last ? ((int)(last - mine) + 1) / 2 * 2 : 0;
                const uint32_t n0 = mine - item;
                // The second row tile begins when half of the first one's weights are there, and the groups then take turns at the
                // softmax. (A few looks: whether it has begun, and not how often since, is all that the barrier can tell.)
                if (nt == 2 && n0 == 1)
                    for (int z = 0; z < STAGGER && !__all_sync(0xFFFFFFFFu, test_at(bar(C::B_PFULL, 2 * (1 - b)), (item >> 1) & 1)); ++z) {}
                uint32_t k = 0, q = 0;
                auto keys = [&](uint32_t n) {        // waits for the keys of item n, and finds its operands
                    const uint32_t t = tile + (nt == 2 ? n >> 1 : n);
                    k = lower(KD, base + C::OFF_K + t % NK * C::KSLOT);
                    q = lower(KD, base + C::OFF_Q + (nt == 2 ? n & 1 : 0) * C::QTILE);
                    return warp_wait_at(bar(C::B_KFULL, t % NK), (t / NK) & 1, stop);
                };
#pragma unroll 1
                for (int z = -2; z < halves; ++z) {
                    const int h = z & 1;
                    // what the next scores need is found before the wait that the softmax ends
                    if (C::NT == 2 && h == 0 && z + 2 < halves && !keys(n0 + z + 2)) { ok = false; break; }
                    if (z >= 0) {
                        const uint32_t n = n0 + (z & ~1), at = mine + (z & ~1);
                        const uint32_t bi = (tile + (nt == 2 ? n >> 1 : n)) * C::PIECES + h * PH;
                        const uint32_t o = __shfl_sync(0xFFFFFFFFu, tm + C::TMEM_O + (C::NT == 2 && nt == 1 ? b : nt == 2 ? n & 1 : 0) * D, 0);
                        const uint32_t p = __shfl_sync(0xFFFFFFFFu, s_tm + h * 64, 0);
                        const uint32_t add = __shfl_sync(0xFFFFFFFFu, (C::NT == 2 ? n < 2 : n == 0) && h == 0 ? 0u : 1u, 0);
                        uint32_t v[PH];
#pragma unroll
                        for (int pc = 0; pc < PH; ++pc) v[pc] = lower(VD, base + C::OFF_B + (bi + pc) % NB * C::BSLOT);
                        // Outputs of one O add up in order: the other buffer's last is complete. (Its values then have arrived,
                        // without which the parity of the next ones' barriers would say nothing.)
                        if (C::NT == 1 && h == 0 && at > 0 &&
                            (!warp_wait_at(bar(C::B_PFULL, 2 * b), (at >> 1) & 1, stop) ||
                             !warp_wait_at(bar(C::B_ODONE, 1 - b), ((at - 1) >> 1) & 1, stop))) { ok = false; break; }
#pragma unroll
                        for (int pc = 0; pc < PH; ++pc) ok = ok && warp_wait_at(bar(C::B_BFULL, (bi + pc) % NB), ((bi + pc) / NB) & 1, stop);
                        if (!ok || !warp_wait_at(bar(C::B_PFULL, 2 * b + h), (at >> 1) & 1, stop)) { ok = false; break; }
                        tc_fence_after();
                        if (elect_one()) {
#pragma unroll
                            for (int pc = 0; pc < PH; ++pc) {
#pragma unroll
                                for (int kk = 0; kk < C::VR / 16; ++kk)
                                    tc_mma_f16_ts(o, p + pc * (C::VR / 2) + kk * 8, desc(VD, v[pc] + kk * (2048 >> 4)), ID_PV, pc == 0 && kk == 0 ? add : 1u);
                                if (two)
#pragma unroll
                                    for (int kk = 0; kk < C::VR / 16; ++kk)
                                        tc_mma_f16_ts(o, p + 32 + pc * (C::VR / 2) + kk * 8, desc(VD, v[pc] + kk * (2048 >> 4)), ID_PV, 1u);
                                for (int w = nt; w < 3; ++w) commit_at(bar(C::B_BEMPTY, (bi + pc) % NB));
                            }
                            commit_at(bar(h ? C::B_ODONE : C::B_OHALF, b));
                        }
                        __syncwarp();
                        if (h) progress[b] = at;
                    }
                    // (With one row tile to a unit the next keys come when this output is done: the scores of a whole tile after its
                    // second half's. Products of 128 columns read the queries once, of 64 twice.)
                    const int y = z + 2;
                    if (y < halves && (C::NT == 2 || h)) {
                        const int n = (int)n0 + (y & ~1), i = nt == 2 ? n >> 1 : n;
                        if (C::NT == 1 && !keys(n)) { ok = false; break; }
                        // Q is free when all scores of the part are made, of both buffers
                        const int frees = nt == 2 ? i == tiles - 1 : (i == tiles - 1) + (i == tiles - 2 || tiles == 1);
                        const uint32_t s_half = __shfl_sync(0xFFFFFFFFu, s_tm + (C::NT == 2 ? h * 64 : 0), 0);
                        const uint32_t k_half = __shfl_sync(0xFFFFFFFFu, k + (C::NT == 2 ? h * (64 * C::ROWB) >> 4 : 0), 0);
                        tc_fence_after();
                        if (elect_one()) {
#pragma unroll
                            for (int kk = 0; kk < 2 * D / 32; ++kk) {
                                constexpr int STEPS = C::ROWB / 32, HALF = D / 32;
                                const int kq = kk % HALF;
                                tc_mma_f8(s_half, desc(KD, q + (((kq / STEPS) * C::QPANEL + (kk / HALF) * TILE * C::ROWB + (kq % STEPS) * 32) >> 4)),
                                          desc(KD, k_half + (((kq / STEPS) * C::KPANEL + (kq % STEPS) * 32) >> 4)), ID_S, kk ? 1u : 0u);
                            }
                            if (C::NT == 1) commit_at(bar(C::B_SFULL, 2 * b));
                            commit_at(bar(C::B_SFULL, 2 * b + h));
                            if (h) {
                                for (int w = nt; w < 3; ++w) commit_at(bar(C::B_KEMPTY, (tile + i) % NK));       // one row tile arrives for two
                                for (int w = 0; w < frees; ++w) commit_at(bar(C::B_QFREE));
                            }
                        }
                        __syncwarp();
                    }
                }
                mine += halves;
                item = last;
                tile += tiles;
            }
        } else {
            // -------------------------------------------------------- scales: a lane takes four rows; scales are under way SA tiles
            // ahead and page ids another SA, both into shared memory (a register handed on would wait for its load)
            constexpr int A = C::SA;
            const uint32_t ids = base + C::OFF_SID + lane * 4, sc0 = base + C::OFF_SC + lane * 4;
            uint32_t tiles = 0, piece = 0;
            // This warp's waits bound those of all: where the pipeline stands, it waits, and stops the block when nothing has moved for
            // the bound.
            uint32_t seen = 0;
            uint64_t since = global_timer_ns();
            const bool nap = a.wait_ns >= 40000ull;  // (asleep for some 20 us, whatever less is asked for)
            auto wait = [&](uint32_t b, uint32_t parity) -> bool {
                while (!__all_sync(0xFFFFFFFFu, nap ? try_at_for(b, parity, 20000) : test_at(b, parity))) {
                    if (__any_sync(0xFFFFFFFFu, stopped(stop))) return false;
                    const uint32_t now_at = progress[0] + progress[1] + progress[2];
                    const uint64_t now = global_timer_ns();
                    if (now_at != seen) {
                        seen = now_at;
                        since = now;
                    } else if (__any_sync(0xFFFFFFFFu, now - since >= a.wait_ns)) {
                        stop_all(stop);
                        return false;
                    }
                }
                return true;
            };
            bool ok = true;
            Part x;
            while (ok && wait(bar(C::B_PDFULL, piece % C::NPD), (piece / C::NPD) & 1) && part_at(piece, x)) {
                const int t0 = x.t0, nt = x.t1 - t0, hp = x.h * P;
                const int first = t0 * TILE + lane * 4;
                const int32_t* table = a.table + (int64_t)x.b * a.width;
                auto look = [&](int d) {
                    const int j = first + d * TILE;
                    if (d < nt && j < x.end) cp_async_4(ids + (d % (2 * A)) * 128, table + (j >> a.page_shift));
                };
                auto load = [&](int d) {                     // its id has arrived
                    if (d >= nt) return true;
                    const uint32_t e = tiles + d, sc = e % NSC;
                    if (!wait(bar(C::B_SCEMPTY, sc), ((e / NSC) & 1) ^ 1)) return false;
                    const int j = first + d * TILE;
                    const uint32_t dst = sc0 + sc * C::SC_BYTES;
                    if (j < x.end) {
                        const int row = checked(read_at(ids + (d % (2 * A)) * 128), false) * a.c.n_kv_heads * P + hp + (j & (P - 1));
                        cp_async_4(dst, a.c.k_scales + row);
                        cp_async_4(dst + TILE, a.c.v_scales + row);
                    } else {
                        write_at(dst, 0x7F7F7F7Fu);
                        write_at(dst + TILE, 0x7F7F7F7Fu);
                    }
                    return true;
                };
                const int ahead = nt < A ? nt : A;
#pragma unroll 1
                for (int d = 0; d < ahead; ++d) look(d);
                cp_async_commit();
                cp_async_wait<0>();
                float unit = 0.0f;
#pragma unroll 1
                for (int d = -ahead; d < nt; ++d) {
                    if (d >= 0) {
                        if (nt < A) cp_async_wait<0>(); else cp_async_wait<A - 1>();
                    }
                    if (!load(d + ahead)) { ok = false; break; }
                    look(d + 2 * A);
                    cp_async_commit();
                    if (d < 0) continue;
                    if (d == 0) {
                        if (!wait(bar(C::B_QFULL, piece % QB), (piece / QB) & 1)) { ok = false; break; }
                        unit = *reinterpret_cast<const float*>(smem + C::OFF_QU + (piece % QB) * 8) * a.scale_log2;
                    }
                    const uint32_t sc = (tiles + d) % NSC, dst = sc0 + sc * C::SC_BYTES;
                    const uint32_t ks = read_at(dst);
                    uint32_t vs = read_at(dst + TILE);
                    float f[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint32_t k = (ks >> (8 * e)) & 255u, v = (vs >> (8 * e)) & 255u;
                        // scores stay finite where they can; values past bf16's range, and NaN, make a NaN of the weight and count as zeros
                        f[e] = fminf(e8m0_to_float(k) * unit, 0x1p126f);
                        if (k == 255u || v > 246u) f[e] = __uint_as_float(0x7FC00000u);
                        if (v > 246u) vs &= ~(255u << (8 * e));
                    }
                    write_at(dst + TILE, vs);
                    *reinterpret_cast<float4*>(smem + C::OFF_SC + sc * C::SC_BYTES + 2 * TILE + lane * 16) = make_float4(f[0], f[1], f[2], f[3]);
                    __syncwarp();
                    if (lane == 0) arrive_at(bar(C::B_SCFULL, sc));
                }
                tiles += nt;
                ++piece;
            }
            cp_async_wait<0>();
            if (ok) (void)wait(bar(C::B_DONE), 0);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (*abort_flag) {                               // final after the barrier: nothing new is issued past it
        if (warp == 16 && lane == 0) {
            drain_stage_fills(bar_ptr(C::B_KFULL), NK, issued_k);
            drain_stage_fills(bar_ptr(C::B_RFULL), NR, issued_r);
        }
        if ((warp == 17 || warp == 18) && elect_one()) tc_drain(bar_ptr(C::B_DRAIN) + (warp - 17));
        tc_fence_before();
        __syncthreads();
    }
    if (warp == 17) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
    if (tid == 0 && *abort_flag) record_error(a.err, MOE_DEV_TIMEOUT);
}

// ------------------------------------------------------------------ join

// The parts of a unit that several CTAs share, added in the order of the cache rows. blockIdx.x + 1 is the first CTA whose
// part begins inside the unit; 32 rows a block, a lane a row, a warp an eighth of the columns: a lane's output is whole
// sectors where it has 16 columns or more. The references come first, of all parts, and the sums need not wait for one another.
constexpr int JOIN_WARPS = 8, JOIN_ROWS = 32;

template <int D>
__global__ void __launch_bounds__(JOIN_WARPS * 32) chunk_attention_join(const __grid_constant__ ChunkArgs a, int ctas) {
    using C = Cfg<D>;
    constexpr int ROWS = C::ROWS;
    pdl_trigger();
    pdl_wait();
    const Pos* places = reinterpret_cast<const Pos*>(a.ws);
    const int k = blockIdx.x + 1;
    const Pos p = places[k], before_p = places[k - 1];
    if (p.lane >= a.lanes || p.tile == 0 || (same_unit(p, before_p) && before_p.tile > 0)) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, row = blockIdx.y * JOIN_ROWS + lane;
    // CTA k - 1 + i holds a part: one more in which the unit begins, and those that begin in it, but for CTAs without tiles
    auto parts_from = [&](int i0, bool* more) {
        const int c = k - 1 + i0 + lane;
        bool in = i0 + lane == 0, some = in;
        if (!in && c < ctas) {
            const Pos here = places[c], next = places[c + 1];
            in = same_unit(here, p);
            some = in && !(same_unit(next, here) && next.tile == here.tile);
        }
        *more = __all_sync(0xFFFFFFFFu, in);
        return __ballot_sync(0xFFFFFFFFu, some);
    };
    bool more;
    const uint32_t first = parts_from(0, &more);
    const Unit x = unit_at<D>(a, p.lane, p.unit);
    if ((int)blockIdx.y * JOIN_ROWS >= x.rows) return;
    const float* parts = reinterpret_cast<const float*>(a.ws + parts_offset(ctas));
    // f(each part)
    auto each = [&](auto f) {
        uint32_t some = first;
        bool on = more;
        for (int i0 = 0;;) {
            for (; some; some &= some - 1) {
                const int c = k - 1 + i0 + __ffs(some) - 1;
                const float* part = parts + (size_t)(2 * c + (c == k - 1 ? 1 : 0)) * C::PART_FLOATS;
                f(part);
            }
            if (!on) break;
            i0 += 32;
            some = parts_from(i0, &on);
        }
    };
    float m = NEVER;
    each([&](const float* part) { m = fmaxf(m, part[ROWS * D + row]); });
    constexpr int N = D / 4 / JOIN_WARPS;            // groups of four columns of a thread
    float4 acc[N];
#pragma unroll
    for (int e = 0; e < N; ++e) acc[e] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    float l = 0.0f;
    each([&](const float* part) {
        const float mc = part[ROWS * D + row], lc = part[ROWS * D + ROWS + row];
        if (row >= x.rows || (mc == NEVER && lc == 0.0f)) return;            // nothing seen: no O either
        float4 v[N];
#pragma unroll
        for (int e = 0; e < N; ++e) v[e] = *reinterpret_cast<const float4*>(part + ((size_t)(warp * N + e) * ROWS + row) * 4);
        const float f = ex2(mc - m);
        l += lc * f;
#pragma unroll
        for (int e = 0; e < N; ++e) {
            acc[e].x += v[e].x * f;
            acc[e].y += v[e].y * f;
            acc[e].z += v[e].z * f;
            acc[e].w += v[e].w * f;
        }
    });
    if (row >= x.rows) return;
    const int t = (int)((uint32_t)row * a.by_group >> 16);
    const int64_t to = (int64_t)(x.tok0 + t) * a.n_q + x.h * a.group + row - t * a.group;
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    uint32_t o[2 * N];
#pragma unroll
    for (int e = 0; e < N; ++e) {
        o[2 * e] = pack_bf16(acc[e].x * inv, acc[e].y * inv);
        o[2 * e + 1] = pack_bf16(acc[e].z * inv, acc[e].w * inv);
    }
    __nv_bfloat16* dst = a.out + to * D + warp * N * 4;
    if constexpr (N == 2) {
        *reinterpret_cast<uint4*>(dst) = make_uint4(o[0], o[1], o[2], o[3]);
    } else {
#pragma unroll
        for (int e = 0; e < 2 * N; e += 8) store_32(dst + 2 * e, o[e], o[e + 1], o[e + 2], o[e + 3], o[e + 4], o[e + 5], o[e + 6], o[e + 7]);
    }
    if (a.lse && warp == 0) a.lse[to] = l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
}

// ------------------------------------------------------------------ host side

cudaError_t codes_map(CUtensorMap* m, const void* base, const moe_kv_cache& c, int box_bytes, int box_rows, CUtensorMapSwizzle swizzle) {
    auto enc = encoder();
    if (!enc) return cudaErrorNotSupported;
    const cuuint64_t dims[2] = {(cuuint64_t)c.head_dim, (cuuint64_t)c.n_pages * c.n_kv_heads * c.page_size};
    const cuuint64_t strides[1] = {(cuuint64_t)c.head_dim};
    const cuuint32_t box[2] = {(cuuint32_t)box_bytes, (cuuint32_t)(c.page_size < box_rows ? c.page_size : box_rows)};
    const cuuint32_t estr[2] = {1, 1};
    const CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
                           CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <int D>
cudaError_t launch(ChunkArgs a, cudaStream_t s) {
    using C = Cfg<D>;
    const int64_t tiles = ((int64_t)a.width * a.c.page_size + TILE - 1) / TILE;
    const int64_t units = ((int64_t)a.n_tokens * a.group + C::ROWS - 1) / C::ROWS * a.c.n_kv_heads;      // if they are full
    a.whole = tiles <= SHORT_TILES || (tiles <= WHOLE_TILES && units <= 2 * moe_sm_count());
    // Few units that are not cut: of one row tile each, for twice as many CTAs (300 tokens, 8 kv heads: 19 us, not 23).
    a.block = (C::NT == 2 && a.whole && units * 2 <= moe_sm_count() ? TILE : C::ROWS) / a.group;
    ChunkMaps maps;
    cudaError_t e = codes_map(&maps.k, a.c.k_codes, a.c, C::ROWB, TILE, C::ROWB == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B);
    if (e == cudaSuccess) e = codes_map(&maps.v, a.c.v_codes, a.c, D, C::VR, CU_TENSOR_MAP_SWIZZLE_NONE);
    if (e != cudaSuccess) return e;
    static bool attr_set[64] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev >= 0 && dev < 64 && !attr_set[dev]) {
        e = cudaFuncSetAttribute(chunk_attention<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
        if (e != cudaSuccess) return e;
        attr_set[dev] = true;
    }
    const int ctas = moe_sm_count();
    moe_prof_begin(MK_CHUNK_ATTENTION, s);
    e = moe_launch(chunk_attention<D>, dim3((unsigned)ctas), dim3(C::THREADS), C::SMEM, s, maps, a);
    moe_prof_end(MK_CHUNK_ATTENTION, s);
    moe_count_launches(1);
    if (e != cudaSuccess || ctas < 2 || a.whole) return e;
    moe_prof_begin(MK_CHUNK_JOIN, s);
    e = moe_launch(chunk_attention_join<D>, dim3((unsigned)(ctas - 1), C::ROWS / JOIN_ROWS), dim3(JOIN_WARPS * 32), 0, s, a, ctas);
    moe_prof_end(MK_CHUNK_JOIN, s);
    moe_count_launches(1);
    return e;
}

}  // namespace

size_t moe_chunk_attention_workspace_bytes(int n_tokens, int n_q_heads, int n_kv_heads, int head_dim, int lanes) {
    if (n_tokens < 1 || n_q_heads < 1 || n_kv_heads < 1 || head_dim < 1 || lanes < 1) return 0;
    const int ctas = moe_sm_count();
    const size_t part = head_dim == 256 ? Cfg<256>::PART_FLOATS : head_dim == 64 ? Cfg<64>::PART_FLOATS : Cfg<128>::PART_FLOATS;
    return parts_offset(ctas) + (size_t)2 * ctas * part * sizeof(float);
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
    if ((((uintptr_t)q | (uintptr_t)workspace) & 15) || ((uintptr_t)out & 31)) return MOE_EINVAL;
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
    a.by_group = (65536u + a.group - 1) / a.group;
    a.table = page_table;
    a.width = table_width;
    a.lanes = lanes;
    a.page_shift = log2_of(cache->page_size);
    a.kv_len = kv_len;
    a.cu = cu_tokens;
    a.scale_log2 = scale * 1.4426950408889634f;
    a.out = static_cast<__nv_bfloat16*>(out);
    a.lse = lse;
    a.ws = static_cast<uint8_t*>(workspace);
    a.err = err;
    a.wait_ns = moe_wait_limit_ns();
    const cudaError_t e = cache->head_dim == 64 ? launch<64>(a, s) : cache->head_dim == 128 ? launch<128>(a, s) : launch<256>(a, s);
    return e == cudaSuccess ? MOE_OK : MOE_ECUDA;
}
