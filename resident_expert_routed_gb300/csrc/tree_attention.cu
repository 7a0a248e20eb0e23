// Attention of drafted tokens over the paged 8-bit key/value cache.
//
// For the rows r = (node, query head) of one kv head and the cache rows j:
//   s[r,j] = scale log2(e) q_r . k_j        (k_j = codes * 2^ek_j)
//   out[r] = sum_j 2^s[r,j] v_j / sum_j 2^s[r,j]      (v_j = codes * 2^ev_j)
// over the j that r sees. Both products run on the tensor cores on the codes
// as they lie in the cache (tcgen05 kind::f8f6f4, fp32 accumulators in TMEM):
// no byte of the cache is converted or scaled outside the MMA, so TMA moves it
// from HBM to the operand buffers untouched.
//   - The other operand is split in 8-bit parts. A bf16 query has 8
//     significant bits and e4m3 has 4: with its row scaled by a power of two to
//     128 <= max|q| < 256, hi = e4m3(q), lo = e4m3(q - hi) hold it exactly down
//     to 2^-9 of the row's maximum and within 2^-17 of the maximum below.
//   - A probability p, rounded to fp16, is the sum of three e5m2: an e5m2 is the upper byte of an fp16, so hi is that
//     byte of p, mid that of p - hi (rounded by an integer add), lo that of the rest. Together 10 significant bits,
//     as long as lo's smallest, 2^-16, allows.
//   - The scale of a key row multiplies its column of scores; the scale of a
//     value row is added to the exponent: s' = s + ev_j, p = 2^(s' - m + 11), so
//     values of any size keep their precision; the sum of weights gets p 2^-ev_j (and 2^-16, for its range).
//   - m is a running reference, not each tile's maximum: it is the maximum of s'
//     when it is set, and stays until a score passes it by 4.9 (p = 2^15.9; fp16 ends at 2^16);
//     then it is set again and what has been added up is scaled down. Most tiles
//     so need no maximum at all: one compare, a vote, no reduction over the rows.
//     A weight (2^s') is held to 2^-9 of itself, or to 2^-28 of the largest: weights that are small but many keep
//     their share, 2^17 of one size to 2^-11 of the peak above them. (Two parts, e5m2 and e4m3, reach 2^-9 of a weight
//     only down to 2^-8 of the largest, and equal weights below round the same way: up to 11 % of a tail's share was
//     lost.)
//   - A value vector of zeros has the scale 2^0 in the cache, far above those of ordinary values. Taken as it is it would
//     raise m by 8 and more and cost the weights that count as many bits. Rows of that scale byte have their codes looked at,
//     and zeros count as 2^-100: they add to the sum of weights and to nothing else.
//   - References hold a value exponent, so two of them can be 2^220 apart where the scores are not. The sum of weights,
//     which holds the inverse, is taken from one to the other by the root of the factor, twice: 2^-220 is no
//     fp32, its product with the sum is.
// Scores, sums, the accumulators O and the parts that the join adds up are fp32; the output is rounded to bf16 once.
//
// Orientation: cache rows are the MMA's M (128), tree rows its N, so a single
// token costs N = 16 and a wide tree 32 or 64, and nothing is padded to 128;
// hi and lo accumulate:
//   S^T[128 rows, R] = K[128, D] Q^T            O^T[D, R] += V^T[D, 128] P^T[128, R]
// A thread of a softmax group is a cache row: the rows' scales are its own
// registers, the sums of weights are kept per thread and added up once at the end.
//
// Two softmax groups take the tiles of 128 cache rows in turn, each with an O of
// its own, four warps for up to 32 tree rows and eight for 64 (32 tree rows are what a
// thread can hold next to their sums).
//
// Work: the (lane, kv head, tile of tree rows) units, each a run of cache
// tiles, are laid end to end and cut into equal parts, one per CTA. (A few tiles are added for each unit.) A unit that one
// CTA does whole is written at once; the others leave their parts (output, maximum, sum)
// in the workspace and tree_attention_join adds them up in order. One CTA an SM, so one long lane and many uneven
// ones fill the machine alike.
//
// What bounds it (measured, a call's whole time, calls back to back in a graph; head_dim 128, 8 kv heads, 2,064 bytes of
// cache a row): up to 32 tree rows HBM: one token in 64 lanes of uneven lengths up to 8,192 rows 94.5 us (543 MB, 5.7 TB/s;
// even lengths 6.5 TB/s, head_dim 256 6.5, head_dim 64 4.3: there the copies' warp, 1,090 clocks a tile for four pages where
// HBM would allow 780), a tree of 7 nodes in two lanes of 131,072 rows 101 us (541 MB). Of the 95 us the tile loop takes 78,
// the cut 4, the first tile 4, the last outputs, the join and its launch 6. With 64 tree rows the softmax's instructions and
// their latency: 2,400 clocks a tile where HBM would allow 1,550 (trees of up to 16 nodes, 64 query heads, 32 lanes of up to
// 8,001 rows: 148 us; at head_dim 64 2,600 clocks). A chain without a mask (the chunk of a prompt) runs over all its tiles,
// those that nobody sees too: 8,192 rows, 32 query heads 2.58 ms. Below some thousand rows the chain of one unit: 8.7 us
// for a lane of 300.
//
// Roles: 8 or 16 warps of softmax, then
//   four warps       the next unit's queries (split and laid out), a finished unit's output
//   a warp           TMA, one copy per page
//   a warp           MMA issue, TMEM
//   a warp           the rows' scales
//   a warp           what the join has to know, then the watchdog
// Waits are bounded as in the expert GEMMs, by a watchdog warp. Loops that run beside the softmax are kept short and
// rolled: their instructions compete with its unrolled ones for the instruction cache (TMA and scale loops unrolled
// by four and eight cost a third of the rate).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <climits>
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
    int whole;                                   // units are not cut: the table holds WHOLE_TILES tiles at most
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
constexpr int LANE_CACHE = 256;                  // lanes whose facts are kept in shared memory

// Units of at most this many tiles are not cut between CTAs, and the join is not launched: a unit's tiles one after the other
// take less than the join and its launch. Known on the host, from the rows that the page table can hold. (One token, 8 kv
// heads of 128, us whole / cut: 300 rows 8.7 / 10.8 in one lane, 20.2 / 25.0 in 64; 1,000 rows 12.1 / 11.6 and 33.3 / 35.7;
// 2,000 rows 17.5 / 13.6 and 54.6 / 53.3.)
constexpr int WHOLE_TILES = 8;

// The run's measure: what a tile costs, and a tile of which half the unit's tree rows are missing, where the halves are
// different warps' (the cache is then read as fast, the softmax does half the work; 2, 3, 4: trees of up to 10 nodes 147, 125,
// 128 us). A unit costs R / 8 tiles beside its own: its queries, its first reference, its output (0, R / 8, R / 4: trees of up to
// 16 nodes 207, 148, 154 us; 64 uneven lanes of one token 110, 94, 92.5 us). The parts are cut evenly in this measure; below four
// tiles a CTA in tiles alone, as there the longest part counts.
constexpr int FULL_COST = 4, HALF_COST = 3;
__host__ __device__ constexpr int unit_cost(int R) { return FULL_COST * R / 8; }

// What the join needs, at the start of the workspace: for each CTA the unit that its part begins in.
struct JoinUnit {
    int32_t join;                                // 1: its part is the second of the unit, whose parts are
    int32_t first, last;                         // those of CTAs first .. last,
    int32_t second;                              // the first of them its CTA's second part (else its first)
    int32_t node0, rows, head, row0;             // first node of the lane, tree rows of the unit, kv head, first row in the lane
};

__host__ __device__ constexpr size_t part_floats(int R, int D) { return (size_t)R * (D + 2); }
__host__ __device__ inline size_t parts_offset(int ctas) { return ((size_t)ctas * sizeof(JoinUnit) + 255) / 256 * 256; }

// Where part k begins: total / parts each, one more in the first total % parts. (64-bit divisions only where needed.)
MOE_DEV int64_t part_begin(unsigned long long total, int parts, int k) {
    const unsigned long long each = total >> 32 ? total / parts : (uint32_t)total / (uint32_t)parts;
    const int more = (int)(total - each * parts);
    return (int64_t)(each * k) + (k < more ? k : more);
}
// The part that x is in.
MOE_DEV int part_of(unsigned long long total, int parts, unsigned long long x) {
    const unsigned long long each = total / parts, more = total - each * parts;
    return (int)(x < more * (each + 1) ? x / (each + 1) : more + (x - more * (each + 1)) / each);
}

template <int D, int R>                          // R: tree rows of a unit
struct Cfg {
    static constexpr int RH = R < 32 ? R : 32;                // tree rows of a softmax warpgroup: its threads' registers
    static constexpr int HALVES = R / RH;                     // warpgroups of a softmax group
    static constexpr int SW = 8 * HALVES;                     // softmax warps, of two groups
    static constexpr int THREADS = (SW + 8) * 32;             // then four of queries and outputs, TMA, MMA, scales, join
    static constexpr int ROWB = D >= 128 ? 128 : 64;          // bytes of an operand row: one swizzle atom
    static constexpr int PANELS = D / ROWB;
    static constexpr int PANEL = TILE * ROWB;
    static constexpr int SLOT = TILE * D;
    static constexpr int QROWS = 2 * R;                       // hi, then lo
    static constexpr int QBUF = QROWS * D;
    static constexpr int PBUF = 3 * TILE * R;                 // hi, mid, lo
    static constexpr int SB = 4;                              // buffers of S
    static constexpr int NS = D == 64 ? 16 : D == 256 ? (R == 32 ? 4 : 5) : R == 64 ? 7 : R == 32 ? 10 : 12;     // ring of key and value tiles: what fits
    static constexpr int SA = 8;                              // tiles that scales are under way ahead, and page ids another as many
    static constexpr int PT = 8;                              // tiles that the page ids of keys and values are under way ahead
    static constexpr int NSC = 2 * SA;                        // ring of the rows' scales:
    static constexpr int SC_BYTES = 2 * TILE + 16;            // key bytes, value bytes, largest and smallest value byte (int)
    static constexpr int MB = D == 256 ? 2 : 1;               // M blocks of O^T
    static constexpr int OFF_RING = 0;
    static constexpr int OFF_P = OFF_RING + NS * SLOT;
    static constexpr int OFF_Q = OFF_P + 2 * PBUF;
    static constexpr int OFF_SC = OFF_Q + 2 * QBUF;
    static constexpr int OFF_SID = OFF_SC + NSC * SC_BYTES;   // page ids, [2 SA][32]
    static constexpr int OFF_TID = OFF_SID + 2 * SA * 128;    // [PT][8]
    static constexpr int OFF_F = OFF_TID + PT * 32;           // floats from here
    static constexpr int F_O = 0;                             // [2 groups][R] P_EXP - m, as added to s'
    static constexpr int F_AL = F_O + 2 * R;                  // [2: root, whole][2][R] scale-down of what has been added up
    static constexpr int F_WMAX = F_AL + 4 * R;               // [2 groups][HALVES][2][4 warps][RH]
    static constexpr int F_QF = F_WMAX + 16 * R;              // [4][R] 2^-a of the queries' rows
    static constexpr int F_QU = F_QF + 4 * R;                // [4][2] 2^-a of all rows of a unit; whether the rows' differ instead
    static constexpr int F_QX = F_QU + 8;                     // [largest, smallest][unit parity][4 warps] |q| of the rows, as bits
    static constexpr int F_L = F_QX + 16;                 // [2][4][R] sums at a part's end
    static constexpr int F_M = F_L + 8 * R;                   // [2][R] their references
    static constexpr int F_ST = F_M + 2 * R;                  // [4 warps][3][R] factors of the output, and its rows' places (int)
    static constexpr int F_END = F_ST + 12 * R;
    static constexpr int OFF_LANE = OFF_F + F_END * 4;        // int n0, n, len [LANE_CACHE]
    static constexpr int OFF_SCAN = OFF_LANE + 3 * LANE_CACHE * 4;
    static constexpr int OFF_BAR = OFF_SCAN + 2 * 32 * 8 + 64;       // two sums, Cut
    // barriers, as byte offsets
    static constexpr int B_FULL = OFF_BAR;                    // [NS] a tile of keys or values has arrived
    static constexpr int B_EMPTY = B_FULL + 8 * NS;           // [NS] ... has been used
    static constexpr int B_SCFULL = B_EMPTY + 8 * NS;         // [NSC] the scales of a tile are there
    static constexpr int B_SCEMPTY = B_SCFULL + 8 * NSC;      // [NSC] ... have been read
    static constexpr int B_SFULL = B_SCEMPTY + 8 * NSC;       // [SB] S of a tile is ready
    static constexpr int B_VOTE = B_SFULL + 8 * SB;           // [4 warpgroups] the four warps have compared a tile's scores
    static constexpr int B_MAXIMA = B_VOTE + 32;              // [4 warpgroups] ... have written a tile's maxima
    static constexpr int B_PFULL = B_MAXIMA + 32;             // [2 groups] P is written (and S has been read)
    static constexpr int B_PFREE = B_PFULL + 16;              // [2] P has been read (and added to O)
    static constexpr int B_QFULL = B_PFREE + 16;              // [2] the queries of a part are there
    static constexpr int B_QFREE = B_QFULL + 16;              // [2] ... have been used
    static constexpr int B_OFULL = B_QFREE + 16;              // [2] O of a part is complete
    static constexpr int B_OFREE = B_OFULL + 16;              // [2] ... and has been read
    static constexpr int B_LFULL = B_OFREE + 16;              // the sums of a part are written
    static constexpr int B_LFREE = B_LFULL + 8;               // ... and read
    static constexpr int B_QMAX = B_LFREE + 8;                // the four query warps have their maxima
    static constexpr int B_DONE = B_QMAX + 8;                 // the block's last output is written
    static constexpr int B_DRAIN = B_DONE + 8;
    static constexpr int OFF_MISC = (B_DRAIN + 8 + 15) / 16 * 16;     // tmem slot, abort flag, votes [4 warpgroups][2][4]
    static constexpr int SMEM = OFF_MISC + 16 + 128 + 1024;
    // Tiles whose S may be under way: the buffers, and (an odd ring) not past a slot whose values are still to be used
    static constexpr int LOOK = NS % 2 && NS / 2 + 1 < SB ? NS / 2 + 1 : SB;
    // O of the three parts of P in columns of their own where TMEM has room (they are added up with the output): one MMA of
    // N = 3 R takes 32 rows, not three of N = R (us, so / three: one token in 64 uneven lanes 93.9 / 103.7, a tree of 7 nodes
    // in two lanes of 131,072 rows 100.6 / 107.4).
    static constexpr int PARTS = 4 * R + 4 * R * MB * 3 <= 512 ? 3 : 1;
    static constexpr int OC = PARTS * R;                      // columns of one O block
    static constexpr int TMEM_O = 4 * R;                      // after S (4 R columns): O [group][unit parity][MB][PARTS][R]
    static constexpr int TMEM_USED = 4 * R + 4 * OC * MB;
    static constexpr int TMEM_COLS = TMEM_USED <= 128 ? 128 : TMEM_USED <= 256 ? 256 : 512;
    static_assert(TMEM_USED <= 512 && SMEM <= 227 * 1024, "TMEM, shared memory");
    static_assert(OFF_F % 16 == 0 && OFF_SCAN % 8 == 0 && OFF_BAR % 8 == 0 && OFF_MISC % 16 == 0, "alignment");
    static_assert(R == 16 || R == 32 || R == 64, "R");
};

constexpr float P_EXP = 11.0f;                   // p = 2^11 at the reference
constexpr float P_EXP_MAX = 15.9f;               // below fp16's largest, 65,504
// The sums of weights hold 2^(s - m + P_EXP - L_EXP), with value exponents of -100 to 120 in m: 2^99 at most for a row (so 2^28
// rows do not overflow), 2^-125 for the largest weight at least. An exponential of its own is taken 2^26 larger, as
// ex2 has no subnormal results.
constexpr int L_EXP = 16, L_OWN = 26;
constexpr uint32_t ZERO_BYTE = 127u, LEAST_BYTE = 27u;      // scale bytes: of a vector of zeros, of the smallest vectors
// A row's value scale this far (in binades) below the largest so far, or a row that may be one of zeros, is looked after. (p
// ends at 2^-126: what the sum of weights could miss is 2^-37 of the largest weight.)
constexpr int WIDE = 100, MAY_BE_ZERO = -1000;

// ------------------------------------------------------------------ small device pieces

MOE_DEV float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
MOE_DEV float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
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
// The barrier and copy instructions of common.cuh on 32-bit shared-memory addresses: one register holds the base, the
// rest is an immediate. (Registers bound this kernel; a table of 64-bit pointers costs it dozens.)
MOE_DEV bool test_at(uint32_t bar, uint32_t parity) {         // without waiting
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
MOE_DEV bool try_at(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
MOE_DEV bool try_at_for(uint32_t bar, uint32_t parity, uint32_t ns) {       // asleep for about ns at most
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity), "r"(ns)
        : "memory");
    return ok != 0;
}
MOE_DEV void cp_async_4(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
MOE_DEV void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> MOE_DEV void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
MOE_DEV int read_at(uint32_t at) {
    int v;
    asm volatile("ld.shared.s32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
    return v;
}
MOE_DEV void write_at(uint32_t at, uint32_t v) { asm volatile("st.shared.u32 [%0], %1;" ::"r"(at), "r"(v) : "memory"); }
MOE_DEV uint32_t stopped(uint32_t stop) {
    uint32_t v;
    asm volatile("ld.volatile.shared.u32 %0, [%1];" : "=r"(v) : "r"(stop) : "memory");
    return v;
}
MOE_DEV void stop_all(uint32_t stop) { asm volatile("st.volatile.shared.u32 [%0], 1;" ::"r"(stop) : "memory"); }
// A wait of a whole warp, with the same outcome in every lane: false when the block has been stopped. The watchdog warp bounds all
// of a block's waits in one place: a bound in each of some thirty inlined waits drives the kernel out of the instruction cache.
MOE_DEV bool warp_wait_at(uint32_t bar, uint32_t parity, uint32_t stop) {
    while (!__all_sync(0xFFFFFFFFu, try_at(bar, parity)))
        if (__any_sync(0xFFFFFFFFu, stopped(stop))) return false;
    return true;
}
MOE_DEV void arrive_at(uint32_t bar) { asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory"); }
MOE_DEV void arrive_expect_tx_at(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
MOE_DEV void commit_at(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
MOE_DEV void tma_load_at(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];"
        ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y)
        : "memory");
}

MOE_DEV void tc_mma_f8(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}"
        ::"r"(d_tmem), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Moves registers between warpgroups: of 768 threads launched with 80 each (R = 64), 4 x 96 + 56 + 40 = 6 x 80.
template <int N> MOE_DEV void regs_up() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N> MOE_DEV void regs_down() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

// kind::f8f6f4, e4m3 x e4m3 (or x e5m2) -> fp32; a_mn, b_mn: whether A and B lie with M and N (instead of K) contiguous.
__host__ __device__ constexpr uint32_t idesc_f8(int m, int n, int a_mn, int b_mn, int b_e5m2) {
    return (1u << 4) | ((uint32_t)b_e5m2 << 10) | ((uint32_t)a_mn << 15) | ((uint32_t)b_mn << 16) | ((uint32_t)(n >> 3) << 17) |
           ((uint32_t)(m >> 4) << 24);
}

// 2^p down to the smallest subnormal, 2^-149.
MOE_DEV float exp2_whole(int p) { return p >= -126 ? exp2_int(p) : __uint_as_float(p >= -149 ? 1u << (p + 149) : 0u); }

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

// N consecutive columns of this lane of TMEM, complete on return. One wide load, not several: beside running
// MMAs each wait costs 250 to 400 clocks.
MOE_DEV void tc_load(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {"
        "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}
MOE_DEV void tc_load(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {"
        "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr)
        : "memory");
}

// Shared-memory matrix descriptor without its address: swizzle 2 = 128 B, 4 = 64 B, 6 = 32 B, 0 = none; the two
// strides in bytes. With a swizzle `lead` is from one atom of the contiguous axis to the next and `group` from one group of
// eight rows (of the strided axis) to the next, without one the other way round. Operands that are one atom wide on
// their contiguous axis hold the group stride in both.
__host__ __device__ constexpr uint64_t desc_base(int swizzle, int lead, int group) {
    return ((uint64_t)(lead >> 4) << 16) | ((uint64_t)(group >> 4) << 32) | ((uint64_t)1 << 46) | ((uint64_t)swizzle << 61);
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

// This CTA's part: its first lane, unit of the lane and tile of the unit, its number of tiles.
struct Cut {
    int lane, unit, t, count;
    unsigned long long unit_at, before, next;        // that unit's first place in the run; tiles before the part, before the next one
    unsigned long long total;                        // of the run
    int cost, weight, parts;                         // of a unit beside its tiles, of a tile of that unit; parts of the run
};

// Inclusive sums over the block's threads of two values, and their totals. scratch: 64 values. One barrier, after one that
// lets scratch be written again.
MOE_DEV void scan2(unsigned long long& x, unsigned long long& y, unsigned long long* scratch, unsigned long long* tx, unsigned long long* ty) {
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, nw = blockDim.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const unsigned long long a = __shfl_up_sync(0xFFFFFFFFu, x, o), b = __shfl_up_sync(0xFFFFFFFFu, y, o);
        if (lane >= o) { x += a; y += b; }
    }
    __syncthreads();
    if (lane == 31) { scratch[wid] = x; scratch[32 + wid] = y; }
    __syncthreads();
    unsigned long long sx = lane < nw ? scratch[lane] : 0ull, sy = lane < nw ? scratch[32 + lane] : 0ull;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const unsigned long long a = __shfl_up_sync(0xFFFFFFFFu, sx, o), b = __shfl_up_sync(0xFFFFFFFFu, sy, o);
        if (lane >= o) { sx += a; sy += b; }
    }
    *tx = __shfl_sync(0xFFFFFFFFu, sx, 31);
    *ty = __shfl_sync(0xFFFFFFFFu, sy, 31);
    const unsigned long long bx = __shfl_sync(0xFFFFFFFFu, sx, wid - 1 & 31), by = __shfl_sync(0xFFFFFFFFu, sy, wid - 1 & 31);
    if (wid > 0) { x += bx; y += by; }
}

// One CTA's way through its part of the run: the unit it is in and the tile within it.
struct Walk {
    int b, h, rt, t, tiles, nrt;                     // lane, kv head, tile of tree rows, cache tile; tiles of the unit, units of a head
};
template <int R>                                     // R: tree rows of a unit
struct Walker {
    const AttnArgs& a;
    const int* facts;

    MOE_DEV Lane lane(int b) const {
        if (b < LANE_CACHE) return Lane{facts[b], facts[LANE_CACHE + b], facts[2 * LANE_CACHE + b]};
        bool bad;
        return lane_facts(a, b, &bad);
    }
    MOE_DEV void enter(Walk& w) const {
        const Lane l = lane(w.b);
        w.tiles = l.len > 0 ? (l.len + TILE - 1) / TILE : 1;
        w.nrt = l.n > 0 ? (l.n * a.group + R - 1) / R : 1;
    }
    MOE_DEV Walk start(int b, int u, int tile) const {
        Walk w;
        w.b = b;
        enter(w);
        w.t = tile;
        w.h = u / w.nrt;
        w.rt = u - w.h * w.nrt;
        return w;
    }
    // past n tiles, which do not lead out of the unit; more: whether tiles are left after them
    MOE_DEV void advance(Walk& w, int n, bool more) const {
        w.t += n;
        if (w.t < w.tiles || !more) return;
        w.t = 0;
        if (++w.rt < w.nrt) return;
        w.rt = 0;
        if (++w.h < a.c.n_kv_heads) return;
        w.h = 0;
        do ++w.b; while (lane(w.b).n == 0 && w.b + 1 < a.lanes);
        enter(w);
    }
    MOE_DEV int rows(const Walk& w) const {                   // tree rows of this unit
        const int left = lane(w.b).n * a.group - w.rt * R;
        return left < R ? left : R;
    }
};

// The cut: every CTA adds up all lanes' tiles and finds its own part. A function of its own, so that nothing of it is
// live in the roles.
template <int R>
__device__ __noinline__ void cut_run(const AttnArgs& a, int* facts, unsigned long long* scratch, Cut* here) {
    const int tid = threadIdx.x, H = a.c.n_kv_heads, G = a.group;
    // this thread's lane of a round: units a head, tiles a unit, costs of a full unit's tile and of the last one's; sizes of
    // the lanes before it, in the run's measure and in tiles
    unsigned long long size_all = 0, tiles_all = 0, size_in = 0, tiles_in = 0, lane_size = 0, lane_tiles = 0;
    uint32_t nrt = 0, tiles = 0, last = 0;
    auto scan_lanes = [&](int b0, bool tell) {
        const int b = b0 + tid;
        Lane l{0, 0, 0};
        if (b < a.lanes) {
            bool bad;
            l = lane_facts(a, b, &bad);
            if (bad && tell && blockIdx.x == 0) record_error(a.err, MOE_DEV_BAD_PAGE);
            if (b < LANE_CACHE) {
                facts[b] = l.n0;
                facts[LANE_CACHE + b] = l.n;
                facts[2 * LANE_CACHE + b] = l.len;
            }
        }
        nrt = (l.n * G + R - 1) / R;
        tiles = l.len > 0 ? (l.len + TILE - 1) / TILE : 1;
        last = Cfg<64, R>::HALVES > 1 && l.n * G - (int)(nrt - 1) * R <= R / 2 ? HALF_COST : FULL_COST;
        lane_tiles = (unsigned long long)H * nrt * tiles;
        lane_size = nrt == 0  ? 0
                    : a.whole ? (unsigned long long)H * nrt
                              : H * ((unsigned long long)tiles * ((nrt - 1) * FULL_COST + last) + (unsigned long long)nrt * unit_cost(R));
        unsigned long long x = lane_size, y = lane_tiles, tx, ty;
        scan2(x, y, scratch, &tx, &ty);
        size_in = size_all + x - lane_size;
        tiles_in = tiles_all + y - lane_tiles;
        size_all += tx;
        tiles_all += ty;
    };
    for (int b0 = 0; b0 < a.lanes; b0 += (int)blockDim.x) scan_lanes(b0, true);
    const unsigned long long n_tiles = tiles_all;
    const bool plain = !a.whole && n_tiles <= 4ull * gridDim.x;      // a tile is a tile
    const uint32_t cost = a.whole || plain ? 0 : unit_cost(R), full = plain ? 1 : FULL_COST;
    const unsigned long long total = plain ? n_tiles : size_all, pieces = a.whole ? size_all : n_tiles;
    const int parts = pieces < gridDim.x ? (int)pieces : (int)gridDim.x;
    const bool active = (int)blockIdx.x < parts;
    const unsigned long long first = active ? part_begin(total, parts, blockIdx.x) : 0;
    const unsigned long long next = active ? part_begin(total, parts, blockIdx.x + 1) : 0;
    auto divide = [](unsigned long long x, unsigned long long y) { return (x | y) >> 32 ? (uint32_t)(x / y) : (uint32_t)x / (uint32_t)y; };
    auto locate = [&](int b0) {                      // by the thread whose lane it is in
        const unsigned long long at = plain ? tiles_in : size_in, size = plain ? lane_tiles : lane_size;
        const uint32_t wl = plain ? 1 : last;
        const uint32_t each = tiles * full + cost;                   // of a full unit; of all units of a head:
        const unsigned long long head = (unsigned long long)(nrt - 1) * each + tiles * wl + cost;
#pragma unroll
        for (int z = 0; z < 2; ++z) {
            const unsigned long long x = z ? next : first;
            if (x < at || x >= at + size) continue;
            const unsigned long long off = x - at;
            uint32_t u, tile = 0, w = wl;
            unsigned long long in_lane;              // where the unit begins
            if (a.whole) {
                u = (uint32_t)off;
                in_lane = off;
            } else {
                const uint32_t h = divide(off, head);
                const unsigned long long rest = off - h * head;
                uint32_t rt = divide(rest, each);
                if (rt >= nrt - 1) rt = nrt - 1;
                else w = full;
                const uint32_t in = (uint32_t)(rest - (unsigned long long)rt * each);
                if (in > cost) tile = (in - cost) / w;
                u = h * nrt + rt;
                in_lane = off - in;
            }
            const unsigned long long before = tiles_in + (unsigned long long)u * tiles + tile;
            if (z == 0) {
                here->lane = b0 + tid;
                here->unit = (int)u;
                here->t = (int)tile;
                here->unit_at = at + in_lane;
                here->before = before;
                here->weight = (int)w;
            }
            else here->next = before;
        }
    };
    if (active) {
        if (a.lanes <= (int)blockDim.x) {
            locate(0);
        } else {
            size_all = tiles_all = 0;
            for (int b0 = 0; b0 < a.lanes; b0 += (int)blockDim.x) {
                scan_lanes(b0, false);
                locate(b0);
            }
        }
    }
    __syncthreads();
    if (tid == 0) {
        if (!active) here->lane = here->unit = here->t = here->count = here->weight = 0;
        else here->count = (int)((next == total ? n_tiles : here->next) - here->before);      // of at most 2^31 rows
        here->total = total;
        here->cost = (int)cost;
        here->parts = parts;
    }
}

// What the join has to know of this part.
template <int R>
__device__ __noinline__ void tell_join(const AttnArgs& a, const int* facts, const Cut* here) {
    const Walker<R> walk{a, facts};
    const Walk w = walk.start(here->lane, here->unit, here->t);
    JoinUnit u{0, 0, 0, 0, walk.lane(w.b).n0, walk.rows(w), w.h, w.rt * R};
    if (here->count > 0 && w.t > 0) {
        // a part that begins within a tile's span has that tile
        u.first = part_of(here->total, here->parts, here->unit_at + here->cost + here->weight - 1);
        u.last = part_of(here->total, here->parts, here->unit_at + here->cost + (unsigned long long)w.tiles * here->weight - 1);
        u.second = (unsigned long long)part_begin(here->total, here->parts, u.first) < here->unit_at;
        u.join = u.first == (int)blockIdx.x - 1;
    }
    reinterpret_cast<JoinUnit*>(a.ws)[blockIdx.x] = u;
}

// Whether all codes of a value row in its ring slot are zeros. (A function of its own, as it is rare: its instructions within the
// tile loop cost trees of up to 16 nodes 1 %.)
template <int D, int ROWB, int PANEL>
__device__ __noinline__ bool all_zero(const uint8_t* row) {
    for (int q = 0; q < D / 16; ++q) {
        const uint4 c = *reinterpret_cast<const uint4*>(row + q / (ROWB / 16) * PANEL + q % (ROWB / 16) * 16);
        if ((c.x | c.y | c.z | c.w) & 0x7F7F7F7Fu) return false;
    }
    return true;
}

template <int D, int R>
__global__ void __launch_bounds__(Cfg<D, R>::THREADS, 1) tree_attention(const __grid_constant__ AttnMaps maps,
                                                                          const __grid_constant__ AttnArgs a) {
    using C = Cfg<D, R>;
    constexpr int RH = C::RH, SW = C::SW;
    constexpr int NS = C::NS, NSC = C::NSC;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    const uint32_t base = smem_u32(smem), stop = base + C::OFF_MISC + 4;
    auto bar = [&](int offset, uint32_t i = 0) { return base + offset + 8 * i; };
    auto bar_ptr = [&](int offset) { return reinterpret_cast<uint64_t*>(smem + offset); };
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 4);
    volatile uint32_t* progress = reinterpret_cast<volatile uint32_t*>(smem + C::OFF_MISC + 8);      // tiles done; parts out
    volatile int* votes = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 16);       // [warpgroups][2][4 warps]
    float* F = reinterpret_cast<float*>(smem + C::OFF_F);
    int* facts = reinterpret_cast<int*>(smem + C::OFF_LANE);
    unsigned long long* scratch = reinterpret_cast<unsigned long long*>(smem + C::OFF_SCAN);
    Cut* here = reinterpret_cast<Cut*>(smem + C::OFF_SCAN + 512);

    const int tid = threadIdx.x, warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0), lane = tid & 31;
    const int H = a.c.n_kv_heads, G = a.group;
    pdl_trigger();
    if (tid == 0) {
        auto init = [&](int offset, int n, int arrivals) {
            for (int i = 0; i < n; ++i) mbar_init(bar_ptr(offset) + i, arrivals);
        };
        init(C::B_FULL, NS, 1); init(C::B_EMPTY, NS, 1); init(C::B_SCFULL, NSC, 1); init(C::B_SCEMPTY, NSC, SW / 2);
        init(C::B_SFULL, C::SB, 1); init(C::B_VOTE, 4, 4); init(C::B_MAXIMA, 4, 4); init(C::B_PFULL, 2, SW / 2); init(C::B_PFREE, 2, 1);
        init(C::B_QFULL, 2, 4); init(C::B_QFREE, 2, 1); init(C::B_OFULL, 2, 1); init(C::B_OFREE, 2, 4);
        init(C::B_LFULL, 1, SW); init(C::B_LFREE, 1, 4); init(C::B_QMAX, 1, 4); init(C::B_DONE, 1, 1); init(C::B_DRAIN, 1, 1);
        *abort_flag = 0;
        progress[0] = progress[1] = 0;
        fence_barrier_init();
        prefetch_tmap(&maps.k);
        prefetch_tmap(&maps.v);
    }
    if (warp == SW + 5) { tmem_alloc(tmem_slot, C::TMEM_COLS); tmem_relinquish(); }
    pdl_wait();

    // ---------------------------------------------------------------- the cut
    cut_run<R>(a, facts, scratch, here);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const int count = here->count;
    const Walker<R> walk{a, facts};
    Walk w = walk.start(here->lane, here->unit, here->t);
    int left = count;
    uint32_t issued = 0;                             // ring fills, by the producer

    if (warp < SW) {
        // ------------------------------------------------------------ softmax
        if constexpr (R == 64) regs_up<96>();
        const int wg = warp >> 2, wl = warp & 3;     // warpgroup, warp in it
        const int g = wg / C::HALVES, h = wg % C::HALVES;             // group, which of its tree rows
        const int j = tid & 127;                     // this thread's row of the tile
        const uint32_t trow = tmem + ((uint32_t)(wl * 32) << 16) + h * RH;
        float* off = F + C::F_O + g * R + h * RH;
        float* alpha = F + C::F_AL + g * R + h * RH;
        uint32_t i = 0, k = 0, sets = 0, polls = 0, piece = 0;       // tile of the CTA; of this group; references set; votes; part
        bool ok = true;
        while (left > 0 && ok) {
            const int nt = left < w.tiles - w.t ? left : w.tiles - w.t;
            f32x2 l2[RH / 2];
            float M = -INFINITY;                     // reference of tree row `lane`
#pragma unroll
            for (int r = 0; r < RH / 2; ++r) l2[r] = 0ull;
            const float* qf = F + C::F_QF + (piece & 3) * R + h * RH;
            const Lane ln = walk.lane(w.b);
            const int len = ln.len, prefix = ln.len - ln.n;
            const int row0 = w.rt * R + h * RH;      // this warpgroup's tree rows in the lane
            const int live = ln.n * G - row0;        // how many of them there are (more than RH: all; none or less: none)
            int ev_most = 0;                         // largest value scale byte so far
            bool set = true;                         // the reference is to be set (a part's first tile)
            const uint32_t i1 = i + nt;              // the part's tiles are taken in turn by the two groups
            int t = w.t + (int)((i ^ (uint32_t)g) & 1);
            for (i += (i ^ (uint32_t)g) & 1; i < i1; i += 2, t += 2) {
                if (C::HALVES > 1 && live <= 0) {    // the last unit of a lane: its first half has all the rows
                    const int sc = (int)(i % NSC);
                    if (!warp_wait_at(bar(C::B_SCFULL, sc), (i / NSC) & 1, stop)) { ok = false; break; }
                    if (k > 0 && !warp_wait_at(bar(C::B_PFREE, g), (k - 1) & 1, stop)) { ok = false; break; }
                    if (lane == 0) {
                        arrive_at(bar(C::B_SCEMPTY, sc));
                        arrive_at(bar(C::B_PFULL, g));
                    }
                    ++k;
                    continue;
                }
                const int j0 = t * TILE;
                const int valid = len - j0;      // rows of the tile that exist (can be <= 0 or > 128)
                const bool masked = j0 + TILE > prefix;
                // what this row is to each tree row
                uint32_t sees = ~0u;
                if (masked) {
                    const int n = j0 + j - prefix;
                    if (j >= valid) {
                        sees = 0u;
                    } else if (n >= 0) {
                        sees = 0u;
                        const Lane ln = walk.lane(w.b);
                        const int end = ln.n * G < row0 + RH ? ln.n * G : row0 + RH;
                        for (int t1 = row0 / G; t1 * G < end; ++t1) {
                            const bool see = a.mask ? (a.mask[(int64_t)(ln.n0 + t1) * a.mask_words + (n >> 5)] >> (n & 31)) & 1
                                                    : n <= t1;
                            if (!see) continue;
                            int lo = t1 * G - row0, hi = lo + G;
                            lo = lo < 0 ? 0 : lo;
                            hi = hi > RH ? RH : hi;
                            sees |= (hi == 32 ? ~0u : (1u << hi) - 1u) & ~((1u << lo) - 1u);
                        }
                    }
                }
                const int sc = (int)(i % NSC);
                if (!warp_wait_at(bar(C::B_SCFULL, sc), (i / NSC) & 1, stop)) { ok = false; break; }
                const uint8_t* scales = smem + C::OFF_SC + sc * C::SC_BYTES;
                const uint32_t ks = scales[j];
                uint32_t vs = scales[TILE + j];
                const int2 range = *reinterpret_cast<const int2*>(scales + 2 * TILE);
                __syncwarp();
                if (lane == 0) arrive_at(bar(C::B_SCEMPTY, sc));
                ev_most = max(ev_most, range.x);
                bool wide = false;
                if (ev_most > range.y + WIDE) {
                    if (__any_sync(0xFFFFFFFFu, vs == ZERO_BYTE && sees != 0u)) {
                        // The values have arrived when their slot's fill is complete. The fill before it in the slot, which the
                        // parity cannot tell from it, is one of a tile before this group's last or that tile itself.
                        const uint32_t f = 2 * i + 1;
                        if (k > 0 && !warp_wait_at(bar(C::B_PFREE, g), (k - 1) & 1, stop)) { ok = false; break; }
                        if (!warp_wait_at(bar(C::B_FULL, f % NS), (f / NS) & 1, stop)) { ok = false; break; }
                        if (vs == ZERO_BYTE && all_zero<D, C::ROWB, C::PANEL>(smem + C::OFF_RING + (f % NS) * C::SLOT + j * C::ROWB)) vs = LEAST_BYTE;
                        __syncwarp();
                    }
                    // p could underflow in a row that matters to the sum of weights, p 2^-ev: the warp's weights then get an
                    // exponential of their own.
                    wide = __any_sync(0xFFFFFFFFu, sees != 0u && ev_most > (int)vs + WIDE);
                }
                const int evi = vs == 255u ? 0 : (int)vs - 127;       // a NaN row that is not seen weighs nothing
                const float ev = vs == 255u ? __uint_as_float(0x7FC00000u) : (float)evi;
                const f32x2 ev2 = pack2(ev, ev);
                const uint32_t sb = i % C::SB;
                if (!warp_wait_at(bar(C::B_SFULL, sb), (i / C::SB) & 1, stop)) { ok = false; break; }
                tc_fence_after();
                const uint32_t srow = trow + sb * R;
                const float2 unit = *reinterpret_cast<const float2*>(F + C::F_QU + (piece & 3) * 2);
                const bool rowwise = unit.y != 0.0f;
                const float cj = a.scale_log2 * e8m0_to_float(ks) * unit.x;
                const f32x2 cj2 = pack2(cj, cj);
                // One pass over the tile, a second one where a score has passed the limit
                f32x2 y[RH / 2];                     // s' + off, the exponent of p, then p; rows not seen are -inf
                bool setting = set;
                for (;;) {
                    {
                        uint32_t s[RH];
                        tc_load(srow, s);
#pragma unroll
                        for (int q = 0; q < RH / 2; ++q) y[q] = pack2(__uint_as_float(s[2 * q]), __uint_as_float(s[2 * q + 1]));
                    }
                    if (rowwise) {
#pragma unroll
                        for (int q = 0; q < RH / 2; ++q) y[q] = mul2(y[q], *reinterpret_cast<const f32x2*>(qf + 2 * q));
                    }
#pragma unroll
                    for (int q = 0; q < RH / 2; ++q) y[q] = fma2(y[q], cj2, ev2);
                    if (masked) {
#pragma unroll
                        for (int q = 0; q < RH / 2; ++q) {
                            const float2 s = unpack2(y[q]);
                            y[q] = pack2((sees >> (2 * q)) & 1 ? s.x : -INFINITY, (sees >> (2 * q + 1)) & 1 ? s.y : -INFINITY);
                        }
                    }
                    if (setting) {
                        // The tile's maximum of s' in every tree row, over the warpgroup's 128 threads. Rows are halved while
                        // lanes are paired: lane l ends with row l (of 16: l / 2). Shuffles, not redux.sync: its
                        // results come one by one through the uniform registers (100 clocks each).
                        float* wmax = F + C::F_WMAX + (wg * 2 + (sets & 1)) * 4 * RH;
                        constexpr int HALF = RH / 2;
                        float v[HALF];
#pragma unroll
                        for (int r = 0; r < HALF; r += 2) {
                            const float2 x0 = unpack2(y[r / 2]), x1 = unpack2(y[(r + HALF) / 2]);
                            const bool up = lane & 16;
                            v[r] = fmaxf(up ? x1.x : x0.x, __shfl_xor_sync(0xFFFFFFFFu, up ? x0.x : x1.x, 16));
                            v[r + 1] = fmaxf(up ? x1.y : x0.y, __shfl_xor_sync(0xFFFFFFFFu, up ? x0.y : x1.y, 16));
                        }
                        int n = HALF;
#pragma unroll
                        for (int o = 8; o > 0; o >>= 1) {
                            n /= 2;
                            const bool up = lane & o;
#pragma unroll
                            for (int r = 0; r < HALF / 2; ++r) {
                                if (r >= n) break;
                                v[r] = fmaxf(up ? v[r + n] : v[r], __shfl_xor_sync(0xFFFFFFFFu, up ? v[r] : v[r + n], o));
                            }
                            if (n == 0) v[0] = fmaxf(v[0], __shfl_xor_sync(0xFFFFFFFFu, v[0], o));
                        }
                        wmax[wl * RH + (RH < 32 ? lane >> 1 : lane)] = v[0];
                        __syncwarp();
                        if (lane == 0) arrive_at(bar(C::B_MAXIMA, wg));
                        if (!warp_wait_at(bar(C::B_MAXIMA, wg), sets & 1, stop)) { ok = false; break; }
                        ++sets;
                        if (RH == 32 || lane < RH) { // every warp writes the same factors
                            const float m = fmaxf(fmaxf(wmax[lane], wmax[RH + lane]), fmaxf(wmax[2 * RH + lane], wmax[3 * RH + lane]));
                            const float Mn = fmaxf(M, m);
                            // a row that has seen nothing: the first score it sees passes any limit
                            off[lane] = Mn == -INFINITY ? 1e30f : P_EXP - Mn;
                            const float root = M == -INFINITY ? 0.0f : ex2(0.5f * (M - Mn));
                            alpha[lane] = root;
                            alpha[2 * R + lane] = root * root;
                            M = Mn;
                        }
                        __syncwarp();
#pragma unroll
                        for (int q = 0; q < RH / 2; ++q) {
                            const f32x2 al = *reinterpret_cast<const f32x2*>(alpha + 2 * q);
                            l2[q] = mul2(mul2(l2[q], al), al);
                        }
                    }
                    float top = -INFINITY;
#pragma unroll
                    for (int q = 0; q < RH / 2; q += 2) {
                        const ulonglong2 o = *reinterpret_cast<const ulonglong2*>(off + 2 * q);
                        y[q] = add2(y[q], o.x);
                        y[q + 1] = add2(y[q + 1], o.y);
                        const float2 s0 = unpack2(y[q]), s1 = unpack2(y[q + 1]);
                        top = max3(max3(top, s0.x, s0.y), s1.x, s1.y);
                    }
                    if (!setting) {
                        const bool over = __any_sync(0xFFFFFFFFu, top > P_EXP_MAX);
                        if (lane == 0) {
                            votes[wg * 8 + (polls & 1) * 4 + wl] = over;
                            arrive_at(bar(C::B_VOTE, wg));
                        }
                    }
                    // P of this group's previous tile has been read, and its O added up
                    if (k > 0 && !warp_wait_at(bar(C::B_PFREE, g), (k - 1) & 1, stop)) { ok = false; break; }
                    if (setting && !set) {           // what has been added up is scaled down to the new reference
                        tc_fence_after();
                        const uint32_t orow = tmem + ((uint32_t)(wl * 32) << 16) + C::TMEM_O + (g * 2 + (piece & 1)) * C::MB * C::OC + h * RH;
                        for (int c0 = 0; c0 < C::MB * C::PARTS * RH; c0 += 8) {
                            const uint32_t at = orow + (c0 / RH) * R + c0 % RH;
                            uint32_t o[8];
                            tc_ld_x8(at, o);
                            tc_wait_ld();
                            const float* al = alpha + 2 * R + c0 % RH;
#pragma unroll
                            for (int q = 0; q < 8; ++q) o[q] = __float_as_uint(__uint_as_float(o[q]) * al[q]);
                            tc_st_x8(at, make_uint4(o[0], o[1], o[2], o[3]), make_uint4(o[4], o[5], o[6], o[7]));
                        }
                        tc_wait_st();
                    }
                    uint8_t* P = smem + C::OFF_P + g * C::PBUF + j * R;
                    const int swz = R == 64 ? (j >> 1) & 3 : R == 32 ? (j >> 2) & 1 : 0;
#pragma unroll
                    for (int c0 = 0; c0 < RH; c0 += 16) {
                        if (c0 >= live) break;       // what P then holds there becomes columns of O that nobody reads
                        uint32_t hi[4], mid[4], lo[4];
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            uint32_t a2[2], b2[2], c2[2];
#pragma unroll
                            for (int z = 0; z < 2; ++z) {
                                f32x2& e = y[c0 / 2 + 2 * q + z];
                                const float2 s = unpack2(e);
                                const float p0 = ex2(s.x), p1 = ex2(s.y);
                                if (!wide) e = pack2(p0, p1);
                                auto bits = [](__half2 x) { return *reinterpret_cast<const uint32_t*>(&x); };
                                auto halves = [](uint32_t x) { return *reinterpret_cast<const __half2*>(&x); };
                                // hi is cut off (NaN, 0x7FFF, stays NaN), the rests are exact, mid and lo rounded to
                                // nearest. No sum carries out of its half.
                                const __half2 ph = __floats2half2_rn(p0, p1);
                                a2[z] = bits(ph);
                                const __half2 r1 = __hsub2(ph, halves(a2[z] & 0xFF00FF00u));
                                b2[z] = bits(r1) + 0x00800080u;
                                c2[z] = bits(__hsub2(r1, halves(b2[z] & 0xFF00FF00u))) + 0x00800080u;
                            }
                            hi[q] = __byte_perm(a2[0], a2[1], 0x7531);
                            mid[q] = __byte_perm(b2[0], b2[1], 0x7531);
                            lo[q] = __byte_perm(c2[0], c2[1], 0x7531);
                        }
                        uint8_t* at = P + (((h * (RH / 16) + c0 / 16) ^ swz) << 4);
                        *reinterpret_cast<uint4*>(at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                        *reinterpret_cast<uint4*>(at + TILE * R) = make_uint4(mid[0], mid[1], mid[2], mid[3]);
                        *reinterpret_cast<uint4*>(at + 2 * TILE * R) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                    }
                    if (setting) break;
                    if (!warp_wait_at(bar(C::B_VOTE, wg), polls & 1, stop)) { ok = false; break; }
                    const volatile int* got = votes + wg * 8 + (polls & 1) * 4;
                    ++polls;
                    if (!(got[0] | got[1] | got[2] | got[3])) break;
                    setting = true;
                }
                if (!ok) break;
                set = false;
                if (valid < TILE && h == 0) {
                    // rows past the lane's end hold anything: their values are cleared, so that 0 * NaN does not arise
                    const uint32_t f = 2 * i + 1;
                    if (!warp_wait_at(bar(C::B_FULL, f % NS), (f / NS) & 1, stop)) { ok = false; break; }
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
                if (lane == 0) arrive_at(bar(C::B_PFULL, g));
                if (wide) {
                    const float evf = (float)(evi - (L_OWN - L_EXP)), wj = exp2_int(-L_OWN);
                    const f32x2 wj2 = pack2(wj, wj);
#pragma unroll
                    for (int q = 0; q < RH / 2; ++q) {
                        const float2 s = unpack2(y[q]);
                        l2[q] = fma2(pack2(ex2(s.x - evf), ex2(s.y - evf)), wj2, l2[q]);
                    }
                } else {
                    const float wj = exp2_whole(-evi - L_EXP);
                    const f32x2 wj2 = pack2(wj, wj);
#pragma unroll
                    for (int q = 0; q < RH / 2; ++q) l2[q] = fma2(y[q], wj2, l2[q]);
                }
                ++k;
            }
            if (!ok) break;
            i = i1;
            // the part's sums over this group's rows
            if (piece > 0 && !warp_wait_at(bar(C::B_LFREE), (piece - 1) & 1, stop)) break;
            float v[RH];
#pragma unroll
            for (int r = 0; r < RH / 2; ++r) {
                const float2 p = unpack2(l2[r]);
                v[2 * r] = p.x;
                v[2 * r + 1] = p.y;
            }
            int n = RH;                              // as for the maxima
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                n /= 2;
                const bool up = lane & o;
#pragma unroll
                for (int r = 0; r < RH / 2; ++r) {
                    if (r >= n) break;
                    v[r] = (up ? v[r + n] : v[r]) + __shfl_xor_sync(0xFFFFFFFFu, up ? v[r] : v[r + n], o);
                }
                if (n == 0) v[0] += __shfl_xor_sync(0xFFFFFFFFu, v[0], o);
            }
            F[C::F_L + (g * 4 + wl) * R + h * RH + (RH < 32 ? lane >> 1 : lane)] = v[0];
            if (wl == 0 && (RH == 32 || lane < RH)) F[C::F_M + g * R + h * RH + lane] = M;
            __syncwarp();
            if (lane == 0) arrive_at(bar(C::B_LFULL));
            left -= nt;
            walk.advance(w, nt, left > 0);
            ++piece;
        }
    } else if (warp < SW + 4) {
        // ------------------------------------------------------------ queries and outputs
        if constexpr (R == 64) regs_down<56>();
        const int wl = warp & 3;
        // the queries of the next unit; all loads of a batch are under way before the first is used
        Walk wq = w;
        int qleft = left;
        uint32_t qpiece = 0;
        const int row_step = 4 * (32 / (D / 8));     // tree rows the four warps take at once
        auto convert = [&]() -> bool {
            constexpr int LPR = D / 8, RPW = 32 / LPR;                // lanes a row, rows a warp takes at once
            constexpr int ITER = R / (4 * RPW) > 0 ? R / (4 * RPW) : 1;
            const int part = lane % LPR, sub = lane / LPR;
            const uint32_t qb = qpiece & 1;
            const int rows = walk.rows(wq), row0 = wq.rt * R, n0 = walk.lane(wq.b).n0;
            uint8_t* Q = smem + C::OFF_Q + qb * C::QBUF;
            float* qf = F + C::F_QF + (qpiece & 3) * R;
            static_assert(ITER <= 8, "a lane's rows are held in registers");
            const int first = row0 + wl * RPW + sub;
            int node = first / G, head = first - node * G;
            uint4 raw[ITER];
#pragma unroll
            for (int b = 0; b < ITER; ++b) {
                raw[b] = make_uint4(0u, 0u, 0u, 0u);
                if ((b * 4 + wl) * RPW + sub < rows)
                    raw[b] = *reinterpret_cast<const uint4*>(a.q + (n0 + node) * a.q_token_stride + (wq.h * G + head) * a.q_head_stride + part * 8);
                node += row_step / G;
                head += row_step % G;
                if (head >= G) { head -= G; ++node; }
            }
            // max |x| of each row (bf16 bits; NaN stays), and of the unit's rows the largest and the smallest but zero
            uint32_t* keys = reinterpret_cast<uint32_t*>(qf);
            uint32_t most = 0, least = 0x7FFFu;
#pragma unroll
            for (int b = 0; b < ITER; ++b) {
                auto abs2 = [](uint32_t v) {
                    v &= 0x7FFF7FFFu;
                    return *reinterpret_cast<const __nv_bfloat162*>(&v);
                };
                __nv_bfloat162 m = __hmax2_nan(__hmax2_nan(abs2(raw[b].x), abs2(raw[b].y)), __hmax2_nan(abs2(raw[b].z), abs2(raw[b].w)));
                m = __hmax2_nan(m, __lowhigh2highlow(m));
#pragma unroll
                for (int o = LPR / 2; o > 0; o >>= 1) m = __hmax2_nan(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
                const uint32_t key = *reinterpret_cast<const uint32_t*>(&m) & 0xFFFFu;
                const int u = (b * 4 + wl) * RPW + sub;
                if (part == 0 && u < R) keys[u] = key;
                most = max(most, key);
                if (key) least = min(least, key);
            }
            uint32_t* qx = reinterpret_cast<uint32_t*>(F + C::F_QX);
            most = __reduce_max_sync(0xFFFFFFFFu, most);
            least = __reduce_min_sync(0xFFFFFFFFu, least);
            if (lane == 0) {
                qx[(qpiece & 1) * 4 + wl] = most;
                qx[8 + (qpiece & 1) * 4 + wl] = least;
                arrive_at(bar(C::B_QMAX));
            }
            if (!warp_wait_at(bar(C::B_QMAX), qpiece & 1, stop)) return false;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                most = max(most, qx[(qpiece & 1) * 4 + q]);
                least = min(least, qx[8 + (qpiece & 1) * 4 + q]);
            }
            // Rows within 2^4 of one another share one power of two, and the scores need no factor of their row's;
            // the smallest rows' low parts then end 2^-13 below their own maximum. (Subnormal rows count as 2^-126.)
            auto up_of = [](uint32_t k) {            // 2^up * maximum is in [128, 256)
                const int up = k ? 134 - (int)(k >> 7) : 0;
                return up > 120 ? 120 : (up < -120 ? -120 : up);
            };
            const int unit_up = up_of(most);
            const bool rowwise = most >= 0x7F80u || (least < most && up_of(least) - unit_up > 4);
            if (!warp_wait_at(bar(C::B_QFREE, qb), ((qpiece >> 1) & 1) ^ 1, stop)) return false;
            if (wl == 0 && lane == 0)
                *reinterpret_cast<float2*>(F + C::F_QU + (qpiece & 3) * 2) = make_float2(rowwise ? 1.0f : exp2_int(-unit_up), rowwise ? 1.0f : 0.0f);
            const int byte = part * 8, panel = byte / C::ROWB, in_row = byte % C::ROWB;
#pragma unroll
            for (int b = 0; b < ITER; ++b) {
                const int u = (b * 4 + wl) * RPW + sub;
                const uint32_t key = rowwise && u < R ? keys[u] : 0u;
                __syncwarp();
                const int up = rowwise ? up_of(key) : unit_up;
                const float gain = exp2_int(up);
                const f32x2 gain2 = pack2(gain, gain);
                const uint32_t in[4] = {raw[b].x, raw[b].y, raw[b].z, raw[b].w};
                uint32_t hi[4], lo[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    // a scaled bf16 value is exact in fp16 (down to 2^-16, far below what lo resolves)
                    const float2 x = unpack2(mul2(pack2(__uint_as_float(in[e] << 16), __uint_as_float(in[e] & 0xFFFF0000u)), gain2));
                    const __half2 xh = __floats2half2_rn(x.x, x.y);
                    hi[e] = __nv_cvt_halfraw2_to_fp8x2(xh, __NV_SATFINITE, __NV_E4M3);
                    const __half2 rest = __hsub2(xh, __half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)hi[e], __NV_E4M3)));
                    lo[e] = __nv_cvt_halfraw2_to_fp8x2(rest, __NV_SATFINITE, __NV_E4M3);
                }
                if (u < R) {
                    // a row that is not finite: its scores become NaN
                    if (rowwise && part == 0) qf[u] = key >= 0x7F80u ? __uint_as_float(0x7FC00000u) : exp2_int(-up);
                    const int swz = C::ROWB == 128 ? u & 7 : (u >> 1) & 3;     // the same for row R + u
                    uint8_t* at = Q + panel * C::QROWS * C::ROWB + u * C::ROWB + (((in_row >> 4) ^ swz) << 4) + (in_row & 15);
                    *reinterpret_cast<uint2*>(at) = make_uint2(__byte_perm(hi[0], hi[1], 0x5410), __byte_perm(hi[2], hi[3], 0x5410));
                    *reinterpret_cast<uint2*>(at + R * C::ROWB) = make_uint2(__byte_perm(lo[0], lo[1], 0x5410), __byte_perm(lo[2], lo[3], 0x5410));
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) arrive_at(bar(C::B_QFULL, qb));
            const int nt = qleft < wq.tiles - wq.t ? qleft : wq.tiles - wq.t;
            qleft -= nt;
            ++qpiece;
            walk.advance(wq, nt, qleft > 0);
            return true;
        };

        constexpr int RL = R > 32 ? R / 32 : 1;    // tree rows a lane looks after
        float* st = F + C::F_ST + wl * 3 * R;
        int* place = reinterpret_cast<int*>(st + 2 * R);
        const bool on = D >= 128 || lane < 16;       // M = 64 leaves 16 rows in each quarter of the lanes
        const int d0 = D >= 128 ? wl * 32 + lane : wl * 16 + (lane & 15);
        uint32_t i0 = 0, piece = 0;                  // the part's first tile
        if (left > 0) (void)convert();
        while (left > 0) {
            const int nt = left < w.tiles - w.t ? left : w.tiles - w.t;
            if (qleft > 0 && !convert()) break;
            const uint32_t ob = piece & 1;
            if (!warp_wait_at(bar(C::B_LFULL), piece & 1, stop) || !warp_wait_at(bar(C::B_OFULL, ob), (piece >> 1) & 1, stop)) break;
            tc_fence_after();
            const int rows = walk.rows(w), row0 = w.rt * R, n0 = walk.lane(w.b).n0;
            const bool whole = nt == w.tiles;
            // a group without a tile in this part has no O
            const bool has0 = nt > 1 || (i0 & 1) == 0, has1 = nt > 1 || (i0 & 1) == 1;
            float* part = reinterpret_cast<float*>(a.ws + parts_offset(gridDim.x)) +
                          (size_t)(2 * blockIdx.x + (left == count ? 0 : 1)) * part_floats(R, D);
#pragma unroll
            for (int r = 0; r < RL; ++r) {
                const int u = r * 32 + lane;
                if (R < 32 && u >= R) break;
                auto sum = [&](int g) {
                    const float* ls = F + C::F_L + g * 4 * R + u;
                    return (ls[0] + ls[R]) + (ls[2 * R] + ls[3 * R]);
                };
                const float M0 = F[C::F_M + u], M1 = F[C::F_M + R + u], M = fmaxf(M0, M1);
                float f0 = M0 == -INFINITY ? 0.0f : ex2(0.5f * (M0 - M)), f1 = M1 == -INFINITY ? 0.0f : ex2(0.5f * (M1 - M));
                const float L = sum(0) * f0 * f0 + sum(1) * f1 * f1;  // sums may be NaN
                f0 *= f0;
                f1 *= f1;
                const int node = (row0 + u) / G, row = node * a.n_q_heads + row0 + u - node * G;      // of the lane and kv head: 2^26 at most
                if (whole) {
                    // out = O / (L 2^L_EXP); lse = ln 2 (M - P_EXP + L_EXP + log2 L): p carries 2^P_EXP, L 2^-L_EXP
                    const float inv = L == 0.0f ? 0.0f : exp2_int(-L_EXP) / L;
                    f0 *= inv;
                    f1 *= inv;
                    if (wl == 0 && a.lse && u < rows)
                        a.lse[(int64_t)n0 * a.n_q_heads + w.h * G + row] = L == 0.0f ? -INFINITY : (M - (P_EXP - L_EXP) + log2f(L)) * 0.69314718055994531f;
                } else if (wl == 0 && u < rows) {
                    part[R * D + u] = M;
                    part[R * D + R + u] = L;
                }
                // a group without a tile has no O: what lies there is read, and cleared below
                st[u] = f0;
                st[R + u] = f1;
                place[u] = row;                  // in vectors of D: the offset in values can pass 32 bits
            }
            __syncwarp();
            if (lane == 0) arrive_at(bar(C::B_LFREE));
            __nv_bfloat16* out = a.out + ((int64_t)n0 * a.n_q_heads + w.h * G) * D + d0;
            const uint32_t orow = tmem + ((uint32_t)(wl * 32) << 16) + C::TMEM_O + ob * C::MB * C::OC;
            for (int c0 = 0; c0 < rows; c0 += 16) {
#pragma unroll
                for (int m = 0; m < C::MB; ++m) {
                    uint32_t o0[16], o1[16];
                    tc_ld_x16(orow + m * C::OC + c0, o0);
                    tc_ld_x16(orow + (2 * C::MB + m) * C::OC + c0, o1);
                    tc_wait_ld();
#pragma unroll
                    for (int z = 1; z < C::PARTS; ++z) {
                        uint32_t x0[16], x1[16];
                        tc_ld_x16(orow + m * C::OC + z * R + c0, x0);
                        tc_ld_x16(orow + (2 * C::MB + m) * C::OC + z * R + c0, x1);
                        tc_wait_ld();
#pragma unroll
                        for (int q = 0; q < 16; ++q) {
                            o0[q] = __float_as_uint(__uint_as_float(o0[q]) + __uint_as_float(x0[q]));
                            o1[q] = __float_as_uint(__uint_as_float(o1[q]) + __uint_as_float(x1[q]));
                        }
                    }
#pragma unroll
                    for (int q = 0; q < 16; q += 4) {
                        const float4 f0 = *reinterpret_cast<const float4*>(st + c0 + q), f1 = *reinterpret_cast<const float4*>(st + R + c0 + q);
                        const int4 at = *reinterpret_cast<const int4*>(place + c0 + q);
                        const float g0[4] = {f0.x, f0.y, f0.z, f0.w}, g1[4] = {f1.x, f1.y, f1.z, f1.w};
                        const int to[4] = {at.x, at.y, at.z, at.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float x = (has0 ? __uint_as_float(o0[q + e]) * g0[e] : 0.0f) + (has1 ? __uint_as_float(o1[q + e]) * g1[e] : 0.0f);
                            if (!on || c0 + q + e >= rows) continue;
                            if (whole) out[(int64_t)to[e] * D + m * 128] = __float2bfloat16_rn(x);
                            else part[(c0 + q + e) * D + m * 128 + d0] = x;
                        }
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive_at(bar(C::B_OFREE, ob));
            i0 += nt;
            left -= nt;
            walk.advance(w, nt, left > 0);
            ++piece;
            progress[1] = piece;
        }
        __syncwarp();
        if (wl == 0 && lane == 0) arrive_at(bar(C::B_DONE));           // the block's last work, or it has been stopped
    } else {
        if (warp == SW + 7 && lane == 0) tell_join<R>(a, facts, here);       // (before registers are handed back: the call may use them)
        __syncwarp();
        if constexpr (R == 64) regs_down<40>();
        const int P = 1 << a.page_shift;
        // A warp of its own has few instructions a tile to spare (each waits for the one before: five clocks): within a part the
        // way through the table is one add a tile. Ids are looked at when used, so that lookups stay under way.
        auto checked = [&](int page, bool tell) {
            if (page >= 0 && page < a.c.n_pages) return page;
            if (tell) record_error(a.err, MOE_DEV_BAD_PAGE);
            return 0;
        };
        if (warp == SW + 4) {
            // -------------------------------------------------------- TMA: lane l copies the tile's l-th page (or 128 rows of it)
            const int rows_a_page = P < TILE ? P : TILE;
            const uint32_t ids = base + C::OFF_TID + (lane & 7) * 4;         // eight pages a tile at most: [PT][8]
            bool ok = true;
            uint32_t f = 0, slot = 0, round = 1;     // fill of the ring, its slot, the parity of the slot's last use
            while (left > 0 && ok) {
                const int nt = left < w.tiles - w.t ? left : w.tiles - w.t;
                const int first = w.t * TILE + lane * rows_a_page;
                // past the part or the lane's rows, or no piece of a tile for this lane: nothing to copy
                const int end = lane * rows_a_page >= TILE ? 0 : min(walk.lane(w.b).len, (w.t + nt) * TILE), hp = w.h * P;
                const int32_t* table = a.table + (int64_t)w.b * a.width;
                // Ids come PT tiles ahead through shared memory: a register handed from one to the next would wait for its load.
                constexpr int PT = C::PT;
                auto look = [&](int d) {
                    const int at = first + d * TILE;
                    if (d < nt && at < end) cp_async_4(ids + (d % PT) * 32, table + (at >> a.page_shift));
                    cp_async_commit();
                };
                const bool few = nt < PT;            // then all at once
#pragma unroll 1
                for (int d = 0; d < (few ? nt : PT); ++d) look(d);
#pragma unroll 1
                for (int d = 0; d < nt && ok; ++d) {
                    const int at = first + d * TILE;
                    const bool some = at < end;
                    if (few) cp_async_wait<0>(); else cp_async_wait<PT - 1>();
                    int row = 0;
                    if (some) row = checked(read_at(ids + (d % PT) * 32), true) * H * P + hp + (at & (P - 1));
                    const uint32_t bytes = __popc(__ballot_sync(0xFFFFFFFFu, some)) * rows_a_page * D;
                    look(d + PT);                    // into the place that has just been read
#pragma unroll 1
                    for (int v = 0; v < 2; ++v) {
                        if (!warp_wait_at(bar(C::B_EMPTY, slot), round, stop)) { ok = false; break; }
                        if (lane == 0) arrive_expect_tx_at(bar(C::B_FULL, slot), bytes);
                        ++f;
                        __syncwarp();
                        if (some)
#pragma unroll
                            for (int q = 0; q < C::PANELS; ++q)
                                tma_load_at(base + C::OFF_RING + slot * C::SLOT + q * C::PANEL + lane * rows_a_page * C::ROWB,
                                            v ? &maps.v : &maps.k, bar(C::B_FULL, slot), q * 128, row);
                        if (++slot == NS) { slot = 0; round ^= 1; }
                    }
                }
                left -= nt;
                walk.advance(w, nt, left > 0);
            }
            cp_async_wait<0>();
            issued = f;
        } else if (warp == SW + 5) {
            // -------------------------------------------------------- MMA issue. The loop is uniform over the warp and one elected
            // lane issues, so that descriptors stay in uniform registers (39 clocks an MMA of N = 16 against 120
            // from a loop that one lane runs).
            constexpr uint64_t KD = desc_base(C::ROWB == 128 ? 2 : 4, 8 * C::ROWB, 8 * C::ROWB);       // K, Q (along K) and V (along M): one atom, 8 rows
            // P: 8 R bytes from eight cache rows to the next, TILE R from hi to mid to lo. (Without a swizzle the strides of
            // the contiguous axis and of the groups stand in each other's fields.)
            constexpr uint64_t PD = R == 16 ? desc_base(0, 8 * R, TILE * R) : desc_base(R == 64 ? 4 : 6, TILE * R, 8 * R);
            constexpr uint32_t ID_S = idesc_f8(128, R, 0, 0, 0);
            constexpr uint32_t ID_PV = idesc_f8(D < 128 ? 64 : 128, C::OC, 1, 1, 1);
            const uint32_t tm = __shfl_sync(0xFFFFFFFFu, tmem, 0);
            const uint64_t ring = desc_at(KD, smem_u32(smem + C::OFF_RING));
            const uint64_t qd = desc_at(KD, smem_u32(smem + C::OFF_Q)), pd = desc_at(PD, smem_u32(smem + C::OFF_P));
            // S of tile i = K (Q hi)^T + K (Q lo)^T; `last` of its part
            auto qk = [&](uint32_t i, uint32_t qb, bool last) {
                const uint32_t s = (2 * i) % NS;
                const uint64_t kd = ring + (uint64_t)(s * (C::SLOT >> 4)), q = qd + (uint64_t)(qb * (C::QBUF >> 4));
                const uint32_t d = tm + (i % C::SB) * R;
                if (elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < 2 * D / 32; ++kk) {
                        constexpr int STEPS = C::ROWB / 32, HALF = D / 32;
                        const int k = kk % HALF;
                        tc_mma_f8(d, kd + (((k / STEPS) * C::PANEL + (k % STEPS) * 32) >> 4),
                                  q + (((k / STEPS) * C::QROWS * C::ROWB + (kk / HALF) * R * C::ROWB + (k % STEPS) * 32) >> 4), ID_S,
                                  kk ? 1u : 0u);
                    }
                    commit_at(bar(C::B_EMPTY, s));
                    commit_at(bar(C::B_SFULL, i % C::SB));
                    if (last) commit_at(bar(C::B_QFREE, qb));
                }
                __syncwarp();
            };
            // O of the tile's group += tile n; fresh: the group's first of the part, ends: the part's last
            auto pv = [&](uint32_t n, uint32_t part, bool fresh, bool ends) {
                const uint32_t g = n & 1, s = (2 * n + 1) % NS;
                const uint64_t vd = ring + (uint64_t)(s * (C::SLOT >> 4)), p = pd + (uint64_t)(g * (C::PBUF >> 4));
                const uint32_t o = tm + C::TMEM_O + (g * 2 + (part & 1)) * C::MB * C::OC;
                const uint32_t add = fresh ? 0u : 1u;
                if (elect_one()) {
#pragma unroll
                    for (int m = 0; m < C::MB; ++m)
#pragma unroll
                        for (int kk = 0; kk < 12 / C::PARTS; ++kk)     // four steps of 32 rows; with hi, with mid and with lo
                            tc_mma_f8(o + m * C::OC, vd + ((m * C::PANEL + (kk & 3) * 32 * C::ROWB) >> 4),
                                      p + (((kk >> 2) * TILE * R + (kk & 3) * 32 * R) >> 4), ID_PV, kk ? 1u : add);
                    commit_at(bar(C::B_EMPTY, s));
                    commit_at(bar(C::B_PFREE, g));
                    if (ends) commit_at(bar(C::B_OFULL, part & 1));
                }
                __syncwarp();
            };
            // Whatever is ready is issued: a finished P frees its values' place in the ring, the next keys keep the softmax
            // groups supplied (waiting for either in turn holds up the other).
            auto ready = [&](uint32_t at, uint32_t parity) { return __all_sync(0xFFFFFFFFu, test_at(at, parity)) != 0; };
            auto tiles_of = [&](const Walk& x, int rest) {
                return __shfl_sync(0xFFFFFFFFu, rest < x.tiles - x.t ? rest : x.tiles - x.t, 0);
            };
            Walk wv = w;                         // the tile whose O is added next, on its own way through the parts
            int vleft = left;
            uint32_t i = 0, n = 0, piece = 0, vpart = 0;
            int nt = left > 0 ? tiles_of(w, left) : 0, t = 0, vnt = nt, vt = 0;
            while (vnt > 0) {
                bool moved = false;
                const uint32_t vf = 2 * n + 1;
                if (n < i && ready(bar(C::B_PFULL, n & 1), (n >> 1) & 1) && ready(bar(C::B_FULL, vf % NS), (vf / NS) & 1) &&
                    (vt > 0 || ready(bar(C::B_OFREE, vpart & 1), ((vpart >> 1) & 1) ^ 1))) {
                    tc_fence_after();
                    pv(n, vpart, vt < 2, vt == vnt - 1);
                    progress[0] = ++n;
                    if (++vt == vnt) {
                        vleft -= vnt;
                        ++vpart;
                        vt = 0;
                        walk.advance(wv, vnt, vleft > 0);
                        vnt = vleft > 0 ? tiles_of(wv, vleft) : 0;
                    }
                    moved = true;
                }
                // S of tile i - SB has been read: its O, or a later one, has been added
                const uint32_t kf = 2 * i;
                if (nt > 0 && i < n + C::LOOK && (t > 0 || ready(bar(C::B_QFULL, piece & 1), (piece >> 1) & 1)) &&
                    ready(bar(C::B_FULL, kf % NS), (kf / NS) & 1)) {
                    tc_fence_after();
                    qk(i, piece & 1, t == nt - 1);
                    ++i;
                    if (++t == nt) {
                        left -= nt;
                        ++piece;
                        t = 0;
                        walk.advance(w, nt, left > 0);
                        nt = left > 0 ? tiles_of(w, left) : 0;
                    }
                    moved = true;
                }
                if (!moved && __any_sync(0xFFFFFFFFu, stopped(stop))) break;
            }
        } else if (warp == SW + 7) {
            // -------------------------------------------------------- watchdog: stops the block when nothing has moved for the bound
            uint32_t seen = 0;
            uint64_t since = global_timer_ns();
            const bool nap = a.wait_ns >= 40000ull;  // (asleep for some 20 us, whatever less is asked for)
            while (!(nap ? try_at_for(bar(C::B_DONE), 0, 20000) : test_at(bar(C::B_DONE), 0)) && !stopped(stop)) {
                const uint32_t now_at = progress[0] + progress[1];
                const uint64_t now = global_timer_ns();
                if (now_at != seen) {
                    seen = now_at;
                    since = now;
                } else if (now - since >= a.wait_ns) {
                    stop_all(stop);
                    break;
                }
            }
        } else {
            // -------------------------------------------------------- scales: a lane takes four rows. Scales are under way A tiles
            // ahead and page ids another A, both into shared memory (a register handed from one to the next waits for its load:
            // a tile then takes an access): a tile takes 750 (head_dim 64) to 2,500 clocks (64 tree rows) and an
            // access to loaded HBM some 5,500.
            constexpr int A = C::SA;
            const uint32_t ids = base + C::OFF_SID + lane * 4, sc0 = base + C::OFF_SC + lane * 4;
            bool ok = true;
            uint32_t i = 0;
            while (left > 0 && ok) {
                const int nt = left < w.tiles - w.t ? left : w.tiles - w.t;
                const int first = w.t * TILE + lane * 4, end = min(walk.lane(w.b).len, (w.t + nt) * TILE), hp = w.h * P;
                const int32_t* table = a.table + (int64_t)w.b * a.width;
                auto look = [&](int d) {
                    const int at = first + d * TILE;
                    if (d < nt && at < end) cp_async_4(ids + (d % (2 * A)) * 128, table + (at >> a.page_shift));
                };
                auto load = [&](int d) {                     // its id has arrived
                    if (d >= nt) return true;
                    const uint32_t e = i + d, sc = e % NSC;
                    if (!warp_wait_at(bar(C::B_SCEMPTY, sc), ((e / NSC) & 1) ^ 1, stop)) return false;
                    const int at = first + d * TILE;
                    const uint32_t dst = sc0 + sc * C::SC_BYTES;
                    if (at < end) {
                        const int row = checked(read_at(ids + (d % (2 * A)) * 128), false) * H * P + hp + (at & (P - 1));
                        cp_async_4(dst, a.c.k_scales + row);
                        cp_async_4(dst + TILE, a.c.v_scales + row);
                    } else {
                        write_at(dst, 0x01010101u * (ZERO_BYTE - 1));              // any scale but that of zeros
                        write_at(dst + TILE, 0x01010101u * (ZERO_BYTE - 1));
                    }
                    return true;
                };
                const int ahead = nt < A ? nt : A;
#pragma unroll 1
                for (int d = 0; d < ahead; ++d) look(d);
                cp_async_commit();
                cp_async_wait<0>();
                // at d: scales of tile d + A and ids of tile d + 2 A are sent for, tile d is handed over; few tiles wait for all
#pragma unroll 1
                for (int d = -ahead; d < nt; ++d) {
                    if (d >= 0) {
                        if (nt < A) cp_async_wait<0>(); else cp_async_wait<A - 1>();
                    }
                    if (!load(d + ahead)) { ok = false; break; }
                    look(d + 2 * A);
                    cp_async_commit();
                    if (d < 0) continue;
                    const uint32_t sc = (i + d) % NSC;
                    const uint32_t mine = read_at(sc0 + sc * C::SC_BYTES + TILE);
                    const uint32_t hi = __vmaxu4(mine, mine >> 16);
                    const uint32_t lo = __vminu4(mine, __byte_perm(mine, 0, 0x1032));
                    const uint32_t most = __reduce_max_sync(0xFFFFFFFFu, max(hi & 255u, (hi >> 8) & 255u));
                    uint32_t least = __reduce_min_sync(0xFFFFFFFFu, min(lo & 255u, (lo >> 8) & 255u));
                    if (__any_sync(0xFFFFFFFFu, __vcmpeq4(mine, 0x01010101u * ZERO_BYTE) != 0u)) least = (uint32_t)MAY_BE_ZERO;
                    if (lane == 0) {
                        write_at(base + C::OFF_SC + sc * C::SC_BYTES + 2 * TILE, most);
                        write_at(base + C::OFF_SC + sc * C::SC_BYTES + 2 * TILE + 4, least);
                    }
                    __syncwarp();
                    if (lane == 0) arrive_at(bar(C::B_SCFULL, sc));
                }
                i += nt;
                left -= nt;
                walk.advance(w, nt, left > 0);
            }
            cp_async_wait<0>();
        }
    }
    tc_fence_before();
    __syncthreads();
    if (*abort_flag) {                               // final after the barrier: nothing new is issued past it
        if (warp == SW + 4 && lane == 0) drain_stage_fills(bar_ptr(C::B_FULL), NS, issued);
        if (warp == SW + 5 && elect_one()) tc_drain(bar_ptr(C::B_DRAIN));
        tc_fence_before();
        __syncthreads();
    }
    if (warp == SW + 5) {
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

template <int D, int R>
__global__ void __launch_bounds__(JOIN_WARPS * 32) tree_attention_join(const AttnArgs a, int ctas) {
    pdl_trigger();
    pdl_wait();
    const JoinUnit u = reinterpret_cast<const JoinUnit*>(a.ws)[blockIdx.x + 1];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int r = blockIdx.y * JOIN_WARPS + warp;
    if (!u.join || r >= u.rows) return;
    const float* parts = reinterpret_cast<const float*>(a.ws + parts_offset(ctas));
    auto part = [&](int k) { return parts + (size_t)(2 * k + (k == u.first ? u.second : 0)) * part_floats(R, D); };
    constexpr int V = D / 32, AT_ONCE = D == 256 ? 4 : 8;      // columns a lane; parts whose loads are under way together
    float acc[V] = {}, L = 0.0f, M = -INFINITY;
#pragma unroll 1
    for (int k0 = u.first; k0 <= u.last; k0 += AT_ONCE) {
        float m[AT_ONCE], l[AT_ONCE], x[AT_ONCE][V], Mn = M;
#pragma unroll
        for (int k = 0; k < AT_ONCE; ++k) {
            const float* p = part(k0 + k <= u.last ? k0 + k : u.last);
            m[k] = p[R * D + r];
            l[k] = p[R * D + R + r];
#pragma unroll
            for (int e = 0; e < V; ++e) x[k][e] = p[r * D + e * 32 + lane];
        }
#pragma unroll
        for (int k = 0; k < AT_ONCE; ++k) {
            if (k0 + k > u.last) { m[k] = -INFINITY; l[k] = 0.0f; }
            Mn = fmaxf(Mn, m[k]);
        }
        const float f0 = M == -INFINITY ? 0.0f : ex2(0.5f * (M - Mn));
        L = L * f0 * f0;
#pragma unroll
        for (int e = 0; e < V; ++e) acc[e] *= f0 * f0;
#pragma unroll
        for (int k = 0; k < AT_ONCE; ++k) {
            const float f = m[k] == -INFINITY ? 0.0f : ex2(0.5f * (m[k] - Mn));
            L += f * l[k] * f;                       // NaN stays, also with a weight of zero
#pragma unroll
            for (int e = 0; e < V; ++e)
                if (k0 + k <= u.last) acc[e] += f * f * x[k][e];
        }
        M = Mn;
    }
    const float inv = L == 0.0f ? 0.0f : exp2_int(-L_EXP) / L;
    const int tr = u.row0 + r, node = tr / a.group;
    const int64_t at = (int64_t)(u.node0 + node) * a.n_q_heads + u.head * a.group + tr - node * a.group;
#pragma unroll
    for (int e = 0; e < V; ++e) a.out[at * D + e * 32 + lane] = __float2bfloat16_rn(acc[e] * inv);
    if (a.lse && lane == 0) a.lse[at] = L == 0.0f ? -INFINITY : (M - (P_EXP - L_EXP) + log2f(L)) * 0.69314718055994531f;
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

constexpr int max_unit(int D) { return D == 256 ? 32 : 64; }         // R: what shared memory holds

template <int D, int R>
cudaError_t launch(const AttnArgs& a, cudaStream_t s) {
    using C = Cfg<D, R>;
    AttnMaps maps;
    cudaError_t e = codes_map(&maps.k, a.c.k_codes, a.c);
    if (e == cudaSuccess) e = codes_map(&maps.v, a.c.v_codes, a.c);
    if (e != cudaSuccess) return e;
    static bool attr_set[64] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev >= 0 && dev < 64 && !attr_set[dev]) {
        e = cudaFuncSetAttribute(tree_attention<D, R>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
        if (e != cudaSuccess) return e;
        attr_set[dev] = true;
    }
    const int ctas = moe_sm_count();
    moe_prof_begin(MK_ATTENTION, s);
    e = moe_launch(tree_attention<D, R>, dim3((unsigned)ctas), dim3(C::THREADS), C::SMEM, s, maps, a);
    moe_prof_end(MK_ATTENTION, s);
    moe_count_launches(1);
    if (e != cudaSuccess || ctas < 2 || a.whole) return e;
    moe_prof_begin(MK_ATTENTION_JOIN, s);
    e = moe_launch(tree_attention_join<D, R>, dim3((unsigned)(ctas - 1), R / JOIN_WARPS), dim3(JOIN_WARPS * 32), 0, s, a, ctas);
    moe_prof_end(MK_ATTENTION_JOIN, s);
    moe_count_launches(1);
    return e;
}

// The tile of tree rows: the smallest that takes a lane's rows of one kv head at once, else the largest. Measured, us,
// taken / the other: 4 rows, 64 lanes of up to 8,192 rows, 16 / 32: 94 / 104. 28 rows, two lanes of 131,072, 32 / 64:
// 101 / 124. Up to 128 rows, 32 lanes of up to 8,001, 64 / 32: 148 / 171. Up to 64 rows at head_dim 64, 32 lanes of up
// to 8,000, 64 / 32: 182 / 189 (nine lanes of up to 2,047, their trees uneven: 38 / 33; a second rule, on the rows that the page
// table can hold, could tell these apart). Two groups on one tile for
// twice the rows read the cache once where two units read it twice, but above 64 rows the softmax
// bounds, not the reading: 3 % faster with 128 rows in every lane, 8 % slower with uneven trees (with weights in two parts).
template <int D>
cudaError_t launch_rows(const AttnArgs& a, cudaStream_t s) {
    const int64_t rows = (int64_t)(a.max_nodes < a.n_nodes ? a.max_nodes : a.n_nodes) * a.group;
    if (rows <= 16) return launch<D, 16>(a, s);
    if (rows <= 32 || D == 256) return launch<D, 32>(a, s);
    return launch<D, max_unit(D)>(a, s);
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
    a.whole = (int64_t)table_width * cache->page_size <= WHOLE_TILES * TILE;
    a.scale_log2 = scale * 1.4426950408889634f;
    a.out = static_cast<__nv_bfloat16*>(out);
    a.lse = lse;
    a.ws = static_cast<uint8_t*>(workspace);
    a.err = err;
    a.wait_ns = moe_wait_limit_ns();
    const cudaError_t e = cache->head_dim == 64    ? launch_rows<64>(a, s)
                          : cache->head_dim == 128 ? launch_rows<128>(a, s)
                                                   : launch_rows<256>(a, s);
    return e == cudaSuccess ? MOE_OK : MOE_ECUDA;
}
