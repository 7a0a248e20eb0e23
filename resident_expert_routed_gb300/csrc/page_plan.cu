// The plan of a batch of new tokens: pages for the lanes, positions and cache slots for the tokens.
//
// With new_b tokens for lane b, which has kept rows_b rows in held_b pages:
//   need_b   = max(0, ceil((rows_b + new_b) / page) - held_b)
//   served_b = need_0 + ... + need_b <= pages on the stack
//   position = rows_b + i,   slot = table[b, position / page] * page + position % page     (token i of the lane)
// Two prefix sums over the lanes (tokens and returned pages, then needs), then
// every token, new page and returned page on its own: a binary search over the
// sums finds its lane.
//
// Nothing here is large (12 bytes a token), so the launch and the chain of
// dependent steps bound it. One launch: a cluster of up to eight CTAs, each of which
// does the sums for itself and takes its share of the tokens; the cluster's first
// barrier keeps the state's old values until all have read them, the second (0.1 to
// 0.5 us) tells all whether a lane has met a page id outside the pool. One after the
// other in a graph: two lanes of one token 3.2 us, 256 lanes of 9 tokens 6.8, 48 of
// 1,000 9.1.
#include <climits>

#include "common.cuh"

namespace {

constexpr int PLAN_THREADS = 1024;
constexpr int PLAN_MAX_LANES = 4096;
constexpr int PLAN_MAX_CTAS = 8;            // 1 / 4 / 8, before the second barrier: 48 lanes of 1,000 tokens 32.3 / 12.4 / 8.6 us, 4,096 lanes of 4 28.3 / 17.7 / 15.9

struct PlanArgs {
    const int32_t* n_new;
    int32_t* rows;
    int32_t* held;
    int32_t* table;
    int width, lanes, n_pages, page_shift, max_tokens;
    int32_t* free_pages;
    int32_t* n_free;
    int32_t* kv_len;
    int32_t* cu;
    int32_t* positions;
    int64_t* slots;
    uint32_t* err;
};

typedef unsigned long long u64;

MOE_DEV void cluster_sync() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Sets a flag in shared memory of a block of the cluster.
MOE_DEV void tell_block(int* flag, int rank) {
    asm volatile(
        "{\n\t.reg .u32 at;\n\t"
        "mapa.shared::cluster.u32 at, %0, %1;\n\t"
        "st.shared::cluster.u32 [at], 1;\n\t}" ::"r"(smem_u32(flag)), "r"(rank) : "memory");
}

// The first index in [0, n) with upto[index] > x; n where there is none.
MOE_DEV int lane_of(const int* upto, int n, int x) {
    int lo = 0, hi = n;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (upto[mid] <= x) lo = mid + 1; else hi = mid;
    }
    return lo;
}

__global__ void __launch_bounds__(PLAN_THREADS) page_plan(const PlanArgs a) {
    extern __shared__ int plan_smem[];
    const int B = a.lanes, tid = threadIdx.x, nt = blockDim.x;
    const int rank = blockIdx.x, ranks = gridDim.x;
    int* tok = plan_smem;                   // [B] tokens of the lanes up to this one, at most max_tokens
    int* got = tok + B;                     // [B] new pages
    int* back = got + B;                    // [B] returned pages
    int* rows = back + B;                   // [B] the lane's rows; ~rows where it is refused
    int* held = rows + B;                   // [B]
    __shared__ u64 scratch[64];
    __shared__ int spoilt;                  // some token's page is none of the pool's
    if (tid == 0) spoilt = 0;
    pdl_trigger();
    pdl_wait();
    int n_free = a.n_free[0];
    uint32_t bad = 0;
    if (n_free < 0 || n_free > a.n_pages) {
        bad |= MOE_DEV_BAD_PAGE;
        n_free = n_free < 0 ? 0 : a.n_pages;
    }
    // ---- tokens and returned pages
    u64 tok_all = 0, back_all = 0;
    for (int b0 = 0; b0 < B; b0 += nt) {
        const int b = b0 + tid;
        int n = 0, r = 0, h = 0;
        if (b < B) { n = a.n_new[b]; r = a.rows[b]; h = a.held[b]; }
        bool fine = r >= 0 && h >= 0 && h <= a.width;
        if (!fine) { bad |= MOE_DEV_BAD_PAGE; h = h < 0 ? 0 : (h > a.width ? a.width : h); }
        const u64 own = n > 0 ? n : 0, gone = n < 0 ? h : 0;
        u64 x = own, y = gone, tx, ty;
        scan2(x, y, scratch, &tx, &ty);
        x += tok_all;
        y += back_all;
        tok_all += tx;
        back_all += ty;
        if (b < B) {
            tok[b] = (int)min(x, (u64)a.max_tokens);
            back[b] = (int)min(y, (u64)INT_MAX);
            held[b] = h;
            if (n > 0) fine &= x <= (u64)a.max_tokens;                          // (a lane that waits fits any batch)
            const int64_t pages = ((int64_t)(fine ? r : 0) + (int64_t)own + (1 << a.page_shift) - 1) >> a.page_shift;
            if (n > 0) fine &= pages <= a.width;
            rows[b] = fine ? r : ~(r < 0 ? 0 : r);
            got[b] = fine && n > 0 && pages > h ? (int)(pages - h) : 0;          // the need, for now
        }
    }
    if ((u64)n_free + back_all > (u64)a.n_pages) bad |= MOE_DEV_BAD_PAGE;        // pages that come back twice: the last are dropped
    const int there = (int)min((u64)a.n_pages, (u64)n_free + back_all);
    // ---- needs: a lane is served where those of all lanes up to it are there
    u64 need_all = 0, given = 0;
    for (int b0 = 0; b0 < B; b0 += nt) {
        const int b = b0 + tid;
        const int need = b < B ? got[b] : 0;
        u64 x = need, y = 0, tx, ty;
        scan2(x, y, scratch, &tx, &ty);
        x += need_all;
        need_all += tx;
        bool served = true;
        if (b < B && need > 0 && x > (u64)there) served = false;
        u64 g = served ? need : 0, z = 0, tg, tz;
        scan2(g, z, scratch, &tg, &tz);
        g += given;
        given += tg;
        if (b < B) {
            if (!served) rows[b] = ~rows[b];
            if (rows[b] < 0 && a.n_new[b] > 0) bad |= MOE_DEV_NO_PAGES;
            got[b] = (int)g;                                                    // pages given to the lanes up to this one
            if (rank == 0) a.kv_len[b] = a.n_new[b] < 0 || rows[b] < 0 ? 0 : rows[b] + a.n_new[b];
        }
    }
    if (bad && rank == 0) record_error(a.err, bad);
    __syncthreads();
    // ---- returned pages go to the top of the stack, in the lanes' order
    const int step = ranks * nt, first = rank * nt + tid;
    for (int i = first; i < there - n_free; i += step) {
        const int b = lane_of(back, B, i);
        const int at = i - (b ? back[b - 1] : 0);
        a.free_pages[n_free + i] = a.table[(int64_t)b * a.width + at];
    }
    if (ranks > 1) cluster_sync(); else __syncthreads();
    // ---- from here on the state changes, and nobody reads its old values
    if (rank == 0) {
        for (int b = tid; b < B; b += nt) {
            const int n = a.n_new[b], h = held[b];
            a.cu[b + 1] = tok[b];
            if (n < 0) {
                a.rows[b] = 0;
                a.held[b] = 0;
            } else if (got[b] > (b ? got[b - 1] : 0)) {
                a.held[b] = h + got[b] - (b ? got[b - 1] : 0);
            }
        }
        if (tid == 0) {
            a.cu[0] = 0;
            a.n_free[0] = there - (int)given;
        }
    }
    for (int i = first; i < (int)given; i += step) {
        const int b = lane_of(got, B, i);
        const int at = held[b] + i - (b ? got[b - 1] : 0);
        a.table[(int64_t)b * a.width + at] = a.free_pages[there - 1 - i];
    }
    const int returned = back[B - 1];
    for (int i = first; i < returned; i += step) {
        const int b = lane_of(back, B, i);
        a.table[(int64_t)b * a.width + i - (b ? back[b - 1] : 0)] = -1;
    }
    const int page = 1 << a.page_shift, tokens = tok[B - 1];
    bool lost = false;
    for (int t = first; t < a.max_tokens; t += step) {
        int64_t slot = -1;
        int pos = 0;
        if (t < tokens) {
            const int b = lane_of(tok, B, t), r = rows[b];
            pos = (r < 0 ? ~r : r) + t - (b ? tok[b - 1] : 0);
            if (r >= 0) {
                const int p = pos >> a.page_shift, h = held[b];
                const int id = p < h ? a.table[(int64_t)b * a.width + p] : a.free_pages[there - 1 - ((b ? got[b - 1] : 0) + p - h)];
                if (id >= 0 && id < a.n_pages) {
                    slot = (int64_t)id * page + (pos & (page - 1));
                } else {
                    lost = true;
                    a.kv_len[b] = 0;
                }
            }
        }
        a.positions[t] = pos;
        a.slots[t] = slot;
    }
    // A lane with an id outside the pool among its tokens' pages is refused as a whole: whichever block met it, those of its
    // tokens that have got slots on other pages lose them.
    if (lost) {
        record_error(a.err, MOE_DEV_BAD_PAGE);
        for (int r = 0; r < ranks; ++r) tell_block(&spoilt, r);
    }
    if (ranks > 1) cluster_sync(); else __syncthreads();
    if (spoilt)
        for (int t = first; t < tokens; t += step)
            if (__ldcg(a.kv_len + lane_of(tok, B, t)) == 0) a.slots[t] = -1;
}

}  // namespace

moe_status moe_page_plan(const int32_t* n_new, int32_t* rows, int32_t* held, int32_t* page_table, int table_width, int lanes,
                         int32_t* free_pages, int n_pages, int32_t* n_free, int page_size, int32_t* kv_len, int32_t* cu_tokens,
                         int32_t* positions, int64_t* slots, int max_tokens, void* stream) {
    MOE_RANGE("moe_page_plan");
    if (!n_new || !rows || !held || !page_table || !free_pages || !n_free || !kv_len || !cu_tokens) return MOE_EINVAL;
    if (lanes < 1 || table_width < 1 || n_pages < 1 || max_tokens < 0 || page_size < 1 || (page_size & (page_size - 1))) return MOE_EINVAL;
    if (max_tokens > 0 && (!positions || !slots)) return MOE_EINVAL;
    if (lanes > PLAN_MAX_LANES || page_size < 16 || page_size > 1024 || max_tokens > (1 << 24) || table_width > (1 << 20)) return MOE_EUNSUPPORTED;
    if ((int64_t)n_pages * page_size >= ((int64_t)1 << 31)) return MOE_EUNSUPPORTED;
    uint32_t* err = moe_err_word();
    if (!err) return MOE_ECUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const PlanArgs a{n_new, rows, held, page_table, table_width, lanes, n_pages, log2_of(page_size), max_tokens, free_pages, n_free,
                     kv_len, cu_tokens, positions, slots, err};
    const size_t smem = (size_t)5 * lanes * sizeof(int);
    cudaError_t e = cudaSuccess;
    // (48 KB need no opt-in, but the block's static shared memory is among them)
    if (smem > 40 * 1024) e = cudaFuncSetAttribute(page_plan, cudaFuncAttributeMaxDynamicSharedMemorySize, 5 * PLAN_MAX_LANES * (int)sizeof(int));
    if (e != cudaSuccess) return MOE_ECUDA;
    // threads for the lanes and the tokens; more CTAs where a thread would take more than two tokens
    int threads = (lanes > max_tokens ? lanes : max_tokens) + 31;
    threads = threads > PLAN_THREADS ? PLAN_THREADS : threads / 32 * 32;
    int ctas = (max_tokens + 2 * PLAN_THREADS - 1) / (2 * PLAN_THREADS);
    ctas = ctas < 1 ? 1 : ctas > PLAN_MAX_CTAS ? PLAN_MAX_CTAS : ctas;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)ctas;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    moe_prof_begin(MK_PAGE_PLAN, s);
    e = cudaLaunchKernelEx(&cfg, page_plan, a);
    moe_prof_end(MK_PAGE_PLAN, s);
    moe_count_launches(1);
    return e == cudaSuccess ? MOE_OK : MOE_ECUDA;
}
