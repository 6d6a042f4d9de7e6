// paged_chunk.cu -- attention of chunks of new tokens over a paged cache, on
// the tcgen05 tensor cores.
//
// The mathematics is paged_attn.cu's (one pass over the keys, running maximum
// and sum per row, both in fp32).  With many rows per key the bound is no longer
// memory but the tensor cores (4 d operations per row and key) and, as near, the
// exponential unit: a 128 x 128 tile of scores takes 1024 tensor cycles at d =
// 128 (scores and values together) and as many cycles of 2^x at 16 a cycle.  So
// both have to run all the time:
// - an item is 256 rows (tokens x query heads of one key head) in two tiles of
//   128.  A tile's scores, 128 fp32 TMEM columns, become weights in place (64
//   columns of 16-bit pairs) that the second product reads from TMEM; while one
//   tile's warps form weights, the tensor cores work on the other tile.
// - one warp issues every product, one loads pages by TMA into a ring (key and
//   value tiles of 128 keys in turn), eight own a row per thread.
// - the sums stay in TMEM.  They are rescaled only when a row's maximum grows by
//   more than 2^8 over the one in use (weights up to 2^8 lose nothing: 16-bit
//   rounding is relative and the sums are fp32), so after the first keys hardly
//   ever.
// - the rows of masked keys behind the sequence's end are zeroed in the last
//   value tile: a page holds anything there, and 0 x NaN is NaN.
//
// Work: a plan kernel (one block; the others meanwhile write the new tokens to
// their pages) cuts the items' keys into pieces of a common length, chosen among
// sixteen by the time it models for all SMs, longest items first; CTAs, one per
// SM, claim pieces from a counter.  Pieces of a split item are joined by
// paged_join_kernel in a fixed order.
#include "kda_internal.cuh"
#include "paged_params.cuh"

namespace kda {

constexpr int CK_M = 128, CK_KT = 128, CK_ROWS = 2 * CK_M;  // rows of a tile, keys of a tile, rows of an item
constexpr int CK_THREADS = 320, CK_MMA = 8, CK_LOAD = 9;    // warps 0-7: rows; 8: products; 9: loads

// One piece of work: keys [kv0, kv1) in tiles of rows [t 256, t 256 + 256) of
// (n, h); part_row: where its partial sums go, or -1 when it is the whole item.
struct ChunkPiece {
    int n, h, t, kv0, kv1;
    int part_row;
    int pad[2];
};
struct ChunkPlanHead {
    int pieces, ticket, entries, pad;
};
struct ChunkParams {
    PagedParams p;
    ChunkPlanHead *head;
    ChunkPiece *pieces;
    int *base;             // [N] the plan's scratch
    int max_pieces, max_entries, max_rows, sms;
};

template <int D>
struct CkShape {
    static constexpr int TILE = CK_KT * D * 2;                    // a key or value tile
    static constexpr int STAGES = D == 128 ? 5 : 8;
    static constexpr int OFF_RING = 2 * CK_M * D * 2;             // behind the two query tiles
    static constexpr int OFF_BAR = OFF_RING + STAGES * TILE;
    static constexpr int B_Q = 0, B_S = 1, B_P = 3, B_TAIL = 5, B_DRAIN = 6, B_FULL = 7, B_EMPTY = B_FULL + STAGES, NBAR = B_EMPTY + STAGES;
    static constexpr int SMEM = OFF_BAR + NBAR * 8 + 1024;        // and room to align the base
    static constexpr uint32_t TM_S = 0, TM_O = 256;               // columns: S0, S1, O0, O1
};

// ------------------------------------------------------------------- plan ----
__device__ __forceinline__ int ck_tiles(const PagedSeq &s, int G) { return (int)(((long long)s.nq * G + CK_ROWS - 1) / CK_ROWS); }
__device__ __forceinline__ int ck_keys(const PagedSeq &s, int G, int t) {  // key tiles of row tile t
    return max(1, (paged_kv_end(s, G, (t + 1) * CK_ROWS - 1) + CK_KT - 1) / CK_KT);
}
// rows that row tile t holds
__device__ __forceinline__ int ck_rows(const PagedSeq &s, int G, int t) { return min(CK_ROWS, s.nq * G - t * CK_ROWS); }

constexpr int CK_CAND = 16;
__device__ __constant__ int ck_div[CK_CAND] = {1, 2, 3, 4, 5, 6, 7, 8, 10, 12, 16, 24, 32, 64, 128, 256};

__device__ void ck_plan(const ChunkParams &c, int d) {
    __shared__ unsigned long long s_w;
    __shared__ unsigned long long s_pieces[CK_CAND], s_rows[CK_CAND];
    __shared__ int s_max, s_step, s_entries, s_part, s_sum[33];
    const PagedParams &p = c.p;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, warps = blockDim.x >> 5, G = p.G;
    if (tid == 0) { s_w = 0; s_max = 1; s_entries = 0; s_part = 0; }
    if (tid < CK_CAND) s_pieces[tid] = s_rows[tid] = 0;
    __syncthreads();
    // a warp a sequence, a lane a row tile
    unsigned long long w = 0;
    int mx = 1;
    for (int n = warp; n < p.N; n += warps) {
        const PagedSeq s = paged_seq(p, n, lane == 0);
        for (int t = lane; t < ck_tiles(s, G); t += 32) {
            const int k = ck_keys(s, G, t);
            w += k;
            mx = max(mx, k);
        }
    }
    atomicAdd(&s_w, w);
    atomicMax(&s_max, mx);
    __syncthreads();
    int pieces[CK_CAND] = {};
    unsigned long long rows[CK_CAND] = {};
    for (int n = warp; n < p.N; n += warps) {
        const PagedSeq s = paged_seq(p, n, false);
        for (int t = lane; t < ck_tiles(s, G); t += 32) {
            const int k = ck_keys(s, G, t), r = ck_rows(s, G, t);
#pragma unroll
            for (int j = 0; j < CK_CAND; ++j) {
                const int step = (s_max + ck_div[j] - 1) / ck_div[j], ns = (k + step - 1) / step;
                pieces[j] += ns;
                if (ns > 1) rows[j] += (unsigned long long)ns * r;
            }
        }
    }
#pragma unroll
    for (int j = 0; j < CK_CAND; ++j) {
        atomicAdd(&s_pieces[j], (unsigned long long)pieces[j]);
        atomicAdd(&s_rows[j], rows[j]);
    }
    __syncthreads();
    if (warp == 0) {
        // modelled time in key tiles: the waves of pieces, each with a fixed cost of about
        // three tiles, no less than the longest piece; joins at the memory's rate
        float cost = 3.0e38f;
        int step = s_max;
        if (lane < CK_CAND) {
            step = (s_max + ck_div[lane] - 1) / ck_div[lane];
            const float P = (float)s_pieces[lane] * p.Hkv, W = (float)s_w * p.Hkv, R = (float)s_rows[lane] * p.Hkv;
            const float waves = ceilf(P / c.sms);
            if (lane == 0 || (P <= c.max_pieces && R <= c.max_rows))
                cost = fmaxf(waves * (W / P + 3.f), step + 3.f) + (R > 0.f ? 3.f + R * d * 8.f * 1.2e-7f : 0.f);
        }
        float best = cost;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) best = fminf(best, __shfl_xor_sync(0xffffffffu, best, o));
        const int who = __ffs(__ballot_sync(0xffffffffu, cost == best)) - 1;
        step = __shfl_sync(0xffffffffu, step, who);
        if (lane == 0) s_step = step;
    }
    __syncthreads();
    const int step = s_step;
    // pieces of each sequence and key head, then where each sequence's begin
    for (int n = warp; n < p.N; n += warps) {
        const PagedSeq s = paged_seq(p, n, false);
        int k = 0;
        for (int t = lane; t < ck_tiles(s, G); t += 32) k += (ck_keys(s, G, t) + step - 1) / step;
        k = __reduce_add_sync(0xffffffffu, k);
        if (lane == 0) c.base[n] = k * p.Hkv;
    }
    __syncthreads();
    const int per = (p.N + blockDim.x - 1) / blockDim.x;
    int mine = 0;
    for (int n = tid * per; n < min(p.N, (tid + 1) * per); ++n) mine += c.base[n];
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += up;
    }
    if (lane == 31) s_sum[warp] = incl;
    __syncthreads();
    int at = incl - mine, total = 0;
    for (int k = 0; k < warps; ++k) {
        if (k < warp) at += s_sum[k];
        total += s_sum[k];
    }
    for (int n = tid * per; n < min(p.N, (tid + 1) * per); ++n) {
        const int k = c.base[n];
        c.base[n] = at;
        at += k;
    }
    __syncthreads();
    for (int n = warp; n < p.N; n += warps) {
        const PagedSeq s = paged_seq(p, n, false);
        const int tiles = ck_tiles(s, G);
        const int first = c.base[n], head_pieces = (n + 1 < p.N ? c.base[n + 1] : total) - first;
        const int per_head = head_pieces / p.Hkv;
        int before = 0;
        for (int t0 = 0; t0 < tiles; t0 += 32) {
            const int t = tiles - 1 - (t0 + lane);  // the longest first
            const int k = t >= 0 ? ck_keys(s, G, t) : 0, ns = t >= 0 ? (k + step - 1) / step : 0;
            int inc = ns;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int up = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o) inc += up;
            }
            if (t >= 0) {
                const int r = ck_rows(s, G, t);
                for (int h = 0; h < p.Hkv; ++h) {
                    const long long i = (long long)first + (long long)h * per_head + before + inc - ns;
                    int part = -1;
                    if (ns > 1) {
                        part = atomicAdd(&s_part, ns * r);
                        const int e = atomicAdd(&s_entries, 1);
                        if (e < c.max_entries && part + ns * r <= c.max_rows)
                            p.entries[e] = {n, h, t, part, part + r, ns - 1, r};
                        else report(p.st, DEV_BAD_ARG);  // only where sequences overlap
                    }
                    for (int j = 0; j < ns; ++j) {
                        if (i + j >= c.max_pieces) { report(p.st, DEV_BAD_ARG); break; }
                        const int row = part < 0 ? -1 : part + j * r;
                        // a piece without room for its sums is left empty
                        const bool room = part < 0 || part + ns * r <= c.max_rows;
                        c.pieces[i + j] = {n, h, t, j * step, room ? min(k, (j + 1) * step) : j * step, row, {0, 0}};
                    }
                }
            }
            before += __shfl_sync(0xffffffffu, inc, 31);
        }
    }
    __syncthreads();
    if (tid == 0) {
        c.head->pieces = min(total, c.max_pieces);
        c.head->ticket = 0;
        c.head->entries = min(s_entries, c.max_entries);
    }
}

// The new tokens' keys and values to their pages: 16 bytes a thread.
template <int D>
__device__ void ck_append(const ChunkParams &c, long long first, long long step) {
    const PagedParams &p = c.p;
    constexpr int CH = D / 8;
    const int per_tok = p.Hkv * CH;
    for (long long i = first; i < (long long)p.total_q * per_tok; i += step) {
        const int tok = (int)(i / per_tok), in_tok = (int)(i % per_tok), h = in_tok / CH, ch = in_tok % CH;
        int lo = 0, hi = p.N;  // the last sequence that begins at or before the token
        while (hi - lo > 1) {
            const int mid = (lo + hi) / 2;
            if (p.cu[mid] <= tok) lo = mid; else hi = mid;
        }
        const PagedSeq s = paged_seq(p, lo, false);
        const int at = tok - s.q0, pos = s.len - s.nq + at;
        if (at < 0 || at >= s.nq || pos < 0) continue;
        const int page = p.table[(long long)s.row * p.P + pos / p.page_size], in = pos % p.page_size;
        if (page < 0 || page >= p.num_pages) { report(p.st, DEV_BAD_ARG); continue; }
        const uint4 kx = *reinterpret_cast<const uint4 *>(p.k_new + tok * p.kn_ts + h * D + ch * 8);
        const uint4 vx = *reinterpret_cast<const uint4 *>(p.v_new + tok * p.vn_ts + h * D + ch * 8);
        *reinterpret_cast<uint4 *>(p.kp + page * p.k_ps + in * p.k_ts + h * p.k_hs + ch * 8) = kx;
        *reinterpret_cast<uint4 *>(p.vp + page * p.v_ps + in * p.v_ts + h * p.v_hs + ch * 8) = vx;
    }
}

template <int D>
__global__ void __launch_bounds__(512) paged_plan_kernel(const ChunkParams c) {
    if (blockIdx.x == 0) ck_plan(c, D);
    else ck_append<D>(c, (long long)(blockIdx.x - 1) * blockDim.x + threadIdx.x, (long long)(gridDim.x - 1) * blockDim.x);
}

// -------------------------------------------------------------- tensor memory ----
__device__ __forceinline__ void tm_ld32(uint32_t a, uint32_t *r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(a));
}
__device__ __forceinline__ void tm_st32(uint32_t a, const uint32_t *r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(a),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
        "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
        "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}
__device__ __forceinline__ void tm_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// D[tmem] (+)= A[tmem] B[smem]: A's rows are lanes, two 16-bit values a column.
__device__ __forceinline__ void umma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}

// ------------------------------------------------------------------ kernel ----
template <int D, bool BF>
__global__ void __launch_bounds__(CK_THREADS, 1)
paged_chunk_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v, const ChunkParams c) {
    using S = CkShape<D>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint32_t s_tmem;
    __shared__ int s_piece;
    __shared__ volatile int s_abort;
    const PagedParams &p = c.p;
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    uint8_t *sm = smem_raw + (base - smem_u32(smem_raw));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, G = p.G;
    const uint64_t polls = p.st.wait_polls;
    auto bar = [&](int i) { return base + S::OFF_BAR + i * 8; };

    if (tid == 0) {
        for (int i = 0; i < S::NBAR; ++i) mbar_init(bar(i), i == S::B_Q ? 8u : (i >= S::B_P && i < S::B_P + 2) ? 4u : 1u);
        s_abort = 0;
        fence_mbar_init();
    }
    if (warp == CK_MMA) {
        tmem_alloc(smem_u32(&s_tmem), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    const int pieces = c.head->pieces;

    auto wait1 = [&](int i, uint32_t par) -> bool {
        if (mbar_wait(bar(i), par, polls, p.st)) return true;
        s_abort = 1;
        return false;
    };
    auto wait_warp = [&](int i, uint32_t par) -> bool {
        const bool ok = __all_sync(0xffffffffu, mbar_wait(bar(i), par, polls, p.st));
        if (!ok) s_abort = 1;
        return ok;
    };
    auto arrive1 = [&](int i) { asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar(i)) : "memory"); };

    uint32_t done = 0;          // pieces with work that this CTA has finished (completions of B_Q)
    uint32_t tick = 0;          // ring tiles loaded (loader) or read (issuer) so far
    uint32_t s_phase = 0;       // rows: completions of this tile's B_S so far
    uint32_t p_phase0 = 0, p_phase1 = 0;  // issuer: completions of B_P
    uint32_t tails = 0;         // loader: completions of B_TAIL

    for (;;) {
        if (tid == 0) s_piece = atomicAdd(&c.head->ticket, 1);
        __syncthreads();
        const int at = s_piece;
        if (at >= pieces || s_abort) break;
        const ChunkPiece pc = c.pieces[at];
        const PagedSeq sq = paged_seq(p, pc.n, false);
        const int rows = ck_rows(sq, G, pc.t), nt = pc.kv1 - pc.kv0;
        const int act = rows > CK_M ? 2 : 1;
        const int first_new = sq.len - sq.nq;

        if (nt <= 0) {
            // nothing to do for this piece
        } else if (warp == CK_LOAD) {
            // ------------------------------------------------ loader (lane 0; all for the tail)
            const int kv_end = paged_kv_end(sq, G, (pc.t + 1) * CK_ROWS - 1);
            const int *trow = p.table + (long long)sq.row * p.P;
            const int box = min(p.page_size, CK_KT);  // tokens of one copy
            bool ok = true;
            for (int i = 0; ok && i < 2 * nt; ++i) {
                const bool val = i & 1;
                const int k0 = (pc.kv0 + (i >> 1)) * CK_KT;
                const int st = tick % S::STAGES;
                const uint32_t use = tick / S::STAGES;
                const int valid = max(0, min(CK_KT, kv_end - k0));  // keys of the tile that some row sees
                const int copies = (valid + box - 1) / box;
                const bool tail = val && valid < CK_KT;
                if (use > 0) ok = wait_warp(S::B_EMPTY + st, (use - 1) & 1);
                if (!ok) break;
                const uint32_t dst = base + S::OFF_RING + st * S::TILE;
                const int bi = tail ? S::B_TAIL : S::B_FULL + st;
                if (lane == 0) mbar_expect_tx(bar(bi), (uint32_t)copies * box * D * 2);
                __syncwarp();
                for (int k = lane; k < copies; k += 32) {
                    const int pos = k0 + k * box;
                    int page = trow[pos / p.page_size];
                    if (page < 0 || page >= p.num_pages) { report(p.st, DEV_BAD_ARG); page = 0; }
#pragma unroll
                    for (int kb = 0; kb < D / 64; ++kb)
                        tma_load_4d(dst + kb * CK_KT * 128 + k * box * 128, val ? &tm_v : &tm_k, bar(bi), kb * 64,
                                    pos % p.page_size, pc.h, page);
                }
                if (tail) {  // rows behind the end become zeros before the products see them
                    ok = wait_warp(S::B_TAIL, tails & 1);
                    ++tails;
                    for (int k = lane; k < (CK_KT - valid) * (D / 64) * 8; k += 32) {
                        const int row = valid + k / (D / 64 * 8), kb = k / 8 % (D / 64), ch = k % 8;
                        *reinterpret_cast<uint4 *>(sm + S::OFF_RING + st * S::TILE + kb * CK_KT * 128 + row * 128 + ch * 16) =
                            make_uint4(0u, 0u, 0u, 0u);
                    }
                    fence_async_smem();
                    __syncwarp();
                    if (lane == 0) arrive1(S::B_FULL + st);
                }
                ++tick;
            }
            if (!ok && lane == 0)  // leave no copy in flight into this CTA's memory
                for (uint32_t st = 0; st < S::STAGES && st < tick; ++st)
                    mbar_wait(bar(S::B_FULL + st), ((tick + S::STAGES - 1 - st) / S::STAGES - 1) & 1, ~0ull, p.st);
        } else if (warp == CK_MMA) {
            // ------------------------------------------------ issuer (lane 0; the rest idle)
            if (lane == 0) {
                const uint32_t id_s = make_idesc(BF ? 1 : 0, false, false, CK_M, CK_KT);
                const uint32_t id_o = make_idesc(BF ? 1 : 0, false, true, CK_M, D);
                auto full = [&](uint32_t tk) { return wait1(S::B_FULL + tk % S::STAGES, (tk / S::STAGES) & 1); };
                auto scores = [&](int w, uint32_t tk) {  // S[w] = Q[w] K^T
                    const uint32_t qa = base + w * CK_M * D * 2, ka = base + S::OFF_RING + tk % S::STAGES * S::TILE;
#pragma unroll
                    for (int k = 0; k < D; k += 16)
                        umma<0>(tmem + S::TM_S + w * 128, desc_kmaj<128, 2>(qa, CK_M, k), desc_kmaj<128, 2>(ka, CK_KT, k), id_s, k > 0);
                };
                auto values = [&](int w, uint32_t tk, bool add) {  // O[w] (+)= P[w] V
                    const uint32_t va = base + S::OFF_RING + tk % S::STAGES * S::TILE;
#pragma unroll
                    for (int k = 0; k < CK_KT; k += 16)
                        umma_ts(tmem + S::TM_O + w * D, tmem + S::TM_S + w * 128 + k / 2, desc_mnmaj<128>(va, CK_KT, k), id_o,
                                add || k > 0);
                };
                bool ok = wait1(S::B_Q, done & 1) && full(tick);
                if (ok) {
                    tc_fence_after();
                    for (int w = 0; w < act; ++w) {
                        scores(w, tick);
                        umma_commit(bar(S::B_S + w));
                    }
                    umma_commit(bar(S::B_EMPTY + tick % S::STAGES));
                }
                for (int i = 0; ok && i < nt; ++i) {
                    const uint32_t kt = tick + 2 * i + 2, vt = tick + 2 * i + 1;
                    const bool more = i + 1 < nt;
                    if (!(ok = full(vt))) break;
                    for (int w = 0; ok && w < act; ++w) {
                        if (!(ok = wait1(S::B_P + w, ((w ? p_phase1 : p_phase0) + i) & 1))) break;
                        tc_fence_after();
                        values(w, vt, i > 0);
                        if (w == act - 1) umma_commit(bar(S::B_EMPTY + vt % S::STAGES));
                        if (more) {
                            if (w == 0 && !(ok = full(kt))) break;
                            scores(w, kt);
                        }
                        umma_commit(bar(S::B_S + w));
                    }
                    if (ok && more) umma_commit(bar(S::B_EMPTY + kt % S::STAGES));
                }
                if (!ok) {  // leave no product in flight
                    umma_commit(bar(S::B_DRAIN));
                    mbar_wait(bar(S::B_DRAIN), 0, ~0ull, p.st);
                }
            }
            tick += 2 * nt;
            p_phase0 += nt;
            if (act == 2) p_phase1 += nt;
            __syncwarp();
        } else {
            // ------------------------------------------------ rows: thread (w, r) owns one
            const int w = warp >> 2, r = (warp & 3) * 32 + lane;
            const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
            const int row = w * CK_M + r;                           // in the item
            const bool real = row < rows;
            const int tok = (pc.t * CK_ROWS + row) / G, head = pc.h * G + (pc.t * CK_ROWS + row) % G;
            bool ok = true;
            {   // its query, to the swizzled tile
                const uint4 *src = reinterpret_cast<const uint4 *>(p.q + (real ? (sq.q0 + tok) * p.q_ts + (long long)head * D : 0));
                uint4 x[D / 8];
#pragma unroll
                for (int k = 0; k < D / 8; ++k) x[k] = real ? src[k] : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
                for (int k = 0; k < D / 8; ++k)
                    *reinterpret_cast<uint4 *>(sm + w * CK_M * D * 2 + kmaj<128, 2>(r, k * 8, CK_M)) = x[k];
                fence_async_smem();
                __syncwarp();
                if (lane == 0) arrive1(S::B_Q);
            }
            const int last = real ? first_new + tok : -1;            // the last key that the row sees
            float m = -INFINITY, l = 0.f;                            // m in the scores' units
            const float sc = p.scale_log2;
            const uint32_t ts = tmem + lanes + S::TM_S + w * 128, to = tmem + lanes + S::TM_O + w * D;
            if (w < act) {
                for (int i = 0; i < nt; ++i) {
                    if (!(ok = wait_warp(S::B_S + w, (s_phase + i) & 1))) break;
                    tc_fence_after();
                    uint32_t x[128];
                    tm_ld32(ts, x);
                    tm_ld32(ts + 32, x + 32);
                    tm_ld32(ts + 64, x + 64);
                    tm_ld32(ts + 96, x + 96);
                    tmem_wait_ld();
                    const int lim = last - (pc.kv0 + i) * CK_KT;     // columns 0 .. lim are seen
                    if (__any_sync(0xffffffffu, lim < CK_KT - 1)) {
#pragma unroll
                        for (int k = 0; k < 128; ++k)
                            if (k > lim) x[k] = 0xff800000u;
                    }
                    float m4[4] = {m, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int k = 0; k < 128; ++k) m4[k & 3] = fmaxf(m4[k & 3], __uint_as_float(x[k]));
                    const float mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
                    // a new reference where the row has none yet or its maximum outgrew it
                    const bool grow = mx > -INFINITY && (m == -INFINITY || (mx - m) * sc > 8.f);
                    if (__any_sync(0xffffffffu, grow)) {
                        const float f = grow ? ex2((m - mx) * sc) : 1.f;  // 2^-inf = 0 at first
                        if (grow) m = mx;
                        l *= f;
                        if (i > 0) {  // the products into O so far are done: B_S completed after them
#pragma unroll
                            for (int k = 0; k < D; k += 32) {
                                uint32_t y[32];
                                tm_ld32(to + k, y);
                                tmem_wait_ld();
#pragma unroll
                                for (int e = 0; e < 32; ++e) y[e] = __float_as_uint(__uint_as_float(y[e]) * f);
                                tm_st32(to + k, y);
                            }
                        }
                    }
                    const float ref = m == -INFINITY ? 0.f : m * sc;
                    float l4[4] = {};
#pragma unroll
                    for (int k0 = 0; k0 < 128; k0 += 64) {
                        uint32_t y[32];
#pragma unroll
                        for (int k = 0; k < 64; k += 2) {
                            const float a = ex2(fmaf(__uint_as_float(x[k0 + k]), sc, -ref));
                            const float b = ex2(fmaf(__uint_as_float(x[k0 + k + 1]), sc, -ref));
                            l4[k & 2] += a;
                            l4[(k & 2) + 1] += b;
                            y[k / 2] = pack16x2<BF>(a, b);
                        }
                        tm_st32(ts + k0 / 2, y);
                    }
                    l += (l4[0] + l4[1]) + (l4[2] + l4[3]);
                    tm_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) arrive1(S::B_P + w);
                }
                // the sums, after the last product
                if (ok && (ok = wait_warp(S::B_S + w, (s_phase + nt) & 1))) {
                    tc_fence_after();
                    const bool whole = pc.part_row < 0;
                    const float inv = l > 0.f || l != l ? 1.f / l : 0.f;  // a row that sees nothing: 0
                    uint16_t *dst = p.out + ((long long)(sq.q0 + tok) * p.Hq + head) * D;
                    float *part = p.part_o + ((long long)pc.part_row + row) * D;
#pragma unroll
                    for (int k = 0; k < D; k += 32) {
                        uint32_t y[32];
                        tm_ld32(to + k, y);
                        tmem_wait_ld();
                        if (!real) continue;
                        if (whole) {
#pragma unroll
                            for (int e = 0; e < 32; e += 8) {
                                uint4 z;
                                z.x = pack16x2<BF>(__uint_as_float(y[e]) * inv, __uint_as_float(y[e + 1]) * inv);
                                z.y = pack16x2<BF>(__uint_as_float(y[e + 2]) * inv, __uint_as_float(y[e + 3]) * inv);
                                z.z = pack16x2<BF>(__uint_as_float(y[e + 4]) * inv, __uint_as_float(y[e + 5]) * inv);
                                z.w = pack16x2<BF>(__uint_as_float(y[e + 6]) * inv, __uint_as_float(y[e + 7]) * inv);
                                *reinterpret_cast<uint4 *>(dst + k + e) = z;
                            }
                        } else {
#pragma unroll
                            for (int e = 0; e < 32; e += 4)
                                *reinterpret_cast<uint4 *>(part + k + e) = make_uint4(y[e], y[e + 1], y[e + 2], y[e + 3]);
                        }
                    }
                    if (real) {
                        if (!whole) p.part_ml[pc.part_row + row] = make_float2(m == -INFINITY ? m : m * sc, l);
                        else if (p.lse != nullptr)
                            p.lse[(long long)(sq.q0 + tok) * p.Hq + head] = m == -INFINITY ? -INFINITY : m * sc * LN2 + logf(l);
                    }
                    tc_fence_before();
                }
                s_phase += nt + 1;
            }
        }
        if (nt > 0) ++done;
        __syncthreads();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == CK_MMA) tmem_dealloc(tmem, 512);
}

// ------------------------------------------------------------------- host ----
int paged_chunk_tile() { return CK_ROWS; }

// Whether pages of this shape can be loaded by tensor copies: a copy is a page, or 128 tokens
// of it, and begins on an 8-row swizzle atom of the tile.
bool paged_chunk_pages(int page_size) {
    return page_size >= 8 && (page_size % CK_KT == 0 || CK_KT % page_size == 0);
}

// Sizes of the plan for these bounds; sms: of the device.
ChunkLimits paged_chunk_limits(int N, int total_q, int G, int Hkv, int span, int sms) {
    ChunkLimits m;
    const long long seqs = N < total_q ? N : total_q;
    const long long tiles = (long long)total_q * G / CK_ROWS + seqs, items = tiles * Hkv;
    const long long keys = (span + CK_KT - 1) / CK_KT;  // an item's tiles at most
    // room to cut the items into eight pieces per SM more than there are items, and for
    // four per SM of whole partial sums
    long long pieces = items + 8LL * sms, rows = 4LL * sms * CK_ROWS;
    if (keys < pieces / items + 1 && items * keys < pieces) pieces = items * keys;
    const long long all = pieces * CK_ROWS < (long long)total_q * G * Hkv * keys ? pieces * CK_ROWS : (long long)total_q * G * Hkv * keys;
    if (all < rows) rows = all;
    if (keys == 1) rows = 0;  // nothing to cut
    m.pieces = (int)(pieces < 0x7fffffffLL ? pieces : 0x7fffffffLL);
    m.rows = (int)rows;
    m.entries = (int)(rows / 2 + 1 < m.pieces ? rows / 2 + 1 : m.pieces);
    return m;
}
size_t paged_chunk_piece_bytes() { return sizeof(ChunkPiece); }

static bool page_map(CUtensorMap *map, PFN_cuTensorMapEncodeTiled_v12000 enc, const void *ptr, bool bf, int d, int page_size,
                     int Hkv, int pages, long long ps, long long ts, long long hs) {
    cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)page_size, (cuuint64_t)Hkv, (cuuint64_t)pages};
    cuuint64_t strides[3] = {(cuuint64_t)ts * 2, (cuuint64_t)hs * 2, (cuuint64_t)ps * 2};
    cuuint32_t box[4] = {64u, (cuuint32_t)(page_size < CK_KT ? page_size : CK_KT), 1u, 1u};
    cuuint32_t one[4] = {1u, 1u, 1u, 1u};
    return enc(map, bf ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4, const_cast<void *>(ptr), dims,
               strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool BF>
static cudaError_t launch_chunk_t(const CUtensorMap &tk, const CUtensorMap &tv, const ChunkParams &c, cudaStream_t stream) {
    cudaError_t e = cudaFuncSetAttribute(paged_chunk_kernel<D, BF>, cudaFuncAttributeMaxDynamicSharedMemorySize, CkShape<D>::SMEM);
    if (e != cudaSuccess) return e;
    // one block plans; with new tokens to place, two an SM place them meanwhile
    const long long vecs = (long long)c.p.total_q * c.p.Hkv * (D / 8), blocks = (vecs + 511) / 512;
    const int more = c.p.k_new == nullptr ? 0 : (int)(blocks < 2LL * c.sms ? blocks : 2LL * c.sms);
    paged_plan_kernel<D><<<1 + more, 512, 0, stream>>>(c);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    paged_chunk_kernel<D, BF><<<c.max_pieces < c.sms ? c.max_pieces : c.sms, CK_THREADS, CkShape<D>::SMEM, stream>>>(tk, tv, c);
    return cudaGetLastError();
}

// ws: the plan's part of the workspace: head (256 bytes), base [N], pieces.
cudaError_t launch_paged_chunk(const PagedParams &p, const ChunkLimits &m, void *ws, int d, bool bf, int sms, cudaStream_t stream) {
    PFN_cuTensorMapEncodeTiled_v12000 enc = nullptr;
    if (host_encoder(&enc) != 0) return cudaErrorUnknown;
    CUtensorMap tk, tv;
    if (!page_map(&tk, enc, p.kp, bf, d, p.page_size, p.Hkv, p.num_pages, p.k_ps, p.k_ts, p.k_hs) ||
        !page_map(&tv, enc, p.vp, bf, d, p.page_size, p.Hkv, p.num_pages, p.v_ps, p.v_ts, p.v_hs))
        return cudaErrorInvalidValue;
    ChunkParams c;
    c.p = p;
    c.head = static_cast<ChunkPlanHead *>(ws);
    c.base = reinterpret_cast<int *>(static_cast<uint8_t *>(ws) + 256);
    c.pieces = reinterpret_cast<ChunkPiece *>(reinterpret_cast<uint8_t *>(c.base) + ((size_t)p.N * 4 + 255) / 256 * 256);
    c.max_pieces = m.pieces;
    c.max_entries = m.entries;
    c.max_rows = m.rows;
    c.sms = sms;
    if (d == 128)
        return bf ? launch_chunk_t<128, true>(tk, tv, c, stream) : launch_chunk_t<128, false>(tk, tv, c, stream);
    return bf ? launch_chunk_t<64, true>(tk, tv, c, stream) : launch_chunk_t<64, false>(tk, tv, c, stream);
}

}  // namespace kda
