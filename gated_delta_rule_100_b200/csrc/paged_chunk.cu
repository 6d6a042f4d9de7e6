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
// - one warp issues every product, one loads pages by TMA (the values of one key
//   tile with the keys of the next, as the steps read them, in two stages), eight
//   own a row per thread.
// - weights are formed with the reference there is and looked at afterwards, so
//   no maximum stands between scores and weights; the sums stay in TMEM and are
//   rescaled only when 64 weights add up to more than 2^7 times what the
//   reference allows (16-bit rounding is relative and the sums are fp32), so
//   after the first keys hardly ever.
// - one weight in sixteen is a polynomial's, which takes work off the exponential
//   unit.  (Both this and sums rescaled only past a threshold are published ideas; the
//   thresholds, the share and the coefficients are this file's own.)
// - the rows of masked keys behind the sequence's end are zeroed in the last
//   value tile: a page holds anything there, and 0 x NaN is NaN.
//
// Measured, 2048 new tokens over 65,536 keys, 32 query heads, 8 key heads of 128:
// 1.62 to 1.67 ms a call in a short run, 1300 to 1340 TFLOP/s or 77 to 80 % of a
// library product's rate in a burst, and 1.91 ms a call in a long one under the power
// limit, 1130 TFLOP/s or 79 % of that product's sustained rate.  At d = 64, 2048 tokens
// over 16,384 keys: 698 TFLOP/s, where half the tensor work comes with each
// exponential (1173 at d = 128; fp16 698 and 1145).  A 256 x 128 tile takes about
// 3000 cycles at d = 128, of which the
// tensor cores work 2048: the rest is the way from scores to weights (TMEM load,
// 2^x, TMEM store and three hand-offs) where a tile's own warps are the only ones
// that can go on.  Four row tiles would hide it; registers (a row's 64 scores and
// their weights) and TMEM (two tiles' scores and sums are all 512 columns at d =
// 128) hold two.  Slower forms measured: 64 keys a step with scores in two
// buffers (1.93 ms: products of 64 columns take 57 cycles, not 32), two floats an
// instruction (3.3 cycles for two), 16 warps of rows, two a row (2 % faster here,
// 3 % slower on mixed batches, and the hand-offs twice as many).
//
// Work: a plan kernel (one block; the others meanwhile write the new tokens to
// their pages) cuts the items' keys into pieces, by the shortest of 32 modelled
// times; CTAs, one per SM, claim pieces from a counter.  Pieces of a split item
// are joined by paged_join_kernel in a fixed order.
#include "kda_internal.cuh"
#include "paged_params.cuh"

namespace kda {

constexpr int CK_M = 128, CK_KT = 128, CK_ROWS = 2 * CK_M;  // rows of a tile, keys of a loaded tile, rows of an item
constexpr int CK_STEP = 64;                                  // keys whose weights are formed at a time
constexpr int CK_RW = 8;                                     // warps of rows, four a tile
constexpr int CK_MMA = CK_RW, CK_LOAD = CK_RW + 1;           // one for the products, one for the loads, two idle
constexpr int CK_THREADS = (CK_RW + 4) * 32;
constexpr int CK_REGS_ROWS = 216, CK_REGS_REST = 72;         // 256 x 216 + 128 x 72 = 384 x 168, the launch's registers

// One piece of work: keys [kv0, kv1) in tiles of rows [t 256, t 256 + 256) of
// (n, h); part_row: where its partial sums go, or -1 when it is the whole item.
struct ChunkPiece {
    int n, h, t, kv0, kv1;
    int part_row;
    PagedSeq s;  // the sequence's numbers, checked
    int pad[2];
};
struct ChunkPlanHead {
    int pieces, ticket, entries, pad;
};
struct ChunkParams {
    PagedParams p;
    ChunkPlanHead *head;
    ChunkPiece *pieces;
    int *base;             // [3][N] the plan's scratch
    int max_pieces, max_entries, max_rows, sms;
};

template <int D>
struct CkShape {
    static constexpr int TILE = CK_KT * D * 2;                    // a key or value tile
    // two stages of keys, then two of values
    static constexpr int OFF_K = 2 * CK_M * D * 2, OFF_V = OFF_K + 2 * TILE;  // behind the two query tiles
    static constexpr int OFF_BAR = OFF_V + 2 * TILE;
    // barriers: queries [tile], scores [tile], weights [tile][half], a half's products [tile], a pair of tiles loaded [stage],
    // read [stage], a tail's copies, the end of all products, pieces handed on [2], taken [2]
    static constexpr int B_Q = 0, B_S = 2, B_P = 4, B_HALF = 8, B_FULL = 10, B_EMPTY = 12, B_TAIL = 14, B_DRAIN = 15, B_WORK = 16,
                         B_FREE = 18, NBAR = 20;
    static constexpr int SMEM = OFF_BAR + NBAR * 8 + 32;          // and five words
    static constexpr uint32_t TM_S = 0, TM_O = 256;               // columns: S0, S1, O0, O1
};

// ------------------------------------------------------------------- plan ----
__device__ __forceinline__ int ck_tiles(const PagedSeq &s, int G) { return (int)(((long long)s.nq * G + CK_ROWS - 1) / CK_ROWS); }
__device__ __forceinline__ int ck_keys(const PagedSeq &s, int G, int t) {  // key tiles of row tile t
    return max(1, (paged_kv_end(s, G, (t + 1) * CK_ROWS - 1) + CK_KT - 1) / CK_KT);
}
// rows that row tile t holds
__device__ __forceinline__ int ck_rows(const PagedSeq &s, int G, int t) { return min(CK_ROWS, s.nq * G - t * CK_ROWS); }

// Cutting the items.  In each sequence the row tiles with the most keys stay
// whole (a share `phi` of the tiles: none, or as many as fill whole waves of
// SMs), the others are cut into pieces of `step` key tiles, one of sixteen
// divisors of the longest.  The 32 candidates are compared by a modelled time in
// key tiles: a piece costs its tiles and about three more; the whole items' waves
// first, their last wave's idle SMs already at the pieces; then the pieces' waves;
// and the join of what was cut, at the memory's rate.
constexpr int CK_CAND = 16;
__device__ __constant__ int ck_div[CK_CAND] = {1, 2, 3, 4, 5, 6, 7, 8, 10, 12, 16, 24, 32, 64, 128, 256};

__device__ void ck_plan(const ChunkParams &c, int d) {
    // of one key head; rows in eights.  32 bits hold them: there are below 2^24 tiles, and rows of
    // candidates with more pieces than there is room for do not count
    __shared__ unsigned s_pieces[2 * CK_CAND], s_rows8[2 * CK_CAND], s_a;
    __shared__ unsigned long long s_w, s_wa, s_q;
    __shared__ int s_max, s_ma, s_items, s_step, s_phi, s_entries, s_part, s_sum[33];
    const PagedParams &p = c.p;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, warps = blockDim.x >> 5, G = p.G;
    if (tid == 0) { s_w = s_q = 0; s_wa = s_a = 0; s_max = 1; s_ma = s_items = s_entries = s_part = 0; }
    if (tid < 2 * CK_CAND) s_pieces[tid] = s_rows8[tid] = 0;
    __syncthreads();
    // a warp a sequence, a lane a row tile
    unsigned long long w = 0, tokens = 0;
    int mx = 1, items = 0;
    for (int n = warp; n < p.N; n += warps) {
        const PagedSeq s = paged_seq(p, n, lane == 0);
        tokens += s.nq;
        for (int t = lane; t < ck_tiles(s, G); t += 32) {
            const int k = ck_keys(s, G, t);
            w += k;
            mx = max(mx, k);
            ++items;
        }
    }
    // a warp's sum first: 32 lanes' atomics on one 64-bit word of shared memory wait for one another
    auto warp_sum = [](unsigned long long v) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        return v;
    };
    w = warp_sum(w);
    mx = __reduce_max_sync(0xffffffffu, mx);
    items = __reduce_add_sync(0xffffffffu, items);
    if (lane == 0 && items) {
        atomicAdd(&s_w, w);
        atomicAdd(&s_q, tokens);
        atomicMax(&s_max, mx);
        atomicAdd(&s_items, items);
    }
    __syncthreads();
    if (s_q > (unsigned long long)p.total_q) {  // sequences overlap, which was reported: more work than there is room for
        if (tid == 0) c.head->pieces = c.head->ticket = c.head->entries = 0;
        return;
    }
    const long long all = (long long)s_items * p.Hkv;
    const float phi1 = (float)(all / c.sms * c.sms) / fmaxf((float)all, 1.f);
    // whole tiles of a sequence: ranks below, counted from the one with the most keys
    auto whole = [&](int tiles, int phi) { return phi ? (int)(tiles * phi1) : 0; };
    const int split = max(1, warps / p.N);  // few sequences share the warps: here among their tiles, below among the heads
    {   // a lane a candidate
        const int q = lane / CK_CAND;
        const int step = (s_max + ck_div[lane % CK_CAND] - 1) / ck_div[lane % CK_CAND];
        unsigned long long wa = 0;
        unsigned na = 0, pieces = 0, rows8 = 0;
        int ma = 0;
        for (int v = warp; v < p.N * split; v += warps) {
            const PagedSeq s = paged_seq(p, v % p.N, false);
            const int tiles = ck_tiles(s, G), a = whole(tiles, 1);
            for (int t = v / p.N; t < tiles; t += split) {
                const int k = ck_keys(s, G, t), ns = (k + step - 1) / step;
                const bool in_a = tiles - 1 - t < a;
                if (in_a) { wa += k; ++na; ma = max(ma, k); }
                if (!(q && in_a)) {
                    pieces += ns;
                    if (ns > 1) rows8 += ns * ((ck_rows(s, G, t) + 7) / 8);
                }
            }
        }
        atomicAdd(&s_pieces[lane], pieces);
        atomicAdd(&s_rows8[lane], rows8);
        if (lane == 0) {
            atomicAdd(&s_wa, wa);
            atomicAdd(&s_a, na);
            atomicMax(&s_ma, ma);
        }
    }
    __syncthreads();
    if (warp == 0) {
        const int q = lane / CK_CAND, j = lane % CK_CAND, step = (s_max + ck_div[j] - 1) / ck_div[j];
        const float S = (float)c.sms, R = (float)s_rows8[lane] * 8.f * p.Hkv;
        const float pa = q ? (float)s_a * p.Hkv : 0.f, ta = q && s_a ? __fdividef((float)s_wa, (float)s_a) + 3.f : 0.f;
        const float pb = (float)s_pieces[lane] * p.Hkv,
                    tb = pb > 0.f ? __fdividef((float)(s_w - (q ? s_wa : 0)) * p.Hkv, pb) + 3.f : 3.f;
        const float ka = ceilf(__fdividef(pa, S)), early = (ka * S - pa) * floorf(__fdividef(ta, tb));
        float cost = ka * ta + (pb > early ? ceilf(__fdividef(pb - early, S)) * tb : 0.f);
        cost = fmaxf(cost, max(pa > 0.f ? s_ma : 0, pb > 0.f ? step : 0) + 3.f);  // no less than the longest
        if (R > 0.f) cost += 3.f + R * d * 8.f * 1.2e-7f;
        // what the workspace has no room for is out (not the uncut items, which it always has room for)
        const unsigned long long np = (unsigned long long)(s_pieces[lane] + (q ? s_a : 0u)) * p.Hkv, nr = s_rows8[lane] * 8ull * p.Hkv;
        if (lane > 0 && (np > (unsigned long long)c.max_pieces || nr > (unsigned long long)c.max_rows)) cost = 3.0e38f;
        float best = cost;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) best = fminf(best, __shfl_xor_sync(0xffffffffu, best, o));
        const int who = __ffs(__ballot_sync(0xffffffffu, cost == best)) - 1;
        if (lane == who) { s_step = step; s_phi = q; }
    }
    __syncthreads();
    const int step = s_step, phi = s_phi;
    // The order of the pieces, for CTAs that claim them one by one: whole items, then pieces of the
    // full length and rests of half of it, then the other rests, so that what is claimed last is
    // short.  Pieces of each kind per key head of a sequence; then where each sequence's begin.
    for (int n = warp; n < p.N; n += warps) {
        const PagedSeq s = paged_seq(p, n, false);
        const int tiles = ck_tiles(s, G), a = whole(tiles, phi);
        int full = 0, rest = 0;
        for (int t = lane; t < tiles - a; t += 32) {
            const int k = ck_keys(s, G, t);
            const int big = 2 * (k % step) >= step;
            full += k / step + big;
            rest += !big && k % step != 0;
        }
        full = __reduce_add_sync(0xffffffffu, full);
        rest = __reduce_add_sync(0xffffffffu, rest);
        if (lane == 0) {
            c.base[n] = a * p.Hkv;
            c.base[n + p.N] = full * p.Hkv;
            c.base[n + 2 * p.N] = rest * p.Hkv;
        }
    }
    __syncthreads();
    const int cells = 3 * p.N, per = (cells + blockDim.x - 1) / blockDim.x;
    int mine = 0;
    for (int n = tid * per; n < min(cells, (tid + 1) * per); ++n) mine += c.base[n];
    int incl = mine, total = 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += up;
    }
    if (lane == 31) s_sum[warp] = incl;
    __syncthreads();
    int at = incl - mine;
    for (int k = 0; k < warps; ++k) {
        if (k < warp) at += s_sum[k];
        total += s_sum[k];
    }
    for (int n = tid * per; n < min(cells, (tid + 1) * per); ++n) {
        const int k = c.base[n];
        c.base[n] = at;
        at += k;
    }
    __syncthreads();
    for (int v = warp; v < p.N * split; v += warps) {
        const int n = v % p.N, h0 = v / p.N, heads = (p.Hkv - h0 + split - 1) / split;  // key heads h0, h0 + split, ..
        const PagedSeq s = paged_seq(p, n, false);
        const int tiles = ck_tiles(s, G), a = whole(tiles, phi);
        const int w0 = c.base[n], f0 = c.base[n + p.N], r0 = c.base[n + 2 * p.N];
        const int full_head = (c.base[n + p.N + 1] - f0) / p.Hkv;
        const int rest_head = ((n + 1 < p.N ? c.base[n + 2 * p.N + 1] : total) - r0) / p.Hkv;
        int full_before = 0, rest_before = 0;
        for (int t0 = 0; t0 < tiles && heads > 0; t0 += 32) {
            const int tl = tiles - 1 - t0 - lane;  // a lane a tile, the longest first
            const bool wl = t0 + lane < a;
            const int kl = tl >= 0 ? ck_keys(s, G, tl) : 0, big = 2 * (kl % step) >= step,
                      full = wl ? 0 : kl / step + big, rest = !wl && !big && kl % step != 0;
            int fi = full, ri = rest;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int uf = __shfl_up_sync(0xffffffffu, fi, o), ur = __shfl_up_sync(0xffffffffu, ri, o);
                if (lane >= o) { fi += uf; ri += ur; }
            }
            const int work = min(32, tiles - t0) * heads;
            for (int b = 0; b < work; b += 32) {  // then a lane an item: a tile of a head
                const int of = min((b + lane) / heads, 31), h = h0 + (b + lane) % heads * split;
                const int k = __shfl_sync(0xffffffffu, kl, of), nf = __shfl_sync(0xffffffffu, full, of),
                          nr = __shfl_sync(0xffffffffu, rest, of), fb = full_before + __shfl_sync(0xffffffffu, fi, of) - nf,
                          rb = rest_before + __shfl_sync(0xffffffffu, ri, of) - 1;
                if (b + lane >= work) continue;
                const int rank = t0 + of, t = tiles - 1 - rank;
                const bool w1 = rank < a;
                const int r = ck_rows(s, G, t), ns = w1 ? 1 : nf + nr;
                int part = -1;
                if (ns > 1) {
                    part = atomicAdd(&s_part, ns * r);
                    const int e = atomicAdd(&s_entries, 1);
                    if (e < c.max_entries && part + ns * r <= c.max_rows)
                        p.entries[e] = {n, h, t, part, part + r, ns - 1, r};
                    else report(p.st, DEV_BAD_ARG);  // only where cu_q or length change meanwhile
                }
                // a piece without room for its sums is left empty
                const bool room = part < 0 || part + ns * r <= c.max_rows;
                for (int j = 0; j < ns; ++j) {
                    const unsigned i = w1 ? w0 + h * a + rank : j < nf ? f0 + h * full_head + fb + j : r0 + h * rest_head + rb;
                    if (i >= (unsigned)c.max_pieces) { report(p.st, DEV_BAD_ARG); continue; }
                    const int kv0 = j * step;
                    c.pieces[i] = {n, h, t, kv0, !room ? kv0 : w1 ? k : min(k, kv0 + step), part < 0 ? -1 : part + j * r, s, {0, 0}};
                }
            }
            full_before += __shfl_sync(0xffffffffu, fi, 31);
            rest_before += __shfl_sync(0xffffffffu, ri, 31);
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
        if (!KDA_CHECK(p.st, h < p.Hkv && pos < p.P * p.page_size)) continue;
        const uint4 kx = *reinterpret_cast<const uint4 *>(p.k_new + tok * p.kn_ts + h * D + ch * 8);
        const uint4 vx = *reinterpret_cast<const uint4 *>(p.v_new + tok * p.vn_ts + h * D + ch * 8);
        *reinterpret_cast<uint4 *>(p.kp + page * p.k_ps + in * p.k_ts + h * p.k_hs + ch * 8) = kx;
        *reinterpret_cast<uint4 *>(p.vp + page * p.v_ps + in * p.v_ts + h * p.v_hs + ch * 8) = vx;
    }
}

template <int D>
__global__ void __launch_bounds__(512) paged_plan_kernel(const ChunkParams c) {
    launch_dependents();  // the chunk kernel sets itself up meanwhile
    if (blockIdx.x == 0) ck_plan(c, D);
    else ck_append<D>(c, (long long)(blockIdx.x - 1) * blockDim.x + threadIdx.x, (long long)(gridDim.x - 1) * blockDim.x);
}

// A bounded wait of at most `tries` tries, in five instructions.  mbar_wait reads
// %globaltimer after its first miss, which takes longer than most waits here (it
// cost each contended wait 300 to 600 cycles), and is long where the
// instruction cache is short of room.  A try that misses sleeps for 4 us (measured, with
// one warp waiting and with twelve), so CK_TRIES of them are the second that a bounded
// wait lasts elsewhere.
constexpr uint32_t CK_TRIES = 1u << 18;
__device__ __forceinline__ bool ck_wait(uint32_t bar, uint32_t parity, uint32_t tries) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .u32 n;\n\tmov.u32 n, %3;\n"
        "again_%=:\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t@p bra done_%=;\n\t"
        "sub.u32 n, n, 1;\n\tsetp.ne.u32 q, n, 0;\n\t@q bra again_%=;\n"
        "done_%=:\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok) : "r"(bar), "r"(parity), "r"(tries) : "memory");
    return ok != 0;
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
__device__ __forceinline__ void tm_st16(uint32_t a, const uint32_t *r) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(a),
                 "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
                 "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
                 : "memory");
}
// Waits for the loads; the registers go through it, so that nothing reads them before.
__device__ __forceinline__ void tm_wait_ld32(uint32_t *r) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]),
                   "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
                 :: "memory");
    asm volatile("" : "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]),
                 "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31]) :: "memory");
}
__device__ __forceinline__ void tm_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// The products, with descriptors by their low word (address and leading stride);
// the high word is the same for all of them here: 1024 bytes between 8-row atoms,
// 128-byte swizzle.  Few instructions between products count: the issuing warp
// runs alone, at some ten cycles each.
constexpr uint32_t DESC_HI = (1024u >> 4) | 1u << 14 | 2u << 29;
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr, uint32_t lead) { return (addr >> 4) | (lead >> 4) << 16; }
// D[tmem] (+)= A[smem] B[smem]
__device__ __forceinline__ void umma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\tsetp.ne.b32 p, %4, 0;\n\tmov.b64 a, {%1, %5};\n\tmov.b64 b, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "n"(DESC_HI)
        : "memory");
}
// D[tmem] (+)= A[tmem] B[smem]: A's rows are lanes, two 16-bit values a column.
__device__ __forceinline__ void umma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\tsetp.ne.b32 p, %4, 0;\n\tmov.b64 b, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "n"(DESC_HI)
        : "memory");
}

// One lane of a converged warp.  The compiler knows that the branch on it holds
// for a single lane, and keeps descriptors in uniform registers: products issued
// under `lane == 0` cost 73 to 87 cycles each, under this 64, the tensor
// cores' own time for 128 x 128 x 16.
__device__ __forceinline__ bool elect_lane() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}

// 2^x without the exponential unit, for x = s sc - ref: y = (x + LOW) / 128 in one
// operation that also holds it in [0, 1] (x in [-LOW, 128 - LOW]); x = n + r with n
// the nearest integer (128 y - LOW added to 1.5 2^23, whose last place is 1, leaves
// n in the low bits) and r in [-1/2, 1/2]; 2^r by the polynomial of degree 4 with
// the least largest relative error there, 2.7e-6 (a least-squares fit with its
// weights moved to the error's peaks); n added to the exponent.  y's last place
// is another 2.6e-6; a weight's 16-bit rounding is 50 times both or more.  A score
// far below the maximum weighs 2^-LOW and not 0: not for masked keys.
template <bool BF>
struct Poly {
    static constexpr float LOW = BF ? 120.f : 112.f, SHIFT = 12582912.f - LOW;
    float a, b;  // y = s a + b
    __device__ __forceinline__ Poly(float sc, float ref) : a(sc * 0.0078125f), b((LOW - ref) * 0.0078125f) {}
    __device__ __forceinline__ float operator()(float s) const {
        float y;
        asm("fma.rn.sat.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(s), "f"(a), "f"(b));
        const float t = fmaf(y, 128.f, SHIFT);
        const float r = fmaf(y, 128.f, SHIFT - t);
        float q = fmaf(r, 0.0095701003447f, 0.0559178590775f);
        q = fmaf(q, r, 0.2402474433184f);
        q = fmaf(q, r, 0.6931217908859f);
        q = fmaf(q, r, 0.9999992847443f);
        return __uint_as_float(__float_as_uint(q) + (__float_as_uint(t) << 23));
    }
};

// Weights 2^(x sc - ref) of a row's N scores as 16-bit pairs, and their sum
// before the rounding.  MIX: one of sixteen by the polynomial, which takes work
// off the exponential unit (512 cycles a warp for 64); it has no 0 for masked keys.
// 2048 tokens over 65,536 keys: 1.68 ms with none, 1.635 with one in 32, 1.62 with
// one in 16, 1.625 with one in 8, 1.68 with three in 16 and one in 4.
template <bool BF, bool MIX, int N>
__device__ __forceinline__ float ck_weights(const uint32_t (&x)[N], uint32_t *y, float sc, float ref) {
    const Poly<BF> poly(sc, ref);
    float l[4] = {}, nan = 0.f;
#pragma unroll
    for (int k = 0; k < N; k += 2) {
        const float u = __uint_as_float(x[k]), v = __uint_as_float(x[k + 1]);
        const float a = ex2(fmaf(u, sc, -ref));
        const float b = MIX && k % 16 == 0 ? poly(v) : ex2(fmaf(v, sc, -ref));
        l[k & 2] += a;
        l[(k & 2) + 1] += b;
        if (MIX && k % 16 == 0) asm("max.NaN.f32 %0, %0, %1;" : "+f"(nan) : "f"(v));  // which the polynomial's clamp drops
        y[k / 2] = pack16x2<BF>(a, b);
    }
    const float sum = (l[0] + l[1]) + (l[2] + l[3]);
    return MIX && nan != nan ? nan : sum;
}

// The issuing lane's walk over a piece.  Its loop holds the steps of one key tile
// and no more: it runs alone, at some ten cycles an instruction, so a loop
// over the steps cost 400 cycles each; and the instruction cache that it shares
// with two of the rows' warps is short, so unrolled over the stages too it slowed
// those two by half.
template <int D, bool BF>
struct Issuer {
    using S = CkShape<D>;
    uint32_t base, tmem, tries;
    uint32_t q_par0 = 0, q_par1 = 0, p_par0 = 0, p_par1 = 0, f_par = 0;  // parities waited for next

    __device__ __forceinline__ uint32_t bar(int i) const { return base + S::OFF_BAR + i * 8; }
    template <int W>
    __device__ __forceinline__ void scores(uint32_t k) const {  // S[W] = Q[W] K^T, k: the key tile's descriptor
        constexpr uint32_t idesc = make_idesc(BF ? 1 : 0, false, false, CK_M, CK_KT);
        uint32_t q = desc_lo(base, 16) + W * (CK_M * D * 2 / 16);
        asm volatile("" : "+r"(q), "+r"(k));  // the products' descriptors are formed here, not kept
#pragma unroll
        for (int e = 0; e < D; e += 16) {
            constexpr int KB = CK_KT * 128 / 16;  // 16-byte units of 64 channels
            umma_ss(tmem + S::TM_S + W * 128, q + e / 64 * KB + e % 64 / 8, k + e / 64 * KB + e % 64 / 8, idesc, e > 0);
        }
    }
    template <int W, int H>
    __device__ __forceinline__ bool values(uint32_t v, bool add) const {  // O[W] (+)= P[W][H] V, half H of the value tile
        constexpr uint32_t idesc = make_idesc(BF ? 1 : 0, false, true, CK_M, D);
        if (!ck_wait(bar(S::B_P + W * 2 + H), W ? p_par1 : p_par0, tries)) return false;
        tc_fence_after();
        asm volatile("" : "+r"(v));
#pragma unroll
        for (int e = 0; e < CK_STEP; e += 16)
            umma_ts(tmem + S::TM_O + W * D, tmem + S::TM_S + W * 128 + (H * CK_STEP + e) / 2, v + (H * CK_STEP + e) * 128 / 16, idesc,
                    H || e ? 1u : (uint32_t)add);
        return true;
    }
    // a tile's weights times their values as the halves come, then its scores of the next keys
    template <int W>
    __device__ __forceinline__ bool step(uint32_t v, uint32_t k, bool add, bool more) const {
        if (!values<W, 0>(v, add)) return false;
        umma_commit(bar(S::B_HALF + W));
        if (!values<W, 1>(v, true)) return false;
        if (more) scores<W>(k);
        umma_commit(bar(S::B_S + W));  // and every product before it
        return true;
    }
    // Tiles come in pairs, the values of key tile i with the keys of tile i + 1: that is what
    // tile i's steps read, so one barrier says that both are there and one that both are free.
    // The pair of tile i is in stage (i + 1) & 1; its values lie in that stage of their ring, its
    // keys in the other.  A piece's first pair is its first keys alone, and it takes an even
    // number of pairs (the last one empty if need be), so that it begins at stage 0.
    __device__ __forceinline__ bool full(uint32_t st) {
        if (!ck_wait(bar(S::B_FULL) + st * 8, f_par, tries)) return false;
        f_par ^= st;
        return true;
    }
    __device__ __forceinline__ bool run(int nt, bool both) {
        const uint32_t k0 = desc_lo(base + S::OFF_K, 16), v0 = desc_lo(base + S::OFF_V, CK_KT * 128);
        if (!full(0) || !ck_wait(bar(S::B_Q), q_par0, tries)) return false;
        q_par0 ^= 1;
        tc_fence_after();
        scores<0>(k0 + S::TILE / 16);
        umma_commit(bar(S::B_S));
        if (both) {
            if (!ck_wait(bar(S::B_Q + 1), q_par1, tries)) return false;
            q_par1 ^= 1;
            tc_fence_after();
            scores<1>(k0 + S::TILE / 16);
            umma_commit(bar(S::B_S + 1));
        }
        umma_commit(bar(S::B_EMPTY));
        uint32_t st = 1;
#pragma unroll 1
        for (int i = 0; i < nt; ++i, st ^= 1) {
            const uint32_t v = v0 + st * (S::TILE / 16), k = k0 + (st ^ 1) * (S::TILE / 16);
            const bool more = i + 1 < nt;
            if (!full(st) || !step<0>(v, k, i > 0, more)) return false;
            if (both && !step<1>(v, k, i > 0, more)) return false;
            umma_commit(bar(S::B_EMPTY) + st * 8);
            p_par0 ^= 1;
            p_par1 ^= (uint32_t)both;
        }
        if ((nt & 1) == 0) {  // the empty pair
            if (!full(1)) return false;
            umma_commit(bar(S::B_EMPTY + 1));
        }
        return true;
    }
};

// ------------------------------------------------------------------ kernel ----
template <int D, bool BF>
__global__ void __launch_bounds__(CK_THREADS, 1)
paged_chunk_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v, const ChunkParams c) {
    using S = CkShape<D>;
    extern __shared__ __align__(1024) uint8_t sm[];  // swizzle atoms are 1024 bytes
    const PagedParams &p = c.p;
    const uint32_t base = smem_u32(sm);
    volatile int *words = reinterpret_cast<volatile int *>(sm + S::OFF_BAR + S::NBAR * 8);
    volatile int *s_piece = words;       // [2] the pieces handed on
    volatile int &s_abort = words[2];
    volatile int &s_loaded = words[4];   // pairs of tiles loaded so far
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, G = p.G;
    const uint32_t tries = p.st.wait_polls < CK_TRIES ? (uint32_t)p.st.wait_polls : CK_TRIES;
    auto bar = [&](int i) { return base + S::OFF_BAR + i * 8; };

    if (tid == 0) {
        for (int i = 0; i < S::NBAR; ++i)
            mbar_init(bar(i), (i < S::B_S || (i >= S::B_P && i < S::B_P + 4)) ? 4u : (i == S::B_FREE || i == S::B_FREE + 1) ? CK_RW + 1u : 1u);
        s_abort = s_loaded = 0;
        fence_mbar_init();
    }
    if (warp == CK_MMA) {
        tmem_alloc(base + S::OFF_BAR + S::NBAR * 8 + 12, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = (uint32_t)words[3];
    wait_for_primary();  // the plan, and the new tokens in their pages
    asm volatile("fence.proxy.async;" ::: "memory");  // which the tensor copies read
    const int pieces = c.head->pieces;
    auto wait1 = [&](int i, uint32_t par) -> bool {
        if (ck_wait(bar(i), par, tries)) return true;
        s_abort = 1;
        report(p.st, DEV_TIMEOUT);
        return false;
    };
    auto wait_warp = [&](int i, uint32_t par) -> bool {
        const bool ok = __all_sync(0xffffffffu, ck_wait(bar(i), par, tries));
        if (!ok) {
            s_abort = 1;
            report(p.st, DEV_TIMEOUT);
        }
        return ok;
    };
    auto arrive1 = [&](int i) { asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar(i)) : "memory"); };

    // The loader claims pieces and hands each on through two slots, so that it can run ahead:
    // it loads the next piece's keys while the rows of this one are being finished.
    // take(): the k-th piece (-1: no more); a warp is done with its slot once it has read it.
    // A tile without rows of its own waits here while the other one works on a piece, which may
    // take longer than a wait may: this one goes on for as long as something is loaded meanwhile.
    auto take = [&](uint32_t k) -> int {
        if (!__all_sync(0xffffffffu, ck_wait(bar(S::B_WORK + (k & 1)), (k >> 1) & 1, tries))) {
            int seen, now = 0;
            do {
                seen = now;
                now = s_loaded;
                if (!__any_sync(0xffffffffu, now != seen)) {
                    s_abort = 1;
                    report(p.st, DEV_TIMEOUT);
                    return -1;
                }
            } while (!__all_sync(0xffffffffu, ck_wait(bar(S::B_WORK + (k & 1)), (k >> 1) & 1, tries)));
        }
        const int at = s_piece[k & 1];
        __syncwarp();
        if (lane == 0) arrive1(S::B_FREE + (k & 1));
        return at;
    };

    if (warp >= CK_RW) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(CK_REGS_REST));
        if (warp == CK_LOAD) {
            // ------------------------------------------------ loader
            uint32_t g = 0, tails = 0;  // pairs begun, completions of B_TAIL
            bool ok = true;
            for (uint32_t w = 0; ok; ++w) {
                if (w >= 2 && !(ok = wait_warp(S::B_FREE + (w & 1), ((w >> 1) - 1) & 1))) break;
                int at = 0;
                if (lane == 0) {
                    at = atomicAdd(&c.head->ticket, 1);
                    if (at >= pieces || s_abort) at = -1;
                    s_piece[w & 1] = at;
                    arrive1(S::B_WORK + (w & 1));
                }
                at = __shfl_sync(0xffffffffu, at, 0);
                if (at < 0) break;
                const ChunkPiece pc = c.pieces[at];
                const PagedSeq sq = pc.s;
                const int kv_end = paged_kv_end(sq, G, (pc.t + 1) * CK_ROWS - 1);
                const int *trow = p.table + (long long)sq.row * p.P;
                const int box = min(p.page_size, CK_KT);  // tokens of one copy
                const int per_tile = CK_KT / box, per_page = p.page_size / box;  // copies of a tile, tiles of a page
                int pi = pc.kv0 / per_page * per_tile, tok0 = pc.kv0 % per_page * CK_KT;  // page and token the tile begins at
                // The row's page numbers, 32 at a time, a lane each, and the 32 after them: a table
                // entry read when its tile is due would cost its latency for every 128 keys.
                auto pages_at = [&](int i) { return trow[min(i + lane, p.P - 1)]; };
                int window = pi & ~31, cur = pages_at(window), next = pages_at(window + 32);
                const int cp = lane / (D / 64), kb = lane % (D / 64);  // a lane a copy and 64 channels
                const int put = kb * CK_KT * 128 + cp * box * 128;
                const int nt = pc.kv1 - pc.kv0;
                if (nt <= 0) continue;
                const int pairs = (nt + 2) & ~1;  // see Issuer
                int vpage = 0, vtok = 0, vcopies = 0, vvalid = 0;  // the keys' tile of the pair before, whose values come now
                for (int i = 0; ok && i < pairs; ++i, ++g) {
                    const int st = g & 1;
                    const int kt = pc.kv0 + i;
                    const int valid = i < nt ? max(0, min(CK_KT, kv_end - kt * CK_KT)) : 0;  // keys of the tile that some row sees
                    const int copies = (valid + box - 1) / box;
                    if (i < nt && (pi & ~31) != window) {
                        window += 32;
                        cur = next;
                        next = pages_at(window + 32);
                    }
                    int page = __shfl_sync(0xffffffffu, cur, (pi & 31) + cp);
                    if (cp < copies && (page < 0 || page >= p.num_pages)) { report(p.st, DEV_BAD_ARG); page = 0; }
                    if (g >= 2 && !(ok = wait_warp(S::B_EMPTY + st, ((g >> 1) - 1) & 1))) break;
                    // values behind the sequence's end become zeros before the products see them:
                    // such a tile is a piece's last, and comes with no keys
                    const bool tail = i > 0 && i <= nt && vvalid < CK_KT;
                    const int bi = tail ? S::B_TAIL : S::B_FULL + st;
                    if (lane == 0) mbar_expect_tx(bar(bi), (uint32_t)(vcopies + copies) * box * D * 2);
                    __syncwarp();
                    if (cp < vcopies) tma_load_4d(base + S::OFF_V + st * S::TILE + put, &tm_v, bar(bi), kb * 64, vtok, pc.h, vpage);
                    if (cp < copies) tma_load_4d(base + S::OFF_K + (st ^ 1) * S::TILE + put, &tm_k, bar(bi), kb * 64, tok0, pc.h, page);
                    if (tail) {
                        if (!(ok = wait_warp(S::B_TAIL, tails & 1))) {
                            // the values are on their way still: nothing is zeroed or handed on, and this
                            // memory stays the CTA's until they are here
                            if (lane == 0) mbar_wait(bar(S::B_TAIL), tails & 1, ~0ull, p.st);
                            __syncwarp();
                            break;
                        }
                        ++tails;
                        for (int k = lane; k < (CK_KT - vvalid) * (D / 64) * 8; k += 32) {
                            const int row = vvalid + k / (D / 64 * 8), b = k / 8 % (D / 64), ch = k % 8;
                            *reinterpret_cast<uint4 *>(sm + S::OFF_V + st * S::TILE + b * CK_KT * 128 + row * 128 + ch * 16) =
                                make_uint4(0u, 0u, 0u, 0u);
                        }
                        fence_async_smem();
                        __syncwarp();
                        if (lane == 0) arrive1(S::B_FULL + st);
                    }
                    if (lane == 0) s_loaded = (int)g + 1;
                    vpage = page;
                    vtok = tok0;
                    vcopies = copies;
                    vvalid = valid;
                    if (per_page == 1) pi += per_tile;
                    else if ((tok0 += CK_KT) == p.page_size) { tok0 = 0; ++pi; }
                }
            }
            // Leave no copy in flight into this CTA's memory.  This warp may have loaded all there is when another
            // one gives up, so it looks whether it has itself or not.
            if (lane == 0)
                for (uint32_t b = g >= 2 ? g - 2 : 0; b < g; ++b) mbar_wait(bar(S::B_FULL + (b & 1)), (b >> 1) & 1, ~0ull, p.st);
            __syncwarp();
        } else if (warp == CK_MMA) {
            // ------------------------------------------------ issuer (one lane issues)
            Issuer<D, BF> is = {base, tmem, tries};
            bool ok = true;
            for (uint32_t k = 0; ok; ++k) {
                const int at = take(k);
                if (at < 0) break;
                const ChunkPiece pc = c.pieces[at];
                const PagedSeq sq = pc.s;
                const int nt = pc.kv1 - pc.kv0;
                if (nt <= 0) continue;
                if (elect_lane()) ok = is.run(nt, ck_rows(sq, G, pc.t) > CK_M);
                __syncwarp();
                ok = __all_sync(0xffffffffu, ok);
            }
            if (!ok) {
                s_abort = 1;
                if (lane == 0) report(p.st, DEV_TIMEOUT);
            }
            // Leave no product in flight: the rows that wait for the last ones may give up after this warp is
            // done.  A commit tracks the products of the thread that it is made by, which is the one elected.
            if (elect_lane()) {
                umma_commit(bar(S::B_DRAIN));
                mbar_wait(bar(S::B_DRAIN), 0, ~0ull, p.st);
            }
            __syncwarp();
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(CK_REGS_ROWS));
        // ------------------------------------------------------------ rows: thread (w, r) owns one
        const int w = warp >> 2, r = (warp & 3) * 32 + lane;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t ts = tmem + lanes + S::TM_S + w * 128, to = tmem + lanes + S::TM_O + w * D;
        // weights are shifted up by SH; sums of 64 of them may reach 2^7 times the reference's own
        constexpr float SH = weight_shift<BF>(), MOST = BF ? 128.f : 32768.f;
        uint32_t s_phase = 0, h_phase = 0;  // completions of this tile's B_S, B_HALF
        bool ok = true;
        for (uint32_t kp = 0; ok; ++kp) {
            const int at = take(kp);
            if (at < 0) break;
            int nt, key0, last;     // key tiles; the first key; the last key that the row sees
            float m = -INFINITY;    // the row's reference, in the scores' units
            bool idle;              // the warp has no row: what its lanes of TMEM hold goes nowhere
            {
                const ChunkPiece pc = c.pieces[at];
                const PagedSeq sq = pc.s;
                const int rows = ck_rows(sq, G, pc.t), row = pc.t * CK_ROWS + w * CK_M + r, tok = row / G;
                nt = pc.kv1 - pc.kv0;
                if (nt <= 0 || (w == 1 && rows <= CK_M)) continue;
                idle = w * CK_M + (warp & 3) * 32 >= rows;
                const bool real = w * CK_M + r < rows && KDA_CHECK(p.st, sq.q0 + tok < p.total_q && pc.h < p.Hkv);
                key0 = pc.kv0 * CK_KT;
                last = sq.len - sq.nq + tok;
                if (!real) { last = 0x7ffffff0; m = 0.f; }  // no row: nothing to mask, a reference that never moves
                const uint4 *src = reinterpret_cast<const uint4 *>(
                    p.q + (real ? (sq.q0 + tok) * p.q_ts + (long long)(pc.h * G + row % G) * D : 0));
                uint4 x[D / 8];  // its query, to the swizzled tile
#pragma unroll
                for (int k = 0; k < D / 8; ++k) x[k] = real ? src[k] : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
                for (int k = 0; k < D / 8; ++k)
                    *reinterpret_cast<uint4 *>(sm + w * CK_M * D * 2 + kmaj<128, 2>(r, k * 8, CK_M)) = x[k];
                fence_async_smem();
                __syncwarp();
                if (lane == 0) arrive1(S::B_Q + w);
            }
            if (idle) {  // the products' turns, and nothing else
                for (int i = 0; i < nt && (ok = wait_warp(S::B_S + w, (s_phase + i) & 1)); ++i)
                    if (lane < 2) arrive1(S::B_P + w * 2 + lane);
                ok = ok && wait_warp(S::B_S + w, (s_phase + nt) & 1);
                s_phase += nt + 1;
                h_phase += nt;
                continue;
            }
            // the first step that some row of the warp does not see whole
            const int mask_from = __reduce_min_sync(0xffffffffu, last < key0 ? 0 : (last - key0 + 1) / CK_STEP);
            bool unset = true;  // some row has no reference yet
            float l = 0.f;
            const float sc = p.scale_log2;
            auto hand_on = [&](int h) {  // the products may begin on this half
                tm_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) arrive1(S::B_P + w * 2 + h);
            };
            for (int i = 0; i < nt; ++i) {
                if (!(ok = wait_warp(S::B_S + w, (s_phase + i) & 1))) break;
                tc_fence_after();
                // Both halves' weights lie over the first half's scores, which are read by then.
                // Unmasked keys: the weights with the reference there is, looked at afterwards, so that no
                // maximum stands between scores and weights.  A sum of the 64 up to MOST keeps every weight
                // there too; past it the half is done again below, from the scores still in TMEM.  Scores are
                // loaded 32 ahead (1.67 ms from 1.74) and weights handed on at once (1.75 ms with half 0's
                // store left in flight under the next 32 exponentials).
                int from = 0;  // the first half without weights
                if (2 * i + 1 < mask_from && !unset) {
                    uint32_t a[32], b[32], y[32], z[32];
                    const float ref = m * sc - SH;
                    tm_ld32(ts, a);
                    tm_wait_ld32(a);
                    tm_ld32(ts + 32, b);
                    float sum = ck_weights<BF, true>(a, y, sc, ref);
                    tm_wait_ld32(b);
                    tm_ld32(ts + 64, a);
                    sum += ck_weights<BF, true>(b, y + 16, sc, ref);
                    if (!__any_sync(0xffffffffu, sum > MOST)) {
                        tm_st32(ts, y);
                        l += sum;
                        from = 1;
                        hand_on(0);
                        tm_wait_ld32(a);
                        tm_ld32(ts + 96, b);
                        sum = ck_weights<BF, true>(a, z, sc, ref);
                        tm_wait_ld32(b);
                        sum += ck_weights<BF, true>(b, z + 16, sc, ref);
                        tm_st32(ts + 32, z);  // over scores of the half before: before the look at the sum, 1.5 % off
                        if (!__any_sync(0xffffffffu, sum > MOST)) {
                            l += sum;
                            from = 2;
                            hand_on(1);
                        }
                    } else {
                        tm_wait_ld32(a);  // nothing may land in registers that are others' by then
                    }
                }
#pragma unroll 1
                for (int h = from; h < 2; ++h) {
                    const int j = 2 * i + h;
                    const uint32_t sb = ts + h * CK_STEP, pb = ts + h * (CK_STEP / 2);
                    uint32_t x[CK_STEP], y[CK_STEP / 2];
                    tm_ld32(sb, x);
                    tm_ld32(sb + 32, x + 32);
                    tmem_wait_ld();
                    const int lim = last - key0 - j * CK_STEP;  // columns 0 .. lim are seen
                    float mx = -INFINITY;
#pragma unroll
                    for (int k = 0; k < CK_STEP; ++k) {
                        if (k > lim) x[k] = 0xff800000u;
                        mx = fmaxf(mx, __uint_as_float(x[k]));
                    }
                    // the row's first reference, or its next one where a weight would pass 2
                    const bool move = mx > -INFINITY && (m == -INFINITY || (mx - m) * sc > 1.f);
                    if (__any_sync(0xffffffffu, move)) {
                        const float f = move ? ex2((m - mx) * sc) : 1.f;  // 2^-inf = 0 at first
                        if (move) m = mx;
                        l *= f;
                        if (j > 0) {  // the products of earlier tiles are done, those of this one's first half have to be
                            if (h == 1) {
                                if (!(ok = wait_warp(S::B_HALF + w, (h_phase + i) & 1))) break;
                                tc_fence_after();
                            }
#pragma unroll 1
                            for (int k = 0; k < D; k += 16) {
                                float o[16];
                                uint32_t z[16];
                                tmem_ld16(to + k, o);
                                tmem_wait_ld();
#pragma unroll
                                for (int e = 0; e < 16; ++e) z[e] = __float_as_uint(o[e] * f);
                                tm_st16(to + k, z);
                            }
                        }
                    }
                    if (unset) unset = __any_sync(0xffffffffu, m == -INFINITY);
                    l += ck_weights<BF, false>(x, y, sc, (m == -INFINITY ? 0.f : m * sc) - SH);
                    tm_st32(pb, y);
                    hand_on(h);
                }
                if (!ok) break;
            }
            // the sums, after the last product
            if (ok && (ok = wait_warp(S::B_S + w, (s_phase + nt) & 1))) {
                tc_fence_after();
                const ChunkPiece pc = c.pieces[at];  // read again: the loop above needs the registers
                const PagedSeq sq = pc.s;
                const int row = w * CK_M + r, tok = (pc.t * CK_ROWS + row) / G, head = pc.h * G + (pc.t * CK_ROWS + row) % G;
                const bool whole = pc.part_row < 0;
                const bool real = row < ck_rows(sq, G, pc.t) && KDA_CHECK(p.st, sq.q0 + tok < p.total_q && head < p.Hq) &&
                                  KDA_CHECK(p.st, whole || pc.part_row + row < p.part_rows);
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
                    if (!whole) p.part_ml[pc.part_row + row] = make_float2(m == -INFINITY ? m : m * sc - SH, l);
                    else if (p.lse != nullptr)
                        p.lse[(long long)(sq.q0 + tok) * p.Hq + head] = row_lse(m * sc - SH, l);
                }
                tc_fence_before();
            }
            s_phase += nt + 1;
            h_phase += nt;
        }
        __syncwarp();
        tm_wait_st();  // weights that are done again, where the wait before that gave up
    }
    __syncwarp();
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
    cudaError_t e = allow_smem(paged_chunk_kernel<D, BF>, CkShape<D>::SMEM);
    if (e != cudaSuccess) return e;
    // one block plans; with new tokens to place, two an SM place them meanwhile
    const long long vecs = (long long)c.p.total_q * c.p.Hkv * (D / 8), blocks = (vecs + 511) / 512;
    const int more = c.p.k_new == nullptr ? 0 : (int)(blocks < 2LL * c.sms ? blocks : 2LL * c.sms);
    paged_plan_kernel<D><<<1 + more, 512, 0, stream>>>(c);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(c.max_pieces < c.sms ? c.max_pieces : c.sms);
    cfg.blockDim = dim3(CK_THREADS);
    cfg.dynamicSmemBytes = CkShape<D>::SMEM;
    cfg.stream = stream;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, paged_chunk_kernel<D, BF>, tk, tv, c);
}

// ws: the plan's part of the workspace: head (256 bytes), base [3][N], pieces.
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
    c.pieces = reinterpret_cast<ChunkPiece *>(reinterpret_cast<uint8_t *>(c.base) + ((size_t)p.N * 12 + 255) / 256 * 256);
    c.max_pieces = m.pieces;
    c.max_entries = m.entries;
    c.max_rows = m.rows;
    c.sms = sms;
    if (d == 128)
        return bf ? launch_chunk_t<128, true>(tk, tv, c, stream) : launch_chunk_t<128, false>(tk, tv, c, stream);
    return bf ? launch_chunk_t<64, true>(tk, tv, c, stream) : launch_chunk_t<64, false>(tk, tv, c, stream);
}

}  // namespace kda
