// pages.cu -- the pages of a cache: reserve, fork, free, compact, copy.
//
// A cache is one or more pools of num_pages pages, a table [R][P] of page
// numbers (row r holds the sequence in slot r, its first ceil(length[r] /
// page_size) entries in use, -1 behind them), length[R], and ref[num_pages],
// the number of rows that hold each page (0: free).
//
// Nothing here computes; each kernel's bound is the memory it touches, and for
// the small ones the latency of a few dependent reads.  Pages are handed out
// lowest number first, in the order of the caller's list, so results are the
// same whatever the timing.  A call whose list is bad (a row out of range, a
// row named twice, a length that shrinks or does not fit) changes nothing and is
// reported; so is a reservation for which there are too few pages, through its
// info word.
#include <cooperative_groups.h>
#include <stddef.h>

#include "kda_internal.cuh"
#include "pages_params.cuh"

namespace kda {

namespace cg = cooperative_groups;

constexpr int PG_THREADS = 1024, PG_WARPS = PG_THREADS / 32, PG_CLUSTER = 8;

// Exclusive prefix of v over the block, and the block's total.  sm: PG_WARPS + 1 ints.
__device__ __forceinline__ int block_prefix(int v, int *sm, int &total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += up;
    }
    __syncthreads();  // sm may still be read from the call before
    if (lane == 31) sm[warp] = incl;
    __syncthreads();
    if (warp == 0) {
        const int x = lane < (int)blockDim.x / 32 ? sm[lane] : 0;
        int y = x;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int up = __shfl_up_sync(0xffffffffu, y, o);
            if (lane >= o) y += up;
        }
        sm[lane] = y - x;
        if (lane == 31) sm[32] = y;
    }
    __syncthreads();
    total = sm[32];
    return sm[warp] + incl - v;
}

__device__ __forceinline__ int pages_of(int len, int ps) { return (int)(((long long)len + ps - 1) / ps); }
__device__ __forceinline__ bool length_ok(int len, int P, int ps) { return len >= 0 && pages_of(len, ps) <= P; }

// Marks rows[0..n) in the bitmap; false where one is out of range or marked already.
// Called by the whole block; needs a barrier before the bitmap is read.
__device__ __forceinline__ bool mark_rows(const int *rows, int n, int R, uint32_t *bits) {
    bool ok = true;
    for (int i = threadIdx.x; i < n; i += blockDim.x) {
        const int r = rows[i];
        if (r < 0 || r >= R) { ok = false; continue; }
        const uint32_t b = 1u << (r & 31);
        if (atomicOr(&bits[r >> 5], b) & b) ok = false;
    }
    return ok;
}

// ------------------------------------------------------------------- free ----
// Every block checks the whole list (a few reads a thread), then takes rows in
// turn: 256 entries at a time, so a row of 750 pages costs three round trips to
// the counts (a warp a row took 24: 15.7 us for 200 rows, from 7).
__global__ void __launch_bounds__(256) pages_free_kernel(const PagesParams p) {
    __shared__ uint32_t bits[PG_MAX_ROWS / 32];
    wait_for_primary();
    for (int i = threadIdx.x; i < (p.R + 31) / 32; i += blockDim.x) bits[i] = 0;
    __syncthreads();
    const bool ok = mark_rows(p.rows, p.n, p.R, bits);
    if (__syncthreads_or(!ok)) {
        if (threadIdx.x == 0) report(p.st, DEV_BAD_ARG);
        return;
    }
    for (int i = blockIdx.x; i < p.n; i += gridDim.x) {
        const int row = p.rows[i];
        int *tr = p.table + (long long)row * p.P;
        const int len = p.length[row], held = min(pages_of(max(len, 0), p.ps), p.P);
        if (threadIdx.x == 0 && !length_ok(len, p.P, p.ps)) report(p.st, DEV_BAD_ARG);
        for (int j = threadIdx.x; j < held; j += blockDim.x) {
            const int page = tr[j];
            tr[j] = -1;
            if (page < 0 || page >= p.num_pages) { report(p.st, DEV_BAD_ARG); continue; }
            if (atomicSub(&p.ref[page], 1) <= 0) {  // held by nobody: the count stays at zero
                atomicAdd(&p.ref[page], 1);
                report(p.st, DEV_BAD_ARG);
            }
        }
        __syncthreads();  // every thread has read the length
        if (threadIdx.x == 0) p.length[row] = 0;
    }
}

// -------------------------------------------------------- reserve and fork ----
// One cluster of eight CTAs, one launch: every CTA checks the list and sums the
// pages that its sequences need, each counts the free pages of its eighth of
// ref, the counts meet over distributed shared memory, and each hands out the
// free pages of its own eighth: the f-th free page goes to the sequence whose
// needs cover rank f.  A second pass over ref hands out; up to 262,144 pages it
// has the first one's flags in registers (1.4 us of a turnover of 200 rows).
struct GrantShared {
    int sm[33];
    uint32_t bits[PG_MAX_ROWS / 32];
    int warp_free[PG_WARPS];
    int cta_free;
    int found[PG_WARPS][128];    // a step's free pages, in order
    int start[PG_MAX_LIST + 1];  // exclusive prefix of the sequences' needs
    int row[PG_MAX_LIST];        // their rows
    int held[PG_MAX_LIST];       // entries that the rows hold before (a fork's: full pages of the source)
};
// what of it a list of n needs
__host__ __device__ constexpr size_t grant_bytes(int n) { return offsetof(GrantShared, start) + sizeof(int) * (3 * (size_t)n + 1); }

// Free flags of pages [4 i, 4 i + 4).
__device__ __forceinline__ uint32_t free_nibble(const int *ref, int num_pages, int i) {
    uint32_t m = 0;
    if (4 * i + 3 < num_pages && (reinterpret_cast<uintptr_t>(ref) & 15u) == 0) {
        const int4 x = *reinterpret_cast<const int4 *>(ref + 4 * i);
        m = (x.x == 0) | (x.y == 0) << 1 | (x.z == 0) << 2 | (x.w == 0) << 3;
    } else {
        for (int k = 0; k < 4; ++k)
            if (4 * i + k < num_pages && ref[4 * i + k] == 0) m |= 1u << k;
    }
    return m;
}

template <bool FORK>
__global__ void __cluster_dims__(PG_CLUSTER, 1, 1) __launch_bounds__(PG_THREADS) pages_grant_kernel(const PagesParams p) {
    extern __shared__ __align__(16) uint8_t raw[];
    GrantShared &s = *reinterpret_cast<GrantShared *>(raw);
    int *s_start = s.start, *s_row = s.start + p.n + 1, *s_held = s_row + p.n;  // packed for n
    cg::cluster_group cluster = cg::this_cluster();
    const int cta = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    wait_for_primary();
    // ---- the list: rows in range and named once; what each needs
    for (int i = tid; i < (p.R + 31) / 32; i += PG_THREADS) s.bits[i] = 0;
    __syncthreads();
    bool ok = mark_rows(p.rows, p.n, p.R, s.bits);
    __syncthreads();
    int total = 0;
    for (int base = 0; base < p.n; base += PG_THREADS) {
        const int i = base + tid;
        int need = 0, held = 0;
        if (i < p.n) {
            const int row = p.rows[i];
            s_row[i] = row;
            if (row >= 0 && row < p.R) {
                const int have = p.length[row];
                if constexpr (FORK) {
                    const int from = p.src[i];
                    if (from < 0 || from >= p.R || (s.bits[from >> 5] >> (from & 31) & 1u) || have != 0) {
                        ok = false;
                    } else {
                        const int len = p.length[from];
                        if (!length_ok(len, p.P, p.ps)) ok = false;
                        else { need = len % p.ps != 0; held = len / p.ps; }
                    }
                } else {
                    const int want = p.new_length[i];
                    if (have < 0 || want < have || pages_of(want, p.ps) > p.P) ok = false;
                    else { held = pages_of(have, p.ps); need = pages_of(want, p.ps) - held; }
                }
            }
        }
        int sum;
        const int at = block_prefix(need, s.sm, sum);
        if (i < p.n) { s_start[i] = total + at; s_held[i] = held; }
        total += sum;  // at most the table's entries, which the host holds below 2^31
    }
    if (tid == 0) s_start[p.n] = total;
    auto no_copies = [&]() {
        if constexpr (FORK)
            for (int i = cta * PG_THREADS + tid; i < p.n; i += PG_CLUSTER * PG_THREADS) p.copy_src[i] = p.copy_dst[i] = -1;
    };
    if (__syncthreads_or(!ok)) {  // the same in every CTA: all return before the cluster's barrier
        if (tid == 0 && cta == 0) report(p.st, DEV_BAD_ARG);
        no_copies();
        return;
    }

    // ---- free pages of this CTA's eighth, a warp a contiguous run of 128-page steps
    const int steps = (p.num_pages + 127) / 128, warps = PG_CLUSTER * PG_WARPS, gw = cta * PG_WARPS + warp;
    const int s0 = (int)((long long)steps * gw / warps), s1 = (int)((long long)steps * (gw + 1) / warps);
    int cnt = 0;
    uint32_t kept = 0;  // the first eight steps' flags (262,144 pages), for the second pass
#pragma unroll
    for (int k = 0; k < 8; ++k)
        if (s0 + k < s1) kept |= free_nibble(p.ref, p.num_pages, (s0 + k) * 32 + lane) << 4 * k;
    cnt = __popc(kept);
#pragma unroll 8
    for (int k = s0 + 8; k < s1; ++k) cnt += __popc(free_nibble(p.ref, p.num_pages, k * 32 + lane));
    cnt = __reduce_add_sync(0xffffffffu, cnt);
    if (lane == 0) s.warp_free[warp] = cnt;
    __syncthreads();
    if (warp == 0) {
        const int x = s.warp_free[lane];
        int y = x;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int up = __shfl_up_sync(0xffffffffu, y, o);
            if (lane >= o) y += up;
        }
        s.warp_free[lane] = y - x;
        if (lane == 31) s.cta_free = y;
    }
    cluster.sync();
    int rank = s.warp_free[warp], free_all = 0;
    for (int r = 0; r < PG_CLUSTER; ++r) {
        const int f = *cluster.map_shared_rank(&s.cta_free, r);
        if (r < cta) rank += f;
        free_all += f;
    }
    cluster.sync();  // no CTA leaves while its count is read; every read of length, and the count of ref, is done
    const bool fits = free_all >= total;
    if (cta == 0 && tid == 0 && p.info != nullptr) *p.info = free_all - total;  // negative: pages missing
    if (!fits) {
        no_copies();
        return;
    }

    // ---- the free pages of ranks below `total` go to their sequences.  A step's are listed, then a lane takes
    // one, so that a warp's stores lie together; ranks only grow, so a lane goes on from the sequence that it
    // served last and searches only past two of them (11,800 pages of one CTA's eighth, with the free before it: 18.9
    // us; with a search a page 23.5, with a lane's own four pages and a search for them 23.3: one SM's stores).
    int lo = 0;  // the last sequence with start <= f
    for (int k = s0; k < s1 && rank < total; ++k) {
        const uint32_t m = k - s0 < 8 ? kept >> 4 * (k - s0) & 15u : free_nibble(p.ref, p.num_pages, k * 32 + lane);
        const int c = __popc(m);
        int incl = c;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int up = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += up;
        }
        const int all = __shfl_sync(0xffffffffu, incl, 31);
        for (int b = 0, at = incl - c; b < 4; ++b)
            if (m >> b & 1u) s.found[warp][at++] = (k * 32 + lane) * 4 + b;
        __syncwarp();
        for (int q = lane; q < all && rank + q < total; q += 32) {
            const int f = rank + q, page = s.found[warp][q];
            if (s_start[lo + 1] <= f && s_start[++lo + 1] <= f && s_start[++lo + 1] <= f) {  // s_start[n] = total > f
                int hi = p.n - 1;
                ++lo;
                while (lo < hi) {
                    const int mid = (lo + hi + 1) / 2;
                    if (s_start[mid] <= f) lo = mid; else hi = mid - 1;
                }
            }
            // its entries so far come first
            if (!KDA_CHECK(p.st, lo < p.n && s_held[lo] + f - s_start[lo] < p.P && page < p.num_pages)) continue;
            p.table[(long long)s_row[lo] * p.P + s_held[lo] + f - s_start[lo]] = page;
            p.ref[page] = 1;
            if constexpr (FORK) {
                const int came = p.table[(long long)p.src[lo] * p.P + s_held[lo]];
                if (came < 0 || came >= p.num_pages) report(p.st, DEV_BAD_ARG);
                p.copy_src[lo] = came;
                p.copy_dst[lo] = page;
            }
        }
        rank += all;
        __syncwarp();
    }
    if constexpr (!FORK) {
        for (int i = cta * PG_THREADS + tid; i < p.n; i += PG_CLUSTER * PG_THREADS) p.length[p.rows[i]] = p.new_length[i];
    } else {
        // the full pages, shared: the warps share out the branches
        const int each = max(1, warps / max(1, p.n));  // warps of a branch
        for (int v = gw; v < p.n * each; v += warps) {
            const int i = v / each, sub = v % each, full = s_held[i], len = p.length[p.src[i]];
            const int *a = p.table + (long long)p.src[i] * p.P;
            int *b = p.table + (long long)s_row[i] * p.P;
            for (int j = sub * 32 + lane; j < full; j += each * 32) {
                const int page = a[j];
                b[j] = page;
                if (page >= 0 && page < p.num_pages) atomicAdd(&p.ref[page], 1);
                else report(p.st, DEV_BAD_ARG);
            }
            if (lane == 0 && sub == 0) {
                p.length[s_row[i]] = len;
                if (len % p.ps == 0) p.copy_src[i] = p.copy_dst[i] = -1;
            }
        }
    }
}

// ---------------------------------------------------------------- compact ----
// With n live pages, the i-th free page below n (a hole) takes the i-th live
// page at or above n, both in ascending order: the fewest moves, and no page is
// both read and written.  Three launches over ref (one for a small cache): counts of blocks of pages;
// ranks of holes and of pages to move; the table, ref and info.  The pools'
// pages move in pages_copy_kernel.
constexpr int CP_BLOCK = 4096, CP_THREADS = 1024;

__global__ void __launch_bounds__(CP_THREADS) compact_count_kernel(const PagesParams p) {
    wait_for_primary();
    const int i = blockIdx.x * CP_THREADS + threadIdx.x;
    const int dead = __popc(free_nibble(p.ref, p.num_pages, i));
    const int in = min(4, max(0, p.num_pages - 4 * i));
    __shared__ int sm[33];
    int total;
    block_prefix(in - dead, sm, total);
    if (threadIdx.x == 0) p.ws_counts[blockIdx.x] = total;
}

__global__ void __launch_bounds__(CP_THREADS) compact_rank_kernel(const PagesParams p, int blocks) {
    __shared__ int sm[33];
    const int tid = threadIdx.x;
    wait_for_primary();
    // live pages in all, before this block, and in the blocks before the one that page n lies in
    int mine = 0, before = 0;
    for (int b = tid; b < blocks; b += CP_THREADS) {
        const int c = p.ws_counts[b];
        mine += c;
        if (b < (int)blockIdx.x) before += c;
    }
    int n, lp0, below;
    block_prefix(mine, sm, n);
    block_prefix(before, sm, lp0);
    const int edge = n / CP_BLOCK;
    int x = 0;
    for (int b = tid; b < min(edge, blocks); b += CP_THREADS) x += p.ws_counts[b];
    for (int q = edge * CP_BLOCK + tid; q < n; q += CP_THREADS) x += p.ref[q] != 0;
    block_prefix(x, sm, below);  // live pages below n
    const int i = blockIdx.x * CP_THREADS + tid;
    const int in = min(4, max(0, p.num_pages - 4 * i));
    const uint32_t dead = free_nibble(p.ref, p.num_pages, i);
    int total;
    int lp = lp0 + block_prefix(in - __popc(dead), sm, total);
    for (int k = 0; k < in; ++k) {
        const int q = 4 * i + k;
        const bool live = !(dead >> k & 1u);
        if (q < n && !live && KDA_CHECK(p.st, q >= lp)) p.ws_hole[q - lp] = q;
        if (q >= n && live && KDA_CHECK(p.st, lp >= below)) {
            p.ws_move[lp - below] = q;
            p.ws_rank[q] = lp - below;
        }
        lp += live;
    }
    if (blockIdx.x == 0 && tid == 0) {
        p.ws_n[0] = n;
        p.ws_n[1] = n - below;  // pages to move
        if (p.info != nullptr) *p.info = p.num_pages - n;
    }
}

// Table, ref and the moved pages' counts, by `all` threads of which this is `me`.
__device__ __forceinline__ void compact_apply(const PagesParams &p, int n, int moves, long long me, long long all) {
    for (long long i = me; i < p.num_pages; i += all) {
        // below n: a hole's new count comes from the page that moves in; above: a moved page's old count is read first
        const int v = p.ref[i];
        if (i < n ? v != 0 : v == 0) p.ref_out[i] = i < n ? v : 0;
    }
    for (long long i = me; i < moves; i += all) {
        const int from = p.ws_move[i], to = p.ws_hole[i];
        if (!KDA_CHECK(p.st, from >= 0 && from < p.num_pages && to >= 0 && to < n)) continue;
        p.ref_out[to] = p.ref[from];
        p.ref_out[from] = 0;
    }
    for (long long i = me; i < (long long)p.R * p.P; i += all) {
        const int row = (int)(i / p.P), j = (int)(i % p.P);
        const int page = p.table[i];
        int to = page;
        const int len = p.length[row];
        if (j == 0 && !length_ok(len, p.P, p.ps)) report(p.st, DEV_BAD_ARG);
        if (len > 0 && j < pages_of(len, p.ps)) {
            if (page < 0 || page >= p.num_pages) report(p.st, DEV_BAD_ARG);
            else if (page >= n) {
                const int r = p.ws_rank[page];
                // a page that the table holds but ref does not count has no place to go
                if (r >= 0 && r < moves && p.ws_move[r] == page) to = p.ws_hole[r];
                else report(p.st, DEV_BAD_ARG);
            }
        }
        if (to != page || p.table_out != p.table) p.table_out[i] = to;
    }
}

__global__ void __launch_bounds__(256) compact_apply_kernel(const PagesParams p) {
    wait_for_primary();
    compact_apply(p, p.ws_n[0], p.ws_n[1], (long long)blockIdx.x * blockDim.x + threadIdx.x, (long long)gridDim.x * blockDim.x);
}

// All three in one launch for a small cache, by a cluster of eight CTAs: counts meet over
// distributed shared memory, lists through memory.
__global__ void __cluster_dims__(PG_CLUSTER, 1, 1) __launch_bounds__(PG_THREADS) compact_small_kernel(const PagesParams p) {
    __shared__ int warp_live[PG_WARPS], warp_below[PG_WARPS], cta_live, cta_below;
    cg::cluster_group cluster = cg::this_cluster();
    const int cta = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    wait_for_primary();
    // a warp a contiguous run of 128-page steps, as in pages_grant_kernel
    const int steps = (p.num_pages + 127) / 128, warps = PG_CLUSTER * PG_WARPS, gw = cta * PG_WARPS + warp;
    const int s0 = (int)((long long)steps * gw / warps), s1 = (int)((long long)steps * (gw + 1) / warps);
    auto live = [&](int k) {  // live flags of pages [4 i, 4 i + 4), i = 32 k + lane
        const int i = k * 32 + lane, in = min(4, max(0, p.num_pages - 4 * i));
        return ~free_nibble(p.ref, p.num_pages, i) & ((1u << in) - 1u);
    };
    int cnt = 0;
    for (int k = s0; k < s1; ++k) cnt += __popc(live(k));
    cnt = __reduce_add_sync(0xffffffffu, cnt);
    if (lane == 0) warp_live[warp] = cnt;
    __syncthreads();
    int lp = 0;  // live pages before this warp's
    if (tid == 0) {
        int x = 0;
        for (int w = 0; w < PG_WARPS; ++w) x += warp_live[w];
        cta_live = x;
    }
    for (int w = 0; w < warp; ++w) lp += warp_live[w];
    cluster.sync();
    int n = 0;
    for (int r = 0; r < PG_CLUSTER; ++r) {
        const int x = *cluster.map_shared_rank(&cta_live, r);
        if (r < cta) lp += x;
        n += x;
    }
    // live pages below n
    int below = 0;
    for (int k = s0; k < s1 && k * 128 < n; ++k) {
        const int in = min(4, max(0, n - 4 * (k * 32 + lane)));
        below += __popc(live(k) & ((1u << in) - 1u));
    }
    below = __reduce_add_sync(0xffffffffu, below);
    if (lane == 0) warp_below[warp] = below;
    __syncthreads();
    if (tid == 0) {
        int x = 0;
        for (int w = 0; w < PG_WARPS; ++w) x += warp_below[w];
        cta_below = x;
    }
    cluster.sync();
    below = 0;
    for (int r = 0; r < PG_CLUSTER; ++r) below += *cluster.map_shared_rank(&cta_below, r);
    for (int k = s0; k < s1; ++k) {
        const uint32_t m = live(k);
        int incl = __popc(m);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int up = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += up;
        }
        int at = lp + incl - __popc(m);
        for (int b = 0; b < 4; ++b) {
            const int q = (k * 32 + lane) * 4 + b;
            const bool is = m >> b & 1u;
            if (q < n && !is && KDA_CHECK(p.st, q >= at)) p.ws_hole[q - at] = q;
            if (q >= n && is && KDA_CHECK(p.st, at >= below)) {
                p.ws_move[at - below] = q;
                p.ws_rank[q] = at - below;
            }
            at += is;
        }
        lp += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (cta == 0 && tid == 0) {
        p.ws_n[0] = n;
        p.ws_n[1] = n - below;
        if (p.info != nullptr) *p.info = p.num_pages - n;
    }
    cluster.sync();  // the lists are written, and nobody's counts are read any more
    compact_apply(p, n, n - below, cta * PG_THREADS + tid, PG_CLUSTER * PG_THREADS);
}

// ------------------------------------------------------------------- copy ----
// pool[o][dst[i]] = pool[o][src[i]] for every pair and outer index, in units of
// at most 64 KB: 256 threads with sixteen 16-byte loads in flight each, then the
// stores.  128 pages of 32 x 131 KB take 173 us (6.2 TB/s moved, 95 % of the
// card's copy rate), from 188, 184 and 176 us with units of 8, 16 and 32 KB; cache
// hints for data read and written once (187 us at 16 KB) and half the blocks (187
// us at 32 KB) were slower.  Where that is more than an SM's share units are
// halved, to 8 KB at least (a 256 KB state: 2.9 us from 3.7; 33 MB in units of 8 KB
// took 9 us longer than in 64).  A pair whose destination the list names elsewhere too
// (as a destination or as a source) is not copied: the others read what was there
// before the call.
//
// Whether a destination is named elsewhere takes a look through the list.  Blocks
// with few pairs look once a pair; with more than COPY_EACH of them a block looks once
// for up to COPY_BATCH, their destinations in a hash table in shared memory, so that
// the work grows with the list and not with its square (once a pair / by batches, us,
// pages of 4 KB: 2600 pairs 20 / 30, 5000 pairs 38 / 48, 8192 pairs 58 / 69, 16,384
// pairs 176 / 153, 65,536 pairs 3340 / 680; tables of half the size 155 and 715).
constexpr int COPY_THREADS = 256, COPY_VECS = 16, COPY_UNIT = COPY_THREADS * COPY_VECS * 16;
constexpr int COPY_EACH = 8;
enum { CHECK_NONE, CHECK_EACH, CHECK_BATCH };  // a compaction's pairs need none
constexpr int COPY_BATCH = 1024, COPY_SLOT_BITS = 11, COPY_SLOTS = 1 << COPY_SLOT_BITS;

// Destinations, and how often the list names them: open addressing, at most half full.
struct NamedPages {
    int page[COPY_SLOTS], times[COPY_SLOTS];

    // the page's slot, or the empty one where it would go
    __device__ __forceinline__ int slot(int q) const {
        int at = (int)((uint32_t)q * 0x9e3779b1u >> (32 - COPY_SLOT_BITS));  // by the golden ratio: neighbours part
        while (page[at] != q && page[at] != -1) at = (at + 1) & (COPY_SLOTS - 1);
        return at;
    }
    // by the whole block: the destinations of pairs [i0, i1) and their count in the list
    __device__ void fill(const PoolParams &p, int n, int i0, int i1) {
        __syncthreads();  // the batch before may still be read
        for (int k = threadIdx.x; k < COPY_SLOTS; k += COPY_THREADS) {
            page[k] = -1;
            times[k] = 0;
        }
        __syncthreads();
        for (int i = i0 + threadIdx.x; i < i1; i += COPY_THREADS) {
            const int q = p.dst[i];
            if (q < 0 || q >= p.num_pages || p.src[i] == q) continue;  // not copied
            int at = (int)((uint32_t)q * 0x9e3779b1u >> (32 - COPY_SLOT_BITS));
            for (;;) {
                const int was = atomicCAS(&page[at], -1, q);
                if (was == -1 || was == q) break;
                at = (at + 1) & (COPY_SLOTS - 1);
            }
        }
        __syncthreads();
        constexpr int V = 4;
        for (int j0 = threadIdx.x; j0 < n; j0 += V * COPY_THREADS) {
            int q[2 * V];
#pragma unroll
            for (int k = 0; k < V; ++k) {
                const int j = j0 + k * COPY_THREADS;
                q[2 * k] = j < n ? p.dst[j] : -1;
                q[2 * k + 1] = j < n ? p.src[j] : -1;
            }
#pragma unroll
            for (int k = 0; k < 2 * V; ++k) {
                if (q[k] < 0) continue;
                const int at = slot(q[k]);
                if (page[at] == q[k]) atomicAdd(&times[at], 1);
            }
        }
        __syncthreads();
    }
};

template <int CHECK>
__global__ void __launch_bounds__(COPY_THREADS) pages_copy_kernel(const PoolParams p) {
    __shared__ NamedPages named;  // CHECK_BATCH only
    wait_for_primary();
    const int n = p.count != nullptr ? min(max(*p.count, 0), p.n) : p.n;
    const long long per_page = (p.page_bytes + p.unit - 1) / p.unit, per_pair = per_page * p.outer;
    const long long units = n * per_pair;
    const long long u0 = units * blockIdx.x / gridDim.x, u1 = units * (blockIdx.x + 1) / gridDim.x;
    int pair = -1, from = 0, to = 0;
    bool ok = false;
    const int first = (int)(u0 / per_pair), last = u1 > u0 ? (int)((u1 - 1) / per_pair) : first;
    for (long long u = u0; u < u1; ++u) {
        const int i = (int)(u / per_pair);
        if (i != pair) {
            pair = i;
            from = p.src[i];
            to = p.dst[i];
            ok = from >= 0 && from < p.num_pages && to >= 0 && to < p.num_pages;
            bool bad = !ok && !(from == -1 && to == -1);
            bool twice = false;
            if constexpr (CHECK == CHECK_EACH) {
                if (ok && from != to) {
                    for (int j = threadIdx.x; j < n; j += COPY_THREADS) {
                        const int a = p.dst[j], b = p.src[j];
                        twice |= j != i && (a == to || b == to);
                    }
                    twice = __syncthreads_or(twice);
                }
            } else if constexpr (CHECK == CHECK_BATCH) {
                if ((i - first) % COPY_BATCH == 0) named.fill(p, n, i, min(i + COPY_BATCH, last + 1));
                if (ok && from != to) twice = named.times[named.slot(to)] > 1;  // once by the pair itself
            }
            if (twice) { ok = false; bad = true; }
            if (bad && threadIdx.x == 0) report(p.st, DEV_BAD_ARG);
        }
        if (!ok || from == to) continue;
        const long long in_pair = u % per_pair, o = in_pair / per_page, at = (in_pair % per_page) * p.unit;
        const int vecs = (int)(min((long long)p.unit, p.page_bytes - at) / 16);
        const uint8_t *base = p.pool + o * p.outer_stride + at;
        const uint4 *a = reinterpret_cast<const uint4 *>(base + from * p.page_stride);
        uint4 *b = reinterpret_cast<uint4 *>(const_cast<uint8_t *>(base) + to * p.page_stride);
        uint4 x[COPY_VECS];
        if (vecs == COPY_UNIT / 16) {
#pragma unroll
            for (int k = 0; k < COPY_VECS; ++k) x[k] = a[k * COPY_THREADS + threadIdx.x];
#pragma unroll
            for (int k = 0; k < COPY_VECS; ++k) b[k * COPY_THREADS + threadIdx.x] = x[k];
        } else {
#pragma unroll
            for (int k = 0; k < COPY_VECS; ++k)
                if (k * COPY_THREADS + threadIdx.x < vecs) x[k] = a[k * COPY_THREADS + threadIdx.x];
#pragma unroll
            for (int k = 0; k < COPY_VECS; ++k)
                if (k * COPY_THREADS + threadIdx.x < vecs) b[k * COPY_THREADS + threadIdx.x] = x[k];
        }
    }
}

// ------------------------------------------------------------------- host ----
// Every kernel here is launched so that its blocks may be in place when the one
// before it ends (each waits for that end first): a fork's three launches on
// small lists are mostly launches.
template <class K, class... A>
static cudaError_t launch_behind(K *kernel, dim3 grid, int threads, size_t smem, cudaStream_t stream, const A &...args) {
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

cudaError_t launch_pages_free(const PagesParams &p, int sms, cudaStream_t stream) {
    return launch_behind(pages_free_kernel, dim3(p.n < 8 * sms ? p.n : 8 * sms), 256, 0, stream, p);
}
cudaError_t launch_pages_grant(const PagesParams &p, bool fork, cudaStream_t stream) {
    auto *k = fork ? pages_grant_kernel<true> : pages_grant_kernel<false>;
    const size_t smem = grant_bytes(p.n);
    if (smem > 48 * 1024) {
        const cudaError_t e = fork ? allow_smem(pages_grant_kernel<true>, (int)grant_bytes(PG_MAX_LIST))
                                   : allow_smem(pages_grant_kernel<false>, (int)grant_bytes(PG_MAX_LIST));
        if (e != cudaSuccess) return e;
    }
    return launch_behind(k, dim3(PG_CLUSTER), PG_THREADS, smem, stream, p);
}
int compact_blocks(int num_pages) { return (num_pages + CP_BLOCK - 1) / CP_BLOCK; }
// Pages and table entries up to which one launch compacts: one launch / three, for 300 pages and 1024 entries
// 5.9 / 6.8 us, 16,384 of each 9.2 / 8.7 us, 65,536 of each 17.0 / 9.7 us, and for the host two launches
// (4 us of 20) less.
constexpr int COMPACT_SMALL = 16384;
cudaError_t launch_pages_compact(const PagesParams &p, int sms, cudaStream_t stream) {
    if (p.num_pages <= COMPACT_SMALL && (long long)p.R * p.P <= COMPACT_SMALL)
        return launch_behind(compact_small_kernel, dim3(PG_CLUSTER), PG_THREADS, 0, stream, p);
    const int blocks = compact_blocks(p.num_pages);
    cudaError_t e = launch_behind(compact_count_kernel, dim3(blocks), CP_THREADS, 0, stream, p);
    if (e == cudaSuccess) e = launch_behind(compact_rank_kernel, dim3(blocks), CP_THREADS, 0, stream, p, blocks);
    if (e != cudaSuccess) return e;
    const long long want = ((long long)p.R * p.P + 255) / 256, want2 = (p.num_pages + 255) / 256, top = 8LL * sms;
    const long long grid = want > want2 ? want : want2;
    return launch_behind(compact_apply_kernel, dim3((unsigned)(grid < top ? grid : top)), 256, 0, stream, p);
}
cudaError_t launch_pages_copy(PoolParams p, bool check, int sms, cudaStream_t stream) {
    const double each = (double)p.page_bytes * p.outer * p.n / sms;  // bytes an SM
    for (p.unit = COPY_UNIT; p.unit > COPY_UNIT / 8 && p.unit > each; p.unit /= 2) {}
    const long long units = (p.page_bytes + p.unit - 1) / p.unit * p.outer * p.n, top = 8LL * sms;
    const unsigned grid = (unsigned)(units < top ? units : top);
    auto *kernel = !check ? pages_copy_kernel<CHECK_NONE>
                   : p.n > (long long)COPY_EACH * grid ? pages_copy_kernel<CHECK_BATCH> : pages_copy_kernel<CHECK_EACH>;
    return launch_behind(kernel, dim3(grid), COPY_THREADS, 0, stream, p);
}

}  // namespace kda
