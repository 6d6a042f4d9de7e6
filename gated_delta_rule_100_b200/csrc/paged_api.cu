// paged_api.cu -- the extern "C" boundary of the paged cache: argument checks,
// workspace layout, the choice of kernel, launches.  Contracts in include/kda.h.
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "../../include/kda.h"
#include "kda_internal.cuh"
#include "paged_params.cuh"
#include "pages_params.cuh"

namespace kda {
int paged_rows_slots(int ctas);
int paged_rows_ctas_per_sm(int d);
int paged_rows_tile();
cudaError_t launch_paged_rows(const PagedParams &p, int d, bool bf, bool whole, int ctas, cudaStream_t stream);
cudaError_t launch_paged_join(const PagedParams &p, int d, bool bf, const int *count, int max_entries, int tile_rows, int sms,
                              cudaStream_t stream);
int paged_chunk_tile();
bool paged_chunk_pages(int page_size);
ChunkLimits paged_chunk_limits(int N, int total_q, int G, int Hkv, int span, int sms);
size_t paged_chunk_piece_bytes();
cudaError_t launch_paged_chunk(const PagedParams &p, const ChunkLimits &m, void *ws, int d, bool bf, int sms, cudaStream_t stream);
cudaError_t launch_pages_free(const PagesParams &p, int sms, cudaStream_t stream);
cudaError_t launch_pages_grant(const PagesParams &p, bool fork, cudaStream_t stream);
int compact_blocks(int num_pages);
cudaError_t launch_pages_compact(const PagesParams &p, int sms, cudaStream_t stream);
cudaError_t launch_pages_copy(PoolParams p, bool check, int sms, cudaStream_t stream);
}  // namespace kda

namespace {

bool al(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
size_t up256(size_t x) { return (x + 255) & ~size_t(255); }
int device() {
    int dev = 0;
    return cudaGetDevice(&dev) == cudaSuccess ? dev : 0;
}
int to_status(cudaError_t e) { return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA; }

// Whether cells of `width`, extent[i] of them stride[i] apart along axis i, lie clear of one
// another: along the axes by stride, each step leads past all that the axes before it reach.
// (Layouts that mesh without that, such as steps of 2 and 3 cells, count as overlapping.)
template <int N>
bool apart(const long long (&stride)[N], const long long (&extent)[N], long long width) {
    int order[N];
    for (int i = 0; i < N; ++i) order[i] = i;
    std::sort(order, order + N, [&](int a, int b) { return stride[a] < stride[b]; });
    __int128 reach = width;
    for (const int i : order) {
        if (extent[i] < 2) continue;
        if (stride[i] < reach) return false;
        reach += (__int128)(extent[i] - 1) * stride[i];
    }
    return true;
}

// ------------------------------------------------------------- attention ----
// Sizes that paged attention takes at all (0: yes).
int attn_sizes(int N, int total_q, int max_q, int Hq, int Hkv, int d, int page_size, int P) {
    if (N < 1 || total_q < 0 || max_q < 0 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || page_size < 1 || P < 1)
        return KDA_ERR_INVALID_ARG;
    if (total_q > 0 && max_q < 1) return KDA_ERR_INVALID_ARG;
    if (d != 64 && d != 128) return KDA_ERR_UNSUPPORTED;
    if (N > (1 << 22) || (long long)P * page_size > 0x7ffff000LL || (long long)total_q * Hq > 0x7ffff000LL)
        return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

// The kernel of few rows runs up to kFewRows rows of a sequence and key head (new tokens times
// query heads), and where there are at most kFewUnits 64-key units a CTA, as many as the sizes
// allow; the chunk kernel otherwise.  Few rows are bound by memory and want many CTAs' loads; the
// chunk kernel's tiles are 128 rows whatever there is, and its plan, pieces and join take some 12 us.
// The units are those that the table has room for, as the host reads no lengths: with a table wider
// than its sequences the chunk kernel comes sooner.  Every figure by units below is for a table as wide
// as the keys; for 131,072 keys a row they are the chunk kernel's (100 over 3000 26 -> 33 us, 64 over
// 4000 17 -> 27, 256 over 1024 20 -> 25).  Page sizes that it cannot load (paged_chunk_pages) stay with few
// rows whatever there is: 2048 tokens over 16,384 keys take 3.7 ms on pages of 48 or 272 tokens, 4.0 ms on
// pages of 4, and 0.44 on pages of 64.
// Measured (few rows / chunk kernel, us), 4 key heads of 128, 64 sequences of 128 to 8192 keys: 24
// rows 81 / 84, 32 rows 83 / 83, 40 rows 132 / 95, 64 rows 143 / 89; of 64: 32 rows 51 / 72, 64 rows
// 88 / 77.  By units a CTA: 5 (256 tokens over 1024, 8 heads of 64) 21 / 24, 5 (64 over 4000, 4 of 64
// with 2 queries) 17 / 26, 6 (300 over 1500, 4 of 128) 31 / 31, 8 (512 over 512, 8 of 128) 39 / 28, 8
// (100 over 3000, 2 of 128 with 4) 26 / 33, 9 (16 chunks of 16 over 500) 17 / 25, 11 (200 over 2000, 2
// of 128 with 4) 33 / 31.  (The units leave out how often rows read their keys again: many rows over
// few keys are where the rule is off.)
constexpr int kFewRows = 32, kFewUnits = 9;

// Keys of a full table up to which the kernel of few rows takes items whole: one launch, no join
// (one token over 257 keys, 4 heads of 64: 7.8 us from 9.4, and a launch less for the host).
constexpr int kWholeKeys = 512;

struct AttnPlan {
    bool chunk, whole;
    int ctas, entries, tile, sms;
    kda::ChunkLimits lim;
    int rows;  // of partial sums
    size_t off_entries, off_ml, off_o, bytes;
};
AttnPlan attn_plan(int N, int total_q, int max_q, int Hq, int Hkv, int d, int page_size, int P) {
    AttnPlan a = {};
    const int G = Hq / Hkv;
    if (max_q > total_q) max_q = total_q;
    a.sms = kda::host_num_sms(device());
    const int few = kda::paged_rows_tile();
    // units that there can be: every sequence's tiles, each over a full table
    const long long seqs = N < total_q ? N : total_q;
    const long long tiles = ((long long)total_q * G / few + seqs) * Hkv, span = ((long long)P * page_size + 63) / 64;
    const long long top = (long long)a.sms * kda::paged_rows_ctas_per_sm(d);
    a.chunk = (long long)max_q * G > kFewRows && (double)tiles * span > (double)(kFewUnits * top) &&
              kda::paged_chunk_pages(page_size);
    long long rows;
    if (a.chunk) {
        a.tile = kda::paged_chunk_tile();
        a.lim = kda::paged_chunk_limits(N, total_q, G, Hkv, P * page_size, a.sms);
        a.entries = a.lim.entries;
        a.off_entries = 256 + up256(3 * (size_t)N * sizeof(int)) + up256((size_t)a.lim.pieces * kda::paged_chunk_piece_bytes());
        rows = a.lim.rows;
    } else {
        a.tile = few;
        a.whole = (long long)P * page_size <= kWholeKeys;
        a.ctas = (int)top;
        if (tiles < top && (a.whole || tiles * span < top)) a.ctas = (int)(a.whole ? tiles : tiles * span);
        a.entries = a.whole ? 0 : a.ctas;
        rows = a.whole ? 0 : (long long)kda::paged_rows_slots(a.ctas) * a.tile;
    }
    a.rows = (int)rows;
    a.off_ml = a.off_entries + up256((size_t)a.entries * sizeof(kda::SplitEntry));
    a.off_o = a.off_ml + up256((size_t)rows * sizeof(float2));
    a.bytes = a.whole ? 0 : a.off_o + (size_t)rows * d * sizeof(float);
    return a;
}

// ----------------------------------------------------------------- pages ----
int table_sizes(int R, int P, int num_pages, int page_size) {
    if (R < 1 || P < 1 || num_pages < 1 || page_size < 1) return KDA_ERR_INVALID_ARG;
    if (R > kda::PG_MAX_ROWS || (long long)R * P > 0x7fffffffLL || num_pages > (1 << 30) ||
        (long long)P * page_size > 0x7fffffffLL)
        return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}
int list_size(int n, int R) {
    if (n < 0 || n > R) return KDA_ERR_INVALID_ARG;  // a row is named once
    return n > kda::PG_MAX_LIST ? KDA_ERR_UNSUPPORTED : KDA_OK;
}
int device_status(kda::DeviceStatus *st) {
    if (kda::host_status_word(&st->word) != KDA_OK) return KDA_ERR_CUDA;
    st->wait_polls = kda::host_wait_polls();
    return KDA_OK;
}
kda::PagesParams pages_params(int *table, int *length, int *ref, int R, int P, int num_pages, int page_size) {
    kda::PagesParams p = {};
    p.table = table;
    p.length = length;
    p.ref = ref;
    p.R = R;
    p.P = P;
    p.num_pages = num_pages;
    p.ps = page_size;
    return p;
}
int pool_check(const void *pool, long long outer, long long outer_stride, long long page_stride, long long page_bytes,
               int num_pages) {
    // a pool of no layers has no memory
    if ((pool == nullptr && outer != 0) || outer < 0 || page_bytes < 1 || num_pages < 1 || outer_stride < 0 || page_stride < 0)
        return KDA_ERR_INVALID_ARG;
    // pages that overlap would be read and written at once
    const long long extent[2] = {num_pages, outer};
    if (!apart({page_stride, outer_stride}, extent, page_bytes)) return KDA_ERR_INVALID_ARG;
    if (!al(pool, 16) || page_bytes % 16 || page_stride % 16 || outer_stride % 16) return KDA_ERR_ALIGNMENT;
    if (outer > (1 << 24)) return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}
int copy_pages(void *pool, long long outer, long long outer_stride, long long page_stride, long long page_bytes,
               int num_pages, const int *src, const int *dst, const int *count, int n, cudaStream_t stream) {
    kda::PoolParams p = {};
    if (device_status(&p.st) != KDA_OK) return KDA_ERR_CUDA;
    p.pool = static_cast<uint8_t *>(pool);
    p.src = src;
    p.dst = dst;
    p.count = count;
    p.outer = outer;
    p.outer_stride = outer_stride;
    p.page_stride = page_stride;
    p.page_bytes = page_bytes;
    p.num_pages = num_pages;
    p.n = n;
    return to_status(kda::launch_pages_copy(p, count == nullptr, kda::host_num_sms(device()), stream));
}

// The workspace of a compaction: block counts, {live, moves}, holes, moves, ranks.
struct CompactPlan {
    size_t off_n, off_hole, off_move, off_rank, bytes;
};
CompactPlan compact_plan(int num_pages) {
    CompactPlan c;
    const size_t list = up256((size_t)num_pages * sizeof(int));
    c.off_n = up256((size_t)kda::compact_blocks(num_pages) * sizeof(int));
    c.off_hole = c.off_n + 256;
    c.off_move = c.off_hole + list;
    c.off_rank = c.off_move + list;
    c.bytes = c.off_rank + list;
    return c;
}

}  // namespace

extern "C" {

size_t kda_paged_attn_workspace_bytes(int N, int total_q, int max_q, int Hq, int Hkv, int d, int page_size, int P) {
    if (attn_sizes(N, total_q, max_q, Hq, Hkv, d, page_size, P) != KDA_OK || total_q == 0) return 0;
    return attn_plan(N, total_q, max_q, Hq, Hkv, d, page_size, P).bytes;
}

int kda_paged_attn(const void *q, const void *k_new, const void *v_new, void *k_pages, void *v_pages, const int *cu_q,
                   const int *page_table, const int *length, const int *rows, float scale, void *out, float *lse, int N,
                   int total_q, int max_q, int Hq, int Hkv, int d, int page_size, int num_pages, int P, int R,
                   long long q_stride, long long k_stride, long long v_stride, const long long *page_strides, int dtype,
                   void *workspace, size_t workspace_bytes, void *stream) {
    if (const int st = attn_sizes(N, total_q, max_q, Hq, Hkv, d, page_size, P); st != KDA_OK) return st;
    if (num_pages < 1 || R < 1 || (rows == nullptr && R < N)) return KDA_ERR_INVALID_ARG;
    if (!(scale > 0.f) || scale > 1.0e30f) return KDA_ERR_INVALID_ARG;  // also rejects NaN
    if (dtype != KDA_BF16 && dtype != KDA_FP16) return KDA_ERR_UNSUPPORTED;
    if (!cu_q || !page_table || !length || !k_pages || !v_pages || (k_new == nullptr) != (v_new == nullptr))
        return KDA_ERR_INVALID_ARG;
    if (total_q > 0 && (!q || !out)) return KDA_ERR_INVALID_ARG;
    const long long row = (long long)Hkv * d;
    const long long dense[6] = {page_size * row, row, d, page_size * row, row, d};
    const long long *ps = page_strides ? page_strides : dense;
    if (q_stride < (long long)Hq * d || (k_new && (k_stride < row || v_stride < row))) return KDA_ERR_INVALID_ARG;
    for (int i = 0; i < 6; ++i) {
        if (ps[i] < d || ps[i] > (1LL << 38)) return KDA_ERR_INVALID_ARG;
        if (ps[i] % 8) return KDA_ERR_ALIGNMENT;
    }
    if (q_stride % 8 || (k_new && (k_stride % 8 || v_stride % 8)) || !al(q, 16) || !al(k_new, 16) || !al(v_new, 16) ||
        !al(k_pages, 16) || !al(v_pages, 16) || !al(out, 16) || !al(lse, 4) || !al(cu_q, 4) || !al(page_table, 4) ||
        !al(length, 4) || !al(rows, 4) || !al(workspace, 16))
        return KDA_ERR_ALIGNMENT;
    // the new tokens would be written over one another
    const long long places[3] = {num_pages, page_size, Hkv};
    if (k_new && !(apart({ps[0], ps[1], ps[2]}, places, d) && apart({ps[3], ps[4], ps[5]}, places, d))) return KDA_ERR_INVALID_ARG;
    if (total_q == 0) return KDA_OK;
    const AttnPlan pl = attn_plan(N, total_q, max_q, Hq, Hkv, d, page_size, P);
    if (pl.bytes > 0 && (!workspace || workspace_bytes < pl.bytes)) return KDA_ERR_INVALID_ARG;
    kda::PagedParams p = {};
    if (device_status(&p.st) != KDA_OK) return KDA_ERR_CUDA;
    p.q = static_cast<const uint16_t *>(q);
    p.k_new = static_cast<const uint16_t *>(k_new);
    p.v_new = static_cast<const uint16_t *>(v_new);
    p.kp = static_cast<uint16_t *>(k_pages);
    p.vp = static_cast<uint16_t *>(v_pages);
    p.cu = cu_q;
    p.table = page_table;
    p.length = length;
    p.rows = rows;
    p.out = static_cast<uint16_t *>(out);
    p.lse = lse;
    p.scale_log2 = scale * 1.4426950408889634f;
    p.N = N;
    p.total_q = total_q;
    p.max_q = max_q < total_q ? max_q : total_q;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.G = Hq / Hkv;
    p.page_size = page_size;
    p.num_pages = num_pages;
    p.P = P;
    p.R = R;
    p.q_ts = q_stride;
    p.kn_ts = k_stride;
    p.vn_ts = v_stride;
    p.k_ps = ps[0];
    p.k_ts = ps[1];
    p.k_hs = ps[2];
    p.v_ps = ps[3];
    p.v_ts = ps[4];
    p.v_hs = ps[5];
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    p.entries = reinterpret_cast<kda::SplitEntry *>(ws + pl.off_entries);
    p.part_ml = reinterpret_cast<float2 *>(ws + pl.off_ml);
    p.part_o = reinterpret_cast<float *>(ws + pl.off_o);
    p.part_rows = pl.rows;
    p.max_entries = pl.entries;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool bf = dtype == KDA_BF16;
    if (pl.chunk) {
        if (kda::launch_paged_chunk(p, pl.lim, ws, d, bf, pl.sms, s) != cudaSuccess) return KDA_ERR_CUDA;
        if (pl.lim.rows == 0) return KDA_OK;  // nothing can be split
        const int *count = reinterpret_cast<const int *>(ws) + 2;  // ChunkPlanHead::entries
        return to_status(kda::launch_paged_join(p, d, bf, count, pl.entries, pl.tile, pl.sms, s));
    }
    if (kda::launch_paged_rows(p, d, bf, pl.whole, pl.ctas, s) != cudaSuccess) return KDA_ERR_CUDA;
    if (pl.whole) return KDA_OK;
    return to_status(kda::launch_paged_join(p, d, bf, nullptr, pl.entries, pl.tile, pl.sms, s));
}

int kda_pages_reserve(int *table, int *length, int *ref, const int *rows, const int *new_length, int n, int *info, int R,
                      int P, int num_pages, int page_size, void *stream) {
    if (const int st = table_sizes(R, P, num_pages, page_size); st != KDA_OK) return st;
    if (const int st = list_size(n, R); st != KDA_OK) return st;
    if (!table || !length || !ref || (n > 0 && (!rows || !new_length))) return KDA_ERR_INVALID_ARG;
    if (!al(table, 4) || !al(length, 4) || !al(ref, 4) || !al(rows, 4) || !al(new_length, 4) || !al(info, 4))
        return KDA_ERR_ALIGNMENT;
    kda::PagesParams p = pages_params(table, length, ref, R, P, num_pages, page_size);
    if (device_status(&p.st) != KDA_OK) return KDA_ERR_CUDA;
    p.rows = rows;
    p.new_length = new_length;
    p.n = n;
    p.info = info;
    return to_status(kda::launch_pages_grant(p, false, static_cast<cudaStream_t>(stream)));
}

int kda_pages_fork(int *table, int *length, int *ref, const int *src_rows, const int *dst_rows, int n, int *copy_src,
                   int *copy_dst, int *info, int R, int P, int num_pages, int page_size, void *stream) {
    if (const int st = table_sizes(R, P, num_pages, page_size); st != KDA_OK) return st;
    if (const int st = list_size(n, R); st != KDA_OK) return st;
    if (!table || !length || !ref || (n > 0 && (!src_rows || !dst_rows || !copy_src || !copy_dst))) return KDA_ERR_INVALID_ARG;
    if (!al(table, 4) || !al(length, 4) || !al(ref, 4) || !al(src_rows, 4) || !al(dst_rows, 4) || !al(copy_src, 4) ||
        !al(copy_dst, 4) || !al(info, 4))
        return KDA_ERR_ALIGNMENT;
    kda::PagesParams p = pages_params(table, length, ref, R, P, num_pages, page_size);
    if (device_status(&p.st) != KDA_OK) return KDA_ERR_CUDA;
    p.rows = dst_rows;
    p.src = src_rows;
    p.copy_src = copy_src;
    p.copy_dst = copy_dst;
    p.n = n;
    p.info = info;
    return to_status(kda::launch_pages_grant(p, true, static_cast<cudaStream_t>(stream)));
}

int kda_pages_free(int *table, int *length, int *ref, const int *rows, int n, int R, int P, int num_pages, int page_size,
                   void *stream) {
    if (const int st = table_sizes(R, P, num_pages, page_size); st != KDA_OK) return st;
    if (n < 0 || n > R) return KDA_ERR_INVALID_ARG;
    if (!table || !length || !ref || (n > 0 && !rows)) return KDA_ERR_INVALID_ARG;
    if (!al(table, 4) || !al(length, 4) || !al(ref, 4) || !al(rows, 4)) return KDA_ERR_ALIGNMENT;
    if (n == 0) return KDA_OK;
    kda::PagesParams p = pages_params(table, length, ref, R, P, num_pages, page_size);
    if (device_status(&p.st) != KDA_OK) return KDA_ERR_CUDA;
    p.rows = rows;
    p.n = n;
    return to_status(kda::launch_pages_free(p, kda::host_num_sms(device()), static_cast<cudaStream_t>(stream)));
}

size_t kda_pages_compact_workspace_bytes(int num_pages) {
    return num_pages < 1 || num_pages > (1 << 30) ? 0 : compact_plan(num_pages).bytes;
}

int kda_pages_compact(const int *table, const int *length, const int *ref, int *table_out, int *ref_out, int *info, int R,
                      int P, int num_pages, int page_size, void *workspace, size_t workspace_bytes, void *stream) {
    if (const int st = table_sizes(R, P, num_pages, page_size); st != KDA_OK) return st;
    if (!table || !length || !ref || !table_out || !ref_out || !workspace) return KDA_ERR_INVALID_ARG;
    if (!al(table, 4) || !al(length, 4) || !al(ref, 4) || !al(table_out, 4) || !al(ref_out, 4) || !al(info, 4) ||
        !al(workspace, 16))
        return KDA_ERR_ALIGNMENT;
    const CompactPlan c = compact_plan(num_pages);
    if (workspace_bytes < c.bytes) return KDA_ERR_INVALID_ARG;
    kda::PagesParams p = pages_params(const_cast<int *>(table), const_cast<int *>(length), const_cast<int *>(ref), R, P,
                                      num_pages, page_size);
    if (device_status(&p.st) != KDA_OK) return KDA_ERR_CUDA;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    p.table_out = table_out;
    p.ref_out = ref_out;
    p.info = info;
    p.ws_counts = reinterpret_cast<int *>(ws);
    p.ws_n = reinterpret_cast<int *>(ws + c.off_n);
    p.ws_hole = reinterpret_cast<int *>(ws + c.off_hole);
    p.ws_move = reinterpret_cast<int *>(ws + c.off_move);
    p.ws_rank = reinterpret_cast<int *>(ws + c.off_rank);
    return to_status(kda::launch_pages_compact(p, kda::host_num_sms(device()), static_cast<cudaStream_t>(stream)));
}

int kda_pages_compact_pool(void *pool, long long outer, long long outer_stride, long long page_stride, long long page_bytes,
                           int num_pages, const void *workspace, size_t workspace_bytes, void *stream) {
    if (const int st = pool_check(pool, outer, outer_stride, page_stride, page_bytes, num_pages); st != KDA_OK) return st;
    if (!workspace || num_pages > (1 << 30)) return KDA_ERR_INVALID_ARG;
    if (!al(workspace, 16)) return KDA_ERR_ALIGNMENT;
    const CompactPlan c = compact_plan(num_pages);
    if (workspace_bytes < c.bytes) return KDA_ERR_INVALID_ARG;
    if (outer == 0) return KDA_OK;
    const uint8_t *ws = static_cast<const uint8_t *>(workspace);
    // at most half of the pages move: a move needs a hole
    return copy_pages(pool, outer, outer_stride, page_stride, page_bytes, num_pages,
                      reinterpret_cast<const int *>(ws + c.off_move), reinterpret_cast<const int *>(ws + c.off_hole),
                      reinterpret_cast<const int *>(ws + c.off_n) + 1, (num_pages + 1) / 2, static_cast<cudaStream_t>(stream));
}

int kda_pages_copy(void *pool, long long outer, long long outer_stride, long long page_stride, long long page_bytes,
                   int num_pages, const int *src, const int *dst, int n, void *stream) {
    if (const int st = pool_check(pool, outer, outer_stride, page_stride, page_bytes, num_pages); st != KDA_OK) return st;
    if (n < 0 || (n > 0 && (!src || !dst))) return KDA_ERR_INVALID_ARG;
    if (n > kda::PG_MAX_COPY) return KDA_ERR_UNSUPPORTED;
    if (!al(src, 4) || !al(dst, 4)) return KDA_ERR_ALIGNMENT;
    if (n == 0 || outer == 0) return KDA_OK;
    return copy_pages(pool, outer, outer_stride, page_stride, page_bytes, num_pages, src, dst, nullptr, n,
                      static_cast<cudaStream_t>(stream));
}

}  // extern "C"
