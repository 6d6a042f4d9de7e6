// paged_params.cuh -- what the paged-attention kernels share: their
// parameters, the geometry of a sequence, and the join of split rows.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "kda_device.cuh"
#include "launch_order.cuh"

namespace kda {

// One row's partial result over part of its keys: unnormalised sums against a
// reference m (log2 units, the weights' shift taken off) and l = sum of 2^(x - m).
// The first piece of a split item has its rows from part row `head`, the `count`
// others from `next`, `stride` rows apart.
struct SplitEntry {
    int n, h, t;     // sequence, key head, row tile
    int head, next, count, stride;  // count = 0: nothing to join
};

// Upper bounds of the chunk kernel's plan: pieces of work, split items, rows of
// partial sums.
struct ChunkLimits {
    int pieces, entries, rows;
};

struct PagedParams {
    const uint16_t *q, *k_new, *v_new;  // 16-bit [total_q][heads][d], token strides below
    uint16_t *kp, *vp;                  // pages
    const int *cu, *table, *length, *rows;
    uint16_t *out;
    float *lse;
    float scale_log2;                   // scale * log2(e)
    int N, total_q, max_q, Hq, Hkv, G, page_size, num_pages, P, R;
    long long q_ts, kn_ts, vn_ts;       // elements between tokens
    long long k_ps, k_ts, k_hs;         // key pages: elements between pages, tokens, heads
    long long v_ps, v_ts, v_hs;         // value pages
    float *part_o;                      // [part rows][d]
    float2 *part_ml;                    // [part rows]
    SplitEntry *entries;
    int part_rows, max_entries;         // room of the workspace
    DeviceStatus st;
};

// Sequence n of the batch, from arrays the host never reads: every value is
// bounded here before it is used as an index, and a change is reported.
struct PagedSeq {
    int q0, nq, len, row;  // first token, new tokens, cache length with them, table row
};
__device__ __forceinline__ PagedSeq paged_seq(const PagedParams &p, int n, bool tell) {
    PagedSeq s;
    const int a = p.cu[n], b = p.cu[n + 1];
    s.row = p.rows != nullptr ? p.rows[n] : n;
    const bool row_ok = s.row >= 0 && s.row < p.R;
    if (!row_ok) s.row = 0;
    const int len = row_ok ? p.length[s.row] : 0;
    bool ok = row_ok && a >= 0 && b >= a && b <= p.total_q && b - a <= p.max_q && len >= 0 &&
              (long long)len <= (long long)p.P * p.page_size;
    s.q0 = min(max(a, 0), p.total_q);
    s.nq = min(min(max(b, s.q0), p.total_q) - s.q0, p.max_q);
    s.len = (int)min((long long)max(len, 0), (long long)p.P * p.page_size);
    if (tell && !ok) report(p.st, DEV_BAD_ARG);
    return s;
}

// Rows of a sequence are its tokens times the G query heads of one key head,
// row r = token r / G, head r % G.  Keys that rows [0, r] see at most.
__device__ __forceinline__ int paged_kv_end(const PagedSeq &s, int G, int last_row) {
    const int r = min(last_row, s.nq * G - 1);
    return max(0, s.len - s.nq + r / G + 1);
}

template <bool BF>
__device__ __forceinline__ uint32_t pack16x2(float lo, float hi) {
    if constexpr (BF) return pack_bf16x2(lo, hi);
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// 2^x by the hardware's unit (relative error about 2^-22); 2^-inf = 0.
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Binary orders that a weight is shifted up by before it is rounded to 16 bits.
// bf16 reaches as far as fp32.  fp16 has full precision down to 2^-14 only, and a
// row whose first key outweighs the others (an attention sink) may have most of
// its other keys below that: shifted, weights keep it down to 2^-22 of the
// reference, with 2^7 left above it (as many orders up as the chunk kernel needs:
// with 2^3 it moved references so often that a mixed batch took 110 us for 81).
template <bool BF>
__host__ __device__ constexpr float weight_shift() { return BF ? 0.f : 8.f; }

constexpr float LN2 = 0.69314718055994531f;

// lse of a row from its reference m (log2 units) and sum l.  What tells a row without keys is
// l == 0: a row whose every score is NaN has m = -inf as well (maxima pass NaN over), and l = NaN,
// which is its lse.
__device__ __forceinline__ float row_lse(float m, float l) { return l == 0.f ? -INFINITY : m * LN2 + logf(l); }

}  // namespace kda
