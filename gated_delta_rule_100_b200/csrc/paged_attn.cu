// paged_attn.cu -- attention of new tokens over a paged cache for few rows
// (single tokens, a few drafted tokens, any page size), and the join of rows
// whose keys were split.
//
// For token i of sequence n (n_q new tokens, cache length L with them), head h:
//   o = sum_{j <= L - n_q + i} p_j v_j / sum_j p_j,  p_j = exp(scale q.k_j)
// in one pass over the keys with a running maximum m and sum l per row:
//   m' = max(m, x),  o <- o 2^(m-m') + 2^(x-m') v,  l <- l 2^(m-m') + 2^(x-m').
// Statistics and sums are fp32; the weights 2^(x-m) are rounded to the inputs'
// 16-bit type as the operand of the second product (relative error at most half
// a step each, and the roundings of many keys average out), while l sums them
// before that rounding.
//
// Bound: HBM.  A key head's keys and values are read once for every 16 of its
// rows (new tokens times the G query heads): once for up to 16, which is what
// single tokens are, twice for 17 to 32 (64 sequences of 3 tokens, 8 query heads a
// key head of 128: 83 us, twice the 41 that one reading takes).  That is 4 d bytes a
// key against at most 64 d operations, far under the card's ratio.  So the kernel is
// laid out for loads in flight: the rows of an item, at most 16, fill an mma.sync tile;
// each of the four warps walks its own 16 keys of every 64 with its own ring of
// asynchronous 16-byte copies and no block-wide barrier; rows out of the
// sequence's end are filled with zeros, so whatever lies behind it (NaN too)
// never meets the products.
//
// Work is cut into equal runs of 64-key units over all (sequence, key head, row
// tile) items, one run per CTA: lengths from 1 to the cache's end load every SM
// alike.  An item's own cost counts as PA_HEAD units: for 256 sequences of 128 to
// 16,384 keys, 8 key heads of 128, the call took 653 us with none, 618, 596, 559
// and 570 us with 1, 2, 4 and 8.  Those are replays on the same inputs, some of which
// the L2 cache still holds (3 % of them would fill it); on other inputs each time the
// call takes 592 to 598 us, 6.2 TB/s, where a plain sum over 4 GB reads 6.5.  A run
// has at most one item that began before it and one that ends after it; these
// write their sums to slots, joined by the second kernel in a fixed order (no
// atomics, so results do not depend on timing).
#include "kda_internal.cuh"
#include "paged_params.cuh"

namespace kda {

constexpr int PA_THREADS = 128, PA_WARPS = 4, PA_ROWS = 16, PA_UNIT = 64, PA_WKEYS = 16;
constexpr int PA_HEAD = 4;  // units that an item's own cost (queries, sums, output) counts as

template <int D>
struct PaShape {
    static constexpr int ROWB = D * 2;                        // bytes of a key
    static constexpr int TILE = PA_WKEYS * ROWB;              // one warp's keys of a stage
    static constexpr int STAGE = 2 * TILE;                    // keys and values
    static constexpr int STAGES = D == 128 ? 3 : 4;
    static constexpr int RING = STAGE * STAGES;               // per warp
    static constexpr int MSTRIDE = D + 8;                     // floats of a row of sums (padded: eight rows at a time)
    static constexpr int SMEM = PA_WARPS * RING + PA_ROWS * MSTRIDE * 4;
};

__device__ __forceinline__ void cp16(uint32_t dst, const void *src, bool valid) {
    const int n = valid ? 16 : 0;  // 0: the 16 bytes are filled with zeros
    asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
template <bool BF>
__device__ __forceinline__ void mma16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (BF)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// 64-key units of row tile t.  A tile that sees nothing keeps one, so that its
// rows are written.
__device__ __forceinline__ int pa_units(const PagedSeq &s, int G, int t) {
    return max(1, (paged_kv_end(s, G, (t + 1) * PA_ROWS - 1) + PA_UNIT - 1) / PA_UNIT);
}
__device__ __forceinline__ int pa_tiles(const PagedSeq &s, int G) { return (s.nq * G + PA_ROWS - 1) / PA_ROWS; }
// A run's part of one item.
struct PaPiece {
    PagedSeq s;
    int n, h, t, off, cnt, units;
};

// WHOLE: an item is one unit of the plan, so nothing is split or joined (short caches).
template <int D, bool BF, bool WHOLE>
__global__ void __launch_bounds__(PA_THREADS) paged_rows_kernel(const PagedParams p) {
    using S = PaShape<D>;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ long long s_sum[PA_WARPS];
    __shared__ long long s_start;                 // first unit of the item found
    __shared__ int s_n, s_h, s_t;
    __shared__ float2 s_ml[PA_WARPS][PA_ROWS];

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int G = p.G, c = blockIdx.x, grid = gridDim.x;
    launch_dependents();
    auto plan_units = [&](const PagedSeq &s, int t) { return WHOLE ? 1 : PA_HEAD + pa_units(s, G, t); };
    auto head_units = [&](const PagedSeq &s) {
        if (WHOLE) return (long long)pa_tiles(s, G);
        long long w = 0;
        for (int t = 0; t < pa_tiles(s, G); ++t) w += plan_units(s, t);
        return w;
    };

    // ---- plan: the units of every sequence, and the item that this run begins in
    const int per = (p.N + PA_THREADS - 1) / PA_THREADS;
    long long mine = 0;
    for (int n = tid * per; n < min(p.N, (tid + 1) * per); ++n) mine += head_units(paged_seq(p, n, c == 0)) * p.Hkv;
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long up = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += up;
    }
    if (lane == 31) s_sum[warp] = incl;
    __syncthreads();
    long long before = incl - mine, W = 0;
    for (int w = 0; w < PA_WARPS; ++w) {
        if (w < warp) before += s_sum[w];
        W += s_sum[w];
    }
    const long long runs = W < grid ? W : grid;  // every run has at least one unit
    if (!WHOLE && tid == 0 && KDA_CHECK(p.st, c < p.max_entries)) p.entries[c].count = 0;
    if (c >= runs) return;
    long long u = c * W / runs;
    const long long u_end = (c + 1) * W / runs;
    if (u >= before && u < before + mine) {      // exactly one thread
        long long left = u - before, start = before;
        int n = tid * per;
        for (;; ++n) {
            const PagedSeq s = paged_seq(p, n, false);
            const long long hu = head_units(s), w = hu * p.Hkv;
            if (left >= w) { left -= w; start += w; continue; }
            const int h = (int)(left / hu);
            left -= h * hu;
            start += h * hu;
            int t = 0;
            for (int k; left >= (k = plan_units(s, t)); ++t) { left -= k; start += k; }
            s_n = n; s_h = h; s_t = t; s_start = start;
            break;
        }
    }
    __syncthreads();
    long long start = s_start;                   // the item's first unit

    const uint32_t ring = smem_u32(smem) + warp * S::RING;
    float *sums = reinterpret_cast<float *>(smem + PA_WARPS * S::RING);
    const int g8 = lane >> 2, t4 = lane & 3;

    // the run's part of the item that unit u lies in and that begins at unit `start`: its first
    // PA_HEAD units stand for no keys, so a part may be empty
    auto take = [&](PaPiece &pc) {
        pc.units = pa_units(pc.s, G, pc.t);
        const int to = (int)min((long long)(PA_HEAD + pc.units), u_end - start);
        pc.off = WHOLE ? 0 : max(0, (int)(u - start) - PA_HEAD);
        pc.cnt = WHOLE ? pc.units : max(0, to - PA_HEAD) - pc.off;
        u = WHOLE ? u + 1 : start + to;
    };
    // ---- the warp's loads: 16 keys of each unit
    const uint16_t *kptr = p.kp, *vptr = p.vp;
    bool kvalid = false;
    auto locate = [&](const PaPiece &pc, int step) {  // lane l < 16: where key l of the step lies
        const int pos = (pc.off + step) * PA_UNIT + warp * PA_WKEYS + (lane & 15), first_new = pc.s.len - pc.s.nq;
        kvalid = step < pc.cnt && pos < paged_kv_end(pc.s, G, (pc.t + 1) * PA_ROWS - 1);
        kptr = p.kp;
        vptr = p.vp;
        if (kvalid) {
            if (p.k_new != nullptr && pos >= first_new) {
                const long long tok = pc.s.q0 + pos - first_new;
                kptr = p.k_new + tok * p.kn_ts + pc.h * D;
                vptr = p.v_new + tok * p.vn_ts + pc.h * D;
            } else {
                const int page = p.table[(long long)pc.s.row * p.P + pos / p.page_size], in = pos % p.page_size;
                if (page >= 0 && page < p.num_pages) {
                    kptr = p.kp + page * p.k_ps + in * p.k_ts + pc.h * p.k_hs;
                    vptr = p.vp + page * p.v_ps + in * p.v_ts + pc.h * p.v_hs;
                } else {
                    kvalid = false;
                    report(p.st, DEV_BAD_ARG);
                }
            }
        }
    };
    auto issue = [&](int step) {
        constexpr int CPR = D / 8, RPI = 32 / CPR;  // 16-byte pieces of a key, keys of one copy
        const uint32_t kb = ring + (step % S::STAGES) * S::STAGE, vb = kb + S::TILE;
        const int ch = lane % CPR;
#pragma unroll
        for (int i = 0; i < PA_WKEYS / RPI; ++i) {
            const int r = i * RPI + lane / CPR;
            const uint16_t *ks = reinterpret_cast<const uint16_t *>(__shfl_sync(0xffffffffu, (unsigned long long)kptr, r));
            const uint16_t *vs = reinterpret_cast<const uint16_t *>(__shfl_sync(0xffffffffu, (unsigned long long)vptr, r));
            const bool ok = __shfl_sync(0xffffffffu, (int)kvalid, r) != 0;
            const uint32_t o = r * S::ROWB + ((ch ^ (r & 7)) << 4);
            cp16(kb + o, ks + ch * 8, ok);
            cp16(vb + o, vs + ch * 8, ok);
        }
    };
    // a piece's new tokens to their pages, and its first loads
    auto begin = [&](const PaPiece &pc) {
        // The new tokens' keys and values of this run go to their pages; they are read from where
        // they came, so nothing waits for these stores.  (Row tile 0's last unit writes what no
        // unit of it covers: a tile sees at least the first token.)
        if (p.k_new != nullptr && pc.t == 0) {
            const int first_new = pc.s.len - pc.s.nq;
            const int lo = max(max(pc.off * PA_UNIT, first_new), 0);
            const int hi = pc.off + pc.cnt == pc.units ? pc.s.len : min(pc.s.len, (pc.off + pc.cnt) * PA_UNIT);
            constexpr int CH = D / 8;
            for (int i = tid; i < max(hi - lo, 0) * CH; i += PA_THREADS) {
                const int pos = lo + i / CH, ch = i % CH, tok = pc.s.q0 + pos - first_new;
                const int page = p.table[(long long)pc.s.row * p.P + pos / p.page_size], in = pos % p.page_size;
                if (page < 0 || page >= p.num_pages) { report(p.st, DEV_BAD_ARG); continue; }
                if (!KDA_CHECK(p.st, tok >= 0 && tok < p.total_q && pos < p.P * p.page_size)) continue;
                const uint4 kx = *reinterpret_cast<const uint4 *>(p.k_new + tok * p.kn_ts + pc.h * D + ch * 8);
                const uint4 vx = *reinterpret_cast<const uint4 *>(p.v_new + tok * p.vn_ts + pc.h * D + ch * 8);
                *reinterpret_cast<uint4 *>(p.kp + page * p.k_ps + in * p.k_ts + pc.h * p.k_hs + ch * 8) = kx;
                *reinterpret_cast<uint4 *>(p.vp + page * p.v_ps + in * p.v_ts + pc.h * p.v_hs + ch * 8) = vx;
            }
        }
        locate(pc, 0);
#pragma unroll
        for (int i = 0; i < S::STAGES - 1; ++i) {
            if (i < pc.cnt) issue(i);
            cp_commit();
            locate(pc, i + 1);
        }
    };

    PaPiece pc;
    pc.n = s_n;
    pc.h = s_h;
    pc.t = s_t;
    pc.s = paged_seq(p, pc.n, false);
    take(pc);
    if (pc.cnt == 0) return;
    begin(pc);
    for (;;) {
        const int rows = pc.s.nq * G, first_new = pc.s.len - pc.s.nq;  // first_new may be negative: tokens without a place
        // ---- the rows' queries as mma operands, straight from memory
        uint32_t qf[D / 16][4];
        int qpos[2];  // last key that the thread's two rows see; -1: none
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int r = pc.t * PA_ROWS + g8 + 8 * e;
            const bool ok = r < rows && KDA_CHECK(p.st, pc.s.q0 + r / G < p.total_q && pc.h < p.Hkv);
            qpos[e] = ok ? first_new + r / G : -1;
            const uint16_t *qr = p.q + (ok ? (pc.s.q0 + r / G) * p.q_ts + (long long)(pc.h * G + r % G) * D : 0);
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
                qf[k][e] = ok ? *reinterpret_cast<const uint32_t *>(qr + k * 16 + t4 * 2) : 0u;
                qf[k][2 + e] = ok ? *reinterpret_cast<const uint32_t *>(qr + k * 16 + 8 + t4 * 2) : 0u;
            }
        }
        const int low_pos = first_new + (pc.t * PA_ROWS) / G;  // the smallest last key of the tile's rows

        float o[D / 8][4];
#pragma unroll
        for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

        for (int step = 0; step < pc.cnt; ++step) {
            cp_wait<S::STAGES - 2>();
            __syncwarp();
            if (step + S::STAGES - 1 < pc.cnt) issue(step + S::STAGES - 1);  // the stage read in the step before
            cp_commit();
            if (step + S::STAGES < pc.cnt) locate(pc, step + S::STAGES);
            const uint32_t kb = ring + (step % S::STAGES) * S::STAGE, vb = kb + S::TILE;
            const int base = (pc.off + step) * PA_UNIT + warp * PA_WKEYS;
            float x[2][4] = {};
            {
                const int r = (lane >> 4) * 8 + (lane & 7), hi = (lane >> 3) & 1;
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    uint32_t b[4];
                    ldsm4(b, kb + r * S::ROWB + (((k * 2 + hi) ^ (r & 7)) << 4));
                    mma16<BF>(x[0], qf[k], b[0], b[1]);
                    mma16<BF>(x[1], qf[k], b[2], b[3]);
                }
            }
            const bool all = base + PA_WKEYS - 1 <= low_pos;  // no row's mask reaches these keys
#pragma unroll
            for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float y = x[nt][e] * p.scale_log2;
                    x[nt][e] = all || base + nt * 8 + t4 * 2 + (e & 1) <= qpos[e >> 1] ? y : -INFINITY;
                }
            float f[2];
            uint32_t pa[4];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float mx = fmaxf(fmaxf(x[0][2 * e], x[0][2 * e + 1]), fmaxf(x[1][2 * e], x[1][2 * e + 1]));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                mx = fmaxf(mx, m[e]);
                const float top = mx == -INFINITY ? 0.f : mx;  // nothing seen yet: every weight is 2^-inf = 0
                const float ref = top - weight_shift<BF>();
                f[e] = ex2(m[e] - top);
                m[e] = mx;
                float sum = 0.f;
#pragma unroll
                for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        x[nt][2 * e + j] = ex2(x[nt][2 * e + j] - ref);
                        sum += x[nt][2 * e + j];
                    }
                l[e] = l[e] * f[e] + sum;
                pa[e] = pack16x2<BF>(x[0][2 * e], x[0][2 * e + 1]);
                pa[2 + e] = pack16x2<BF>(x[1][2 * e], x[1][2 * e + 1]);
            }
            if (__any_sync(0xffffffffu, f[0] != 1.f || f[1] != 1.f)) {
#pragma unroll
                for (int i = 0; i < D / 8; ++i) {
                    o[i][0] *= f[0]; o[i][1] *= f[0];
                    o[i][2] *= f[1]; o[i][3] *= f[1];
                }
            }
            {
                const int r = ((lane >> 3) & 1) * 8 + (lane & 7), hi = lane >> 4;
#pragma unroll
                for (int i = 0; i < D / 16; ++i) {
                    uint32_t b[4];
                    ldsm4t(b, vb + r * S::ROWB + (((i * 2 + hi) ^ (r & 7)) << 4));
                    mma16<BF>(o[2 * i], pa, b[0], b[1]);
                    mma16<BF>(o[2 * i + 1], pa, b[2], b[3]);
                }
            }
        }
        cp_wait<0>();
        __syncwarp();

        // ---- the next item's loads begin before this one's sums are joined
        const PaPiece done = pc;
        const long long item_end = start + (WHOLE ? 1 : PA_HEAD + done.units);
        bool again = u < u_end;
        if (again) {
            start = item_end;
            if (++pc.t == pa_tiles(pc.s, G)) {
                pc.t = 0;
                if (++pc.h == p.Hkv) {
                    pc.h = 0;
                    do pc.s = paged_seq(p, ++pc.n, false); while (pc.s.nq == 0);
                }
            }
            take(pc);
            again = pc.cnt > 0;
            if (again) begin(pc);
        }

        // ---- the four warps' sums, one after the other onto 16 rows in shared memory
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
            l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
            m[e] -= weight_shift<BF>();
            if (t4 == 0) s_ml[warp][g8 + 8 * e] = make_float2(m[e], l[e]);
        }
        __syncthreads();
        float fw[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float M = -INFINITY;
            for (int w = 0; w < PA_WARPS; ++w) M = fmaxf(M, s_ml[w][g8 + 8 * e].x);
            fw[e] = ex2(m[e] - (M == -INFINITY ? 0.f : M));
        }
        for (int w = 0; w < PA_WARPS; ++w) {
            if (warp == w) {
#pragma unroll
                for (int i = 0; i < D / 8; ++i)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float2 *at = reinterpret_cast<float2 *>(sums + (g8 + 8 * e) * S::MSTRIDE + i * 8 + t4 * 2);
                        float2 y = make_float2(fw[e] * o[i][2 * e], fw[e] * o[i][2 * e + 1]);
                        if (w > 0) { const float2 z = *at; y.x += z.x; y.y += z.y; }
                        *at = y;
                    }
            }
            __syncthreads();
        }
        const bool begins = done.off == 0, ends = done.off + done.cnt == done.units;
        const int slot = begins ? grid + c : c;
#pragma unroll
        for (int i = 0; i < PA_ROWS * D / 4 / PA_THREADS; ++i) {
            const int at = i * PA_THREADS + tid, r = at / (D / 4), col = (at % (D / 4)) * 4;
            float M = -INFINITY, L = 0.f;
            for (int w = 0; w < PA_WARPS; ++w) M = fmaxf(M, s_ml[w][r].x);
            for (int w = 0; w < PA_WARPS; ++w) L += ex2(s_ml[w][r].x - (M == -INFINITY ? 0.f : M)) * s_ml[w][r].y;
            const float4 a = *reinterpret_cast<const float4 *>(sums + r * S::MSTRIDE + col);
            const int row = done.t * PA_ROWS + r;
            if (begins && ends) {
                if (row < done.s.nq * G && KDA_CHECK(p.st, done.s.q0 + row / G < p.total_q && done.h < p.Hkv)) {
                    const float inv = L == 0.f ? 0.f : 1.f / L;
                    const long long tok = done.s.q0 + row / G;
                    const int head = done.h * G + row % G;
                    uint2 y;
                    y.x = pack16x2<BF>(a.x * inv, a.y * inv);
                    y.y = pack16x2<BF>(a.z * inv, a.w * inv);
                    *reinterpret_cast<uint2 *>(p.out + (tok * p.Hq + head) * D + col) = y;
                    if (p.lse != nullptr && col == 0)
                        p.lse[tok * p.Hq + head] = row_lse(M, L);
                }
            } else if (KDA_CHECK(p.st, slot * PA_ROWS + r < p.part_rows)) {
                *reinterpret_cast<float4 *>(p.part_o + ((long long)slot * PA_ROWS + r) * D + col) = a;
                if (col == 0) p.part_ml[(long long)slot * PA_ROWS + r] = make_float2(M, L);
            }
        }
        if (!WHOLE && begins && !ends && tid == 0 && KDA_CHECK(p.st, c < p.max_entries)) {
            // runs c + 1 .. last hold the rest: the last is the one with the item's last unit
            const int last = (int)((item_end * runs + W - 1) / W) - 1;
            p.entries[c] = {done.n, done.h, done.t, (grid + c) * PA_ROWS, (c + 1) * PA_ROWS, last - c, PA_ROWS};
        }
        if (!again) break;
        __syncthreads();
    }
}

// Joins the pieces of split items, one warp per row: entries in turn over
// blockIdx.x, rows over blockIdx.y.  The pieces have just been written and lie
// in L2: what a row costs is the round trip to it.
template <int D, bool BF>
__global__ void __launch_bounds__(256) paged_join_kernel(const PagedParams p, int tile_rows, const int *count, int max_entries) {
    wait_for_primary();
    const int entries = count != nullptr ? min(*count, max_entries) : max_entries;
    const int lane = threadIdx.x & 31, warps = gridDim.y * (blockDim.x >> 5);
    for (int i = blockIdx.x; i < entries; i += gridDim.x) {
        const SplitEntry e = p.entries[i];
        if (e.count == 0) continue;
        const PagedSeq s = paged_seq(p, e.n, false);
        const int rows = min(tile_rows, s.nq * p.G - e.t * tile_rows);
        for (int r = blockIdx.y * (blockDim.x >> 5) + (threadIdx.x >> 5); r < rows; r += warps) {
            auto at = [&](int k) { return (long long)(k == 0 ? e.head : e.next + (k - 1) * e.stride) + r; };
            // pieces four at a time with a running maximum, so that a row's loads are one round trip
            constexpr int V = D / 32;
            float M = -INFINITY, L = 0.f, a[V] = {};
            for (int k0 = 0; k0 <= e.count; k0 += 4) {
                float2 ml[4], y[4][V / 2];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const bool in = k0 + k <= e.count;
                    const long long x0 = at(in ? k0 + k : k0), x = KDA_CHECK(p.st, x0 >= 0 && x0 < p.part_rows) ? x0 : 0;
                    ml[k] = __ldcg(p.part_ml + x);
                    if (!in) ml[k] = make_float2(-INFINITY, 0.f);
#pragma unroll
                    for (int j = 0; j < V / 2; ++j) y[k][j] = __ldcg(reinterpret_cast<const float2 *>(p.part_o + x * D + lane * V) + j);
                }
                const float Mn = fmaxf(fmaxf(fmaxf(ml[0].x, ml[1].x), fmaxf(ml[2].x, ml[3].x)), M), ref = Mn == -INFINITY ? 0.f : Mn;
                const float f0 = ex2(M - ref);
                M = Mn;
                L *= f0;
#pragma unroll
                for (int j = 0; j < V; ++j) a[j] *= f0;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float f = ex2(ml[k].x - ref);
                    L += f * ml[k].y;
#pragma unroll
                    for (int j = 0; j < V / 2; ++j) {
                        a[2 * j] += f * y[k][j].x;
                        a[2 * j + 1] += f * y[k][j].y;
                    }
                }
            }
            const float inv = L == 0.f ? 0.f : 1.f / L;
            const int row = e.t * tile_rows + r, head = e.h * p.G + row % p.G;
            const long long tok = s.q0 + row / p.G;
            if (!KDA_CHECK(p.st, tok < p.total_q && head < p.Hq)) continue;
#pragma unroll
            for (int j = 0; j < V; j += 2)
                *reinterpret_cast<uint32_t *>(p.out + (tok * p.Hq + head) * D + lane * V + j) =
                    pack16x2<BF>(a[j] * inv, a[j + 1] * inv);
            if (p.lse != nullptr && lane == 0)
                p.lse[tok * p.Hq + head] = row_lse(M, L);
        }
    }
}

// ------------------------------------------------------------------- host ----
int paged_rows_slots(int ctas) { return 2 * ctas; }
int paged_rows_ctas_per_sm(int d) { return d == 128 ? 2 : 3; }
int paged_rows_tile() { return PA_ROWS; }

template <int D, bool BF, bool WHOLE>
static cudaError_t launch_rows_t(const PagedParams &p, int ctas, cudaStream_t stream) {
    const cudaError_t e = allow_smem(paged_rows_kernel<D, BF, WHOLE>, PaShape<D>::SMEM);
    if (e != cudaSuccess) return e;
    paged_rows_kernel<D, BF, WHOLE><<<ctas, PA_THREADS, PaShape<D>::SMEM, stream>>>(p);
    return cudaGetLastError();
}
template <int D, bool BF>
static cudaError_t launch_join_t(const PagedParams &p, const int *count, int max_entries, int tile_rows, int sms, cudaStream_t stream) {
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    // blocks of eight warps over an item's rows: of 256 rows a warp takes two, one after the other (four, with
    // half the blocks and twice the entries at once: 0.6 us more)
    const int groups = tile_rows > 64 ? 16 : 2, entries = tile_rows > 64 ? sms : 2 * sms;
    cfg.gridDim = dim3(max_entries < entries ? max_entries : entries, groups);
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, paged_join_kernel<D, BF>, p, tile_rows, count, max_entries);
}

cudaError_t launch_paged_rows(const PagedParams &p, int d, bool bf, bool whole, int ctas, cudaStream_t stream) {
    if (d == 128) {
        if (whole) return bf ? launch_rows_t<128, true, true>(p, ctas, stream) : launch_rows_t<128, false, true>(p, ctas, stream);
        return bf ? launch_rows_t<128, true, false>(p, ctas, stream) : launch_rows_t<128, false, false>(p, ctas, stream);
    }
    if (whole) return bf ? launch_rows_t<64, true, true>(p, ctas, stream) : launch_rows_t<64, false, true>(p, ctas, stream);
    return bf ? launch_rows_t<64, true, false>(p, ctas, stream) : launch_rows_t<64, false, false>(p, ctas, stream);
}
// count: entries, on the device, or NULL for max_entries of them (some with count 0).
cudaError_t launch_paged_join(const PagedParams &p, int d, bool bf, const int *count, int max_entries, int tile_rows, int sms,
                              cudaStream_t stream) {
    if (d == 128)
        return bf ? launch_join_t<128, true>(p, count, max_entries, tile_rows, sms, stream)
                  : launch_join_t<128, false>(p, count, max_entries, tile_rows, sms, stream);
    return bf ? launch_join_t<64, true>(p, count, max_entries, tile_rows, sms, stream)
              : launch_join_t<64, false>(p, count, max_entries, tile_rows, sms, stream);
}

}  // namespace kda
