// Backward of the selective scan.  With yb' = yb silu(z) and, from the last
// row to the first,
//   g_t = C_t yb'_t + a_{t+1} g_{t+1},   q_t = g_t a_t h_{t-1}
// the cotangents are
//   xb = dt' (g . B) + D yb'        dt'b = x (g . B) + q . A     Ab = sum_t q dt'
//   Bb = sum_d g dt' x              Cb = sum_d h yb'             Db = sum_t yb' x
//   zb = yb silu'(z) (h . C + D x)  dtb = dt'b softplus'(dt + dt_bias).
// A block works on SCAN_WARPS neighbouring warp tiles of channels and one
// segment of a line, SCAN_R rows at a time from the end: the states inside
// come again from the one kept before those rows, and wait in shared memory.
// The sums over channels (Bb, Cb) leave a block as one partial sum per row,
// those over rows (Ab, Db, dt_biasb) as one per segment; scan_sums_kernel
// adds them in a fixed order.
#pragma once

#include "scan.cuh"

namespace selinv {
namespace {

template <class K> struct ScanBwdSmem {
    using C = typename K::C;
    C dt[SCAN_R][K::PITCH], u[SCAN_R][K::PITCH], yb[SCAN_R][K::PITCH];
    C gb[SCAN_R][K::PITCH], qa[SCAN_R][K::PITCH], hc[SCAN_R][K::PITCH];
    C bc[SCAN_R][2 * K::NP];                                     // this warp's sums for Bb and Cb
    typename K::V h[SCAN_R][K::TP * K::TN / 2][32][2];           // states after each row, by thread
};
template <class K> struct ScanBwdBlock {
    using C = typename K::C;
    ScanBwdSmem<K> warp[SCAN_WARPS];
    C b[SCAN_R][2 * K::NP], c[SCAN_R][2 * K::NP];
};

// MAIN: all outputs.  Otherwise only what each segment hands to the row before it: a g from nothing behind it, and the
// sum of its steps.
template <class K, bool MAIN>
__global__ void __launch_bounds__(SCAN_WARPS * 32)
    scan_backward_kernel(const __grid_constant__ ScanArgs p, const __grid_constant__ ScanGrads o)
{
    using T = typename K::T;
    using C = typename K::C;
    using V = typename K::V;
    constexpr int R = SCAN_R, CW = K::CW, E = K::E, EB = K::EB, NP = K::NP, TD = K::TD, TN = K::TN, TP = K::TP;
    extern __shared__ __align__(16) char smem_raw[];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    ScanBwdBlock<K> &block = *reinterpret_cast<ScanBwdBlock<K> *>(smem_raw);
    ScanBwdSmem<K> *all = block.warp;
    ScanBwdSmem<K> &sm = all[warp];
    ScanPlace w;
    scan_place<K>(p, warp, w);              // a warp without channels (nch <= 0) still meets the others
    const int nch = max(w.nch, 0);
    if (nch == 0) w.c0 = 0;                 // its addresses are never used

    const int n = p.n, d0 = (lane / K::LN) * TD, n0 = (lane % K::LN) * TN;
    const T *x = static_cast<const T *>(p.x.p) + w.line * p.x.line + w.c0;
    const T *dt = static_cast<const T *>(p.dt.p) + w.line * p.dt.line + w.c0;
    const T *z = p.z.p ? static_cast<const T *>(p.z.p) + w.line * p.z.line + w.c0 : nullptr;
    const T *B = static_cast<const T *>(p.B.p) + w.line * p.B.line + w.group * p.B_group;
    const T *Cc = static_cast<const T *>(p.C.p) + w.line * p.C.line + w.group * p.C_group;
    const T *yb = static_cast<const T *>(o.yb.p) + w.line * o.yb.line + w.c0;
    T *xb = static_cast<T *>(o.xb.p) + w.line * o.xb.line + w.c0;
    T *dtb = static_cast<T *>(o.dtb.p) + w.line * o.dtb.line + w.c0;
    T *zb = o.zb.p ? static_cast<T *>(o.zb.p) + w.line * o.zb.line + w.c0 : nullptr;
    const int64_t part = (int64_t)w.c0 * n, dn = p.d * n;
    const C *state = static_cast<const C *>(p.state), *stateb = static_cast<const C *>(o.stateb);
    C *stateb_out = static_cast<C *>(o.stateb_out);

    if (MAIN && stateb_out && p.rows.table && blockIdx.x == 0) {
        for (int64_t e = 0; e < p.sequences - p.rows.live; ++e) {
            const int64_t at = p.rows.table[2 * p.rows.live + 1 + e] * dn + part;
            for (int i = lane; i < nch * n; i += 32) stateb_out[at + i] = stateb ? stateb[at + i] : (C)0;
        }
    }

    V A2[TP][TN], g[TP][TN], ab[TP][TN];       // g: what the row behind hands on, a_{t+1} g_{t+1}
    load_part<K>(static_cast<const C *>(p.A) + part, n, nch, lane, A2, (C)0);
#pragma unroll
    for (int q = 0; q < TP; ++q)
#pragma unroll
        for (int j = 0; j < TN; ++j) {
            A2[q][j] = mul2(A2[q][j], make2(log2e<C>(), log2e<C>()));
            g[q][j] = ab[q][j] = make2((C)0, (C)0);
        }
    const int ce = (lane % (CW / E)) * E;
    C bias[E], skip[E], sum_d[E], sum_bias[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const bool in = ce + e < nch;
        bias[e] = in && p.dt_bias ? static_cast<const C *>(p.dt_bias)[w.c0 + ce + e] : (C)0;
        skip[e] = in && p.D ? static_cast<const C *>(p.D)[w.c0 + ce + e] : (C)0;
        sum_d[e] = sum_bias[e] = 0;
    }
    V total[TP];
#pragma unroll
    for (int q = 0; q < TP; ++q) total[q] = make2((C)0, (C)0);

    int64_t k = w.r1 > w.r0 ? p.rows.find(w.r1 - 1) : 0;     // the sequence of the row at hand
    if (MAIN && w.r1 > w.r0 && p.rows.end(k) > w.r1) {
        // what the segments behind this one hand on, from the last that holds rows of this sequence
        const C *ends = static_cast<const C *>(p.ends) + w.line * p.segs * dn + part;
        const C *sums = static_cast<const C *>(p.sums) + w.line * p.segs * p.d + w.c0;
        int s = (int)((p.rows.end(k) - 1) / p.seg_rows);
        load_part<K>(ends + s * dn, n, nch, lane, g, (C)0);
        for (--s; s > w.seg; --s) {
            V e[TP][TN];
            load_part<K>(ends + s * dn, n, nch, lane, e, (C)0);
#pragma unroll
            for (int q = 0; q < TP; ++q) {
                V t;
                t.x = d0 + 2 * q < nch ? sums[s * p.d + d0 + 2 * q] : (C)0;
                t.y = d0 + 2 * q + 1 < nch ? sums[s * p.d + d0 + 2 * q + 1] : (C)0;
#pragma unroll
                for (int j = 0; j < TN; ++j) {
                    const V a = mul2(t, A2[q][j]);
                    g[q][j] = fma2(make2(exp2_(a.x), exp2_(a.y)), g[q][j], e[q][j]);
                }
            }
        }
    }
    const bool pad_n = n < NP;
    const int64_t tiles = (p.rows.rows + R - 1) / R;

    for (int64_t rt = w.r0 + (w.r1 > w.r0 ? (w.r1 - w.r0 - 1) / R * R : 0); rt >= w.r0 && rt < w.r1; rt -= R) {
        const int nr = (int)min((int64_t)R, w.r1 - rt);
        // the live sequence of this tile's first row, and the rows that begin one
        int64_t k0 = k;
        while (p.rows.start(k0) > rt) --k0;
        const uint32_t st = p.rows.starts(rt, R, k0, lane);
        // stage
#pragma unroll
        for (int i = 0; i < K::PER; ++i) {
            const int row = (lane + 32 * i) / (CW / E);
            if (row >= R) break;
            C a[E], b[E], c[E];
            Pack<T, E> xv, dv, yv, zv;
            xv.clear(), dv.clear(), yv.clear(), zv.clear();
            if (row < nr && nch > 0) {
                xv.load(x + (rt + row) * p.x.row + ce, nch - ce, p.x.wide);
                dv.load(dt + (rt + row) * p.dt.row + ce, nch - ce, p.dt.wide);
                yv.load(yb + (rt + row) * o.yb.row + ce, nch - ce, o.yb.wide);
                if (z) zv.load(z + (rt + row) * p.z.row + ce, nch - ce, p.z.wide);
            }
#pragma unroll
            for (int e = 0; e < E; ++e) {
                a[e] = dv.get(e) + bias[e];
                if (p.softplus) a[e] = softplus_(a[e]);
                b[e] = a[e] * xv.get(e);
                c[e] = yv.get(e);
                if (z) c[e] *= zv.get(e) * sigmoid_(zv.get(e));
            }
            put<E>(&sm.dt[row][ce], a);
            put<E>(&sm.u[row][ce], b);
            put<E>(&sm.yb[row][ce], c);
        }
#pragma unroll
        for (int i = 0; i < (K::BVECS + SCAN_WARPS * 32 - 1) / (SCAN_WARPS * 32); ++i) {
            const int vec = threadIdx.x + SCAN_WARPS * 32 * i, row = vec / (NP / EB), e0 = (vec % (NP / EB)) * EB;
            if (row >= R) break;
            C a[2 * EB], b[2 * EB];
            Pack<T, EB> bv, cv;
            bv.clear(), cv.clear();
            if (row < nr) {
                if (MAIN) bv.load(B + (rt + row) * p.B.row + e0, n - e0, p.B.wide);
                cv.load(Cc + (rt + row) * p.C.row + e0, n - e0, p.C.wide);
            }
#pragma unroll
            for (int e = 0; e < EB; ++e) {
                a[2 * e] = a[2 * e + 1] = bv.get(e);
                b[2 * e] = b[2 * e + 1] = cv.get(e);
            }
            if (MAIN) put<2 * EB>(&block.b[row][2 * e0], a);
            put<2 * EB>(&block.c[row][2 * e0], b);
        }
        __syncthreads();
        V h[TP][TN];
        if (MAIN) {
            // the states after each row but the last, again
            load_part<K>(static_cast<const C *>(o.kept) + (w.line * tiles + rt / R) * dn + part, n, nch, lane, h, (C)0);
            int64_t kk = k0;
            for (int t = 0; t < nr; ++t) {
                if ((st >> t) & 1u) {
                    if (rt + t > p.rows.start(kk)) ++kk;
                    if (state) {
                        load_part<K>(state + p.rows.number(kk, w.line) * dn + part, n, nch, lane, h, (C)0);
                    } else {
#pragma unroll
                        for (int q = 0; q < TP; ++q)
#pragma unroll
                            for (int j = 0; j < TN; ++j) h[q][j] = make2((C)0, (C)0);
                    }
                }
                V dt2[TP], u2[TP], b2[TN];
                get<TP>(&sm.dt[t][d0], dt2);
                get<TP>(&sm.u[t][d0], u2);
                get<TN>(&block.b[t][2 * n0], b2);
#pragma unroll
                for (int q = 0; q < TP; ++q)
#pragma unroll
                    for (int j = 0; j < TN; ++j) {
                        const V e = mul2(dt2[q], A2[q][j]);
                        h[q][j] = fma2(make2(exp2_(e.x), exp2_(e.y)), h[q][j], mul2(u2[q], b2[j]));
                        if (pad_n && n0 + j >= n) h[q][j] = make2((C)0, (C)0);
                    }
#pragma unroll
                for (int i = 0; i < TP * TN; ++i) sm.h[t][i / 2][lane][i % 2] = h[i / TN][i % TN];
            }
        }
        // from the last row to the first
        for (int t = nr - 1; t >= 0; --t) {
            if ((st >> (t + 1)) & 1u) {         // the last row of its sequence
                if (rt + t < p.rows.start(k)) --k;
                if (stateb) {
                    load_part<K>(stateb + p.rows.number(k, w.line) * dn + part, n, nch, lane, g, (C)0);
                } else {
#pragma unroll
                    for (int q = 0; q < TP; ++q)
#pragma unroll
                        for (int j = 0; j < TN; ++j) g[q][j] = make2((C)0, (C)0);
                }
            }
            const bool first = (st >> t) & 1u;
            V dt2[TP], yb2[TP], c2[TN];
            get<TP>(&sm.dt[t][d0], dt2);
            get<TP>(&sm.yb[t][d0], yb2);
            get<TN>(&block.c[t][2 * n0], c2);
            if constexpr (!MAIN) {
#pragma unroll
                for (int q = 0; q < TP; ++q) {
#pragma unroll
                    for (int j = 0; j < TN; ++j) {
                        const V e = mul2(dt2[q], A2[q][j]);
                        g[q][j] = mul2(make2(exp2_(e.x), exp2_(e.y)), fma2(c2[j], yb2[q], g[q][j]));
                    }
                    total[q] = add2(total[q], dt2[q]);
                }
            } else {
                V u2[TP], b2[TN], past[TP][TN], gb[TP], qa[TP], hc[TP];
                C bc[2 * TN];
                get<TP>(&sm.u[t][d0], u2);
                get<TN>(&block.b[t][2 * n0], b2);
                if (first) {
                    if (state) {
                        load_part<K>(state + p.rows.number(k, w.line) * dn + part, n, nch, lane, past, (C)0);
                    } else {
#pragma unroll
                        for (int q = 0; q < TP; ++q)
#pragma unroll
                            for (int j = 0; j < TN; ++j) past[q][j] = make2((C)0, (C)0);
                    }
                } else if (t > 0) {
#pragma unroll
                    for (int i = 0; i < TP * TN; ++i) past[i / TN][i % TN] = sm.h[t - 1][i / 2][lane][i % 2];
                } else {
                    load_part<K>(static_cast<const C *>(o.kept) + (w.line * tiles + rt / R) * dn + part, n, nch, lane,
                                 past, (C)0);
                }
#pragma unroll
                for (int q = 0; q < TP; ++q) gb[q] = qa[q] = hc[q] = make2((C)0, (C)0);
#pragma unroll
                for (int j = 0; j < TN; ++j) {
                    V sb = make2((C)0, (C)0), sc = make2((C)0, (C)0);
#pragma unroll
                    for (int q = 0; q < TP; ++q) {
                        const V e = mul2(dt2[q], A2[q][j]);
                        const V a = make2(exp2_(e.x), exp2_(e.y));
                        const V gt = fma2(c2[j], yb2[q], g[q][j]);
                        sb = fma2(gt, u2[q], sb);
                        sc = fma2(h[q][j], yb2[q], sc);
                        gb[q] = fma2(gt, b2[j], gb[q]);
                        hc[q] = fma2(h[q][j], c2[j], hc[q]);
                        g[q][j] = mul2(a, gt);
                        const V m = mul2(g[q][j], past[q][j]);
                        qa[q] = fma2(m, A2[q][j], qa[q]);
                        ab[q][j] = fma2(m, dt2[q], ab[q][j]);
                        h[q][j] = past[q][j];
                        if (pad_n && n0 + j >= n) g[q][j] = make2((C)0, (C)0);
                    }
                    bc[j] = sb.x + sb.y, bc[TN + j] = sc.x + sc.y;
                }
                if (first) {
                    if (stateb_out) store_part<K>(stateb_out + p.rows.number(k, w.line) * dn + part, n, nch, lane, g);
                    // the row before is another sequence's last
                    if (t > 0) {
#pragma unroll
                        for (int i = 0; i < TP * TN; ++i) h[i / TN][i % TN] = sm.h[t - 1][i / 2][lane][i % 2];
                    }
                }
                scatter_sum<2 * TN, K::LN, 32>(bc, lane);
                {
                    constexpr int KEEP = 2 * TN > K::LD ? 2 * TN / K::LD : 1;
                    if (scatter_writes<2 * TN, K::LN, 32>(lane)) {
                        const int f = scatter_first<2 * TN, K::LN, 32>(lane);
#pragma unroll
                        for (int i = 0; i < KEEP; ++i) sm.bc[t][((f + i) / TN) * NP + n0 + (f + i) % TN] = bc[i];
                    }
                }
                C v[TD * 2], y1[TD];
#pragma unroll
                for (int q = 0; q < TP; ++q) {
                    v[2 * q] = gb[q].x, v[2 * q + 1] = gb[q].y;
                    v[TD + 2 * q] = qa[q].x, v[TD + 2 * q + 1] = qa[q].y;
                    y1[2 * q] = hc[q].x, y1[2 * q + 1] = hc[q].y;
                }
                scatter_sum<2 * TD, 1, K::LN>(v, lane);
                {
                    constexpr int KEEP = 2 * TD > K::LN ? 2 * TD / K::LN : 1;
                    if (scatter_writes<2 * TD, 1, K::LN>(lane)) {
                        const int f = scatter_first<2 * TD, 1, K::LN>(lane);
#pragma unroll
                        for (int i = 0; i < KEEP; ++i) {
                            if (f + i < TD)
                                sm.gb[t][d0 + f + i] = v[i];
                            else
                                sm.qa[t][d0 + f + i - TD] = v[i] * ln2<C>();
                        }
                    }
                }
                if (z) {
                    scatter_sum<TD, 1, K::LN>(y1, lane);
                    constexpr int KEEP = TD > K::LN ? TD / K::LN : 1;
                    if (scatter_writes<TD, 1, K::LN>(lane)) {
                        const int f = scatter_first<TD, 1, K::LN>(lane);
#pragma unroll
                        for (int i = 0; i < KEEP; ++i) sm.hc[t][d0 + f + i] = y1[i];
                    }
                }
            }
        }
        k = k0;
        __syncthreads();
        if constexpr (MAIN) {
#pragma unroll
            for (int i = 0; i < K::PER; ++i) {
                const int row = (lane + 32 * i) / (CW / E);
                if (row >= nr || nch == 0) break;
                Pack<T, E> xv, dv, yv, zv, out;
                xv.load(x + (rt + row) * p.x.row + ce, nch - ce, p.x.wide);
                dv.load(dt + (rt + row) * p.dt.row + ce, nch - ce, p.dt.wide);
                C s[E], gb[E], qa[E], hc[E], xo[E], so[E], zo[E], ys[E];
                get<E>(&sm.dt[row][ce], s);
                get<E>(&sm.yb[row][ce], ys);
                get<E>(&sm.gb[row][ce], gb);
                get<E>(&sm.qa[row][ce], qa);
                if (z) {
                    get<E>(&sm.hc[row][ce], hc);
                    yv.load(yb + (rt + row) * o.yb.row + ce, nch - ce, o.yb.wide);
                    zv.load(z + (rt + row) * p.z.row + ce, nch - ce, p.z.wide);
                }
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    const C xe = xv.get(e);
                    xo[e] = gb[e] * s[e] + skip[e] * ys[e];
                    so[e] = gb[e] * xe + qa[e];
                    if (p.softplus) so[e] *= sigmoid_(dv.get(e) + bias[e]);
                    sum_d[e] += ys[e] * xe;
                    sum_bias[e] += so[e];
                    if (z) {
                        const C ze = zv.get(e);
                        zo[e] = yv.get(e) * (hc[e] + skip[e] * xe) * silu_slope(ze, sigmoid_(ze));
                    }
                }
                out.set(xo);
                out.store(xb + (rt + row) * o.xb.row + ce, nch - ce, o.xb.wide);
                out.set(so);
                out.store(dtb + (rt + row) * o.dtb.row + ce, nch - ce, o.dtb.wide);
                if (z) {
                    out.set(zo);
                    out.store(zb + (rt + row) * o.zb.row + ce, nch - ce, o.zb.wide);
                }
            }
            // Bb and Cb: the block's warps, in order, into this block's partial sums [blocks of a group][line, row][group]
            const int per = (int)(p.d / p.groups), tiles_c = (per + CW - 1) / CW;
            const int blocks = (tiles_c + SCAN_WARPS - 1) / SCAN_WARPS;
            const int64_t all_rows = p.lines * p.rows.rows;
            C *out = static_cast<C *>(o.part_bc) +
                     (((int64_t)((int)blockIdx.y % blocks) * all_rows + w.line * p.rows.rows + rt) * p.groups + w.group) * 2 * NP;
            const int live = min(SCAN_WARPS, tiles_c - ((int)blockIdx.y % blocks) * SCAN_WARPS);
            for (int i = threadIdx.x; i < nr * 2 * NP; i += SCAN_WARPS * 32) {
                const int t = i / (2 * NP), j = i % (2 * NP);
                C v = all[0].bc[t][j];
                for (int a = 1; a < live; ++a) v += all[a].bc[t][j];
                out[(int64_t)t * p.groups * 2 * NP + j] = v;
            }
            __syncthreads();
        }
    }
    if (nch == 0) return;
    const int64_t at = w.line * p.segs + w.seg;
    if constexpr (!MAIN) {
        C *ends = static_cast<C *>(p.ends) + at * dn + part;
        C *sums = static_cast<C *>(p.sums) + at * p.d + w.c0;
        store_part<K>(ends, n, nch, lane, g);
        if (lane % K::LN == 0) {
#pragma unroll
            for (int q = 0; q < TP; ++q) {
                if (d0 + 2 * q < nch) sums[d0 + 2 * q] = total[q].x;
                if (d0 + 2 * q + 1 < nch) sums[d0 + 2 * q + 1] = total[q].y;
            }
        }
    } else {
        store_part<K>(static_cast<C *>(o.part_a) + at * dn + part, n, nch, lane, ab);
        // lanes that converted the same channels
#pragma unroll
        for (int e = 0; e < E; ++e) {
#pragma unroll
            for (int m = CW / E; m < 32; m *= 2) {
                sum_d[e] += shfl_xor_(sum_d[e], m);
                sum_bias[e] += shfl_xor_(sum_bias[e], m);
            }
            if (lane < CW / E && ce + e < nch) {
                static_cast<C *>(o.part_d)[at * p.d + w.c0 + ce + e] = sum_d[e];
                static_cast<C *>(o.part_bias)[at * p.d + w.c0 + ce + e] = sum_bias[e];
            }
        }
    }
}

// Bb and Cb from the blocks' sums, and Ab, Db, dt_biasb from the segments': the first `bc_blocks` blocks take one
// (row, group) entry of B and C per thread, the others 32 parameters each, in 8 strands of segments; every sum in
// one order.
template <class T, int NP>
__global__ void __launch_bounds__(256)
    scan_sums_kernel(const __grid_constant__ ScanArgs p, const __grid_constant__ ScanGrads o, int64_t bc_blocks, int parts)
{
    using C = typename Elem<T>::C;
    const int64_t rows = p.lines * p.rows.rows;
    if (blockIdx.x < bc_blocks) {
        const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, total = rows * p.groups * 2 * NP;
        if (i >= total) return;
        const int j = (int)(i % (2 * NP)), m = j % NP;
        const int64_t at = i / (2 * NP), r = at / p.groups, g = at % p.groups;
        if (m >= p.n) return;
        C v = 0;
        for (int b = 0; b < parts; ++b) v += static_cast<const C *>(o.part_bc)[b * total + i];
        const int64_t line = r / p.rows.rows, row = r % p.rows.rows;
        const Out &out = j < NP ? o.Bb : o.Cb;
        const int64_t gs = j < NP ? o.Bb_group : o.Cb_group;
        static_cast<T *>(out.p)[line * out.line + row * out.row + g * gs + m] = Elem<T>::down(v);
        return;
    }
    __shared__ C s[8][32];
    const int64_t dn = p.d * p.n, i = ((int64_t)blockIdx.x - bc_blocks) * 32 + threadIdx.x % 32;
    const int strand = threadIdx.x / 32;
    const C *from = nullptr;
    C *to = nullptr;
    int64_t stride = 0;
    if (i < dn) {
        from = static_cast<const C *>(o.part_a) + i, to = static_cast<C *>(o.Ab) + i, stride = dn;
    } else if (i < dn + p.d) {
        from = static_cast<const C *>(o.part_d) + (i - dn), stride = p.d;
        to = o.Db ? static_cast<C *>(o.Db) + (i - dn) : nullptr;
    } else if (i < dn + 2 * p.d) {
        from = static_cast<const C *>(o.part_bias) + (i - dn - p.d), stride = p.d;
        to = o.dt_biasb ? static_cast<C *>(o.dt_biasb) + (i - dn - p.d) : nullptr;
    }
    C v = 0;
    if (to)
        for (int64_t e = strand; e < p.lines * p.segs; e += 8) v += from[e * stride];
    s[strand][threadIdx.x % 32] = v;
    __syncthreads();
    if (strand == 0 && to) {
        for (int e = 1; e < 8; ++e) v += s[e][threadIdx.x];
        *to = v;
    }
}

// Blocks of one group of channels: how many partial sums of B and C there are.
template <class K> int scan_parts(const ScanArgs &p)
{
    const int64_t per = p.d / p.groups, tiles = (per + K::CW - 1) / K::CW;
    return (int)((tiles + SCAN_WARPS - 1) / SCAN_WARPS);
}

template <class K> cudaError_t scan_backward_run(const ScanArgs &p, const ScanGrads &o, cudaStream_t s)
{
    const int parts = scan_parts<K>(p);
    const dim3 grid((unsigned)(p.lines * p.segs), (unsigned)(p.groups * parts));
    static_assert(sizeof(ScanBwdSmem<K>) % 16 == 0 && offsetof(ScanBwdSmem<K>, h) % 16 == 0 &&
                      offsetof(ScanBwdBlock<K>, b) % 16 == 0 && offsetof(ScanBwdBlock<K>, c) % 16 == 0,
                  "staged rows lie on 16 bytes");
    constexpr int bytes = (int)sizeof(ScanBwdBlock<K>);
    static_assert(bytes <= 227 * 1024, "fits an SM");
    if (p.segs > 1) {
        cudaError_t e =
            cudaFuncSetAttribute(scan_backward_kernel<K, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != cudaSuccess) return e;
        scan_backward_kernel<K, false><<<grid, SCAN_WARPS * 32, bytes, s>>>(p, o);
    }
    cudaError_t e =
        cudaFuncSetAttribute(scan_backward_kernel<K, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    scan_backward_kernel<K, true><<<grid, SCAN_WARPS * 32, bytes, s>>>(p, o);
    const int64_t bc = (p.lines * p.rows.rows * p.groups * 2 * K::NP + 255) / 256;
    const int64_t params = (p.d * (p.n + 2) + 31) / 32;
    scan_sums_kernel<typename K::T, K::NP><<<(unsigned)(bc + params), 256, 0, s>>>(p, o, bc, parts);
    return cudaGetLastError();
}

}  // namespace
}  // namespace selinv
