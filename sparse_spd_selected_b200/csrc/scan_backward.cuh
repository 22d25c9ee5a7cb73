// Backward of the selective scan.  With yb' = yb silu(z) and, from the last
// row to the first,
//   g_t = C_t yb'_t + a_{t+1} g_{t+1},   q_t = g_t a_t h_{t-1}
// the cotangents are
//   xb = dt' (g . B) + D yb'        dt'b = x (g . B) + q . A     Ab = sum_t q dt'
//   Bb = sum_d g dt' x              Cb = sum_d h yb'             Db = sum_t yb' x
//   zb = yb silu'(z) (h . C + D x)  dtb = dt'b softplus'(dt + dt_bias).
// A block works on SCAN_WARPS neighbouring warp tiles of channels and one
// segment of a line, SCAN_R rows at a time from the end.  The states inside
// come again from the one kept before those rows: a first run leaves every
// SCAN_S-th in shared memory, a second one fills the registers with the
// states and decays of SCAN_S rows, which the backward recurrence then uses
// up.  The sums over states and over channels go through shared memory, not
// shuffles: one store of 16 bytes per thread and row, added by the lanes that
// finish the rows.  The sums over channels (Bb, Cb) leave a block as one
// partial sum per row, those over rows (Ab, Db, dt_biasb) as one per segment;
// scan_sums_kernel adds them in a fixed order.
#pragma once

#include "scan.cuh"

namespace selinv {
namespace {

constexpr int SCAN_S = 4;       // rows whose states and decays are in registers together

template <class K> struct ScanBwdSmem {
    using C = typename K::C;
    using V = typename K::V;
    C dt[SCAN_R][K::CW], u[SCAN_R][K::CW], yb[SCAN_R][K::CW];
    C gb[SCAN_S][K::LN][K::CW], qa[SCAN_S][K::LN][K::CW], hc[SCAN_S][K::LN][K::CW];     // parts of the sums over states
    C part[SCAN_S][K::LN][2 * K::TN / K::TD][K::LD][K::TD];     // parts of the sums over channels: B's states, then C's
    C bc[SCAN_R][2 * K::NP];                                    // those sums of this warp
    V h[SCAN_R / SCAN_S - 1][K::TP * K::TN][32];                // states before rows SCAN_S, 2 SCAN_S, ...
};
template <class K> struct ScanBwdBlock {
    using C = typename K::C;
    ScanBwdSmem<K> warp[SCAN_WARPS];
    C b[SCAN_R][2 * K::NP], c[SCAN_R][2 * K::NP];
};

// a and h of row t.
template <class K, bool POLY, int ROW>
SELINV_DEVINL void scan_again(const ScanBwdSmem<K> &sm, const ScanBwdBlock<K> &block, int t, int d0, int n0, int n,
                              const typename K::V (*A2)[K::TN], typename K::V (*h)[K::TN], typename K::V (*a)[K::TN])
{
    using V = typename K::V;
    using C = typename K::C;
    V dt2[K::TP], u2[K::TP], b2[K::TN];
    get<K::TP>(&sm.dt[t][d0], dt2);
    get<K::TP>(&sm.u[t][d0], u2);
    get<K::TN>(&block.b[t][2 * n0], b2);
    scan_pairs<K, POLY, ROW>([&](auto poly, int q, int j) {
        a[q][j] = decay2<poly.value>(mul2(dt2[q], A2[q][j]));
        h[q][j] = fma2(a[q][j], h[q][j], mul2(u2[q], b2[j]));
    });
    if (n < K::NP) {
#pragma unroll
        for (int j = 0; j < K::TN; ++j)
            if (n0 + j >= n) {
#pragma unroll
                for (int q = 0; q < K::TP; ++q) h[q][j] = make2((C)0, (C)0);
            }
    }
}

// What a thread of the backward knows of its place.
template <class K> struct ScanBwd {
    using T = typename K::T;
    using C = typename K::C;
    using V = typename K::V;
    const ScanArgs &p;
    const ScanGrads &o;
    ScanBwdBlock<K> &block;
    ScanBwdSmem<K> &sm;
    int lane, nl, d0, n0, nch;
    int64_t line, part, dn;         // part: the warp's first channel in a [d, n] array

    SELINV_DEVINL void states(const void *from, int64_t sequence, V (*v)[K::TN]) const
    {
        if (from)
            load_part<K>(static_cast<const C *>(from) + p.rows.number(sequence, line) * dn + part, p.n, nch, lane, v);
        else
            zero_part<K>(v);
    }
    // The live sequence of row t of a tile whose first row lies in k0; st: the rows that begin one.
    SELINV_DEVINL static int64_t sequence(int64_t k0, uint32_t st, int t) { return k0 + __popc(st & ((2u << t) - 2u)); }

    // Rows t0 .. t0 + SCAN_S - 1, `before` the state before them.  EDGE: some row begins or ends a sequence; st has the
    // rows that begin one and the row behind the last, of which only those below nr are rows.
    template <bool POLY, bool EDGE>
    SELINV_DEVINL void rows(int t0, int nr, uint32_t st, int64_t k0, const V (*A2)[K::TN], const V (*before)[K::TN], V (*g)[K::TN],
                            V (*ab)[K::TN]) const
    {
        constexpr int S = SCAN_S, TP = K::TP, TN = K::TN;
        V h[S][TP][TN], a[S][TP][TN];
        const uint32_t begins = st & ((1u << nr) - 1u);
        run<POLY, EDGE, 0>(t0, begins, k0, A2, before, h, a);
#pragma unroll
        for (int r = S - 1; r >= 0; --r) {
            const int t = t0 + r;
            if (EDGE && ((st >> (t + 1)) & 1u)) states(o.stateb, sequence(k0, st, t), g);
            const bool first = EDGE && ((begins >> t) & 1u);
            V start[TP][TN];
            if (EDGE) {
                if (first) {
                    states(p.state, sequence(k0, st, t), start);
                } else {
#pragma unroll
                    for (int q = 0; q < TP; ++q)
#pragma unroll
                        for (int j = 0; j < TN; ++j) start[q][j] = r > 0 ? h[r > 0 ? r - 1 : 0][q][j] : before[q][j];
                }
            }
            V dt2[TP], u2[TP], yb2[TP], b2[TN], c2[TN], gb[TP], qa[TP];
            get<TP>(&sm.dt[t][d0], dt2);
            get<TP>(&sm.u[t][d0], u2);
            get<TP>(&sm.yb[t][d0], yb2);
            get<TN>(&block.b[t][2 * n0], b2);
            get<TN>(&block.c[t][2 * n0], c2);
            C sum[2 * TN];
#pragma unroll
            for (int j = 0; j < TN; ++j) {
                V sb, sc;
#pragma unroll
                for (int q = 0; q < TP; ++q) {
                    const V past = EDGE ? start[q][j] : r > 0 ? h[r > 0 ? r - 1 : 0][q][j] : before[q][j];
                    const V gt = fma2(c2[j], yb2[q], g[q][j]);
                    sb = q ? fma2(gt, u2[q], sb) : mul2(gt, u2[q]);
                    sc = q ? fma2(h[r][q][j], yb2[q], sc) : mul2(h[r][q][j], yb2[q]);
                    gb[q] = j ? fma2(gt, b2[j], gb[q]) : mul2(gt, b2[j]);
                    g[q][j] = mul2(a[r][q][j], gt);
                    const V m = mul2(g[q][j], past);
                    qa[q] = j ? fma2(m, A2[q][j], qa[q]) : mul2(m, A2[q][j]);
                    ab[q][j] = fma2(m, dt2[q], ab[q][j]);
                }
                sum[j] = sb.x + sb.y, sum[TN + j] = sc.x + sc.y;
            }
            if (p.n < K::NP) {
#pragma unroll
                for (int j = 0; j < TN; ++j)
                    if (n0 + j >= p.n) {
#pragma unroll
                        for (int q = 0; q < TP; ++q) g[q][j] = make2((C)0, (C)0);
                    }
            }
            put<TP>(&sm.gb[r][nl][d0], gb);
            put<TP>(&sm.qa[r][nl][d0], qa);
            if (p.z.p) {
                V hc[TP];
#pragma unroll
                for (int q = 0; q < TP; ++q) {
                    hc[q] = mul2(c2[0], h[r][q][0]);
#pragma unroll
                    for (int j = 1; j < TN; ++j) hc[q] = fma2(c2[j], h[r][q][j], hc[q]);
                }
                put<TP>(&sm.hc[r][nl][d0], hc);
            }
#pragma unroll
            for (int i = 0; i < 2 * TN / K::TD; ++i) put<K::TD>(&sm.part[r][nl][i][lane % K::LD][0], sum + i * K::TD);
            if (first && o.stateb_out)
                store_part<K>(static_cast<C *>(o.stateb_out) + p.rows.number(sequence(k0, st, t), line) * dn + part, p.n, nch,
                              lane, g);
        }
    }
    // The states and decays of rows t0 + R on.
    template <bool POLY, bool EDGE, int R>
    SELINV_DEVINL void run(int t0, uint32_t st, int64_t k0, const V (*A2)[K::TN], const V (*before)[K::TN],
                           V (*h)[K::TP][K::TN], V (*a)[K::TP][K::TN]) const
    {
        if constexpr (R < SCAN_S) {
#pragma unroll
            for (int q = 0; q < K::TP; ++q)
#pragma unroll
                for (int j = 0; j < K::TN; ++j) h[R][q][j] = R ? h[R ? R - 1 : 0][q][j] : before[q][j];
            if (EDGE && ((st >> (t0 + R)) & 1u)) states(p.state, sequence(k0, st, t0 + R), h[R]);
            scan_again<K, POLY, R>(sm, block, t0 + R, d0, n0, p.n, A2, h[R], a[R]);
            run<POLY, EDGE, R + 1>(t0, st, k0, A2, before, h, a);
        }
    }
    // SCAN_S rows of the first run.
    template <bool POLY, bool EDGE, int R = 0>
    SELINV_DEVINL void skip(int t0, uint32_t st, int64_t k0, const V (*A2)[K::TN], V (*h)[K::TN]) const
    {
        if constexpr (R < SCAN_S) {
            V a[K::TP][K::TN];
            if (EDGE && ((st >> (t0 + R)) & 1u)) states(p.state, sequence(k0, st, t0 + R), h);
            scan_again<K, POLY, R>(sm, block, t0 + R, d0, n0, p.n, A2, h, a);
            skip<POLY, EDGE, R + 1>(t0, st, k0, A2, h);
        }
    }
};

template <class K>
__global__ void __launch_bounds__(SCAN_WARPS * 32)
    scan_backward_kernel(const __grid_constant__ ScanArgs p, const __grid_constant__ ScanGrads o)
{
    using T = typename K::T;
    using C = typename K::C;
    using V = typename K::V;
    constexpr int R = SCAN_R, S = SCAN_S, LN = K::LN, LD = K::LD, NP = K::NP, TD = K::TD, TN = K::TN, TP = K::TP;
    constexpr int PERS = S > LN ? S / LN : 1;       // rows of S that a lane finishes
    extern __shared__ __align__(16) char smem_raw[];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    ScanBwdBlock<K> &block = *reinterpret_cast<ScanBwdBlock<K> *>(smem_raw);
    ScanBwdSmem<K> &sm = block.warp[warp];
    ScanPlace w;
    scan_place<K>(p, warp, w);              // a warp without channels (nch <= 0) still meets the others
    w.nch = max(w.nch, 0);
    if (w.nch == 0) w.c0 = 0;               // its addresses are never used

    const int n = p.n, nl = lane / LD, d0 = (lane % LD) * TD, n0 = nl * TN, nd = w.nch - d0;
    const T *x = static_cast<const T *>(p.x.p) + w.line * p.x.line + w.c0 + d0;
    const T *dt = static_cast<const T *>(p.dt.p) + w.line * p.dt.line + w.c0 + d0;
    const T *z = p.z.p ? static_cast<const T *>(p.z.p) + w.line * p.z.line + w.c0 + d0 : nullptr;
    const T *B = static_cast<const T *>(p.B.p) + w.line * p.B.line + w.group * p.B_group;
    const T *Cc = static_cast<const T *>(p.C.p) + w.line * p.C.line + w.group * p.C_group;
    const T *yb = static_cast<const T *>(o.yb.p) + w.line * o.yb.line + w.c0 + d0;
    T *xb = static_cast<T *>(o.xb.p) + w.line * o.xb.line + w.c0 + d0;
    T *dtb = static_cast<T *>(o.dtb.p) + w.line * o.dtb.line + w.c0 + d0;
    T *zb = o.zb.p ? static_cast<T *>(o.zb.p) + w.line * o.zb.line + w.c0 + d0 : nullptr;
    const int64_t part = (int64_t)w.c0 * n, dn = p.d * n;
    const ScanBwd<K> at{p, o, block, sm, lane, nl, d0, n0, w.nch, w.line, part, dn};

    if (o.stateb_out && p.rows.table && blockIdx.x == 0) {      // sequences without rows
        C *out = static_cast<C *>(o.stateb_out);
        const C *in = static_cast<const C *>(o.stateb);
        for (int64_t e = 0; e < p.sequences - p.rows.live; ++e) {
            const int64_t a = p.rows.table[2 * p.rows.live + 1 + e] * dn + part;
            for (int i = lane; i < w.nch * n; i += 32) out[a + i] = in ? in[a + i] : (C)0;
        }
    }

    V A2[TP][TN], g[TP][TN], ab[TP][TN];       // g: what the row behind hands on, a_{t+1} g_{t+1}
    V bias[TP], skip[TP], sum_d[TP], sum_bias[TP];
    const bool plain = load_decay<K>(p.A, part, n, w.nch, lane, A2) && p.softplus;
    zero_part<K>(g);
    zero_part<K>(ab);
#pragma unroll
    for (int q = 0; q < TP; ++q) {
        bias[q] = pair_of<K>(p.dt_bias, w.c0 + d0, nd, q);
        skip[q] = pair_of<K>(p.D, w.c0 + d0, nd, q);
        sum_d[q] = sum_bias[q] = make2((C)0, (C)0);
    }
    int64_t k0 = w.r1 > w.r0 ? p.rows.find(w.r1 - 1) : 0;
    if (w.r1 > w.r0 && p.rows.end(k0) > w.r1)       // what the segments behind this one hand on
        scan_join<K>(p, w, (int)((p.rows.end(k0) - 1) / p.seg_rows), w.seg, -1, lane, A2, g);
    const int64_t tiles = (p.rows.rows + R - 1) / R;
    const int per = (int)(p.d / p.groups), tiles_c = (per + K::CW - 1) / K::CW;
    const int blocks = (tiles_c + SCAN_WARPS - 1) / SCAN_WARPS, bi = (int)blockIdx.y % blocks;
    const int live = min(SCAN_WARPS, tiles_c - bi * SCAN_WARPS);
    C *part_bc = static_cast<C *>(o.part_bc) +
                 (((int64_t)bi * p.lines + w.line) * p.rows.rows * p.groups + w.group) * 2 * NP;

    for (int64_t rt = w.r0 + (w.r1 > w.r0 ? (w.r1 - w.r0 - 1) / R * R : 0); rt >= w.r0 && rt < w.r1; rt -= R) {
        const int nr = (int)min((int64_t)R, w.r1 - rt);
        while (p.rows.start(k0) > rt) --k0;         // the live sequence of this tile's first row
        const uint32_t st = p.rows.starts(rt, R, k0, lane);
        // stage; rows that are not there (behind the last) change nothing: no step, no input, no cotangent
        {
            ScanLoad<K> xl, dl, yl, zl;
            ScanLoadN<K, SCAN_WARPS * 32> bl, cl;
            dl.load(dt, p.dt.row, rt, w.r1, nd, p.dt.wide, nl);
            xl.load(x, p.x.row, rt, w.r1, nd, p.x.wide, nl);
            yl.load(yb, o.yb.row, rt, w.r1, nd, o.yb.wide, nl);
            if (z) zl.load(z, p.z.row, rt, w.r1, nd, p.z.wide, nl);
            bl.load(B, p.B.row, rt, w.r1, n, p.B.wide, threadIdx.x);
            cl.load(Cc, p.C.row, rt, w.r1, n, p.C.wide, threadIdx.x);
#pragma unroll
            for (int i = 0; i < K::PER; ++i) {
                const int row = nl + LN * i;
                if (row >= R) break;
                V a[TP], b[TP], c[TP];
#pragma unroll
                for (int q = 0; q < TP; ++q) {
                    a[q] = add2(make2(dl.v[i].get(2 * q), dl.v[i].get(2 * q + 1)), bias[q]);
                    if (p.softplus) a[q] = softplus2(a[q]);
                    if (row >= nr) a[q] = make2((C)0, (C)0);
                    b[q] = mul2(a[q], make2(xl.v[i].get(2 * q), xl.v[i].get(2 * q + 1)));
                    c[q] = make2(yl.v[i].get(2 * q), yl.v[i].get(2 * q + 1));
                    if (z) {
                        const V v = make2(zl.v[i].get(2 * q), zl.v[i].get(2 * q + 1));
                        c[q] = mul2(c[q], mul2(v, sigmoid2(v)));
                    }
                }
                put<TP>(&sm.dt[row][d0], a);
                put<TP>(&sm.u[row][d0], b);
                put<TP>(&sm.yb[row][d0], c);
            }
            bl.stage(block.b, threadIdx.x);
            cl.stage(block.c, threadIdx.x);
        }
        __syncthreads();

        V h[TP][TN];
        const C *kept = static_cast<const C *>(o.kept) + (w.line * tiles + rt / R) * dn + part;
        load_part<K>(kept, n, w.nch, lane, h);
        for (int b = 0; b < R / S - 1 && (b + 1) * S < nr; ++b) {
            if ((st >> (b * S)) & ((1u << S) - 1u))
                at.template skip<false, true>(b * S, st, k0, A2, h);
            else if (plain)
                at.template skip<true, false>(b * S, st, k0, A2, h);
            else
                at.template skip<false, false>(b * S, st, k0, A2, h);
#pragma unroll
            for (int q = 0; q < TP; ++q)
#pragma unroll
                for (int j = 0; j < TN; ++j) sm.h[b][q * TN + j][lane] = h[q][j];
        }
        for (int b = (nr - 1) / S; b >= 0; --b) {
            const int t0 = b * S;
            if (b > 0) {
#pragma unroll
                for (int q = 0; q < TP; ++q)
#pragma unroll
                    for (int j = 0; j < TN; ++j) h[q][j] = sm.h[b - 1][q * TN + j][lane];
            } else {
                load_part<K>(kept, n, w.nch, lane, h);
            }
            Pack<T, TD> xv[PERS], dv[PERS], yv[PERS], zv[PERS];
#pragma unroll
            for (int i = 0; i < PERS; ++i) {
                const int row = t0 + nl + LN * i;
                xv[i].clear(), dv[i].clear(), yv[i].clear(), zv[i].clear();
                if (nl < S && row < nr) {
                    xv[i].load(x + (rt + row) * p.x.row, nd, p.x.wide);
                    dv[i].load(dt + (rt + row) * p.dt.row, nd, p.dt.wide);
                    if (z) {
                        yv[i].load(yb + (rt + row) * o.yb.row, nd, o.yb.wide);
                        zv[i].load(z + (rt + row) * p.z.row, nd, p.z.wide);
                    }
                }
            }
            if ((st >> t0) & ((2u << S) - 1u))
                at.template rows<false, true>(t0, nr, st, k0, A2, h, g, ab);
            else if (plain)
                at.template rows<true, false>(t0, nr, st, k0, A2, h, g, ab);
            else
                at.template rows<false, false>(t0, nr, st, k0, A2, h, g, ab);
            __syncwarp();
            // finish the rows: the sums over states
#pragma unroll
            for (int i = 0; i < PERS; ++i) {
                const int r = nl + LN * i, row = t0 + r;
                if (nl >= S || row >= nr) break;
                V gb[TP], qa[TP], hc[TP], s[TP], ys[TP];
                get<TP>(&sm.gb[r][nl][d0], gb);
                get<TP>(&sm.qa[r][nl][d0], qa);
                get<TP>(&sm.hc[r][nl][d0], hc);
#pragma unroll
                for (int e = 1; e < LN; ++e) {
                    V v[TP];
                    const int from = (nl + e) % LN;
                    get<TP>(&sm.gb[r][from][d0], v);
#pragma unroll
                    for (int q = 0; q < TP; ++q) gb[q] = add2(gb[q], v[q]);
                    get<TP>(&sm.qa[r][from][d0], v);
#pragma unroll
                    for (int q = 0; q < TP; ++q) qa[q] = add2(qa[q], v[q]);
                    if (z) {
                        get<TP>(&sm.hc[r][from][d0], v);
#pragma unroll
                        for (int q = 0; q < TP; ++q) hc[q] = add2(hc[q], v[q]);
                    }
                }
                get<TP>(&sm.dt[row][d0], s);
                get<TP>(&sm.yb[row][d0], ys);
                C xo[TD], so[TD], zo[TD];
#pragma unroll
                for (int q = 0; q < TP; ++q) {
                    const V xe = make2(xv[i].get(2 * q), xv[i].get(2 * q + 1));
                    const V vx = fma2(gb[q], s[q], mul2(skip[q], ys[q]));
                    V vs = fma2(qa[q], make2(ln2<C>(), ln2<C>()), mul2(gb[q], xe));
                    if (p.softplus) vs = mul2(vs, sigmoid2(add2(make2(dv[i].get(2 * q), dv[i].get(2 * q + 1)), bias[q])));
                    sum_d[q] = fma2(ys[q], xe, sum_d[q]);
                    sum_bias[q] = add2(sum_bias[q], vs);
                    xo[2 * q] = vx.x, xo[2 * q + 1] = vx.y;
                    so[2 * q] = vs.x, so[2 * q + 1] = vs.y;
                    if (z) {
                        const V ze = make2(zv[i].get(2 * q), zv[i].get(2 * q + 1)), pe = sigmoid2(ze);
                        const V vz = mul2(make2(yv[i].get(2 * q), yv[i].get(2 * q + 1)), fma2(skip[q], xe, hc[q]));
                        zo[2 * q] = vz.x * silu_slope(ze.x, pe.x), zo[2 * q + 1] = vz.y * silu_slope(ze.y, pe.y);
                    }
                }
                Pack<T, TD> out;
                out.set(xo);
                out.store(xb + (rt + row) * o.xb.row, nd, o.xb.wide);
                out.set(so);
                out.store(dtb + (rt + row) * o.dtb.row, nd, o.dtb.wide);
                if (z) {
                    out.set(zo);
                    out.store(zb + (rt + row) * o.zb.row, nd, o.zb.wide);
                }
            }
            // and the sums over this warp's channels: TD of a row's 2 NP values at a time, from another lane's part on
            // each, so that the lanes read other banks
            constexpr int QUADS = LN * (2 * TN / TD);
            for (int i = lane; i < S * QUADS; i += 32) {
                const int r = i / QUADS, quad = i % QUADS, m = quad / (2 * TN / TD), half = quad % (2 * TN / TD);
                C v[TD], e[TD];
                get<TD>(&sm.part[r][m][half][quad % LD][0], v);
#pragma unroll
                for (int f = 1; f < LD; ++f) {
                    get<TD>(&sm.part[r][m][half][(quad + f) % LD][0], e);
#pragma unroll
                    for (int c = 0; c < TD; ++c) v[c] += e[c];
                }
#pragma unroll
                for (int c = 0; c < TD; ++c) {
                    const int j = half * TD + c;
                    sm.bc[t0 + r][(j / TN) * NP + m * TN + j % TN] = v[c];
                }
            }
            __syncwarp();
        }
        __syncthreads();
        // Bb and Cb: the block's warps, in order, into this block's partial sums [blocks of a group][line, row][group]
        for (int i = threadIdx.x; i < nr * 2 * NP; i += SCAN_WARPS * 32) {
            const int t = i / (2 * NP), j = i % (2 * NP);
            C v = block.warp[0].bc[t][j];
            for (int a = 1; a < live; ++a) v += block.warp[a].bc[t][j];
            part_bc[(rt + t) * p.groups * 2 * NP + j] = v;
        }
    }
    if (w.nch == 0) return;
    const int64_t piece = w.line * p.segs + w.seg;
    store_part<K>(static_cast<C *>(o.part_a) + piece * dn + part, n, w.nch, lane, ab);
    // lanes that finished the same channels
    C *pd = static_cast<C *>(o.part_d) + piece * p.d + w.c0 + d0, *pb = static_cast<C *>(o.part_bias) + piece * p.d + w.c0 + d0;
#pragma unroll
    for (int q = 0; q < TP; ++q) {
#pragma unroll
        for (int m = LD; m < 32; m *= 2) {
            sum_d[q] = add2(sum_d[q], make2(shfl_xor_(sum_d[q].x, m), shfl_xor_(sum_d[q].y, m)));
            sum_bias[q] = add2(sum_bias[q], make2(shfl_xor_(sum_bias[q].x, m), shfl_xor_(sum_bias[q].y, m)));
        }
        if (nl == 0) {
            if (2 * q < nd) pd[2 * q] = sum_d[q].x, pb[2 * q] = sum_bias[q].x;
            if (2 * q + 1 < nd) pd[2 * q + 1] = sum_d[q].y, pb[2 * q + 1] = sum_bias[q].y;
        }
    }
}

// What each segment hands to the row before it, from nothing behind it, and the sum of its steps.
template <class K> struct ScanEndsSmem {
    using C = typename K::C;
    C dt[SCAN_R][K::CW], yb[SCAN_R][K::CW], c[SCAN_R][2 * K::NP];
};
template <class K, bool POLY, int ROW>
SELINV_DEVINL void scan_ends_row(const ScanEndsSmem<K> &sm, int t, int d0, int n0, const typename K::V (*A2)[K::TN],
                                 typename K::V (*g)[K::TN], typename K::V *total)
{
    using V = typename K::V;
    V dt2[K::TP], yb2[K::TP], c2[K::TN];
    get<K::TP>(&sm.dt[t][d0], dt2);
    get<K::TP>(&sm.yb[t][d0], yb2);
    get<K::TN>(&sm.c[t][2 * n0], c2);
    scan_pairs<K, POLY, ROW>([&](auto poly, int q, int j) {
        g[q][j] = mul2(decay2<poly.value>(mul2(dt2[q], A2[q][j])), fma2(c2[j], yb2[q], g[q][j]));
    });
#pragma unroll
    for (int q = 0; q < K::TP; ++q) total[q] = add2(total[q], dt2[q]);
}
template <class K>
__global__ void __launch_bounds__(SCAN_WARPS * 32)
    scan_backward_ends_kernel(const __grid_constant__ ScanArgs p, const __grid_constant__ ScanGrads o)
{
    using T = typename K::T;
    using C = typename K::C;
    using V = typename K::V;
    constexpr int R = SCAN_R, LN = K::LN, TP = K::TP, TN = K::TN;
    extern __shared__ __align__(16) char smem_raw[];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    ScanEndsSmem<K> &sm = reinterpret_cast<ScanEndsSmem<K> *>(smem_raw)[warp];
    ScanPlace w;
    if (!scan_place<K>(p, warp, w) || w.r0 >= w.r1 || w.seg == 0) return;
    const int n = p.n, nl = lane / K::LD, d0 = (lane % K::LD) * K::TD, n0 = nl * TN, nd = w.nch - d0;
    const T *dt = static_cast<const T *>(p.dt.p) + w.line * p.dt.line + w.c0 + d0;
    const T *z = p.z.p ? static_cast<const T *>(p.z.p) + w.line * p.z.line + w.c0 + d0 : nullptr;
    const T *Cc = static_cast<const T *>(p.C.p) + w.line * p.C.line + w.group * p.C_group;
    const T *yb = static_cast<const T *>(o.yb.p) + w.line * o.yb.line + w.c0 + d0;
    const int64_t part = (int64_t)w.c0 * n, dn = p.d * n;
    V A2[TP][TN], g[TP][TN], bias[TP], total[TP];
    const bool plain = load_decay<K>(p.A, part, n, w.nch, lane, A2) && p.softplus;
    zero_part<K>(g);
#pragma unroll
    for (int q = 0; q < TP; ++q) {
        bias[q] = pair_of<K>(p.dt_bias, w.c0 + d0, nd, q);
        total[q] = make2((C)0, (C)0);
    }
    ScanLoad<K> dl, yl, zl;
    ScanLoadN<K, 32> cl;
    auto fetch = [&](int64_t r) {
        dl.load(dt, p.dt.row, r, w.r1, nd, p.dt.wide, nl);
        yl.load(yb, o.yb.row, r, w.r1, nd, o.yb.wide, nl);
        if (z) zl.load(z, p.z.row, r, w.r1, nd, p.z.wide, nl);
        cl.load(Cc, p.C.row, r, w.r1, n, p.C.wide, lane);
    };
    int64_t k = p.rows.find(w.r1 - 1);          // the sequence of the row at hand
    int64_t rt = w.r0 + (w.r1 - w.r0 - 1) / R * R;
    fetch(rt);
    for (; rt >= w.r0; rt -= R) {
        const int nr = (int)min((int64_t)R, w.r1 - rt);
        int64_t k0 = k;
        while (p.rows.start(k0) > rt) --k0;
        const uint32_t st = p.rows.starts(rt, R, k0, lane);
#pragma unroll
        for (int i = 0; i < K::PER; ++i) {
            const int row = nl + LN * i;
            if (row >= R) break;
            V a[TP], c[TP];
#pragma unroll
            for (int q = 0; q < TP; ++q) {
                a[q] = add2(make2(dl.v[i].get(2 * q), dl.v[i].get(2 * q + 1)), bias[q]);
                if (p.softplus) a[q] = softplus2(a[q]);
                c[q] = make2(yl.v[i].get(2 * q), yl.v[i].get(2 * q + 1));
                if (z) {
                    const V v = make2(zl.v[i].get(2 * q), zl.v[i].get(2 * q + 1));
                    c[q] = mul2(c[q], mul2(v, sigmoid2(v)));
                }
            }
            put<TP>(&sm.dt[row][d0], a);
            put<TP>(&sm.yb[row][d0], c);
        }
        cl.stage(sm.c, lane);
        if (rt > w.r0) fetch(rt - R);
        __syncwarp();
        for (int t = nr - 1; t >= 0;) {
            if ((st >> (t + 1)) & 1u) {         // the last row of its sequence
                if (rt + t < p.rows.start(k)) --k;
                if (o.stateb)
                    load_part<K>(static_cast<const C *>(o.stateb) + p.rows.number(k, w.line) * dn + part, n, w.nch, lane, g);
                else
                    zero_part<K>(g);
            }
            // down to the row behind the next such row
            const uint32_t earlier = st & ((2u << t) - 2u);
            const int te = earlier ? 31 - __clz(earlier) : 0;
            if (plain) {
                for (; t - 3 >= te; t -= 4) {
                    scan_ends_row<K, true, 3>(sm, t, d0, n0, A2, g, total);
                    scan_ends_row<K, true, 2>(sm, t - 1, d0, n0, A2, g, total);
                    scan_ends_row<K, true, 1>(sm, t - 2, d0, n0, A2, g, total);
                    scan_ends_row<K, true, 0>(sm, t - 3, d0, n0, A2, g, total);
                }
            }
#pragma unroll 1
            for (; t >= te; --t) scan_ends_row<K, false, 0>(sm, t, d0, n0, A2, g, total);
        }
        __syncwarp();
    }
    scan_leave<K>(p, w, lane, g, total);
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
                      offsetof(ScanBwdSmem<K>, gb) % 16 == 0 && offsetof(ScanBwdSmem<K>, qa) % 16 == 0 &&
                      offsetof(ScanBwdSmem<K>, hc) % 16 == 0 && offsetof(ScanBwdSmem<K>, part) % 16 == 0 &&
                      offsetof(ScanBwdBlock<K>, b) % 16 == 0 && offsetof(ScanBwdBlock<K>, c) % 16 == 0,
                  "staged rows lie on 16 bytes");
    constexpr int bytes = (int)sizeof(ScanBwdBlock<K>);
    static_assert(bytes <= 227 * 1024, "fits an SM");
    if (p.segs > 1) {
        constexpr int ends = SCAN_WARPS * (int)sizeof(ScanEndsSmem<K>);
        static_assert(sizeof(ScanEndsSmem<K>) % 16 == 0 && offsetof(ScanEndsSmem<K>, c) % 16 == 0, "rows on 16 bytes");
        cudaError_t e =
            cudaFuncSetAttribute(scan_backward_ends_kernel<K>, cudaFuncAttributeMaxDynamicSharedMemorySize, ends);
        if (e != cudaSuccess) return e;
        scan_backward_ends_kernel<K><<<grid, SCAN_WARPS * 32, ends, s>>>(p, o);
    }
    cudaError_t e = cudaFuncSetAttribute(scan_backward_kernel<K>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    scan_backward_kernel<K><<<grid, SCAN_WARPS * 32, bytes, s>>>(p, o);
    const int64_t bc = (p.lines * p.rows.rows * p.groups * 2 * K::NP + 255) / 256;
    const int64_t params = (p.d * (p.n + 2) + 31) / 32;
    scan_sums_kernel<typename K::T, K::NP><<<(unsigned)(bc + params), 256, 0, s>>>(p, o, bc, parts);
    return cudaGetLastError();
}

}  // namespace
}  // namespace selinv
