// Backward of the selective scan.  With yb' = yb silu(z) and, from the last
// row to the first,
//   g_t = C_t yb'_t + a_{t+1} g_{t+1},   q_t = g_t a_t h_{t-1}
// the cotangents are
//   xb = dt' (g . B) + D yb'        dt'b = x (g . B) + q . A     Ab = sum_t q dt'
//   Bb = sum_d g dt' x              Cb = sum_d h yb'             Db = sum_t yb' x
//   zb = yb silu'(z) (h . C + D x)  dtb = dt'b softplus'(dt + dt_bias).
// A thread keeps eight states (pairs in one instruction) of two channels, or
// four where shared memory then holds three blocks per SM or there are few; a
// block works on SCAN_WARPS neighbouring warp tiles of channels and one
// segment of a line, SCAN_R rows at a time from the end.  The states inside
// come again from the one kept before those rows: a first run leaves every
// SCAN_S-th in shared memory, a second one fills the registers with the
// states and decays of SCAN_S rows, which the backward recurrence then uses
// up.  Sums over a channel's states end in a thread or a few lanes; those
// over channels (Bb, Cb) go through shared memory, 16 bytes a store, and leave
// a block as one partial sum per row; those over rows (Ab, Db, dt_biasb) leave
// it as one per segment.  scan_sums_kernel adds the partial sums in a fixed
// order.
//
// Bounded by the issue of instructions and their latency: a warp of 32 channels
// takes about 370 per row, at 255 registers two warps per scheduler hide part of
// each other's waits (0.45 instructions a cycle).  4 x 2048 x 4096 x 16 in
// bfloat16: 969 us, of which 180 the run over the segments' ends and 14 the
// partial sums, against 137 us for the powers of two and sigmoids of one pass
// and 92 us of memory.  Three quarters of the rows' states are formed twice, and
// at 255 registers a thread spills 72 bytes of stores and 356 of loads (float64
// up to 476 and 996).  Keeping the first run's powers for the second would take
// 32 KB a warp, and so half of the warps.
#pragma once

#include "scan_forward.cuh"

namespace selinv {
namespace {

constexpr int SCAN_S = 4;       // rows whose states and decays are in registers together

// lane = nl * LD + dl holds the channels 2 dl, 2 dl + 1 and the states nl * SN on.
template <class T_, int NP_> struct ScanBwdTile {
    using T = T_;
    using C = typename Elem<T>::C;
    using V = typename Two<C>::V;
    static constexpr int NP = NP_, SN = NP == 4 && sizeof(C) == 8 ? 2 : NP > 16 - (sizeof(T) == 2) && sizeof(C) == 4 ? 8 : 4, KP = SN / 2, LN = NP / SN, LD = 32 / LN, CW = 2 * LD;
    static constexpr int PER = (SCAN_R + LN - 1) / LN;          // rows whose steps and outputs a lane forms
    static constexpr int P = SN == 4 && sizeof(T) == 2 ? 4 : 2;     // rows whose parts of Bb and Cb are in shared memory together
    static constexpr int Q = 16 / (int)sizeof(C), CHUNKS = 2 * SN / Q;      // 16 bytes of sums; B's states, then C's
};
template <class K> struct ScanBwdSmem {
    using C = typename K::C;
    using T = typename K::T;
    alignas(16) T x[SCAN_R][K::CW], dt_raw[SCAN_R][K::CW], z[SCAN_R][K::CW], yb_raw[SCAN_R][K::CW];
    alignas(16) C dt[SCAN_R][K::CW], yb[SCAN_R][K::CW], gb[SCAN_R][K::CW], qa[SCAN_R][K::CW], hc[SCAN_R][K::CW];
    alignas(16) C part[K::P][K::LN][K::CHUNKS][K::LD][K::Q];
    alignas(16) C bc[SCAN_R][2 * K::NP];
    alignas(16) typename K::V h[SCAN_R / SCAN_S - 1][2 * K::KP][32];    // states before rows SCAN_S, 2 SCAN_S, ...
};
template <class K> struct ScanBwdBlock {
    using C = typename K::C;
    using T = typename K::T;
    ScanBwdSmem<K> warp[SCAN_WARPS];
    alignas(16) T b_raw[SCAN_R][K::NP], c_raw[SCAN_R][K::NP];
    alignas(16) C b[SCAN_R][K::NP], c[SCAN_R][K::NP];
};

// What a thread of the backward knows of its place.
template <class K> struct ScanBwd {
    using T = typename K::T;
    using C = typename K::C;
    using V = typename K::V;
    static constexpr int KP = K::KP, SN = K::SN;
    const ScanArgs &p;
    const ScanGrads &o;
    ScanBwdBlock<K> &block;
    ScanBwdSmem<K> &sm;
    int lane, nl, c, n0, nch;       // c: the first of the two channels, among the warp's
    int64_t line, part, dn;         // part: that channel's place in a [d, n] array

    SELINV_DEVINL void load(const C *from, V (*v)[KP]) const
    {
        load_states<SN>(from + part + n0, p.n - n0, c < nch, v[0]);
        load_states<SN>(from + part + p.n + n0, p.n - n0, c + 1 < nch, v[1]);
    }
    SELINV_DEVINL void store(C *to, const V (*v)[KP]) const
    {
        store_states<SN>(to + part + n0, p.n - n0, c < nch, v[0]);
        store_states<SN>(to + part + p.n + n0, p.n - n0, c + 1 < nch, v[1]);
    }
    SELINV_DEVINL void states(const void *from, int sequence, V (*v)[KP]) const
    {
        if (from) {
            load(static_cast<const C *>(from) + p.rows.number(sequence, line) * dn, v);
        } else {
            zero_states<SN>(v[0]);
            zero_states<SN>(v[1]);
        }
    }
    // The live sequence of row t of a tile whose first row lies in k0; st: the rows that begin one.
    SELINV_DEVINL static int sequence(int k0, uint32_t st, int t) { return k0 + __popc(st & ((2u << t) - 2u)); }

    // dt' and x of the two channels of row t
    SELINV_DEVINL void inputs(int t, V &dt, V &x) const
    {
        dt = *reinterpret_cast<const V *>(&sm.dt[t][c]);
        Pack<T, 2> v;
        v.load(&sm.x[t][c], 2, true);
        x = make2(v.get(0), v.get(1));
    }
    // How many of this lane's states channel i of its two has.
    SELINV_DEVINL int real(int i) const { return c + i < nch ? p.n - n0 : 0; }
    // Row t: the state before it becomes the state after it; its decays.  REAL: with zeros for what does not exist.
    template <bool REAL> SELINV_DEVINL void row(int t, const V (*A2)[KP], V (*h)[KP], V (*a)[KP]) const
    {
        V dt, x, b[KP];
        inputs(t, dt, x);
        get<KP>(&block.b[t][n0], b);
        const V u = mul2(dt, x), d0 = make2(dt.x, dt.x), d1 = make2(dt.y, dt.y), u0 = make2(u.x, u.x), u1 = make2(u.y, u.y);
#pragma unroll
        for (int j = 0; j < KP; ++j) {
            a[0][j] = decay2(d0, A2[0][j]);
            a[1][j] = decay2(d1, A2[1][j]);
            h[0][j] = fma2(a[0][j], h[0][j], mul2(u0, b[j]));
            h[1][j] = fma2(a[1][j], h[1][j], mul2(u1, b[j]));
            if (REAL) {
#pragma unroll
                for (int i = 0; i < 2; ++i) a[i][j] = real_states(a[i][j], j, real(i)), h[i][j] = real_states(h[i][j], j, real(i));
            }
        }
    }
    // SCAN_S rows of the first run.  EDGE: some row begins a sequence.
    template <bool EDGE, bool REAL> SELINV_DEVINL void skip(int t0, uint32_t begins, int k0, const V (*A2)[KP], V (*h)[KP]) const
    {
#pragma unroll
        for (int r = 0; r < SCAN_S; ++r) {
            V a[2][KP];
            if (EDGE && ((begins >> (t0 + r)) & 1u)) states(p.state, sequence(k0, begins, t0 + r), h);
            row<REAL>(t0 + r, A2, h, a);
        }
    }
    // Rows t0 .. t0 + SCAN_S - 1, `before` the state before them.  EDGE: some row begins or ends a sequence; st has the
    // rows that begin one and the row behind the last, of which only those below nr are rows.
    template <bool EDGE, bool REAL>
    SELINV_DEVINL void rows(int t0, int nr, uint32_t st, int k0, const V (*A2)[KP], const V (*before)[KP], V (*g)[KP],
                            V (*ab)[KP]) const
    {
        constexpr int S = SCAN_S;
        const uint32_t begins = st & ((1u << nr) - 1u);
        V h[S][2][KP], a[S][2][KP];
#pragma unroll
        for (int r = 0; r < S; ++r) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < KP; ++j) h[r][i][j] = r ? h[r ? r - 1 : 0][i][j] : before[i][j];
            if (EDGE && ((begins >> (t0 + r)) & 1u)) states(p.state, sequence(k0, begins, t0 + r), h[r]);
            row<REAL>(t0 + r, A2, h[r], a[r]);
        }
#pragma unroll
        for (int r = S - 1; r >= 0; --r) {
            const int t = t0 + r;
            if (EDGE && ((st >> (t + 1)) & 1u)) {
                states(o.stateb, sequence(k0, st, t), g);
                // A line's last row, the first that this block comes to but for up to three behind it that are none: their
                // cotangents are zero, but zero times an infinite state is not a number.
                if (t + 1 == nr && nr < SCAN_R) zero_states<SN>(ab[0]), zero_states<SN>(ab[1]);
            }
            const bool first = EDGE && ((begins >> t) & 1u);
            V start[2][KP];
            if (EDGE) {
                if (first) {
                    states(p.state, sequence(k0, st, t), start);
                } else {
#pragma unroll
                    for (int i = 0; i < 2; ++i)
#pragma unroll
                        for (int j = 0; j < KP; ++j) start[i][j] = r > 0 ? h[r > 0 ? r - 1 : 0][i][j] : before[i][j];
                }
            }
            V dt, x, b[KP], c2[KP], gb[2], qa[2], hc[2], sb[KP], sc[KP];
            inputs(t, dt, x);
            const V yb = *reinterpret_cast<const V *>(&sm.yb[t][c]), u = mul2(dt, x);
            get<KP>(&block.b[t][n0], b);
            get<KP>(&block.c[t][n0], c2);
            const V d2[2] = {make2(dt.x, dt.x), make2(dt.y, dt.y)}, u2[2] = {make2(u.x, u.x), make2(u.y, u.y)};
            const V y2[2] = {make2(yb.x, yb.x), make2(yb.y, yb.y)};
#pragma unroll
            for (int i = 0; i < 2; ++i) {
#pragma unroll
                for (int j = 0; j < KP; ++j) {
                    const V past = EDGE ? start[i][j] : r > 0 ? h[r > 0 ? r - 1 : 0][i][j] : before[i][j];
                    V gt = fma2(c2[j], y2[i], g[i][j]);
                    if (REAL) gt = real_states(gt, j, real(i));
                    sb[j] = i ? fma2(gt, u2[i], sb[j]) : mul2(gt, u2[i]);
                    sc[j] = i ? fma2(h[r][i][j], y2[i], sc[j]) : mul2(h[r][i][j], y2[i]);
                    gb[i] = j ? fma2(gt, b[j], gb[i]) : mul2(gt, b[j]);
                    hc[i] = j ? fma2(h[r][i][j], c2[j], hc[i]) : mul2(h[r][i][j], c2[j]);
                    g[i][j] = mul2(a[r][i][j], gt);
                    const V m = mul2(g[i][j], past);
                    qa[i] = j ? fma2(m, A2[i][j], qa[i]) : mul2(m, A2[i][j]);
                    ab[i][j] = fma2(m, d2[i], ab[i][j]);
                }
            }
            C v[3][2];
#pragma unroll
            for (int i = 0; i < 2; ++i) v[0][i] = gb[i].x + gb[i].y, v[1][i] = qa[i].x + qa[i].y, v[2][i] = hc[i].x + hc[i].y;
#pragma unroll
            for (int e = 0; e < 3; ++e) scatter_sum<2, K::LD, 32>(v[e], lane);
            constexpr int KEEP = K::LN == 1 ? 2 : 1;
            if (scatter_writes<2, K::LD, 32>(lane)) {
                const int f = c + scatter_first<2, K::LD, 32>(lane);
#pragma unroll
                for (int i = 0; i < KEEP; ++i) sm.gb[t][f + i] = v[0][i], sm.qa[t][f + i] = v[1][i], sm.hc[t][f + i] = v[2][i];
            }
            C out[2 * SN];
#pragma unroll
            for (int j = 0; j < KP; ++j) {
                out[2 * j] = sb[j].x, out[2 * j + 1] = sb[j].y;
                out[SN + 2 * j] = sc[j].x, out[SN + 2 * j + 1] = sc[j].y;
            }
#pragma unroll
            for (int i = 0; i < K::CHUNKS; ++i) put<K::Q>(&sm.part[r % K::P][nl][i][lane % K::LD][0], out + i * K::Q);
            if (first && o.stateb_out) store(static_cast<C *>(o.stateb_out) + p.rows.number(sequence(k0, st, t), line) * dn, g);
            if (r % K::P == 0) {
                __syncwarp();
                sums(t);
                __syncwarp();
            }
        }
    }
    // The nr rows of a tile, from the state kept before them; begins and st as above.
    template <bool REAL>
    SELINV_DEVINL void tile(const C *kept, int nr, uint32_t begins, uint32_t st, int k0, const V (*A2)[KP], V (*g)[KP],
                            V (*ab)[KP]) const
    {
        constexpr int S = SCAN_S;
        V h[2][KP];
        load(kept, h);
        for (int b = 0; b < SCAN_R / S - 1 && (b + 1) * S < nr; ++b) {
            if (REAL || ((begins >> (b * S)) & ((1u << S) - 1u)))
                skip<true, REAL>(b * S, begins, k0, A2, h);
            else
                skip<REAL, REAL>(b * S, begins, k0, A2, h);
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < KP; ++j) sm.h[b][i * KP + j][lane] = h[i][j];
        }
        for (int b = (nr - 1) / S; b >= 0; --b) {
            if (b > 0) {
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int j = 0; j < KP; ++j) h[i][j] = sm.h[b - 1][i * KP + j][lane];
            } else {
                load(kept, h);
            }
            if (REAL || ((st >> (b * S)) & ((2u << S) - 1u)))
                rows<true, REAL>(b * S, nr, st, k0, A2, h, g, ab);
            else
                rows<REAL, REAL>(b * S, nr, st, k0, A2, h, g, ab);
        }
    }
    // Bb's and Cb's sums over this warp's channels for rows t .. t + P - 1: a pair of states at a time, from another
    // lane's part on each, so that the lanes read other banks.
    SELINV_DEVINL void sums(int t) const
    {
        constexpr int HALVES = K::Q / 2, PAIRS = K::LN * K::CHUNKS * HALVES;
#pragma unroll
        for (int i = lane; i < K::P * PAIRS; i += 32) {
            const int r = i / PAIRS, pair = i % PAIRS, half = pair % HALVES, chunk = pair / HALVES;
            const int m = chunk / K::CHUNKS, ch = chunk % K::CHUNKS;
            V v[K::LD];
#pragma unroll
            for (int f = 0; f < K::LD; ++f)
                v[f] = *reinterpret_cast<const V *>(&sm.part[r][m][ch][(chunk + f) % K::LD][2 * half]);
#pragma unroll
            for (int s = K::LD / 2; s > 0; s /= 2)
#pragma unroll
                for (int f = 0; f < s; ++f) v[f] = add2(v[f], v[f + s]);
            const int j = ch * K::Q + 2 * half;         // among B's states and then C's of lane group m
            *reinterpret_cast<V *>(&sm.bc[t + r][(j / SN) * K::NP + m * SN + j % SN]) = v[0];
        }
    }
};

// Blocks per SM that shared memory and registers allow; three keep to 168 registers, where eight states would spill (16
// states: in 16-bit types 963 us with eight and two blocks, 1036 with four and three, 4 x 2048 x 4096; in float four are
// a fifth faster, 3 x 517 x 1250).
template <class K> constexpr int scan_bwd_blocks = K::SN <= 4 && 3 * (sizeof(ScanBwdBlock<K>) + 1024) <= 228 * 1024   ? 3
                                                   : 2 * (sizeof(ScanBwdBlock<K>) + 1024) <= 228 * 1024 ? 2
                                                                                                        : 1;

// A block's work.  States and channels that do not exist stay zero as long as all that is there is finite; with PADDED the
// call says whether it is not, and with REAL they are kept at zero whatever comes.
template <class K, bool PADDED, bool REAL>
SELINV_DEVINL bool scan_backward_block(const ScanArgs &p, const ScanGrads &o, char *smem_raw)
{
    using T = typename K::T;
    using C = typename K::C;
    using V = typename K::V;
    constexpr int R = SCAN_R, S = SCAN_S, LN = K::LN, LD = K::LD, NP = K::NP, SN = K::SN, KP = K::KP, CW = K::CW, PER = K::PER;
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    ScanBwdBlock<K> &block = *reinterpret_cast<ScanBwdBlock<K> *>(smem_raw);
    ScanBwdSmem<K> &sm = block.warp[warp];
    ScanPlace w;
    scan_place(p, warp, SCAN_WARPS, CW, w);     // a warp without channels (nch <= 0) still meets the others
    w.nch = max(w.nch, 0);
    if (w.nch == 0) w.c0 = 0;                   // its addresses are never used

    const int n = p.n, nl = lane / LD, c = 2 * (lane % LD), n0 = nl * SN;
    const T *x = static_cast<const T *>(p.x.p) + w.line * p.x.line + w.c0;
    const T *dt = static_cast<const T *>(p.dt.p) + w.line * p.dt.line + w.c0;
    const T *z = p.z.p ? static_cast<const T *>(p.z.p) + w.line * p.z.line + w.c0 : nullptr;
    const T *B = static_cast<const T *>(p.B.p) + w.line * p.B.line + w.group * p.B_group;
    const T *Cc = static_cast<const T *>(p.C.p) + w.line * p.C.line + w.group * p.C_group;
    const T *yb = static_cast<const T *>(o.yb.p) + w.line * o.yb.line + w.c0;
    T *xb = static_cast<T *>(o.xb.p) + w.line * o.xb.line + w.c0 + c;
    T *dtb = static_cast<T *>(o.dtb.p) + w.line * o.dtb.line + w.c0 + c;
    T *zb = o.zb.p ? static_cast<T *>(o.zb.p) + w.line * o.zb.line + w.c0 + c : nullptr;
    const int64_t dn = p.d * n, part = (int64_t)(w.c0 + c) * n;
    const ScanBwd<K> at{p, o, block, sm, lane, nl, c, n0, w.nch, w.line, part, dn};

    if (o.stateb_out && p.rows.table && blockIdx.x == 0 && nl == 0) {       // sequences without rows
        C *out = static_cast<C *>(o.stateb_out);
        const C *in = static_cast<const C *>(o.stateb);
        for (int64_t e = 0; e < p.sequences - p.rows.live; ++e) {
            const int64_t a = p.rows.empty(e) * dn + part;
            for (int i = 0; i < n * min(2, w.nch - c); ++i) out[a + i] = in ? in[a + i] : (C)0;
        }
    }

    V A2[2][KP], g[2][KP], ab[2][KP];       // g: what the row behind hands on, a_{t+1} g_{t+1}
    at.load(static_cast<const C *>(p.A), A2);
    C bias[2], skip[2];
    V sum_d = make2((C)0, (C)0), sum_bias = sum_d;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int j = 0; j < KP; ++j) A2[i][j] = mul2(A2[i][j], make2(log2e<C>(), log2e<C>()));
        zero_states<SN>(g[i]);
        zero_states<SN>(ab[i]);
        bias[i] = c + i < w.nch && p.dt_bias ? static_cast<const C *>(p.dt_bias)[w.c0 + c + i] : (C)0;
        skip[i] = c + i < w.nch && p.D ? static_cast<const C *>(p.D)[w.c0 + c + i] : (C)0;
    }
    int k0 = w.r1 > w.r0 ? p.rows.find(w.r1 - 1) : 0;
    if (w.r1 > w.r0 && p.rows.end(k0) > w.r1) {         // what the segments behind this one hand on
#pragma unroll
        for (int i = 0; i < 2; ++i)
            scan_join<SN, C>(p, w.line, (p.rows.end(k0) - 1) / p.seg_rows, w.seg, -1, w.c0 + c + i, part + i * n + n0, n - n0,
                             c + i < w.nch, A2[i], g[i]);
    }
    const int tiles = (p.rows.rows + R - 1) / R;
    const int per = (int)(p.d / p.groups), tiles_c = (per + CW - 1) / CW;
    const int blocks = (tiles_c + SCAN_WARPS - 1) / SCAN_WARPS, bi = (int)blockIdx.y % blocks;
    C *part_bc = static_cast<C *>(o.part_bc) +
                 (((int64_t)bi * p.lines + w.line) * p.rows.rows * p.groups + w.group) * 2 * NP;
    const bool out_wide = o.xb.wide && o.dtb.wide && (!z || o.zb.wide);
    // rows rt + r, rt + r + LN, ... of an output, below rt + rows
    const auto put_rows = [](T *to, int stride, int rt, int r, int rows, int have, bool wide, const auto &v) {
        constexpr int F = sizeof(v) / sizeof(V);
        to += (int64_t)(rt + r) * stride;
        Pack<T, 2> out[F];
#pragma unroll
        for (int i = 0; i < F; ++i) {
            const C q[2] = {v[i].x, v[i].y};
            out[i].set(q);
        }
        if (wide && have >= 2 && r + LN * (F - 1) < rows) {
#pragma unroll
            for (int i = 0; i < F; ++i) out[i].store(to + (int64_t)(LN * i) * stride, 2, true);
        } else {
#pragma unroll
            for (int i = 0; i < F; ++i)
                if (r + LN * i < rows) out[i].store(to + (int64_t)(LN * i) * stride, have, false);
        }
    };
    const bool full = p.x.wide && p.dt.wide && o.yb.wide && (!z || p.z.wide) && p.B.wide && p.C.wide && w.nch == CW && whole_n<T>(n);
    auto fetch_as = [&](auto whole, int r) {
        constexpr bool F = whole.value;
        raw_fetch<CW, F>(sm.x, x, p.x, r, w.r1, w.nch, lane);
        raw_fetch<CW, F>(sm.dt_raw, dt, p.dt, r, w.r1, w.nch, lane);
        raw_fetch<CW, F>(sm.yb_raw, yb, o.yb, r, w.r1, w.nch, lane);
        if (z) raw_fetch<CW, F>(sm.z, z, p.z, r, w.r1, w.nch, lane);
        raw_fetch_n<SCAN_WARPS * 32, F>(block.b_raw, B, p.B.row, r, w.r1, n, p.B.wide, threadIdx.x);
        raw_fetch_n<SCAN_WARPS * 32, F>(block.c_raw, Cc, p.C.row, r, w.r1, n, p.C.wide, threadIdx.x);
        cp_async_commit();
    };
    auto fetch = [&](int r) {
        if (full && r + R <= w.r1)
            fetch_as(std::true_type(), r);
        else
            fetch_as(std::false_type(), r);
    };
    raw_clear_n<SCAN_WARPS * 32>(block.b_raw, n, threadIdx.x);
    raw_clear_n<SCAN_WARPS * 32>(block.c_raw, n, threadIdx.x);
    C probe = 0;            // of zb; not a number once something is not finite
    __syncthreads();
    int rt = w.r0 + (w.r1 > w.r0 ? (w.r1 - w.r0 - 1) / R * R : 0);
    if (w.r1 > w.r0) fetch(rt);
    for (; rt >= w.r0 && rt < w.r1; rt -= R) {
        const int nr = min(R, w.r1 - rt);
        while (p.rows.start(k0) > rt) --k0;         // the live sequence of this tile's first row
        const uint32_t st = p.rows.starts(rt, R, k0, lane), begins = st & ((1u << nr) - 1u);
        cp_async_wait_all();
        __syncthreads();
        raw_stage_n<SCAN_WARPS * 32>(block.b, block.b_raw, threadIdx.x);
        raw_stage_n<SCAN_WARPS * 32>(block.c, block.c_raw, threadIdx.x);
        if (rt > w.r0) {
            raw_prefetch(x, p.x.row, rt - R, w.r1, w.nch, lane);
            raw_prefetch(dt, p.dt.row, rt - R, w.r1, w.nch, lane);
            raw_prefetch(yb, o.yb.row, rt - R, w.r1, w.nch, lane);
            if (z) raw_prefetch(z, p.z.row, rt - R, w.r1, w.nch, lane);
        }
        {       // steps and gated cotangents; rows and channels that are not there have no step, no input, no cotangent
            V a[PER], y[PER];
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const int row = min(nl + LN * i, R - 1);
                Pack<T, 2> v;
                v.load(&sm.dt_raw[row][c], 2, true);
                a[i] = make2(v.get(0) + bias[0], v.get(1) + bias[1]);
                v.load(&sm.yb_raw[row][c], 2, true);
                y[i] = make2(v.get(0), v.get(1));
            }
            if (p.softplus) {
#pragma unroll
                for (int i = 0; i < PER; ++i) a[i] = make2(softplus_of<T>(a[i].x), softplus_of<T>(a[i].y));
            }
            if (z) {
#pragma unroll
                for (int i = 0; i < PER; ++i) {
                    Pack<T, 2> v;
                    v.load(&sm.z[min(nl + LN * i, R - 1)][c], 2, true);
                    const V q = make2(v.get(0), v.get(1));
                    y[i] = mul2(y[i], mul2(q, sigmoid2(q)));
                }
            }
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const int row = nl + LN * i;
                if (row >= R) break;
                const bool in0 = row < nr && c < w.nch, in1 = row < nr && c + 1 < w.nch;
                *reinterpret_cast<V *>(&sm.dt[row][c]) = make2(in0 ? a[i].x : (C)0, in1 ? a[i].y : (C)0);
                *reinterpret_cast<V *>(&sm.yb[row][c]) = make2(in0 ? y[i].x : (C)0, in1 ? y[i].y : (C)0);
                if (!in0) sm.x[row][c] = Elem<T>::down((C)0);
                if (!in1) sm.x[row][c + 1] = Elem<T>::down((C)0);
            }
        }
        __syncthreads();

        const C *kept = static_cast<const C *>(o.kept) + (w.line * tiles + rt / R) * dn;
        at.template tile<REAL>(kept, nr, begins, st, k0, A2, g, ab);
        __syncwarp();
        // finish the rows, four of a lane's at a time: all loads, then the arithmetic, then the stores
        constexpr int F = PER < 4 ? PER : 4;
#pragma unroll
        for (int i0 = 0; i0 < PER; i0 += F) {
            V xe[F], de[F], gb[F], qa[F], s[F], ys[F], vx[F], vs[F];
            const V sk = make2(skip[0], skip[1]);
#pragma unroll
            for (int i = 0; i < F; ++i) {
                const int row = min(nl + LN * (i0 + i), R - 1);
                Pack<T, 2> v;
                v.load(&sm.x[row][c], 2, true);
                xe[i] = make2(v.get(0), v.get(1));
                v.load(&sm.dt_raw[row][c], 2, true);
                de[i] = make2(v.get(0) + bias[0], v.get(1) + bias[1]);
                gb[i] = *reinterpret_cast<const V *>(&sm.gb[row][c]);
                qa[i] = *reinterpret_cast<const V *>(&sm.qa[row][c]);
                s[i] = *reinterpret_cast<const V *>(&sm.dt[row][c]);
                ys[i] = *reinterpret_cast<const V *>(&sm.yb[row][c]);
            }
#pragma unroll
            for (int i = 0; i < F; ++i) {
                vx[i] = fma2(gb[i], s[i], mul2(sk, ys[i]));
                vs[i] = fma2(qa[i], make2(ln2<C>(), ln2<C>()), mul2(gb[i], xe[i]));
            }
            if (p.softplus) {
#pragma unroll
                for (int i = 0; i < F; ++i) vs[i] = mul2(vs[i], sigmoid2(de[i]));
            }
#pragma unroll
            for (int i = 0; i < F; ++i) {
                const bool have = nl + LN * (i0 + i) < nr;
                if (have) sum_d = fma2(ys[i], xe[i], sum_d);
                if (have && c < w.nch) sum_bias.x += vs[i].x;
                if (have && c + 1 < w.nch) sum_bias.y += vs[i].y;
            }
            put_rows(xb, o.xb.row, rt, nl + LN * i0, nr, w.nch - c, out_wide, vx);
            put_rows(dtb, o.dtb.row, rt, nl + LN * i0, nr, w.nch - c, out_wide, vs);
            if (z) {
#pragma unroll
                for (int i = 0; i < F; ++i) {
                    const int row = min(nl + LN * (i0 + i), R - 1);
                    Pack<T, 2> v;
                    v.load(&sm.yb_raw[row][c], 2, true);
                    ys[i] = make2(v.get(0), v.get(1));
                    v.load(&sm.z[row][c], 2, true);
                    de[i] = make2(v.get(0), v.get(1));
                    s[i] = *reinterpret_cast<const V *>(&sm.hc[row][c]);
                }
#pragma unroll
                for (int i = 0; i < F; ++i)
                    vs[i] = mul2(mul2(ys[i], fma2(sk, xe[i], s[i])), silu_slope2(de[i], sigmoid2(de[i])));
                if constexpr (PADDED) {
#pragma unroll
                    for (int i = 0; i < F; ++i) {
                        const bool have = nl + LN * (i0 + i) < nr;
                        if (have && c < w.nch) probe = fma(vs[i].x, (C)0, probe);
                        if (have && c + 1 < w.nch) probe = fma(vs[i].y, (C)0, probe);
                    }
                }
                put_rows(zb, o.zb.row, rt, nl + LN * i0, nr, w.nch - c, out_wide, vs);
            }
        }
        __syncthreads();        // the warps' sums are there, and the staged rows are used up
        if (rt > w.r0) fetch(rt - R);
        // Bb and Cb: the block's warps, in order, into this block's partial sums [blocks of a group][line, row][group]
#pragma unroll
        for (int i = threadIdx.x; i < R * 2 * NP; i += SCAN_WARPS * 32) {
            const int t = i / (2 * NP), j = i % (2 * NP);
            C v = 0;
#pragma unroll
            for (int a = 0; a < SCAN_WARPS; ++a) v += block.warp[a].bc[t][j];       // zero where a warp has no channels
            if (t < nr) part_bc[(int64_t)(rt + t) * p.groups * 2 * NP + j] = v;
        }
    }
    if (w.nch > 0) {
        const int64_t piece = w.line * p.segs + w.seg;
        at.store(static_cast<C *>(o.part_a) + piece * dn, ab);
        // lanes that finished the same channels
#pragma unroll
        for (int m = LD; m < 32; m *= 2) {
            sum_d = add2(sum_d, make2(shfl_xor_(sum_d.x, m), shfl_xor_(sum_d.y, m)));
            sum_bias = add2(sum_bias, make2(shfl_xor_(sum_bias.x, m), shfl_xor_(sum_bias.y, m)));
        }
        if (nl == 0) {
            C *pd = static_cast<C *>(o.part_d) + piece * p.d + w.c0 + c, *pb = static_cast<C *>(o.part_bias) + piece * p.d + w.c0 + c;
            if (c < w.nch) pd[0] = sum_d.x, pb[0] = sum_bias.x;
            if (c + 1 < w.nch) pd[1] = sum_d.y, pb[1] = sum_bias.y;
        }
    }
    // Every infinity that can make something of what does not exist shows in the block's channels: x and yb' in Db, dt' in
    // Ab, B and C in dt_biasb, and a product dt' x in Ab or, where no row of its sequence follows, in zb.
    if (!PADDED) return false;
    probe = fma(sum_d.x + sum_d.y, (C)0, fma(sum_bias.x + sum_bias.y, (C)0, probe));
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < KP; ++j) probe = fma(ab[i][j].x, (C)0, fma(ab[i][j].y, (C)0, probe));
    return __syncthreads_or(probe != (C)0);
}
// PADDED: some states or channels of the blocks do not exist.  Where something is not finite the block then begins again: what
// tells is in no tile's way, and not in the kernel that has no use for it (4 x 2048 x 4096 in bfloat16, backward: 987 us
// with 12 states, 955 without any of this, 1062 with infinities in one channel; 16 states, all there, 969.  Told apart
// tile by tile, inside the loop, its registers cost those 60 us.)
template <class K, bool PADDED>
__global__ void __launch_bounds__(SCAN_WARPS * 32, scan_bwd_blocks<K>)
    scan_backward_kernel(const __grid_constant__ ScanArgs p, const __grid_constant__ ScanGrads o)
{
    extern __shared__ __align__(16) char smem_raw[];
    const bool odd = scan_backward_block<K, PADDED, false>(p, o, smem_raw);
    if constexpr (PADDED)
        if (odd) scan_backward_block<K, false, true>(p, o, smem_raw);
}
template <class K, bool PADDED> cudaError_t scan_backward_start(const ScanArgs &p, const ScanGrads &o, const dim3 &grid, cudaStream_t s)
{
    constexpr int bytes = (int)sizeof(ScanBwdBlock<K>);
    static_assert(bytes <= 227 * 1024, "fits an SM");
    const cudaError_t e =
        cudaFuncSetAttribute(scan_backward_kernel<K, PADDED>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    scan_backward_kernel<K, PADDED><<<grid, SCAN_WARPS * 32, bytes, s>>>(p, o);
    return cudaSuccess;
}

// What each segment hands to the row before it, from nothing behind it, and the sum of its steps: LN lanes per channel, as
// in the forward.
template <class K> struct ScanEndsSmem {
    using C = typename K::C;
    using T = typename K::T;
    struct Raw {
        alignas(16) T dt[SCAN_R][K::CW], yb[SCAN_R][K::CW], z[SCAN_R][K::CW], c[SCAN_R][K::NP];
    } raw[2];
    alignas(16) C dt[SCAN_R][K::CW], yb[SCAN_R][K::CW], c[SCAN_R][K::NP];
};
template <class K>
SELINV_DEVINL void scan_ends_row(const ScanEndsSmem<K> &sm, int t, int dl, int n0, const typename K::V *A2, typename K::V *g)
{
    using C = typename K::C;
    using V = typename K::V;
    const C dt = sm.dt[t][dl], yb = sm.yb[t][dl];
    const V d2 = make2(dt, dt), y2 = make2(yb, yb);
#pragma unroll
    for (int j = 0; j < K::KP; j += 2) {
        V c[2];
        get<2>(&sm.c[t][n0 + 2 * j], c);
#pragma unroll
        for (int i = 0; i < 2; ++i) g[j + i] = mul2(decay2(d2, A2[j + i]), fma2(c[i], y2, g[j + i]));
    }
}
template <class K>
__global__ void __launch_bounds__(SCAN_WARPS * 32)
    scan_backward_ends_kernel(const __grid_constant__ ScanArgs p, const __grid_constant__ ScanGrads o)
{
    using T = typename K::T;
    using C = typename K::C;
    using V = typename K::V;
    constexpr int R = SCAN_R, LN = K::LN, SN = K::SN, KP = K::KP, CW = K::CW, PER = K::PER;
    extern __shared__ __align__(16) char smem_raw[];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    ScanEndsSmem<K> &sm = reinterpret_cast<ScanEndsSmem<K> *>(smem_raw)[warp];
    ScanPlace w;
    if (!scan_place(p, warp, blockDim.x / 32, CW, w) || w.r0 >= w.r1 || w.seg == 0) return;
    const int nl = lane / CW, dl = lane % CW, n0 = nl * SN, n = p.n - n0;
    const bool in = dl < w.nch;
    const T *dt = static_cast<const T *>(p.dt.p) + w.line * p.dt.line + w.c0;
    const T *z = p.z.p ? static_cast<const T *>(p.z.p) + w.line * p.z.line + w.c0 : nullptr;
    const T *Cc = static_cast<const T *>(p.C.p) + w.line * p.C.line + w.group * p.C_group;
    const T *yb = static_cast<const T *>(o.yb.p) + w.line * o.yb.line + w.c0;
    const int64_t own = (int64_t)(w.c0 + dl) * p.n + n0, dn = p.d * p.n;
    V A2[KP], g[KP];
    load_states<SN>(static_cast<const C *>(p.A) + own, n, in, A2);
#pragma unroll
    for (int j = 0; j < KP; ++j) A2[j] = mul2(A2[j], make2(log2e<C>(), log2e<C>()));
    zero_states<SN>(g);
    const C bias = in && p.dt_bias ? static_cast<const C *>(p.dt_bias)[w.c0 + dl] : (C)0;
    C total = 0;
    const bool full = p.dt.wide && o.yb.wide && (!z || p.z.wide) && p.C.wide && w.nch == CW && whole_n<T>(p.n);
    auto fetch_as = [&](auto whole, int r, int to) {
        constexpr bool F = whole.value;
        raw_fetch<CW, F>(sm.raw[to].dt, dt, p.dt, r, w.r1, w.nch, lane);
        raw_fetch<CW, F>(sm.raw[to].yb, yb, o.yb, r, w.r1, w.nch, lane);
        if (z) raw_fetch<CW, F>(sm.raw[to].z, z, p.z, r, w.r1, w.nch, lane);
        raw_fetch_n<32, F>(sm.raw[to].c, Cc, p.C.row, r, w.r1, p.n, p.C.wide, lane);
        cp_async_commit();
    };
    auto fetch = [&](int r, int to) {
        if (full && r + R <= w.r1)
            fetch_as(std::true_type(), r, to);
        else
            fetch_as(std::false_type(), r, to);
    };
    raw_clear_n<32>(sm.raw[0].c, p.n, lane);
    raw_clear_n<32>(sm.raw[1].c, p.n, lane);
    __syncwarp();
    int k = p.rows.find(w.r1 - 1);          // the sequence of the row at hand
    int rt = w.r0 + (w.r1 - w.r0 - 1) / R * R, now = 0;
    fetch(rt, 0);
    for (; rt >= w.r0; rt -= R, now ^= 1) {
        const int nr = min(R, w.r1 - rt);
        int k0 = k;
        while (p.rows.start(k0) > rt) --k0;
        const uint32_t st = p.rows.starts(rt, R, k0, lane);
        const auto &raw = sm.raw[now];
        cp_async_wait_all();
        __syncwarp();
        if (rt > w.r0) fetch(rt - R, now ^ 1);
        raw_stage_n<32>(sm.c, raw.c, lane);
        {
            C a[PER], y[PER];
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                a[i] = Elem<T>::up(raw.dt[nl + LN * i][dl]) + bias;
                y[i] = Elem<T>::up(raw.yb[nl + LN * i][dl]);
            }
            if (p.softplus) {
#pragma unroll
                for (int i = 0; i < PER; ++i) a[i] = softplus_of<T>(a[i]);
            }
            if (z) {
#pragma unroll
                for (int i = 0; i < PER; ++i) {
                    const C v = Elem<T>::up(raw.z[nl + LN * i][dl]);
                    y[i] *= v * sigmoid_(v);
                }
            }
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const int t = nl + LN * i;
                sm.dt[t][dl] = a[i];
                sm.yb[t][dl] = y[i];
                if (t < nr) total += a[i];
            }
        }
        __syncwarp();
        for (int t = nr - 1; t >= 0;) {
            if ((st >> (t + 1)) & 1u) {         // the last row of its sequence
                if (rt + t < p.rows.start(k)) --k;
                if (o.stateb)
                    load_states<SN>(static_cast<const C *>(o.stateb) + p.rows.number(k, w.line) * dn + own, n, in, g);
                else
                    zero_states<SN>(g);
            }
            // down to the row behind the next such row
            const uint32_t earlier = st & ((2u << t) - 2u);
            const int te = earlier ? 31 - __clz(earlier) : 0;
            for (; t - 3 >= te; t -= 4) {
#pragma unroll
                for (int i = 0; i < 4; ++i) scan_ends_row(sm, t - i, dl, n0, A2, g);
            }
            for (; t >= te; --t) scan_ends_row(sm, t, dl, n0, A2, g);
        }
        __syncwarp();
    }
#pragma unroll
    for (int m = CW; m < 32; m *= 2) total += shfl_xor_(total, m);
    if (in) {
        const int64_t piece = w.line * p.segs + w.seg;
        store_states<SN>(static_cast<C *>(p.ends) + piece * dn + own, n, in, g);
        if (nl == 0) static_cast<C *>(p.sums)[piece * p.d + w.c0 + dl] = total;
    }
}
template <class K> cudaError_t scan_ends_run(const ScanArgs &p, const ScanGrads &o, cudaStream_t s)
{
    constexpr int warps = SCAN_WARPS;
    constexpr int bytes = warps * (int)sizeof(ScanEndsSmem<K>);
    static_assert(bytes <= 227 * 1024, "fits an SM");
    const int64_t tiles = (p.d / p.groups + K::CW - 1) / K::CW;
    const dim3 grid((unsigned)(p.lines * p.segs), (unsigned)(p.groups * ((tiles + warps - 1) / warps)));
    const cudaError_t e =
        cudaFuncSetAttribute(scan_backward_ends_kernel<K>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    scan_backward_ends_kernel<K><<<grid, warps * 32, bytes, s>>>(p, o);
    return cudaSuccess;
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
#pragma unroll 8
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

template <class T, int NP> cudaError_t scan_backward_run(const ScanArgs &p, const ScanGrads &o, cudaStream_t s)
{
    using K = ScanBwdTile<T, NP>;
    const int64_t per = p.d / p.groups, tiles = (per + K::CW - 1) / K::CW;
    const int parts = (int)((tiles + SCAN_WARPS - 1) / SCAN_WARPS);
    const dim3 grid((unsigned)(p.lines * p.segs), (unsigned)(p.groups * parts));
    if (p.segs > 1) {
        const cudaError_t e = with_lanes<T, NP>(p.ends_lanes, [&](auto k) { return scan_ends_run<decltype(k)>(p, o, s); });
        if (e != cudaSuccess) return e;
    }
    const bool padded = p.n != NP || per % (K::CW * SCAN_WARPS) != 0;
    const cudaError_t e = padded ? scan_backward_start<K, true>(p, o, grid, s) : scan_backward_start<K, false>(p, o, grid, s);
    if (e != cudaSuccess) return e;
    const int64_t bc = (p.lines * p.rows.rows * p.groups * 2 * NP + 255) / 256;
    const int64_t params = (p.d * (p.n + 2) + 31) / 32;
    scan_sums_kernel<T, NP><<<(unsigned)(bc + params), 256, 0, s>>>(p, o, bc, parts);
    return cudaGetLastError();
}

}  // namespace
}  // namespace selinv
