// Forward of the selective scan.  One warp works on CW channels of one
// segment of a line, row after row: a thread keeps TD x TN states in
// registers, packed in pairs of channels, and forms the TD partial sums of
// y, which the LN lanes that share those channels then add up.  Rows are
// staged SCAN_R at a time in the warp's own shared memory (steps, steps times
// x, B and C as pairs of equal values); the next rows' loads are in flight
// meanwhile.  No two warps wait for one another.
#pragma once

#include "scan.cuh"

namespace selinv {
namespace {

template <class K> struct ScanFwdSmem {
    using C = typename K::C;
    C dt[SCAN_R][K::PITCH], u[SCAN_R][K::PITCH], y[SCAN_R][K::PITCH];
    C b[SCAN_R][2 * K::NP], c[SCAN_R][2 * K::NP];
};
template <class K> constexpr bool scan_fwd_aligned =
    sizeof(ScanFwdSmem<K>) % 16 == 0 && offsetof(ScanFwdSmem<K>, b) % 16 == 0 && offsetof(ScanFwdSmem<K>, y) % 16 == 0;

// MAIN: outputs.  Otherwise only what each segment leaves behind: its end state from a zero state, its sum of steps.
template <class K, bool MAIN>
__global__ void __launch_bounds__(SCAN_WARPS * 32) scan_kernel(const __grid_constant__ ScanArgs p)
{
    using T = typename K::T;
    using C = typename K::C;
    using V = typename K::V;
    constexpr int R = SCAN_R, CW = K::CW, E = K::E, EB = K::EB, NP = K::NP, TD = K::TD, TN = K::TN, TP = K::TP;
    extern __shared__ __align__(16) char smem_raw[];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    ScanFwdSmem<K> &sm = reinterpret_cast<ScanFwdSmem<K> *>(smem_raw)[warp];
    ScanPlace w;
    if (!scan_place<K>(p, warp, w)) return;

    const int n = p.n, d0 = (lane / K::LN) * TD, n0 = (lane % K::LN) * TN;
    const T *x = static_cast<const T *>(p.x.p) + w.line * p.x.line + w.c0;
    const T *dt = static_cast<const T *>(p.dt.p) + w.line * p.dt.line + w.c0;
    const T *z = p.z.p ? static_cast<const T *>(p.z.p) + w.line * p.z.line + w.c0 : nullptr;
    const T *B = static_cast<const T *>(p.B.p) + w.line * p.B.line + w.group * p.B_group;
    const T *Cc = static_cast<const T *>(p.C.p) + w.line * p.C.line + w.group * p.C_group;
    T *y = static_cast<T *>(p.y.p) + w.line * p.y.line + w.c0;
    const int64_t part = (int64_t)w.c0 * n, dn = p.d * n;
    const C *state = static_cast<const C *>(p.state);
    C *state_out = static_cast<C *>(p.state_out);

    // sequences without rows end as they began
    if (MAIN && state_out && p.rows.table && blockIdx.x == 0) {
        for (int64_t e = 0; e < p.sequences - p.rows.live; ++e) {
            const int64_t at = p.rows.table[2 * p.rows.live + 1 + e] * dn + part;
            for (int i = lane; i < w.nch * n; i += 32) state_out[at + i] = state ? state[at + i] : (C)0;
        }
    }
    if (w.r0 >= w.r1) return;

    V A2[TP][TN], h[TP][TN];
    load_part<K>(static_cast<const C *>(p.A) + part, n, w.nch, lane, A2, (C)0);
#pragma unroll
    for (int q = 0; q < TP; ++q)
#pragma unroll
        for (int j = 0; j < TN; ++j) {
            A2[q][j] = mul2(A2[q][j], make2(log2e<C>(), log2e<C>()));
            h[q][j] = make2((C)0, (C)0);
        }
    const int ce = (lane % (CW / E)) * E;       // the channels this lane converts
    C bias[E], skip[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const bool in = ce + e < w.nch;
        bias[e] = in && p.dt_bias ? static_cast<const C *>(p.dt_bias)[w.c0 + ce + e] : (C)0;
        skip[e] = MAIN && in && p.D ? static_cast<const C *>(p.D)[w.c0 + ce + e] : (C)0;
    }

    int64_t k = p.rows.find(w.r0);
    if (MAIN && w.seg > 0 && p.rows.start(k) < w.r0) {
        // the state that the segments before this one leave: of the first that holds rows of this sequence, its end
        // state; each later one decays what came before by its own sum of steps
        const C *ends = static_cast<const C *>(p.ends) + w.line * p.segs * dn + part;
        const C *sums = static_cast<const C *>(p.sums) + w.line * p.segs * p.d + w.c0;
        int s = (int)(p.rows.start(k) / p.seg_rows);
        load_part<K>(ends + s * dn, n, w.nch, lane, h, (C)0);
        for (++s; s < w.seg; ++s) {
            V e[TP][TN];
            load_part<K>(ends + s * dn, n, w.nch, lane, e, (C)0);
#pragma unroll
            for (int q = 0; q < TP; ++q) {
                V t;
                t.x = d0 + 2 * q < w.nch ? sums[s * p.d + d0 + 2 * q] : (C)0;
                t.y = d0 + 2 * q + 1 < w.nch ? sums[s * p.d + d0 + 2 * q + 1] : (C)0;
#pragma unroll
                for (int j = 0; j < TN; ++j) {
                    const V a = mul2(t, A2[q][j]);
                    h[q][j] = fma2(make2(exp2_(a.x), exp2_(a.y)), h[q][j], e[q][j]);
                }
            }
        }
    }

    ScanLoad<K, K::PER, E, CW / E> xl, dl, zl;
    ScanLoad<K, K::BPER, EB, NP / EB> bl, cl;
    auto fetch = [&](int64_t r) {
        xl.load(x, p.x.row, r, w.r1, w.nch, p.x.wide, lane);
        dl.load(dt, p.dt.row, r, w.r1, w.nch, p.dt.wide, lane);
        bl.load(B, p.B.row, r, w.r1, n, p.B.wide, lane);
        if (MAIN) cl.load(Cc, p.C.row, r, w.r1, n, p.C.wide, lane);
    };
    fetch(w.r0);
    V total[TP];
#pragma unroll
    for (int q = 0; q < TP; ++q) total[q] = make2((C)0, (C)0);
    const bool pad = n < NP;

    for (int64_t rt = w.r0; rt < w.r1; rt += R) {
        // stage
#pragma unroll
        for (int i = 0; i < K::PER; ++i) {
            const int row = (lane + 32 * i) / (CW / E);
            if (row >= R) break;
            C a[E], b[E];
#pragma unroll
            for (int e = 0; e < E; ++e) {
                a[e] = dl.v[i].get(e) + bias[e];
                if (p.softplus) a[e] = softplus_(a[e]);
                b[e] = a[e] * xl.v[i].get(e);
            }
            put<E>(&sm.dt[row][ce], a);
            put<E>(&sm.u[row][ce], b);
        }
#pragma unroll
        for (int i = 0; i < K::BPER; ++i) {
            const int vec = lane + 32 * i, row = vec / (NP / EB), e0 = (vec % (NP / EB)) * EB;
            if (row >= R) break;
            C a[2 * EB], b[2 * EB];
#pragma unroll
            for (int e = 0; e < EB; ++e) {
                a[2 * e] = a[2 * e + 1] = bl.v[i].get(e);
                if (MAIN) b[2 * e] = b[2 * e + 1] = cl.v[i].get(e);
            }
            put<2 * EB>(&sm.b[row][2 * e0], a);
            if (MAIN) put<2 * EB>(&sm.c[row][2 * e0], b);
        }
        const auto xc = xl;
        if (MAIN && z) zl.load(z, p.z.row, rt, w.r1, w.nch, p.z.wide, lane);
        if (rt + R < w.r1) fetch(rt + R);
        const uint32_t st = p.rows.starts(rt, R, k, lane);
        const int nr = (int)min((int64_t)R, w.r1 - rt);
        __syncwarp();
        if (MAIN && p.kept) {
            const int64_t tiles = (p.rows.rows + R - 1) / R;
            store_part<K>(static_cast<C *>(p.kept) + (w.line * tiles + rt / R) * dn + part, n, w.nch, lane, h);
        }
        for (int t = 0; t < nr;) {
            if ((st >> t) & 1u) {
                if (rt + t > p.rows.start(k)) ++k;
                if (state) {
                    load_part<K>(state + p.rows.number(k, w.line) * dn + part, n, w.nch, lane, h, (C)0);
                } else {
#pragma unroll
                    for (int q = 0; q < TP; ++q)
#pragma unroll
                        for (int j = 0; j < TN; ++j) h[q][j] = make2((C)0, (C)0);
                }
            }
            const uint32_t later = st >> (t + 1);
            const int te = later ? min(nr, t + __ffs(later)) : nr;
#pragma unroll 4
            for (; t < te; ++t) {
                V dt2[TP], u2[TP], b2[TN], c2[TN], y2[TP];
                get<TP>(&sm.dt[t][d0], dt2);
                get<TP>(&sm.u[t][d0], u2);
                get<TN>(&sm.b[t][2 * n0], b2);
                if (MAIN) get<TN>(&sm.c[t][2 * n0], c2);
#pragma unroll
                for (int q = 0; q < TP; ++q) {
#pragma unroll
                    for (int j = 0; j < TN; ++j) {
                        const V e = mul2(dt2[q], A2[q][j]);
                        h[q][j] = fma2(make2(exp2_(e.x), exp2_(e.y)), h[q][j], mul2(u2[q], b2[j]));
                    }
                    if (!MAIN) total[q] = add2(total[q], dt2[q]);
                }
                if (pad) {      // an infinite x must not reach y through a state that is not there
#pragma unroll
                    for (int j = 0; j < TN; ++j)
                        if (n0 + j >= n) {
#pragma unroll
                            for (int q = 0; q < TP; ++q) h[q][j] = make2((C)0, (C)0);
                        }
                }
                if (MAIN) {
                    C v[TD];
#pragma unroll
                    for (int q = 0; q < TP; ++q) {
                        y2[q] = mul2(c2[0], h[q][0]);
#pragma unroll
                        for (int j = 1; j < TN; ++j) y2[q] = fma2(c2[j], h[q][j], y2[q]);
                        v[2 * q] = y2[q].x, v[2 * q + 1] = y2[q].y;
                    }
                    scatter_sum<TD, 1, K::LN>(v, lane);
                    constexpr int KEEP = TD > K::LN ? TD / K::LN : 1;
                    if (scatter_writes<TD, 1, K::LN>(lane)) {
                        const int f = d0 + scatter_first<TD, 1, K::LN>(lane);
#pragma unroll
                        for (int i = 0; i < KEEP; ++i) sm.y[t][f + i] = v[i];
                    }
                }
            }
            if (MAIN && state_out && ((st >> t) & 1u))
                store_part<K>(state_out + p.rows.number(k, w.line) * dn + part, n, w.nch, lane, h);
        }
        __syncwarp();
        if (MAIN) {
#pragma unroll
            for (int i = 0; i < K::PER; ++i) {
                const int row = (lane + 32 * i) / (CW / E);
                if (row >= nr) break;
                C v[E];
                get<E>(&sm.y[row][ce], v);
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    v[e] += skip[e] * xc.v[i].get(e);
                    if (z) {
                        const C g = zl.v[i].get(e);
                        v[e] *= g * sigmoid_(g);
                    }
                }
                Pack<T, E> out;
                out.set(v);
                out.store(y + (rt + row) * p.y.row + ce, w.nch - ce, p.y.wide);
            }
            __syncwarp();
        }
    }
    if (!MAIN) {
        C *ends = static_cast<C *>(p.ends) + (w.line * p.segs + w.seg) * dn + part;
        C *sums = static_cast<C *>(p.sums) + (w.line * p.segs + w.seg) * p.d + w.c0;
        store_part<K>(ends, n, w.nch, lane, h);
        if (lane % K::LN == 0) {
#pragma unroll
            for (int q = 0; q < TP; ++q) {
                if (d0 + 2 * q < w.nch) sums[d0 + 2 * q] = total[q].x;
                if (d0 + 2 * q + 1 < w.nch) sums[d0 + 2 * q + 1] = total[q].y;
            }
        }
    }
}

template <class K> cudaError_t scan_run(const ScanArgs &p, cudaStream_t s)
{
    const int64_t per = p.d / p.groups, tiles = (per + K::CW - 1) / K::CW;
    const int64_t gy = p.groups * ((tiles + SCAN_WARPS - 1) / SCAN_WARPS), gx = p.lines * p.segs;
    const dim3 grid((unsigned)gx, (unsigned)gy);
    static_assert(scan_fwd_aligned<K>, "staged rows lie on 16 bytes");
    constexpr int bytes = SCAN_WARPS * (int)sizeof(ScanFwdSmem<K>);
    if (p.segs > 1) {
        cudaError_t e = cudaFuncSetAttribute(scan_kernel<K, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != cudaSuccess) return e;
        scan_kernel<K, false><<<grid, SCAN_WARPS * 32, bytes, s>>>(p);
    }
    cudaError_t e = cudaFuncSetAttribute(scan_kernel<K, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    scan_kernel<K, true><<<grid, SCAN_WARPS * 32, bytes, s>>>(p);
    return cudaGetLastError();
}

}  // namespace
}  // namespace selinv
