// Forward of the selective scan.  A lane owns one channel and keeps its
// states in registers, in pairs, so that y needs no other lane; a warp works
// on 32 neighbouring channels of one segment of a line, row after row, and
// waits for no other warp.  SCAN_R rows at a time: x, dt and z arrive in the
// warp's shared memory asynchronously, one tile ahead; a first run over the
// rows forms the steps and their products with x, a second one the states and
// the sums of y, a third one the outputs.  What bounds it is the special
// function unit: one power of two per row, channel and state, 16 a cycle and
// SM, and two to three more per row and channel.
#pragma once

#include "scan.cuh"

namespace selinv {
namespace {

// SCAN_R rows as they lie in memory.
template <class T, int NP> struct ScanRaw {
    alignas(16) T x[SCAN_R][32], dt[SCAN_R][32], z[SCAN_R][32], b[SCAN_R][NP], c[SCAN_R][NP];
};
template <class T, int NP> struct ScanFwdSmem {
    using C = typename Elem<T>::C;
    ScanRaw<T, NP> raw[2];
    // steps, and then the outputs in T, row by row; steps times x, and then the sums of y
    alignas(16) C dt[SCAN_R][32], u[SCAN_R][32];
    alignas(16) C b[SCAN_R][NP], c[SCAN_R][NP];
};

// One row: states on, this channel's sum of y.
template <class T, int NP, bool MAIN>
SELINV_DEVINL typename Elem<T>::C scan_row(const ScanFwdSmem<T, NP> &sm, int t, int lane, const typename Two<typename Elem<T>::C>::V *A2,
                                           typename Two<typename Elem<T>::C>::V *h)
{
    using C = typename Elem<T>::C;
    using V = typename Two<C>::V;
    const C dt = sm.dt[t][lane], u = sm.u[t][lane];
    const V dt2 = make2(dt, dt), u2 = make2(u, u);
    V y[2] = {make2((C)0, (C)0), make2((C)0, (C)0)};
#pragma unroll
    for (int j = 0; j < NP / 2; j += 2) {
        V b[2], c[2];
        get<2>(&sm.b[t][2 * j], b);
        if (MAIN) get<2>(&sm.c[t][2 * j], c);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            h[j + i] = fma2(exp2_2(mul2(dt2, A2[j + i])), h[j + i], mul2(u2, b[i]));
            if (MAIN) y[i] = fma2(c[i], h[j + i], y[i]);
        }
    }
    const V s = add2(y[0], y[1]);
    return s.x + s.y;
}

// MAIN: outputs.  Otherwise only what each segment leaves behind: its end state from a zero state, its sum of steps.
template <class T, int NP, bool MAIN>
__global__ void __launch_bounds__(SCAN_WARPS * 32) scan_kernel(const __grid_constant__ ScanArgs p)
{
    using C = typename Elem<T>::C;
    using V = typename Two<C>::V;
    constexpr int R = SCAN_R, E = 16 / (int)sizeof(T);
    extern __shared__ __align__(16) char smem_raw[];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    ScanFwdSmem<T, NP> &sm = reinterpret_cast<ScanFwdSmem<T, NP> *>(smem_raw)[warp];
    ScanPlace w;
    if (!scan_place(p, warp, blockDim.x / 32, 32, w) || (!MAIN && w.seg == p.segs - 1)) return;

    const int n = p.n;
    const bool in = lane < w.nch;
    const T *x = static_cast<const T *>(p.x.p) + w.line * p.x.line + w.c0;
    const T *dt = static_cast<const T *>(p.dt.p) + w.line * p.dt.line + w.c0;
    const T *z = p.z.p ? static_cast<const T *>(p.z.p) + w.line * p.z.line + w.c0 : nullptr;
    const T *B = static_cast<const T *>(p.B.p) + w.line * p.B.line + w.group * p.B_group;
    const T *Cc = static_cast<const T *>(p.C.p) + w.line * p.C.line + w.group * p.C_group;
    T *y = static_cast<T *>(p.y.p) + w.line * p.y.line + w.c0;
    const int64_t own = (int64_t)(w.c0 + lane) * n, dn = p.d * n;       // this lane's place in a [d, n] array
    const C *state = static_cast<const C *>(p.state);
    C *state_out = static_cast<C *>(p.state_out);

    // sequences without rows end as they began
    if (MAIN && state_out && p.rows.table && blockIdx.x == 0 && in) {
        for (int64_t e = 0; e < p.sequences - p.rows.live; ++e) {
            const int64_t at = p.rows.empty(e) * dn + own;
            for (int i = 0; i < n; ++i) state_out[at + i] = state ? state[at + i] : (C)0;
        }
    }
    if (w.r0 >= w.r1) return;

    V A2[NP / 2], h[NP / 2];
    load_states<NP>(static_cast<const C *>(p.A) + own, n, in, A2);
#pragma unroll
    for (int j = 0; j < NP / 2; ++j) A2[j] = mul2(A2[j], make2(log2e<C>(), log2e<C>()));
    zero_states<NP>(h);
    const C bias = in && p.dt_bias ? static_cast<const C *>(p.dt_bias)[w.c0 + lane] : (C)0;
    const C skip = MAIN && in && p.D ? static_cast<const C *>(p.D)[w.c0 + lane] : (C)0;

    int k = p.rows.find(w.r0);
    if (MAIN && w.seg > 0 && p.rows.start(k) < w.r0) {
        // the state that the segments before this one leave: of the first that holds rows of this sequence, its end
        // state; each later one decays what came before by its own sum of steps
        scan_join<NP, C>(p, w.line, p.rows.start(k) / p.seg_rows, w.seg, 1, w.c0 + lane, own, n, in, A2, h);
    }

    auto fetch = [&](int r, int to) {
        raw_fetch<32>(sm.raw[to].x, x, p.x.row, r, w.r1, w.nch, p.x.wide, lane);
        raw_fetch<32>(sm.raw[to].dt, dt, p.dt.row, r, w.r1, w.nch, p.dt.wide, lane);
        if (MAIN && z) raw_fetch<32>(sm.raw[to].z, z, p.z.row, r, w.r1, w.nch, p.z.wide, lane);
        raw_fetch_n<32>(sm.raw[to].b, B, p.B.row, r, w.r1, n, p.B.wide, lane);
        if (MAIN) raw_fetch_n<32>(sm.raw[to].c, Cc, p.C.row, r, w.r1, n, p.C.wide, lane);
        cp_async_commit();
    };
    fetch(w.r0, 0);
    C total = 0;

    for (int rt = w.r0; rt < w.r1; rt += R) {
        const int at = ((rt - w.r0) / R) & 1;
        const ScanRaw<T, NP> &raw = sm.raw[at];
        cp_async_wait_all();
        __syncwarp();
        if (rt + R < w.r1) fetch(rt + R, at ^ 1);
        raw_stage_n<32>(sm.b, raw.b, lane);
        if (MAIN) raw_stage_n<32>(sm.c, raw.c, lane);
        const int nr = min(R, w.r1 - rt);
        {       // all rows' loads before the stores: the chains of one row are long, those of sixteen run side by side
            C v[R], u[R];
#pragma unroll
            for (int t = 0; t < R; ++t) {
                v[t] = Elem<T>::up(raw.dt[t][lane]) + bias;
                u[t] = Elem<T>::up(raw.x[t][lane]);
            }
            if (p.softplus) {
#pragma unroll
                for (int t = 0; t < R; ++t) v[t] = softplus_(v[t]);
            }
#pragma unroll
            for (int t = 0; t < R; ++t) {
                sm.dt[t][lane] = v[t];
                sm.u[t][lane] = v[t] * u[t];
                if (!MAIN && t < nr) total += v[t];
            }
        }
        __syncwarp();
        const uint32_t st = p.rows.starts(rt, R, k, lane);
        if (MAIN && p.kept) {
            const int tiles = (p.rows.rows + R - 1) / R;
            store_states<NP>(static_cast<C *>(p.kept) + (w.line * tiles + rt / R) * dn + own, n, in, h);
        }
        for (int t = 0; t < nr;) {
            if ((st >> t) & 1u) {
                if (rt + t > p.rows.start(k)) ++k;
                if (state) {
                    load_states<NP>(state + p.rows.number(k, w.line) * dn + own, n, in, h);
                } else {
                    zero_states<NP>(h);
                }
            }
            const uint32_t later = st >> (t + 1);
            const int te = later ? min(nr, t + __ffs(later)) : nr;
            for (; t + 4 <= te; t += 4) {       // four rows' loads before their stores
                C v[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = scan_row<T, NP, MAIN>(sm, t + i, lane, A2, h);
                if (MAIN) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) sm.u[t + i][lane] = v[i];
                }
            }
            for (; t < te; ++t) {
                const C v = scan_row<T, NP, MAIN>(sm, t, lane, A2, h);
                if (MAIN) sm.u[t][lane] = v;
            }
            if (MAIN && state_out && ((st >> t) & 1u))
                store_states<NP>(state_out + p.rows.number(k, w.line) * dn + own, n, in, h);
        }
        if (MAIN) {
            C v[R];
#pragma unroll
            for (int t = 0; t < R; ++t) v[t] = sm.u[t][lane] + skip * Elem<T>::up(raw.x[t][lane]);
            if (z) {
#pragma unroll
                for (int t = 0; t < R; ++t) {
                    const C g = Elem<T>::up(raw.z[t][lane]);
                    v[t] *= g * sigmoid_(g);
                }
            }
            T(*out)[32] = reinterpret_cast<T(*)[32]>(&sm.dt[0][0]);
            __syncwarp();       // all lanes are done with the steps
#pragma unroll
            for (int t = 0; t < R; ++t) out[t][lane] = Elem<T>::down(v[t]);
            __syncwarp();
            if (p.y.wide && w.nch == 32) {
                constexpr int LANES = 32 / E, ROWS = 32 / LANES;
                const int row = lane / LANES, e = (lane % LANES) * E;
#pragma unroll
                for (int i = 0; i < R; i += ROWS)
                    if (row + i < nr)
                        *reinterpret_cast<uint4 *>(y + (int64_t)(rt + row + i) * p.y.row + e) =
                            *reinterpret_cast<const uint4 *>(&out[row + i][e]);
            } else if (in) {
                for (int t = 0; t < nr; ++t) y[(int64_t)(rt + t) * p.y.row + lane] = out[t][lane];
            }
        }
        __syncwarp();
    }
    if (!MAIN && in) {
        const int64_t piece = w.line * p.segs + w.seg;
        store_states<NP>(static_cast<C *>(p.ends) + piece * dn + own, n, in, h);
        static_cast<C *>(p.sums)[piece * p.d + w.c0 + lane] = total;
    }
}

template <class T, int NP> cudaError_t scan_run(const ScanArgs &p, cudaStream_t s)
{
    // float64 with many states: fewer warps fit
    constexpr int warps = SCAN_WARPS * sizeof(ScanFwdSmem<T, NP>) <= 227 * 1024 ? SCAN_WARPS : SCAN_WARPS / 2;
    constexpr int bytes = warps * (int)sizeof(ScanFwdSmem<T, NP>);
    static_assert(bytes <= 227 * 1024, "fits an SM");
    const int64_t per = p.d / p.groups, tiles = (per + 31) / 32;
    const dim3 grid((unsigned)(p.lines * p.segs), (unsigned)(p.groups * ((tiles + warps - 1) / warps)));
    if (p.segs > 1) {
        cudaError_t e = cudaFuncSetAttribute(scan_kernel<T, NP, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != cudaSuccess) return e;
        scan_kernel<T, NP, false><<<grid, warps * 32, bytes, s>>>(p);
    }
    cudaError_t e = cudaFuncSetAttribute(scan_kernel<T, NP, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    scan_kernel<T, NP, true><<<grid, warps * 32, bytes, s>>>(p);
    return cudaGetLastError();
}

}  // namespace
}  // namespace selinv
