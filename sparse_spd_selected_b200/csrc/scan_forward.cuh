// Forward of the selective scan.  A lane owns SN = NP / LN states of one
// channel and keeps them in registers, in pairs; the LN lanes of a channel add
// their parts of y.  A warp works on 32 / LN neighbouring channels of one
// segment of a line, row after row, and waits for no other warp.  SCAN_R rows
// at a time: x, dt and z arrive in the warp's shared memory asynchronously,
// one tile ahead; a first run over the rows forms the steps and their products
// with x, a second one the states and the sums of y, a third one the outputs.
// What bounds it is the special function unit: one power of two per row,
// channel and state, 16 a cycle and SM, and three more per row and
// channel (one with the softplus, two with z).  4 x 2048 x 4096 x 16 in bfloat16,
// states kept: 306 us for 5.4e8 states, 137 us of that unit alone and 62 us of
// memory; one or two warps per scheduler do not keep it busy.  Cut into segments
// (one line of 4096 x 2048 x 16: 117 us, 46 of them the summary run) it is 65 to
// 75 % busy, but the powers are formed twice.  A polynomial for a part of the
// powers on the FMA pipe gave nothing (issue slots are the next bound), joining
// the segments in batches of four took 125 us, for its registers.
#pragma once

#include "scan.cuh"

namespace selinv {
namespace {

// A warp's tile: lane = nl * CW + dl holds channel dl and the states nl * SN on.
template <class T_, int NP_, int LN_> struct ScanFwdTile {
    using T = T_;
    using C = typename Elem<T>::C;
    using V = typename Two<C>::V;
    static constexpr int NP = NP_, LN = LN_, SN = NP / LN, KP = SN / 2, CW = 32 / LN, PER = SCAN_R / LN;
    static_assert(SN >= 4 && CW >= 8, "whole vectors of states and of channels");
};
// SCAN_R rows as they lie in memory.
template <class K> struct ScanRaw {
    using T = typename K::T;
    alignas(16) T x[SCAN_R][K::CW], dt[SCAN_R][K::CW], z[SCAN_R][K::CW], b[SCAN_R][K::NP], c[SCAN_R][K::NP];
};
template <class K> struct ScanFwdSmem {
    using C = typename K::C;
    ScanRaw<K> raw[2];
    // steps, and then the outputs in T, row by row; steps times x, and then the sums of y
    alignas(16) C dt[SCAN_R][K::CW], u[SCAN_R][K::CW];
    alignas(16) C b[SCAN_R][K::NP], c[SCAN_R][K::NP];
};

// One row: states on, this lane's part of y.  REAL: keeps those that do not exist (from n on) at zero whatever comes.
template <class K, bool MAIN, bool REAL>
SELINV_DEVINL typename K::C scan_row(const ScanFwdSmem<K> &sm, int t, int dl, int n0, int n, const typename K::V *A2,
                                     typename K::V *h)
{
    using C = typename K::C;
    using V = typename K::V;
    const C dt = sm.dt[t][dl], u = sm.u[t][dl];
    const V dt2 = make2(dt, dt), u2 = make2(u, u);
    V y[2] = {make2((C)0, (C)0), make2((C)0, (C)0)};
#pragma unroll
    for (int j = 0; j < K::KP; j += 2) {
        V b[2], c[2];
        get<2>(&sm.b[t][n0 + 2 * j], b);
        if (MAIN) get<2>(&sm.c[t][n0 + 2 * j], c);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            h[j + i] = fma2(decay2(dt2, A2[j + i]), h[j + i], mul2(u2, b[i]));
            if (REAL) h[j + i] = real_states(h[j + i], j + i, n);
            if (MAIN) y[i] = fma2(c[i], h[j + i], y[i]);
        }
    }
    const V s = add2(y[0], y[1]);
    return s.x + s.y;
}

// MAIN: outputs.  Otherwise only what each segment leaves behind: its end state from a zero state, its sum of steps.
// BLOCKS per SM that the registers are kept to.  Four (128 registers), as many as segments are planned for, where they
// fill the GPU (4096 x 2048 x 16: 121 us, 132 without); none where no more than two come to an SM, whose warps work
// better with all they want (4 x 2048 x 4096 x 16, one lane: 358 us, 404 with).
// PADDED: some of a tile's states do not exist.  A tile with infinities then goes on row by row with zeros for them; a kernel of
// its own, since the choice costs the others 3 % (4 x 2048 x 4096 x 8 in bfloat16: 234 us for 226).
template <class K, bool MAIN, int BLOCKS, bool PADDED>
__global__ void __launch_bounds__(SCAN_WARPS * 32, BLOCKS) scan_kernel(const __grid_constant__ ScanArgs p)
{
    using T = typename K::T;
    using C = typename K::C;
    using V = typename K::V;
    constexpr int R = SCAN_R, E = 16 / (int)sizeof(T), LN = K::LN, SN = K::SN, CW = K::CW, KP = K::KP, PER = K::PER;
    extern __shared__ __align__(16) char smem_raw[];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    ScanFwdSmem<K> &sm = reinterpret_cast<ScanFwdSmem<K> *>(smem_raw)[warp];
    ScanPlace w;
    if (!scan_place(p, warp, blockDim.x / 32, CW, w) || (!MAIN && w.seg == p.segs - 1)) return;

    const int nl = lane / CW, dl = lane % CW, n0 = nl * SN, n = p.n - n0;       // n: of this lane's states and those behind
    const bool in = dl < w.nch;
    const T *x = static_cast<const T *>(p.x.p) + w.line * p.x.line + w.c0;
    const T *dt = static_cast<const T *>(p.dt.p) + w.line * p.dt.line + w.c0;
    const T *z = p.z.p ? static_cast<const T *>(p.z.p) + w.line * p.z.line + w.c0 : nullptr;
    const T *B = static_cast<const T *>(p.B.p) + w.line * p.B.line + w.group * p.B_group;
    const T *Cc = static_cast<const T *>(p.C.p) + w.line * p.C.line + w.group * p.C_group;
    T *y = static_cast<T *>(p.y.p) + w.line * p.y.line + w.c0;
    const int64_t own = (int64_t)(w.c0 + dl) * p.n + n0, dn = p.d * p.n;        // this lane's place in a [d, n] array
    const C *state = static_cast<const C *>(p.state);
    C *state_out = static_cast<C *>(p.state_out);

    // sequences without rows end as they began
    if (MAIN && state_out && p.rows.table && blockIdx.x == 0 && in) {
        for (int64_t e = 0; e < p.sequences - p.rows.live; ++e) {
            const int64_t at = p.rows.empty(e) * dn + own;
            for (int i = 0; i < min(n, SN); ++i) state_out[at + i] = state ? state[at + i] : (C)0;
        }
    }
    if (w.r0 >= w.r1) return;

    V A2[KP], h[KP];
    load_states<SN>(static_cast<const C *>(p.A) + own, n, in, A2);
#pragma unroll
    for (int j = 0; j < KP; ++j) A2[j] = mul2(A2[j], make2(log2e<C>(), log2e<C>()));
    zero_states<SN>(h);
    const C bias = in && p.dt_bias ? static_cast<const C *>(p.dt_bias)[w.c0 + dl] : (C)0;
    const C skip = MAIN && in && p.D ? static_cast<const C *>(p.D)[w.c0 + dl] : (C)0;

    int k = p.rows.find(w.r0);
    if (MAIN && w.seg > 0 && p.rows.start(k) < w.r0) {
        // the state that the segments before this one leave: of the first that holds rows of this sequence, its end
        // state; each later one decays what came before by its own sum of steps
        scan_join<SN, C>(p, w.line, p.rows.start(k) / p.seg_rows, w.seg, 1, w.c0 + dl, own, n, in, A2, h);
    }

    const bool full = p.x.wide && p.dt.wide && (!z || p.z.wide) && p.B.wide && p.C.wide && w.nch == CW && whole_n<T>(p.n);
    auto fetch_as = [&](auto whole, int r, int to) {
        constexpr bool F = whole.value;
        raw_fetch<CW, F>(sm.raw[to].x, x, p.x, r, w.r1, w.nch, lane);
        raw_fetch<CW, F>(sm.raw[to].dt, dt, p.dt, r, w.r1, w.nch, lane);
        if (MAIN && z) raw_fetch<CW, F>(sm.raw[to].z, z, p.z, r, w.r1, w.nch, lane);
        raw_fetch_n<32, F>(sm.raw[to].b, B, p.B.row, r, w.r1, p.n, p.B.wide, lane);
        if (MAIN) raw_fetch_n<32, F>(sm.raw[to].c, Cc, p.C.row, r, w.r1, p.n, p.C.wide, lane);
        cp_async_commit();
    };
    auto fetch = [&](int r, int to) {
        if (full && r + R <= w.r1)
            fetch_as(std::true_type(), r, to);
        else
            fetch_as(std::false_type(), r, to);
    };
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        raw_clear_n<32>(sm.raw[i].b, p.n, lane);
        if (MAIN) raw_clear_n<32>(sm.raw[i].c, p.n, lane);
    }
    C total = 0;

    for (int rt = w.r0 - R; rt < w.r1; rt += R) {       // the first time only to fetch: one place in the code that does
        const int at = ((rt - w.r0) / R) & 1;
        const ScanRaw<K> &raw = sm.raw[at];
        cp_async_wait_all();
        __syncwarp();
        if (rt + R < w.r1) fetch(rt + R, at ^ 1);
        if (rt < w.r0) continue;
        raw_stage_n<32>(sm.b, raw.b, lane);
        if (MAIN) raw_stage_n<32>(sm.c, raw.c, lane);
        const int nr = min(R, w.r1 - rt);
        bool finite = true;
        {       // all rows' loads before the stores: the chains of one row are long, those of sixteen run side by side
            C v[PER], u[PER];
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                v[i] = Elem<T>::up(raw.dt[nl + LN * i][dl]) + bias;
                u[i] = Elem<T>::up(raw.x[nl + LN * i][dl]);
            }
            if (p.softplus) {
#pragma unroll
                for (int i = 0; i < PER; ++i) v[i] = softplus_of<T>(v[i]);
            }
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const int t = nl + LN * i;
                sm.dt[t][dl] = v[i];
                sm.u[t][dl] = v[i] * u[i];
                if (!MAIN && t < nr) total += v[i];
            }
            if constexpr (PADDED) {     // an infinite step makes this not finite too
                C probe = 0;
#pragma unroll
                for (int i = 0; i < PER; ++i)
                    if (in && nl + LN * i < nr) probe = fma(v[i] * u[i], (C)0, probe);
                finite = !__any_sync(FULL_MASK, probe != (C)0);
            }
        }
        __syncwarp();
        const uint32_t st = p.rows.starts(rt, R, k, lane);
        if (MAIN && p.kept) {
            const int tiles = (p.rows.rows + R - 1) / R;
            store_states<SN>(static_cast<C *>(p.kept) + (w.line * tiles + rt / R) * dn + own, n, in, h);
        }
        for (int t = 0; t < nr;) {
            if ((st >> t) & 1u) {
                if (rt + t > p.rows.start(k)) ++k;
                if (state) {
                    load_states<SN>(state + p.rows.number(k, w.line) * dn + own, n, in, h);
                } else {
                    zero_states<SN>(h);
                }
            }
            const uint32_t later = st >> (t + 1);
            const int te = later ? min(nr, t + __ffs(later)) : nr;
            for (; (!PADDED || finite) && t + 4 <= te; t += 4) {        // four rows' loads before their stores
                C v[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = scan_row<K, MAIN, false>(sm, t + i, dl, n0, n, A2, h);
                if (MAIN) {
                    scatter_sum<4, CW, 32>(v, lane);
                    if (LN > 1) __syncwarp();       // a row's sum lands where other lanes read its product
#pragma unroll
                    for (int i = 0; i < 4 / LN; ++i) sm.u[t + scatter_first<4, CW, 32>(lane) + i][dl] = v[i];
                }
            }
            for (; t < te; ++t) {
                C v[1] = {scan_row<K, MAIN, PADDED>(sm, t, dl, n0, n, A2, h)};
                if (MAIN) {
                    scatter_sum<1, CW, 32>(v, lane);
                    if (LN > 1) __syncwarp();
                    if (nl == 0) sm.u[t][dl] = v[0];
                }
            }
            if (MAIN && state_out && ((st >> t) & 1u))
                store_states<SN>(state_out + p.rows.number(k, w.line) * dn + own, n, in, h);
        }
        if (MAIN) {
            if (LN > 1) __syncwarp();
            C v[PER];
#pragma unroll
            for (int i = 0; i < PER; ++i) v[i] = sm.u[nl + LN * i][dl] + skip * Elem<T>::up(raw.x[nl + LN * i][dl]);
            if (z) {
#pragma unroll
                for (int i = 0; i < PER; ++i) {
                    const C g = Elem<T>::up(raw.z[nl + LN * i][dl]);
                    v[i] *= g * sigmoid_(g);
                }
            }
            T(*out)[CW] = reinterpret_cast<T(*)[CW]>(&sm.dt[0][0]);
            __syncwarp();       // all lanes are done with the steps
#pragma unroll
            for (int i = 0; i < PER; i += 2) down2(&out[nl + LN * i][dl], &out[nl + LN * (i + 1)][dl], v[i], v[i + 1]);
            __syncwarp();
            if (p.y.wide && w.nch == CW) {
                constexpr int LANES = CW / E, ROWS = 32 / LANES;
                const int row = lane / LANES, e = (lane % LANES) * E;
#pragma unroll
                for (int i = 0; i < R; i += ROWS)
                    if (row + i < nr)
                        *reinterpret_cast<uint4 *>(y + (int64_t)(rt + row + i) * p.y.row + e) =
                            *reinterpret_cast<const uint4 *>(&out[row + i][e]);
            } else if (in) {
#pragma unroll
                for (int i = 0; i < PER; ++i)
                    if (nl + LN * i < nr) y[(int64_t)(rt + nl + LN * i) * p.y.row + dl] = out[nl + LN * i][dl];
            }
        }
        __syncwarp();
    }
    if (!MAIN) {
#pragma unroll
        for (int m = CW; m < 32; m *= 2) total += shfl_xor_(total, m);
    }
    if (!MAIN && in) {
        const int64_t piece = w.line * p.segs + w.seg;
        store_states<SN>(static_cast<C *>(p.ends) + piece * dn + own, n, in, h);
        if (nl == 0) static_cast<C *>(p.sums)[piece * p.d + w.c0 + dl] = total;
    }
}

template <class K, bool MAIN, int BLOCKS, bool PADDED>
cudaError_t scan_start(const ScanArgs &p, const dim3 &grid, int threads, int bytes, cudaStream_t s)
{
    const cudaError_t e =
        cudaFuncSetAttribute(scan_kernel<K, MAIN, BLOCKS, PADDED>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    scan_kernel<K, MAIN, BLOCKS, PADDED><<<grid, threads, bytes, s>>>(p);
    return cudaGetLastError();
}
template <class K> cudaError_t scan_run(const ScanArgs &p, cudaStream_t s)
{
    constexpr int warps = SCAN_WARPS;
    constexpr int bytes = warps * (int)sizeof(ScanFwdSmem<K>);
    static_assert(bytes <= 227 * 1024, "fits an SM");
    const int64_t per = p.d / p.groups, tiles = (per + K::CW - 1) / K::CW;
    const dim3 grid((unsigned)(p.lines * p.segs), (unsigned)(p.groups * ((tiles + warps - 1) / warps)));
    constexpr int full = sizeof(typename K::C) == 4 ? 4 : 1;
    if (p.segs > 1) {
        const cudaError_t e = scan_start<K, false, full, false>(p, grid, warps * 32, bytes, s);
        if (e != cudaSuccess) return e;
    }
    const auto start = [&](auto blocks) {
        return p.n != K::NP ? scan_start<K, true, blocks.value, true>(p, grid, warps * 32, bytes, s)
                            : scan_start<K, true, blocks.value, false>(p, grid, warps * 32, bytes, s);
    };
    if (full > 1 && (int64_t)grid.x * grid.y <= 2 * p.sms) return start(std::integral_constant<int, 1>());
    return start(std::integral_constant<int, full>());
}

// Calls f with the tile of NP states and so many lanes per channel.
template <class T, int NP, class F> cudaError_t with_lanes(int lanes, F f)
{
    if constexpr (NP <= 16) {
        if (lanes == 1) return f(ScanFwdTile<T, NP, 1>());
    }
    if constexpr (NP == 8 || NP == 16 || NP == 32) {
        if (lanes == 2) return f(ScanFwdTile<T, NP, 2>());
    }
    if constexpr (NP >= 16) {
        if (lanes == 4) return f(ScanFwdTile<T, NP, 4>());
    }
    return cudaErrorInvalidValue;
}

}  // namespace
}  // namespace selinv
