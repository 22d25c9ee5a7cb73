// Shared pieces of the sequence operators (selective scan, causal
// convolution): element types, pair arithmetic, exponentials, the row ranges
// of lines and ragged sequences, and lane reductions.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/selinv.h"
#include <cstddef>
#include <cstring>
#include <type_traits>

#include "common.cuh"
#include "pieces.h"

namespace selinv {

// ---- element types: storage T, arithmetic C (32 bits for the 16-bit types) --

template <class T> struct Elem;
template <> struct Elem<float> {
    using C = float;
    SELINV_DEVINL static float up(float v) { return v; }
    SELINV_DEVINL static float down(float v) { return v; }
};
template <> struct Elem<double> {
    using C = double;
    SELINV_DEVINL static double up(double v) { return v; }
    SELINV_DEVINL static double down(double v) { return v; }
};
template <> struct Elem<__nv_bfloat16> {
    using C = float;
    // two elements of a word, and back: one instruction
    SELINV_DEVINL static float low(uint32_t w) { return __uint_as_float(w << 16); }
    SELINV_DEVINL static float high(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
    SELINV_DEVINL static uint32_t pair(float a, float b)
    {
        const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
        uint32_t w;
        memcpy(&w, &v, 4);
        return w;
    }
    SELINV_DEVINL static float up(__nv_bfloat16 v) { return __bfloat162float(v); }
    SELINV_DEVINL static __nv_bfloat16 down(float v) { return __float2bfloat16_rn(v); }
};
template <> struct Elem<__half> {
    using C = float;
    SELINV_DEVINL static float low(uint32_t w)
    {
        __half2 v;
        memcpy(&v, &w, 4);
        return __low2float(v);
    }
    SELINV_DEVINL static float high(uint32_t w)
    {
        __half2 v;
        memcpy(&v, &w, 4);
        return __high2float(v);
    }
    SELINV_DEVINL static uint32_t pair(float a, float b)
    {
        const __half2 v = __floats2half2_rn(a, b);
        uint32_t w;
        memcpy(&w, &v, 4);
        return w;
    }
    SELINV_DEVINL static float up(__half v) { return __half2float(v); }
    SELINV_DEVINL static __half down(float v) { return __float2half_rn(v); }
};

// Rounds two values to two places: the 16-bit types in one instruction (one value alone takes the special function unit).
template <class T> SELINV_DEVINL void down2(T *p, T *q, typename Elem<T>::C x, typename Elem<T>::C y)
{
    if constexpr (sizeof(T) == 2) {
        const uint32_t w = Elem<T>::pair(x, y);
        *reinterpret_cast<unsigned short *>(p) = (unsigned short)w;
        *reinterpret_cast<unsigned short *>(q) = (unsigned short)(w >> 16);
    } else {
        *p = Elem<T>::down(x);
        *q = Elem<T>::down(y);
    }
}

// E consecutive elements as they lie in memory, held in 32-bit words.
template <class T, int E> struct Pack {
    static_assert(E * sizeof(T) % 4 == 0 && E * sizeof(T) <= 16, "4, 8 or 16 bytes");
    static constexpr int W = E * (int)sizeof(T) / 4;
    uint32_t w[W];

    SELINV_DEVINL void clear()
    {
#pragma unroll
        for (int i = 0; i < W; ++i) w[i] = 0u;
    }
    SELINV_DEVINL typename Elem<T>::C get(int e) const
    {
        if constexpr (sizeof(T) == 2) {
            return e & 1 ? Elem<T>::high(w[e >> 1]) : Elem<T>::low(w[e >> 1]);
        } else if constexpr (sizeof(T) == 4) {
            return __uint_as_float(w[e]);
        } else {
            return __hiloint2double((int)w[2 * e + 1], (int)w[2 * e]);
        }
    }
    SELINV_DEVINL void set(const typename Elem<T>::C *v)
    {
#pragma unroll
        for (int e = 0; e < E; ++e) {
            if constexpr (sizeof(T) == 2) {
                if (e % 2 == 0) w[e / 2] = Elem<T>::pair(v[e], v[e + 1]);
            } else if constexpr (sizeof(T) == 4) {
                w[e] = __float_as_uint(v[e]);
            } else {
                w[2 * e] = (uint32_t)__double2loint(v[e]);
                w[2 * e + 1] = (uint32_t)__double2hiint(v[e]);
            }
        }
    }
    // The first `n` of the elements at p; `wide`: p is aligned to the whole pack.
    SELINV_DEVINL void load(const T *p, int n, bool wide)
    {
        if (wide && n >= E) {
            if constexpr (W == 4) {
                const uint4 v = *reinterpret_cast<const uint4 *>(p);
                w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
            } else if constexpr (W == 2) {
                const uint2 v = *reinterpret_cast<const uint2 *>(p);
                w[0] = v.x, w[1] = v.y;
            } else {
                w[0] = *reinterpret_cast<const uint32_t *>(p);
            }
            return;
        }
        clear();
#pragma unroll
        for (int e = 0; e < E; ++e)
            if (e < n) {
                if constexpr (sizeof(T) == 2) {
                    const uint32_t h = reinterpret_cast<const unsigned short *>(p)[e];
                    w[e >> 1] |= (e & 1) ? h << 16 : h;
                } else if constexpr (sizeof(T) == 4) {
                    w[e] = reinterpret_cast<const uint32_t *>(p)[e];
                } else {
                    w[2 * e] = reinterpret_cast<const uint32_t *>(p)[2 * e];
                    w[2 * e + 1] = reinterpret_cast<const uint32_t *>(p)[2 * e + 1];
                }
            }
    }
    SELINV_DEVINL void store(T *p, int n, bool wide) const
    {
        if (wide && n >= E) {
            if constexpr (W == 4)
                *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
            else if constexpr (W == 2)
                *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
            else
                *reinterpret_cast<uint32_t *>(p) = w[0];
            return;
        }
#pragma unroll
        for (int e = 0; e < E; ++e)
            if (e < n) {
                if constexpr (sizeof(T) == 2)
                    reinterpret_cast<unsigned short *>(p)[e] = (unsigned short)(w[e >> 1] >> (16 * (e & 1)));
                else if constexpr (sizeof(T) == 4)
                    reinterpret_cast<uint32_t *>(p)[e] = w[e];
                else {
                    reinterpret_cast<uint32_t *>(p)[2 * e] = w[2 * e];
                    reinterpret_cast<uint32_t *>(p)[2 * e + 1] = w[2 * e + 1];
                }
            }
    }
};

// ---- pairs: two neighbouring channels in one instruction (FFMA2) -----------

template <class C> struct Two;
template <> struct Two<float> {
    using V = float2;
};
template <> struct Two<double> {
    using V = double2;
};

SELINV_DEVINL unsigned long long bits2(float2 v)
{
    unsigned long long r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(v.x), "f"(v.y));
    return r;
}
SELINV_DEVINL float2 from_bits2(unsigned long long r)
{
    float2 v;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(v.x), "=f"(v.y) : "l"(r));
    return v;
}
SELINV_DEVINL float2 fma2(float2 a, float2 b, float2 c)
{
    unsigned long long r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(bits2(a)), "l"(bits2(b)), "l"(bits2(c)));
    return from_bits2(r);
}
SELINV_DEVINL float2 mul2(float2 a, float2 b)
{
    unsigned long long r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits2(a)), "l"(bits2(b)));
    return from_bits2(r);
}
SELINV_DEVINL float2 add2(float2 a, float2 b)
{
    unsigned long long r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits2(a)), "l"(bits2(b)));
    return from_bits2(r);
}
SELINV_DEVINL double2 fma2(double2 a, double2 b, double2 c)
{
    return make_double2(fma(a.x, b.x, c.x), fma(a.y, b.y, c.y));
}
SELINV_DEVINL double2 mul2(double2 a, double2 b) { return make_double2(a.x * b.x, a.y * b.y); }
SELINV_DEVINL double2 add2(double2 a, double2 b) { return make_double2(a.x + b.x, a.y + b.y); }
SELINV_DEVINL float2 make2(float x, float y) { return make_float2(x, y); }
SELINV_DEVINL double2 make2(double x, double y) { return make_double2(x, y); }

// ---- exponentials ----------------------------------------------------------

template <class C> __host__ __device__ constexpr C log2e() { return (C)1.4426950408889634073599246810018921; }
template <class C> __host__ __device__ constexpr C ln2() { return (C)0.69314718055994530941723212145817657; }

// 2^x.  Results below the normal range become zero in float: a decay that small leaves nothing of a state.
SELINV_DEVINL float exp2_(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
SELINV_DEVINL double exp2_(double x) { return exp2(x); }
SELINV_DEVINL float rcp_(float x)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
SELINV_DEVINL double rcp_(double x) { return 1.0 / x; }

SELINV_DEVINL float2 exp2_2(float2 e) { return make_float2(exp2_(e.x), exp2_(e.y)); }
SELINV_DEVINL double2 exp2_2(double2 e) { return make_double2(exp2(e.x), exp2(e.y)); }
// The decays 2^(dt A2) of a pair.  The special function's results are low by 0.6e-8 (arguments over -0.001) to 2.5e-8 on
// average; a state that lives for many rows collects that, so the argument is raised by half of it, in the product's
// own instruction (the error of A's cotangent over 517 rows in float falls from 1.0e-6 to 5.2e-7).
SELINV_DEVINL float2 decay2(float2 dt, float2 A2) { return exp2_2(fma2(dt, A2, make_float2(1.8e-8f, 1.8e-8f))); }
SELINV_DEVINL double2 decay2(double2 dt, double2 A2) { return exp2_2(mul2(dt, A2)); }

// 1 / (1 + e^-x): in float to 7 units in the last place and, where e^-x counts, the 1.3 |x| of its rounded argument.
SELINV_DEVINL float sigmoid_(float x) { return rcp_(1.0f + exp2_(-log2e<float>() * x)); }
SELINV_DEVINL double sigmoid_(double x) { return 1.0 / (1.0 + exp(-x)); }
SELINV_DEVINL float2 sigmoid2(float2 x)
{
    const float2 t = mul2(x, make_float2(-log2e<float>(), -log2e<float>()));
    const float2 v = add2(make_float2(exp2_(t.x), exp2_(t.y)), make_float2(1.0f, 1.0f));
    return make_float2(rcp_(v.x), rcp_(v.y));
}
SELINV_DEVINL double2 sigmoid2(double2 x) { return make_double2(sigmoid_(x.x), sigmoid_(x.y)); }

// d/dx of x sigmoid(x), given p = sigmoid(x).
template <class C> SELINV_DEVINL C silu_slope(C x, C p) { return p * ((C)1 + x * ((C)1 - p)); }

SELINV_DEVINL float2 silu_slope2(float2 x, float2 p)
{
    const float2 one = make_float2(1.0f, 1.0f);
    return mul2(p, fma2(x, fma2(p, make_float2(-1.0f, -1.0f), one), one));
}
SELINV_DEVINL double2 silu_slope2(double2 x, double2 p) { return make_double2(silu_slope(x.x, p.x), silu_slope(x.y, p.y)); }

// log(1 + e^x) = max(x, 0) + log1p(e), e = e^-|x| in (0, 1].  In float log1p(e) = e + e^2 r(e), r of degree 7, minimax
// for the relative error by Remez's exchange (3.3e-8; 6.0e-8 with float coefficients): log(1 + e) itself would lose e's
// low bits for far negative x, and would use the special function unit, which bounds the scan, a second time.  There the
// result is e, whose argument, up to 125, must not be rounded: with EXACT what the product and log2 e lose is put back into
// e, and the result is good to some 10 units in its last place over the whole range (from |x| = 256 on e is nothing).
// Without, 1.3 |x| units are added to them, nothing to steps that come from 16-bit inputs and lead to 16-bit outputs
// (EXACT for those too: 1288 us for 1275, 4 x 2048 x 4096 x 16 forward and backward).
SELINV_DEVINL float max_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
template <bool EXACT> SELINV_DEVINL float softplus_(float x)
{
    float e;
    if (EXACT) {
        const float a = fminf(fabsf(x), 256.0f), t = -log2e<float>() * a;
        const float lost = fmaf(-1.9259630e-8f, a, fmaf(-log2e<float>(), a, -t));   // log2 e beyond a float; the product's rounding
        e = exp2_(t);
        e = fmaf(e * lost, ln2<float>(), e);
    } else {
        e = exp2_(-log2e<float>() * fabsf(x));
    }
    float r = 0.005364798475056887f;
    r = fmaf(r, e, -0.030065692961215973f);
    r = fmaf(r, e, 0.07920438051223755f);
    r = fmaf(r, e, -0.1375378966331482f);
    r = fmaf(r, e, 0.19153648614883423f);
    r = fmaf(r, e, -0.24857161939144135f);
    r = fmaf(r, e, 0.333213210105896f);
    r = fmaf(r, e, -0.49999648332595825f);
    return fmaf(e * e, r, e) + max_nan(x, 0.0f);
}
template <bool EXACT> SELINV_DEVINL double softplus_(double x)
{
    return x == x ? fmax(x, 0.0) + log1p(exp(-fabs(x))) : x;
}
// A step, from inputs of type T.
template <class T> SELINV_DEVINL typename Elem<T>::C softplus_of(typename Elem<T>::C x) { return softplus_<(sizeof(T) > 2)>(x); }

// ---- reductions over lanes -------------------------------------------------

template <class C> SELINV_DEVINL C shfl_xor_(C v, int m) { return __shfl_xor_sync(FULL_MASK, v, m); }

// Sums of V values over the lanes that differ in the bits [LO, HI) of the lane number (powers of two); the values
// are dealt out over those lanes as they are summed, so that a lane ends with max(1, V * LO / HI) of them, in v[0..]:
// those from scatter_first() on.  With more lanes than values, lanes that differ in the lowest bits hold the same.
template <int V, int LO, int HI, class C> SELINV_DEVINL void scatter_sum(C *v, int lane)
{
    if constexpr (HI > LO) {
        constexpr int B = HI / 2;
        if constexpr (V > 1) {
            const bool up = lane & B;
#pragma unroll
            for (int i = 0; i < V / 2; ++i) {
                const C send = up ? v[i] : v[i + V / 2], keep = up ? v[i + V / 2] : v[i];
                v[i] = keep + shfl_xor_(send, B);
            }
            scatter_sum<V / 2, LO, B>(v, lane);
        } else {
            v[0] += shfl_xor_(v[0], B);
            scatter_sum<1, LO, B>(v, lane);
        }
    }
}
template <int V, int LO, int HI> SELINV_DEVINL int scatter_first(int lane)
{
    if constexpr (HI > LO && V > 1)
        return ((lane & (HI / 2)) ? V / 2 : 0) + scatter_first<V / 2, LO, HI / 2>(lane);
    else
        return 0;
}
// Whether this lane is the one of its equals that writes.
template <int V, int LO, int HI> SELINV_DEVINL bool scatter_writes(int lane)
{
    if constexpr (HI > LO && V > 1)
        return scatter_writes<V / 2, LO, HI / 2>(lane);
    else if constexpr (HI > LO)
        return (lane & (HI - LO)) == 0;
    else
        return true;
}

// ---- rows ------------------------------------------------------------------
//
// A call covers `lines` lines of `rows` rows.  Without a table every line is
// one sequence.  With one there is a single line, cut into sequences: the
// table (device memory, int64) holds the first rows of the `live` sequences
// that have any, ascending, then `rows`, then those sequences' numbers.

struct Rows {
    const int64_t *table;
    int live, rows;
    // The live sequence that row r lies in (r < rows).
    SELINV_DEVINL int find(int r) const
    {
        if (!table) return 0;
        int lo = 0, hi = live;
        while (hi - lo > 1) {
            const int m = lo + (hi - lo) / 2;
            if (table[m] <= r)
                lo = m;
            else
                hi = m;
        }
        return lo;
    }
    SELINV_DEVINL int start(int k) const { return table ? (int)table[k] : 0; }
    SELINV_DEVINL int end(int k) const { return table ? (int)table[k + 1] : rows; }
    SELINV_DEVINL int64_t number(int k, int64_t line) const { return table ? table[live + 1 + k] : line; }
    // The sequences without rows, e of them.
    SELINV_DEVINL int64_t empty(int64_t e) const { return table[2 * (int64_t)live + 1 + e]; }
    // Which of the rows r0 .. r0 + n (n <= 30) begin a sequence, given that row r0 lies in the live sequence k; `rows`
    // itself counts as one.  Every lane of the warp calls it.
    SELINV_DEVINL uint32_t starts(int r0, int n, int k, int lane) const
    {
        if (!table) return (r0 == 0 ? 1u : 0u) | (rows - r0 <= n ? 1u << (rows - r0) : 0u);
        uint32_t bit = 0;
        if (lane <= live - k) {
            const int at = (int)table[k + lane] - r0;
            if (at >= 0 && at <= n) bit = 1u << at;
        }
        return __reduce_or_sync(FULL_MASK, bit);
    }
};

// An array [lines, rows, channels]: strides in elements, channels contiguous.  `wide`: base, strides and the first
// channel of every group lie on 16 bytes, so that packs may be moved whole; `words`: on 4 (8 in float64).
template <class P> struct Strided {
    P p;
    int64_t line;
    int row;
    bool wide, words;
};
using In = Strided<const void *>;
using Out = Strided<void *>;

struct ScanArgs {
    Rows rows;
    int64_t lines, d, sequences;
    int n, groups;
    bool softplus;
    In x, dt, z, B, C;          // z.p may be null
    int64_t B_group, C_group;
    const void *A, *D, *dt_bias, *state;     // D, dt_bias, state may be null
    Out y;
    void *state_out, *kept;     // may be null
    // lines cut into segments of seg_rows rows: the state each leaves behind from zero, and the sum of its steps
    int segs, seg_rows;
    int sms;                    // multiprocessors of the device
    int ends_lanes;             // lanes per channel of the backward's run over the segments' ends
    void *ends, *sums;
};

struct ScanGrads {
    const void *kept;
    In yb;
    const void *stateb;         // cotangent of the final states, or null
    Out xb, dtb, zb, Bb, Cb;    // zb.p may be null
    int64_t Bb_group, Cb_group;
    void *Ab, *Db, *dt_biasb, *stateb_out;   // the last three may be null
    // partial sums: of B and C over the channels of a block, of the parameters over a segment
    void *part_bc, *part_a, *part_d, *part_bias;
};

struct ScanStepArgs {
    int64_t batch, d, slots;
    int n, groups;
    bool softplus;
    const void *x, *dt, *z, *B, *C;
    int64_t x_row, dt_row, z_row, B_row, C_row, B_group, C_group, y_row;
    const void *A, *D, *dt_bias;
    const void *cache;
    void *cache_out, *y;
    const int32_t *index;
    int32_t *info;
};

struct ConvArgs {
    Rows rows;
    int64_t lines, d, sequences;
    int k;
    bool silu;
    In x;
    const void *weight, *bias, *state;
    Out y;
    void *state_out;
    // backward
    In yb;
    const void *stateb;
    Out xb;
    void *weightb, *biasb, *stateb_out;
    void *part;
    int chunk_rows, chunks;
};

struct ConvStepArgs {
    int64_t batch, d, slots;
    int k;
    bool silu;
    const void *x, *weight, *bias, *cache;
    int64_t x_row, y_row;
    void *cache_out, *y;
    const int32_t *index;
    int32_t *info;
};

// Status of a row of a step (info): done, its slot lies outside the cache, or an earlier row names the same slot.
constexpr int32_t STEP_OK = -1, STEP_RANGE = 0, STEP_TWICE = 1;

}  // namespace selinv
