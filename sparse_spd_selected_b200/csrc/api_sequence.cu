// C ABI of the sequence operators (selective scan, causal convolution):
// argument validation, workspace sizing, how lines are cut, and dispatch.
// Declarations and the full contract are in include/selinv.h.
#include <stdint.h>

#include "sequence.h"

using namespace selinv;

namespace {

constexpr int64_t MAX_D = 1 << 20, MAX_ROWS = 0x7fffffff - 64, MAX_STRIDE = 0x7fffffff, MAX_SEGS = 160, MAX_GRID_X = 0x7fffffff, MAX_GRID_Y = 65535;

bool aligned(const void *p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
size_t round_up(size_t x) { return (x + 255) / 256 * 256; }
int64_t div_up(int64_t a, int64_t b) { return (a + b - 1) / b; }
selinv_status from_cuda(cudaError_t e) { return e == cudaSuccess ? SELINV_OK : SELINV_ERR_CUDA; }

// bytes of an element and of the arithmetic (states, A, D, dt_bias, parameter gradients)
size_t elem(int64_t dtype) { return dtype == SELINV_F64 ? 8 : dtype == SELINV_F32 ? 4 : 2; }
size_t arith(int64_t dtype) { return dtype == SELINV_F64 ? 8 : 4; }
bool valid(int64_t dtype)
{
    return dtype == SELINV_F64 || dtype == SELINV_F32 || dtype == SELINV_BF16 || dtype == SELINV_F16;
}

// Calls f with a value of the element type.
template <class F> auto with_type(int64_t dtype, F f)
{
    switch (dtype) {
    case SELINV_F64: return f(double());
    case SELINV_F32: return f(float());
    case SELINV_BF16: return f(__nv_bfloat16());
    default: return f(__half());
    }
}

int sm_count()
{
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms < 1) {
        cudaGetLastError();
        return 148;
    }
    return sms;
}

bool view_ok(const selinv_view &v, size_t es) { return v.data && aligned(v.data, es) && v.line >= 0 && v.row >= 0 && v.row <= MAX_STRIDE; }

// Whether packs of 16 bytes along the channels are aligned in every row, line and group (`group` elements apart).
bool wide(const selinv_view &v, size_t es, int64_t group, size_t pack = 16)
{
    return aligned(v.data, pack) && v.line * es % pack == 0 && v.row * es % pack == 0 && group * es % pack == 0;
}
In in_of(const selinv_view &v, size_t es, int64_t group, size_t pack = 16)
{
    return In{v.data, v.line, (int)v.row, wide(v, es, group, pack), wide(v, es, group, es < 4 ? 4 : es)};
}
Out out_of(const selinv_view &v, size_t es, int64_t group)
{
    return Out{const_cast<void *>(v.data), v.line, (int)v.row, wide(v, es, group), wide(v, es, group, es < 4 ? 4 : es)};
}

selinv_status rows_check(int64_t lines, int64_t rows, const int64_t *table, int64_t sequences, int64_t live)
{
    if (lines < 0 || rows < 0) return SELINV_ERR_INVALID_ARG;
    if (table && (lines != 1 || sequences < 0 || live < 0 || live > sequences || live > rows || (live == 0) != (rows == 0) ||
                  !aligned(table, 8)))
        return SELINV_ERR_INVALID_ARG;
    return rows > MAX_ROWS ? SELINV_ERR_UNSUPPORTED : SELINV_OK;
}

// The cache that a step writes, n elements of the given size: its rows are done in no order, so nothing else lies in it.
struct Written {
    uintptr_t lo, hi;
    Written(const void *p, int64_t n, size_t size) : lo(reinterpret_cast<uintptr_t>(p)), hi(lo + n * size) {}
    // Whether n elements at p lie beside it (or p is null).
    bool beside(const void *p, int64_t n, size_t size) const
    {
        const uintptr_t at = reinterpret_cast<uintptr_t>(p);
        return !p || at >= hi || at + n * size <= lo;
    }
};

// ---- selective scan ----------------------------------------------------------

selinv_status scan_check(const selinv_scan_inputs &a)
{
    if (!valid(a.dtype) || (a.flags & ~(int64_t)SELINV_SOFTPLUS)) return SELINV_ERR_INVALID_ARG;
    if (a.d < 1 || a.n < 1 || a.groups < 1 || a.d % a.groups) return SELINV_ERR_INVALID_ARG;
    if (a.n > SCAN_MAX_N || a.d > MAX_D) return SELINV_ERR_UNSUPPORTED;
    const selinv_status st = rows_check(a.lines, a.rows, a.table, a.sequences, a.live);
    if (st != SELINV_OK) return st;
    const size_t es = elem(a.dtype), cs = arith(a.dtype);
    if (!aligned(a.A, cs) || !aligned(a.D, cs) || !aligned(a.dt_bias, cs) || !aligned(a.state, cs) || !a.A)
        return SELINV_ERR_INVALID_ARG;
    if (a.lines == 0 || a.rows == 0) return SELINV_OK;
    if (!view_ok(a.x, es) || !view_ok(a.dt, es) || !view_ok(a.B, es) || !view_ok(a.C, es) || a.B_group < 0 || a.C_group < 0)
        return SELINV_ERR_INVALID_ARG;
    if (a.z.data && !view_ok(a.z, es)) return SELINV_ERR_INVALID_ARG;
    return SELINV_OK;
}

// How a scan is spread over the GPU.
struct Spread {
    int lanes, segs;                        // lanes of a channel (forward), segments of a line
    int64_t seg_rows, blocks, ends_blocks;  // blocks over all groups' channels; of the backward's run over segment ends
};
Spread scan_spread(const selinv_scan_inputs &a, bool backward)
{
    const int n = (int)a.n;
    const int64_t per = a.d / a.groups, sms = sm_count(), lines = a.lines > 0 ? a.lines : 1;
    const auto blocks = [&](int64_t channels) { return lines * a.groups * div_up(div_up(per, channels), SCAN_BLOCK_TILES); };
    Spread s{scan_least_lanes(n), 1, a.rows, 0, 0};
    int64_t cw = backward ? with_type(a.dtype, [&](auto t) { return scan_backward_channels<decltype(t)>(n); }) : 32 / s.lanes;
    // A line that is cut is run twice but for its last segment, first for the states that segments leave behind.  So it
    // is cut only where its blocks come to less than about one per SM (forward; 128 blocks of 4 x 2048 x 4096 x 16 take
    // 306 us whole, 366 in 16 segments) or to less than 0.7 of those resident (backward; with two resident per SM 128
    // blocks take 1297 us whole and 994 in 8 segments, 256 blocks 895 whole and 965 in 4).
    const int64_t resident =
        (backward ? with_type(a.dtype, [&](auto t) { return scan_backward_blocks<decltype(t)>(n); }) : 4) * sms;
    if (blocks(cw) * 10 < (backward ? 7 * resident : 8 * sms)) {
        // more lanes per channel where segments alone do not fill the GPU (1 x 300 x 1024 x 16: 35 us with one, 27 with four)
        if (!backward)
            while (s.lanes < scan_most_lanes(n) && blocks(cw) * (a.rows / 64 > 1 ? a.rows / 64 : 1) < 3 * sms)
                s.lanes *= 2, cw /= 2;
        // As many segments as are resident at once, or where that leaves SMs with fewer than the others, so many that they
        // end together (128 blocks forward: 409 us in 4 segments, 352 in 8); none under 64 rows unless SMs would be idle.
        const int64_t b = blocks(cw);
        int64_t segs = resident / b;
        if (segs * b * 100 < 93 * resident) segs = 7 * sms / b;
        if (segs > a.rows / 64) segs = a.rows / 64;
        if (b * segs < 2 * sms) segs = 2 * sms / b < a.rows / 32 ? 2 * sms / b : a.rows / 32;
        s.segs = (int)(segs < 1 ? 1 : segs < MAX_SEGS ? segs : MAX_SEGS);
    } else if (!backward && s.lanes == 1 && scan_most_lanes(n) > 1 && 2 * blocks(cw) <= 3 * sms) {
        // Whole lines, one or two blocks per SM: twice the warps of half the channels hide more of each other's waits
        // and spread more evenly (x 1024 x 4096 x 16: 4 lines 184 us with one lane, 158 with two; 5 lines 256 and 206;
        // 7 lines 257 either way, 12 lines 367 and 386).
        s.lanes = 2, cw = 16;
    }
    // the backward's run over the segments' ends: lanes until there are three blocks per SM
    if (backward)
        while (s.lanes < scan_most_lanes(n) && blocks(32 / s.lanes) * s.segs < 3 * sms) s.lanes *= 2;
    s.blocks = a.groups * div_up(div_up(per, cw), SCAN_BLOCK_TILES);
    s.ends_blocks = backward ? a.groups * div_up(div_up(per, 32 / s.lanes), SCAN_BLOCK_TILES) : 0;
    s.seg_rows = div_up(div_up(a.rows, s.segs), SCAN_KEEP_ROWS) * SCAN_KEEP_ROWS;
    if (s.seg_rows < SCAN_KEEP_ROWS) s.seg_rows = SCAN_KEEP_ROWS;
    s.segs = (int)div_up(a.rows, s.seg_rows);
    if (s.segs < 1) s.segs = 1;
    return s;
}

// Workspace of a scan: what segments hand on, and the backward's partial sums.
struct ScanSpace {
    size_t ends, sums, bc, a, d, bias, total;
};
ScanSpace scan_space(const selinv_scan_inputs &a, const Spread &s, bool backward)
{
    const size_t cs = arith(a.dtype), pieces = (size_t)a.lines * s.segs;
    ScanSpace w{};
    size_t at = 0;
    const auto take = [&](size_t bytes) {
        const size_t here = at;
        at += round_up(bytes);
        return here;
    };
    if (s.segs > 1) {
        w.ends = take(pieces * a.d * a.n * cs);
        w.sums = take(pieces * a.d * cs);
    }
    if (backward) {
        const size_t parts = s.blocks / a.groups;
        w.bc = take(parts * a.lines * a.rows * a.groups * 2 * scan_padded((int)a.n) * cs);
        w.a = take(pieces * a.d * a.n * cs);
        w.d = take(pieces * a.d * cs);
        w.bias = take(pieces * a.d * cs);
    }
    w.total = at;
    return w;
}

size_t scan_workspace(const selinv_scan_inputs *a, bool backward)
{
    if (!a || !valid(a->dtype) || a->d < 1 || a->d > MAX_D || a->n < 1 || a->n > SCAN_MAX_N || a->groups < 1 ||
        a->d % a->groups || a->lines < 1 || a->rows < 0 || (a->rows == 0 && !a->table))
        return 0;
    return scan_space(*a, scan_spread(*a, backward), backward).total;
}

selinv_status scan_args(const selinv_scan_inputs &a, const Spread &s, ScanArgs &p)
{
    const size_t es = elem(a.dtype);
    const int64_t per = a.groups > 1 ? a.d / a.groups : 0;
    if (a.lines * s.segs > MAX_GRID_X || s.blocks > MAX_GRID_Y || s.ends_blocks > MAX_GRID_Y) return SELINV_ERR_UNSUPPORTED;
    const size_t pack = es == 2 ? 8 : 16;        // B and C: four elements at a time, two in float64
    p.rows = Rows{a.table, (int)a.live, (int)a.rows};
    p.lines = a.lines, p.d = a.d, p.sequences = a.sequences;
    p.n = (int)a.n, p.groups = (int)a.groups;
    p.softplus = a.flags & SELINV_SOFTPLUS;
    p.x = in_of(a.x, es, per), p.dt = in_of(a.dt, es, per), p.z = in_of(a.z, es, per);
    p.B = in_of(a.B, es, a.B_group, pack), p.C = in_of(a.C, es, a.C_group, pack);
    p.B_group = a.B_group, p.C_group = a.C_group;
    p.A = a.A, p.D = a.D, p.dt_bias = a.dt_bias, p.state = a.state;
    p.segs = s.segs, p.seg_rows = (int)s.seg_rows;
    p.ends_lanes = s.lanes;
    p.sms = sm_count();
    return SELINV_OK;
}

// No rows: sequences end as they began.
selinv_status copy_states(void *to, const void *from, size_t bytes, cudaStream_t s)
{
    if (!to || bytes == 0) return SELINV_OK;
    return from_cuda(from ? cudaMemcpyAsync(to, from, bytes, cudaMemcpyDeviceToDevice, s) : cudaMemsetAsync(to, 0, bytes, s));
}
selinv_status zero(void *to, size_t bytes, cudaStream_t s)
{
    return to ? from_cuda(cudaMemsetAsync(to, 0, bytes, s)) : SELINV_OK;
}

// ---- causal convolution --------------------------------------------------------

selinv_status conv_check(const selinv_conv_inputs &a)
{
    if (!valid(a.dtype) || (a.flags & ~(int64_t)SELINV_SILU) || a.d < 1 || a.k < 1) return SELINV_ERR_INVALID_ARG;
    if (a.k < CONV_MIN_K || a.k > CONV_MAX_K || a.d > MAX_D) return SELINV_ERR_UNSUPPORTED;
    const selinv_status st = rows_check(a.lines, a.rows, a.table, a.sequences, a.live);
    if (st != SELINV_OK) return st;
    const size_t es = elem(a.dtype);
    if (!a.weight || !aligned(a.weight, es) || !aligned(a.bias, es) || !aligned(a.state, es)) return SELINV_ERR_INVALID_ARG;
    if (a.lines > 0 && a.rows > 0 && !view_ok(a.x, es)) return SELINV_ERR_INVALID_ARG;
    return SELINV_OK;
}

// Rows per thread: enough threads to keep every SM's loads in flight, but chunks long enough that the K - 1 rows before
// each cost little.
int64_t conv_chunk(const selinv_conv_inputs &a)
{
    const int64_t per = a.dtype == SELINV_F64 ? 2 : 4, vecs = div_up(a.d, per) * (a.lines > 0 ? a.lines : 1);
    const int64_t want = 1024 * (int64_t)sm_count(), least = 16, most = 128;
    int64_t rows = div_up(a.rows, div_up(want, vecs));
    rows = rows < least ? least : rows > most ? most : rows;
    return div_up(rows, 4) * 4;
}
size_t conv_space(const selinv_conv_inputs &a)
{
    const int64_t chunks = div_up(a.rows, conv_chunk(a));
    return round_up((size_t)a.lines * (chunks > 1 ? chunks : 1) * (a.k + 1) * a.d * arith(a.dtype));
}

selinv_status conv_args(const selinv_conv_inputs &a, ConvArgs &p)
{
    const size_t es = elem(a.dtype);
    p.rows = Rows{a.table, (int)a.live, (int)a.rows};
    p.lines = a.lines, p.d = a.d, p.sequences = a.sequences;
    p.k = (int)a.k;
    p.silu = a.flags & SELINV_SILU;
    p.x = in_of(a.x, es, 0);
    p.weight = a.weight, p.bias = a.bias, p.state = a.state;
    p.chunk_rows = (int)conv_chunk(a);
    const int64_t chunks = div_up(a.rows, p.chunk_rows);
    if (div_up(div_up(a.d, es == 8 ? 2 : 4) * a.lines * chunks, 128) > MAX_GRID_X) return SELINV_ERR_UNSUPPORTED;
    p.chunks = (int)(chunks > 1 ? chunks : 1);
    return SELINV_OK;
}

}  // namespace

size_t selinv_selective_scan_kept_size(const selinv_scan_inputs *a)
{
    if (!a || !valid(a->dtype) || a->d < 1 || a->n < 1 || a->lines < 0 || a->rows < 0) return 0;
    return (size_t)a->lines * div_up(a->rows, SCAN_KEEP_ROWS) * a->d * a->n * arith(a->dtype);
}

size_t selinv_selective_scan_workspace_size(const selinv_scan_inputs *a) { return scan_workspace(a, false); }
size_t selinv_selective_scan_backward_workspace_size(const selinv_scan_inputs *a) { return scan_workspace(a, true); }

selinv_status selinv_selective_scan(const selinv_scan_inputs *a, const selinv_view *y, void *state_out, void *kept,
                                    void *workspace, size_t workspace_bytes, void *stream)
{
    if (!a || !y) return SELINV_ERR_INVALID_ARG;
    selinv_status st = scan_check(*a);
    if (st != SELINV_OK) return st;
    const size_t es = elem(a->dtype), cs = arith(a->dtype);
    if (!aligned(state_out, cs) || !aligned(kept, cs) || !aligned(workspace, 16)) return SELINV_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (a->lines == 0 || (a->rows == 0 && !a->table))
        return copy_states(state_out, a->state, (size_t)a->lines * a->d * a->n * cs, s);
    if (a->rows > 0 && !view_ok(*y, es)) return SELINV_ERR_INVALID_ARG;
    const Spread spread = scan_spread(*a, false);
    const ScanSpace w = scan_space(*a, spread, false);
    if (w.total > 0 && (!workspace || workspace_bytes < w.total)) return SELINV_ERR_WORKSPACE;
    ScanArgs p{};
    st = scan_args(*a, spread, p);
    if (st != SELINV_OK) return st;
    p.y = out_of(*y, es, a->groups > 1 ? a->d / a->groups : 0);
    p.state_out = state_out, p.kept = kept;
    p.ends = static_cast<char *>(workspace) + w.ends, p.sums = static_cast<char *>(workspace) + w.sums;
    return from_cuda(with_type(a->dtype, [&](auto t) { return scan_launch<decltype(t)>(p, spread.lanes, s); }));
}

selinv_status selinv_selective_scan_backward(const selinv_scan_inputs *a, const selinv_scan_grads *g, void *workspace,
                                             size_t workspace_bytes, void *stream)
{
    if (!a || !g) return SELINV_ERR_INVALID_ARG;
    selinv_status st = scan_check(*a);
    if (st != SELINV_OK) return st;
    const size_t es = elem(a->dtype), cs = arith(a->dtype);
    if (!g->Ab || !aligned(g->Ab, cs) || !aligned(g->Db, cs) || !aligned(g->dt_biasb, cs) || !aligned(g->stateb_out, cs) ||
        !aligned(g->stateb, cs) || !aligned(g->kept, cs) || !aligned(workspace, 16))
        return SELINV_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (a->lines == 0 || (a->rows == 0 && !a->table)) {
        st = copy_states(g->stateb_out, g->stateb, (size_t)a->lines * a->d * a->n * cs, s);
        if (st == SELINV_OK) st = zero(g->Ab, (size_t)a->d * a->n * cs, s);
        if (st == SELINV_OK) st = zero(g->Db, (size_t)a->d * cs, s);
        return st == SELINV_OK ? zero(g->dt_biasb, (size_t)a->d * cs, s) : st;
    }
    if (a->rows > 0) {
        if (!g->kept || !view_ok(g->yb, es) || !view_ok(g->xb, es) || !view_ok(g->dtb, es) || !view_ok(g->Bb, es) ||
            !view_ok(g->Cb, es) || (a->z.data && !view_ok(g->zb, es)) || g->Bb_group < 0 || g->Cb_group < 0)
            return SELINV_ERR_INVALID_ARG;
    }
    const Spread spread = scan_spread(*a, true);
    const ScanSpace w = scan_space(*a, spread, true);
    if (!workspace || workspace_bytes < w.total) return SELINV_ERR_WORKSPACE;
    ScanArgs p{};
    st = scan_args(*a, spread, p);
    if (st != SELINV_OK) return st;
    char *ws = static_cast<char *>(workspace);
    p.ends = ws + w.ends, p.sums = ws + w.sums;
    const int64_t per = a->groups > 1 ? a->d / a->groups : 0;
    ScanGrads o{};
    o.kept = g->kept;
    o.yb = in_of(g->yb, es, per);
    o.stateb = g->stateb;
    o.xb = out_of(g->xb, es, per), o.dtb = out_of(g->dtb, es, per);
    o.zb = a->z.data ? out_of(g->zb, es, per) : Out{};
    o.Bb = out_of(g->Bb, es, 0), o.Cb = out_of(g->Cb, es, 0);
    o.Bb_group = g->Bb_group, o.Cb_group = g->Cb_group;
    o.Ab = g->Ab, o.Db = g->Db, o.dt_biasb = g->dt_biasb, o.stateb_out = g->stateb_out;
    o.part_bc = ws + w.bc, o.part_a = ws + w.a, o.part_d = ws + w.d, o.part_bias = ws + w.bias;
    const int64_t sums = div_up(a->lines * a->rows * a->groups * 2 * scan_padded((int)a->n), 256) +
                         div_up(a->d * (a->n + 2), 32);
    if (sums > MAX_GRID_X) return SELINV_ERR_UNSUPPORTED;
    return from_cuda(with_type(a->dtype, [&](auto t) { return scan_backward_launch<decltype(t)>(p, o, s); }));
}

selinv_status selinv_selective_scan_step(const selinv_scan_step *a, void *stream)
{
    if (!a || !valid(a->dtype) || (a->flags & ~(int64_t)SELINV_SOFTPLUS) || a->batch < 0 || a->slots < 0 || a->d < 1 ||
        a->n < 1 || a->groups < 1 || a->d % a->groups)
        return SELINV_ERR_INVALID_ARG;
    if (a->n > SCAN_MAX_N || a->d > MAX_D) return SELINV_ERR_UNSUPPORTED;
    if (a->batch == 0) return SELINV_OK;
    if (!a->index && a->slots < a->batch) return SELINV_ERR_INVALID_ARG;
    const size_t es = elem(a->dtype), cs = arith(a->dtype);
    const void *const elems[] = {a->x, a->dt, a->B, a->C, a->y};
    for (const void *p : elems)
        if (!p || !aligned(p, es)) return SELINV_ERR_INVALID_ARG;
    if (!aligned(a->z, es) || !a->A || !aligned(a->A, cs) || !aligned(a->D, cs) || !aligned(a->dt_bias, cs) || !a->cache ||
        !a->cache_out || !aligned(a->cache, cs) || !aligned(a->cache_out, cs) || !aligned(a->index, 4) || !aligned(a->info, 4))
        return SELINV_ERR_INVALID_ARG;
    if (a->x_row < 0 || a->dt_row < 0 || a->z_row < 0 || a->B_row < 0 || a->C_row < 0 || a->B_group < 0 || a->C_group < 0 ||
        a->y_row < 0)
        return SELINV_ERR_INVALID_ARG;
    const int64_t last = a->batch - 1, states = a->slots * a->d * a->n;
    const Written w(a->cache_out, states, cs);
    const auto row = [&](const void *v, int64_t stride) { return w.beside(v, last * stride + a->d, es); };
    const auto groups = [&](const void *v, int64_t stride, int64_t group) {
        return w.beside(v, last * stride + (a->groups - 1) * group + a->n, es);
    };
    if (!row(a->x, a->x_row) || !row(a->dt, a->dt_row) || !row(a->z, a->z_row) || !row(a->y, a->y_row) ||
        !groups(a->B, a->B_row, a->B_group) || !groups(a->C, a->C_row, a->C_group) || !w.beside(a->A, a->d * a->n, cs) ||
        !w.beside(a->D, a->d, cs) || !w.beside(a->dt_bias, a->d, cs) || !w.beside(a->index, a->batch, 4) ||
        !w.beside(a->info, a->batch, 4) || (a->cache != a->cache_out && !w.beside(a->cache, states, cs)))
        return SELINV_ERR_INVALID_ARG;
    if (a->batch * div_up(a->d, 128) > MAX_GRID_X) return SELINV_ERR_UNSUPPORTED;
    ScanStepArgs p{};
    p.batch = a->batch, p.d = a->d, p.slots = a->slots, p.n = (int)a->n, p.groups = (int)a->groups;
    p.softplus = a->flags & SELINV_SOFTPLUS;
    p.x = a->x, p.dt = a->dt, p.z = a->z, p.B = a->B, p.C = a->C;
    p.x_row = a->x_row, p.dt_row = a->dt_row, p.z_row = a->z_row, p.B_row = a->B_row, p.C_row = a->C_row;
    p.B_group = a->B_group, p.C_group = a->C_group, p.y_row = a->y_row;
    p.A = a->A, p.D = a->D, p.dt_bias = a->dt_bias, p.cache = a->cache, p.cache_out = a->cache_out, p.y = a->y;
    p.index = a->index, p.info = a->info;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return from_cuda(with_type(a->dtype, [&](auto t) { return scan_step_launch<decltype(t)>(p, s); }));
}

size_t selinv_causal_conv_backward_workspace_size(const selinv_conv_inputs *a)
{
    if (!a || !valid(a->dtype) || a->d < 1 || a->d > MAX_D || a->k < CONV_MIN_K || a->k > CONV_MAX_K || a->lines < 1 ||
        a->rows < 0)
        return 0;
    return conv_space(*a);
}

selinv_status selinv_causal_conv(const selinv_conv_inputs *a, const selinv_view *y, void *state_out, void *stream)
{
    if (!a || !y) return SELINV_ERR_INVALID_ARG;
    selinv_status st = conv_check(*a);
    if (st != SELINV_OK) return st;
    const size_t es = elem(a->dtype);
    if (!aligned(state_out, es)) return SELINV_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (a->lines == 0 || (a->rows == 0 && !a->table))
        return copy_states(state_out, a->state, (size_t)a->lines * a->d * (a->k - 1) * es, s);
    if (a->rows > 0 && !view_ok(*y, es)) return SELINV_ERR_INVALID_ARG;
    ConvArgs p{};
    st = conv_args(*a, p);
    if (st != SELINV_OK) return st;
    p.y = out_of(*y, es, 0);
    p.state_out = state_out;
    return from_cuda(with_type(a->dtype, [&](auto t) { return conv_launch<decltype(t)>(p, s); }));
}

selinv_status selinv_causal_conv_backward(const selinv_conv_inputs *a, const selinv_conv_grads *g, void *workspace,
                                          size_t workspace_bytes, void *stream)
{
    if (!a || !g) return SELINV_ERR_INVALID_ARG;
    selinv_status st = conv_check(*a);
    if (st != SELINV_OK) return st;
    const size_t es = elem(a->dtype), cs = arith(a->dtype);
    if (!g->weightb || !aligned(g->weightb, cs) || !aligned(g->biasb, cs) || !aligned(g->stateb, es) ||
        !aligned(g->stateb_out, es) || !aligned(workspace, 16))
        return SELINV_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (a->lines == 0 || (a->rows == 0 && !a->table)) {
        st = copy_states(g->stateb_out, g->stateb, (size_t)a->lines * a->d * (a->k - 1) * es, s);
        if (st == SELINV_OK) st = zero(g->weightb, (size_t)a->d * a->k * cs, s);
        return st == SELINV_OK ? zero(g->biasb, (size_t)a->d * cs, s) : st;
    }
    if (a->rows > 0 && (!view_ok(g->yb, es) || !view_ok(g->xb, es))) return SELINV_ERR_INVALID_ARG;
    if (!workspace || workspace_bytes < conv_space(*a)) return SELINV_ERR_WORKSPACE;
    ConvArgs p{};
    st = conv_args(*a, p);
    if (st != SELINV_OK) return st;
    p.yb = in_of(g->yb, es, 0);
    p.xb = out_of(g->xb, es, 0);
    p.stateb = g->stateb, p.stateb_out = g->stateb_out, p.weightb = g->weightb, p.biasb = g->biasb, p.part = workspace;
    return from_cuda(with_type(a->dtype, [&](auto t) { return conv_backward_launch<decltype(t)>(p, s); }));
}

selinv_status selinv_causal_conv_step(const selinv_conv_step *a, void *stream)
{
    if (!a || !valid(a->dtype) || (a->flags & ~(int64_t)SELINV_SILU) || a->batch < 0 || a->slots < 0 || a->d < 1 || a->k < 1)
        return SELINV_ERR_INVALID_ARG;
    if (a->k < CONV_MIN_K || a->k > CONV_MAX_K || a->d > MAX_D) return SELINV_ERR_UNSUPPORTED;
    if (a->batch == 0) return SELINV_OK;
    if (!a->index && a->slots < a->batch) return SELINV_ERR_INVALID_ARG;
    const size_t es = elem(a->dtype);
    const void *const elems[] = {a->x, a->weight, a->cache, a->cache_out, a->y};
    for (const void *p : elems)
        if (!p || !aligned(p, es)) return SELINV_ERR_INVALID_ARG;
    if (!aligned(a->bias, es) || !aligned(a->index, 4) || !aligned(a->info, 4) || a->x_row < 0 || a->y_row < 0)
        return SELINV_ERR_INVALID_ARG;
    const int64_t last = a->batch - 1, states = a->slots * (a->k - 1) * a->d;
    const Written w(a->cache_out, states, es);
    if (!w.beside(a->x, last * a->x_row + a->d, es) || !w.beside(a->y, last * a->y_row + a->d, es) ||
        !w.beside(a->weight, a->d * a->k, es) || !w.beside(a->bias, a->d, es) || !w.beside(a->index, a->batch, 4) ||
        !w.beside(a->info, a->batch, 4) || (a->cache != a->cache_out && !w.beside(a->cache, states, es)))
        return SELINV_ERR_INVALID_ARG;
    if (a->batch * div_up(a->d, 128) > MAX_GRID_X) return SELINV_ERR_UNSUPPORTED;
    ConvStepArgs p{};
    p.batch = a->batch, p.d = a->d, p.slots = a->slots, p.k = (int)a->k;
    p.silu = a->flags & SELINV_SILU;
    p.x = a->x, p.weight = a->weight, p.bias = a->bias, p.cache = a->cache;
    p.x_row = a->x_row, p.y_row = a->y_row, p.cache_out = a->cache_out, p.y = a->y;
    p.index = a->index, p.info = a->info;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return from_cuda(with_type(a->dtype, [&](auto t) { return conv_step_launch<decltype(t)>(p, s); }));
}
