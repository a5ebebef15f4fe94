// Reordering of beam-search states, for gfx950: row j of every item becomes a copy
// of row parent[j], for many tensors in one launch.
//
// Pure data movement, bound by HBM: each distinct parent row is read once and each
// moved row written once. One thread owns one 16-byte column of all the rows of an
// item: it reads that column of every row that moves, then writes them. No other
// thread touches the column, so the same kernel moves in place, without a second
// buffer and whatever cycles or repetitions the parents hold.
#include <algorithm>

#include "qg_device.h"
#include "qg_host.h"

namespace {

// 16 bytes as a vector type of the compiler's, which keeps arrays of it in registers
typedef uint32_t u16B __attribute__((ext_vector_type(4)));

struct RArgs {
    qg_beam_state st[QG_BEAM_MAX_STATES];
    uint32_t end[QG_BEAM_MAX_STATES];  // workgroups of the states up to this one
    const int32_t* parent;
    int32_t beams_in, beams_out;
};

template <typename U, int W>
__global__ __launch_bounds__(256) void beam_reorder_kernel(RArgs a) {
    int k = 0;  // the state this workgroup belongs to: the first whose end is beyond it
#pragma unroll
    for (int step = 32; step; step >>= 1)
        if (k + step < QG_BEAM_MAX_STATES && a.end[k + step - 1] <= blockIdx.x) k += step;
    const qg_beam_state& s = a.st[k];
    const uint32_t first = k ? a.end[k - 1] : 0u;
    const int64_t per = s.span / (int64_t)sizeof(U);
    const int64_t c = (int64_t)(blockIdx.x - first) * 256 + threadIdx.x;
    if (c >= s.outer * per) return;
    const int64_t o = c / per, i = c - o * per;
    const int64_t b = blockIdx.y;
    const uint8_t* src = (const uint8_t*)s.src + b * a.beams_in * s.src_row + o * s.src_outer + i * (int64_t)sizeof(U);
    uint8_t* dst = (uint8_t*)s.dst + b * a.beams_out * s.dst_row + o * s.dst_outer + i * (int64_t)sizeof(U);
    const bool inplace = s.src == s.dst;
    const int32_t* par = a.parent + b * a.beams_out;
    U v[W];
    bool mv[W];
#pragma unroll
    for (int j = 0; j < W; ++j) {
        mv[j] = false;
        if (j < a.beams_out) {
            const int p = par[j];
            mv[j] = p >= 0 && p < a.beams_in && !(inplace && p == j);
            if (mv[j]) v[j] = *reinterpret_cast<const U*>(src + p * s.src_row);
        }
    }
#pragma unroll
    for (int j = 0; j < W; ++j)
        if (mv[j]) *reinterpret_cast<U*>(dst + j * s.dst_row) = v[j];
}

// The largest unit of 16, 4 or 1 bytes that a state's pointers, strides and span allow.
int unit_of(const qg_beam_state& s) {
    uintptr_t bits = reinterpret_cast<uintptr_t>(s.src) | reinterpret_cast<uintptr_t>(s.dst) | (uintptr_t)s.src_row |
                     (uintptr_t)s.dst_row | (uintptr_t)s.span;
    if (s.outer > 1) bits |= (uintptr_t)s.src_outer | (uintptr_t)s.dst_outer;
    return (bits & 15) == 0 ? 16 : (bits & 3) == 0 ? 4 : 1;
}
int64_t groups_of(const qg_beam_state& s, int unit) { return qg::ceil_div(s.outer * (s.span / unit), 256); }

// One launch for the states of one unit.
template <typename U>
qg_status launch(const qg_beam_state* states, int count, const int32_t* parent, int64_t batch, int beams_in,
                 int beams_out, hipStream_t stream) {
    RArgs a{};
    int n = 0;
    uint32_t groups = 0;
    for (int k = 0; k < count; ++k)
        if (unit_of(states[k]) == (int)sizeof(U)) {
            a.st[n] = states[k];
            groups += (uint32_t)groups_of(states[k], (int)sizeof(U));
            a.end[n++] = groups;
        }
    if (!n) return QG_OK;
    for (int k = n; k < QG_BEAM_MAX_STATES; ++k) a.end[k] = groups;
    a.parent = parent;
    a.beams_in = beams_in;
    a.beams_out = beams_out;
    const dim3 g(groups, (unsigned)batch);
    if (beams_out <= 4)
        hipLaunchKernelGGL((beam_reorder_kernel<U, 4>), g, dim3(256), 0, stream, a);
    else if (beams_out <= 8)
        hipLaunchKernelGGL((beam_reorder_kernel<U, 8>), g, dim3(256), 0, stream, a);
    else
        hipLaunchKernelGGL((beam_reorder_kernel<U, QG_BEAM_MAX>), g, dim3(256), 0, stream, a);
    return qg::launch_status("qg_beam_reorder");
}

}  // namespace

extern "C" qg_status qg_beam_reorder(const qg_beam_state* states, int count, const int32_t* parent, int64_t batch,
                                     int beams_in, int beams_out, qg_stream_t stream) {
    qg::clear_error();
    if (!states || !parent) return qg::fail(QG_ERR_NULL, "NULL pointer (states, parent)");
    if (count < 1 || count > QG_BEAM_MAX_STATES)
        return qg::fail(QG_ERR_SHAPE, "count=%d not in [1, %d]", count, QG_BEAM_MAX_STATES);
    if (beams_in < 1 || beams_in > QG_BEAM_MAX || beams_out < 1 || beams_out > QG_BEAM_MAX)
        return qg::fail(QG_ERR_SHAPE, "beams_in=%d or beams_out=%d not in [1, %d]", beams_in, beams_out, QG_BEAM_MAX);
    if (batch < 1 || batch > 65535) return qg::fail(QG_ERR_SHAPE, "batch=%lld not in [1, 65535]", (long long)batch);
    if (reinterpret_cast<uintptr_t>(parent) & 3) return qg::fail(QG_ERR_ALIGN, "parent not 4-byte aligned");
    const int64_t most = (int64_t)1 << 40;  // products with 2^21 rows stay below 2^62
    int64_t groups = 0;
    for (int k = 0; k < count; ++k) {
        const qg_beam_state& s = states[k];
        if (!s.src || !s.dst) return qg::fail(QG_ERR_NULL, "state %d: src or dst is NULL", k);
        if (s.outer < 1 || s.span < 1 || s.outer >= most || s.span >= most / s.outer)
            return qg::fail(QG_ERR_SHAPE, "state %d: outer=%lld, span=%lld not in range", k, (long long)s.outer,
                            (long long)s.span);
        if (s.src_row < 0 || s.dst_row < 0 || s.src_outer < 0 || s.dst_outer < 0 || s.src_row > most ||
            s.dst_row > most || s.src_outer > most || s.dst_outer > most)
            return qg::fail(QG_ERR_SHAPE, "state %d: a stride is not in [0, 2^40]", k);
        const int64_t rin = batch * beams_in, rout = batch * beams_out;
        // dst's rows and pieces are apart if the smaller stride clears a span and the
        // larger one everything that the smaller one steps over
        const bool rows_inner = s.outer > 1 && s.dst_row < s.dst_outer;
        const int64_t s1 = rows_inner ? s.dst_row : s.dst_outer, n1 = rows_inner ? rout : s.outer;
        const int64_t s2 = rows_inner ? s.dst_outer : s.dst_row, n2 = rows_inner ? s.outer : rout;
        const int64_t reach = n1 > 1 ? (n1 - 1) * s1 + s.span : s.span;
        if ((n1 > 1 && s1 < s.span) || (n2 > 1 && s2 < reach))
            return qg::fail(QG_ERR_SHAPE, "state %d: dst rows or pieces overlap", k);
        const uintptr_t d0 = reinterpret_cast<uintptr_t>(s.dst), p0 = reinterpret_cast<uintptr_t>(parent);
        const uintptr_t dn = (uintptr_t)((rout - 1) * s.dst_row + (s.outer - 1) * s.dst_outer + s.span);
        if (d0 < p0 + (uintptr_t)rout * 4 && p0 < d0 + dn)
            return qg::fail(QG_ERR_SHAPE, "state %d: dst and parent overlap", k);
        if (s.src == s.dst) {
            if (beams_in != beams_out || s.src_row != s.dst_row || s.src_outer != s.dst_outer)
                return qg::fail(QG_ERR_SHAPE, "state %d: in place needs equal beams and strides", k);
        } else {
            const uintptr_t s0 = reinterpret_cast<uintptr_t>(s.src);
            const uintptr_t sn = (uintptr_t)((rin - 1) * s.src_row + (s.outer - 1) * s.src_outer + s.span);
            if (s0 < d0 + dn && d0 < s0 + sn) return qg::fail(QG_ERR_SHAPE, "state %d: src and dst overlap", k);
        }
        groups += groups_of(s, unit_of(s));
        if (groups >= (int64_t)1 << 24)  // a launch has fewer than 2^32 threads along x
            return qg::fail(QG_ERR_SHAPE, "the states' rows hold over 2^32 units of their alignment");
    }
    qg_status st = qg::check_device();
    if (st) return st;
    hipStream_t s = (hipStream_t)stream;
    st = launch<u16B>(states, count, parent, batch, beams_in, beams_out, s);
    if (!st) st = launch<uint32_t>(states, count, parent, batch, beams_in, beams_out, s);
    if (!st) st = launch<uint8_t>(states, count, parent, batch, beams_in, beams_out, s);
    return st;
}
