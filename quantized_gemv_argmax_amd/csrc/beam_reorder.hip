// Reordering of beam-search states, for gfx950: row j of every item becomes a copy
// of row parent[j], for many tensors in one launch.
//
// Pure data movement, bound by HBM: each distinct parent row is read once and each
// moved row written once. One thread owns one 16-byte column of all the rows of an
// item: it reads that column of every row that moves, then writes them. No other
// thread touches the column, so the same kernel moves in place, without a second
// buffer and whatever cycles or repetitions the parents hold. Measured: 16 tensors of
// 32 rows of 2 MB in 300 us (1.8 GB, 6.0 TB/s); 56 tensors of 4 rows of 38 KB in place in
// 4.4 us, three memory round trips (arguments, parents, rows).
#include <algorithm>

#include "qg_device.h"
#include "qg_host.h"

namespace {

// Units of any alignment: the hardware takes unaligned accesses of up to 16 bytes.
template <int B>
struct Unit;
template <>
struct Unit<16> {
    typedef uint32_t T __attribute__((ext_vector_type(4), aligned(1)));
};
template <>
struct Unit<8> {
    typedef uint32_t T __attribute__((ext_vector_type(2), aligned(1)));
};
template <>
struct Unit<4> {
    typedef uint32_t T __attribute__((aligned(1)));
};
template <>
struct Unit<2> {
    typedef uint16_t T __attribute__((aligned(1)));
};
template <>
struct Unit<1> {
    typedef uint8_t T;
};

struct RState {
    const uint8_t* src;
    uint8_t* dst;
    int64_t src_row, dst_row, src_outer, dst_outer;
    uint32_t per, cols;  // 16-byte columns of a piece and of a row
    uint32_t tail;       // bytes of a piece's last column, 16 or fewer
};
struct RArgs {
    RState st[QG_BEAM_MAX_STATES];
    const int32_t* parent;
    int32_t beams_in, beams_out;
};

// Rows J .. W - 1 of B bytes of a column: all of them are read before the first is
// written (the reads of the later rows lie inside the call between a row's read and its
// write). As a recursion over single values: an array of them became one wide register
// that every branch copied (226 registers at eight beams, here 40).
template <int B, int W, int J>
QG_DEV void move_rows(const uint8_t* src, uint8_t* dst, const RState& s, const int (&p)[W]) {
    typedef typename Unit<B>::T U;
    if constexpr (J < W) {
        U v{};
        if (p[J] >= 0) v = *reinterpret_cast<const U*>(src + p[J] * s.src_row);
        move_rows<B, W, J + 1>(src, dst, s, p);
        if (p[J] >= 0) *reinterpret_cast<U*>(dst + J * s.dst_row) = v;
    }
}

template <int W>
__global__ __launch_bounds__(256) void beam_reorder_kernel(RArgs a) {
    const RState& s = a.st[blockIdx.z];
    const uint32_t c = blockIdx.x * 256u + threadIdx.x;
    const int64_t b = blockIdx.y;
    const int32_t* par = a.parent + b * a.beams_out;
    const bool inplace = s.src == s.dst;
    int p[W];  // parents of the rows that move, else -1
#pragma unroll
    for (int j = 0; j < W; ++j) {
        p[j] = j < a.beams_out ? par[j] : -1;
        if (p[j] < 0 || p[j] >= a.beams_in || (inplace && p[j] == j)) p[j] = -1;
    }
    if (c >= s.cols) return;
    const uint32_t o = c / s.per, i = c - o * s.per;
    const uint8_t* src = s.src + b * a.beams_in * s.src_row + o * s.src_outer + (int64_t)i * 16;
    uint8_t* dst = s.dst + b * a.beams_out * s.dst_row + o * s.dst_outer + (int64_t)i * 16;
    const uint32_t bytes = i + 1 == s.per ? s.tail : 16;
    if (bytes == 16) {
        move_rows<16, W, 0>(src, dst, s, p);
        return;
    }
    uint32_t at = 0;
    if (bytes & 8) move_rows<8, W, 0>(src, dst, s, p), at = 8;
    if (bytes & 4) move_rows<4, W, 0>(src + at, dst + at, s, p), at += 4;
    if (bytes & 2) move_rows<2, W, 0>(src + at, dst + at, s, p), at += 2;
    if (bytes & 1) move_rows<1, W, 0>(src + at, dst + at, s, p);
}

int64_t cols_of(const qg_beam_state& s) { return s.outer * qg::ceil_div(s.span, 16); }

qg_status launch(const RArgs& a, int n, uint32_t cols, int64_t batch, hipStream_t stream) {
    const dim3 g((cols + 255) / 256, (unsigned)batch, (unsigned)n);
    // (no instance for 16: with 9 to 16 beams the one for 32, at three wavefronts per SIMD
    // instead of six, moves 400 MB of 12 beams in 120 us instead of 131; with four beams it
    // takes 435 us where the first takes 300)
    if (a.beams_out <= 4)
        hipLaunchKernelGGL((beam_reorder_kernel<4>), g, dim3(256), 0, stream, a);
    else if (a.beams_out <= 8)
        hipLaunchKernelGGL((beam_reorder_kernel<8>), g, dim3(256), 0, stream, a);
    else
        hipLaunchKernelGGL((beam_reorder_kernel<QG_BEAM_MAX>), g, dim3(256), 0, stream, a);
    return qg::launch_status("qg_beam_reorder");
}

qg_status check(const qg_beam_state* states, int count, const int32_t* parent, int64_t batch, int beams_in,
                int beams_out) {
    if (!states || !parent) return qg::fail(QG_ERR_NULL, "NULL pointer (states, parent)");
    if (count < 1 || count > QG_BEAM_MAX_STATES)
        return qg::fail(QG_ERR_SHAPE, "count=%d not in [1, %d]", count, QG_BEAM_MAX_STATES);
    if (beams_in < 1 || beams_in > QG_BEAM_MAX || beams_out < 1 || beams_out > QG_BEAM_MAX)
        return qg::fail(QG_ERR_SHAPE, "beams_in=%d or beams_out=%d not in [1, %d]", beams_in, beams_out, QG_BEAM_MAX);
    if (batch < 1 || batch > 65535) return qg::fail(QG_ERR_SHAPE, "batch=%lld not in [1, 65535]", (long long)batch);
    if (reinterpret_cast<uintptr_t>(parent) & 3) return qg::fail(QG_ERR_ALIGN, "parent not 4-byte aligned");
    const int64_t most = (int64_t)1 << 40;  // products with 2^21 rows stay below 2^62
    for (int k = 0; k < count; ++k) {
        const qg_beam_state& s = states[k];
        if (!s.src || !s.dst) return qg::fail(QG_ERR_NULL, "state %d: src or dst is NULL", k);
        if (s.outer < 1 || s.span < 1 || s.outer >= most || s.span >= most / s.outer)
            return qg::fail(QG_ERR_SHAPE, "state %d: outer=%lld, span=%lld not in range", k, (long long)s.outer,
                            (long long)s.span);
        if (s.src_row < 0 || s.dst_row < 0 || s.src_outer < 0 || s.dst_outer < 0 || s.src_row > most ||
            s.dst_row > most || s.src_outer > most || s.dst_outer > most)
            return qg::fail(QG_ERR_SHAPE, "state %d: a stride is not in [0, 2^40]", k);
        if (s.outer > 1 && std::max(s.src_outer, s.dst_outer) > ((int64_t)1 << 60) / (s.outer - 1))
            return qg::fail(QG_ERR_SHAPE, "state %d: a row spans over 2^60 bytes", k);
        for (int j = 0; j < k; ++j)
            if (s.dst == states[j].dst || s.dst == states[j].src || s.src == states[j].dst)
                return qg::fail(QG_ERR_SHAPE, "states %d and %d share a result", j, k);
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
        if (cols_of(s) > 0xffffff00ll)  // a launch has fewer than 2^32 threads along x
            return qg::fail(QG_ERR_SHAPE, "state %d: a row holds over 2^32 columns of 16 bytes", k);
    }
    return QG_OK;
}

}  // namespace

extern "C" qg_status qg_beam_reorder_check(const qg_beam_state* states, int count, const int32_t* parent, int64_t batch,
                                           int beams_in, int beams_out) {
    qg::clear_error();
    return check(states, count, parent, batch, beams_in, beams_out);
}

extern "C" qg_status qg_beam_reorder(const qg_beam_state* states, int count, const int32_t* parent, int64_t batch,
                                     int beams_in, int beams_out, qg_stream_t stream) {
    qg::clear_error();
    qg_status st = check(states, count, parent, batch, beams_in, beams_out);
    if (st) return st;
    st = qg::check_device();
    if (st) return st;
    // One launch for the states whose rows are alike in length to a factor of two (a
    // model's layers: one launch): a workgroup finds its state by its index.
    uint64_t left = ((uint64_t)1 << count) - 1;
    while (left) {
        const int64_t c0 = cols_of(states[__builtin_ctzll(left)]);
        RArgs a{};
        a.parent = parent;
        a.beams_in = beams_in;
        a.beams_out = beams_out;
        int n = 0;
        int64_t longest = 0;
        for (int k = __builtin_ctzll(left); k < count; ++k) {
            const qg_beam_state& s = states[k];
            const int64_t c = cols_of(s);
            if (!(left >> k & 1) || c > 2 * c0 || c0 > 2 * c) continue;
            left &= ~((uint64_t)1 << k);
            a.st[n++] = {(const uint8_t*)s.src, (uint8_t*)s.dst, s.src_row, s.dst_row, s.src_outer, s.dst_outer,
                         (uint32_t)qg::ceil_div(s.span, 16), (uint32_t)c, (uint32_t)((s.span - 1) % 16 + 1)};
            longest = std::max(longest, c);
        }
        st = launch(a, n, (uint32_t)longest, batch, (hipStream_t)stream);
        if (st) return st;
    }
    return st;
}
