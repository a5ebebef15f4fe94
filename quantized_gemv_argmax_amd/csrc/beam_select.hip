// Beam search's selection over beams and vocabulary, for gfx950.
//
// Candidate v of live beam w scores score_w + ((z_v - m) - log sum exp(z - m)), m the
// row's maximum; the n best over all beams of an item are wanted. Within a beam the
// score only grows with the logit, so each beam's n best logits (equal ones: the
// lower token) hold all it can contribute, and only those are scored.
//
// Double precision: two beams' candidates are ranked by the difference of numbers
// that went through a sum of up to 262144 exponentials, and float32 sums would
// decide near ties by their own rounding. z - m is exact there, so a constant added
// to a row changes nothing.
//
// Stages.
//  1. beam_stats_kernel, one pass over the logits: per wavefront's segment its
//     maximum m and sum of exp(z - m); per tile (16 lanes' vectors) the key of its
//     best element.
//  2. beam_row_kernel, one workgroup per row: the n-th best of the threads' best
//     tile keys bounds the n-th best element from below (n elements reach it), so
//     only tiles that reach it are read again, and of them only such elements; they
//     are ranked by counting the larger ones.
//  3. beam_item_kernel, one workgroup per item: scores of the rows' n best, ranked by
//     counting.
// Keys are order-preserving value bits above the complement of the token, so that
// no two are equal and every order of arrival gives the same result.
#include <algorithm>
#include <climits>
#include <cmath>

#include "qg_device.h"
#include "qg_host.h"

namespace {

constexpr int kWG = 256;
constexpr int kSegVec = 8;      // 16-byte vectors per lane and segment
constexpr int kBuf = 1024;      // candidate buffer of stage 2
constexpr double kMaxAlpha = 16;
constexpr float kMaxF = 3.4028234663852886e38f;

template <int XT>
struct Log;
template <>
struct Log<QG_F32> {
    static constexpr int N = 4;
    QG_DEV static float get(const uint4& v, int i) { return __builtin_bit_cast(float, (&v.x)[i]); }
    QG_DEV static float at(const void* p, int64_t i) { return reinterpret_cast<const float*>(p)[i]; }
};
template <>
struct Log<QG_F16> {
    static constexpr int N = 8;
    QG_DEV static float get(const uint4& v, int i) {
        return (i & 1) ? qg_half_hi((&v.x)[i >> 1]) : qg_half_lo((&v.x)[i >> 1]);
    }
    QG_DEV static float at(const void* p, int64_t i) { return qg_half_lo(reinterpret_cast<const uint16_t*>(p)[i]); }
};
template <>
struct Log<QG_BF16> {
    static constexpr int N = 8;
    QG_DEV static float get(const uint4& v, int i) {
        const uint32_t w = (&v.x)[i >> 1];
        return __builtin_bit_cast(float, (i & 1) ? (w & 0xffff0000u) : (w << 16));
    }
    QG_DEV static float at(const void* p, int64_t i) {
        return __builtin_bit_cast(float, (uint32_t)reinterpret_cast<const uint16_t*>(p)[i] << 16);
    }
};

struct BArgs {
    const void* logits;
    int64_t ld;
    int32_t rows, beams, vocab, n;
    int32_t tiles, segs;  // per row
    const float* score;
    const uint8_t* finished;
    const int32_t* length;
    double alpha;
    int32_t eos;
    float* segmax;      // [rows][segs]
    double* segsum;     // [rows][segs]
    uint64_t* tkey;     // [rows][tiles]
    uint64_t* rowkey;   // [rows][n], best first, 0: none
    double2* rowstat;   // [rows]: maximum, log of the sum
    qg_beam_out out;
};

// Masked elements (NaN, -inf) become -inf, +inf the largest float.
QG_DEV float clean(float v) {
    const float ninf = -__builtin_huge_valf();
    return v != v ? ninf : fminf(v, kMaxF);
}
QG_DEV uint64_t key_of(float v, int token) {
    return v == -__builtin_huge_valf() ? 0 : ((uint64_t)qg_ord(v) << 32) | (0xffffffffu - (uint32_t)token);
}
QG_DEV float key_value(uint64_t k) { return qg_unord((uint32_t)(k >> 32)); }
QG_DEV int key_token(uint64_t k) { return (int)(0xffffffffu - (uint32_t)k); }

QG_DEV uint64_t shfl_xor64(uint64_t v, int m) {
    const uint32_t lo = (uint32_t)__shfl_xor((int)(uint32_t)v, m), hi = (uint32_t)__shfl_xor((int)(v >> 32), m);
    return ((uint64_t)hi << 32) | lo;
}

// Rows start at any element: vectors are read from the 16-byte boundary at or below
// a row's start, `sh` elements before it. (The base is aligned, so that boundary is
// never before the buffer.)
template <int XT>
struct Row {
    const uint8_t* base;
    int sh, vocab;
    QG_DEV Row(const void* logits, int64_t ld, int64_t row, int vocab_) : vocab(vocab_) {
        constexpr int eb = 16 / Log<XT>::N;
        const uint8_t* p = (const uint8_t*)logits + row * ld * eb;
        sh = (int)((reinterpret_cast<uintptr_t>(p) & 15) / eb);
        base = p - sh * eb;
    }
    // vector i's elements; outside the row -inf. Full vectors are one load, the
    // last one stays inside the row.
    QG_DEV void load(int64_t i, float (&v)[Log<XT>::N]) const {
        constexpr int N = Log<XT>::N;
        const int64_t e0 = i * N - sh;
        const float ninf = -__builtin_huge_valf();
        if (e0 + N <= vocab) {
            const uint4 u = *reinterpret_cast<const uint4*>(base + i * 16);
#pragma unroll
            for (int e = 0; e < N; ++e) v[e] = e0 + e >= 0 ? clean(Log<XT>::get(u, e)) : ninf;
        } else {
#pragma unroll
            for (int e = 0; e < N; ++e)
                v[e] = e0 + e >= 0 && e0 + e < vocab ? clean(Log<XT>::at(base, i * N + e)) : ninf;
        }
    }
};

// ---------------------------------------------------------------- stage 1
template <int XT>
__global__ __launch_bounds__(kWG) void beam_stats_kernel(BArgs a) {
    constexpr int N = Log<XT>::N;
    const int lane = threadIdx.x & 63;
    const int64_t g = (int64_t)blockIdx.x * (kWG / 64) + (threadIdx.x >> 6);
    const int64_t row = g / a.segs;
    if (row >= a.rows) return;
    if (a.finished && a.finished[row]) return;
    const int seg = (int)(g - row * a.segs);
    const Row<XT> r(a.logits, a.ld, row, a.vocab);
    const float ninf = -__builtin_huge_valf();
    float v[kSegVec][N];
#pragma unroll
    for (int j = 0; j < kSegVec; ++j) r.load(((int64_t)seg * kSegVec + j) * 64 + lane, v[j]);
    float mx = ninf;
#pragma unroll
    for (int j = 0; j < kSegVec; ++j) {
        const int64_t i = ((int64_t)seg * kSegVec + j) * 64 + lane;
        float best = v[j][0];
        int at = 0;
#pragma unroll
        for (int e = 1; e < N; ++e)
            if (v[j][e] > best) best = v[j][e], at = e;
        uint64_t k = key_of(best, (int)(i * N - r.sh) + at);
#pragma unroll
        for (int m = 1; m < 16; m <<= 1) {
            const uint64_t o = shfl_xor64(k, m);
            k = o > k ? o : k;
        }
        const int64_t tile = ((int64_t)seg * kSegVec + j) * 4 + (lane >> 4);
        if ((lane & 15) == 0 && tile < a.tiles) a.tkey[row * a.tiles + tile] = k;
        mx = fmaxf(mx, best);
    }
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) mx = fmaxf(mx, __shfl_xor(mx, m));
    double s = 0;
    if (mx != ninf)
#pragma unroll
        for (int j = 0; j < kSegVec; ++j)
#pragma unroll
            for (int e = 0; e < N; ++e)
                if (v[j][e] != ninf) s += exp((double)v[j][e] - (double)mx);
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) s += __shfl_xor(s, m);
    if (lane == 0) {
        a.segmax[row * a.segs + seg] = mx;
        a.segsum[row * a.segs + seg] = s;
    }
}

// ---------------------------------------------------------------- stage 2
// Ranks the `c` keys of buf (distinct, nonzero; c <= kBuf) by counting and moves the
// best min(c, n) to buf in order. Every thread of the workgroup calls it.
QG_DEV int rank_buf(uint64_t* buf, int c, int n) {
    uint64_t k[kBuf / kWG];
    int rk[kBuf / kWG];
#pragma unroll
    for (int j = 0; j < kBuf / kWG; ++j) {
        const int i = threadIdx.x + j * kWG;
        k[j] = i < c ? buf[i] : 0;
        rk[j] = 0;
    }
    for (int i = 0; i < c; ++i) {
        const uint64_t o = buf[i];
#pragma unroll
        for (int j = 0; j < kBuf / kWG; ++j) rk[j] += o > k[j];
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kBuf / kWG; ++j)
        if (k[j] && rk[j] < n) buf[rk[j]] = k[j];
    __syncthreads();
    return min(c, n);
}

template <int XT>
__global__ __launch_bounds__(kWG) void beam_row_kernel(BArgs a) {
    constexpr int N = Log<XT>::N;
    __shared__ uint64_t buf[kBuf];
    __shared__ uint64_t bound;
    __shared__ int count, waiting;
    __shared__ float wmx[kWG / 64];
    __shared__ double wsum[kWG / 64];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t row = blockIdx.x;
    if (a.finished && a.finished[row]) return;
    const float ninf = -__builtin_huge_valf();
    const Row<XT> r(a.logits, a.ld, row, a.vocab);

    // the row's maximum and log-sum, in a fixed order
    const float* sm = a.segmax + row * a.segs;
    const double* ss = a.segsum + row * a.segs;
    float mx = ninf;
    for (int i = tid; i < a.segs; i += kWG) mx = fmaxf(mx, sm[i]);
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) mx = fmaxf(mx, __shfl_xor(mx, m));
    if (lane == 0) wmx[wave] = mx;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWG / 64; ++w) mx = fmaxf(mx, wmx[w]);
    double s = 0;
    for (int i = tid; i < a.segs; i += kWG)
        if (sm[i] != ninf) s += ss[i] * exp((double)sm[i] - (double)mx);
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) s += __shfl_xor(s, m);
    if (lane == 0) wsum[wave] = s;

    // a bound that at least n elements reach (or none, with fewer tiles than n)
    const uint64_t* tk = a.tkey + row * a.tiles;
    uint64_t best = 0;
    for (int i = tid; i < a.tiles; i += kWG) best = max(best, tk[i]);
    buf[tid] = best;
    if (tid == 0) {
        bound = 1;
        count = 0;
    }
    __syncthreads();
    if (tid == 0) {
        double t = 0;
        for (int w = 0; w < kWG / 64; ++w) t += wsum[w];
        a.rowstat[row] = make_double2((double)mx, mx == ninf ? 0. : log(t));
    }
    int rk = 0;
    for (int i = 0; i < kWG; ++i) rk += buf[i] > best;
    if (best && rk == a.n - 1) bound = best;
    __syncthreads();

    // Elements that reach the bound, tile by tile. The buffer is cut back to its n
    // best whenever the next round could overflow it, and the bound rises with it.
    uint64_t T0 = bound;
    constexpr int L = 16;  // lanes per tile
    const int grp = tid / L, sub = tid % L;
    for (int t0 = 0; t0 < a.tiles; t0 += kWG / L) {
        const int t = t0 + grp;
        const bool go = t < a.tiles && tk[t] >= T0;
        if (!__syncthreads_or(go)) continue;
        float v[N];
        const int64_t i = (int64_t)t * L + sub;
        if (go) r.load(i, v);
#pragma unroll
        for (int e = 0; e < N; ++e) {
            const uint64_t k = go ? key_of(v[e], (int)(i * N - r.sh) + e) : 0;
            if (tid == 0) waiting = count;
            __syncthreads();
            if (waiting + kWG > kBuf) {
                const int c = rank_buf(buf, waiting, a.n);
                if (c == a.n) T0 = buf[a.n - 1];
                __syncthreads();
                if (tid == 0) count = c;
                __syncthreads();
            }
            if (k && k >= T0) buf[atomicAdd(&count, 1)] = k;
            __syncthreads();
        }
    }
    const int c = rank_buf(buf, count, a.n);
    for (int i = tid; i < a.n; i += kWG) a.rowkey[row * a.n + i] = i < c ? buf[i] : 0;
}

// ---------------------------------------------------------------- stage 3
// Candidate i (beam-major, each beam's in order) of an item. Order: rank descending,
// then i ascending.
__global__ __launch_bounds__(kWG) void beam_item_kernel(BArgs a) {
    __shared__ double rank[QG_BEAM_MAX * QG_BEAM_MAX_SELECT];
    __shared__ int place[QG_BEAM_MAX_SELECT];
    const int tid = threadIdx.x;
    const int64_t item = blockIdx.x;
    const int total = a.beams * a.n;
    const double ninf = -__builtin_huge_val();
    if (tid < a.n) place[tid] = -1;

    auto candidate = [&](int i, double& sc, int& token, int& len, bool& done) {
        const int w = i / a.n, j = i - w * a.n;
        const int64_t row = item * a.beams + w;
        const float cum = a.score[row];
        done = a.finished && a.finished[row];
        const int l = a.length ? a.length[row] : 0;
        len = done ? l : l + 1;
        sc = ninf;
        token = -1;
        if (cum != cum || cum == -__builtin_huge_valf()) return;
        if (done) {
            if (j == 0) {
                sc = cum;
                token = a.eos;
            }
            return;
        }
        const uint64_t k = a.rowkey[row * a.n + j];
        if (!k) return;
        const double2 st = a.rowstat[row];
        token = key_token(k);
        sc = (double)cum + (((double)key_value(k) - st.x) - st.y);
    };

    for (int i = tid; i < total; i += kWG) {
        double sc;
        int token, len;
        bool done;
        candidate(i, sc, token, len, done);
        if (token >= 0 && a.alpha != 0.) sc /= pow((double)max(len, 1), a.alpha);
        rank[i] = sc;
    }
    __syncthreads();
    for (int i = tid; i < total; i += kWG) {
        const double k = rank[i];
        if (k == ninf) continue;
        int before = 0;
        for (int o = 0; o < total; ++o) before += rank[o] > k || (rank[o] == k && o < i);
        if (before < a.n) place[before] = i;
    }
    __syncthreads();
    double sc = ninf;
    int token = -1, parent = -1, len = 0;
    bool done = false;
    if (tid < a.n && place[tid] >= 0) {
        candidate(place[tid], sc, token, len, done);
        parent = place[tid] / a.n;
    }
    __syncthreads();  // every input is read before an output, which may be the same array, is written
    if (tid < a.n) {
        const int64_t o = item * a.n + tid;
        a.out.token[o] = token;
        a.out.parent[o] = parent;
        a.out.score[o] = (float)sc;
        if (a.out.finished) a.out.finished[o] = parent >= 0 && (done || (a.eos >= 0 && token == a.eos));
        if (a.out.length) a.out.length[o] = parent >= 0 ? len : 0;
    }
}

// ---------------------------------------------------------------- host
int vec_elems(int type) { return type == QG_F32 ? 4 : 8; }

struct Plan {
    int64_t rows;
    int tiles, segs;
    size_t segmax, segsum, tkey, rowkey, rowstat, total;
};
Plan plan(int type, int64_t batch, int beams, int64_t vocab, int n) {
    Plan p;
    p.rows = batch * beams;
    const int64_t ve = vec_elems(type);
    const int64_t vecs = qg::ceil_div(vocab + ve - 1, ve);  // a row may start inside a vector
    p.tiles = (int)qg::ceil_div(vecs, 16);
    p.segs = (int)qg::ceil_div(vecs, 64 * kSegVec);
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t o = at;
        at = qg::align_up(at + bytes, 256);
        return o;
    };
    p.segmax = take((size_t)p.rows * p.segs * 4);
    p.segsum = take((size_t)p.rows * p.segs * 8);
    p.tkey = take((size_t)p.rows * p.tiles * 8);
    p.rowkey = take((size_t)p.rows * n * 8);
    p.rowstat = take((size_t)p.rows * 16);
    p.total = at;
    return p;
}

qg_status check_shape(int type, int64_t batch, int beams, int64_t vocab, int n) {
    if (type != QG_F32 && type != QG_F16 && type != QG_BF16)
        return qg::fail(QG_ERR_SHAPE, "logits_type=%d unknown", type);
    if (beams < 1 || beams > QG_BEAM_MAX) return qg::fail(QG_ERR_SHAPE, "beams=%d not in [1, %d]", beams, QG_BEAM_MAX);
    if (batch < 1 || batch > (1 << 20) / beams)
        return qg::fail(QG_ERR_SHAPE, "batch=%lld below 1, or over 2^20 rows", (long long)batch);
    if (vocab < 1 || vocab > QG_TOPK_MAX_ROWS)
        return qg::fail(QG_ERR_SHAPE, "vocab=%lld not in [1, %d]", (long long)vocab, QG_TOPK_MAX_ROWS);
    if (n < 1 || n > QG_BEAM_MAX_SELECT) return qg::fail(QG_ERR_SHAPE, "n=%d not in [1, %d]", n, QG_BEAM_MAX_SELECT);
    return QG_OK;
}

bool overlap(const void* a, size_t na, const void* b, size_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return a && b && x < y + nb && y < x + na;
}

template <int XT>
qg_status launch(const BArgs& a, int64_t batch, hipStream_t s) {
    const int64_t waves = (int64_t)a.rows * a.segs;
    hipLaunchKernelGGL(beam_stats_kernel<XT>, dim3((unsigned)qg::ceil_div(waves, kWG / 64)), dim3(kWG), 0, s, a);
    qg_status st = qg::launch_status("logits_beam_select (statistics)");
    if (st) return st;
    hipLaunchKernelGGL(beam_row_kernel<XT>, dim3((unsigned)a.rows), dim3(kWG), 0, s, a);
    st = qg::launch_status("logits_beam_select (rows)");
    if (st) return st;
    hipLaunchKernelGGL(beam_item_kernel, dim3((unsigned)batch), dim3(kWG), 0, s, a);
    return qg::launch_status("logits_beam_select (items)");
}

}  // namespace

extern "C" {

size_t logits_beam_select_workspace_bytes(int type, int64_t batch, int beams, int64_t vocab, int n) {
    if (check_shape(type, batch, beams, vocab, n)) {
        qg::clear_error();
        return 0;
    }
    return plan(type, batch, beams, vocab, n).total;
}

qg_status logits_beam_select(const qg_beam_in* in, int n, void* ws, size_t ws_bytes, const qg_beam_out* out,
                             qg_stream_t stream) {
    qg::clear_error();
    if (!in || !out) return qg::fail(QG_ERR_NULL, "NULL descriptor (in, out)");
    if (!in->logits || !in->score) return qg::fail(QG_ERR_NULL, "in->logits or in->score is NULL");
    if (!out->token || !out->parent || !out->score)
        return qg::fail(QG_ERR_NULL, "out->token, out->parent or out->score is NULL");
    qg_status st = check_shape(in->logits_type, in->batch, in->beams, in->vocab, n);
    if (st) return st;
    const int64_t rows = in->batch * in->beams, sel = in->batch * n;
    if (in->ld < in->vocab || in->ld > ((int64_t)1 << 40) / rows)
        return qg::fail(QG_ERR_SHAPE, "ld=%lld not in [vocab, 2^40 / rows]", (long long)in->ld);
    if (in->eos < -1 || in->eos >= in->vocab)
        return qg::fail(QG_ERR_SHAPE, "eos=%d not -1 and not in [0, vocab)", in->eos);
    if (in->finished && in->eos < 0) return qg::fail(QG_ERR_SHAPE, "finished beams need an eos token");
    if (!(std::fabs(in->length_penalty) <= kMaxAlpha))  // keeps len^length_penalty and the ranks finite
        return qg::fail(QG_ERR_SHAPE, "length_penalty not in [-%g, %g]", kMaxAlpha, kMaxAlpha);
    if (!in->length && (in->length_penalty != 0. || out->length))
        return qg::fail(QG_ERR_NULL, "in->length is NULL while a length penalty or out->length asks for it");
    if (!qg::aligned16(in->logits)) return qg::fail(QG_ERR_ALIGN, "logits not 16-byte aligned");
    const void* four[6] = {in->score, in->length, out->token, out->parent, out->score, out->length};
    for (const void* p : four)
        if (reinterpret_cast<uintptr_t>(p) & 3)
            return qg::fail(QG_ERR_ALIGN, "score, length, token and parent arrays must be 4-byte aligned");
    // outputs against inputs (the same array in place with n == beams) and each other
    const int eb = in->logits_type == QG_F32 ? 4 : 2;
    struct Span {
        const void* p;
        size_t n;
        bool written;
    };
    const Span spans[9] = {{in->logits, ((size_t)(rows - 1) * in->ld + in->vocab) * eb, false},
                           {in->score, (size_t)rows * 4, false},
                           {in->finished, (size_t)rows, false},
                           {in->length, (size_t)rows * 4, false},
                           {out->token, (size_t)sel * 4, true},
                           {out->parent, (size_t)sel * 4, true},
                           {out->score, (size_t)sel * 4, true},
                           {out->finished, (size_t)sel, true},
                           {out->length, (size_t)sel * 4, true}};
    for (int i = 0; i < 9; ++i)
        for (int j = i + 1; j < 9; ++j) {
            if (!spans[j].written || !overlap(spans[i].p, spans[i].n, spans[j].p, spans[j].n)) continue;
            const bool step = n == in->beams && spans[i].p == spans[j].p &&
                              ((i == 1 && j == 6) || (i == 2 && j == 7) || (i == 3 && j == 8));
            if (!step) return qg::fail(QG_ERR_SHAPE, "an output overlaps an input or another output");
        }
    const Plan p = plan(in->logits_type, in->batch, in->beams, in->vocab, n);
    if (!ws || ws_bytes < p.total)
        return qg::fail(QG_ERR_WORKSPACE, "workspace of %zu bytes required, got %zu", p.total, ws ? ws_bytes : 0);
    if (!qg::aligned16(ws)) return qg::fail(QG_ERR_ALIGN, "workspace not 16-byte aligned");
    for (const Span& s : spans)
        if (overlap(s.p, s.n, ws, p.total)) return qg::fail(QG_ERR_SHAPE, "the workspace overlaps an operand");
    st = qg::check_device();
    if (st) return st;
    uint8_t* w8 = (uint8_t*)ws;
    BArgs a{};
    a.logits = in->logits;
    a.ld = in->ld;
    a.rows = (int32_t)rows;
    a.beams = in->beams;
    a.vocab = (int32_t)in->vocab;
    a.n = n;
    a.tiles = p.tiles;
    a.segs = p.segs;
    a.score = in->score;
    a.finished = in->finished;
    a.length = in->length;
    a.alpha = in->length_penalty;
    a.eos = in->eos;
    a.segmax = (float*)(w8 + p.segmax);
    a.segsum = (double*)(w8 + p.segsum);
    a.tkey = (uint64_t*)(w8 + p.tkey);
    a.rowkey = (uint64_t*)(w8 + p.rowkey);
    a.rowstat = (double2*)(w8 + p.rowstat);
    a.out = *out;
    hipStream_t s = (hipStream_t)stream;
    if (in->logits_type == QG_F32) return launch<QG_F32>(a, in->batch, s);
    if (in->logits_type == QG_F16) return launch<QG_F16>(a, in->batch, s);
    return launch<QG_BF16>(a, in->batch, s);
}

}  // extern "C"
