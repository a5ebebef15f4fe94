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
// Stages, two launches.
//  1. beam_stats_kernel, one pass over the logits: per wavefront's segment its
//     maximum m and sum of exp(z - m), and the maximum of every tile of 8 vectors of
//     16 bytes.
//  2. beam_rank_kernel, one workgroup per row: the n-th largest of the threads' best
//     tile maxima is a bound that at least n elements reach, so only tiles that reach
//     it are read again, and of them only such elements; they are ranked by counting
//     the better ones. The item's last workgroup to finish scores its rows' n best
//     and ranks those the same way.
// Elements are ranked by keys, order-preserving value bits above the complement of
// the token, no two equal: every order of arrival gives the same result.
#include <algorithm>
#include <climits>
#include <cmath>
#include <type_traits>

#include "qg_device.h"
#include "qg_host.h"

namespace {

constexpr int kWG = 256;
constexpr int kMaxRows = 65536;
constexpr int kBuf = 1024;      // candidate buffer of stage 2
constexpr int kList = 1024;     // tiles of one listing
constexpr double kMaxAlpha = 16;
constexpr float kMaxF = 3.4028234663852886e38f;

template <int XT>
struct Log;
template <>
struct Log<QG_F32> {
    static constexpr int N = 4;  // elements of a 16-byte vector
    typedef uint32_t V __attribute__((ext_vector_type(4), aligned(4)));
    QG_DEV static float get(const uint4& v, int i) { return __builtin_bit_cast(float, (&v.x)[i]); }
    QG_DEV static float at(const void* p, int64_t i) { return reinterpret_cast<const float*>(p)[i]; }
};
template <>
struct Log<QG_F16> {
    static constexpr int N = 8;
    typedef uint32_t V __attribute__((ext_vector_type(4), aligned(2)));
    QG_DEV static float get(const uint4& v, int i) {
        return (i & 1) ? qg_half_hi((&v.x)[i >> 1]) : qg_half_lo((&v.x)[i >> 1]);
    }
    QG_DEV static float at(const void* p, int64_t i) { return qg_half_lo(reinterpret_cast<const uint16_t*>(p)[i]); }
};
template <>
struct Log<QG_BF16> {
    static constexpr int N = 8;
    typedef uint32_t V __attribute__((ext_vector_type(4), aligned(2)));
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
    float* tmax;        // [rows][tiles], rows of a multiple of 4
    uint64_t* rowkey;   // [rows][n], best first, 0: none
    double* rowstat;    // [rows][2]: maximum, log of the sum
    uint32_t* arrived;  // [items]: rows ranked so far
    qg_beam_out out;
};

QG_DEV float neg_inf() { return -__builtin_huge_valf(); }

// Masked elements (NaN, -inf) become -inf, +inf the largest float.
QG_DEV float clean(float v) { return v == v ? fminf(v, kMaxF) : neg_inf(); }
QG_DEV uint64_t key_of(float v, int token) {
    return v == neg_inf() ? 0 : ((uint64_t)qg_ord(v) << 32) | (0xffffffffu - (uint32_t)token);
}
QG_DEV float key_value(uint64_t k) { return qg_unord((uint32_t)(k >> 32)); }
QG_DEV int key_token(uint64_t k) { return (int)(0xffffffffu - (uint32_t)k); }

// exp(v - m) for float32 v <= m, m finite, to 1e-12 of the result: x = v - m is exact in
// double, x = k ln 2 + r with |r| <= ln 2 / 2, exp(r) by the polynomial of degree 8 that
// is 1 at 0 and whose largest relative error over that range is least (8.2e-13; found by
// iterated least squares), and k added to the exponent. k comes from the low bits of a
// sum with 1.5 * 2^52, and x is bounded below through v, one operation each: the
// stage is bound by its instructions. With the bound at m - 600 (not for a large m,
// where float32 steps are wide: there x is bounded), v below it, -inf among them, counts
// as exp(-600), which keeps the result normal and far below what a sum can show.
template <bool WIDE>
QG_DEV double exp_diff(float v, float m) {
    const double x = WIDE ? __builtin_fmax((double)v - (double)m, -600.) : (double)fmaxf(v, m - 600.f) - (double)m;
    const double big = 6755399441055744.;
    const double t = __builtin_fma(x, 1.4426950408889634074, big);
    const double r = __builtin_fma(t - big, -0.69314718055994530942, x);
    double p = 2.473297530561428e-05;
    p = __builtin_fma(p, r, 0.0001991468052941343);
    p = __builtin_fma(p, r, 0.001388915504606253);
    p = __builtin_fma(p, r, 0.00833326875520095);
    p = __builtin_fma(p, r, 0.041666664536176984);
    p = __builtin_fma(p, r, 0.16666666873332264);
    p = __builtin_fma(p, r, 0.5000000000458368);
    p = __builtin_fma(p, r, 0.9999999999830598);
    p = __builtin_fma(p, r, 1.);
    const uint64_t b = __builtin_bit_cast(uint64_t, p);
    const uint32_t hi = (uint32_t)(b >> 32) + ((uint32_t)__builtin_bit_cast(uint64_t, t) << 20);
    return __builtin_bit_cast(double, ((uint64_t)hi << 32) | (uint32_t)b);
}
// Whether m is too large for the narrow form.
QG_DEV bool wide(float m) { return fabsf(m) > 1e6f; }

template <int CTRL>
QG_DEV float dpp(float v) {
    return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), CTRL, 0xf, 0xf, true));
}
template <int CTRL>
QG_DEV double dpp(double v) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_mov_dpp((int)(uint32_t)b, CTRL, 0xf, 0xf, true);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_mov_dpp((int)(b >> 32), CTRL, 0xf, 0xf, true);
    return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}
QG_DEV double readlane(double v, int l) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)b, l);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(b >> 32), l);
    return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}
// Maximum and sum over the wavefront, the same in every lane: quads, 8-lane and
// 16-lane mirrors, then the four rows in order.
QG_DEV float wave_max(float v) {
    v = fmaxf(v, dpp<0xb1>(v));
    v = fmaxf(v, dpp<0x4e>(v));
    v = fmaxf(v, dpp<0x141>(v));
    v = fmaxf(v, dpp<0x140>(v));
    return fmaxf(fmaxf(qg_readlane(v, 0), qg_readlane(v, 16)), fmaxf(qg_readlane(v, 32), qg_readlane(v, 48)));
}
QG_DEV double wave_sum(double v) {
    v += dpp<0xb1>(v);
    v += dpp<0x4e>(v);
    v += dpp<0x141>(v);
    v += dpp<0x140>(v);
    return ((readlane(v, 0) + readlane(v, 16)) + readlane(v, 32)) + readlane(v, 48);
}

// A row's 16-byte vectors, cut from the row's own first element, whatever its address
// (the hardware takes unaligned loads): which lane and segment an element falls to, and
// so the order of every sum, depends on the vocabulary alone, and rows that are equal
// wherever they lie, or equal but for a constant, get equal sums to the last bit. Vector
// i holds the elements i N .. i N + N - 1; only the one that holds the row's end is read
// element by element.
template <int XT>
struct Row {
    static constexpr int N = Log<XT>::N;
    typedef typename Log<XT>::V vec;
    const uint8_t* base;
    int vocab;
    QG_DEV Row(const void* logits, int64_t ld, int64_t row, int vocab_)
        : base((const uint8_t*)logits + row * ld * (16 / N)), vocab(vocab_) {}
    QG_DEV bool whole(int i) const { return i * N + N <= vocab; }  // ends inside the row
    QG_DEV bool cut(int i) const { return i * N < vocab && !whole(i); }
    QG_DEV uint4 get(int i) const {
        const vec v = *reinterpret_cast<const vec*>(base + (int64_t)i * 16);
        return make_uint4(v.x, v.y, v.z, v.w);
    }
    // elements beyond the row: -inf
    QG_DEV void mask(int i, float (&v)[N]) const {
#pragma unroll
        for (int e = 0; e < N; ++e)
            if (i * N + e >= vocab) v[e] = neg_inf();
    }
    QG_DEV void last(int i, float (&v)[N]) const {
#pragma unroll
        for (int e = 0; e < N; ++e) v[e] = clean(Log<XT>::at(base, min(i * N + e, vocab - 1)));
        mask(i, v);
    }
    QG_DEV void load(int i, float (&v)[N]) const {
        uint4 u = make_uint4(0, 0, 0, 0);
        if (whole(i)) u = get(i);
#pragma unroll
        for (int e = 0; e < N; ++e) v[e] = clean(Log<XT>::get(u, e));
        if (cut(i)) last(i, v);
        mask(i, v);
    }
};

// ---------------------------------------------------------------- stage 1
// A segment per wavefront, SV vectors of each lane; 8 / SV lanes' make a tile. Bound by
// its double-precision instructions, about 14 of 25 per element and at half the rate of
// float32's: 16 x 8 rows of 152064 bf16 (39 MB) take 21 us (a fifth of them finished:
// 20.7); with the exponentials replaced by a subtraction 20 became 12. (Walking wavefronts with the next segment's loads ahead
// of the work on one: 22 us. Splitting the polynomial between float32 and double, or a
// table of powers, trades as many instructions as it saves.)
template <int XT, int SV>
__global__ __launch_bounds__(kWG) void beam_stats_kernel(BArgs a) {
    constexpr int N = Log<XT>::N;
    constexpr int L = 8 / SV;  // lanes of a tile
    const int lane = threadIdx.x & 63;
    const uint32_t g = blockIdx.x * (kWG / 64) + (uint32_t)__builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (g < (uint32_t)(a.rows / a.beams) && lane == 0) a.arrived[g] = 0;  // (there are more wavefronts than items)
    const uint32_t row = g / (uint32_t)a.segs;
    if (row >= (uint32_t)a.rows) return;
    if (a.finished && a.finished[row]) return;
    const int seg = (int)(g - row * (uint32_t)a.segs);
    const Row<XT> r(a.logits, a.ld, row, a.vocab);
    const int first = seg * SV * 64;  // vector j of this lane: first + 64 j + lane
    uint4 u[SV];
    float v[SV][N];
#pragma unroll
    for (int j = 0; j < SV; ++j) {
        u[j] = make_uint4(0, 0, 0, 0);
        if (r.whole(first + 64 * j + lane)) u[j] = r.get(first + 64 * j + lane);
    }
#pragma unroll
    for (int j = 0; j < SV; ++j)
#pragma unroll
        for (int e = 0; e < N; ++e) v[j][e] = clean(Log<XT>::get(u[j], e));
    if (!r.whole(first + SV * 64 - 1)) {  // a row's last segment
#pragma unroll
        for (int j = 0; j < SV; ++j) {
            const int i = first + 64 * j + lane;
            if (r.cut(i))
                r.last(i, v[j]);
            else
                r.mask(i, v[j]);
        }
    }
    float best = neg_inf();
#pragma unroll
    for (int j = 0; j < SV; ++j)
#pragma unroll
        for (int e = 0; e < N; ++e) best = fmaxf(best, v[j][e]);
    static_assert(L == 4 || L == 2, "tiles are lanes of a quad");
    best = fmaxf(best, dpp<0xb1>(best));
    if (L == 4) best = fmaxf(best, dpp<0x4e>(best));
    if (lane % L == 0) a.tmax[(int64_t)row * a.tiles + seg * (64 / L) + lane / L] = best;
    const float mx = wave_max(best);
    double sum[2] = {0., 0.};
    auto add = [&](auto w) {
#pragma unroll
        for (int j = 0; j < SV; ++j)
#pragma unroll
            for (int e = 0; e < N; ++e) sum[e & 1] += exp_diff<decltype(w)::value>(v[j][e], mx);
    };
    if (wide(mx)) {
        if (mx != neg_inf()) add(std::true_type());
    } else {
        add(std::false_type());
    }
    const double all = wave_sum(sum[0] + sum[1]);
    if (lane == 0) {
        a.segmax[(int64_t)row * a.segs + seg] = mx;
        a.segsum[(int64_t)row * a.segs + seg] = all;
    }
}

// ---------------------------------------------------------------- stage 2
// Values that other workgroups of the launch read: past this XCD's L2.
template <typename V>
QG_DEV void put(V* p, V v) {
    __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
template <typename V>
QG_DEV V take(const V* p) {
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// Tile maxima of a thread, tiles of 32 (fp32) or 64 elements, and its segments, of at
// least 512 (both divide the longest row).
constexpr int kMine = (QG_TOPK_MAX_ROWS / 32 + kWG - 1) / kWG;
constexpr int kSegs = (QG_TOPK_MAX_ROWS / 512 + kWG - 1) / kWG;
static_assert(QG_TOPK_MAX_ROWS % (4 * 64 * 8) == 0, "whole segments in the longest row");
static_assert(kMine <= 64, "a thread's tiles are marked in 64 bits");

// Rows of up to so many tiles, of eight vectors each, take their bound from the vectors:
// with theirs from the tiles, 15 rows of 933 fp16 with n = 6 took 55 us, now under 20.
constexpr int kFew = kWG / 2;

struct RowShared {
    uint64_t buf[kBuf];
    float tops[kWG / 2];
    int list[kList];
    int count, listed, more;
    float wmx[kWG / 64], wlow[kWG / 64];
    double wsum[kWG / 64];
    uint64_t pairs[kWG / 2], least;
    int left;
};

// Ranks the c keys of the buffer (distinct, nonzero; c <= kBuf) by counting the larger
// ones and leaves the best min(c, n) in order. Every thread of the workgroup calls it.
// Counting takes c steps for every kWG keys, so more than kWG are first cut to those
// that reach the n-th best of the 128 pairs' maxima (distinct, so one pair holds it);
// rows of ties fill the buffer again and again.
QG_DEV int rank_buf(RowShared& sh, int c, int n) {
    constexpr int R = kBuf / kWG;
    const int tid = threadIdx.x;
    uint64_t k[R];
#pragma unroll
    for (int j = 0; j < R; ++j) k[j] = tid + j * kWG < c ? sh.buf[tid + j * kWG] : 0;
    if (c > kWG) {
        uint64_t best = k[0];
#pragma unroll
        for (int j = 1; j < R; ++j) best = max(best, k[j]);
        best = max(best, (uint64_t)__shfl_xor((unsigned long long)best, 1));
        if (!(tid & 1)) sh.pairs[tid >> 1] = best;
        if (tid == 0) sh.left = 0;
        __syncthreads();
        int reached = 0;
#pragma unroll 8
        for (int i = 0; i < kWG / 4; ++i) reached += sh.pairs[(tid & 1) * (kWG / 4) + i] >= best;
        reached += __shfl_xor(reached, 1);
        if (reached == n && !(tid & 1)) sh.least = best;
        __syncthreads();
        const uint64_t least = sh.least;
#pragma unroll
        for (int j = 0; j < R; ++j)
            if (k[j] >= least) sh.buf[atomicAdd(&sh.left, 1)] = k[j];
        __syncthreads();
        c = sh.left;
#pragma unroll
        for (int j = 0; j < R; ++j) k[j] = tid + j * kWG < c ? sh.buf[tid + j * kWG] : 0;
    }
    int rk[R] = {};
    if (c <= kWG) {
#pragma unroll 4
        for (int i = 0; i < c; ++i) rk[0] += sh.buf[i] > k[0];
    } else {
        for (int i = 0; i < c; ++i) {
            const uint64_t o = sh.buf[i];
#pragma unroll
            for (int j = 0; j < R; ++j) rk[j] += o > k[j];
        }
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < R; ++j)
        if (k[j] && rk[j] < n) sh.buf[rk[j]] = k[j];
    __syncthreads();
    return min(c, n);
}

// The row's n best keys, in order, to rowkey, and its maximum and log-sum to rowstat.
template <int XT, int SV>
QG_DEV void rank_row(const BArgs& a, int64_t row, RowShared& sh) {
    constexpr int N = Log<XT>::N;
    constexpr int L = 8 / SV;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const Row<XT> r(a.logits, a.ld, row, a.vocab);

    // maximum and log-sum, in a fixed order; meanwhile the threads' best tile maxima
    const float* sm = a.segmax + row * a.segs;
    const double* ss = a.segsum + row * a.segs;
    const float* tm = a.tmax + row * a.tiles;
    float mx = neg_inf(), best = neg_inf();
    float tv[kMine];  // this thread's tile maxima: tiles tid + kWG q
#pragma unroll
    for (int q = 0; q < kMine; ++q) tv[q] = tid + kWG * q < a.tiles ? tm[tid + kWG * q] : neg_inf();
    float segm[kSegs];
    double segs[kSegs];
#pragma unroll
    for (int q = 0; q < kSegs; ++q) {
        const int i = tid + kWG * q;
        segm[q] = i < a.segs ? sm[i] : neg_inf();
        segs[q] = i < a.segs ? ss[i] : 0.;
    }
#pragma unroll
    for (int q = 0; q < kSegs; ++q) mx = fmaxf(mx, segm[q]);
#pragma unroll
    for (int q = 0; q < kMine; ++q) best = fmaxf(best, tv[q]);
    // A row of few tiles: the best of its vectors tid + kWG q instead, since tiles would
    // leave most groups empty, and the bound low or without a value.
    if (a.tiles <= kFew) {
        best = neg_inf();
#pragma unroll
        for (int q = 0; q < kFew * 8 / kWG; ++q) {
            float v[N];
            r.load(tid + kWG * q, v);
#pragma unroll
            for (int e = 0; e < N; ++e) best = fmaxf(best, v[e]);
        }
    }
    mx = wave_max(mx);
    if (lane == 0) sh.wmx[wave] = mx;
    const bool quads = a.n <= 16;
    best = fmaxf(best, dpp<0xb1>(best));
    if (quads) best = fmaxf(best, dpp<0x4e>(best));
    if (quads ? !(tid & 3) : !(tid & 1)) sh.tops[quads ? tid >> 2 : tid >> 1] = best;
    if (tid == 0) {
        sh.count = sh.listed = 0;
    }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWG / 64; ++w) mx = fmaxf(mx, sh.wmx[w]);
    double s = 0;
    if (mx != neg_inf())
#pragma unroll
        for (int q = 0; q < kSegs; ++q) s += segs[q] * exp_diff<true>(segm[q], mx);
    s = wave_sum(s);
    if (lane == 0) sh.wsum[wave] = s;
    // The n-th largest of the 64 quads' (for up to 16) or 128 pairs' maxima: the largest
    // value that n of them reach. The threads of a group count a share of them each.
    int reached = 0;
    auto count = [&](const float* tops, auto of) {
#pragma unroll
        for (int i = 0; i < decltype(of)::value; i += 4) {
            const float4 o = *reinterpret_cast<const float4*>(tops + i);
            reached += (o.x >= best) + (o.y >= best) + (o.z >= best) + (o.w >= best);
        }
    };
    if (quads)
        count(sh.tops + (tid & 3) * (kWG / 16), std::integral_constant<int, kWG / 16>());
    else
        count(sh.tops + (tid & 1) * (kWG / 4), std::integral_constant<int, kWG / 4>());
    reached += __shfl_xor(reached, 1);
    if (quads) reached += __shfl_xor(reached, 2);
    const float low = wave_max(reached >= a.n ? best : neg_inf());
    if (lane == 0) sh.wlow[wave] = low;
    __syncthreads();
    if (tid == 0) {
        double t = 0;
        for (int w = 0; w < kWG / 64; ++w) t += sh.wsum[w];
        put(a.rowstat + 2 * row, (double)mx);
        put(a.rowstat + 2 * row + 1, mx == neg_inf() ? 0. : log(t));
    }

    // The tiles that reach the bound are listed, all at once where the list holds them,
    // else those of one round q at a time; each listed tile's eight vectors go to eight
    // threads. Keys from the bound's value on go to the buffer; when they would not fit,
    // it is cut back to its n best, which raises the bound.
    float bound = -kMaxF;  // (every element that is not masked, where fewer than n groups hold one)
#pragma unroll
    for (int w = 0; w < kWG / 64; ++w) bound = fmaxf(bound, sh.wlow[w]);
    uint64_t T0 = (uint64_t)qg_ord(bound) << 32;
    uint64_t marked = 0;
#pragma unroll
    for (int q = 0; q < kMine; ++q) marked |= (uint64_t)(tv[q] >= bound) << q;
    const int mine_t = __builtin_popcountll(marked);
    int at = mine_t ? atomicAdd(&sh.listed, mine_t) : 0;
    __syncthreads();
    const int reach = sh.listed;
    const bool whole = reach <= kList;
    for (int turn = 0; turn < (whole ? 1 : kMine); ++turn) {
        if (!whole) {
            __syncthreads();
            if (tid == 0) sh.listed = 0;
            __syncthreads();
        }
        uint64_t now = whole ? marked : marked & (1ull << turn);
        if (!whole && now) at = atomicAdd(&sh.listed, 1);
        while (now) {
            sh.list[at++] = tid + kWG * __builtin_ctzll(now);
            now &= now - 1;
        }
        __syncthreads();
        const int scanned = whole ? reach : sh.listed;
        for (int v0 = 0; v0 < scanned * 8; v0 += kWG) {
            const int o = v0 + tid;
            float v[N];
            uint64_t key[N];
            int mine = 0;
            const bool on = o < scanned * 8;
            int i = 0;
            if (on) {
                const int t = sh.list[o >> 3], part = o & 7;
                const int seg = t / (64 / L), l = t % (64 / L) * L + part % L;
                i = seg * SV * 64 + part / L * 64 + l;
            }
            if (on) r.load(i, v);
#pragma unroll
            for (int e = 0; e < N; ++e) {
                key[e] = on ? key_of(v[e], i * N + e) : 0;
                mine += key[e] >= T0;
            }
            if (tid == 0) sh.more = 0;
            __syncthreads();
            if (mine) atomicAdd(&sh.more, mine);
            __syncthreads();
            if (sh.count + sh.more <= kBuf) {
                __syncthreads();
#pragma unroll
                for (int e = 0; e < N; ++e)
                    if (key[e] >= T0) sh.buf[atomicAdd(&sh.count, 1)] = key[e];
                __syncthreads();
            } else {  // one element of every thread at a time
#pragma unroll 1
                for (int e = 0; e < N; ++e) {
                    uint64_t k = key[0];
#pragma unroll
                    for (int d = 1; d < N; ++d) k = d == e ? key[d] : k;
                    const int c = sh.count;
                    __syncthreads();
                    if (c + kWG > kBuf) {
                        const int left = rank_buf(sh, c, a.n);
                        if (left == a.n) T0 = sh.buf[a.n - 1];
                        if (tid == 0) sh.count = left;
                        __syncthreads();
                    }
                    if (k && k >= T0) sh.buf[atomicAdd(&sh.count, 1)] = k;
                    __syncthreads();
                }
            }
        }
        __syncthreads();
    }
    const int c = rank_buf(sh, sh.count, a.n);
    for (int i = tid; i < a.n; i += kWG) put(a.rowkey + row * a.n + i, i < c ? sh.buf[i] : (uint64_t)0);
}

struct ItemShared {
    double rank[QG_BEAM_MAX * QG_BEAM_MAX_SELECT];  // of candidate i = beam * n + place in the beam
    uint64_t key[QG_BEAM_MAX * QG_BEAM_MAX_SELECT];
    double over[QG_BEAM_MAX];                       // len^alpha
    double2 stat[QG_BEAM_MAX];
    float cum[QG_BEAM_MAX];
    int len[QG_BEAM_MAX];
    bool done[QG_BEAM_MAX];
    int place[QG_BEAM_MAX_SELECT];
    int list[QG_BEAM_MAX * QG_BEAM_MAX_SELECT];
    double head[2 * QG_BEAM_MAX_SELECT + QG_BEAM_MAX];
    double bound;
    int kept;
};
struct Beam {  // of thread `beam`, read before the workgroup is counted
    float cum;
    int len;
    bool done;
    double over;  // len^alpha
};

// An item's n best over its beams' n best. Order: rank descending, then i ascending.
QG_DEV void rank_item(const BArgs& a, int64_t item, const Beam& beam, ItemShared& sh) {
    const int tid = threadIdx.x;
    const int total = a.beams * a.n;
    const double ninf = -__builtin_huge_val();
    for (int i = tid; i < total; i += kWG) sh.key[i] = take(a.rowkey + item * total + i);
    if (tid < a.n) sh.place[tid] = -1;
    if (tid < a.beams) {
        const int64_t row = item * a.beams + tid;
        const double2 st = beam.done ? make_double2(0., 0.) : make_double2(take(a.rowstat + 2 * row), take(a.rowstat + 2 * row + 1));
        sh.cum[tid] = beam.cum;
        sh.done[tid] = beam.done;
        sh.len[tid] = beam.len;
        sh.over[tid] = beam.over;
        sh.stat[tid] = st;
    }
    __syncthreads();
    auto candidate = [&](int i, int& token) -> double {
        const int w = i / a.n;
        const float cum = sh.cum[w];
        token = -1;
        if (cum != cum || cum == neg_inf()) return ninf;
        if (sh.done[w]) {
            if (i != w * a.n) return ninf;
            token = a.eos;
            return cum;
        }
        const uint64_t k = sh.key[i];
        if (!k) return ninf;
        token = key_token(k);
        return (double)cum + (((double)key_value(k) - sh.stat[w].x) - sh.stat[w].y);
    };
    for (int i = tid; i < total; i += kWG) {
        int token;
        const double sc = candidate(i, token);
        sh.rank[i] = a.alpha != 0. && token >= 0 ? sc / sh.over[i / a.n] : sc;
    }
    __syncthreads();
    // Four threads compare a candidate with the others. With many candidates only those
    // that reach a bound are compared: the n-th best of the beams' first few (2 n of them
    // or a few more). A call of 16 beams with n = 16 takes 28 us if all are compared, 21
    // with the bound; of 8 beams 17.6 and 16.3; up to 64 candidates, one each for every
    // four threads, the bound costs 0.4 us (8 beams with n = 8: 15.1 and 15.5).
    auto place = [&](int c, auto listed) {
        for (int j0 = 0; j0 < c; j0 += kWG / 4) {
            const int j = j0 + (tid >> 2);
            const int i = j < c ? (listed ? sh.list[j] : j) : 0;
            const double k = sh.rank[i];
            int before = 0;
#pragma unroll 4
            for (int l = tid & 3; l < c; l += 4) {
                const int o = listed ? sh.list[l] : l;
                const double r = sh.rank[o];
                before += (int)(r > k) | ((int)(r == k) & (int)(o < i));
            }
            before += __shfl_xor(before, 1);
            before += __shfl_xor(before, 2);
            if (j < c && k != ninf && before < a.n && !(tid & 3)) sh.place[before] = i;
        }
    };
    if (total <= kWG / 4) {
        place(total, std::false_type());
    } else {
        const int heads = min(a.n, (2 * a.n + a.beams - 1) / a.beams);
        const int of = a.beams * heads;  // <= 2 n + beams <= 160
        if (tid == 0) {
            sh.bound = ninf;
            sh.kept = 0;
        }
        __syncthreads();
        if (tid < of) sh.head[tid] = sh.rank[tid / heads * a.n + tid % heads];
        __syncthreads();
        for (int j0 = 0; j0 < of; j0 += kWG / 4) {
            const int j = min(j0 + (tid >> 2), of - 1);
            const double k = sh.head[j];
            int above = 0, reach = 0;
#pragma unroll 4
            for (int o = tid & 3; o < of; o += 4) {
                const double r = sh.head[o];
                above += r > k;
                reach += r >= k;
            }
            above += __shfl_xor(above, 1), reach += __shfl_xor(reach, 1);
            above += __shfl_xor(above, 2), reach += __shfl_xor(reach, 2);
            if (above < a.n && reach >= a.n) sh.bound = k;  // (all threads that write it hold the same)
        }
        __syncthreads();
        const double bound = sh.bound;
        for (int i = tid; i < total; i += kWG)
            if (sh.rank[i] >= bound && sh.rank[i] > ninf) sh.list[atomicAdd(&sh.kept, 1)] = i;
        __syncthreads();
        place(sh.kept, std::true_type());
    }
    __syncthreads();
    if (tid < a.n) {
        const int i = sh.place[tid];
        int token = -1, w = -1;
        double sc = ninf;
        if (i >= 0) {
            sc = candidate(i, token);
            w = i / a.n;
        }
        const int64_t o = item * a.n + tid;
        a.out.token[o] = token;
        a.out.parent[o] = w;
        a.out.score[o] = (float)sc;
        if (a.out.finished) a.out.finished[o] = w >= 0 && (sh.done[max(w, 0)] || (a.eos >= 0 && token == a.eos));
        if (a.out.length) a.out.length[o] = w >= 0 ? sh.len[max(w, 0)] : 0;
    }
}

// Bound by latency: 9.6 us for 4 rows of 152064 fp32 and n = 8, of them about 1 us each for
// reading the tile maxima, for the bound, for the listed tiles' elements and for the
// candidates of the other rows, under 1 us for each ranking and for the arrival.
template <int XT, int SV>
__global__ __launch_bounds__(kWG) void beam_rank_kernel(BArgs a) {
    __shared__ union {
        RowShared row;
        ItemShared item;
    } sh;
    __shared__ bool last;
    const int64_t row = blockIdx.x;
    const int64_t item = row / a.beams;
    // The item's inputs, which its outputs may replace: read by every one of its
    // workgroups before it is counted, while only the last one counted writes.
    Beam beam{0.f, 0, false, 1.};
    if ((int)threadIdx.x < a.beams) {
        const int64_t b = item * a.beams + threadIdx.x;
        beam.done = a.finished && a.finished[b];
        beam.cum = a.score[b];
        beam.len = (a.length ? a.length[b] : 0) + (beam.done ? 0 : 1);
        if (a.alpha != 0.) beam.over = pow((double)max(beam.len, 1), a.alpha);
    }
    if (!(a.finished && a.finished[row])) rank_row<XT, SV>(a, row, sh.row);
    // The row's results are out (each wavefront waits for its stores before the barrier)
    // before it is counted; the item's last row sees the others' counts, hence their
    // results. No workgroup waits for another.
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();
    if (threadIdx.x == 0)
        last = __hip_atomic_fetch_add(a.arrived + item, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) ==
               (uint32_t)(a.beams - 1);
    __syncthreads();
    if (last) rank_item(a, item, beam, sh.item);
}

// ---------------------------------------------------------------- host
int vec_elems(int type) { return type == QG_F32 ? 4 : 8; }

struct Plan {
    int64_t rows;
    int sv, tiles, segs;
    size_t segmax, segsum, tmax, rowkey, rowstat, arrived, total;
};
Plan plan(int type, int64_t batch, int beams, int64_t vocab, int n) {
    Plan p;
    p.rows = batch * beams;
    const int64_t ve = vec_elems(type);
    const int64_t vecs = qg::ceil_div(vocab, ve);
    // Segments of four vectors a lane, or of two where four would leave most of the
    // chip without one.
    p.sv = p.rows * qg::ceil_div(vecs, 64 * 4) >= 2048 ? 4 : 2;
    p.segs = (int)qg::ceil_div(vecs, 64 * p.sv);
    p.tiles = p.segs * 8 * p.sv;
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t o = at;
        at = qg::align_up(at + bytes, 256);
        return o;
    };
    p.segmax = take((size_t)p.rows * p.segs * 4);
    p.segsum = take((size_t)p.rows * p.segs * 8);
    p.tmax = take((size_t)p.rows * p.tiles * 4);
    p.rowkey = take((size_t)p.rows * n * 8);
    p.rowstat = take((size_t)p.rows * 16);
    p.arrived = take((size_t)batch * 4);
    p.total = at;
    return p;
}

qg_status check_shape(int type, int64_t batch, int beams, int64_t vocab, int n) {
    if (type != QG_F32 && type != QG_F16 && type != QG_BF16)
        return qg::fail(QG_ERR_SHAPE, "logits_type=%d unknown", type);
    if (beams < 1 || beams > QG_BEAM_MAX) return qg::fail(QG_ERR_SHAPE, "beams=%d not in [1, %d]", beams, QG_BEAM_MAX);
    if (batch < 1 || batch > kMaxRows / beams)
        return qg::fail(QG_ERR_SHAPE, "batch=%lld below 1, or over 65536 rows", (long long)batch);
    if (vocab < 1 || vocab > QG_TOPK_MAX_ROWS)
        return qg::fail(QG_ERR_SHAPE, "vocab=%lld not in [1, %d]", (long long)vocab, QG_TOPK_MAX_ROWS);
    if (n < 1 || n > QG_BEAM_MAX_SELECT) return qg::fail(QG_ERR_SHAPE, "n=%d not in [1, %d]", n, QG_BEAM_MAX_SELECT);
    return QG_OK;
}

bool overlap(const void* a, size_t na, const void* b, size_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return a && b && x < y + nb && y < x + na;
}

template <int XT, int SV>
qg_status launch(const BArgs& a, hipStream_t s) {
    const int64_t waves = (int64_t)a.rows * a.segs;
    hipLaunchKernelGGL((beam_stats_kernel<XT, SV>), dim3((unsigned)qg::ceil_div(waves, kWG / 64)), dim3(kWG), 0, s, a);
    const qg_status st = qg::launch_status("logits_beam_select (statistics)");
    if (st) return st;
    hipLaunchKernelGGL((beam_rank_kernel<XT, SV>), dim3((unsigned)a.rows), dim3(kWG), 0, s, a);
    return qg::launch_status("logits_beam_select (ranking)");
}
template <int XT>
qg_status launch_for(const BArgs& a, int sv, hipStream_t s) {
    return sv == 4 ? launch<XT, 4>(a, s) : launch<XT, 2>(a, s);
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
    a.tmax = (float*)(w8 + p.tmax);
    a.rowkey = (uint64_t*)(w8 + p.rowkey);
    a.rowstat = (double*)(w8 + p.rowstat);
    a.arrived = (uint32_t*)(w8 + p.arrived);
    a.out = *out;
    hipStream_t s = (hipStream_t)stream;
    if (in->logits_type == QG_F32) return launch_for<QG_F32>(a, p.sv, s);
    if (in->logits_type == QG_F16) return launch_for<QG_F16>(a, p.sv, s);
    return launch_for<QG_BF16>(a, p.sv, s);
}

}  // extern "C"
