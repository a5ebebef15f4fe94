// Products on 8-bit floating-point (e4m3) weights and activations with block scales, for
// gfx950: the load-time layout of the weights, the row quantizer, the product and the
// product grouped by expert.
//
//   y[n, m] = sum_b x_scale[n, b] * w_scale[m / 128, b] * sum_{k in b} xq[n, k] * wq[m, k]  (+ bias[m])
//
// over blocks b of 128 values of K. A block is one matrix-core operand (16 x 16 x 128),
// whose sum is scaled once, by one multiply-add per output.
#include <algorithm>
#include <climits>
#include <type_traits>

#include "qg_device.h"
#include "qg_host.h"
#include "qg_rows.h"

namespace {

using namespace qg;

constexpr int T = QG_TILE_ROWS;
constexpr int kPair = 2 * T;  // weight rows of two operands, which share them in fours
constexpr int kB = QG_F8_BLOCK;
constexpr int kUnit = T * kB;  // bytes of one operand: 16 rows x 128 k

typedef int v8i __attribute__((ext_vector_type(8)));
typedef _Float16 h8 __attribute__((ext_vector_type(8)));

// ---------------------------------------------------------------- weight layout
// Operands in pairs of 32 weight rows: row r of operand i of a pair is the weight row 8 (r /
// 4) + 4 i + r % 4, so that a lane, which gets four rows of a product, gets eight
// consecutive ones of a pair's. Once per model; bound by memory (37888 x 3584: 43 us, 6.3 TB/s read and
// written; 128 x 1536 x 2048: 146 us, 5.5).
__global__ __launch_bounds__(256) void pack_f8_kernel(const uint8_t* __restrict__ src, int64_t ldw, int64_t w_expert,
                                                      uint4* __restrict__ dst, int64_t M, int K, int nb,
                                                      int64_t mtiles, int64_t units) {
    const int64_t stride = (int64_t)gridDim.x * 256;
    for (int64_t u = (int64_t)blockIdx.x * 256 + threadIdx.x; u < units; u += stride) {
        const int l = (int)(u & 63);
        const int64_t th = u >> 6;  // (expert, tile, half of a block)
        const int64_t t = th / (2 * nb), m = t % mtiles;
        const int64_t row = m / 2 * kPair + (l >> 2 & 3) * 8 + (m & 1) * 4 + (l & 3);
        const int k0 = (int)(th % (2 * nb)) * (kB / 2) + (l >> 4) * 16;
        union {
            uint4 v;
            uint8_t b[16];
        } o;
        o.v = make_uint4(0, 0, 0, 0);
        if (row < M) {
            typedef uint32_t vec __attribute__((ext_vector_type(4), aligned(1)));  // rows start anywhere
            const uint8_t* p = src + t / mtiles * w_expert + row * ldw + k0;
            if (k0 + 16 <= K) {
                const vec v = *reinterpret_cast<const vec*>(p);
                o.v = make_uint4(v.x, v.y, v.z, v.w);
            } else {
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    if (k0 + e < K) o.b[e] = p[e];
            }
        }
        dst[u] = o.v;
    }
}

// ---------------------------------------------------------------- row quantizer
// The largest of a value's 16 lanes, in all of them (DPP: within quads, then across them).
QG_DEV uint32_t row_max(uint32_t v) {
    v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xb1, 0xf, 0xf, true));   // quad_perm [1, 0, 3, 2]
    v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4e, 0xf, 0xf, true));   // quad_perm [2, 3, 0, 1]
    v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x141, 0xf, 0xf, true));  // row_half_mirror
    return max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x140, 0xf, 0xf, true));  // row_mirror
}

QG_DEV uint2 to_f8(const float (&t)[8]) {
    uint2 o;
    o.x = __builtin_amdgcn_cvt_pk_fp8_f32(t[0], t[1], 0, false);
    o.x = __builtin_amdgcn_cvt_pk_fp8_f32(t[2], t[3], o.x, true);
    o.y = __builtin_amdgcn_cvt_pk_fp8_f32(t[4], t[5], 0, false);
    o.y = __builtin_amdgcn_cvt_pk_fp8_f32(t[6], t[7], o.y, true);
    return o;
}

// Eight values divided by a d below 2^-90, as e4m3 bytes: in double precision the quotient of
// two floats is never rounded onto a border between two results that it does not meet. Three
// bits after the leading one from 2^-6 on, multiples of 2^-9 below, ties to even.
QG_DEV uint2 quant8_tiny(const float (&x)[8], float d) {
    float t[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const double v = (double)x[i] / (double)d, a = fabs(v);
        const int e = a < 0x1p-6 ? -6 : ilogb(a);
        t[i] = fminf(fmaxf((float)ldexp(rint(ldexp(v, 3 - e)), e - 3), -448.f), 448.f);  // (over it where d is subnormal)
    }
    return to_f8(t);
}

// Eight values divided by d, as e4m3 bytes, by x * inv with inv within a unit in the last place
// of 1/d. The product is off by three units at most; where it lies within four of a border
// (as bf16 values often do: in one block of seven the largest value is a multiple of 7, d a power of two
// times few bits), the remainder of that border, exact in one fused operation, says on which side the quotient lies.
QG_DEV uint2 quant8(const float (&x)[8], float d, float inv) {
    float t[8];
    auto shifted = [](float a) { return a < 0x1p-6f ? a + 0x1p-6f : a; };  // below 2^-6: the next octave's borders, shifted
    auto off = [](float b) { return (__builtin_bit_cast(uint32_t, b) + (4u - 0x80000u)) << 12; };  // from 4 below a border on
    uint32_t least = ~0u;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        t[e] = x[e] * inv;
        least = min(least, off(shifted(fabsf(t[e]))));
    }
    if (__ballot(least <= 8u << 12)) {
        asm volatile("");  // (a branch: without it both sides are computed and one is taken)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float a = fabsf(t[e]), b = shifted(a);
            const float at = __builtin_bit_cast(float, (__builtin_bit_cast(uint32_t, b) & 0xfff00000u) | 0x80000u);
            const float border = a < 0x1p-6f ? at - 0x1p-6f : at;
            const float rest = __builtin_fmaf(-border, d, fabsf(x[e]));
            const float side = rest > 0.f ? 0x1p-22f : rest < 0.f ? -0x1p-22f : 0.f;
            if (off(b) <= 8u << 12) t[e] = copysignf(__builtin_fmaf(border, side, border), t[e]);
        }
    }
    return to_f8(t);
}

// z / (1 + exp(-z)): the exponential by a power of two, whose argument's rounding error is
// added back; within a few units in the last place. For |z| below kFarGate: the exponential and
// 1 + it stay normal and the sum's reciprocal too (the hardware's is zero below 2^-126).
constexpr float kFarGate = 87.f;
QG_DEV float silu(float z) {
    const float p = z * -1.44269504f;
    const float e = __builtin_amdgcn_exp2f(p);
    const float low = __builtin_fmaf(z, -1.44269504f, -p) + z * -1.925963033e-8f;
    return z * __builtin_amdgcn_rcpf(1.f + __builtin_fmaf(e * 0.693147181f, low, e));
}
// The same for any z: from exponentials of 2^64 on with numerator and denominator times 2^-64,
// so that they last until the quotient itself is below the floats (z = -190 / log2(e)); below the normal
// floats it is rounded to their step. As the formula has it, zero beyond and NaN for -infinity.
QG_DEV float silu_far(float z) {
#pragma clang fp contract(off)  // (p - 64 is exact for the rounded p, whose error is what `low` adds)
    const float p = z * -1.44269504f;
    const float one = p > 64.f ? 0x1p-64f : 1.f, q = p > 64.f ? p - 64.f : p;
    const float e = __builtin_amdgcn_exp2f(q);
    // (where e is infinite or zero, its correction would not be a number)
    const float low = __builtin_fmaf(z, -1.925963033e-8f, __builtin_fmaf(z, -1.44269504f, -p));
    const float c = q < 128.f && q > -126.f ? __builtin_fmaf(e * 0.693147181f, low, e) : e;
    return z * __builtin_amdgcn_rcpf(one + c) * one;
}

struct QArgs {
    const void* x;
    int64_t ldx;
    const int32_t* count;  // rows to do, or NULL
    uint8_t* q;
    int64_t ldq;
    float* scale;
    int64_t lds;
    int32_t N, K;
    uint32_t quads;  // quads: groups of four blocks of a row
};

// A block's scale is d = max |x| / 448, its values are x / d rounded to e4m3, ties to even.
// Sixteen lanes per block, a wavefront per four blocks of a row: one pass, every value read
// once (four groups to a wavefront at a time, with their loads ahead, took 90 us for 4096 x
// 18944 gated bf16 where one took 84, and 4.9 for 64 x 3584 where it took 3.0). Bound by memory and by
// as many cycles of instructions: that gated case 71 to 73 us in a trace, up to 87 in a row of calls
// (390 MB, 4.5 to 5.5 TB/s), the plain one 59 us (235 MB, 4.0 TB/s) by the instructions.
template <int XT, bool GATED>
__global__ __launch_bounds__(256) void quantize_f8_kernel(QArgs a) {
    typedef typename XVec<XT>::E E;
    constexpr int VN = XVec<XT>::N, V = 8 / VN;  // vectors of a lane's eight values
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t rows = a.count ? min(max(*a.count, 0), a.N) : a.N;
    const uint32_t total = rows * a.quads;  // below 2^31
    for (uint32_t at = blockIdx.x * 4 + wave; at < total; at += gridDim.x * 4) {
        const uint32_t n = at / a.quads;
        const int b0 = (int)(at - n * a.quads) * 4, b = b0 + (lane >> 4), k = b0 * kB + lane * 8;
        const E* p = reinterpret_cast<const E*>(a.x) + n * a.ldx;
        uint4 v[V], g[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            v[i] = row_vec<XT>(GATED ? p + a.K : p, a.K, k / VN + i);
            if constexpr (GATED) g[i] = row_vec<XT>(p, a.K, k / VN + i);
        }
        float x[8], z[8];
        if constexpr (GATED) {
            float far = 0.f;  // (a NaN among the gates needs no care)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                z[e] = XVec<XT>::get(g[e / VN], e % VN);
                far = fmaxf(far, fabsf(z[e]));
            }
            if (__ballot(far >= kFarGate)) {
                asm volatile("");
#pragma unroll
                for (int e = 0; e < 8; ++e) z[e] = silu_far(z[e]);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) z[e] = silu(z[e]);
            }
        }
        uint32_t mx = 0;  // the largest |x| by its bits: above every finite value an infinity, above it a NaN
        if constexpr (!GATED && VN == 8) {
            // 16-bit values in pairs
            typedef uint16_t h2 __attribute__((ext_vector_type(2)));
            h2 m = {0, 0};
#pragma unroll
            for (int e = 0; e < 4; ++e) m = __builtin_elementwise_max(m, __builtin_bit_cast(h2, (&v[0].x)[e] & 0x7fff7fffu));
            const uint4 one = make_uint4(max(m[0], m[1]), 0, 0, 0);
            mx = __builtin_bit_cast(uint32_t, XVec<XT>::get(one, 0));
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            x[e] = XVec<XT>::get(v[e / VN], e % VN);
            if constexpr (GATED) x[e] *= z[e];
            if constexpr (GATED || VN == 4) mx = max(mx, __builtin_bit_cast(uint32_t, x[e]) & 0x7fffffffu);
        }
        mx = row_max(mx);
        const bool finite = mx < 0x7f800000u;
        const float top = __builtin_bit_cast(float, mx);
        // top / 448 rounded to nearest: the product with 1/448 and its exact remainder's correction
        const float q0 = top * (1.f / 448.f);
        float d = __builtin_fmaf(__builtin_fmaf(-448.f, q0, top), 1.f / 448.f, q0);
        if (!finite) d = __builtin_nanf("");
        uint2 o = quant8(x, d, __builtin_amdgcn_rcpf(d));
        const bool tiny = d < 0x1p-90f && top > 0.f;  // (the remainders could be subnormal, and 1/d infinite)
        if (__ballot(tiny)) {
            asm volatile("");
            if (tiny) {
                d = top / 448.f;
                o = quant8_tiny(x, d);
            }
        }
        if (!(d > 0.f)) o = make_uint2(0, 0);
        const bool in = b * kB < a.K;
        if (in) *reinterpret_cast<uint2*>(a.q + n * a.ldq + b * kB + (lane & 15) * 8) = o;
        if ((lane & 15) == 0) a.scale[n * a.lds + b] = in ? d : 0.f;
    }
}

// ---------------------------------------------------------------- product
struct GArgs {
    const uint8_t* w;
    const float* ws;
    const uint8_t* x;
    int64_t ldx;
    const float* xs;
    int64_t ldxs;
    const float* bias;
    void* Y;
    int64_t ldy;
    const int32_t* offsets;  // grouped: rows offsets[e] .. offsets[e + 1] of Y meet expert e
    const int32_t* row;      // grouped: rows of x that rows of Y come from, or NULL: the same
    qg_f4* part;             // partial sums of a product split along K
    int32_t M, N, X;         // N: rows of Y, X: rows of x
    int32_t E, nb, mb;       // experts, blocks of 128 along K and M
    int32_t mtiles;          // 16-row tiles of an expert's weights
    int32_t kper;            // blocks of a split
    int32_t total;           // tiles of Y
};

// Rows of Y that meet one expert.
struct Group {
    int e, r0, r1;
};

QG_DEV void group_range(const GArgs& a, int e, int& r0, int& r1) {
    r0 = r1 = 0;
    if (e < a.E) {
        r0 = min(max(a.offsets[e], 0), a.N);
        r1 = min(max(a.offsets[e + 1], r0), a.N);
    }
}

// The slot-th expert that has rows; false if there are fewer. By every wavefront alike.
QG_DEV bool used_group(const GArgs& a, int slot, Group& g) {
    const int lane = threadIdx.x & 63;
    for (int e0 = 0; e0 < a.E; e0 += 64) {
        int r0, r1;
        group_range(a, e0 + lane, r0, r1);
        const uint64_t used = __ballot(r1 > r0);
        const int before = __builtin_amdgcn_mbcnt_hi((uint32_t)(used >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)used, 0));
        const uint64_t hit = __ballot(r1 > r0 && before == slot);
        if (hit) {
            const int l = __builtin_ctzll(hit);
            g = {e0 + l, __builtin_amdgcn_readlane(r0, l), __builtin_amdgcn_readlane(r1, l)};
            return true;
        }
        slot -= __builtin_popcountll(used);
    }
    return false;
}

QG_DEV int source_row(const GArgs& a, int r) { return a.row ? min(max(a.row[r], 0), a.X - 1) : r; }

// Eight e4m3 values as fp16, exactly.
QG_DEV h8 to_half(uint32_t lo, uint32_t hi) {
    typedef _Float16 h2 __attribute__((ext_vector_type(2)));
    union {
        h2 p[4];
        h8 v;
    } o;
    o.p[0] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.f, false);
    o.p[1] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.f, true);
    o.p[2] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.f, false);
    o.p[3] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.f, true);
    return o.v;
}

// A 16 x 128 operand in a lane: row lane % 16, k = 16 (lane / 16) .. + 15 of each half.
union Op8 {
    v8i v;
    qi4 h[2];
};
struct Op16 {
    h8 v[4];
    QG_DEV void set(const Op8& o) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = to_half((uint32_t)o.v[2 * i], (uint32_t)o.v[2 * i + 1]);
    }
};
// The 16 x 16 sums of one block. On the 8-bit matrix cores, which align each eight
// products to the largest and keep 13 bits below its leading one (measured with single
// products: one of 2^-13 of the largest counts, of 2^-14 it does not), so that a block's
// sum is off by 1.5e-5 for normally distributed values: for outputs that are rounded to
// 2^-9 or 2^-12 in the end ...
QG_DEV qg_f4 block_sum(const Op8& a, const Op8& b) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a.v, b.v, qg_f4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0, 0, 0);
}
// ... and on the fp16 ones at half the rate, exactly but for the float32 additions.
QG_DEV qg_f4 block_sum(const Op16& a, const Op16& b) {
    qg_f4 s = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 4; ++i) s = __builtin_amdgcn_mfma_f32_16x16x32_f16(a.v[i], b.v[i], s, 0, 0, 0);
    return s;
}
QG_DEV void add_scaled(qg_f4& acc, const qg_f4& s, float scale) {
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[e] = __builtin_fmaf(s[e], scale, acc[e]);
}

// The biases of C consecutive weight rows from m on, rows beyond M repeating the last one.
template <int C>
QG_DEV void row_bias(const GArgs& a, int e, int m, float (&sb)[C]) {
#pragma unroll
    for (int i = 0; i < C; ++i) sb[i] = a.bias ? a.bias[(int64_t)e * a.M + min(m + i, a.M - 1)] : 0.f;
}

// ---------------------------------------------------------------- few rows
// One 16-row tile of an expert's weights and 16 rows of Y after the other per workgroup; its
// wavefronts take blocks of K in turn, and their sums meet in LDS, in order. The weights go
// from memory straight to registers, in the packed order, and are what bounds it: latency
// where they are few (4608 x 3584 by 1: 6.2 us, 16.5 MB in 3.5 at the copy's rate; 8 of 128 experts of
// 1536 x 2048, one token: 9.4 us, of which the offsets, the weights and the joining of sums are one
// round trip after the other), memory where they are many (152064 x 3584 by 1: 87 us, 6.3 TB/s).
// Products are exact on the fp16 cores, whose rate does not matter here.
constexpr int kStreamWaves = 8;
template <int YT>
__global__ __launch_bounds__(64 * kStreamWaves) void gemm_f8_stream_kernel(GArgs a) {
    constexpr int W = kStreamWaves;
    __shared__ qg_f4 part[W][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int t = blockIdx.x, slot = blockIdx.y;
    Group g = {0, 0, a.N};
    if (a.offsets && !used_group(a, slot, g)) return;
    const uint8_t* w = a.w + ((size_t)g.e * a.mtiles + t) * a.nb * kUnit + lane * 16;
    const float* ws = a.ws + ((size_t)g.e * a.mb + t * T / kB) * a.nb;
    for (int c0 = g.r0; c0 < g.r1; c0 += 16) {
        // (rows beyond the last repeat it; their sums are not stored)
        const int n = c0 + (lane & 15);
        const int64_t r = source_row(a, min(n, g.r1 - 1));
        const uint8_t* const xr = a.x + r * a.ldx + (lane >> 4) * 16;
        const float* const sr = a.xs + r * a.ldxs;
        qg_f4 acc = {0.f, 0.f, 0.f, 0.f};
        Op8 wv[2], xv[2];
        float sv[2];
        auto load = [&](int p, int b) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                wv[p].h[h] = __builtin_nontemporal_load(reinterpret_cast<const qi4*>(w + (size_t)b * kUnit + h * 1024));
                xv[p].h[h] = *reinterpret_cast<const qi4*>(xr + b * kB + h * 64);
            }
            sv[p] = sr[b] * ws[b];
        };
        auto mma = [&](int p) {
            Op16 wh, xh;
            wh.set(wv[p]);
            xh.set(xv[p]);
            add_scaled(acc, block_sum(wh, xh), sv[p]);
        };
        int b = wave;
        for (; b + W < a.nb; b += 2 * W) {
            load(0, b);
            load(1, b + W);
            mma(0);
            mma(1);
        }
        if (b < a.nb) {
            load(0, b);
            mma(0);
        }
        part[wave][lane] = acc;
        __syncthreads();
        if (wave == 0) {
            const int m = (t >> 1) * kPair + (lane >> 4) * 8 + (t & 1) * 4;
            qg_f4 s = part[0][lane];
#pragma unroll
            for (int k = 1; k < W; ++k) s += part[k][lane];
            if (n < g.r1 && m < a.M) {
                float sb[4], y[4];
                row_bias(a, g.e, m, sb);
#pragma unroll
                for (int e = 0; e < 4; ++e) y[e] = s[e] + sb[e];
                store_row<YT>(a.Y, n * a.ldy + m, y, a.M - m);
            }
        }
        __syncthreads();  // (the next rows' sums go to the same places)
    }
}

// ---------------------------------------------------------------- many rows
// Tiles of Y (Tile in qg_rows.h: a K tile of 128 bytes is one block), one after the other
// per workgroup. Beside a tile's stages LDS holds the row scales and the weight scales of
// GB blocks, in GS places. H: parts of a K tile that are loaded apart (of two, the first has
// half of each wavefront's weights and all activations).
template <int BM, int BN, int WM, int WN, int NS, int H_, int GB_, int GS_>
struct F8Tile : Tile<BM, BN, WM, WN, NS> {
    typedef Tile<BM, BN, WM, WN, NS> P;
    static constexpr int H = H_, GB = GB_, GS = GS_;
    static constexpr int SU = GB / 4 * BN / 64;         // 1 KB loads of the row scales of GB blocks
    static constexpr int MB = (BM + kB - 1) / kB;       // blocks of weight rows
    static constexpr int SB = SU * 1024 + MB * 256;     // bytes of all scales of GB blocks
    static constexpr int LDS = P::LDS + GS * SB;
    static_assert(SU <= P::W && GB <= 64, "a wavefront loads row scales and weight scales once");
    static constexpr int MH = P::MT / H, AH = P::AU / H;  // weight operands and loads of a part
    static constexpr int FIRST = AH + P::XU;            // loads of the first part
    static_assert(MH * H == P::MT && AH * H == P::AU, "parts of a K tile");
    static_assert(BM / WM <= kB && kB % (BM / WM) == 0 && BN % 64 == 0, "a wavefront's rows share a weight scale");
};

template <int N>
using number = std::integral_constant<int, N>;

// Outputs of a wavefront's accumulators: a lane's pair is eight consecutive outputs, four
// lanes' pairs are 32.
template <int YT, int CT>
QG_DEV void store_pair(const GArgs& a, const qg_f4 (&lo)[CT], const qg_f4 (&hi)[CT], const float (&sb)[8], int m, int n0,
                       int n1) {
    const int count = a.M - m;
    if (count <= 0) return;
#pragma unroll
    for (int j = 0; j < CT; ++j) {
        const int n = n0 + 16 * j;
        if (n < n1) {
            float y[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                y[e] = lo[j][e] + sb[e];
                y[4 + e] = hi[j][e] + sb[4 + e];
            }
            store_row<YT>(a.Y, n * a.ldy + m, y, count);
        }
    }
}

// The bound of a buffer's loads, whose offsets are 32 bits.
QG_DEV int buffer_bytes(int64_t n) { return (int)(uint32_t)min(n, (int64_t)0xffffffffll); }

// The same outputs in 16 bits for whole pairs, by as many stores whatever rows there are: a
// lane's row beyond the last one is out of the bounds of Yr, which begins at column m of row n0.
template <int YT, int CT>
QG_DEV void store_pair_counted(const __amdgpu_buffer_rsrc_t Yr, const qg_f4 (&lo)[CT], const qg_f4 (&hi)[CT],
                               const float (&sb)[8], uint32_t at, uint32_t step, int rows) {
#pragma unroll
    for (int j = 0; j < CT; ++j) {
        float y[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            y[e] = lo[j][e] + sb[e];
            y[4 + e] = hi[j][e] + sb[4 + e];
        }
        qg_u4v v;
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = pack2<YT>(y[2 * e], y[2 * e + 1]);
        __builtin_amdgcn_raw_buffer_store_b128(v, Yr, 16 * j < rows ? at + j * step : 0xfffffff0u, 0, 0);
    }
}

// A tile of Y: the expert, its first 16-row weight tile, first row and end of the expert's rows.
struct TileOf {
    int e, t0, n0, n1;
};

// What a grouped product's workgroups know of the experts, in LDS: how many tiles of BN
// rows come before each one's, and its first row.
struct Experts {
    int* all;    // tiles of all
    int* first;  // [experts rounded up to 64]
    int* from;   // [the same and one more]
    __host__ QG_DEV static int bytes(int E) { return (2 + 2 * ((E + 63) & ~63)) * 4; }
    QG_DEV Experts(uint8_t* lds, int E)
        : all(reinterpret_cast<int*>(lds)), first(all + 1), from(first + ((E + 63) & ~63)) {}
    // By one wavefront.
    template <int BN>
    QG_DEV void fill(const GArgs& a) {
        const int lane = threadIdx.x & 63;
        int sum = 0;
        for (int e0 = 0; e0 < a.E; e0 += 64) {
            int r0, r1;
            group_range(a, e0 + lane, r0, r1);
            const int n = (r1 - r0 + BN - 1) / BN;
            int upto = n;
#pragma unroll
            for (int m = 1; m < 64; m <<= 1) {
                const int v = __shfl_up(upto, m);
                if (lane >= m) upto += v;
            }
            first[e0 + lane] = sum + upto - n;
            from[e0 + lane] = r0;
            sum += __builtin_amdgcn_readlane(upto, 63);
        }
        if (lane == 0) {
            from[a.E] = min(max(a.offsets[a.E], 0), a.N);
            *all = sum;
        }
    }
    // Tile `id`: the experts in order, of each one's the tiles of a weight tile and 1024 rows together,
    // so that they read both from the L2 (4 experts of 3584 x 3584, 4096 rows each: 203 us, with all rows
    // together 213); the XCDs take contiguous runs. False beyond the last one.
    template <int BM, int BN>
    QG_DEV bool tile(const GArgs& a, int id, TileOf& o) const {
        const int lane = threadIdx.x & 63;
        const int mts = (a.mtiles * 16 + BM - 1) / BM;
        const int total = __builtin_amdgcn_readfirstlane(*all) * mts, q = total / 8, r = total % 8, x = id % 8;
        if (id / 8 >= q + (x < r)) return false;
        id = x * q + min(x, r) + id / 8;
        const int at = id / mts;
        // the last expert whose first tile is not beyond this one (it has rows: one without would
        // share its first tile with the next)
        int e = -1;
        for (int e0 = 0; e0 < a.E; e0 += 64) {
            const int c = __builtin_popcountll(__ballot(e0 + lane < a.E && first[e0 + lane] <= at));
            e += c;
            if (c < 64) break;
        }
        const int r0 = __builtin_amdgcn_readfirstlane(from[e]);
        o.e = e;
        o.n1 = max(r0, __builtin_amdgcn_readfirstlane(from[e + 1]));
        constexpr int C = 1024 / BN;  // tiles of rows
        int n = id - __builtin_amdgcn_readfirstlane(first[e]) * mts;
        const int nts = (o.n1 - r0 + BN - 1) / BN, c = n / (C * mts) * C, w = min(C, nts - c);
        n -= c * mts;
        const int m = n / w;
        o.t0 = m * (BM / 16);
        o.n0 = r0 + (c + n - m * w) * BN;
        return true;
    }
};

// A wavefront's loads of a tile's stages and scales. What lies beyond the operands is out
// of its buffer's bounds and reads as zeros (and its sums are not stored). Weights arrive in
// the packed order. Activations: eight lanes per row of 128 bytes, the 16-byte chunk c of row
// r at place c ^ (r % 8), which spreads the operand reads over the banks.
template <class G, int BM, int BN, bool GROUPED>
struct Loads {
    const GArgs& a;
    uint8_t* const lds;
    const int lane, wave, mine;  // mine: the block of weight rows whose scales this wavefront takes
    const uint8_t* xp;
    int xbytes;
    __amdgpu_buffer_rsrc_t sr, vr;
    uint32_t woff[G::AU], xoff[G::XU], soff;

    QG_DEV Loads(const GArgs& args, uint8_t* l, int ln, int wv, int block) : a(args), lds(l), lane(ln), wave(wv), mine(block) {
#pragma unroll
        for (int u = 0; u < G::AU; ++u) woff[u] = (uint32_t)(unit_of(u) >> 1) * (uint32_t)a.nb * kUnit + lane * 16u;
        rows([](int c) { return (uint32_t)c; });
    }
    QG_DEV bool gathers() const { return GROUPED && a.row; }
    // 1 KB of weights in a stage that load u brings: the operands of the first part of every
    // wavefront's rows come first.
    QG_DEV int unit_of(int u) const {
        const int h = u / G::AH, g = wave * G::AH + u % G::AH, o = g >> 1;
        return (o / G::MH * G::MT + h * G::MH + o % G::MH) * 2 + (g & 1);
    }
    // from(c): the row of x that column c of the tile comes from, counted from the first one of xp.
    template <class F>
    QG_DEV void rows(F&& from) {
#pragma unroll
        for (int u = 0; u < G::XU; ++u)
            xoff[u] = from((wave * G::XU + u) * 8 + (lane >> 3)) * (uint32_t)a.ldx + ((lane & 7) ^ (lane >> 3)) * 16u;
        soff = from(wave % (BN / 64) * 64 + lane) * (uint32_t)a.ldxs * 4u;
    }
    QG_DEV const uint8_t* weights(const TileOf& o) const { return a.w + ((size_t)o.e * a.mtiles + o.t0) * a.nb * kUnit; }
    QG_DEV int weight_bytes(const TileOf& o) const { return buffer_bytes((int64_t)(a.mtiles - o.t0) * a.nb * kUnit); }
    // The activations and scales of tile o.
    QG_DEV void aim(const TileOf& o) {
        const int64_t base = gathers() ? 0 : o.n0, rows = gathers() ? a.X : o.n1 - o.n0;
        xp = a.x + base * a.ldx;
        xbytes = buffer_bytes((rows - 1) * a.ldx + a.nb * kB);
        sr = __builtin_amdgcn_make_buffer_rsrc((void*)(a.xs + base * a.ldxs), (short)0,
                                               buffer_bytes(((rows - 1) * a.ldxs + ((a.nb + 3) & ~3)) * 4), kQgRawBufferFlags);
        const int block = min(o.t0 * T / kB + mine, a.mb - 1);
        vr = __builtin_amdgcn_make_buffer_rsrc((void*)(a.ws + ((size_t)o.e * a.mb + block) * a.nb), (short)0, a.nb * 4,
                                               kQgRawBufferFlags);
    }
    // Load u of a part of K tile t to the stage in buffer buf: the part's weights first.
    QG_DEV void fetch(const uint8_t* wp, int wbytes, int xbytes, int t, int buf, int part, int u) const {
        uint8_t* A = lds + buf * G::STAGE;
        if (u < G::AH) {
            const int v = part * G::AH + u;
            const __amdgpu_buffer_rsrc_t wr = __builtin_amdgcn_make_buffer_rsrc((void*)wp, (short)0, wbytes, kQgRawBufferFlags);
            lds_load(wr, A + unit_of(v) * 1024, woff[v], (2 * t + (unit_of(v) & 1)) * 1024);
        } else {
            const __amdgpu_buffer_rsrc_t xr = __builtin_amdgcn_make_buffer_rsrc((void*)xp, (short)0, xbytes, kQgRawBufferFlags);
            lds_load(xr, A + G::AB + (wave * G::XU + u - G::AH) * 1024, xoff[u - G::AH], t * kB);
        }
    }
    // Scales of the blocks GB g .. + GB - 1: the row scales four blocks to a load, and the
    // weight scales (wavefronts of one block of rows alike).
    QG_DEV uint8_t* scales(int place) const { return lds + G::P::LDS + place * G::SB; }
    QG_DEV void fetch_scales(int g, int place) const {
        uint8_t* S = scales(place);
        if (wave < G::SU)
            lds_load(sr, S + wave * 1024, soff, min(g * (G::GB / 4) + wave / (BN / 64), (a.nb - 1) >> 2) * 16);
        __builtin_amdgcn_raw_ptr_buffer_load_lds(vr, (lds_ptr)(S + G::SU * 1024 + mine * 256), 4, (lane & (G::GB - 1)) * 4,
                                                 g * G::GB * 4, 0, 0);
    }
};

// A wavefront's reads from LDS, of one of its operands or scales.
template <class G, int BN>
struct Reads {
    const uint8_t* const lds;
    int arow, x0, x1, srow, wrow;
    QG_DEV Reads(const uint8_t* l, int lane, int wm, int wn, int mine) : lds(l) {
        const int r = lane & 15, q = lane >> 4, xrow = G::AB + (wn * G::CT * 16 + r) * 128;
        arow = wm * G::MT * kUnit + lane * 16;
        x0 = xrow + ((q ^ (r & 7)) * 16);
        x1 = xrow + (((4 + q) ^ (r & 7)) * 16);
        srow = (wn * G::CT * 16 + r) * 16;
        wrow = G::SU * 1024 + mine * 256;
    }
    QG_DEV void row(Op8& o, int buf, int i) const {
        const uint8_t* A = lds + buf * G::STAGE + arow + i * kUnit;
        o.h[0] = *reinterpret_cast<const qi4*>(A);
        o.h[1] = *reinterpret_cast<const qi4*>(A + 1024);
    }
    QG_DEV void col(Op8& o, int buf, int j) const {
        const uint8_t* X = lds + buf * G::STAGE + j * 2048;
        o.h[0] = *reinterpret_cast<const qi4*>(X + x0);
        o.h[1] = *reinterpret_cast<const qi4*>(X + x1);
    }
    QG_DEV void scales(float (&x)[G::CT], float& w, const uint8_t* S, int t) const {
        const uint8_t* X = S + ((t >> 2) & (G::GB / 4 - 1)) * (BN * 16) + srow + (t & 3) * 4;
#pragma unroll
        for (int j = 0; j < G::CT; ++j) x[j] = *reinterpret_cast<const float*>(X + j * 256);
        w = *reinterpret_cast<const float*>(S + wrow + (t & (G::GB - 1)) * 4);
    }
};

// float32 outputs take the exact block sums, 16-bit ones the faster 8-bit matrix cores.
template <int YT>
using Operand = typename std::conditional<YT == QG_F32, Op16, Op8>::type;
template <int YT>
QG_DEV Operand<YT> operand(const Op8& o) {
    Operand<YT> v;
    if constexpr (YT == QG_F32)
        v.set(o);
    else
        v = o;
    return v;
}

// Tiles of up to 128, several workgroups to a compute unit, whose starts and ends overlap. A K
// tile's products run between the loads of the one NS - 1 ahead; a pair of weight operands is
// read from LDS while the one before is multiplied. Few rows to an expert are bound by
// memory (128 experts of 2048 x 768, 8 to each of 256 tokens: 44 us, 201 MB of weights at 4.6
// TB/s), few tiles by the latency of their K tiles (4608 x 3584 by 32: 11.0 us).
template <int YT, int BM, int BN, int WM, int WN, int NS, bool SPLIT, bool GROUPED>
__global__ __launch_bounds__(64 * WM * WN) void gemm_f8_tile_kernel(GArgs a) {
    typedef F8Tile<BM, BN, WM, WN, NS, 1, 8, 2> G;
    constexpr int NP = G::MT / 2;  // pairs of weight operands
    static_assert(NP % 2 == 0, "the pairs alternate between two sets of registers");
    extern __shared__ __align__(1024) uint8_t lds[];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave % WM, wn = wave / WM, mine = wm * (BM / WM) / kB;
    const int k0 = SPLIT ? blockIdx.y * a.kper : 0;
    const int k1 = SPLIT ? min(a.nb, k0 + a.kper) : a.nb;
    Experts ex(lds + G::LDS, a.E);
    if constexpr (GROUPED) {
        if (wave == 0) ex.fill<BN>(a);
        __syncthreads();
    }
    Loads<G, BM, BN, GROUPED> L(a, lds, lane, wave, mine);
    const Reads<G, BN> R(lds, lane, wm, wn, mine);
    TileOf at{};
    const uint8_t* wp;
    int wbytes;
    auto aim = [&](int id) {
        if (id >= a.total) return false;
        if constexpr (GROUPED) {
            if (!ex.tile<BM, BN>(a, id, at)) return false;
            if (a.row) L.rows([&](int c) { return (uint32_t)source_row(a, min(at.n0 + c, at.n1 - 1)); });
        } else {
            const TileAt o = tile_at<BM, BN>(a.mtiles, a.N, id);
            at = {0, o.t0, o.n0, a.N};
        }
        L.aim(at);
        wp = L.weights(at);
        wbytes = L.weight_bytes(at);
        return true;
    };
    // A share of K tile t's loads. Beyond the last one they are out of bounds and read nothing,
    // so that the loop needs no branch.
    constexpr int U = G::AU + G::XU;
    auto fetch = [&](int t, int buf, int part, int parts) {
#pragma unroll
        for (int u = part * U / parts; u < (part + 1) * U / parts; ++u)
            L.fetch(wp, t < k1 ? wbytes : 0, t < k1 ? L.xbytes : 0, t, buf, 0, u);
    };
    auto start = [&]() {
#pragma unroll
        for (int i = 0; i < NS; ++i) {
            if (i == 0 || (((k0 + i) & 7) == 0 && k0 + i < k1)) L.fetch_scales((k0 + i) >> 3, (k0 + i) >> 3 & 1);
            fetch(k0 + i, i, 0, 1);
        }
    };

    // A tile's products run pair by pair of weight operands, each pair over the columns, and
    // the sums of a step are scaled and added during the next one. The operands of a pair are
    // read during the pair before; before the last pair, whose operands are then in registers,
    // a barrier: the tile's buffer can be refilled, with the tile NS later, and the next tile
    // has arrived, whose operands and scales are read as the last pair frees their registers.
    typedef Operand<YT> Op;
    Op8 fa[2][2], fx[G::CT];
    float xs[G::CT], w, sx[G::CT], before;
    qg_f4 acc[G::MT][G::CT], sum[2];
    auto tile = [&](auto last, int t, int buf, int nbuf) {
        constexpr bool LAST = decltype(last)::value;
        Op cx[G::CT];
#pragma unroll
        for (int j = 0; j < G::CT; ++j) {
            sx[j] = xs[j] * w;
            if constexpr (YT == QG_F32) cx[j] = operand<YT>(fx[j]);
        }
#pragma unroll
        for (int p = 0; p < NP; ++p) {
            if (p == NP - 1 && !LAST) {
                tile_sync<(NS - 2) * U>();
                __builtin_amdgcn_sched_barrier(0);
            }
            const Op ca[2] = {operand<YT>(fa[p & 1][0]), operand<YT>(fa[p & 1][1])};
#pragma unroll
            for (int j = 0; j < G::CT; ++j) {
                qg_f4 now[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    if constexpr (YT == QG_F32)
                        now[i] = block_sum(ca[i], cx[j]);
                    else
                        now[i] = block_sum(ca[i], fx[j]);
                }
                // the step before
                const int pj = j ? j - 1 : G::CT - 1, pp = j ? p : p ? p - 1 : NP - 1;
                const float s = j || p ? sx[pj] : before;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    add_scaled(acc[2 * pp + i][pj], sum[i], s);
                    // (left free, the last tile's additions move behind it and its sums to scratch memory)
                    if constexpr (LAST) asm volatile("" : "+v"(acc[2 * pp + i][pj]));
                    sum[i] = now[i];
                }
                if (p + 1 < NP) {
                    if (j == 0)
#pragma unroll
                        for (int i = 0; i < 2; ++i) R.row(fa[(p + 1) & 1][i], buf, 2 * p + 2 + i);
                } else if constexpr (!LAST) {
                    if (j == 0) {
                        R.scales(xs, w, L.scales((t + 1) >> 3 & 1), t + 1);
#pragma unroll
                        for (int i = 0; i < 2; ++i) R.row(fa[0][i], nbuf, i);
                    }
                    R.col(fx[j], nbuf, j);
                    fetch(t + NS, buf, j, G::CT);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        before = sx[G::CT - 1];
    };
    int id = blockIdx.x;
    if (!aim(id)) return;
    start();
    while (true) {
#pragma unroll
        for (int i = 0; i < G::MT; ++i)
#pragma unroll
            for (int j = 0; j < G::CT; ++j) acc[i][j] = qg_f4{0.f, 0.f, 0.f, 0.f};
        sum[0] = sum[1] = qg_f4{0.f, 0.f, 0.f, 0.f};
        before = 0.f;
        tile_sync<(NS - 1) * U>();
        R.scales(xs, w, L.scales(k0 >> 3 & 1), k0);
#pragma unroll
        for (int i = 0; i < 2; ++i) R.row(fa[0][i], 0, i);
#pragma unroll
        for (int j = 0; j < G::CT; ++j) R.col(fx[j], 0, j);
        int t = k0, buf = 0;
        for (; t + 1 < k1; ++t) {
            const int nbuf = buf + 1 == NS ? 0 : buf + 1;
            if (((t + NS) & 7) == 0 && t + NS < k1) L.fetch_scales((t + NS) >> 3, (t + NS) >> 3 & 1);
            tile(std::false_type{}, t, buf, nbuf);
            buf = nbuf;
        }
        tile(std::true_type{}, t, buf, buf);
#pragma unroll
        for (int i = 0; i < 2; ++i) add_scaled(acc[G::MT - 2 + i][G::CT - 1], sum[i], before);
        const int m0 = (at.t0 + wm * G::MT) * 16 + (lane >> 4) * 8, c0 = at.n0 + wn * G::CT * 16 + (lane & 15);
        if constexpr (SPLIT) {
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // (loads beyond the last tile)
            qg_f4* p = a.part + ((((size_t)blockIdx.y * gridDim.x + blockIdx.x) * G::W + wave) * (G::MT * G::CT)) * 64 + lane;
#pragma unroll
            for (int i = 0; i < G::MT; ++i)
#pragma unroll
                for (int j = 0; j < G::CT; ++j) p[(i * G::CT + j) * 64] = acc[i][j];
            return;
        } else {
            // A workgroup with another tile to do sends that tile's first loads before it
            // stores this one's outputs. (The biases have arrived before: a wait for them in the
            // next tile would be one for its loads.)
            float sb[NP][8];
#pragma unroll
            for (int c = 0; c < NP; ++c) {
                row_bias(a, at.e, m0 + 32 * c, sb[c]);
#pragma unroll
                for (int i = 0; i < 8; ++i) asm volatile("" : "+v"(sb[c][i]));
            }
            const int rows = at.n1;
            id += gridDim.x;
            tile_sync<0>();  // the last tile's buffer has been read by all (and loads beyond it are done)
            const bool more = aim(id);
            if (more) start();
#pragma unroll
            for (int c = 0; c < NP; ++c)
                store_pair<YT, G::CT>(a, acc[2 * c], acc[2 * c + 1], sb[c], m0 + 32 * c, c0, rows);
            if (!more) return;
        }
    }
}

// Large tiles, one workgroup of eight wavefronts to a compute unit, for K of some blocks.
// The wavefronts work in two groups of four, one of each on every SIMD, that take turns: while
// one multiplies a part of a K tile (its operands are in registers, but for the last few,
// which are on their way), the other reads the operands of its next part from LDS. A barrier
// ends each turn; the second group is a turn behind. So turn 2 H t + 2 h of the first group
// reads part h of K tile t, the next one multiplies it, and the second group's are one later.
// A part's place in its buffer is free when the second group has multiplied it. The next
// loads to it go between the products of the first group one turn later, of the second two.
// They have to be there before the first group's turn that reads them: at the end of a turn
// before one, the first group has just multiplied and the second read, and each lets only the
// loads sent after those be on their way.
// The loads run on into the workgroup's next tile. A tile's outputs are stored between its last
// turn and the next one's first, in a known number of stores, so that waits for loads sent
// before them can leave them on their way; where the last columns of Y make that number
// unknown, the loads come first.
// Bound by the reads that the L1 has on their way, about 64 lines at a time: 9 TB/s over the card
// at the L2's latency. So tiles of 256 beat 256 x 128 where they fit (37888 x 3584 by 4096: 492 to 529 us
// on several cards, 2100 to 2260 TFLOP/s, matrix cores busy 58% of the cycles). Experts whose rows are
// few and uneven are where this costs most: 32768 rows over 128 experts of 1536 x 2048, 256 in the
// mean and from 2 to 1400, are 1920 tiles of 256 x 128, a quarter of their rows padding, and 1.5 GB
// (163 to 171 us, busy 40%; memory alone 82 us). In tiles of 256 they are 1.25 GB but 55% more rows than there are.
constexpr int kTurnsBlocks = 4;     // the least blocks of K: the next tile's rows are known after two
constexpr int kTurnsExperts = 512;  // the most experts that leave room in LDS
template <int YT, int BM, int BN, int WM, int WN, int NS, int H, bool GROUPED>
__global__ __launch_bounds__(64 * WM * WN) void gemm_f8_turns_kernel(GArgs a) {
    typedef F8Tile<BM, BN, WM, WN, NS, H, 4, 3> G;  // (scales: see the places below)
    static_assert(G::W == 8 && ((H == 1 && NS == 3) || (H == 2 && NS == 2)), "two groups; the waits below");
    constexpr int AHEAD = 2;  // K tiles from the one that is multiplied to the one whose first part is loaded
    static_assert(AHEAD == NS - 2 + H && kTurnsBlocks >= AHEAD + 2, "the next tile's rows are there when its loads begin");
    extern __shared__ __align__(1024) uint8_t lds[];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave % WM, wn = wave / WM, mine = wm * (BM / WM) / kB;
    Experts ex(lds + G::LDS, a.E);
    int* const next_rows = reinterpret_cast<int*>(lds + G::LDS + Experts::bytes(a.E));
    if constexpr (GROUPED) {
        if (wave == 0) ex.fill<BN>(a);
        __syncthreads();
    }
    Loads<G, BM, BN, GROUPED> L(a, lds, lane, wave, mine);
    const Reads<G, BN> R(lds, lane, wm, wn, mine);
    int id = blockIdx.x;
    auto tile_of = [&](TileOf& o) {
        if (id >= a.total) return false;
        if constexpr (GROUPED) return ex.tile<BM, BN>(a, id, o);
        const TileAt d = tile_at<BM, BN>(a.mtiles, a.N, id);
        o = {0, d.t0, d.n0, a.N};
        return true;
    };
    TileOf at{}, next{};
    bool more = false;
    if (!tile_of(at)) return;
    L.aim(at);
    if (L.gathers()) L.rows([&](int c) { return (uint32_t)source_row(a, min(at.n0 + c, at.n1 - 1)); });
    const int nb = a.nb;
    const uint8_t *wp = L.weights(at), *wnext = wp;
    int wbytes = L.weight_bytes(at), nbytes = 0;
    // Load u of a part of K tile t, from nb on of the next tile (without one, nothing is read).
    auto fetch = [&](int t, int buf, int part, int u) {
        const bool on = t >= nb;
        L.fetch(on ? wnext : wp, on ? nbytes : wbytes, L.xbytes, on ? t - nb : t, buf, part, u);
    };
    L.fetch_scales(0, 0);
#pragma unroll
    for (int i = 0; i < AHEAD; ++i)
#pragma unroll
        for (int h = 0; h < H; ++h)
            if (h == 0 || i < NS - 1)
#pragma unroll
                for (int u = 0; u < (h ? G::AH : G::FIRST); ++u) fetch(i, i, h, u);

    constexpr int U = G::AU + G::XU, STORES = G::MT / 2 * G::CT;
    constexpr int LATE = G::MH >= 4 ? 4 : 0;  // reads that may be on their way when a part's products begin
    constexpr int PRODUCTS = G::MH * G::CT, D = PRODUCTS < 3 ? PRODUCTS : 3;  // D: products whose sums wait to be added
    typedef Operand<YT> Op;
    Op fa[G::MH], fx[G::CT];
    float sx[G::CT], xs[G::CT], w;
    qg_f4 acc[G::MT][G::CT], sum[D];
    auto clear = [&]() {
#pragma unroll
        for (int i = 0; i < G::MT; ++i)
#pragma unroll
            for (int j = 0; j < G::CT; ++j) acc[i][j] = qg_f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int d = 0; d < D; ++d) sum[d] = qg_f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < G::CT; ++j) sx[j] = 0.f;
    };
    auto turn_end = [&](auto reads, auto loads) {
        __builtin_amdgcn_sched_barrier(0);
        constexpr int R = decltype(reads)::value, V = decltype(loads)::value;
        if constexpr (R >= 0) asm volatile("s_waitcnt lgkmcnt(%0)" ::"n"(R) : "memory");
        if constexpr (V >= 0) asm volatile("s_waitcnt vmcnt(%0)" ::"n"(V) : "memory");
        asm volatile("s_barrier" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
    };
    // Adds the sums that part h has left over.
    auto flush = [&](int h) {
#pragma unroll
        for (int d = 0; d < D; ++d) {
            const int p = PRODUCTS - D + d;
            add_scaled(acc[h * G::MH + p / G::CT][p % G::CT], sum[p % D], sx[p % G::CT]);
        }
    };
    auto read = [&](int t, int buf, const uint8_t* S, int h) {
        Op8 ra[G::MH], rx[G::CT];
        if (h == 0) {
#pragma unroll
            for (int j = 0; j < G::CT; ++j) R.col(rx[j], buf, j);
            R.scales(xs, w, S, t);
        }
#pragma unroll
        for (int i = 0; i < G::MH; ++i) {
            if (2 * (G::MH - i) == LATE) __builtin_amdgcn_sched_barrier(0);
            R.row(ra[i], buf, h * G::MH + i);
        }
        flush(H - 1 - h);
        if (h == 0) {
#pragma unroll
            for (int j = 0; j < G::CT; ++j) fx[j] = operand<YT>(rx[j]);
        }
#pragma unroll
        for (int i = 0; i < G::MH; ++i) fa[i] = operand<YT>(ra[i]);
    };
    // The products of part h of K tile t, and between them the loads that may go now.
    auto multiply = [&](int t, int buf, int h) {
        const bool here = H == 2 && h == 1;  // to this tile's first part, or to the last part of the one before
        const int to = here ? t + NS : t - 1 + NS, to_buf = here ? buf : buf ? buf - 1 : NS - 1;
        const int part = H == 2 ? 1 - h : 0, count = part ? G::AH : G::FIRST;
#pragma unroll
        for (int p = 0; p < PRODUCTS; ++p) {
            const qg_f4 now = block_sum(fa[p / G::CT], fx[p % G::CT]);
            if (p >= D) {
                const int b = p - D;
                add_scaled(acc[h * G::MH + b / G::CT][b % G::CT], sum[b % D], sx[b % G::CT]);
            }
            sum[p % D] = now;
            if (h == 0 && p == 0) {
#pragma unroll
                for (int j = 0; j < G::CT; ++j) sx[j] = xs[j] * w;
            }
#pragma unroll
            for (int u = p * count / PRODUCTS; u < (p + 1) * count / PRODUCTS; ++u) fetch(to, to_buf, part, u);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    auto turns = [&](auto behind) {
        constexpr bool BEHIND = decltype(behind)::value;
        // Places of the scales that are read, and of those loaded last. A group of four blocks (of
        // fewer at a tile's end) is loaded when the first of them is two K tiles away, to the
        // place of the group three before: with four blocks of K or more, two groups
        // in a row have five, so that one has long been read.
        int buf = 0, from = 2, to = 0;
        auto after = [](int place) { return place == 2 ? 0 : place + 1; };
        auto k_tile = [&](auto begin, int t) {
            if ((t & 3) == 0) from = after(from);
            auto part = [&](auto which) {
                constexpr int h = decltype(which)::value;
                // loads, and stores of the tile before, sent after those that the next reading turn
                // of the first group needs
                constexpr int stores = decltype(begin)::value && h == 0 ? STORES : 0;
                constexpr int first = U + stores, second = (H == 1 ? 0 : h ? G::AH : G::FIRST) + stores;
                read(t, buf, L.scales(from), h);
                turn_end(number<LATE>{}, number<BEHIND ? second : -1>{});
                multiply(t, buf, h);
                turn_end(number<-1>{}, number<BEHIND ? -1 : first>{});
            };
            part(number<0>{});
            if constexpr (H == 2) part(number<1>{});
            buf = buf + 1 == NS ? 0 : buf + 1;
        };
        while (true) {
            k_tile(std::true_type{}, 0);
            // the next tile, and the rows that it gathers
            id += gridDim.x;
            more = tile_of(next);
            if (more && L.gathers()) {
                const int unit = wave % (BN / 64);
                const __amdgpu_buffer_rsrc_t rr =
                    __builtin_amdgcn_make_buffer_rsrc((void*)a.row, (short)0, a.N * 4, kQgRawBufferFlags);
                __builtin_amdgcn_raw_ptr_buffer_load_lds(rr, (lds_ptr)(next_rows + unit * 64), 4,
                                                         min(next.n0 + unit * 64 + lane, next.n1 - 1) * 4, 0, 0, 0);
            }
            for (int t = 1; t < nb; ++t) {
                const int l = t + AHEAD;
                if (l == nb) {
                    wnext = L.weights(next);
                    nbytes = more ? L.weight_bytes(next) : 0;
                    L.aim(next);
                    if (!more) L.xbytes = 0;
                    if (more && L.gathers()) L.rows([&](int c) { return (uint32_t)min(max(next_rows[c], 0), a.X - 1); });
                    to = after(to);
                    if (more) L.fetch_scales(0, to);
                } else if (l < nb && (l & 3) == 0) {
                    to = after(to);
                    L.fetch_scales(l >> 2, to);
                }
                k_tile(std::false_type{}, t);
            }
            flush(H - 1);
            const int m0 = (at.t0 + wm * G::MT) * 16 + (lane >> 4) * 8, c0 = at.n0 + wn * G::CT * 16 + (lane & 15);
            float sb[G::MT / 2][8];
#pragma unroll
            for (int c = 0; c < G::MT / 2; ++c) {
                row_bias(a, at.e, m0 + 32 * c, sb[c]);
#pragma unroll
                for (int i = 0; i < 8; ++i) asm volatile("" : "+v"(sb[c][i]));
            }
            if (at.t0 * T + BM <= a.M && a.ldy < (1 << 22)) {
                const __amdgpu_buffer_rsrc_t Yr = __builtin_amdgcn_make_buffer_rsrc(
                    (void*)((uint16_t*)a.Y + at.n0 * a.ldy + at.t0 * T), (short)0,
                    buffer_bytes(((int64_t)(min(at.n1 - at.n0, BN) - 1) * a.ldy + BM) * 2), kQgRawBufferFlags);
                const uint32_t ldy = (uint32_t)a.ldy * 2u, o = (uint32_t)(c0 - at.n0) * ldy + (uint32_t)(m0 - at.t0 * T) * 2u;
#pragma unroll
                for (int c = 0; c < G::MT / 2; ++c)
                    store_pair_counted<YT, G::CT>(Yr, acc[2 * c], acc[2 * c + 1], sb[c], o + c * 64, 16 * ldy, at.n1 - c0);
            } else {
                // what the next tile's first turns read
                asm volatile("s_waitcnt vmcnt(%0)" ::"n"(H == 2 ? G::FIRST : 0) : "memory");
#pragma unroll
                for (int c = 0; c < G::MT / 2; ++c)
                    store_pair<YT, G::CT>(a, acc[2 * c], acc[2 * c + 1], sb[c], m0 + 32 * c, c0, at.n1);
            }
            if (!more) return;
            clear();
            at = next;
            wp = wnext;
            wbytes = nbytes;
        }
    };
    clear();
    tile_sync<H == 2 ? G::FIRST : 0>();
    if (wave >= 4) {
        asm volatile("s_barrier" ::: "memory");
        turns(std::true_type{});
    } else {
        turns(std::false_type{});
        asm volatile("s_barrier" ::: "memory");
    }
}

// The partial sums of a split product added in order and stored: one wavefront per pair
// of a tile wavefront's products. A launch of its own (4 to 5 us in a trace), so that a
// workspace needs no preparation and no sum depends on who arrives last.
template <int YT, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(64) void gemm_f8_join_kernel(GArgs a, int tiles, int splits) {
    typedef Tile<BM, BN, WM, WN, 2> G;
    const int lane = threadIdx.x;
    const int c = blockIdx.x % (G::MT / 2), wave = blockIdx.x / (G::MT / 2) % G::W;
    const int id = blockIdx.x / (G::MT / 2 * G::W);
    const TileAt at = tile_at<BM, BN>(a.mtiles, a.N, id);
    const int wm = wave % WM, wn = wave / WM, r = lane & 15, q = lane >> 4;
    const qg_f4* p = a.part + (((size_t)id * G::W + wave) * (G::MT * G::CT) + 2 * c * G::CT) * 64 + lane;
    const size_t step = (size_t)tiles * G::W * (G::MT * G::CT) * 64;
    const int m = (at.t0 + wm * G::MT + 2 * c) * 16 + q * 8, n = at.n0 + wn * G::CT * 16 + r;
    float sb[8];
    row_bias(a, 0, m, sb);
    qg_f4 lo[G::CT], hi[G::CT];
#pragma unroll
    for (int j = 0; j < G::CT; ++j) lo[j] = hi[j] = qg_f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int s = 0; s < splits; ++s, p += step)
#pragma unroll
        for (int j = 0; j < G::CT; ++j) {
            lo[j] += p[j * 64];
            hi[j] += p[(G::CT + j) * 64];
        }
    store_pair<YT, G::CT>(a, lo, hi, sb, m, n, a.N);
}

// ---------------------------------------------------------------- launches
int64_t weight_tiles(int64_t M) { return qg::ceil_div(M, kPair) * 2; }

// The forms and the rule that takes one (bf16 outputs, weights from memory, calls in a graph).
//   STREAM  few rows: 4608 x 3584 by 1 in 6.2 us (64 x 64: 11.0), 152064 x 3584 by 1 in 87 (101);
//           up to 16 rows of weights of up to 8192 rows (by 16: 8.4 and 11.1; 18944 x 3584 by 16
//           18.8 and 15.4). From 17 rows on, tiles (4608 x 3584 by 32: 13.5 and 11.0).
//   S64     tiles of 64 x 64, two workgroups to a unit, until there are over 512 of them.
//   S128x64 the same with fewer reads of the activations, for one column of many (152064 x
//           3584 by 32: 105 us, 64 x 64 120).
//   S128    tiles of 128 in three LDS buffers, one workgroup to a unit, up to 256 of them (4608 x
//           3584 by 512: 19.2 us, 64 x 64 22.4, 256 x 128 26.7).
//   M128    tiles of 128 in two buffers, two workgroups to a unit: what is left where turns cannot be
//           taken (float32, K below four blocks).
//   T128, T256  256 x 128 and 256 x 256 in turns; a round of tiles on all units costs 27
//           and 49 us at K = 3584, so the number of rounds decides: 4608 x 3584 by 4096 takes 82
//           us in 3 of the first, 91 in 2 of the second, 37888 x 3584 by 4096 513 and 495.
// With fewer tiles than units a long K is split until about 256 workgroups share it, each
// keeping some K tiles to repay the second launch (3584 x 18944 by 64: 43 us whole, 19 in 4).
enum { STREAM, S64, S128x64, S128, M128, T128, T256 };
struct Plan {
    int form, tiles, splits, kper;
    size_t ws;
};

Plan plan(int64_t M, int64_t K, int64_t N, int y_type) {
    Plan p{};
    const int kt = (int)qg::ceil_div(K, kB);
    p.splits = 1;
    p.kper = kt;
    auto tiles = [&](int bm, int bn) { return qg::ceil_div(M, bm) * qg::ceil_div(N, bn); };
    auto take = [&](int form, int bm, int bn) {
        p.form = form;
        p.tiles = (int)tiles(bm, bn);
    };
    if (N <= 4 || (N <= 16 && M <= 8192)) {
        p.form = STREAM;
        p.tiles = (int)weight_tiles(M);
        return p;
    }
    if (N <= 64 && tiles(64, 64) > 1024)
        take(S128x64, 128, 64);
    else if (tiles(64, 64) <= 512 && !(N > 64 && kt >= 64))
        take(S64, 64, 64);
    else if (tiles(128, 128) <= 256)
        take(S128, 128, 128);
    else if (y_type == QG_F32 || kt < kTurnsBlocks)
        take(M128, 128, 128);
    else if (qg::ceil_div(tiles(256, 256), 256) * 9 <= qg::ceil_div(tiles(256, 128), 256) * 5)
        take(T256, 256, 256);
    else
        take(T128, 256, 128);
    if (p.form == S64 || p.form == S128) {
        const int side = p.form == S64 ? 64 : 128, s = std::min(256 / p.tiles, kt / (side == 128 ? 18 : 28));
        if (s > 1) {
            p.kper = (int)qg::ceil_div(kt, s);
            p.splits = (int)qg::ceil_div(kt, p.kper);
            p.ws = (size_t)p.splits * p.tiles * side * side * 4;
        }
    }
    return p;
}

// A workgroup takes tile after tile, as many of them at a time as there is LDS for.
template <class K>
qg_status launch_tiles(K kernel, std::atomic<bool>* done, const GArgs& a, const Plan& p, int threads, int lds, bool split,
                       hipStream_t s) {
    if (lds > 65536) {
        const qg_status st = allow_lds(reinterpret_cast<const void*>(kernel), 160 * 1024, done);
        if (st) return st;
    }
    GArgs b = a;
    b.total = p.tiles;
    const int groups = split ? p.tiles : std::min(p.tiles, qg::device_cus() * (160 * 1024 / lds));
    hipLaunchKernelGGL(kernel, dim3(groups, p.splits), dim3(threads), lds, s, b);
    return qg::launch_status("qgemm_f8");
}
template <int YT, int BM, int BN, int WM, int WN, int NS, bool SPLIT, bool GROUPED>
qg_status launch_small(const GArgs& a, const Plan& p, hipStream_t s) {
    typedef F8Tile<BM, BN, WM, WN, NS, 1, 8, 2> G;
    static std::atomic<bool> done[64];
    qg_status st = launch_tiles(gemm_f8_tile_kernel<YT, BM, BN, WM, WN, NS, SPLIT, GROUPED>, done, a, p, 64 * G::W,
                                G::LDS + (GROUPED ? Experts::bytes(a.E) : 0), SPLIT, s);
    if constexpr (SPLIT) {
        if (st) return st;
        hipLaunchKernelGGL((gemm_f8_join_kernel<YT, BM, BN, WM, WN>), dim3(p.tiles * G::W * (G::MT / 2)), dim3(64), 0, s,
                           a, p.tiles, p.splits);
        st = qg::launch_status("qgemm_f8 (join)");
    }
    return st;
}
template <int YT, int BM, int BN, int WM, int WN, int NS, int H, bool GROUPED>
qg_status launch_turns(const GArgs& a, const Plan& p, hipStream_t s) {
    typedef F8Tile<BM, BN, WM, WN, NS, H, 4, 3> G;
    constexpr int rows = GROUPED ? BN * 4 : 0;
    static_assert(G::LDS + rows + (GROUPED ? (2 + 2 * kTurnsExperts) * 4 : 0) <= 160 * 1024, "LDS of a compute unit");
    static std::atomic<bool> done[64];
    return launch_tiles(gemm_f8_turns_kernel<YT, BM, BN, WM, WN, NS, H, GROUPED>, done, a, p, 512,
                        G::LDS + rows + (GROUPED ? Experts::bytes(a.E) : 0), false, s);
}

template <int YT>
qg_status launch_gemm(const GArgs& a, const Plan& p, hipStream_t s) {
    const bool split = p.splits > 1;
    switch (p.form) {
        case S64:
            return split ? launch_small<YT, 64, 64, 1, 4, 4, true, false>(a, p, s)
                         : launch_small<YT, 64, 64, 1, 4, 4, false, false>(a, p, s);
        case S128x64: return launch_small<YT, 128, 64, 2, 2, 3, false, false>(a, p, s);
        case S128:
            return split ? launch_small<YT, 128, 128, 2, 4, 3, true, false>(a, p, s)
                         : launch_small<YT, 128, 128, 2, 4, 3, false, false>(a, p, s);
        case M128: return launch_small<YT, 128, 128, 2, 2, 2, false, false>(a, p, s);
        case T128:
            if constexpr (YT != QG_F32) return launch_turns<YT, 256, 128, 4, 2, 3, 1, false>(a, p, s);
            break;
        case T256:
            if constexpr (YT != QG_F32) return launch_turns<YT, 256, 256, 2, 4, 2, 2, false>(a, p, s);
            break;
    }
    hipLaunchKernelGGL((gemm_f8_stream_kernel<YT>), dim3(a.mtiles), dim3(64 * kStreamWaves), 0, s, a);
    return qg::launch_status("qgemm_f8");
}

// The same by the mean of rows to an expert that can have some, as the host does not know the
// offsets (128 experts of 1536 x 2048, 8 to a token): one token streams (9.8 us, 64 x 64 11.1), as do all
// with fewer than 256 tiles of 64 weight rows; up to 2 rows 64 x 64 (16 tokens 42.9 us, streamed
// 60.5); up to 64 rows 128 x 64 (512 tokens 81 us, 256 x 128 90); up to 512 256 x 128 (4096 tokens
// 166 us, 256 x 256 173), beyond 256 x 256 (8 experts of 4096 x 2048, 2 to each of 4096 tokens: 94 us and 103).
template <int YT>
qg_status launch_grouped(const GArgs& a, hipStream_t s) {
    const int64_t used = std::min(a.E, a.N), each = qg::ceil_div(a.N, used);
    Plan p{};
    p.splits = 1;
    auto tiles = [&](int bm, int bn) {
        return (int)(std::min<int64_t>(a.N, a.N / bn + used) * qg::ceil_div(a.mtiles * 16, bm));
    };
    if (each <= 4 && used * qg::ceil_div(a.mtiles * 16, 64) <= 256) {
        hipLaunchKernelGGL((gemm_f8_stream_kernel<YT>), dim3(a.mtiles, (unsigned)used), dim3(64 * kStreamWaves), 0, s, a);
        return qg::launch_status("qgemm_f8_grouped");
    }
    if (each <= 2) {
        p.tiles = tiles(64, 64);
        return launch_small<YT, 64, 64, 1, 4, 4, false, true>(a, p, s);
    }
    if (each <= 64) {
        p.tiles = tiles(128, 64);
        return launch_small<YT, 128, 64, 2, 2, 3, false, true>(a, p, s);
    }
    if constexpr (YT != QG_F32)
        if (a.nb >= kTurnsBlocks && a.E <= kTurnsExperts) {
            if (each >= 512) {
                p.tiles = tiles(256, 256);
                return launch_turns<YT, 256, 256, 2, 4, 2, 2, true>(a, p, s);
            }
            p.tiles = tiles(256, 128);
            return launch_turns<YT, 256, 128, 4, 2, 3, 1, true>(a, p, s);
        }
    p.tiles = tiles(128, 128);
    return launch_small<YT, 128, 128, 2, 2, 2, false, true>(a, p, s);
}

qg_status check_mk(int64_t M, int64_t K) {
    if (M < 1 || M > QG_F8_MAX_ROWS)
        return qg::fail(QG_ERR_SHAPE, "M=%lld not in [1, %d]", (long long)M, QG_F8_MAX_ROWS);
    if (K < 1 || K > QG_F8_MAX_K)
        return qg::fail(QG_ERR_SHAPE, "K=%lld not in [1, %d]", (long long)K, QG_F8_MAX_K);
    return QG_OK;
}

constexpr int64_t kMost = (int64_t)1 << 40;

template <int XT, bool GATED>
void launch_quantize(const QArgs& a, hipStream_t s) {
    // (a grid of 2^32 threads is too large)
    const int64_t groups = std::min<int64_t>(qg::ceil_div((int64_t)a.N * a.quads, 4), 1 << 22);
    hipLaunchKernelGGL((quantize_f8_kernel<XT, GATED>), dim3((unsigned)groups), dim3(256), 0, s, a);
}

// What the dense and the grouped product check alike. rows: rows of x.
qg_status check_operands(const void* w, const float* ws, const void* xq, int64_t ldx, const float* xs, int64_t ldxs,
                         const float* bias, const void* Y, int y_type, int64_t ldy, int64_t M, int64_t K, int64_t N,
                         int64_t rows, int64_t experts) {
    if (!w || !ws || !xq || !xs || !Y) return qg::fail(QG_ERR_NULL, "NULL pointer (w_packed, w_scale, xq, x_scale, Y)");
    if (!known_type(y_type)) return qg::fail(QG_ERR_SHAPE, "y_type=%d unknown", y_type);
    const qg_status st = check_mk(M, K);
    if (st) return st;
    if (experts < 1 || experts > QG_EXPERTS_MAX)
        return qg::fail(QG_ERR_SHAPE, "experts=%lld not in [1, %d]", (long long)experts, QG_EXPERTS_MAX);
    const int64_t nb = qg::ceil_div(K, kB), kp = nb * kB;
    if (N < 1 || N > QG_F8_MAX_ROWS || M * N > (int64_t)1 << 32)
        return qg::fail(QG_ERR_SHAPE, "%lld rows not in [1, %d], or times M over 2^32", (long long)N, QG_F8_MAX_ROWS);
    if (rows < 1 || rows > QG_F8_MAX_ROWS)
        return qg::fail(QG_ERR_SHAPE, "%lld rows of xq not in [1, %d]", (long long)rows, QG_F8_MAX_ROWS);
    if (ldx < kp || ldx > (1 << 22) || ldx % 16)  // 256 rows stay within 32-bit offsets
        return qg::fail(QG_ERR_SHAPE, "ldx=%lld not a multiple of 16 in [%lld, 2^22]", (long long)ldx, (long long)kp);
    if (ldxs < nb || ldxs > (1 << 20) || ldxs % 4)
        return qg::fail(QG_ERR_SHAPE, "ldxs=%lld not a multiple of 4 in [%lld, 2^20]", (long long)ldxs, (long long)nb);
    if (ldy < M || ldy > kMost / N || ldy % 4)
        return qg::fail(QG_ERR_SHAPE, "ldy=%lld not a multiple of 4 in [M, 2^40 / N]", (long long)ldy);
    if (!qg::aligned16(w) || !qg::aligned16(xq) || !qg::aligned16(xs) || !qg::aligned16(Y))
        return qg::fail(QG_ERR_ALIGN, "w_packed, xq, x_scale and Y must be 16-byte aligned");
    if ((reinterpret_cast<uintptr_t>(ws) | reinterpret_cast<uintptr_t>(bias)) & 3)
        return qg::fail(QG_ERR_ALIGN, "w_scale and bias must be 4-byte aligned");
    return QG_OK;
}

}  // namespace

extern "C" {

size_t qg_f8_bytes(int64_t M, int64_t K, int64_t experts) {
    if (M < 1 || M > QG_F8_MAX_ROWS || K < 1 || K > QG_F8_MAX_K || experts < 1 || experts > QG_EXPERTS_MAX) return 0;
    const int64_t one = weight_tiles(M) * qg::ceil_div(K, kB) * kUnit;
    return one > kMost / experts ? 0 : (size_t)(one * experts);
}

qg_status qg_pack_f8(const void* w, int64_t ldw, int64_t w_expert, void* dst, int64_t M, int64_t K, int64_t experts,
                     qg_stream_t stream) {
    qg::clear_error();
    if (!w || !dst) return qg::fail(QG_ERR_NULL, "NULL pointer (w, dst)");
    qg_status st = check_mk(M, K);
    if (st) return st;
    const size_t n = qg_f8_bytes(M, K, experts);
    if (!n) return qg::fail(QG_ERR_SHAPE, "experts=%lld not in [1, %d], or over 2^40 bytes", (long long)experts, QG_EXPERTS_MAX);
    if (ldw < K || ldw > kMost / M) return qg::fail(QG_ERR_SHAPE, "ldw=%lld not in [K, 2^40 / M]", (long long)ldw);
    if (experts > 1 && (w_expert < (M - 1) * ldw + K || w_expert > kMost / experts))
        return qg::fail(QG_ERR_SHAPE, "w_expert=%lld: experts overlap, or over 2^40 bytes", (long long)w_expert);
    if (!qg::aligned16(dst)) return qg::fail(QG_ERR_ALIGN, "dst not 16-byte aligned");
    const size_t src = (size_t)(experts > 1 ? (experts - 1) * w_expert : 0) + (M - 1) * ldw + K;
    if (overlap(w, src, dst, n)) return qg::fail(QG_ERR_SHAPE, "w and dst overlap");
    st = qg::check_device();
    if (st) return st;
    const int64_t units = (int64_t)(n / 16);
    const unsigned g = (unsigned)std::min<int64_t>(qg::ceil_div(units, 256), 65536);
    hipLaunchKernelGGL(pack_f8_kernel, dim3(g), dim3(256), 0, (hipStream_t)stream, (const uint8_t*)w, ldw, w_expert,
                       (uint4*)dst, M, (int)K, (int)qg::ceil_div(K, kB), weight_tiles(M), units);
    return qg::launch_status("qg_pack_f8");
}

qg_status qg_quantize_f8_rows(const void* x, int x_type, int64_t ldx, int gated, const int32_t* count, int64_t N, int64_t K,
                              void* q, int64_t ldq, float* scale, int64_t lds, qg_stream_t stream) {
    qg::clear_error();
    if (!x || !q || !scale) return qg::fail(QG_ERR_NULL, "NULL pointer (x, q, scale)");
    if (!known_type(x_type)) return qg::fail(QG_ERR_SHAPE, "x_type=%d unknown", x_type);
    if (gated != 0 && gated != 1) return qg::fail(QG_ERR_SHAPE, "gated=%d not 0 or 1", gated);
    if (N < 1 || N > QG_F8_MAX_ROWS)
        return qg::fail(QG_ERR_SHAPE, "N=%lld not in [1, %d]", (long long)N, QG_F8_MAX_ROWS);
    if (K < 1 || K > QG_F8_MAX_K) return qg::fail(QG_ERR_SHAPE, "K=%lld not in [1, %d]", (long long)K, QG_F8_MAX_K);
    const int64_t nb = qg::ceil_div(K, kB), width = gated ? 2 * K : K, most = kMost / N;
    const int64_t sp = qg::ceil_div(nb, 4) * 4;
    if (ldx < width || ldx > most)
        return qg::fail(QG_ERR_SHAPE, "ldx=%lld not in [%lld, 2^40 / N]", (long long)ldx, (long long)width);
    if (ldq < nb * kB || ldq > most || ldq % 16)
        return qg::fail(QG_ERR_SHAPE, "ldq=%lld not a multiple of 16 in [%lld, 2^40 / N]", (long long)ldq, (long long)(nb * kB));
    if (lds < sp || lds > most || lds % 4)
        return qg::fail(QG_ERR_SHAPE, "lds=%lld not a multiple of 4 in [%lld, 2^40 / N]", (long long)lds, (long long)sp);
    const int eb = elem_bytes(x_type);
    if (reinterpret_cast<uintptr_t>(x) % eb) return qg::fail(QG_ERR_ALIGN, "x not aligned to its elements");
    if (!qg::aligned16(q) || !qg::aligned16(scale)) return qg::fail(QG_ERR_ALIGN, "q and scale must be 16-byte aligned");
    if (reinterpret_cast<uintptr_t>(count) & 3) return qg::fail(QG_ERR_ALIGN, "count not 4-byte aligned");
    const size_t xb = ((size_t)(N - 1) * ldx + width) * eb, qb = (size_t)(N - 1) * ldq + nb * kB;
    const size_t sb = ((size_t)(N - 1) * lds + sp) * 4;
    if (overlap(x, xb, q, qb) || overlap(x, xb, scale, sb) || overlap(q, qb, scale, sb) ||
        (count && (overlap(count, 4, q, qb) || overlap(count, 4, scale, sb))))
        return qg::fail(QG_ERR_SHAPE, "x, count, q and scale overlap");
    qg_status st = qg::check_device();
    if (st) return st;
    QArgs a{x, ldx, count, (uint8_t*)q, ldq, scale, lds, (int32_t)N, (int32_t)K, (uint32_t)(sp / 4)};
    hipStream_t s = (hipStream_t)stream;
    if (x_type == QG_F32)
        gated ? launch_quantize<QG_F32, true>(a, s) : launch_quantize<QG_F32, false>(a, s);
    else if (x_type == QG_F16)
        gated ? launch_quantize<QG_F16, true>(a, s) : launch_quantize<QG_F16, false>(a, s);
    else
        gated ? launch_quantize<QG_BF16, true>(a, s) : launch_quantize<QG_BF16, false>(a, s);
    return qg::launch_status("qg_quantize_f8_rows");
}

size_t qgemm_f8_workspace_bytes(int64_t M, int64_t K, int64_t N, int y_type) {
    if (!qg_f8_bytes(M, K, 1) || N < 1 || N > QG_F8_MAX_ROWS || M * N > (int64_t)1 << 32 || !known_type(y_type)) return 0;
    return plan(M, K, N, y_type).ws;
}

qg_status qgemm_f8(const void* w, const float* ws, const void* xq, int64_t ldx, const float* xs, int64_t ldxs,
                   const float* bias, void* Y, int y_type, int64_t ldy, int64_t M, int64_t K, int64_t N,
                   void* workspace, size_t workspace_bytes, qg_stream_t stream) {
    qg::clear_error();
    qg_status st = check_operands(w, ws, xq, ldx, xs, ldxs, bias, Y, y_type, ldy, M, K, N, N, 1);
    if (st) return st;
    const int64_t nb = qg::ceil_div(K, kB), mb = qg::ceil_div(M, kB);
    const size_t yb = ((size_t)(N - 1) * ldy + M) * elem_bytes(y_type), xb = (size_t)(N - 1) * ldx + nb * kB;
    const size_t sb = ((size_t)(N - 1) * ldxs + qg::ceil_div(nb, 4) * 4) * 4, wb = qg_f8_bytes(M, K, 1), wsb = (size_t)mb * nb * 4;
    auto over = [&](const void* p, size_t n) {
        return overlap(p, n, xq, xb) || overlap(p, n, w, wb) || overlap(p, n, ws, wsb) || overlap(p, n, xs, sb) ||
               (bias && overlap(p, n, bias, (size_t)M * 4));
    };
    if (over(Y, yb)) return qg::fail(QG_ERR_SHAPE, "Y overlaps an input");
    const Plan p = plan(M, K, N, y_type);
    if (p.ws) {
        if (!workspace || workspace_bytes < p.ws)
            return qg::fail(QG_ERR_WORKSPACE, "workspace of %zu bytes required, got %zu", p.ws, workspace ? workspace_bytes : 0);
        if (!qg::aligned16(workspace)) return qg::fail(QG_ERR_ALIGN, "workspace not 16-byte aligned");
        if (over(workspace, p.ws) || overlap(workspace, p.ws, Y, yb))
            return qg::fail(QG_ERR_SHAPE, "the workspace overlaps an operand");
    }
    st = qg::check_device();
    if (st) return st;
    GArgs a{};
    a.w = (const uint8_t*)w;
    a.ws = ws;
    a.x = (const uint8_t*)xq;
    a.ldx = ldx;
    a.xs = xs;
    a.ldxs = ldxs;
    a.bias = bias;
    a.Y = Y;
    a.ldy = ldy;
    a.part = (qg_f4*)workspace;
    a.M = (int32_t)M;
    a.N = a.X = (int32_t)N;
    a.E = 1;
    a.nb = (int32_t)nb;
    a.mb = (int32_t)mb;
    a.mtiles = (int32_t)weight_tiles(M);
    a.kper = p.kper;
    a.total = p.tiles;
    hipStream_t s = (hipStream_t)stream;
    if (y_type == QG_F32) return launch_gemm<QG_F32>(a, p, s);
    if (y_type == QG_F16) return launch_gemm<QG_F16>(a, p, s);
    return launch_gemm<QG_BF16>(a, p, s);
}

qg_status qgemm_f8_grouped(const qg_f8_grouped* g, qg_stream_t stream) {
    qg::clear_error();
    if (!g) return qg::fail(QG_ERR_NULL, "NULL pointer (problem)");
    qg_status st = check_operands(g->w_packed, g->w_scale, g->xq, g->ldx, g->x_scale, g->ldxs, g->bias, g->Y, g->y_type,
                                  g->ldy, g->M, g->K, g->rows, g->x_rows, g->experts);
    if (st) return st;
    if (!g->offsets) return qg::fail(QG_ERR_NULL, "NULL pointer (offsets)");
    if ((reinterpret_cast<uintptr_t>(g->offsets) | reinterpret_cast<uintptr_t>(g->row)) & 3)
        return qg::fail(QG_ERR_ALIGN, "offsets and row must be 4-byte aligned");
    if (!g->row && g->x_rows < g->rows)
        return qg::fail(QG_ERR_SHAPE, "x_rows=%lld below rows=%lld without `row`", (long long)g->x_rows, (long long)g->rows);
    const int64_t nb = qg::ceil_div(g->K, kB), mb = qg::ceil_div(g->M, kB);
    const size_t xb = (size_t)(g->x_rows - 1) * g->ldx + nb * kB, sb = ((size_t)(g->x_rows - 1) * g->ldxs + qg::ceil_div(nb, 4) * 4) * 4;
    if (g->row && (xb > UINT32_MAX || sb > UINT32_MAX))
        return qg::fail(QG_ERR_SHAPE, "xq or x_scale of 2^32 bytes or more with `row`");
    const size_t wb = qg_f8_bytes(g->M, g->K, g->experts);
    if (!wb) return qg::fail(QG_ERR_SHAPE, "weights of over 2^40 bytes");
    const size_t yb = ((size_t)(g->rows - 1) * g->ldy + g->M) * elem_bytes(g->y_type);
    if (overlap(g->Y, yb, g->xq, xb) || overlap(g->Y, yb, g->w_packed, wb) || overlap(g->Y, yb, g->x_scale, sb) ||
        overlap(g->Y, yb, g->w_scale, (size_t)g->experts * mb * nb * 4) ||
        overlap(g->Y, yb, g->offsets, (size_t)(g->experts + 1) * 4) || (g->row && overlap(g->Y, yb, g->row, (size_t)g->rows * 4)) ||
        (g->bias && overlap(g->Y, yb, g->bias, (size_t)g->experts * g->M * 4)))
        return qg::fail(QG_ERR_SHAPE, "Y overlaps an input");
    st = qg::check_device();
    if (st) return st;
    GArgs a{};
    a.w = (const uint8_t*)g->w_packed;
    a.ws = g->w_scale;
    a.x = (const uint8_t*)g->xq;
    a.ldx = g->ldx;
    a.xs = g->x_scale;
    a.ldxs = g->ldxs;
    a.bias = g->bias;
    a.Y = g->Y;
    a.ldy = g->ldy;
    a.offsets = g->offsets;
    a.row = g->row;
    a.M = (int32_t)g->M;
    a.N = (int32_t)g->rows;
    a.X = (int32_t)g->x_rows;
    a.E = (int32_t)g->experts;
    a.nb = (int32_t)nb;
    a.mb = (int32_t)mb;
    a.mtiles = (int32_t)weight_tiles(g->M);
    hipStream_t s = (hipStream_t)stream;
    if (g->y_type == QG_F32) return launch_grouped<QG_F32>(a, s);
    if (g->y_type == QG_F16) return launch_grouped<QG_F16>(a, s);
    return launch_grouped<QG_BF16>(a, s);
}

}  // extern "C"
