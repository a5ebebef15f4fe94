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
// consecutive ones of a pair's.
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

// x / d rounded to e4m3's three bits after the leading one (from 2^-6 on; multiples of
// 2^-9 below), ties to even, decided on the exact quotient: in double precision the
// quotient of two floats is never rounded onto a border that it does not meet.
QG_DEV float round_exact(float x, float d) {
    const double v = (double)x / (double)d, a = fabs(v);
    const int e = a < 0x1p-6 ? -6 : ilogb(a);
    return (float)ldexp(rint(ldexp(v, 3 - e)), e - 3);
}

// Eight values divided by d, as e4m3 bytes. x * inv is off by two units in the last place
// at most; where it lies within four of a border between two results, the exact quotient
// decides.
QG_DEV uint2 quant8(const float (&x)[8], float d, float inv) {
    float t[8];
    bool near = false;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        t[e] = x[e] * inv;
        float a = fabsf(t[e]);
        if (a < 0x1p-6f) a += 0x1p-6f;  // (below 2^-6 the borders are those of the next octave, shifted)
        near |= ((__builtin_bit_cast(uint32_t, a) + 4u - 0x80000u) & 0xfffffu) <= 8u;
    }
    if (near) {
#pragma unroll
        for (int e = 0; e < 8; ++e) t[e] = round_exact(x[e], d);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) t[e] = fminf(fmaxf(t[e], -448.f), 448.f);  // (over it where the scale is subnormal)
    uint2 o;
    o.x = __builtin_amdgcn_cvt_pk_fp8_f32(t[0], t[1], 0, false);
    o.x = __builtin_amdgcn_cvt_pk_fp8_f32(t[2], t[3], o.x, true);
    o.y = __builtin_amdgcn_cvt_pk_fp8_f32(t[4], t[5], 0, false);
    o.y = __builtin_amdgcn_cvt_pk_fp8_f32(t[6], t[7], o.y, true);
    return o;
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

// Sixteen lanes per block of 128, a wavefront per four blocks, U of them at a time.
template <int XT, bool GATED, int U>
__global__ __launch_bounds__(256) void quantize_f8_kernel(QArgs a) {
    typedef typename XVec<XT>::E E;
    constexpr int VN = XVec<XT>::N, V = 8 / VN;  // vectors of a lane's eight values
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t rows = a.count ? min(max(*a.count, 0), a.N) : a.N;
    const uint32_t total = rows * a.quads;  // below 2^31
    for (uint32_t first = (blockIdx.x * 4 + wave) * U; first < total; first += gridDim.x * 4 * U) {
    uint4 v[U][V], g[GATED ? U : 1][V];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const uint32_t at = first + u;
        if (at < total) {
            const uint32_t n = at / a.quads;
            const int k = (int)(at - n * a.quads) * 4 * kB + lane * 8;
            const E* p = reinterpret_cast<const E*>(a.x) + n * a.ldx;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                v[u][i] = row_vec<XT>(p, a.K, k / VN + i);
                if constexpr (GATED) {
                    g[u][i] = v[u][i];
                    v[u][i] = row_vec<XT>(p + a.K, a.K, k / VN + i);
                }
            }
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const uint32_t at = first + u;
        if (at >= total) return;
        const uint32_t n = at / a.quads;
        const int b = (int)(at - n * a.quads) * 4 + (lane >> 4);
        float x[8];
        uint32_t mx = 0;  // the largest |x| by its bits: above every finite value an infinity, above it a NaN
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            x[e] = XVec<XT>::get(v[u][e / VN], e % VN);
            if constexpr (GATED) {
                const float z = XVec<XT>::get(g[u][e / VN], e % VN);
                x[e] *= z / (1.f + expf(-z));
            }
            mx = max(mx, __builtin_bit_cast(uint32_t, x[e]) & 0x7fffffffu);
        }
        mx = row_max(mx);
        const bool finite = mx < 0x7f800000u;
        const float d0 = finite ? __builtin_bit_cast(float, mx) / 448.f : __builtin_nanf("");
        const bool ok = d0 > 0.f;
        // tiny scales: x and d scaled alike (exactly), so that 1/d stays finite
        const float s = d0 < 0x1p-90f ? 0x1p60f : 1.f;
        const float d = ok ? d0 * s : 1.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = ok ? x[e] * s : 0.f;
        const uint2 o = quant8(x, d, 1.f / d);
        const bool in = b * kB < a.K;
        if (in) *reinterpret_cast<uint2*>(a.q + n * a.ldq + b * kB + (lane & 15) * 8) = o;
        if ((lane & 15) == 0) a.scale[n * a.lds + b] = in ? d0 : 0.f;
    }
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
// One 16-row tile of an expert's weights and NB blocks of 16 rows of Y per workgroup; its
// KW wavefronts take blocks of K in turn, and their sums meet in LDS, in order. The
// weights go from memory straight to registers, in the packed order.
template <int YT, int NB, int KW>
__global__ __launch_bounds__(64 * KW) void gemm_f8_stream_kernel(GArgs a) {
    __shared__ qg_f4 part[KW][NB][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int t = blockIdx.x, slot = blockIdx.y;
    Group g = {0, 0, a.N};
    if (a.offsets && !used_group(a, slot, g)) return;
    const uint8_t* w = a.w + ((size_t)g.e * a.mtiles + t) * a.nb * kUnit + lane * 16;
    const float* ws = a.ws + ((size_t)g.e * a.mb + t * T / kB) * a.nb;
    for (int c0 = g.r0; c0 < g.r1; c0 += 16 * NB) {
        const uint8_t* xr[NB];
        const float* sr[NB];
#pragma unroll
        for (int c = 0; c < NB; ++c) {  // rows beyond the last repeat it; their sums are not stored
            const int64_t r = source_row(a, min(c0 + 16 * c + (lane & 15), g.r1 - 1));
            xr[c] = a.x + r * a.ldx + (lane >> 4) * 16;
            sr[c] = a.xs + r * a.ldxs;
        }
        qg_f4 acc[NB];
#pragma unroll
        for (int c = 0; c < NB; ++c) acc[c] = qg_f4{0.f, 0.f, 0.f, 0.f};
        Op8 wv[2], xv[2][NB];
        float sv[2][NB];
        auto load = [&](int p, int b) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
                wv[p].h[h] = __builtin_nontemporal_load(reinterpret_cast<const qi4*>(w + (size_t)b * kUnit + h * 1024));
#pragma unroll
            for (int c = 0; c < NB; ++c) {
#pragma unroll
                for (int h = 0; h < 2; ++h) xv[p][c].h[h] = *reinterpret_cast<const qi4*>(xr[c] + b * kB + h * 64);
                sv[p][c] = sr[c][b] * ws[b];
            }
        };
        auto mma = [&](int p) {
            Op16 wh, xh;
            wh.set(wv[p]);
#pragma unroll
            for (int c = 0; c < NB; ++c) {
                xh.set(xv[p][c]);
                add_scaled(acc[c], block_sum(wh, xh), sv[p][c]);
            }
        };
        int b = wave;
        for (; b + KW < a.nb; b += 2 * KW) {
            load(0, b);
            load(1, b + KW);
            mma(0);
            mma(1);
        }
        if (b < a.nb) {
            load(0, b);
            mma(0);
        }
#pragma unroll
        for (int c = 0; c < NB; ++c) part[wave][c][lane] = acc[c];
        __syncthreads();
        if (wave < NB) {
            const int c = wave, n = c0 + 16 * c + (lane & 15), m = (t >> 1) * kPair + (lane >> 4) * 8 + (t & 1) * 4;
            qg_f4 s = part[0][c][lane];
#pragma unroll
            for (int k = 1; k < KW; ++k) s += part[k][c][lane];
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
// Tiles of Y (Tile in qg_rows.h: a K tile of 128 bytes is one block). Beside a tile's
// stages LDS holds the row scales and the weight scales of eight blocks, twice, and of a
// grouped product the experts' first tiles.
template <int BM, int BN, int WM, int WN, int NS, int H>
struct F8Tile : Tile<BM, BN, WM, WN, NS> {
    typedef Tile<BM, BN, WM, WN, NS> P;
    static constexpr int SU = 2 * BN / 64;            // 1 KB loads of the row scales of eight blocks
    static constexpr int MB = (BM + kB - 1) / kB;      // blocks of weight rows
    static constexpr int SB = SU * 1024 + MB * 256;    // bytes of all scales of eight blocks
    static constexpr int LDS = P::LDS + 2 * SB;
    static constexpr int MH = P::MT / H;               // weight operands of a part of a K tile
    static constexpr int AH = P::AU / H;               // loads of them
    static_assert(P::W == 8 && MH * H == P::MT && AH * H == P::AU && ((H == 1 && NS >= 3) || (H == 2 && NS == 2)), "parts of a K tile");
    static_assert(BM / WM <= kB && kB % (BM / WM) == 0 && BN % 64 == 0, "a wavefront's rows share a weight scale");
};

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

template <int N>
using number = std::integral_constant<int, N>;

// The tiles of BN rows before each expert's, in LDS, by the first wavefront; returns the
// number of all of them to it.
template <int BN>
QG_DEV int first_tiles(const GArgs& a, int* first) {
    const int lane = threadIdx.x & 63;
    int all = 0;
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
        first[e0 + lane] = all + upto - n;
        all += __builtin_amdgcn_readlane(upto, 63);
    }
    return all;
}

// Tile of a grouped product: the experts' tiles of BN rows in order, each with all of its
// weight tiles; the XCDs take contiguous runs. False beyond the last one.
struct GroupTile {
    Group g;
    int t0, n0;  // first 16-row weight tile, first row of Y
};
template <int BM, int BN>
QG_DEV bool group_tile_at(const GArgs& a, const int* first, int all, int id, GroupTile& o) {
    const int lane = threadIdx.x & 63;
    const int mts = (a.mtiles * 16 + BM - 1) / BM;
    const int total = all * mts, q = total / 8, r = total % 8, x = id % 8;
    if (id / 8 >= q + (x < r)) return false;
    id = x * q + min(x, r) + id / 8;
    const int at = id / mts;
    o.t0 = (id - at * mts) * (BM / 16);
    // the last expert whose first tile is not beyond this one (it has rows: one without would share
    // its first tile with the next)
    int e = -1;
    for (int e0 = 0; e0 < a.E; e0 += 64) {
        const int c = __builtin_popcountll(__ballot(e0 + lane < a.E && first[e0 + lane] <= at));
        e += c;
        if (c < 64) break;
    }
    o.g.e = e;
    const int r0 = min(max(a.offsets[e], 0), a.N);
    o.g.r0 = __builtin_amdgcn_readfirstlane(r0);
    o.g.r1 = __builtin_amdgcn_readfirstlane(min(max(a.offsets[e + 1], r0), a.N));
    o.n0 = o.g.r0 + (at - __builtin_amdgcn_readfirstlane(first[e])) * BN;
    return true;
}

template <int YT, int BM, int BN, int WM, int WN, int NS, int H, bool SPLIT, bool GROUPED>
__global__ __launch_bounds__(64 * WM * WN) void gemm_f8_tile_kernel(GArgs a) {
    typedef F8Tile<BM, BN, WM, WN, NS, H> G;
    // float32 outputs take the exact block sums, 16-bit ones the faster 8-bit matrix cores
    typedef typename std::conditional<YT == QG_F32, Op16, Op8>::type Op;
    extern __shared__ __align__(1024) uint8_t lds[];
    uint8_t* const sl = lds + G::P::LDS;
    int* const first = reinterpret_cast<int*>(lds + G::LDS);
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int k0 = SPLIT ? blockIdx.y * a.kper : 0;
    const int k1 = SPLIT ? min(a.nb, k0 + a.kper) : a.nb;
    int all = 0;
    if constexpr (GROUPED) {
        if (wave == 0) {
            all = first_tiles<BN>(a, first + 1);
            if (lane == 0) first[0] = all;
        }
        __syncthreads();
        all = __builtin_amdgcn_readfirstlane(first[0]);
    }

    // Loads: rows and tiles beyond the operands repeat the last ones (their sums are
    // not stored). Weights arrive in the packed order. Activations: eight lanes per row
    // of 128 bytes, the 16-byte chunk c of row r at place c ^ (r % 8), which spreads
    // the operand reads over the banks.
    const int chunk = (lane & 7) ^ (lane >> 3);
    const int wm = wave % WM, wn = wave / WM, mine = wm * (BM / WM) / kB;  // (wavefronts of one block of rows load its scales alike)
    const uint8_t *wp, *xp;
    int wbytes, xbytes;
    __amdgpu_buffer_rsrc_t sr, vr;
    uint32_t woff[G::AU], xoff[G::XU], soff;
    int t0, n0, n1, e = 0;
    // 1 KB of weights in a stage that load u of this wavefront brings: the operands of the
    // first part of every wavefront's rows come first.
    auto unit_of = [&](int u) {
        const int h = u / G::AH, g = wave * G::AH + u % G::AH, o = g >> 1;
        return (o / G::MH * G::MT + h * G::MH + o % G::MH) * 2 + (g & 1);
    };
    auto aim = [&](int id) {
        int64_t xbase = 0;
        if constexpr (GROUPED) {
            GroupTile at;
            if (!group_tile_at<BM, BN>(a, first + 1, all, id, at)) return false;
            e = at.g.e;
            t0 = at.t0;
            n0 = at.n0;
            n1 = at.g.r1;
        } else {
            const TileAt at = tile_at<BM, BN>(a.mtiles, a.N, id);
            t0 = at.t0;
            n0 = at.n0;
            n1 = a.N;
        }
        if (!GROUPED || !a.row) xbase = n0;
        const int64_t rows = GROUPED && a.row ? a.X : n1 - n0;
        wp = a.w + ((size_t)e * a.mtiles + t0) * a.nb * kUnit;
        wbytes = buffer_bytes((int64_t)(a.mtiles - t0) * a.nb * kUnit);
        xp = a.x + xbase * a.ldx;
        xbytes = buffer_bytes((rows - 1) * a.ldx + a.nb * kB);
        sr = __builtin_amdgcn_make_buffer_rsrc((void*)(a.xs + xbase * a.ldxs), (short)0,
                                               buffer_bytes(((rows - 1) * a.ldxs + ((a.nb + 3) & ~3)) * 4), kQgRawBufferFlags);
        const int mblock = min((t0 * T + wm * (BM / WM)) / kB, a.mb - 1);
        vr = __builtin_amdgcn_make_buffer_rsrc((void*)(a.ws + ((size_t)e * a.mb + mblock) * a.nb), (short)0, a.nb * 4,
                                               kQgRawBufferFlags);
        auto from = [&](int c) {  // the row, from xbase on, that column c of the tile comes from
            const int n = min(n0 + c, n1 - 1);
            return (uint32_t)(GROUPED && a.row ? source_row(a, n) : n - n0);
        };
#pragma unroll
        for (int u = 0; u < G::AU; ++u)
            woff[u] = (uint32_t)min(unit_of(u) >> 1, a.mtiles - 1 - t0) * (uint32_t)a.nb * kUnit + lane * 16u;
#pragma unroll
        for (int u = 0; u < G::XU; ++u)
            xoff[u] = from((wave * G::XU + u) * 8 + (lane >> 3)) * (uint32_t)a.ldx + chunk * 16u;
        soff = from(wave % (BN / 64) * 64 + lane) * (uint32_t)a.ldxs * 4u;
        return true;
    };
    // Scales of the blocks 8 g .. + 7: the row scales four blocks to a load (wavefronts beyond
    // the units repeat some), and eight weight scales.
    auto fetch_scales = [&](int g) {
        uint8_t* S = sl + (g & 1) * G::SB;
        const int unit = wave % G::SU, c = min(g * 2 + unit / (BN / 64), (a.nb - 1) >> 2);
        lds_load(sr, S + unit * 1024, soff, c * 16);
        __builtin_amdgcn_raw_ptr_buffer_load_lds(vr, (lds_ptr)(S + G::SU * 1024 + mine * 256), 4, (lane & 7) * 4, g * 32, 0, 0);
    };
    // Load u of part `part` of K tile t: its share of the weights, of the first part the
    // activations too. Beyond the last tile every load is out of its buffer's bounds and reads
    // nothing, so that the loop needs no branch.
    constexpr int FIRST = G::AH + G::XU;  // loads of the first part
    auto fetch = [&](int t, int buf, int part, int u) {
        uint8_t* A = lds + buf * G::STAGE;
        if (u < G::AH) {
            const int v = part * G::AH + u;
            const __amdgpu_buffer_rsrc_t wr = __builtin_amdgcn_make_buffer_rsrc((void*)wp, (short)0, t < k1 ? wbytes : 0, kQgRawBufferFlags);
            lds_load(wr, A + unit_of(v) * 1024, woff[v], (2 * t + (unit_of(v) & 1)) * 1024);
        } else {
            const __amdgpu_buffer_rsrc_t xr = __builtin_amdgcn_make_buffer_rsrc((void*)xp, (short)0, t < k1 ? xbytes : 0, kQgRawBufferFlags);
            lds_load(xr, A + G::AB + (wave * G::XU + u - G::AH) * 1024, xoff[u - G::AH], t * kB);
        }
    };
    auto fetch_part = [&](int t, int buf, int part) {
#pragma unroll
        for (int u = 0; u < (part ? G::AH : FIRST); ++u) fetch(t, buf, part, u);
    };
    // What the first turns need.
    auto start = [&]() {
#pragma unroll
        for (int i = 0; i < NS; ++i) {
            if (i == 0 || (((k0 + i) & 7) == 0 && k0 + i < k1)) fetch_scales((k0 + i) >> 3);
            if (H == 2 || i < NS - 1) fetch_part(k0 + i, i, 0);
            if (H == 2 && i < NS - 1) fetch_part(k0 + i, i, 1);
        }
    };

    const int r = lane & 15, q = lane >> 4;
    qg_f4 acc[G::MT][G::CT];
    const int arow = wm * G::MT * kUnit + lane * 16;
    const int xrow = G::AB + (wn * G::CT * 16 + r) * 128;
    const int x0 = xrow + ((q ^ (r & 7)) * 16), x1 = xrow + (((4 + q) ^ (r & 7)) * 16);
    const int srow = (wn * G::CT * 16 + r) * 16;
    auto get = [](Op8& o, const uint8_t* p0, const uint8_t* p1) {
        o.h[0] = *reinterpret_cast<const qi4*>(p0);
        o.h[1] = *reinterpret_cast<const qi4*>(p1);
    };
    auto get_row = [&](Op8& o, int buf, int i) {
        const uint8_t* A = lds + buf * G::STAGE + arow + i * kUnit;
        get(o, A, A + 1024);
    };
    auto get_col = [&](Op8& o, int buf, int j) { get(o, lds + buf * G::STAGE + x0 + j * 2048, lds + buf * G::STAGE + x1 + j * 2048); };
    auto as = [](const Op8& o) {
        Op v;
        if constexpr (YT == QG_F32)
            v.set(o);
        else
            v = o;
        return v;
    };

    // The wavefronts work in two groups of four, one of each on every SIMD, that take turns:
    // while one multiplies a part of a K tile (its operands are in registers, but for the last
    // few, which are on their way), the other reads the operands of its next part from LDS. A
    // barrier ends each turn; the second group is a turn behind. So turn 2 H t + 2 h of the
    // first group reads part h of K tile t, the next one multiplies it, and the second group's
    // are one later. A part's place in its buffer is free when the second group has multiplied
    // it. The next loads to it go between the products of the first group one turn later, of
    // the second two. They have to be there before the first group's turn that reads them: at
    // the end of a turn before one, the first group has just multiplied and the second read, and each lets only
    // the loads sent after those be on their way.
    constexpr int U = G::AU + G::XU;
    Op fa[G::MH], fx[G::CT];
    float sx[G::CT], s[G::CT], w;
    // sums of the last products, not added yet
    constexpr int LATE = G::MH >= 4 ? 4 : 0;  // reads that may be on their way when a part's products begin
    constexpr int PRODUCTS = G::MH * G::CT, D = PRODUCTS < 3 ? PRODUCTS : 3;
    qg_f4 sum[D];
    auto turn_end = [&](auto reads, auto loads) {
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (decltype(reads)::value >= 0) asm volatile("s_waitcnt lgkmcnt(%0)" ::"n"(decltype(reads)::value) : "memory");
        if constexpr (decltype(loads)::value >= 0) asm volatile("s_waitcnt vmcnt(%0)" ::"n"(decltype(loads)::value) : "memory");
        asm volatile("s_barrier" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
    };
    // Adds the sums of the products that the part h before left over.
    auto flush = [&](int h) {
#pragma unroll
        for (int d = 0; d < D; ++d) {
            const int at = PRODUCTS - D + d;
            add_scaled(acc[h * G::MH + at / G::CT][at % G::CT], sum[at % D], sx[at % G::CT]);
        }
    };
    auto read = [&](int t, int buf, int h) {
        Op8 ra[G::MH], rx[G::CT];
        if (h == 0) {
#pragma unroll
            for (int j = 0; j < G::CT; ++j) get_col(rx[j], buf, j);
            const uint8_t* S = sl + ((t >> 3) & 1) * G::SB;
            const uint8_t* X = S + ((t >> 2) & 1) * (BN * 16) + srow + (t & 3) * 4;
#pragma unroll
            for (int j = 0; j < G::CT; ++j) s[j] = *reinterpret_cast<const float*>(X + j * 256);
            w = *reinterpret_cast<const float*>(S + G::SU * 1024 + mine * 256 + (t & 7) * 4);
        }
#pragma unroll
        for (int i = 0; i < G::MH; ++i) {
            if (2 * (G::MH - i) == LATE) __builtin_amdgcn_sched_barrier(0);
            get_row(ra[i], buf, h * G::MH + i);
        }
        flush(H - 1 - h);
        if (h == 0) {
#pragma unroll
            for (int j = 0; j < G::CT; ++j) fx[j] = as(rx[j]);
        }
#pragma unroll
        for (int i = 0; i < G::MH; ++i) fa[i] = as(ra[i]);
    };
    // The products of part h of tile t, and between them the loads that may go now.
    auto multiply = [&](int t, int buf, int h) {
        const bool here = H == 2 && h == 1;  // to this tile's first part, or to the last part of the one before
        const int to = here ? t + NS : t - 1 + NS, at_buf = here ? buf : buf ? buf - 1 : NS - 1;
        const int part = H == 2 ? 1 - h : 0, count = part ? G::AH : FIRST;
#pragma unroll
        for (int at = 0; at < PRODUCTS; ++at) {
            const qg_f4 now = block_sum(fa[at / G::CT], fx[at % G::CT]);
            if (at >= D) {
                const int b = at - D;
                add_scaled(acc[h * G::MH + b / G::CT][b % G::CT], sum[b % D], sx[b % G::CT]);
            }
            sum[at % D] = now;
            if (h == 0 && at == 0) {
#pragma unroll
                for (int j = 0; j < G::CT; ++j) sx[j] = s[j] * w;
            }
#pragma unroll
            for (int u = at * count / PRODUCTS; u < (at + 1) * count / PRODUCTS; ++u)
                fetch(to, at_buf, part, u);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    int id = blockIdx.x;
    if (!aim(id)) return;
    start();
    while (true) {
#pragma unroll
        for (int i = 0; i < G::MT; ++i)
#pragma unroll
            for (int j = 0; j < G::CT; ++j) acc[i][j] = qg_f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int d = 0; d < D; ++d) sum[d] = qg_f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < G::CT; ++j) sx[j] = 0.f;
        tile_sync<H == 2 ? FIRST : (NS - 2) * U>();
        auto turns = [&](auto behind) {
            constexpr bool BEHIND = decltype(behind)::value;
            int buf = 0;
            for (int t = k0; t < k1; ++t) {
                if (((t + NS) & 7) == 0 && t + NS < k1) fetch_scales((t + NS) >> 3);
                auto part = [&](auto which) {
                    constexpr int h = decltype(which)::value;
                    // loads sent after those that the next reading turn of the first group needs
                    constexpr int first = H == 2 ? U : (NS - 2) * U, second = H == 1 ? (NS - 3) * U : h ? G::AH : FIRST;
                    read(t, buf, h);
                    turn_end(number<LATE>{}, number<BEHIND ? second : -1>{});
                    multiply(t, buf, h);
                    turn_end(number<-1>{}, number<BEHIND ? -1 : first>{});
                };
                part(number<0>{});
                if constexpr (H == 2) part(number<1>{});
                buf = buf + 1 == NS ? 0 : buf + 1;
            }
        };
        if (wave >= 4) {
            asm volatile("s_barrier" ::: "memory");
            turns(std::true_type{});
        } else {
            turns(std::false_type{});
            asm volatile("s_barrier" ::: "memory");
        }
        flush(H - 1);
        const int m0 = (t0 + wm * G::MT) * 16 + q * 8, c0 = n0 + wn * G::CT * 16 + r;
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
            // next tile's turns would be one for its loads.)
            float sb[G::MT / 2][8];
#pragma unroll
            for (int c = 0; c < G::MT / 2; ++c) {
                row_bias(a, e, m0 + 32 * c, sb[c]);
#pragma unroll
                for (int i = 0; i < 8; ++i) asm volatile("" : "+v"(sb[c][i]));
            }
            const int rows = n1;
            id += gridDim.x;
            tile_sync<0>();  // the last tile's buffer has been read by all (and loads beyond it are done)
            const bool more = id < a.total && aim(id);
            if (more) start();
#pragma unroll
            for (int c = 0; c < G::MT / 2; ++c)
                store_pair<YT, G::CT>(a, acc[2 * c], acc[2 * c + 1], sb[c], m0 + 32 * c, c0, rows);
            if (!more) return;
        }
    }
}

// The partial sums of a split product added in order and stored: one wavefront per pair
// of a tile wavefront's products.
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
enum { FORM_STREAM, FORM_64, FORM_128, FORM_256 };
struct Plan {
    int form, tiles, splits, kper;
    size_t ws;
};

int64_t weight_tiles(int64_t M) { return qg::ceil_div(M, kPair) * 2; }

Plan plan(int64_t M, int64_t K, int64_t N, int y_type) {
    Plan p{};
    const int kt = (int)qg::ceil_div(K, kB);
    p.splits = 1;
    p.kper = kt;
    auto tiles = [&](int b) { return qg::ceil_div(M, b) * qg::ceil_div(N, b); };
    if (N <= 32) {
        p.form = FORM_STREAM;
        p.tiles = (int)weight_tiles(M);
        return p;
    }
    int side = 64;
    if (N > 64 && tiles(256) >= 192 && y_type != QG_F32)
        side = 256;
    else if (N > 64 && (tiles(128) >= 128 || kt >= 64))
        side = 128;
    p.tiles = (int)tiles(side);
    p.form = side == 256 ? FORM_256 : side == 64 ? FORM_64 : FORM_128;
    const int s = side == 256 ? 1 : std::min(256 / p.tiles, kt / (side == 128 ? 18 : 28));
    if (s > 1) {
        p.kper = (int)qg::ceil_div(kt, s);
        p.splits = (int)qg::ceil_div(kt, p.kper);
        p.ws = (size_t)p.splits * p.tiles * side * side * 4;
    }
    return p;
}

template <int YT, int BM, int BN, int WM, int WN, int NS, int H, bool SPLIT, bool GROUPED>
qg_status launch_tiles(const GArgs& a, const Plan& p, hipStream_t s) {
    typedef F8Tile<BM, BN, WM, WN, NS, H> G;
    constexpr int most = G::LDS + (GROUPED ? (QG_EXPERTS_MAX + 64) * 4 : 0);  // (one number, and whole 64s of experts)
    static_assert(most <= 160 * 1024, "LDS of a compute unit");
    const int lds = G::LDS + (GROUPED ? (1 + (a.E + 63) / 64 * 64) * 4 : 0);
    // a workgroup takes tile after tile, as many of them at a time as there is LDS for
    const int groups = SPLIT ? p.tiles : std::min(p.tiles, qg::device_cus() * (160 * 1024 / lds));
    static std::atomic<bool> done[64];
    const qg_status lst =
        allow_lds(reinterpret_cast<const void*>(&gemm_f8_tile_kernel<YT, BM, BN, WM, WN, NS, H, SPLIT, GROUPED>), most, done);
    if (lst) return lst;
    hipLaunchKernelGGL((gemm_f8_tile_kernel<YT, BM, BN, WM, WN, NS, H, SPLIT, GROUPED>), dim3(groups, p.splits),
                       dim3(64 * G::W), lds, s, a);
    qg_status st = qg::launch_status("qgemm_f8");
    if constexpr (SPLIT) {
        if (st) return st;
        hipLaunchKernelGGL((gemm_f8_join_kernel<YT, BM, BN, WM, WN>), dim3(p.tiles * G::W * (G::MT / 2)), dim3(64), 0, s,
                           a, p.tiles, p.splits);
        st = qg::launch_status("qgemm_f8 (join)");
    }
    return st;
}

template <int YT>
qg_status launch_gemm(const GArgs& a, const Plan& p, hipStream_t s) {
    const bool split = p.splits > 1;
    switch (p.form) {
        case FORM_64:
            return split ? launch_tiles<YT, 64, 64, 2, 4, 4, 1, true, false>(a, p, s)
                         : launch_tiles<YT, 64, 64, 2, 4, 4, 1, false, false>(a, p, s);
        case FORM_128:
            return split ? launch_tiles<YT, 128, 128, 2, 4, 4, 1, true, false>(a, p, s)
                         : launch_tiles<YT, 128, 128, 2, 4, 4, 1, false, false>(a, p, s);
        case FORM_256:
            if constexpr (YT != QG_F32) return launch_tiles<YT, 256, 256, 2, 4, 2, 2, false, false>(a, p, s);
    }
    if (a.N <= 16)
        hipLaunchKernelGGL((gemm_f8_stream_kernel<YT, 1, 8>), dim3(a.mtiles), dim3(512), 0, s, a);
    else
        hipLaunchKernelGGL((gemm_f8_stream_kernel<YT, 2, 8>), dim3(a.mtiles), dim3(512), 0, s, a);
    return qg::launch_status("qgemm_f8");
}

template <int YT>
qg_status launch_grouped(const GArgs& a, hipStream_t s) {
    const int64_t used = std::min(a.E, a.N);  // experts that can have rows
    const int64_t each = qg::ceil_div(a.N, used);
    Plan p{};
    p.splits = 1;
    p.kper = a.nb;
    auto tiles = [&](int bm, int bn) {
        return (int)((std::min<int64_t>(a.N, a.N / bn + used)) * qg::ceil_div(a.mtiles * 16, bm));
    };
    GArgs b = a;
    if (each <= 32) {
        const dim3 g(a.mtiles, (unsigned)used);
        if (each <= 12)
            hipLaunchKernelGGL((gemm_f8_stream_kernel<YT, 1, 8>), g, dim3(512), 0, s, a);
        else
            hipLaunchKernelGGL((gemm_f8_stream_kernel<YT, 2, 8>), g, dim3(512), 0, s, a);
        return qg::launch_status("qgemm_f8_grouped");
    }
    if (each <= 96) {
        b.total = p.tiles = tiles(64, 64);
        return launch_tiles<YT, 64, 64, 2, 4, 4, 1, false, true>(b, p, s);
    }
    b.total = p.tiles = tiles(128, 128);
    return launch_tiles<YT, 128, 128, 2, 4, 4, 1, false, true>(b, p, s);
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
    const int64_t quads = (int64_t)a.N * a.quads;
    if (quads >= 16384)
        hipLaunchKernelGGL((quantize_f8_kernel<XT, GATED, 4>), dim3((unsigned)std::min<int64_t>(qg::ceil_div(quads, 16), 1 << 22)), dim3(256), 0, s, a);
    else
        hipLaunchKernelGGL((quantize_f8_kernel<XT, GATED, 1>), dim3((unsigned)qg::ceil_div(quads, 4)), dim3(256), 0, s, a);
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
