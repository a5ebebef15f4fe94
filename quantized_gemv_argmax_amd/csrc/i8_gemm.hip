// Int8 products with a scale per weight row and per activation row, for gfx950:
// the load-time layout of the weights, the row quantizer and the product.
//
//   y[n, m] = x_scale[n] * w_scale[m] * sum_k xq[n, k] * wq[m, k]  (+ bias[m])
//
// The dotLLM README's integer path quantizes activations per block; one scale per
// row instead lets the integer sum run over all of K on the int8 matrix cores
// (16 x 16 x 64, twice the fp16 rate) with the scales applied once, in the
// epilogue. Integer sums are exact, so every split of K gives the same bits.
#include <algorithm>
#include <atomic>
#include <climits>

#include "qg_device.h"
#include "qg_host.h"

namespace {

typedef int qi4 __attribute__((ext_vector_type(4)));

constexpr int T = QG_TILE_ROWS;
constexpr int kKB = 64;           // k per matrix-core operand
constexpr int kTileB = T * kKB;   // bytes of one operand (16 rows x 64 k)
constexpr int kWalkBlocks = 64;   // k blocks of the walk form (K <= 4096)
constexpr int kWalkGroups = 512;  // its workgroups

// ---------------------------------------------------------------- weight layout
__global__ __launch_bounds__(256) void pack_i8_kernel(const int8_t* __restrict__ src, int64_t ldw,
                                                      uint4* __restrict__ dst, int64_t M, int K, int nb,
                                                      int64_t units) {
    const int64_t stride = (int64_t)gridDim.x * 256;
    for (int64_t u = (int64_t)blockIdx.x * 256 + threadIdx.x; u < units; u += stride) {
        const int l = (int)(u & 63);
        const int64_t tb = u >> 6;
        const int64_t row = tb / nb * T + (l & 15);
        const int k0 = (int)(tb % nb) * kKB + (l >> 4) * 16;
        union {
            uint4 v;
            int8_t b[16];
        } o;
        o.v = make_uint4(0, 0, 0, 0);
        if (row < M) {
            typedef uint32_t vec __attribute__((ext_vector_type(4), aligned(1)));  // rows start anywhere
            const int8_t* p = src + row * ldw + k0;
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
template <int XT>
struct XVec;  // elements per 16-byte vector and their conversion to fp32
template <>
struct XVec<QG_F32> {
    typedef float E;
    typedef uint32_t V __attribute__((ext_vector_type(4), aligned(4)));
    static constexpr int N = 4;
    QG_DEV static float get(const uint4& v, int i) { return __builtin_bit_cast(float, (&v.x)[i]); }
    QG_DEV static float one(E e) { return e; }
};
template <>
struct XVec<QG_F16> {
    typedef uint16_t E;
    typedef uint32_t V __attribute__((ext_vector_type(4), aligned(2)));
    static constexpr int N = 8;
    QG_DEV static float get(const uint4& v, int i) {
        return (i & 1) ? qg_half_hi((&v.x)[i >> 1]) : qg_half_lo((&v.x)[i >> 1]);
    }
    QG_DEV static float one(E e) { return qg_half_lo(e); }
};
template <>
struct XVec<QG_BF16> {
    typedef uint16_t E;
    typedef uint32_t V __attribute__((ext_vector_type(4), aligned(2)));
    static constexpr int N = 8;
    QG_DEV static float get(const uint4& v, int i) {
        const uint32_t w = (&v.x)[i >> 1];
        return __builtin_bit_cast(float, (i & 1) ? (w & 0xffff0000u) : (w << 16));
    }
    QG_DEV static float one(E e) { return __builtin_bit_cast(float, (uint32_t)e << 16); }
};

// The 16-byte vector i of a row of K elements, zeros beyond K. Rows start at any
// element: full vectors are one load whatever their alignment.
template <int XT>
QG_DEV uint4 row_vec(const typename XVec<XT>::E* p, int K, int i) {
    typedef typename XVec<XT>::E E;
    typedef typename XVec<XT>::V vec;
    constexpr int N = XVec<XT>::N;
    const int k0 = i * N;
    if (k0 + N <= K) {
        const vec v = *reinterpret_cast<const vec*>(p + k0);
        return make_uint4(v.x, v.y, v.z, v.w);
    }
    union {
        uint4 v;
        E e[N];
    } o;
    o.v = make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int e = 0; e < N; ++e)
        if (k0 + e < K) o.e[e] = p[k0 + e];
    return o.v;
}

// x / d rounded to the nearest integer, ties to even, decided on the exact
// quotient. r = rint(x * inv) is off by at most one step, and only where the
// product lies near a half; there the remainder x - r d is exact in fp32 (it is a
// multiple of half of d's last place below 2^24 of them), so comparing it with d/2
// decides.
QG_DEV int quant1(float x, float d, float inv) {
    const float t = x * inv;
    float r = rintf(t);
    if (fabsf(t - r) > 0.4999f) {
        const float e = __builtin_fmaf(-r, d, x);
        const float e2 = fabsf(e) * 2.f;
        if (e2 > d || (e2 == d && (((int)r) & 1))) r += (e > 0.f) ? 1.f : -1.f;
    }
    return (int)fminf(fmaxf(r, -127.f), 127.f);
}

template <int XT>
QG_DEV void store_q(int8_t* q, int i, const uint4& v, float s, float d, float inv, bool ok) {
    constexpr int N = XVec<XT>::N;
    uint32_t w[N / 4];
#pragma unroll
    for (int c = 0; c < N / 4; ++c) {
        w[c] = 0;
        if (ok)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                w[c] |= ((uint32_t)quant1(XVec<XT>::get(v, 4 * c + e) * s, d, inv) & 255u) << (8 * e);
    }
    if constexpr (N == 4)
        reinterpret_cast<uint32_t*>(q)[i] = w[0];
    else
        reinterpret_cast<uint2*>(q)[i] = make_uint2(w[0], w[1]);
}

// One workgroup of NT threads per row, bound by HBM where there are rows enough (4096 x
// 18944 bf16: 233 MB in 41 us, 5.7 TB/s; one row of 3584: 2.8 us, its launch and one
// round trip). The row stays in registers between the maximum and the rounding where
// NT threads hold it in R vectors each; a longer one (R == 0) is read twice. Few vectors
// a thread leave room for more rows in flight: 18944 bf16 in 5 vectors of 512 threads
// takes 41 us, in 10 of 256 57; short rows take one wavefront (4096 x 512 bf16: 5.0 us,
// with 256 threads 6.6).
template <int XT, int NT, int R>
__global__ __launch_bounds__(NT) void quantize_i8_kernel(const void* __restrict__ x, int64_t ldx, int K,
                                                         int8_t* __restrict__ q, int64_t ldq,
                                                         float* __restrict__ scale) {
    typedef typename XVec<XT>::E E;
    constexpr int N = XVec<XT>::N;
    __shared__ uint32_t red[NT / 64];
    const int64_t n = blockIdx.x;
    const int tid = threadIdx.x;
    const E* p = reinterpret_cast<const E*>(x) + n * ldx;
    int8_t* o = q + n * ldq;
    const int nv = (K + kKB - 1) / kKB * (kKB / N);  // vectors, the zero padding included

    // the largest |x| by its bits: above every finite value an infinity, above it a NaN
    uint4 v[R ? R : 1];
    uint32_t mx = 0;
    auto peak = [&](const uint4& u) {
#pragma unroll
        for (int e = 0; e < N; ++e)
            mx = max(mx, __builtin_bit_cast(uint32_t, XVec<XT>::get(u, e)) & 0x7fffffffu);
    };
    if constexpr (R > 0) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            v[r] = make_uint4(0, 0, 0, 0);
            if (tid + r * NT < nv) v[r] = row_vec<XT>(p, K, tid + r * NT);
        }
#pragma unroll
        for (int r = 0; r < R; ++r) peak(v[r]);
    } else {
        for (int i = tid; i < nv; i += NT) peak(row_vec<XT>(p, K, i));
    }
#pragma unroll
    for (int m = 32; m; m >>= 1) mx = max(mx, (uint32_t)__shfl_xor((int)mx, m));
    if ((tid & 63) == 0) red[tid >> 6] = mx;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < NT / 64; ++w) mx = max(mx, red[w]);

    const bool finite = mx < 0x7f800000u;
    const float d0 = finite ? __builtin_bit_cast(float, mx) / 127.f : __builtin_nanf("");
    const bool ok = d0 > 0.f;
    // tiny scales: x and d scaled alike (exactly), so that 1/d stays finite and
    // remainders stay normal
    const float s = d0 < 0x1p-90f ? 0x1p60f : 1.f;
    const float d = ok ? d0 * s : 1.f;
    const float inv = 1.f / d;
    if (tid == 0) scale[n] = d0;
    if constexpr (R > 0) {
#pragma unroll
        for (int r = 0; r < R; ++r)
            if (tid + r * NT < nv) store_q<XT>(o, tid + r * NT, v[r], s, d, inv, ok);
    } else {
        for (int i = tid; i < nv; i += NT) store_q<XT>(o, i, row_vec<XT>(p, K, i), s, d, inv, ok);
    }
}

// ---------------------------------------------------------------- product
struct GArgs {
    const uint8_t* w;
    const float* ws;
    const int8_t* x;
    int64_t ldx;
    const float* xs;
    const float* bias;
    void* Y;
    int64_t ldy;
    qi4* part;           // partial sums of a product split along K
    int32_t M, N, nb;    // nb: k blocks of 64
    int32_t mtiles;      // 16-row tiles of W
    int32_t kper;        // K tiles (two blocks) of a split
    int32_t total;       // tiles of Y
};

// Written as one operation, which rounds the product and the bias together: left as a
// product and a sum, their rounding would be the compiler's choice, form by form.
QG_DEV float scaled(int acc, float xs, float ws, float b) { return __builtin_fmaf((float)acc, xs * ws, b); }

template <int YT>
QG_DEV uint32_t pack2(float lo, float hi) {
    // (round to nearest even, a NaN stays one)
    typedef float f2 __attribute__((ext_vector_type(2)));
    typedef _Float16 h2 __attribute__((ext_vector_type(2)));
    typedef __bf16 b2 __attribute__((ext_vector_type(2)));
    const f2 v = {lo, hi};
    if constexpr (YT == QG_F16)
        return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, h2));
    else
        return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, b2));
}

// C (4 or 8) consecutive outputs from element `at` of Y on, `count` of them inside
// the row (rows are at least four elements aligned).
template <int YT, int C>
QG_DEV void store_row(void* Y, int64_t at, const float (&y)[C], int count) {
    if constexpr (YT == QG_F32) {
        float* p = reinterpret_cast<float*>(Y) + at;
        if (count >= C) {
#pragma unroll
            for (int c = 0; c < C / 4; ++c)
                reinterpret_cast<float4*>(p)[c] = make_float4(y[4 * c], y[4 * c + 1], y[4 * c + 2], y[4 * c + 3]);
        } else {
#pragma unroll
            for (int e = 0; e < C; ++e)
                if (e < count) p[e] = y[e];
        }
    } else {
        uint16_t* p = reinterpret_cast<uint16_t*>(Y) + at;
        uint32_t h[C / 2];
#pragma unroll
        for (int e = 0; e < C / 2; ++e) h[e] = pack2<YT>(y[2 * e], y[2 * e + 1]);
        if (count >= C) {
            // (rows are 8 bytes aligned; one store of 16 all the same)
            typedef uint32_t vec __attribute__((ext_vector_type(C / 2), aligned(8)));
            vec v;
#pragma unroll
            for (int e = 0; e < C / 2; ++e) v[e] = h[e];
            *reinterpret_cast<vec*>(p) = v;
        } else {
#pragma unroll
            for (int e = 0; e < C; ++e)
                if (e < count) p[e] = (uint16_t)(h[e >> 1] >> (16 * (e & 1)));
        }
    }
}

// The scales (and biases) of C consecutive weight rows from m on, rows beyond M
// repeating the last one.
template <int C>
QG_DEV void row_scales(const GArgs& a, int m, float (&sw)[C], float (&sb)[C]) {
#pragma unroll
    for (int e = 0; e < C; ++e) {
        const int r = min(m + e, a.M - 1);
        sw[e] = a.ws[r];
        sb[e] = a.bias ? a.bias[r] : 0.f;
    }
}

// A lane's four sums of one 16 x 16 product: rows m .. m + 3 of column n.
template <int YT>
QG_DEV void store_quad(const GArgs& a, const qi4& s, int m, int n) {
    if (n >= a.N || m >= a.M) return;
    float sw[4], sb[4], y[4];
    row_scales(a, m, sw, sb);
    const float xs = a.xs[n];
#pragma unroll
    for (int e = 0; e < 4; ++e) y[e] = scaled(s[e], xs, sw[e], sb[e]);
    store_row<YT>(a.Y, n * a.ldy + m, y, a.M - m);
}

// ---------------------------------------------------------------- few columns
// One 16-row tile and NB blocks of 16 columns per workgroup; its KW wavefronts take
// pairs of k blocks in turn, and their integer sums meet in LDS. The weights go from
// memory straight to the operand registers, in the packed order; a pair's two column
// operands are the halves of 128 bytes of a row, one cache line (block by block over
// the wavefronts: 30000 x 6000 by 16 columns 44.2 us, in pairs 38; 3584 x 18944 by 16
// 19.1 and 17). For few tiles, where it is bound by latency (4608 x 3584 by 4 columns:
// 5.7 us for 16.6 MB; 16 instead of 8 wavefronts: 6.4), and for long K, where the
// columns, read from L2 by every tile, weigh as much as the weights.
template <int YT, int NB, int KW>
__global__ __launch_bounds__(64 * KW) void gemm_i8_stream_kernel(GArgs a) {
    __shared__ qi4 part[KW][NB][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int t = blockIdx.x;
    const uint8_t* w = a.w + ((size_t)t * a.nb) * kTileB + lane * 16;
    const int8_t* xr[NB];
#pragma unroll
    for (int c = 0; c < NB; ++c)  // columns beyond N read the last one; their sums are not stored
        xr[c] = a.x + (int64_t)min(16 * c + (lane & 15), a.N - 1) * a.ldx + (lane >> 4) * 16;
    qi4 acc[NB];
#pragma unroll
    for (int c = 0; c < NB; ++c) acc[c] = qi4{0, 0, 0, 0};
    qi4 wv[2][2], xv[2][2][NB];  // [pair in flight][block]
    auto load = [&](int p, int b, int count) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
            if (h < count) {
                wv[p][h] = __builtin_nontemporal_load(reinterpret_cast<const qi4*>(w + (size_t)(b + h) * kTileB));
#pragma unroll
                for (int c = 0; c < NB; ++c) xv[p][h][c] = *reinterpret_cast<const qi4*>(xr[c] + (b + h) * kKB);
            }
    };
    auto mma = [&](int p, int count) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
            if (h < count)
#pragma unroll
                for (int c = 0; c < NB; ++c)
                    acc[c] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wv[p][h], xv[p][h][c], acc[c], 0, 0, 0);
    };
    const int pairs = a.nb / 2;
    int b = wave;
    for (; b + KW < pairs; b += 2 * KW) {
        load(0, 2 * b, 2);
        load(1, 2 * (b + KW), 2);
        mma(0, 2);
        mma(1, 2);
    }
    // what is left: a pair, and for one wavefront the odd block
    const bool odd = (a.nb & 1) && wave == KW - 1;
    if (b < pairs) load(0, 2 * b, 2);
    if (odd) load(1, a.nb - 1, 1);
    if (b < pairs) mma(0, 2);
    if (odd) mma(1, 1);
#pragma unroll
    for (int c = 0; c < NB; ++c) part[wave][c][lane] = acc[c];
    __syncthreads();
    if (wave < NB) {
        const int c = wave;
        qi4 s = part[0][c][lane];
#pragma unroll
        for (int k = 1; k < KW; ++k) s += part[k][c][lane];
        store_quad<YT>(a, s, t * T + (lane >> 4) * 4, 16 * c + (lane & 15));
    }
}

// The same for many weight tiles and K <= 4096, bound by HBM (152064 x 3584 by 16 columns:
// 555 MB in 95 us, 5.8 TB/s): each wavefront keeps its k blocks of the columns in
// registers (up to XR of them) while its workgroup walks over tiles, so that only
// weights are loaded, a tile ahead. Sums of alternate tiles meet in alternate LDS
// buffers, one barrier a tile; the wavefronts take turns at adding them.
template <int YT, int NB>
__global__ __launch_bounds__(256) void gemm_i8_walk_kernel(GArgs a) {
    constexpr int KW = 4, XR = kWalkBlocks / KW;
    __shared__ qi4 part[2][KW][NB][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int mine = (a.nb - wave + KW - 1) / KW;  // blocks wave, wave + KW, ..
    qi4 wv[XR], xv[XR][NB];
    auto load = [&](int t) {
        const uint8_t* w = a.w + ((size_t)t * a.nb + wave) * kTileB + lane * 16;
#pragma unroll
        for (int i = 0; i < XR; ++i)
            if (i < mine) wv[i] = __builtin_nontemporal_load(reinterpret_cast<const qi4*>(w + (size_t)i * KW * kTileB));
    };
    int t = blockIdx.x;
    load(t);
#pragma unroll
    for (int c = 0; c < NB; ++c) {  // columns beyond N read the last one; their sums are not stored
        const int8_t* x = a.x + (int64_t)min(16 * c + (lane & 15), a.N - 1) * a.ldx + (lane >> 4) * 16 + wave * kKB;
#pragma unroll
        for (int i = 0; i < XR; ++i)
            if (i < mine) xv[i][c] = *reinterpret_cast<const qi4*>(x + i * KW * kKB);
    }
    for (int turn = 0; t < a.mtiles; ++turn) {
        qi4 acc[NB];
#pragma unroll
        for (int c = 0; c < NB; ++c) acc[c] = qi4{0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < XR; ++i)
            if (i < mine)
#pragma unroll
                for (int c = 0; c < NB; ++c)
                    acc[c] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wv[i], xv[i][c], acc[c], 0, 0, 0);
        const int next = t + gridDim.x;
        if (next < a.mtiles) load(next);
        const int buf = turn & 1;
#pragma unroll
        for (int c = 0; c < NB; ++c) part[buf][wave][c][lane] = acc[c];
        // (the loads of the next tile stay on their way across the barrier)
        asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
#pragma unroll
        for (int c = 0; c < NB; ++c)
            if ((turn * NB + c) % KW == wave) {
                qi4 s = part[buf][0][c][lane];
#pragma unroll
                for (int k = 1; k < KW; ++k) s += part[buf][k][c][lane];
                store_quad<YT>(a, s, t * T + (lane >> 4) * 4, 16 * c + (lane & 15));
            }
        t = next;
    }
}

// ---------------------------------------------------------------- many columns
// Y in tiles of BM weight rows x BN columns, one at a time per workgroup of WM x WN
// wavefronts, K in tiles of 128 bytes through NS LDS buffers.
template <int BM, int BN, int WM, int WN, int NS_>
struct Tile {
    static constexpr int NS = NS_;
    static constexpr int W = WM * WN;
    static constexpr int MT = BM / WM / 16, CT = BN / WN / 16;    // 16 x 16 products of a wavefront
    static constexpr int AB = BM * 128, XB = BN * 128, STAGE = AB + XB, LDS = NS * STAGE;
    static constexpr int AU = AB / 1024 / W, XU = XB / 1024 / W;  // 1 KB loads of a wavefront
    static_assert(MT % 2 == 0 && AU * 1024 * W == AB && XU * 1024 * W == XB, "tile does not split evenly");
};

typedef __attribute__((address_space(3))) void* lds_ptr;

// 1 KB from memory to LDS, 16 bytes a lane, lanes in order from dst on.
QG_DEV void lds_load(const __amdgpu_buffer_rsrc_t r, uint8_t* dst, uint32_t voff, int soff) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_ptr)dst, 16, voff, soff, 0, 0);
}

// All but the last LATER of every wavefront's loads have arrived and its LDS reads are
// done, for all wavefronts of the workgroup.
template <int LATER>
QG_DEV void tile_sync() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(LATER) : "memory");
}

// Order of a half tile's instructions: its LDS reads, then its loads, each followed by an
// even share of the products, nothing moved across its end. (Left to itself the compiler
// bunches the reads in front of their first use: 546 us instead of 523 for 37888 x 3584
// by 4096 columns.)
template <int READS, int LOADS, int PRODUCTS>
QG_DEV void interleave() {
    constexpr int share = PRODUCTS / (READS + LOADS) > 0 ? PRODUCTS / (READS + LOADS) : 1;
#pragma unroll
    for (int i = 0; i < READS; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);  // LDS read
        __builtin_amdgcn_sched_group_barrier(0x8, share, 0);  // matrix product
    }
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x20, 1, 0);  // load
        __builtin_amdgcn_sched_group_barrier(0x8, share, 0);
    }
    __builtin_amdgcn_sched_group_barrier(0x8, PRODUCTS, 0);
    __builtin_amdgcn_sched_barrier(0);
}

// Outputs of a wavefront's accumulators. Product i of a pair (2c, 2c + 1) holds in its
// row 4 q + e the weight row 32 c + 8 q + 4 (i % 2) + e, so a lane's pair is eight
// consecutive outputs and four lanes' pairs are 32.
template <int CT>
struct PairScales {
    float sw[8], sb[8], xs[CT];
    QG_DEV PairScales(const GArgs& a, int m, int n0) {
        row_scales(a, m, sw, sb);
#pragma unroll
        for (int j = 0; j < CT; ++j) xs[j] = a.xs[min(n0 + 16 * j, a.N - 1)];
    }
};
template <int YT, int CT>
QG_DEV void store_pair(const GArgs& a, const qi4 (&lo)[CT], const qi4 (&hi)[CT], const PairScales<CT>& p, int m,
                       int n0) {
    const int count = a.M - m;
    if (count <= 0) return;
#pragma unroll
    for (int j = 0; j < CT; ++j) {
        const int n = n0 + 16 * j;
        if (n < a.N) {
            float y[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                y[e] = scaled(lo[j][e], p.xs[j], p.sw[e], p.sb[e]);
                y[4 + e] = scaled(hi[j][e], p.xs[j], p.sw[4 + e], p.sb[4 + e]);
            }
            store_row<YT>(a.Y, n * a.ldy + m, y, count);
        }
    }
}

// Tile of workgroup id: eight XCDs take the tiles in eight contiguous runs, and in a
// run groups of eight tile rows walk the columns together, so that the tiles an XCD
// works on at a time share their weights and activations in its L2.
struct TileAt {
    int t0, n0;  // first 16-row tile, first column
};
template <int BM, int BN>
QG_DEV TileAt tile_at(const GArgs& a, int id) {
    const int mts = (a.mtiles * 16 + BM - 1) / BM, nts = (a.N + BN - 1) / BN;
    const int total = mts * nts, q = total / 8, r = total % 8, x = id % 8;
    id = x * q + min(x, r) + id / 8;
    constexpr int GM = 8;
    const int per = GM * nts, grp = id / per, rem = id - grp * per;
    const int gm = min(GM, mts - grp * GM);
    return {(grp * GM + rem % gm) * (BM / 16), rem / gm * BN};
}

template <int YT, int BM, int BN, int WM, int WN, int NS, bool SPLIT>
__global__ __launch_bounds__(64 * WM * WN) void gemm_i8_tile_kernel(GArgs a) {
    typedef Tile<BM, BN, WM, WN, NS> G;
    extern __shared__ __align__(1024) uint8_t lds[];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int k0 = SPLIT ? blockIdx.y * a.kper : 0;
    const int k1 = SPLIT ? min((a.nb + 1) / 2, k0 + a.kper) : (a.nb + 1) / 2;

    // Loads: rows and tiles beyond the operands repeat the last ones (their sums are
    // not stored). Weights arrive in the packed order. Activations: eight lanes per row
    // of 128 bytes, the 16-byte chunk c of row r at place c ^ (r % 8), which spreads
    // the operand reads over the banks.
    const int chunk = (lane & 7) ^ (lane >> 3);
    // an odd last block: its row ends after half of the 128 bytes, the lanes of the
    // other half read the first one again (and no product uses what they read)
    const uint32_t back = chunk >= 4 ? 64u : 0u;
    __amdgpu_buffer_rsrc_t wr, xr;
    uint32_t woff[G::AU], xoff[G::XU];
    int t0, n0;
    auto aim = [&](int id) {
        const TileAt at = tile_at<BM, BN>(a, id);
        t0 = at.t0;
        n0 = at.n0;
        wr = __builtin_amdgcn_make_buffer_rsrc((void*)(a.w + (size_t)t0 * a.nb * kTileB), (short)0,
                                               (int)min((int64_t)(a.mtiles - t0) * a.nb * kTileB, (int64_t)INT32_MAX),
                                               kQgRawBufferFlags);
        xr = __builtin_amdgcn_make_buffer_rsrc((void*)(a.x + n0 * a.ldx), (short)0,
                                               (int)min((int64_t)(a.N - 1 - n0) * a.ldx + a.nb * kKB, (int64_t)INT32_MAX),
                                               kQgRawBufferFlags);
#pragma unroll
        for (int u = 0; u < G::AU; ++u)
            woff[u] = (uint32_t)min((wave * G::AU + u) >> 1, a.mtiles - 1 - t0) * (uint32_t)a.nb * kTileB + lane * 16u;
#pragma unroll
        for (int u = 0; u < G::XU; ++u)
            xoff[u] = (uint32_t)min((wave * G::XU + u) * 8 + (lane >> 3), a.N - 1 - n0) * (uint32_t)a.ldx + chunk * 16u;
    };
    auto fetch = [&](int t, int buf) {
        uint8_t* A = lds + buf * G::STAGE;
        uint8_t* X = A + G::AB;
#pragma unroll
        for (int u = 0; u < G::AU; ++u) {
            const int unit = wave * G::AU + u;
            lds_load(wr, A + unit * 1024, woff[u], min(2 * t + (unit & 1), a.nb - 1) * kTileB);
        }
        const uint32_t sub = 2 * t + 1 < a.nb ? 0u : back;
#pragma unroll
        for (int u = 0; u < G::XU; ++u) lds_load(xr, X + (wave * G::XU + u) * 1024, xoff[u] - sub, t * 128);
    };
    auto start = [&]() {
#pragma unroll
        for (int i = 0; i < NS; ++i)
            if (k0 + i < k1) fetch(k0 + i, i);
    };

    const int wm = wave % WM, wn = wave / WM;
    const int r = lane & 15, q = lane >> 4;
    qi4 acc[G::MT][G::CT];
    const int arow = (wm * G::MT + (r >> 3)) * 2048 + (q * 16 + ((r >> 2) & 1) * 8 + (r & 3)) * 16;
    const int xrow = (wn * G::CT * 16 + r) * 128;
    auto frags = [&](int buf, int h, qi4(&fa)[G::MT], qi4(&fx)[G::CT]) {
        const uint8_t* A = lds + buf * G::STAGE + arow + h * 1024;
        const uint8_t* X = lds + buf * G::STAGE + G::AB + xrow + (((h * 4 + q) ^ (r & 7)) * 16);
#pragma unroll
        for (int j = 0; j < G::CT; ++j) fx[j] = *reinterpret_cast<const qi4*>(X + j * 2048);
#pragma unroll
        for (int i = 0; i < G::MT; ++i) fa[i] = *reinterpret_cast<const qi4*>(A + (i >> 1) * 4096 + (i & 1) * 64);
    };
    auto mma = [&](const qi4(&fa)[G::MT], const qi4(&fx)[G::CT]) {
#pragma unroll
        for (int i = 0; i < G::MT; ++i)
#pragma unroll
            for (int j = 0; j < G::CT; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fa[i], fx[j], acc[i][j], 0, 0, 0);
    };

    // One barrier per K tile, between its two halves: the second half's operands are in
    // registers then, so its buffer can be refilled, with the tile NS later; the next
    // tile's loads, sent NS - 1 tiles earlier, have arrived, those of the NS - 2 tiles
    // after it may still be on their way.
    // A workgroup with another tile to do sends that tile's first loads before it stores
    // this one's outputs.
    constexpr int U = G::AU + G::XU;
    int id = blockIdx.x;
    aim(id);
    start();
    while (true) {
#pragma unroll
        for (int i = 0; i < G::MT; ++i)
#pragma unroll
            for (int j = 0; j < G::CT; ++j) acc[i][j] = qi4{0, 0, 0, 0};
        qi4 a0[G::MT], x0[G::CT], a1[G::MT], x1[G::CT];
        if (k0 + NS <= k1)
            tile_sync<(NS - 1) * U>();
        else
            tile_sync<0>();
        frags(0, 0, a0, x0);
        int t = k0, buf = 0;
        auto next = [&](int i) { return i + 1 == NS ? 0 : i + 1; };
        for (; t + NS < k1; ++t, buf = next(buf)) {
            frags(buf, 1, a1, x1);
            mma(a0, x0);
            interleave<G::MT + G::CT, 0, G::MT * G::CT>();
            tile_sync<(NS - 2) * U>();
            __builtin_amdgcn_sched_barrier(0);
            frags(next(buf), 0, a0, x0);
            fetch(t + NS, buf);
            mma(a1, x1);
            interleave<G::MT + G::CT, U, G::MT * G::CT>();
        }
        for (; t + 1 < k1; ++t, buf = next(buf)) {
            frags(buf, 1, a1, x1);
            mma(a0, x0);
            tile_sync<0>();
            frags(next(buf), 0, a0, x0);
            mma(a1, x1);
        }
        frags(buf, 1, a1, x1);
        mma(a0, x0);
        const int m0 = (t0 + wm * G::MT) * 16 + q * 8, c0 = n0 + wn * G::CT * 16 + r;
        if constexpr (SPLIT) {
            if (2 * t + 1 < a.nb) mma(a1, x1);
            qi4* p = a.part + ((((size_t)blockIdx.y * gridDim.x + blockIdx.x) * G::W + wave) * (G::MT * G::CT)) * 64 + lane;
#pragma unroll
            for (int i = 0; i < G::MT; ++i)
#pragma unroll
                for (int j = 0; j < G::CT; ++j) p[(i * G::CT + j) * 64] = acc[i][j];
            return;
        } else {
            id += gridDim.x;
            const bool more = id < a.total;
            // (the scales first: waiting for them must not mean waiting for the loads)
            PairScales<G::CT> sc(a, m0, c0);
            if (more) {
                tile_sync<0>();
                aim(id);
                start();
            }
            if (2 * t + 1 < a.nb) mma(a1, x1);
#pragma unroll
            for (int c = 0; c < G::MT / 2; ++c) {
                if (c) row_scales(a, m0 + 32 * c, sc.sw, sc.sb);
                store_pair<YT, G::CT>(a, acc[2 * c], acc[2 * c + 1], sc, m0 + 32 * c, c0);
            }
            if (!more) return;
        }
    }
}

// The partial sums of a split product added and stored: one wavefront per pair of
// a tile wavefront's products.
template <int YT, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(64) void gemm_i8_join_kernel(GArgs a, int tiles, int splits) {
    typedef Tile<BM, BN, WM, WN, 2> G;
    const int lane = threadIdx.x;
    const int c = blockIdx.x % (G::MT / 2), wave = blockIdx.x / (G::MT / 2) % G::W;
    const int id = blockIdx.x / (G::MT / 2 * G::W);
    const TileAt at = tile_at<BM, BN>(a, id);
    const int wm = wave % WM, wn = wave / WM, r = lane & 15, q = lane >> 4;
    const qi4* p = a.part + (((size_t)id * G::W + wave) * (G::MT * G::CT) + 2 * c * G::CT) * 64 + lane;
    const size_t step = (size_t)tiles * G::W * (G::MT * G::CT) * 64;
    const int m = (at.t0 + wm * G::MT + 2 * c) * 16 + q * 8, n = at.n0 + wn * G::CT * 16 + r;
    const PairScales<G::CT> sc(a, m, n);  // (on their way while the sums are)
    qi4 lo[G::CT], hi[G::CT];
#pragma unroll
    for (int j = 0; j < G::CT; ++j) lo[j] = hi[j] = qi4{0, 0, 0, 0};
#pragma unroll 4
    for (int s = 0; s < splits; ++s, p += step)
#pragma unroll
        for (int j = 0; j < G::CT; ++j) {
            lo[j] += p[j * 64];
            hi[j] += p[(G::CT + j) * 64];
        }
    store_pair<YT, G::CT>(a, lo, hi, sc, m, n);
}

// ---------------------------------------------------------------- launches
// How a product runs: few columns stream the weights past them; else a tile form,
// perhaps split along K. 17 to 32 columns take tiles of 64 for K beyond the walk's
// (3584 x 18944 by 32: 19.7 us in 4 splits, streamed 26; 30000 x 6000 by 32: 42 and 61)
// unless the tiles are few (2000 x 8000 by 20: streamed 8.3, tiles of 64 in two splits 14.4).
// (These times and those below: calls in a graph, bf16 outputs, weights from memory.)
enum { FORM_STREAM, FORM_64, FORM_128_DEEP, FORM_128, FORM_256 };
struct Plan {
    int form, tiles, splits, kper;
    size_t ws;
};

// The largest tile that still gives most compute units one, larger tiles reading the
// operands less often (37888 x 3584 by 4096 columns: 485 us in tiles of 256, 548 in 128,
// 1054 in 64; 18944 x 3584 by 256: 33 us in 296 tiles of 128, 52 in 74 of 256; 1000 x 1000
// by 1000: 6.4 us in 256 tiles of 64, 8.3 in 64 of 128), but tiles of 128 where K is long
// (3584 x 18944 by 256: 36 us, tiles of 64 97). The rule does not see how full the last
// round of tiles of 256 is: in 1.1 rounds of them 4608 x 3584 by 4096 takes 86 us (tiles of
// 128: 76), 18944 x 3584 by 1024 89 (84), 37888 x 3584 by 512 105 (89) and by 300 97 (64).
// Tiles of 128 take three LDS buffers up to a workgroup per compute unit, two, with two
// workgroups per unit, beyond (296 tiles: 33 us, with three buffers 41; 144 tiles of
// 4608 x 3584 by 512: 28 us, with three 20).
// With fewer tiles than units a long K is split until about 256 workgroups share it,
// each keeping some K tiles to repay the second launch: 3584 x 18944 by 64 columns takes
// 20 us in 4 splits of tiles of 64 (1: 97, 3: 24, 8: 22), by 128 25 us in 8 of tiles of 128
// (6: 27). The least K tiles of a split, 28 and 18, were chosen with weights in the caches,
// where 4608 x 3584 by 64 takes 10.4 us whole, 10.2 in two; with weights from memory it
// takes 21 whole, 12 in two.
Plan plan(int64_t M, int64_t K, int64_t N) {
    Plan p{};
    const int kt = (int)qg::ceil_div(K, 2 * kKB);
    p.splits = 1;
    p.kper = kt;
    auto tiles = [&](int b) { return qg::ceil_div(M, b) * qg::ceil_div(N, b); };
    if (N <= 16 || (N <= 32 && (K <= kWalkBlocks * kKB || tiles(64) < 48))) {
        p.form = FORM_STREAM;
        p.tiles = (int)qg::ceil_div(M, T);
        return p;
    }
    int side = 64;
    if (N > 64 && tiles(256) >= 192)
        side = 256;
    else if (N > 64 && (tiles(128) >= 128 || kt >= 64))
        side = 128;
    p.tiles = (int)tiles(side);
    p.form = side == 256 ? FORM_256 : side == 64 ? FORM_64 : p.tiles > 256 ? FORM_128 : FORM_128_DEEP;
    const int s = side == 256 ? 1 : std::min(256 / p.tiles, kt / (side == 128 ? 18 : 28));
    if (s > 1) {
        p.kper = (int)qg::ceil_div(kt, s);
        p.splits = (int)qg::ceil_div(kt, p.kper);
        p.ws = (size_t)p.splits * p.tiles * side * side * 4;
    }
    return p;
}

// Allows a kernel more than 64 KB of LDS, once per device.
qg_status allow_lds(const void* f, int bytes, std::atomic<bool>* done) {
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return qg::fail(QG_ERR_DEVICE, "no current device");
    if (done[dev].load(std::memory_order_acquire)) return QG_OK;
    const hipError_t e = hipFuncSetAttribute(f, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != hipSuccess) return qg::fail(QG_ERR_DEVICE, "LDS size: %s", hipGetErrorString(e));
    done[dev].store(true, std::memory_order_release);
    return QG_OK;
}

template <int YT, int B, int WM, int WN, int NS, bool SPLIT>
qg_status launch_tiles(const GArgs& a, const Plan& p, hipStream_t s) {
    typedef Tile<B, B, WM, WN, NS> G;
    // tiles of 256: a workgroup per compute unit takes tile after tile (523 -> 512 us for
    // 37888 x 3584 by 4096 columns); smaller ones share a unit, which overlaps as much
    const int groups = B == 256 ? std::min(p.tiles, qg::device_cus()) : p.tiles;
    if constexpr (G::LDS > 65536) {
        static std::atomic<bool> done[64];
        const qg_status st =
            allow_lds(reinterpret_cast<const void*>(&gemm_i8_tile_kernel<YT, B, B, WM, WN, NS, SPLIT>), G::LDS, done);
        if (st) return st;
    }
    hipLaunchKernelGGL((gemm_i8_tile_kernel<YT, B, B, WM, WN, NS, SPLIT>), dim3(groups, p.splits), dim3(64 * G::W),
                       G::LDS, s, a);
    qg_status st = qg::launch_status("qgemm_i8");
    if constexpr (SPLIT) {
        if (st) return st;
        hipLaunchKernelGGL((gemm_i8_join_kernel<YT, B, B, WM, WN>), dim3(p.tiles * G::W * (G::MT / 2)), dim3(64), 0, s,
                           a, p.tiles, p.splits);
        st = qg::launch_status("qgemm_i8 (join)");
    }
    return st;
}

template <int YT>
qg_status launch_gemm(const GArgs& a, const Plan& p, hipStream_t s) {
    const bool split = p.splits > 1;
    switch (p.form) {
        case FORM_64: return split ? launch_tiles<YT, 64, 2, 2, 4, true>(a, p, s) : launch_tiles<YT, 64, 2, 2, 4, false>(a, p, s);
        case FORM_128_DEEP:
            return split ? launch_tiles<YT, 128, 2, 4, 3, true>(a, p, s) : launch_tiles<YT, 128, 2, 4, 3, false>(a, p, s);
        case FORM_128: return launch_tiles<YT, 128, 2, 4, 2, false>(a, p, s);
        case FORM_256: return launch_tiles<YT, 256, 2, 4, 2, false>(a, p, s);
    }
    // Few columns. The walk needs a tile for each of its workgroups, and K long enough
    // that the barrier of a tile does not show: 152064 x 3584 takes 96 us at 16 columns
    // and 104 at 32 (a tile per workgroup: 122 and 179), 4608 x 3584 at 4 columns 6.8
    // (5.9), 20000 x 512 at 10 columns 5.9 (4.3).
    const bool walk = a.mtiles >= kWalkGroups && a.nb >= 16 && a.nb <= kWalkBlocks;
    if (walk && a.N <= 16)
        hipLaunchKernelGGL((gemm_i8_walk_kernel<YT, 1>), dim3(kWalkGroups), dim3(256), 0, s, a);
    else if (walk)
        hipLaunchKernelGGL((gemm_i8_walk_kernel<YT, 2>), dim3(kWalkGroups), dim3(256), 0, s, a);
    else if (a.N <= 16)
        hipLaunchKernelGGL((gemm_i8_stream_kernel<YT, 1, 8>), dim3(a.mtiles), dim3(512), 0, s, a);
    else
        hipLaunchKernelGGL((gemm_i8_stream_kernel<YT, 2, 8>), dim3(a.mtiles), dim3(512), 0, s, a);
    return qg::launch_status("qgemm_i8");
}

int elem_bytes(int type) { return type == QG_F32 ? 4 : 2; }
bool known_type(int type) { return type == QG_F32 || type == QG_F16 || type == QG_BF16; }
bool overlap(const void* a, size_t na, const void* b, size_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + nb && y < x + na;
}

template <int XT>
void launch_quantize(const void* x, int64_t ldx, int64_t N, int K, int8_t* q, int64_t ldq, float* scale,
                     hipStream_t s) {
    const int nv = (int)qg::ceil_div(K, kKB) * (kKB / XVec<XT>::N);
    const dim3 g((unsigned)N);
    if (nv <= 256)
        hipLaunchKernelGGL((quantize_i8_kernel<XT, 64, 4>), g, dim3(64), 0, s, x, ldx, K, q, ldq, scale);
    else if (nv <= 512)
        hipLaunchKernelGGL((quantize_i8_kernel<XT, 256, 2>), g, dim3(256), 0, s, x, ldx, K, q, ldq, scale);
    else if (nv <= 1280)
        hipLaunchKernelGGL((quantize_i8_kernel<XT, 256, 5>), g, dim3(256), 0, s, x, ldx, K, q, ldq, scale);
    else if (nv <= 2560)
        hipLaunchKernelGGL((quantize_i8_kernel<XT, 512, 5>), g, dim3(512), 0, s, x, ldx, K, q, ldq, scale);
    else if (nv <= 5120)
        hipLaunchKernelGGL((quantize_i8_kernel<XT, 1024, 5>), g, dim3(1024), 0, s, x, ldx, K, q, ldq, scale);
    else
        hipLaunchKernelGGL((quantize_i8_kernel<XT, 1024, 0>), g, dim3(1024), 0, s, x, ldx, K, q, ldq, scale);
}

qg_status check_mk(int64_t M, int64_t K) {
    if (M < 1 || M > QG_I8_MAX_ROWS)
        return qg::fail(QG_ERR_SHAPE, "M=%lld not in [1, %d]", (long long)M, QG_I8_MAX_ROWS);
    if (K < 1 || K > QG_I8_MAX_K)
        return qg::fail(QG_ERR_SHAPE, "K=%lld not in [1, %d]", (long long)K, QG_I8_MAX_K);
    return QG_OK;
}

}  // namespace

extern "C" {

size_t qg_i8_bytes(int64_t M, int64_t K) {
    if (M < 1 || M > QG_I8_MAX_ROWS || K < 1 || K > QG_I8_MAX_K) return 0;
    return (size_t)qg::ceil_div(M, T) * (size_t)qg::ceil_div(K, kKB) * kTileB;
}

qg_status qg_pack_i8(const void* wq, int64_t ldw, void* dst, int64_t M, int64_t K, qg_stream_t stream) {
    qg::clear_error();
    if (!wq || !dst) return qg::fail(QG_ERR_NULL, "NULL pointer (wq, dst)");
    qg_status st = check_mk(M, K);
    if (st) return st;
    if (ldw < K || ldw > ((int64_t)1 << 40) / M) return qg::fail(QG_ERR_SHAPE, "ldw=%lld not in [K, 2^40 / M]", (long long)ldw);
    if (!qg::aligned16(dst)) return qg::fail(QG_ERR_ALIGN, "dst not 16-byte aligned");
    const size_t n = qg_i8_bytes(M, K);
    if (overlap(wq, (size_t)(M - 1) * ldw + K, dst, n)) return qg::fail(QG_ERR_SHAPE, "wq and dst overlap");
    st = qg::check_device();
    if (st) return st;
    const int64_t units = (int64_t)(n / 16);
    const unsigned g = (unsigned)std::min<int64_t>(qg::ceil_div(units, 256), 65536);
    hipLaunchKernelGGL(pack_i8_kernel, dim3(g), dim3(256), 0, (hipStream_t)stream, (const int8_t*)wq, ldw, (uint4*)dst,
                       M, (int)K, (int)qg::ceil_div(K, kKB), units);
    return qg::launch_status("qg_pack_i8");
}

qg_status qg_quantize_i8_rows(const void* x, int x_type, int64_t ldx, int64_t N, int64_t K, void* q, int64_t ldq,
                              float* scale, qg_stream_t stream) {
    qg::clear_error();
    if (!x || !q || !scale) return qg::fail(QG_ERR_NULL, "NULL pointer (x, q, scale)");
    if (!known_type(x_type)) return qg::fail(QG_ERR_SHAPE, "x_type=%d unknown", x_type);
    if (N < 1 || N > QG_I8_MAX_ROWS)
        return qg::fail(QG_ERR_SHAPE, "N=%lld not in [1, %d]", (long long)N, QG_I8_MAX_ROWS);
    if (K < 1 || K > QG_I8_MAX_K)
        return qg::fail(QG_ERR_SHAPE, "K=%lld not in [1, %d]", (long long)K, QG_I8_MAX_K);
    const int64_t kp = qg::ceil_div(K, kKB) * kKB, most = ((int64_t)1 << 40) / N;
    if (ldx < K || ldx > most) return qg::fail(QG_ERR_SHAPE, "ldx=%lld not in [K, 2^40 / N]", (long long)ldx);
    if (ldq < kp || ldq > most || ldq % 16)
        return qg::fail(QG_ERR_SHAPE, "ldq=%lld not a multiple of 16 in [%lld, 2^40 / N]", (long long)ldq, (long long)kp);
    const int eb = elem_bytes(x_type);
    if (reinterpret_cast<uintptr_t>(x) % eb) return qg::fail(QG_ERR_ALIGN, "x not aligned to its elements");
    if (!qg::aligned16(q)) return qg::fail(QG_ERR_ALIGN, "q not 16-byte aligned");
    if (reinterpret_cast<uintptr_t>(scale) & 3) return qg::fail(QG_ERR_ALIGN, "scale not 4-byte aligned");
    const size_t xb = ((size_t)(N - 1) * ldx + K) * eb, qb = (size_t)(N - 1) * ldq + kp;
    if (overlap(x, xb, q, qb) || overlap(x, xb, scale, (size_t)N * 4) || overlap(q, qb, scale, (size_t)N * 4))
        return qg::fail(QG_ERR_SHAPE, "x, q and scale overlap");
    qg_status st = qg::check_device();
    if (st) return st;
    hipStream_t s = (hipStream_t)stream;
    if (x_type == QG_F32)
        launch_quantize<QG_F32>(x, ldx, N, (int)K, (int8_t*)q, ldq, scale, s);
    else if (x_type == QG_F16)
        launch_quantize<QG_F16>(x, ldx, N, (int)K, (int8_t*)q, ldq, scale, s);
    else
        launch_quantize<QG_BF16>(x, ldx, N, (int)K, (int8_t*)q, ldq, scale, s);
    return qg::launch_status("qg_quantize_i8_rows");
}

size_t qgemm_i8_workspace_bytes(int64_t M, int64_t K, int64_t N) {
    if (!qg_i8_bytes(M, K) || N < 1 || N > QG_I8_MAX_ROWS || M * N > (int64_t)1 << 32) return 0;
    return plan(M, K, N).ws;
}

qg_status qgemm_i8(const void* w, const float* ws, const void* xq, int64_t ldx, const float* xs, const float* bias,
                   void* Y, int y_type, int64_t ldy, int64_t M, int64_t K, int64_t N, void* workspace,
                   size_t workspace_bytes, qg_stream_t stream) {
    qg::clear_error();
    if (!w || !ws || !xq || !xs || !Y) return qg::fail(QG_ERR_NULL, "NULL pointer (w_packed, w_scale, xq, x_scale, Y)");
    if (!known_type(y_type)) return qg::fail(QG_ERR_SHAPE, "y_type=%d unknown", y_type);
    qg_status st = check_mk(M, K);
    if (st) return st;
    const int64_t mt = qg::ceil_div(M, T), kp = qg::ceil_div(K, kKB) * kKB;
    if (N < 1 || N > QG_I8_MAX_ROWS || M * N > (int64_t)1 << 32)
        return qg::fail(QG_ERR_SHAPE, "N=%lld not in [1, %d], or M N over 2^32", (long long)N, QG_I8_MAX_ROWS);
    const int64_t most = ((int64_t)1 << 40) / N;
    if (ldx < kp || ldx > (1 << 22) || ldx % 16)  // 256 rows stay within 32-bit offsets
        return qg::fail(QG_ERR_SHAPE, "ldx=%lld not a multiple of 16 in [%lld, 2^22]", (long long)ldx, (long long)kp);
    if (ldy < M || ldy > most || ldy % 4)
        return qg::fail(QG_ERR_SHAPE, "ldy=%lld not a multiple of 4 in [M, 2^40 / N]", (long long)ldy);
    if (!qg::aligned16(w) || !qg::aligned16(xq) || !qg::aligned16(Y))
        return qg::fail(QG_ERR_ALIGN, "w_packed, xq and Y must be 16-byte aligned");
    if ((reinterpret_cast<uintptr_t>(ws) | reinterpret_cast<uintptr_t>(xs) | reinterpret_cast<uintptr_t>(bias)) & 3)
        return qg::fail(QG_ERR_ALIGN, "w_scale, x_scale and bias must be 4-byte aligned");
    const size_t yb = ((size_t)(N - 1) * ldy + M) * elem_bytes(y_type);
    if (overlap(Y, yb, xq, (size_t)(N - 1) * ldx + kp) || overlap(Y, yb, w, qg_i8_bytes(M, K)) ||
        overlap(Y, yb, ws, (size_t)M * 4) || overlap(Y, yb, xs, (size_t)N * 4) ||
        (bias && overlap(Y, yb, bias, (size_t)M * 4)))
        return qg::fail(QG_ERR_SHAPE, "Y overlaps an input");
    const Plan p = plan(M, K, N);
    if (p.ws && (!workspace || workspace_bytes < p.ws))
        return qg::fail(QG_ERR_WORKSPACE, "workspace of %zu bytes required, got %zu", p.ws, workspace ? workspace_bytes : 0);
    if (p.ws) {
        if (!qg::aligned16(workspace)) return qg::fail(QG_ERR_ALIGN, "workspace not 16-byte aligned");
        if (overlap(workspace, p.ws, Y, yb) || overlap(workspace, p.ws, xq, (size_t)(N - 1) * ldx + kp) ||
            overlap(workspace, p.ws, w, qg_i8_bytes(M, K)) || overlap(workspace, p.ws, ws, (size_t)M * 4) ||
            overlap(workspace, p.ws, xs, (size_t)N * 4) || (bias && overlap(workspace, p.ws, bias, (size_t)M * 4)))
            return qg::fail(QG_ERR_SHAPE, "the workspace overlaps an operand");
    }
    st = qg::check_device();
    if (st) return st;
    GArgs a{};
    a.w = (const uint8_t*)w;
    a.ws = ws;
    a.x = (const int8_t*)xq;
    a.ldx = ldx;
    a.xs = xs;
    a.bias = bias;
    a.Y = Y;
    a.ldy = ldy;
    a.M = (int32_t)M;
    a.N = (int32_t)N;
    a.nb = (int32_t)(kp / kKB);
    a.mtiles = (int32_t)mt;
    a.part = (qi4*)workspace;
    a.kper = p.kper;
    a.total = p.tiles;
    hipStream_t s = (hipStream_t)stream;
    if (y_type == QG_F32) return launch_gemm<QG_F32>(a, p, s);
    if (y_type == QG_F16) return launch_gemm<QG_F16>(a, p, s);
    return launch_gemm<QG_BF16>(a, p, s);
}

}  // extern "C"
