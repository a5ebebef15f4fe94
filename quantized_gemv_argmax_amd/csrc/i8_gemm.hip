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

#include "qg_device.h"
#include "qg_host.h"

namespace {

typedef int qi4 __attribute__((ext_vector_type(4)));

constexpr int T = QG_TILE_ROWS;
constexpr int kKB = 64;           // k per matrix-core operand
constexpr int kTileB = T * kKB;   // bytes of one operand (16 rows x 64 k)

QG_DEV uint16_t f32_to_bf16(float v) {
    // round to nearest even; a NaN stays one
    const uint32_t b = __builtin_bit_cast(uint32_t, v);
    if (v != v) return (uint16_t)((b >> 16) | 0x40u);
    return (uint16_t)((b + 0x7fffu + ((b >> 16) & 1u)) >> 16);
}

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
            const int8_t* p = src + row * ldw + k0;
            if (k0 + 16 <= K && (reinterpret_cast<uintptr_t>(p) & 15) == 0) {
                o.v = *reinterpret_cast<const uint4*>(p);
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
    static constexpr int N = 4;
    QG_DEV static float get(const uint4& v, int i) { return __builtin_bit_cast(float, (&v.x)[i]); }
    QG_DEV static float one(E e) { return e; }
};
template <>
struct XVec<QG_F16> {
    typedef uint16_t E;
    static constexpr int N = 8;
    QG_DEV static float get(const uint4& v, int i) {
        return (i & 1) ? qg_half_hi((&v.x)[i >> 1]) : qg_half_lo((&v.x)[i >> 1]);
    }
    QG_DEV static float one(E e) { return qg_half_lo(e); }
};
template <>
struct XVec<QG_BF16> {
    typedef uint16_t E;
    static constexpr int N = 8;
    QG_DEV static float get(const uint4& v, int i) {
        const uint32_t w = (&v.x)[i >> 1];
        return __builtin_bit_cast(float, (i & 1) ? (w & 0xffff0000u) : (w << 16));
    }
    QG_DEV static float one(E e) { return __builtin_bit_cast(float, (uint32_t)e << 16); }
};

// The 16-byte vector i of a row of K elements, zeros beyond K. `vec`: the row is
// 16-byte aligned.
template <int XT>
QG_DEV uint4 row_vec(const typename XVec<XT>::E* p, int K, int i, bool vec) {
    typedef typename XVec<XT>::E E;
    constexpr int N = XVec<XT>::N;
    const int k0 = i * N;
    if (vec && k0 + N <= K) return *reinterpret_cast<const uint4*>(p + k0);
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

// One workgroup of NT threads per row. The row stays in registers between the
// maximum and the rounding where NT threads hold it in R vectors each; a longer one
// (R == 0) is read twice.
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
    const bool vec = (reinterpret_cast<uintptr_t>(p) & 15) == 0;
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
            if (tid + r * NT < nv) v[r] = row_vec<XT>(p, K, tid + r * NT, vec);
        }
#pragma unroll
        for (int r = 0; r < R; ++r) peak(v[r]);
    } else {
        for (int i = tid; i < nv; i += NT) peak(row_vec<XT>(p, K, i, vec));
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
        for (int i = tid; i < nv; i += NT) store_q<XT>(o, i, row_vec<XT>(p, K, i, vec), s, d, inv, ok);
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
    int32_t M, N, nb;  // nb: k blocks of 64
    int32_t mtiles;
};

QG_DEV float scaled(int acc, float xs, float ws, float b) { return (float)acc * (xs * ws) + b; }

// Four consecutive outputs m .. m + 3 of column n.
template <int YT>
QG_DEV void store4(const GArgs& a, int64_t n, int m, qi4 acc) {
    if (m >= a.M) return;
    const float xs = a.xs[n];
    float y[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int r = min(m + e, a.M - 1);
        y[e] = scaled(acc[e], xs, a.ws[r], a.bias ? a.bias[r] : 0.f);
    }
    if constexpr (YT == QG_F32) {
        float* p = reinterpret_cast<float*>(a.Y) + n * a.ldy + m;
        if (m + 4 <= a.M) {
            *reinterpret_cast<float4*>(p) = make_float4(y[0], y[1], y[2], y[3]);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (m + e < a.M) p[e] = y[e];
        }
    } else {
        uint16_t h[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
            h[e] = YT == QG_F16 ? __builtin_bit_cast(uint16_t, (_Float16)y[e]) : f32_to_bf16(y[e]);
        uint16_t* p = reinterpret_cast<uint16_t*>(a.Y) + n * a.ldy + m;
        if (m + 4 <= a.M) {
            *reinterpret_cast<uint2*>(p) = make_uint2(h[0] | (uint32_t)h[1] << 16, h[2] | (uint32_t)h[3] << 16);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (m + e < a.M) p[e] = h[e];
        }
    }
}

// One 16-row tile and NB blocks of 16 columns per workgroup; its KW wavefronts take
// the k blocks in turn, and their integer sums meet in LDS. The weights go from
// memory straight to the operand registers, in the packed order.
template <int YT, int NB, int KW>
__global__ __launch_bounds__(64 * KW) void gemm_i8_stream_kernel(GArgs a) {
    __shared__ qi4 part[KW][NB][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int t = blockIdx.x % a.mtiles;
    const int n0 = blockIdx.x / a.mtiles * (NB * 16);
    const uint8_t* w = a.w + ((size_t)t * a.nb) * kTileB + lane * 16;
    const int8_t* xr[NB];
#pragma unroll
    for (int c = 0; c < NB; ++c)  // columns beyond N read the last one; their sums are not stored
        xr[c] = a.x + (int64_t)min(n0 + 16 * c + (lane & 15), a.N - 1) * a.ldx + (lane >> 4) * 16;
    qi4 acc[NB];
#pragma unroll
    for (int c = 0; c < NB; ++c) acc[c] = qi4{0, 0, 0, 0};
#pragma unroll 2
    for (int b = wave; b < a.nb; b += KW) {
        const qi4 wv = *reinterpret_cast<const qi4*>(w + (size_t)b * kTileB);
#pragma unroll
        for (int c = 0; c < NB; ++c) {
            const qi4 xv = *reinterpret_cast<const qi4*>(xr[c] + b * kKB);
            acc[c] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wv, xv, acc[c], 0, 0, 0);
        }
    }
#pragma unroll
    for (int c = 0; c < NB; ++c) part[wave][c][lane] = acc[c];
    __syncthreads();
    for (int c = wave; c < NB; c += KW) {
        qi4 s = part[0][c][lane];
#pragma unroll
        for (int k = 1; k < KW; ++k) s += part[k][c][lane];
        const int n = n0 + 16 * c + (lane & 15);
        if (n < a.N) store4<YT>(a, n, t * T + (lane >> 4) * 4, s);
    }
}

template <int YT>
qg_status launch_gemm(const GArgs& a, hipStream_t s) {
    const int nblk = (int)qg::ceil_div(a.N, 16);
    if (nblk <= 1) {
        hipLaunchKernelGGL((gemm_i8_stream_kernel<YT, 1, 8>), dim3(a.mtiles), dim3(512), 0, s, a);
    } else if (nblk <= 2) {
        hipLaunchKernelGGL((gemm_i8_stream_kernel<YT, 2, 8>), dim3(a.mtiles), dim3(512), 0, s, a);
    } else {
        const int64_t g = (int64_t)a.mtiles * qg::ceil_div(nblk, 4);
        hipLaunchKernelGGL((gemm_i8_stream_kernel<YT, 4, 8>), dim3((unsigned)g), dim3(512), 0, s, a);
    }
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
    if (nv <= 512)
        hipLaunchKernelGGL((quantize_i8_kernel<XT, 256, 2>), g, dim3(256), 0, s, x, ldx, K, q, ldq, scale);
    else if (nv <= 2560)
        hipLaunchKernelGGL((quantize_i8_kernel<XT, 256, 10>), g, dim3(256), 0, s, x, ldx, K, q, ldq, scale);
    else if (nv <= 5120)
        hipLaunchKernelGGL((quantize_i8_kernel<XT, 512, 10>), g, dim3(512), 0, s, x, ldx, K, q, ldq, scale);
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

size_t qgemm_i8_workspace_bytes(int64_t M, int64_t K, int64_t N) { return 0; }

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
    if (ldx < kp || ldx > most || ldx % 16)
        return qg::fail(QG_ERR_SHAPE, "ldx=%lld not a multiple of 16 in [%lld, 2^40 / N]", (long long)ldx, (long long)kp);
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
    hipStream_t s = (hipStream_t)stream;
    if (y_type == QG_F32) return launch_gemm<QG_F32>(a, s);
    if (y_type == QG_F16) return launch_gemm<QG_F16>(a, s);
    return launch_gemm<QG_BF16>(a, s);
}

}  // extern "C"
