// Rows of fp32, fp16 and bf16 and LDS tiles, shared by the int8 and the 8-bit
// floating-point products: element access, row stores, direct loads to LDS, the order of
// tiles over the XCDs, and host checks.
#pragma once

#include <atomic>

#include "qg_device.h"
#include "qg_host.h"

namespace qg {

typedef int qi4 __attribute__((ext_vector_type(4)));

// ---------------------------------------------------------------- rows
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

// ---------------------------------------------------------------- tiles
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

// Tile of workgroup id: eight XCDs take the tiles in eight contiguous runs, and in a
// run groups of eight tile rows walk the columns together, so that the tiles an XCD
// works on at a time share their weights and activations in its L2.
struct TileAt {
    int t0, n0;  // first 16-row tile, first column
};
template <int BM, int BN>
QG_DEV TileAt tile_at(int mtiles, int N, int id) {
    const int mts = (mtiles * 16 + BM - 1) / BM, nts = (N + BN - 1) / BN;
    const int total = mts * nts, q = total / 8, r = total % 8, x = id % 8;
    id = x * q + min(x, r) + id / 8;
    constexpr int GM = 8;
    const int per = GM * nts, grp = id / per, rem = id - grp * per;
    const int gm = min(GM, mts - grp * GM);
    return {(grp * GM + rem % gm) * (BM / 16), rem / gm * BN};
}

// ---------------------------------------------------------------- host
// Allows a kernel more than 64 KB of LDS, once per device.
inline qg_status allow_lds(const void* f, int bytes, std::atomic<bool>* done) {
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return fail(QG_ERR_DEVICE, "no current device");
    if (done[dev].load(std::memory_order_acquire)) return QG_OK;
    const hipError_t e = hipFuncSetAttribute(f, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != hipSuccess) return fail(QG_ERR_DEVICE, "LDS size: %s", hipGetErrorString(e));
    done[dev].store(true, std::memory_order_release);
    return QG_OK;
}

inline int elem_bytes(int type) { return type == QG_F32 ? 4 : 2; }
inline bool known_type(int type) { return type == QG_F32 || type == QG_F16 || type == QG_BF16; }
inline bool overlap(const void* a, size_t na, const void* b, size_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + nb && y < x + na;
}

}  // namespace qg
