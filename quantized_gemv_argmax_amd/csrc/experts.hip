// Selection of experts and the weighted sum of their outputs, for gfx950: what a
// mixture-of-experts layer runs before and after its grouped products.
//
// The selection ranks each row of E logits within sixteen lanes and orders the rows by
// expert without atomics whose order could change the result: 32 rows are a word of a
// bit map per expert, so a row's place among an expert's rows is a count of bits.
#include <algorithm>
#include <cfloat>
#include <climits>
#include <cmath>

#include "qg_device.h"
#include "qg_host.h"
#include "qg_rows.h"

namespace {

using namespace qg;

// ---------------------------------------------------------------- selection
struct SArgs {
    const void* z;
    int64_t ld;
    int32_t N, E, k, normalize;
    int32_t words, parts, per;  // words of an expert's bit map, its parts (1: not counted), words of one
    float scale;
    uint32_t* bits;  // [E][words]
    int32_t* counts;  // [E][parts]
    qg_experts_out o;
};

QG_DEV float neg_inf() { return -__builtin_inff(); }

// Reductions over groups of 16 lanes, the result in all of them.
template <int CTRL>
QG_DEV int lane_swap(int v) {
    return __builtin_amdgcn_mov_dpp(v, CTRL, 0xf, 0xf, true);
}
template <class F>
QG_DEV int reduce(int v, F&& op) {
    v = op(v, lane_swap<0xb1>(v));   // quad_perm [1, 0, 3, 2]
    v = op(v, lane_swap<0x4e>(v));   // quad_perm [2, 3, 0, 1]
    v = op(v, lane_swap<0x141>(v));  // row_half_mirror
    return op(v, lane_swap<0x140>(v));  // row_mirror
}
QG_DEV float as_float(int v) { return __builtin_bit_cast(float, v); }
QG_DEV int as_int(float v) { return __builtin_bit_cast(int, v); }
QG_DEV float group_max(float v) {
    return as_float(reduce(as_int(v), [](int a, int b) { return as_int(fmaxf(as_float(a), as_float(b))); }));
}
QG_DEV float group_sum(float v) {
    return as_float(reduce(as_int(v), [](int a, int b) { return as_int(as_float(a) + as_float(b)); }));
}
QG_DEV int group_min(int v) {
    return reduce(v, [](int a, int b) { return min(a, b); });
}
QG_DEV int wave_scan(int v, int lane) {  // inclusive
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
        const int u = __shfl_up(v, m);
        if (lane >= m) v += u;
    }
    return v;
}

// The k best of a row of logits z, in 16 lanes of V each (logit 16 v + lane): the maximum and
// its first place, k times, each a reduction within 16 lanes, which costs less than one over 64 (E = 512,
// 4096 rows: the row in 16 lanes 20 us in all, in 64 lanes 35). Lane j gets the j-th and the (j + 16)-th
// (expert -1 where there are fewer) with their weights exp(z - max) / sum, the sum over
// the chosen ones or over all.
constexpr int L = 16;
template <int XT, int V>
struct Row {
    static constexpr int R = QG_EXPERTS_MAX_K / L;  // results of a lane
    float z[V];
    int expert[R];
    float weight[R];
    QG_DEV void load(const SArgs& a, int64_t n, int lane) {
        typedef typename XVec<XT>::E E;
        const E* p = reinterpret_cast<const E*>(a.z) + n * a.ld;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            z[v] = neg_inf();
            if (v * L + lane < a.E) z[v] = XVec<XT>::one(p[v * L + lane]);
        }
    }
    QG_DEV void select(const SArgs& a, int lane) {
#pragma unroll
        for (int v = 0; v < V; ++v) z[v] = z[v] == z[v] ? fminf(z[v], FLT_MAX) : neg_inf();
#pragma unroll
        for (int r = 0; r < R; ++r) {
            expert[r] = -1;
            weight[r] = neg_inf();
        }
        float first = neg_inf(), sum = 0.f;
        for (int j = 0; j < a.k; ++j) {
            float m = z[0];
#pragma unroll
            for (int v = 1; v < V; ++v) m = fmaxf(m, z[v]);
            m = group_max(m);
            if (j == 0) {
                first = m;
                if (!a.normalize) {
                    float part[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int v = 0; v < V; ++v) part[v & 3] += z[v] > neg_inf() ? expf(z[v] - m) : 0.f;
                    sum = group_sum((part[0] + part[1]) + (part[2] + part[3]));
                }
            }
            int at = INT_MAX;
#pragma unroll
            for (int v = V - 1; v >= 0; --v) at = z[v] == m ? v * L + lane : at;
            at = group_min(at);
            const bool there = m > neg_inf();
#pragma unroll
            for (int v = 0; v < V; ++v) z[v] = v * L + lane == at ? neg_inf() : z[v];
#pragma unroll
            for (int r = 0; r < R; ++r)
                if (there && lane + L * r == j) {
                    expert[r] = at;
                    weight[r] = m;
                }
        }
#pragma unroll
        for (int r = 0; r < R; ++r) weight[r] = expert[r] >= 0 ? expf(weight[r] - first) : 0.f;
        if (a.normalize) {
            float s = weight[0];
#pragma unroll
            for (int r = 1; r < R; ++r) s += weight[r];
            sum = group_sum(s);
        }
#pragma unroll
        for (int r = 0; r < R; ++r)
            if (expert[r] >= 0) weight[r] = a.scale * (weight[r] / sum);
    }
};

// Rows of a workgroup: 32, their words to the bit map; or (ONE) all rows, up to 64, and
// their order too, which saves a launch (45 x 37, 3 of them: 4.7 us, in two launches 10).
// Bounded by the chain of k maxima: 4096 x 128, 8 of them, takes 11.4 us in all, 0.4
// of them to read the logits.
constexpr int kOneRows = 64;
template <int XT, int V, bool ONE>
__global__ __launch_bounds__(ONE ? 1024 : 512) void select_kernel(SArgs a) {
    constexpr int W = ONE ? 2 : 1, ROWS = 32 * W, NT = ONE ? 1024 : 512, EP = V * L;
    __shared__ uint32_t word[EP * W];
    __shared__ int base[ONE ? EP : 1], chosen[ONE ? ROWS * QG_EXPERTS_MAX_K : 1], asked;
    const int tid = threadIdx.x, lane = tid & (L - 1), group = tid / L;
    const int64_t n0 = (int64_t)blockIdx.x * ROWS;
    const int rows = (int)min((int64_t)ROWS, a.N - n0);
    Row<XT, V> row;
    if (group < rows) row.load(a, n0 + group, lane);
    for (int e = tid; e < EP * W; e += NT) word[e] = 0;
    __syncthreads();
    for (int i = group; i < rows; i += NT / L) {
        if (i != group) row.load(a, n0 + i, lane);
        row.select(a, lane);
#pragma unroll
        for (int r = 0; r < row.R; ++r) {
            const int j = lane + L * r;
            if (j < a.k) {
                const int64_t at = (n0 + i) * a.k + j;
                const int e = row.expert[r];
                a.o.expert[at] = e;
                a.o.weight[at] = row.weight[r];
                if constexpr (ONE) chosen[i * a.k + j] = e;
                if (e >= 0)
                    atomicOr(&word[e * W + (i >> 5)], 1u << (i & 31));
                else if constexpr (!ONE)
                    a.o.position[at] = -1;  // (the others' come with the order)
            }
        }
    }
    __syncthreads();
    if constexpr (!ONE) {
        for (int e = tid; e < a.E; e += NT) a.bits[(int64_t)e * a.words + blockIdx.x] = word[e];
    } else {
        if (tid < 64) {
            int carry = 0;
            for (int e0 = 0; e0 < a.E; e0 += 64) {
                const int e = e0 + tid, c = __popc(word[e * W]) + __popc(word[e * W + 1]), upto = wave_scan(c, tid) + carry;
                base[e] = upto - c;
                if (e < a.E) a.o.offsets[e] = upto - c;
                carry = __builtin_amdgcn_readlane(upto, 63);
            }
            if (tid == 0) a.o.offsets[a.E] = asked = carry;
        }
        __syncthreads();
        const int all = a.N * a.k;
        for (int i = tid; i < all; i += NT) {
            const int e = chosen[i], n = i / a.k;
            int at = -1;
            if (e >= 0) {
                at = base[e] + __popc(word[e * W + (n >> 5)] & ((1u << (n & 31)) - 1));
                if (n >= 32) at += __popc(word[e * W]);
                a.o.row[at] = n;
            }
            a.o.position[i] = at;
            if (i >= asked) a.o.row[i] = -1;
        }
    }
}

// Sums over a workgroup, the result in all threads. (A barrier first: `red` may be in use.)
template <int NT>
QG_DEV int group_total(int v, int* red) {
    v = reduce(v, [](int x, int y) { return x + y; });
    v += __shfl_xor(v, 16);
    v += __shfl_xor(v, 32);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0;
#pragma unroll
    for (int w = 0; w < NT / 64; ++w) v += red[w];
    return v;
}

// Rows of expert blockIdx.x in part blockIdx.y of its words.
constexpr int kOrder = 512, kChunk = 256;  // threads, words of a chunk
__global__ __launch_bounds__(256) void count_kernel(SArgs a) {
    __shared__ int red[4];
    const int e = blockIdx.x, part = blockIdx.y, w0 = part * a.per;
    int sum = 0;
    for (int w = w0 + threadIdx.x; w < min(w0 + a.per, a.words); w += 256) sum += __popc(a.bits[(int64_t)e * a.words + w]);
    sum = group_total<256>(sum, red);
    if (threadIdx.x == 0) a.counts[e * a.parts + part] = sum;
}

// The order by expert, a workgroup per expert: its rows begin where the bits of all
// experts before it end; its own bits become a list of rows, a chunk of words at a time.
// With more than a chunk to an expert, a workgroup per part of its words, whose rows begin where the
// counts of the parts before end: a launch more, but no reading that grows with the square of the experts
// (16384 x 256: 22.8 us, without counts 26.7; 131072 x 512: 171 and 377; 524288 x 64: 121 and 296).
template <bool PARTS>
__global__ __launch_bounds__(kOrder) void order_kernel(SArgs a) {
    constexpr int C = kChunk, NT = kOrder;
    __shared__ int red[NT / 64];
    __shared__ int list[C * 32];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, e = blockIdx.x, part = PARTS ? blockIdx.y : 0;
    const int begin = PARTS ? part * a.per : 0, end = PARTS ? min(begin + a.per, a.words) : a.words;
    const int64_t before = (int64_t)e * a.words;
    uint32_t bits = tid < C && begin + tid < end ? a.bits[before + begin + tid] : 0;  // (on their way while the others are counted)
    int sum = 0, rest = 0;
    if constexpr (PARTS) {
        const int mine = e * a.parts + part;
        for (int i = tid; i < a.E * a.parts; i += NT) (i < mine ? sum : rest) += a.counts[i];
    } else {
        const uint4* b4 = reinterpret_cast<const uint4*>(a.bits);
#pragma unroll 4
        for (int64_t i = tid; i < before / 4; i += NT) {
            const uint4 v = b4[i];
            sum += __popc(v.x) + __popc(v.y) + __popc(v.z) + __popc(v.w);
        }
        if (tid < (int)(before & 3)) sum += __popc(a.bits[before - 1 - tid]);
    }
    int at = group_total<NT>(sum, red);
    const int asked = PARTS ? at + group_total<NT>(rest, red) : 0;  // rows of all experts
    if (tid == 0 && part == 0) a.o.offsets[e] = at;
    for (int w0 = begin; w0 < end; w0 += C) {
        if (w0 > begin) bits = tid < C && w0 + tid < end ? a.bits[before + w0 + tid] : 0;
        const int c = __popc(bits);
        int upto = wave_scan(c, lane);
        __syncthreads();  // (red and list of the step before have been read)
        if (lane == 63) red[wave] = upto;
        __syncthreads();
        int all = 0;
#pragma unroll
        for (int w = 0; w < C / 64; ++w) {
            if (w < wave) upto += red[w];
            all += red[w];
        }
        int put = upto - c;
        while (bits) {
            list[put++] = (w0 + tid) * 32 + __builtin_ctz(bits);
            bits &= bits - 1;
        }
        __syncthreads();
        for (int i = tid; i < all; i += NT) {
            const int n = list[i];
            a.o.row[at + i] = n;
            const int64_t p = (int64_t)n * a.k;
#pragma unroll 8
            for (int j = 0; j < a.k; ++j)
                if (a.o.expert[p + j] == e) a.o.position[p + j] = at + i;
        }
        at += all;
    }
    // nothing behind the last expert's rows
    if constexpr (PARTS) {
        if (tid == 0 && e == 0 && part == 0) a.o.offsets[a.E] = asked;
        for (int i = asked + (e * a.parts + part) * NT + tid; i < a.N * a.k; i += a.E * a.parts * NT) a.o.row[i] = -1;
    } else if (e == a.E - 1) {
        if (tid == 0) a.o.offsets[a.E] = at;
        for (int i = at + tid; i < a.N * a.k; i += NT) a.o.row[i] = -1;
    }
}

template <int XT, int V>
void launch_select(const SArgs& a, hipStream_t s) {
    if (a.N <= kOneRows)
        hipLaunchKernelGGL((select_kernel<XT, V, true>), dim3(1), dim3(1024), 0, s, a);
    else
        hipLaunchKernelGGL((select_kernel<XT, V, false>), dim3((unsigned)a.words), dim3(512), 0, s, a);
}
template <int XT>
void launch_select(const SArgs& a, hipStream_t s) {
    if (a.E <= 64)
        launch_select<XT, 4>(a, s);
    else if (a.E <= 128)
        launch_select<XT, 8>(a, s);
    else if (a.E <= 256)
        launch_select<XT, 16>(a, s);
    else if (a.E <= 512)
        launch_select<XT, 32>(a, s);
    else
        launch_select<XT, QG_EXPERTS_MAX / L>(a, s);
}

// ---------------------------------------------------------------- combination
struct CArgs {
    const void* y;
    int64_t ldy;
    const int32_t* position;
    const float* weight;
    const void* add;
    int64_t ldadd;
    void* out;
    int64_t ldo;
    uint32_t total, cols;  // threads; eight columns each, so many in a row
    int32_t rows, k, M;
};

// Eight columns from c on of a row of M, zeros beyond.
template <int XT>
QG_DEV void load8(const typename XVec<XT>::E* p, int M, int c, uint4 (&v)[8 / XVec<XT>::N]) {
#pragma unroll
    for (int i = 0; i < 8 / XVec<XT>::N; ++i) v[i] = row_vec<XT>(p, M, c / XVec<XT>::N + i);
}
template <int XT>
QG_DEV float get8(const uint4 (&v)[8 / XVec<XT>::N], int e) {
    return XVec<XT>::get(v[e / XVec<XT>::N], e % XVec<XT>::N);
}

// out = (add +) sum_j weight_j Y[position_j], in float32, in the order of j. Eight columns of a
// row per thread; the rows it adds are all on their way at once, eight at a time. Bound by
// memory: 4096 rows of 8 by 2048 bf16 onto a residual take 34 us, 168 MB at 4.9 TB/s.
template <int YT, int OT>
__global__ __launch_bounds__(256) void combine_kernel(CArgs a) {
    typedef typename XVec<YT>::E E;
    typedef typename XVec<OT>::E O;
    constexpr int J = 8;
    const uint32_t at = blockIdx.x * 256u + threadIdx.x;
    if (at >= a.total) return;
    const uint32_t n = at / a.cols;
    const int c = (int)(at - n * a.cols) * 8;
    float s[8];
    if (a.add) {
        uint4 v[8 / XVec<OT>::N];
        load8<OT>(reinterpret_cast<const O*>(a.add) + n * a.ldadd, a.M, c, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) s[e] = get8<OT>(v, e);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) s[e] = 0.f;
    }
    const int32_t* pos = a.position + (int64_t)n * a.k;
    const float* wt = a.weight + (int64_t)n * a.k;
    for (int j0 = 0; j0 < a.k; j0 += J) {
        uint4 v[J][8 / XVec<YT>::N];
        int p[J];
        float w[J];
#pragma unroll
        for (int j = 0; j < J; ++j) {
            p[j] = j0 + j < a.k ? pos[j0 + j] : -1;
            w[j] = j0 + j < a.k ? wt[j0 + j] : 0.f;
        }
#pragma unroll
        for (int j = 0; j < J; ++j)
            if (p[j] >= 0 && p[j] < a.rows) load8<YT>(reinterpret_cast<const E*>(a.y) + p[j] * a.ldy, a.M, c, v[j]);
#pragma unroll
        for (int j = 0; j < J; ++j)
            if (p[j] >= 0 && p[j] < a.rows)
#pragma unroll
                for (int e = 0; e < 8; ++e) s[e] = __builtin_fmaf(w[j], get8<YT>(v[j], e), s[e]);
    }
    O* o = reinterpret_cast<O*>(a.out) + n * a.ldo + c;
    if (c + 8 <= a.M) {
        typedef typename XVec<OT>::V vec;  // (rows start anywhere)
        if constexpr (OT == QG_F32) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
                *reinterpret_cast<vec*>(o + 4 * i) = vec{__builtin_bit_cast(uint32_t, s[4 * i]), __builtin_bit_cast(uint32_t, s[4 * i + 1]),
                                                         __builtin_bit_cast(uint32_t, s[4 * i + 2]), __builtin_bit_cast(uint32_t, s[4 * i + 3])};
        } else {
            *reinterpret_cast<vec*>(o) = vec{pack2<OT>(s[0], s[1]), pack2<OT>(s[2], s[3]), pack2<OT>(s[4], s[5]), pack2<OT>(s[6], s[7])};
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (c + e < a.M) {
                if constexpr (OT == QG_F32)
                    o[e] = s[e];
                else
                    o[e] = (uint16_t)pack2<OT>(s[e], 0.f);
            }
    }
}

template <int YT>
void launch_combine(const CArgs& a, int out_type, hipStream_t s) {
    const dim3 g((a.total + 255) / 256);
    if (out_type == QG_F32)
        hipLaunchKernelGGL((combine_kernel<YT, QG_F32>), g, dim3(256), 0, s, a);
    else if (out_type == QG_F16)
        hipLaunchKernelGGL((combine_kernel<YT, QG_F16>), g, dim3(256), 0, s, a);
    else
        hipLaunchKernelGGL((combine_kernel<YT, QG_BF16>), g, dim3(256), 0, s, a);
}

bool select_shape(int64_t N, int E, int k) {
    return E >= 1 && E <= QG_EXPERTS_MAX && k >= 1 && k <= E && k <= QG_EXPERTS_MAX_K && N >= 1 && N <= QG_F8_MAX_ROWS / k;
}
// Parts of an expert's words: whole chunks, and counts that every workgroup can sum.
int select_parts(int64_t words, int E) { return (int)std::min<int64_t>(qg::ceil_div(words, kChunk), std::max(1, 4096 / E)); }
size_t select_bits(int64_t N, int E) { return qg::align_up((size_t)E * (size_t)qg::ceil_div(N, 32) * 4, 16); }
size_t select_ws(int64_t N, int E) {
    return N <= kOneRows ? 0 : select_bits(N, E) + qg::align_up((size_t)E * select_parts(qg::ceil_div(N, 32), E) * 4, 16);
}

}  // namespace

extern "C" {

size_t logits_expert_select_workspace_bytes(int64_t N, int E, int k) { return select_shape(N, E, k) ? select_ws(N, E) : 0; }

qg_status logits_expert_select(const void* logits, int logits_type, int64_t ld, int64_t N, int E, int k, int normalize,
                               float scale, void* workspace, size_t workspace_bytes, const qg_experts_out* out,
                               qg_stream_t stream) {
    qg::clear_error();
    if (!logits || !out) return qg::fail(QG_ERR_NULL, "NULL pointer (logits, out)");
    if (!out->expert || !out->weight || !out->position || !out->row || !out->offsets)
        return qg::fail(QG_ERR_NULL, "NULL pointer in out");
    if (!known_type(logits_type)) return qg::fail(QG_ERR_SHAPE, "logits_type=%d unknown", logits_type);
    if (!select_shape(N, E, k))
        return qg::fail(QG_ERR_SHAPE, "N=%lld, E=%d or k=%d out of range (E <= %d, k <= min(E, %d), N k <= %d)", (long long)N, E, k,
                        QG_EXPERTS_MAX, QG_EXPERTS_MAX_K, QG_F8_MAX_ROWS);
    if (ld < E || ld > ((int64_t)1 << 40) / N) return qg::fail(QG_ERR_SHAPE, "ld=%lld not in [E, 2^40 / N]", (long long)ld);
    if (normalize != 0 && normalize != 1) return qg::fail(QG_ERR_SHAPE, "normalize=%d not 0 or 1", normalize);
    if (!std::isfinite(scale)) return qg::fail(QG_ERR_SHAPE, "scale is not finite");
    const int eb = elem_bytes(logits_type);
    if (reinterpret_cast<uintptr_t>(logits) % eb) return qg::fail(QG_ERR_ALIGN, "logits not aligned to their elements");
    const size_t need = select_ws(N, E);
    struct Span {
        const void* p;
        size_t n;
    };
    const size_t nk = (size_t)N * k * 4;
    const Span in = {logits, ((size_t)(N - 1) * ld + E) * eb};
    const Span o[6] = {{out->expert, nk}, {out->weight, nk}, {out->position, nk}, {out->row, nk},
                       {out->offsets, (size_t)(E + 1) * 4}, {workspace, need}};
    for (int i = 0; i < 5; ++i)
        if (reinterpret_cast<uintptr_t>(o[i].p) & 3) return qg::fail(QG_ERR_ALIGN, "outputs must be 4-byte aligned");
    if (need) {
        if (!workspace || workspace_bytes < need)
            return qg::fail(QG_ERR_WORKSPACE, "workspace of %zu bytes required, got %zu", need, workspace ? workspace_bytes : 0);
        if (!qg::aligned16(workspace)) return qg::fail(QG_ERR_ALIGN, "workspace not 16-byte aligned");
    }
    for (int i = 0; i < (need ? 6 : 5); ++i) {
        if (overlap(o[i].p, o[i].n, in.p, in.n)) return qg::fail(QG_ERR_SHAPE, "an output or the workspace overlaps the logits");
        for (int j = 0; j < i; ++j)
            if (overlap(o[i].p, o[i].n, o[j].p, o[j].n)) return qg::fail(QG_ERR_SHAPE, "outputs and workspace overlap");
    }
    qg_status st = qg::check_device();
    if (st) return st;
    const int64_t words = qg::ceil_div(N, 32);
    const int parts = select_parts(words, E);
    const int per = (int)qg::align_up((size_t)qg::ceil_div(words, parts), kChunk);
    const SArgs a{logits, ld, (int32_t)N, E, k, normalize, (int32_t)words, parts, per, scale, (uint32_t*)workspace,
                  (int32_t*)((char*)workspace + select_bits(N, E)), *out};
    hipStream_t s = (hipStream_t)stream;
    if (logits_type == QG_F32)
        launch_select<QG_F32>(a, s);
    else if (logits_type == QG_F16)
        launch_select<QG_F16>(a, s);
    else
        launch_select<QG_BF16>(a, s);
    st = qg::launch_status("logits_expert_select");
    if (st || !need) return st;
    if (parts == 1) {
        hipLaunchKernelGGL((order_kernel<false>), dim3(E), dim3(kOrder), 0, s, a);
    } else {
        hipLaunchKernelGGL(count_kernel, dim3(E, parts), dim3(256), 0, s, a);
        st = qg::launch_status("logits_expert_select (count)");
        if (st) return st;
        hipLaunchKernelGGL((order_kernel<true>), dim3(E, parts), dim3(kOrder), 0, s, a);
    }
    return qg::launch_status("logits_expert_select (order)");
}

qg_status qg_expert_combine(const void* Y, int y_type, int64_t ldy, int64_t rows, const int32_t* position,
                            const float* weight, int k, const void* add, int64_t ldadd, void* out, int out_type,
                            int64_t ldo, int64_t N, int64_t M, qg_stream_t stream) {
    qg::clear_error();
    if (!Y || !position || !weight || !out) return qg::fail(QG_ERR_NULL, "NULL pointer (Y, position, weight, out)");
    if (!known_type(y_type) || !known_type(out_type))
        return qg::fail(QG_ERR_SHAPE, "y_type=%d or out_type=%d unknown", y_type, out_type);
    if (k < 1 || k > QG_EXPERTS_MAX_K) return qg::fail(QG_ERR_SHAPE, "k=%d not in [1, %d]", k, QG_EXPERTS_MAX_K);
    if (N < 1 || N > QG_F8_MAX_ROWS || rows < 1 || rows > QG_F8_MAX_ROWS)
        return qg::fail(QG_ERR_SHAPE, "N=%lld or rows=%lld not in [1, %d]", (long long)N, (long long)rows, QG_F8_MAX_ROWS);
    const int64_t most = (int64_t)1 << 40;
    if (M < 1 || M > INT32_MAX - 8 || N * qg::ceil_div(M, 8) >= ((int64_t)1 << 32) - 256)
        return qg::fail(QG_ERR_SHAPE, "M=%lld not in range, or N ceil(M / 8) over 2^32 - 256", (long long)M);
    if (ldy < M || ldy > most / rows || ldo < M || ldo > most / N || (add && (ldadd < M || ldadd > most / N)))
        return qg::fail(QG_ERR_SHAPE, "ldy=%lld, ldadd=%lld or ldo=%lld below M or over 2^40 / rows", (long long)ldy,
                        (long long)ldadd, (long long)ldo);
    const int yb = elem_bytes(y_type), ob = elem_bytes(out_type);
    if (reinterpret_cast<uintptr_t>(Y) % yb || (reinterpret_cast<uintptr_t>(out) | reinterpret_cast<uintptr_t>(add)) % ob ||
        (reinterpret_cast<uintptr_t>(position) | reinterpret_cast<uintptr_t>(weight)) & 3)
        return qg::fail(QG_ERR_ALIGN, "an array is not aligned to its elements");
    const size_t on = ((size_t)(N - 1) * ldo + M) * ob;
    if (overlap(out, on, Y, ((size_t)(rows - 1) * ldy + M) * yb) || overlap(out, on, position, (size_t)N * k * 4) ||
        overlap(out, on, weight, (size_t)N * k * 4))
        return qg::fail(QG_ERR_SHAPE, "out overlaps an input");
    if (add && !(add == out && ldadd == ldo) && overlap(out, on, add, ((size_t)(N - 1) * ldadd + M) * ob))
        return qg::fail(QG_ERR_SHAPE, "out overlaps add without being it");
    qg_status st = qg::check_device();
    if (st) return st;
    const uint32_t cols = (uint32_t)qg::ceil_div(M, 8);
    const CArgs a{Y, ldy, position, weight, add, ldadd, out, ldo, (uint32_t)N * cols, cols, (int32_t)rows, k, (int32_t)M};
    hipStream_t s = (hipStream_t)stream;
    if (y_type == QG_F32)
        launch_combine<QG_F32>(a, out_type, s);
    else if (y_type == QG_F16)
        launch_combine<QG_F16>(a, out_type, s);
    else
        launch_combine<QG_BF16>(a, out_type, s);
    return qg::launch_status("qg_expert_combine");
}

}  // extern "C"
