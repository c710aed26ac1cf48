// k_norm.cu -- the norms around a block, in one pass over its rows:
//   m = y silu(gate);  v = norm(m) w_post + b_post;  r_out = r + scale v;  o = norm(r_out) w_pre + b_pre
// with norm(v) = v / sqrt(mean(v^2) + eps), of v - mean(v) when centred.
//
// Some tens of operations per element: memory traffic bounds the forward pass, and the backward one
// about as much the instructions of its four sums over a row and the waits between them. A row stays in the
// registers of one warp (narrow rows) or one block from its load to its last store, so every tensor crosses
// HBM once. Means are taken before squares of differences, from registers, so that no cancellation enters.
// Statistics and sums are fp32.
//
// Measured (B200): forward 8192 x 4096, bf16 with an fp32 stream, gate and both norms, 82 us, 5.7 TB/s;
// backward 193 us, 3.8 TB/s. 8190 x 1153, bf16, centred, all parts: 40 us forward (2.4 TB/s), 77 us backward
// (2.0 TB/s), 37 and 72 us at 1152 columns.
#include "norm_shape.h"
#include "seq_common.cuh"

namespace gspn {
namespace seq {
namespace {

constexpr int kMaxC = 16384;
enum { kDwPost, kDbPost, kDscale, kDwPre, kDbPre, kSums };

struct NormArgs {
    int rows, C, center;
    float eps, inv_c;
    long long y_row, gate_row, r_row, least_row;
    const void *y, *gate, *r;
    const float *w_post, *b_post, *scale, *w_pre, *b_pre;
    void *r_out, *o;
    // backward
    const void *dr, *go;
    void *dy, *dr_in, *dgate;
    float* part;                 // [block][slot of sum][C]
    int slot[kSums], slots;      // which sums are wanted, and where; -1: not
    bool wide, aligned;          // every tensor's rows have one phase; that phase is 0, and parameters are aligned
};

// ---------------------------------------------------------------------------- rows of up to 4096
// How a row is held. E elements (8; 16 over 2048 columns, so that no block has over eight warps to sum
// over: from 1024 columns on, 8190 x 1153 backward took 113 us against 77) in each thread of a block of as many
// warps as the row needs, or of one warp where 32 E cover it: V consecutive columns (16 bytes) at a time,
// E / V times over, as E / 2 pairs. Rows of an odd number of columns start at other distances from a 16-byte border: the columns
// of a thread are shifted by that phase, so that every full vector is still one aligned load. A block
// takes rows of one phase only (the grid is a multiple of the phases' period), so a thread keeps its
// columns, and with them its parameters and column sums. Vectors that cross an end of the row, and all
// of a row whose tensors are aligned in different ways, go element by element.
struct Row {
    int C, tid, tpr, phase;
    bool wide, edge;             // edge: a thread of the warp has columns outside the row
};
template <typename T, int E> struct Lay {
    static constexpr int V = Vec<T>::V, K = E / V;
    static __device__ __forceinline__ int col(const Row& w, int e) { return (e / V * w.tpr + w.tid) * V + e % V - w.phase; }
};
// A row's elements of type S as stored, V columns (16 or 32 bytes) at a time.
template <typename T, typename S, int E> struct RowRaw {
    static constexpr int W = Vec<T>::V * sizeof(S) / 4;           // words of a vector
    uint32_t q[E / Vec<T>::V][W];
};
template <typename T, int E>
__device__ __forceinline__ bool inside(const Row& w, int e) { return (unsigned)Lay<T, E>::col(w, e) < (unsigned)w.C; }
// A vector that crosses an end of the row is loaded whole all the same, where its other columns are those
// of rows around (before it they always are; `more`: seven elements follow behind the row too);
// clear_row sets those to zero. Threads whose columns all lie behind the row keep the zeros they began with.
template <typename T, typename S, int E>
__device__ __forceinline__ void ld_row(RowRaw<T, S, E>& r, const S* p, const Row& w, bool more) {
    using Y = Lay<T, E>;
    constexpr int V = Y::V, W = RowRaw<T, S, E>::W;
#pragma unroll
    for (int k = 0; k < Y::K; ++k) {
        const int c = Y::col(w, k * V);
        if (c >= w.C) continue;
        if (w.wide && (more || c + V <= w.C)) {
#pragma unroll
            for (int m = 0; m < W; m += 4) {
                const uint4 v = *((const uint4*)(p + c) + m / 4);
                r.q[k][m] = v.x; r.q[k][m + 1] = v.y; r.q[k][m + 2] = v.z; r.q[k][m + 3] = v.w;
            }
        } else {
#pragma unroll
            for (int j = 0; j < W; ++j) {
                if constexpr (sizeof(S) == 4) {
                    r.q[k][j] = inside<T, E>(w, k * V + j) ? ((const uint32_t*)p)[c + j] : 0u;
                } else {
                    const uint32_t lo = inside<T, E>(w, k * V + 2 * j) ? ((const uint16_t*)p)[c + 2 * j] : 0u;
                    const uint32_t hi = inside<T, E>(w, k * V + 2 * j + 1) ? ((const uint16_t*)p)[c + 2 * j + 1] : 0u;
                    r.q[k][j] = lo | hi << 16;
                }
            }
        }
    }
}
template <typename T, typename S, int E>
__device__ __forceinline__ void clear_row(RowRaw<T, S, E>& r, const Row& w) {
    constexpr int V = Vec<T>::V;
#pragma unroll
    for (int e = 0; e < E; e += 2) {
        const uint32_t a = inside<T, E>(w, e) ? ~0u : 0u, b = inside<T, E>(w, e + 1) ? ~0u : 0u;
        if constexpr (sizeof(S) == 4) {
            r.q[e / V][e % V] &= a;
            r.q[e / V][e % V + 1] &= b;
        } else {
            r.q[e / V][e % V / 2] &= (a & 0xffffu) | (b & 0xffff0000u);
        }
    }
}
template <typename T, typename S, int E>
__device__ __forceinline__ void open_row(const RowRaw<T, S, E>& r, f2 (&v)[E / 2]) {
#pragma unroll
    for (int h = 0; h < E / 2; ++h) {
        const int k = 2 * h / Vec<T>::V, at = 2 * h % Vec<T>::V;
        if constexpr (sizeof(S) == 4) {
            v[h] = pack(__uint_as_float(r.q[k][at]), __uint_as_float(r.q[k][at + 1]));
        } else {
            const uint32_t q = r.q[k][at / 2];
            v[h] = pack(__uint_as_float(q << 16), __uint_as_float(q & 0xffff0000u));
        }
    }
}
template <typename T, typename S, int E>
__device__ __forceinline__ void st_row(S* p, const Row& w, const f2 (&v)[E / 2]) {
    using Y = Lay<T, E>;
    constexpr int V = Y::V;
#pragma unroll
    for (int k = 0; k < Y::K; ++k) {
        const int c = Y::col(w, k * V);
        float f[V];
        to_floats(*(const f2(*)[V / 2])(v + k * V / 2), f);
        if (w.wide && c >= 0 && c + V <= w.C) {
            st_lanes<S, V>(p + c, f);
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (inside<T, E>(w, k * V + j)) Io<S>::st(p + c + j, f[j]);
        }
    }
}

// The parameters of a thread's columns, zero where it has none, wait in shared memory, each thread's apart:
// shifted columns are not aligned in global memory.
template <typename T, int E> struct Params {
    float* at;                   // [parameter][E / 4][tpr][4]: neighbouring threads on neighbouring 16 bytes
    int stride;
    __device__ __forceinline__ void get(int i, const Row& w, f2 (&v)[E / 2]) const {
#pragma unroll
        for (int e = 0; e < E; e += 4)
            ld_pairs(at + i * stride + (e / 4 * w.tpr + w.tid) * 4, v[e / 2], v[e / 2 + 1]);
    }
    __device__ __forceinline__ void put(int i, const float* p, const Row& w) {
        if (!p) return;
        using Y = Lay<T, E>;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int c = Y::col(w, e);
            at[i * stride + (e / 4 * w.tpr + w.tid) * 4 + e % 4] = c >= 0 && c < w.C ? p[c] : 0.f;
        }
    }
};

// Sums over the threads of a row: the lanes of a warp, or (WARP = false) the warps of the block as well.
// Three buffers in turn, so that one barrier a call is enough. Four sums cost little more than one: the
// lanes share them out by halves.
template <bool WARP>
struct RowSum {
    float (*buf)[4][8];          // [turn][sum][warp]
    int turn = 0;
    __device__ __forceinline__ float one(float a) {
#pragma unroll
        for (int o = 16; o; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
        if constexpr (WARP) return a;
        if ((threadIdx.x & 31) == 0) buf[turn][0][threadIdx.x >> 5] = a;
        __syncthreads();
        a = over_warps(0);
        turn = turn == 2 ? 0 : turn + 1;
        return a;
    }
    __device__ __forceinline__ float4 four(float a, float b, float c, float d) {
        constexpr unsigned all = 0xffffffffu;
        const bool up = threadIdx.x & 16, hi = threadIdx.x & 8;
        const float x = (up ? b : a) + __shfl_xor_sync(all, up ? a : b, 16);
        const float y = (up ? d : c) + __shfl_xor_sync(all, up ? c : d, 16);
        float v = (hi ? y : x) + __shfl_xor_sync(all, hi ? x : y, 8);
#pragma unroll
        for (int o = 4; o; o >>= 1) v += __shfl_xor_sync(all, v, o);
        float4 s;
        if constexpr (WARP) {
            s.x = __shfl_sync(all, v, 0);
            s.y = __shfl_sync(all, v, 16);
            s.z = __shfl_sync(all, v, 8);
            s.w = __shfl_sync(all, v, 24);
        } else {
            if ((threadIdx.x & 7) == 0) buf[turn][(up ? 1 : 0) + (hi ? 2 : 0)][threadIdx.x >> 5] = v;
            __syncthreads();
            s.x = over_warps(0);
            s.y = over_warps(1);
            s.z = over_warps(2);
            s.w = over_warps(3);
            turn = turn == 2 ? 0 : turn + 1;
        }
        return s;
    }
    // eight warps at most; the places of those that are not there hold zeros
    __device__ __forceinline__ float over_warps(int i) const {
        f2 a, b, c, d;
        ld_pairs(&buf[turn][i][0], a, b);
        ld_pairs(&buf[turn][i][4], c, d);
        const float2 v = unpack(add2(add2(a, b), add2(c, d)));
        return v.x + v.y;
    }
};
template <int H>
__device__ __forceinline__ float sum_all(const f2 (&v)[H]) {
    f2 s = v[0];
#pragma unroll
    for (int k = 1; k < H; ++k) s = add2(s, v[k]);
    const float2 f = unpack(s);
    return f.x + f.y;
}
template <int H>
__device__ __forceinline__ float dot_all(const f2 (&v)[H], const f2 (&w)[H]) {
    f2 s = mul2(v[0], w[0]);
#pragma unroll
    for (int k = 1; k < H; ++k) s = fma2(v[k], w[k], s);
    const float2 f = unpack(s);
    return f.x + f.y;
}

// Takes the mean off; places that are no columns stay zero.
template <typename T, int E>
__device__ __forceinline__ void shift_row(f2 (&v)[E / 2], float mean, const Row& w) {
    const f2 by = both(-mean);
#pragma unroll
    for (int k = 0; k < E / 2; ++k) v[k] = add2(v[k], by);
    if (w.edge)
#pragma unroll
        for (int k = 0; k < E / 2; ++k) {
            const float2 f = unpack(v[k]);
            v[k] = pack(inside<T, E>(w, 2 * k) ? f.x : 0.f, inside<T, E>(w, 2 * k + 1) ? f.y : 0.f);
        }
}
// Takes v to its normalised form in place.
template <typename T, int E, bool WARP>
__device__ __forceinline__ void to_unit(f2 (&v)[E / 2], const NormArgs& p, const Row& w, RowSum<WARP>& sum) {
    if (p.center) shift_row<T, E>(v, sum.one(sum_all(v)) * p.inv_c, w);
    const float rs = rsqrtf(fmaf(sum.one(dot_all(v, v)), p.inv_c, p.eps));
#pragma unroll
    for (int k = 0; k < E / 2; ++k) v[k] = mul2(v[k], both(rs));
}

template <typename T, int E>
__device__ __forceinline__ void scale_by(f2 (&v)[E / 2], const Params<T, E>& prm, int i, const Row& w) {
    f2 t[E / 2];
    prm.get(i, w, t);
#pragma unroll
    for (int k = 0; k < E / 2; ++k) v[k] = mul2(v[k], t[k]);
}
template <typename T, int E>
__device__ __forceinline__ void scale_shift(f2 (&v)[E / 2], const Params<T, E>& prm, int i, bool shift, const Row& w) {
    scale_by<T, E>(v, prm, i, w);
    if (!shift) return;
    f2 t[E / 2];
    prm.get(i + 1, w, t);
#pragma unroll
    for (int k = 0; k < E / 2; ++k) v[k] = add2(v[k], t[k]);
}

// The block's place: its first row, the step to its next ones, and how it holds them.
template <typename T, int E, bool WARP>
__device__ __forceinline__ Row place(const NormArgs& p, long long& row, long long& step) {
    Row w;
    w.C = p.C;
    w.tid = WARP ? threadIdx.x & 31 : threadIdx.x;
    w.tpr = WARP ? 32 : blockDim.x;
    row = WARP ? (long long)blockIdx.x * 4 + (threadIdx.x >> 5) : blockIdx.x;
    step = WARP ? (long long)gridDim.x * 4 : gridDim.x;
    w.wide = p.wide;
    w.phase = p.wide ? (int)(row * p.C % Lay<T, E>::V) : 0;
    w.edge = __any_sync(0xffffffffu, !inside<T, E>(w, 0) || !inside<T, E>(w, E - 1));
    return w;
}
template <typename T, int E, bool WARP>
__device__ __forceinline__ Params<T, E> params(const NormArgs& p, const Row& w, float* smem, float (*buf)[4][8]) {
    Params<T, E> q{smem + (WARP ? (threadIdx.x >> 5) * kParams * 32 * E : 0), w.tpr * E};
    q.put(kWPost, p.w_post, w);
    q.put(kBPost, p.b_post, w);
    q.put(kScale, p.scale, w);
    q.put(kWPre, p.w_pre, w);
    q.put(kBPre, p.b_pre, w);
    if constexpr (!WARP) {
        if (threadIdx.x < 32)
            for (int i = 0; i < 3; ++i) buf[i][threadIdx.x / 8][threadIdx.x % 8] = 0.f;
        __syncthreads();
    }
    return q;
}

// MAXT: the most threads a block has; 128: four warps with a row each. The next row's loads are in flight
// while the present one is worked on.
template <typename T, typename R, int E, int MAXT, bool WARP = MAXT == 128>
__global__ void __launch_bounds__(MAXT, MAXT == 128 ? 1 : E == 8 ? 4 : 2) k_norm_fwd(const NormArgs p) {
    constexpr int H = E / 2;
    __shared__ __align__(16) float buf[3][4][8];
    static_assert(sizeof(buf) <= kStaticSmem, "over_48k counts it");
    extern __shared__ __align__(16) float smem[];
    RowSum<WARP> sum{buf};
    long long row, step;
    const Row w = place<T, E, WARP>(p, row, step);
    const Params<T, E> prm = params<T, E, WARP>(p, w, smem, buf);
    RowRaw<T, T, E> ny{}, ng{};
    RowRaw<T, R, E> nr{};
    auto load = [&](long long r) {
        const bool more = (p.rows - 1 - r) * p.least_row >= 7;
        ld_row<T, T, E>(ny, (const T*)p.y + r * p.y_row, w, more);
        if (p.r) ld_row<T, R, E>(nr, (const R*)p.r + r * p.r_row, w, more);
        if (p.gate) ld_row<T, T, E>(ng, (const T*)p.gate + r * p.gate_row, w, more);
    };
    if (row < p.rows) load(row);
    for (; row < p.rows; row += step) {
        f2 m[H], r[H], g[H];
        if (w.edge) {
            clear_row<T, T, E>(ny, w);
            clear_row<T, R, E>(nr, w);
            clear_row<T, T, E>(ng, w);
        }
        open_row<T, T, E>(ny, m);
        open_row<T, R, E>(nr, r);
        open_row<T, T, E>(ng, g);
        if (row + step < p.rows) load(row + step);
        if (p.gate) {
#pragma unroll
            for (int k = 0; k < H; ++k) m[k] = mul2(m[k], silu2(g[k]));
        }
        if (p.w_post) {
            to_unit<T, E, WARP>(m, p, w, sum);
            scale_shift<T, E>(m, prm, kWPost, p.b_post != nullptr, w);
        }
        if (p.scale) scale_by<T, E>(m, prm, kScale, w);
#pragma unroll
        for (int k = 0; k < H; ++k) r[k] = add2(r[k], m[k]);
        st_row<T, R, E>((R*)p.r_out + row * p.C, w, r);
        if (p.w_pre) {
            to_unit<T, E, WARP>(r, p, w, sum);
            scale_shift<T, E>(r, prm, kWPre, p.b_pre != nullptr, w);
            st_row<T, T, E>((T*)p.o + row * p.C, w, r);
        }
    }
}

// Backward of one norm: g = gradient of its normalised form (already times the weight) is taken in
// place to the gradient of its input: (g - unit mean(g unit) - mean(g)) / spread, the last mean only
// when centred. `gu`, `gs`: the sums of g unit and of g. Places that are no columns end up with
// -mean(g) / spread: the next weight is zero there, and they are never stored.
template <int H>
__device__ __forceinline__ void unit_back(f2 (&g)[H], const f2 (&unit)[H], float rs, float gu, float gs, const NormArgs& p) {
    const f2 ma = both(-gu * p.inv_c), mb = both(-gs * p.inv_c), k2 = both(rs);
#pragma unroll
    for (int k = 0; k < H; ++k) g[k] = mul2(add2(g[k], fma2(unit[k], ma, mb)), k2);
}

__device__ __forceinline__ float2 pair_of(float4 v) { return make_float2(v.x, v.y); }

// Column sums over the rows of a block, in shared memory: a thread's columns are its own, and a sum is touched
// once a row. In registers they made the compiler spill (8190 x 1153 backward 93 us, so 77; 8192 x 4096 247 and
// 193); with room for a fourth block of 96 or 112 registers it spilled again (93 and 81 us).
template <int E> struct Cols {
    float* at;                   // [sum][E / 4][thread][4]
    __device__ __forceinline__ ulonglong2& place(int slot, int e) {
        return *(ulonglong2*)(at + ((slot * (E / 4) + e / 4) * (int)blockDim.x + (int)threadIdx.x) * 4);
    }
    __device__ __forceinline__ void clear(int slots) {
        for (int i = 0; i < slots; ++i)
#pragma unroll
            for (int e = 0; e < E; e += 4) place(i, e) = make_ulonglong2(both(0.f), both(0.f));
    }
    __device__ __forceinline__ void add(int slot, const f2 (&x)[E / 2]) {
        if (slot < 0) return;
#pragma unroll
        for (int e = 0; e < E; e += 4) {
            ulonglong2& s = place(slot, e);
            const ulonglong2 v = s;
            s = make_ulonglong2(add2(v.x, x[e / 2]), add2(v.y, x[e / 2 + 1]));
        }
    }
    __device__ __forceinline__ void add_product(int slot, const f2 (&x)[E / 2], const f2 (&y)[E / 2]) {
        if (slot < 0) return;
#pragma unroll
        for (int e = 0; e < E; e += 4) {
            ulonglong2& s = place(slot, e);
            const ulonglong2 v = s;
            s = make_ulonglong2(fma2(x[e / 2], y[e / 2], v.x), fma2(x[e / 2 + 1], y[e / 2 + 1], v.y));
        }
    }
    __device__ __forceinline__ float one(int slot, int thread, int e) const {
        return at[((slot * (E / 4) + e / 4) * (int)blockDim.x + thread) * 4 + e % 4];
    }
};

// One block takes rows blockIdx, blockIdx + grid, ... (four at a time, one a warp, where a warp holds a
// row) and keeps its column sums until the end; k_norm_sum adds the blocks in order.
template <typename T, typename R, int E, int MAXT, bool WARP = MAXT == 128>
__global__ void __launch_bounds__(MAXT, MAXT == 256 && E == 8 ? 2 : 1) k_norm_bwd(const NormArgs p) {
    using Y = Lay<T, E>;
    constexpr int H = E / 2;
    __shared__ __align__(16) float buf[3][4][8];
    static_assert(sizeof(buf) <= kStaticSmem, "over_48k counts it");
    extern __shared__ __align__(16) float smem[];
    RowSum<WARP> sum{buf};
    long long row, step;
    const Row w = place<T, E, WARP>(p, row, step);
    const Params<T, E> prm = params<T, E, WARP>(p, w, smem, buf);
    Cols<E> cols{smem + kParams * E * blockDim.x};
    cols.clear(p.slots);
    RowRaw<T, T, E> ny{}, ng{}, no{};
    RowRaw<T, R, E> nu{}, nd{};
    auto load = [&](long long r) {
        const bool more = (p.rows - 1 - r) * p.least_row >= 7;
        ld_row<T, T, E>(ny, (const T*)p.y + r * p.y_row, w, more);
        if (p.gate) ld_row<T, T, E>(ng, (const T*)p.gate + r * p.gate_row, w, more);
        if (p.w_pre) {
            ld_row<T, R, E>(nu, (const R*)p.r + r * p.r_row, w, more);
            ld_row<T, T, E>(no, (const T*)p.go + r * p.C, w, more);
        }
        if (p.dr) ld_row<T, R, E>(nd, (const R*)p.dr + r * p.C, w, more);
    };
    if (row < p.rows) load(row);
    for (; row < p.rows; row += step) {
        f2 d[H], y[H], g[H];                                      // d: the gradient of r_out
        f2 u[H], go[H];
        if (w.edge) {
            clear_row<T, T, E>(ny, w);
            clear_row<T, T, E>(ng, w);
            clear_row<T, R, E>(nd, w);
            clear_row<T, R, E>(nu, w);
            clear_row<T, T, E>(no, w);
        }
        open_row<T, T, E>(ny, y);
        open_row<T, T, E>(ng, g);
        open_row<T, R, E>(nd, d);
        open_row<T, R, E>(nu, u);
        open_row<T, T, E>(no, go);
        if (row + step < p.rows) load(row + step);
        f2 m[H], s[H];
#pragma unroll
        for (int k = 0; k < H; ++k) {
            if (p.gate) s[k] = sigmoid2(g[k]);
            m[k] = p.gate ? mul2(y[k], mul2(g[k], s[k])) : y[k];
        }
        // The sums of both norms that do not need each other go together, with one barrier; (g unit) is
        // (g v) / spread, so that the first norm's gradient does not wait for its spread.
        if (p.center) {
            const float4 means = sum.four(p.w_pre ? sum_all(u) : 0.f, p.w_post ? sum_all(m) : 0.f, 0.f, 0.f);
            if (p.w_pre) shift_row<T, E>(u, means.x * p.inv_c, w);
            if (p.w_post) shift_row<T, E>(m, means.y * p.inv_c, w);
        }
        f2 gw[H];
        float suu = 0.f, sgu = 0.f, sg = 0.f;
        if (p.w_pre) {
            prm.get(kWPre, w, gw);
#pragma unroll
            for (int k = 0; k < H; ++k) gw[k] = mul2(go[k], gw[k]);
            suu = dot_all(u, u);
            sgu = dot_all(gw, u);
            if (p.center) sg = sum_all(gw);
        }
        float4 sums = make_float4(0.f, 0.f, 0.f, 0.f);
        if (p.w_pre || p.w_post) sums = sum.four(suu, sgu, sg, p.w_post ? dot_all(m, m) : 0.f);
        if (p.w_pre) {
            const float rs = rsqrtf(fmaf(sums.x, p.inv_c, p.eps));
#pragma unroll
            for (int k = 0; k < H; ++k) u[k] = mul2(u[k], both(rs));
            cols.add(p.slot[kDbPre], go);
            cols.add_product(p.slot[kDwPre], go, u);
            unit_back<H>(gw, u, rs, sums.y * rs, sums.z, p);
#pragma unroll
            for (int k = 0; k < H; ++k) d[k] = add2(d[k], gw[k]);
        }
        if (p.dr_in) st_row<T, R, E>((R*)p.dr_in + row * p.C, w, d);
        float rs = 1.f;
        if (p.w_post) {
            rs = rsqrtf(fmaf(sums.w, p.inv_c, p.eps));
#pragma unroll
            for (int k = 0; k < H; ++k) m[k] = mul2(m[k], both(rs));
        }
        if (p.slot[kDscale] >= 0) {
            f2 v[H];
#pragma unroll
            for (int k = 0; k < H; ++k) v[k] = m[k];
            if (p.w_post) scale_shift<T, E>(v, prm, kWPost, p.b_post != nullptr, w);
            cols.add_product(p.slot[kDscale], v, d);
        }
        if (p.scale) scale_by<T, E>(d, prm, kScale, w);
        if (p.w_post) {
            cols.add(p.slot[kDbPost], d);
            cols.add_product(p.slot[kDwPost], d, m);
            scale_by<T, E>(d, prm, kWPost, w);
            const float a = dot_all(d, m);
            const float2 back = p.center ? pair_of(sum.four(a, sum_all(d), 0.f, 0.f)) : make_float2(sum.one(a), 0.f);
            unit_back<H>(d, m, rs, back.x, back.y, p);
        }
        if (p.gate) {
            if (p.dgate) {
                f2 o[H];
#pragma unroll
                for (int k = 0; k < H; ++k)                       // slope of silu: s + g s (1 - s)
                    o[k] = mul2(mul2(d[k], y[k]), fma2(mul2(g[k], s[k]), fma2(s[k], both(-1.f), both(1.f)), s[k]));
                st_row<T, T, E>((T*)p.dgate + row * p.C, w, o);
            }
#pragma unroll
            for (int k = 0; k < H; ++k) d[k] = mul2(d[k], mul2(g[k], s[k]));
        }
        st_row<T, T, E>((T*)p.dy + row * p.C, w, d);
    }
    // this block's sums: [sum][C]
    float* part = p.part + (long long)blockIdx.x * p.slots * p.C;
    if constexpr (WARP) {
        // rows of the four warps are shifted by their own phases: a column's sums lie in four places
        __syncthreads();
        for (int i = 0; i < p.slots; ++i)
            for (int c = threadIdx.x; c < p.C; c += blockDim.x) {
                float v[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const long long first = (long long)blockIdx.x * 4 + k;
                    const int at = c + (w.wide ? (int)(first * p.C % Y::V) : 0), vec = at / Y::V;
                    v[k] = cols.one(i, k * 32 + vec % 32, vec / 32 * Y::V + at % Y::V);
                }
                part[i * p.C + c] = (v[0] + v[1]) + (v[2] + v[3]);
            }
    } else {
        for (int i = 0; i < p.slots; ++i)
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const int c = Y::col(w, e);
                if (c >= 0 && c < p.C) part[i * p.C + c] = cols.one(i, threadIdx.x, e);
            }
    }
}

// ------------------------------------------------------------------------------------ wide rows
// Rows of over 4096 columns: 16 elements in each thread of a block of as many warps as the row needs.
// ALIGNED: V consecutive columns (16 bytes) at a time; a row that is not 16-byte aligned goes column by
// column instead, neighbouring threads on neighbouring columns. Parameters are read again for every row
// and column sums wait in shared memory: neither fits the registers.
template <typename T, int E, bool ALIGNED> struct WideLay {
    static constexpr int V = Vec<T>::V;
    static __device__ __forceinline__ int col(int e, int tid, int tpr) {
        return ALIGNED ? (e / V * tpr + tid) * V + e % V : e * tpr + tid;
    }
};

// Reads the thread's columns of a row of elements S (T, the residual's type, or fp32 parameters).
template <typename T, typename S, int E, bool ALIGNED>
__device__ __forceinline__ void wide_ld_row(const S* p, int C, int tid, int tpr, f2 (&v)[E / 2]) {
    using Y = WideLay<T, E, ALIGNED>;
    if constexpr (ALIGNED) {
        constexpr int V = Y::V, Q = 16 / sizeof(S);               // columns of a vector; of a 16-byte load
#pragma unroll
        for (int k = 0; k < E / V; ++k) {
            const int c = Y::col(k * V, tid, tpr);
#pragma unroll
            for (int m = 0; m < V; m += Q) {
                const uint4 q = c < C ? *(const uint4*)(p + c + m) : make_uint4(0, 0, 0, 0);
                to_pairs(q, *(f2(*)[Q / 2])(v + (k * V + m) / 2));
            }
        }
    } else {
#pragma unroll
        for (int e = 0; e < E; e += 2) {
            const int c0 = Y::col(e, tid, tpr), c1 = Y::col(e + 1, tid, tpr);
            v[e / 2] = pack(c0 < C ? Io<S>::ld(p + c0) : 0.f, c1 < C ? Io<S>::ld(p + c1) : 0.f);
        }
    }
}
template <typename T, typename S, int E, bool ALIGNED>
__device__ __forceinline__ void wide_st_row(S* p, int C, int tid, int tpr, const f2 (&v)[E / 2]) {
    using Y = WideLay<T, E, ALIGNED>;
    if constexpr (ALIGNED) {
        constexpr int V = Y::V;
#pragma unroll
        for (int k = 0; k < E / V; ++k) {
            const int c = Y::col(k * V, tid, tpr);
            float f[V];
            to_floats(*(const f2(*)[V / 2])(v + k * V / 2), f);
            if (c < C) st_lanes<S, V>(p + c, f);
        }
    } else {
#pragma unroll
        for (int e = 0; e < E; e += 2) {
            const float2 f = unpack(v[e / 2]);
            const int c0 = Y::col(e, tid, tpr), c1 = Y::col(e + 1, tid, tpr);
            if (c0 < C) Io<S>::st(p + c0, f.x);
            if (c1 < C) Io<S>::st(p + c1, f.y);
        }
    }
}

// Sums of a and b over the threads of a block, three buffers in turn so that one barrier a call is enough.
struct WideSum {
    float2 (*buf)[32];
    int turn = 0;
    __device__ __forceinline__ float2 operator()(float a, float b) {
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            a += __shfl_xor_sync(0xffffffffu, a, o);
            b += __shfl_xor_sync(0xffffffffu, b, o);
        }
        if ((threadIdx.x & 31) == 0) buf[turn][threadIdx.x >> 5] = make_float2(a, b);
        __syncthreads();
        const int warps = blockDim.x >> 5, lane = threadIdx.x & 31;
        float2 s = lane < warps ? buf[turn][lane] : make_float2(0.f, 0.f);
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            s.x += __shfl_xor_sync(0xffffffffu, s.x, o);
            s.y += __shfl_xor_sync(0xffffffffu, s.y, o);
        }
        turn = turn == 2 ? 0 : turn + 1;
        return s;
    }
};

// Takes v to its normalised form in place; returns one over its spread.
template <typename T, int E, bool ALIGNED>
__device__ __forceinline__ float wide_to_unit(f2 (&v)[E / 2], const NormArgs& p, int tid, int tpr, WideSum& sum) {
    using Y = WideLay<T, E, ALIGNED>;
    if (p.center) {
        const f2 mean = both(-sum(sum_all(v), 0.f).x * p.inv_c);
#pragma unroll
        for (int k = 0; k < E / 2; ++k) {
            const float2 f = unpack(add2(v[k], mean));
            v[k] = pack(Y::col(2 * k, tid, tpr) < p.C ? f.x : 0.f, Y::col(2 * k + 1, tid, tpr) < p.C ? f.y : 0.f);
        }
    }
    const float rs = rsqrtf(fmaf(sum(dot_all(v, v), 0.f).x, p.inv_c, p.eps));
#pragma unroll
    for (int k = 0; k < E / 2; ++k) v[k] = mul2(v[k], both(rs));
    return rs;
}

// v w + b for the columns of this thread.
template <typename T, int E, bool ALIGNED>
__device__ __forceinline__ void wide_scale_shift(f2 (&v)[E / 2], const float* w, const float* b, int C, int tid, int tpr) {
    f2 t[E / 2];
    wide_ld_row<T, float, E, ALIGNED>(w, C, tid, tpr, t);
#pragma unroll
    for (int k = 0; k < E / 2; ++k) v[k] = mul2(v[k], t[k]);
    if (!b) return;
    wide_ld_row<T, float, E, ALIGNED>(b, C, tid, tpr, t);
#pragma unroll
    for (int k = 0; k < E / 2; ++k) v[k] = add2(v[k], t[k]);
}

template <typename T, typename R, int E, bool ALIGNED, int MAXT>
__global__ void __launch_bounds__(MAXT, 1) k_norm_fwd_wide(const NormArgs p) {
    constexpr int H = E / 2;
    __shared__ float2 buf[3][32];
    static_assert(sizeof(buf) <= kStaticSmem, "over_48k counts it");
    WideSum sum{buf};
    const int tid = threadIdx.x, tpr = blockDim.x;
    const long long row = blockIdx.x;
    f2 m[H], r[H];
    wide_ld_row<T, T, E, ALIGNED>((const T*)p.y + row * p.y_row, p.C, tid, tpr, m);
#pragma unroll
    for (int k = 0; k < H; ++k) r[k] = both(0.f);
    if (p.r) wide_ld_row<T, R, E, ALIGNED>((const R*)p.r + row * p.r_row, p.C, tid, tpr, r);
    if (p.gate) {
        f2 g[H];
        wide_ld_row<T, T, E, ALIGNED>((const T*)p.gate + row * p.gate_row, p.C, tid, tpr, g);
#pragma unroll
        for (int k = 0; k < H; ++k) m[k] = mul2(m[k], silu2(g[k]));
    }
    if (p.w_post) {
        wide_to_unit<T, E, ALIGNED>(m, p, tid, tpr, sum);
        wide_scale_shift<T, E, ALIGNED>(m, p.w_post, p.b_post, p.C, tid, tpr);
    }
    if (p.scale) wide_scale_shift<T, E, ALIGNED>(m, p.scale, nullptr, p.C, tid, tpr);
#pragma unroll
    for (int k = 0; k < H; ++k) r[k] = add2(r[k], m[k]);
    wide_st_row<T, R, E, ALIGNED>((R*)p.r_out + row * p.C, p.C, tid, tpr, r);
    if (p.w_pre) {
        wide_to_unit<T, E, ALIGNED>(r, p, tid, tpr, sum);
        wide_scale_shift<T, E, ALIGNED>(r, p.w_pre, p.b_pre, p.C, tid, tpr);
        wide_st_row<T, T, E, ALIGNED>((T*)p.o + row * p.C, p.C, tid, tpr, r);
    }
}

template <int H>
__device__ __forceinline__ void wide_unit_back(f2 (&g)[H], const f2 (&unit)[H], float rs, const NormArgs& p, WideSum& sum) {
    const float2 s = sum(dot_all(g, unit), p.center ? sum_all(g) : 0.f);
    const f2 ma = both(-s.x * p.inv_c), mb = both(-s.y * p.inv_c), k2 = both(rs);
#pragma unroll
    for (int k = 0; k < H; ++k) g[k] = mul2(add2(g[k], fma2(unit[k], ma, mb)), k2);
}

// Column sums over the rows of a block, [sum][pair][thread]: a thread's columns are its own.
template <int H> struct WideCols {
    f2* at;
    int tpr;
    __device__ __forceinline__ void clear(int wanted) {
        for (int i = 0; i < wanted * H; ++i) at[i * tpr] = both(0.f);
    }
    __device__ __forceinline__ void add(int slot, const f2 (&x)[H]) {
        if (slot < 0) return;
#pragma unroll
        for (int k = 0; k < H; ++k) at[(slot * H + k) * tpr] = add2(at[(slot * H + k) * tpr], x[k]);
    }
    __device__ __forceinline__ void add_product(int slot, const f2 (&x)[H], const f2 (&y)[H]) {
        if (slot < 0) return;
#pragma unroll
        for (int k = 0; k < H; ++k) at[(slot * H + k) * tpr] = fma2(x[k], y[k], at[(slot * H + k) * tpr]);
    }
};

// One block takes rows blockIdx, blockIdx + grid, ... and keeps its column sums until the end.
template <typename T, typename R, int E, bool ALIGNED, int MAXT>
__global__ void __launch_bounds__(MAXT, 1) k_norm_bwd_wide(const NormArgs p) {
    using Y = WideLay<T, E, ALIGNED>;
    constexpr int H = E / 2;
    __shared__ float2 buf[3][32];
    static_assert(sizeof(buf) <= kStaticSmem, "over_48k counts it");
    extern __shared__ __align__(16) unsigned char smem_raw[];
    WideSum sum{buf};
    const int tid = threadIdx.x, tpr = blockDim.x;
    WideCols<H> cols;
    cols.at = (f2*)smem_raw + tid;
    cols.tpr = tpr;
    cols.clear(p.slots);
    for (long long row = blockIdx.x; row < p.rows; row += gridDim.x) {
        f2 d[H], y[H], g[H], u[H], go[H];                         // d: the gradient of r_out
        wide_ld_row<T, T, E, ALIGNED>((const T*)p.y + row * p.y_row, p.C, tid, tpr, y);
        if (p.gate) wide_ld_row<T, T, E, ALIGNED>((const T*)p.gate + row * p.gate_row, p.C, tid, tpr, g);
        if (p.w_pre) {
            wide_ld_row<T, R, E, ALIGNED>((const R*)p.r + row * p.r_row, p.C, tid, tpr, u);
            wide_ld_row<T, T, E, ALIGNED>((const T*)p.go + row * p.C, p.C, tid, tpr, go);
        }
#pragma unroll
        for (int k = 0; k < H; ++k) d[k] = both(0.f);
        if (p.dr) wide_ld_row<T, R, E, ALIGNED>((const R*)p.dr + row * p.C, p.C, tid, tpr, d);
        if (p.w_pre) {
            const float rs = wide_to_unit<T, E, ALIGNED>(u, p, tid, tpr, sum);
            cols.add(p.slot[kDbPre], go);
            cols.add_product(p.slot[kDwPre], go, u);
            wide_scale_shift<T, E, ALIGNED>(go, p.w_pre, nullptr, p.C, tid, tpr);
            wide_unit_back<H>(go, u, rs, p, sum);
#pragma unroll
            for (int k = 0; k < H; ++k) d[k] = add2(d[k], go[k]);
        }
        if (p.dr_in) wide_st_row<T, R, E, ALIGNED>((R*)p.dr_in + row * p.C, p.C, tid, tpr, d);
        f2 m[H], s[H];
#pragma unroll
        for (int k = 0; k < H; ++k) {
            if (p.gate) s[k] = sigmoid2(g[k]);
            m[k] = p.gate ? mul2(y[k], mul2(g[k], s[k])) : y[k];
        }
        float rs = 1.f;
        if (p.w_post) rs = wide_to_unit<T, E, ALIGNED>(m, p, tid, tpr, sum);
        if (p.slot[kDscale] >= 0) {
            f2 v[H];
#pragma unroll
            for (int k = 0; k < H; ++k) v[k] = m[k];
            if (p.w_post) wide_scale_shift<T, E, ALIGNED>(v, p.w_post, p.b_post, p.C, tid, tpr);
            cols.add_product(p.slot[kDscale], v, d);
        }
        if (p.scale) wide_scale_shift<T, E, ALIGNED>(d, p.scale, nullptr, p.C, tid, tpr);
        if (p.w_post) {
            cols.add(p.slot[kDbPost], d);
            cols.add_product(p.slot[kDwPost], d, m);
            wide_scale_shift<T, E, ALIGNED>(d, p.w_post, nullptr, p.C, tid, tpr);
            wide_unit_back<H>(d, m, rs, p, sum);
        }
        if (p.gate) {
            if (p.dgate) {
                f2 o[H];
#pragma unroll
                for (int k = 0; k < H; ++k)                       // slope of silu: s + g s (1 - s)
                    o[k] = mul2(mul2(d[k], y[k]), fma2(mul2(g[k], s[k]), fma2(s[k], both(-1.f), both(1.f)), s[k]));
                wide_st_row<T, T, E, ALIGNED>((T*)p.dgate + row * p.C, p.C, tid, tpr, o);
            }
#pragma unroll
            for (int k = 0; k < H; ++k) d[k] = mul2(d[k], mul2(g[k], s[k]));
        }
        wide_st_row<T, T, E, ALIGNED>((T*)p.dy + row * p.C, p.C, tid, tpr, d);
    }
    // this block's sums: [sum][C]
    float* part = p.part + (long long)blockIdx.x * p.slots * p.C;
#pragma unroll
    for (int w = 0; w < kSums; ++w) {
        if (p.slot[w] < 0) continue;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int c = Y::col(e, tid, tpr);
            const float2 f = unpack(cols.at[(p.slot[w] * H + e / 2) * tpr]);
            if (c < p.C) part[p.slot[w] * p.C + c] = e & 1 ? f.y : f.x;
        }
    }
}

struct SumOut {
    float* to[kSums];
};
// The blocks' column sums: 32 columns a block, each by 16 threads that take every 16th block; their sums
// are added in order.
__global__ void k_norm_sum(const float* part, int blocks, int n, int C, SumOut out) {
    __shared__ float red[16][32];
    const int i = blockIdx.x * 32 + threadIdx.x;
    float s = 0.f;
    if (i < n) {
#pragma unroll 8
        for (int b = threadIdx.y; b < blocks; b += 16) s += part[(long long)b * n + i];
    }
    red[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.y == 0 && i < n) {
        s = 0.f;
#pragma unroll
        for (int k = 0; k < 16; ++k) s += red[k][threadIdx.x];
        out.to[i / C][i % C] = s;
    }
}

// ---------------------------------------------------------------------------------------- host
bool make_args(const gspn_norm_desc* d, NormArgs* p) {
    if (!d) return false;
    if (d->rows < 0 || d->C < 1 || !dtype_ok(d->dtype)) return false;
    if (d->res_dtype != GSPN_F32 && d->res_dtype != d->dtype) return false;
    if ((d->center != 0 && d->center != 1) || !(d->eps >= 0.f)) return false;
    if (d->y_row < 0 || d->gate_row < 0 || d->r_row < 0) return false;
    *p = NormArgs{};
    p->rows = d->rows; p->C = d->C; p->center = d->center; p->eps = d->eps;
    p->inv_c = 1.f / (float)d->C;
    p->y_row = d->y_row; p->gate_row = d->gate_row; p->r_row = d->r_row;
    return true;
}

// Blocks: what fits the SMs at once by their registers (threads an SM: backward 512, 256 with 16 elements;
// forward twice that), in whole periods of the phases, and no more than there are rows. Wide rows have
// a block each, forward.
int blocks_for(const gspn_norm_desc& d, bool bwd) {
    const Shape s = shape_for(d.C);
    const long long groups = s.warp ? ((long long)d.rows + 3) / 4 : d.rows;
    if (s.wide && !bwd) return d.rows;
    const int fill = bwd ? (s.e == 8 ? 512 : 256) : s.e == 8 ? 1024 : 512;
    long long n = (long long)device_sm_count() * (s.threads >= fill ? 1 : fill / s.threads);
    n = n / 8 * 8;
    n = groups < n ? groups : n;
    return n > 0 ? (int)n : 1;
}

template <bool FWD, typename T, typename R>
cudaError_t by_shape(const NormArgs& p, int blocks, cudaStream_t st) {
    const Shape s = shape_for(p.C);
    const size_t smem = smem_for(s, FWD ? 0 : p.slots);
    auto go = [&](auto kernel) {
        cudaError_t e = cudaSuccess;
        if (over_48k(smem)) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostSmem);
        if (e == cudaSuccess) kernel<<<blocks, s.threads, smem, st>>>(p);
        return e;
    };
    if constexpr (FWD) {
        if (s.warp) return go(k_norm_fwd<T, R, 8, 128>);
        if (!s.wide && s.e == 8) return go(k_norm_fwd<T, R, 8, 256>);
        if (!s.wide) return go(k_norm_fwd<T, R, 16, 256>);
        if (s.threads <= 512) return p.aligned ? go(k_norm_fwd_wide<T, R, 16, true, 512>) : go(k_norm_fwd_wide<T, R, 16, false, 512>);
        return p.aligned ? go(k_norm_fwd_wide<T, R, 16, true, 1024>) : go(k_norm_fwd_wide<T, R, 16, false, 1024>);
    } else {
        if (s.warp) return go(k_norm_bwd<T, R, 8, 128>);
        if (!s.wide && s.e == 8) return go(k_norm_bwd<T, R, 8, 256>);
        if (!s.wide) return go(k_norm_bwd<T, R, 16, 256>);
        if (s.threads <= 512) return p.aligned ? go(k_norm_bwd_wide<T, R, 16, true, 512>) : go(k_norm_bwd_wide<T, R, 16, false, 512>);
        return p.aligned ? go(k_norm_bwd_wide<T, R, 16, true, 1024>) : go(k_norm_bwd_wide<T, R, 16, false, 1024>);
    }
}
template <bool FWD>
cudaError_t by_type(const gspn_norm_desc& d, const NormArgs& p, int blocks, cudaStream_t st) {
    if (d.dtype == GSPN_F32) return by_shape<FWD, float, float>(p, blocks, st);
    if (d.res_dtype == GSPN_F32) return by_shape<FWD, __nv_bfloat16, float>(p, blocks, st);
    return by_shape<FWD, __nv_bfloat16, __nv_bfloat16>(p, blocks, st);
}
// The least stride of the tensors' rows.
long long least_row(const NormArgs& p, bool gate, bool r) {
    long long s = p.C < p.y_row ? p.C : p.y_row;
    if (gate && p.gate_row < s) s = p.gate_row;
    if (r && p.r_row < s) s = p.r_row;
    return s;
}
// True where a tensor's rows start at the phase of rows of C elements from a 16-byte border.
bool phased(const void* p, long long row, int C, int dtype) {
    return aligned_to(p, 16) && (row - C) % (dtype == GSPN_F32 ? 4 : 8) == 0;
}

}  // namespace
}  // namespace seq
}  // namespace gspn

using namespace gspn;
using namespace gspn::seq;

extern "C" {

size_t gspn_norm_workspace_size(const gspn_norm_desc* desc, int for_backward) {
    NormArgs p;
    if (!make_args(desc, &p) || p.C > kMaxC) return 0;
    if (!for_backward) return 256;
    return 256 + align256((size_t)blocks_for(*desc, true) * kSums * p.C * sizeof(float));
}

gspn_status gspn_norm_forward(const gspn_norm_desc* desc, const void* y, const void* gate, const float* w_post,
                              const float* b_post, const float* scale, const void* r, const float* w_pre,
                              const float* b_pre, void* r_out, void* o, void* stream) {
    NormArgs p;
    if (!make_args(desc, &p)) return GSPN_ERR_INVALID_ARG;
    if ((b_post && !w_post) || (b_pre && !w_pre)) return GSPN_ERR_INVALID_ARG;
    if (p.rows > 0 && (!y || !r_out || (w_pre != nullptr) != (o != nullptr))) return GSPN_ERR_INVALID_ARG;
    if (p.C > kMaxC) return GSPN_ERR_UNSUPPORTED;
    const size_t es = dtype_size(desc->dtype), rs = dtype_size(desc->res_dtype);
    for (const void* q : {y, gate, (const void*)o})
        if (!aligned_to(q, es)) return GSPN_ERR_ALIGNMENT;
    for (const void* q : {r, (const void*)r_out})
        if (!aligned_to(q, rs)) return GSPN_ERR_ALIGNMENT;
    for (const float* q : {w_post, b_post, scale, w_pre, b_pre})
        if (!aligned_to(q, 4)) return GSPN_ERR_ALIGNMENT;
    if (p.rows == 0) return GSPN_OK;
    p.y = y; p.gate = gate; p.r = r; p.w_post = w_post; p.b_post = b_post; p.scale = scale; p.w_pre = w_pre;
    p.b_pre = b_pre; p.r_out = r_out; p.o = o;
    // the phase is the storage type's: eight bf16 columns are 32 bytes of an fp32 stream
    p.wide = phased(y, p.y_row, p.C, desc->dtype) && (!gate || phased(gate, p.gate_row, p.C, desc->dtype)) &&
             (!r || phased(r, p.r_row, p.C, desc->dtype)) && aligned_to(r_out, 16) && aligned_to(o, 16);
    p.least_row = least_row(p, gate != nullptr, r != nullptr);
    p.aligned = p.wide && p.C % 8 == 0;
    for (const float* q : {w_post, b_post, scale, w_pre, b_pre}) p.aligned = p.aligned && aligned_to(q, 16);
    if (by_type<true>(*desc, p, blocks_for(*desc, false), (cudaStream_t)stream) != cudaSuccess) return GSPN_ERR_CUDA;
    return last_status();
}

gspn_status gspn_norm_backward(const gspn_norm_desc* desc, const void* y, const void* gate, const float* w_post,
                               const float* b_post, const float* scale, const void* r_out, const float* w_pre,
                               const void* dr, const void* go, void* dy, void* dr_in, void* dgate, float* dw_post,
                               float* db_post, float* dscale, float* dw_pre, float* db_pre, void* ws, size_t ws_bytes,
                               void* stream) {
    NormArgs p;
    if (!make_args(desc, &p)) return GSPN_ERR_INVALID_ARG;
    if (p.rows > 0 && (!y || !dy || (!dr && !w_pre))) return GSPN_ERR_INVALID_ARG;
    if (p.rows > 0 && ((w_pre != nullptr) != (go != nullptr) || (w_pre && !r_out))) return GSPN_ERR_INVALID_ARG;
    if ((dgate && !gate) || ((dw_post || db_post || b_post) && !w_post) || (dscale && !scale) ||
        ((dw_pre || db_pre) && !w_pre) || !ws)
        return GSPN_ERR_INVALID_ARG;
    const size_t es = dtype_size(desc->dtype), rs = dtype_size(desc->res_dtype);
    for (const void* q : {y, gate, go, (const void*)dy, (const void*)dgate})
        if (!aligned_to(q, es)) return GSPN_ERR_ALIGNMENT;
    for (const void* q : {r_out, dr, (const void*)dr_in})
        if (!aligned_to(q, rs)) return GSPN_ERR_ALIGNMENT;
    float* const outs[kSums] = {dw_post, db_post, dscale, dw_pre, db_pre};
    for (const float* q : {w_post, b_post, scale, w_pre, (const float*)dw_post, (const float*)db_post,
                           (const float*)dscale, (const float*)dw_pre, (const float*)db_pre})
        if (!aligned_to(q, 4)) return GSPN_ERR_ALIGNMENT;
    if (!aligned_to(ws, 16)) return GSPN_ERR_ALIGNMENT;
    SumOut to{};
    for (int i = 0; i < kSums; ++i) {
        p.slot[i] = outs[i] ? p.slots : -1;
        if (outs[i]) to.to[p.slots++] = outs[i];
    }
    // the column sums of wide rows live in shared memory
    if (p.C > kMaxC || smem_for(shape_for(p.C), p.slots) > 200 * 1024) return GSPN_ERR_UNSUPPORTED;
    if (ws_bytes < gspn_norm_workspace_size(desc, 1)) return GSPN_ERR_WORKSPACE;
    p.y = y; p.gate = gate; p.r = r_out; p.w_post = w_post; p.b_post = b_post; p.scale = scale; p.w_pre = w_pre;
    p.dr = dr; p.go = go; p.dy = dy; p.dr_in = dr_in; p.dgate = dgate;
    p.part = (float*)((char*)ws + 256);
    p.wide = phased(y, p.y_row, p.C, desc->dtype) && (!gate || phased(gate, p.gate_row, p.C, desc->dtype)) &&
             (!w_pre || phased(r_out, p.r_row, p.C, desc->dtype)) && aligned_to(dr, 16) && aligned_to(go, 16) &&
             aligned_to(dy, 16) && aligned_to(dr_in, 16) && aligned_to(dgate, 16);
    p.least_row = least_row(p, gate != nullptr, w_pre != nullptr);
    p.aligned = p.wide && p.C % 8 == 0;
    for (const float* q : {w_post, b_post, scale, w_pre}) p.aligned = p.aligned && aligned_to(q, 16);
    const int blocks = blocks_for(*desc, true);
    cudaStream_t st = (cudaStream_t)stream;
    if (by_type<false>(*desc, p, blocks, st) != cudaSuccess) return GSPN_ERR_CUDA;
    const int n = p.slots * p.C;
    if (n > 0) k_norm_sum<<<(n + 31) / 32, dim3(32, 16), 0, st>>>(p.part, blocks, n, p.C, to);
    return last_status();
}

}  // extern "C"
