// k_norm.cu -- the norms around a block, in one pass over its rows:
//   m = y silu(gate);  v = norm(m) w_post + b_post;  r_out = r + scale v;  o = norm(r_out) w_pre + b_pre
// with norm(v) = v / sqrt(mean(v^2) + eps), of v - mean(v) when centred.
//
// Some tens of operations per element: memory traffic bounds it. A row stays in the registers of TPR
// threads (one warp for narrow rows, a block for wide ones) from its load to its last store, so every
// tensor crosses HBM once. Means are taken before squares of differences, from registers, so that
// no cancellation enters. Statistics and sums are fp32.
#include "seq_common.cuh"

namespace gspn {
namespace seq {
namespace {

constexpr int kMaxC = 16384;
enum { kDwPost, kDbPost, kDscale, kDwPre, kDbPre, kSums };

struct NormArgs {
    int rows, C, center;
    float eps, inv_c;
    long long y_row, gate_row, r_row;
    const void *y, *gate, *r;
    const float *w_post, *b_post, *scale, *w_pre, *b_pre;
    void *r_out, *o;
    // backward
    const void *dr, *go;
    void *dy, *dr_in, *dgate;
    float* part;                 // [block][slot of sum][C]
    int slot[kSums], slots;      // which sums are wanted, and where; -1: not
};

// Which column an element is: TPR threads hold V consecutive columns each, CH times over. Rows that are
// not 16-byte aligned go column by column instead, neighbouring threads on neighbouring columns.
template <int TPR, int V, bool WIDE>
__device__ __forceinline__ int col_of(int k, int j, int tid) {
    return WIDE ? (k * TPR + tid) * V + j : (k * V + j) * TPR + tid;
}

// V elements of type E (V * sizeof(E) = 16 or 32 bytes), wide.
template <typename E, int V>
__device__ __forceinline__ void ld_wide(const E* p, float (&v)[V]) {
    if constexpr (V * sizeof(E) == 32) {
        float a[V / 2], b[V / 2];
        ld_lanes<E, V / 2>(p, a);
        ld_lanes<E, V / 2>(p + V / 2, b);
#pragma unroll
        for (int j = 0; j < V / 2; ++j) { v[j] = a[j]; v[j + V / 2] = b[j]; }
    } else {
        ld_lanes<E, V>(p, v);
    }
}
template <typename E, int TPR, int CH, int V, bool WIDE>
__device__ __forceinline__ void ld_row(const E* p, int C, int tid, float (&v)[CH][V]) {
#pragma unroll
    for (int k = 0; k < CH; ++k) {
        if constexpr (WIDE) {
            const int c = col_of<TPR, V, true>(k, 0, tid);
            if (c < C) {
                ld_wide<E, V>(p + c, v[k]);
            } else {
#pragma unroll
                for (int j = 0; j < V; ++j) v[k][j] = 0.f;
            }
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int c = col_of<TPR, V, false>(k, j, tid);
                v[k][j] = c < C ? Io<E>::ld(p + c) : 0.f;
            }
        }
    }
}
template <typename E, int TPR, int CH, int V, bool WIDE>
__device__ __forceinline__ void st_row(E* p, int C, int tid, const float (&v)[CH][V]) {
#pragma unroll
    for (int k = 0; k < CH; ++k) {
        if constexpr (WIDE) {
            const int c = col_of<TPR, V, true>(k, 0, tid);
            if (c < C) st_lanes<E, V>(p + c, v[k]);
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int c = col_of<TPR, V, false>(k, j, tid);
                if (c < C) Io<E>::st(p + c, v[k][j]);
            }
        }
    }
}

// Sum of a and b over the TPR threads of a row. `buf`: two floats for each warp, a fresh one each call
// in turn of three, so that one barrier a call is enough.
template <int TPR>
struct RowSum {
    float2 (*buf)[TPR / 32];
    int turn = 0;
    __device__ __forceinline__ float2 operator()(float a, float b) {
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            a += __shfl_xor_sync(0xffffffffu, a, o);
            b += __shfl_xor_sync(0xffffffffu, b, o);
        }
        if constexpr (TPR == 32) {
            return make_float2(a, b);
        } else {
            const int w = threadIdx.x >> 5;
            if ((threadIdx.x & 31) == 0) buf[turn][w] = make_float2(a, b);
            __syncthreads();
            float2 s = make_float2(0.f, 0.f);
#pragma unroll
            for (int i = 0; i < TPR / 32; ++i) {
                const float2 v = buf[turn][i];
                s.x += v.x;
                s.y += v.y;
            }
            turn = turn == 2 ? 0 : turn + 1;
            return s;
        }
    }
};

// Takes v to its normalised form in place; returns one over its spread.
template <int TPR, int CH, int V, bool WIDE>
__device__ __forceinline__ float to_unit(float (&v)[CH][V], const NormArgs& p, int tid, RowSum<TPR>& sum) {
    if (p.center) {
        float s = 0.f;
#pragma unroll
        for (int k = 0; k < CH; ++k)
#pragma unroll
            for (int j = 0; j < V; ++j) s += v[k][j];
        const float mean = sum(s, 0.f).x * p.inv_c;
#pragma unroll
        for (int k = 0; k < CH; ++k)
#pragma unroll
            for (int j = 0; j < V; ++j) v[k][j] = col_of<TPR, V, WIDE>(k, j, tid) < p.C ? v[k][j] - mean : 0.f;
    }
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < CH; ++k)
#pragma unroll
        for (int j = 0; j < V; ++j) s = fmaf(v[k][j], v[k][j], s);
    const float rs = rsqrtf(fmaf(sum(s, 0.f).x, p.inv_c, p.eps));
#pragma unroll
    for (int k = 0; k < CH; ++k)
#pragma unroll
        for (int j = 0; j < V; ++j) v[k][j] *= rs;
    return rs;
}

// v w + b for the columns of this thread.
template <int TPR, int CH, int V, bool WIDE>
__device__ __forceinline__ void scale_shift(float (&v)[CH][V], const float* w, const float* b, int C, int tid) {
    float t[CH][V];
    ld_row<float, TPR, CH, V, WIDE>(w, C, tid, t);
#pragma unroll
    for (int k = 0; k < CH; ++k)
#pragma unroll
        for (int j = 0; j < V; ++j) v[k][j] *= t[k][j];
    if (!b) return;
    ld_row<float, TPR, CH, V, WIDE>(b, C, tid, t);
#pragma unroll
    for (int k = 0; k < CH; ++k)
#pragma unroll
        for (int j = 0; j < V; ++j) v[k][j] += t[k][j];
}

template <typename T, typename R, int TPR, int CH, bool WIDE>
__global__ void __launch_bounds__(TPR == 32 ? 128 : TPR) k_norm_fwd(const NormArgs p) {
    constexpr int V = Vec<T>::V, RPB = TPR == 32 ? 4 : 1;
    __shared__ float2 buf[3][TPR / 32];
    RowSum<TPR> sum{buf};
    const int tid = TPR == 32 ? threadIdx.x & 31 : threadIdx.x;
    const long long row = (long long)blockIdx.x * RPB + (TPR == 32 ? threadIdx.x >> 5 : 0);
    if (row >= p.rows) return;               // whole warps only where RPB > 1; no barrier is used there
    float m[CH][V], r[CH][V];
    ld_row<T, TPR, CH, V, WIDE>((const T*)p.y + row * p.y_row, p.C, tid, m);
    if (p.r) {
        ld_row<R, TPR, CH, V, WIDE>((const R*)p.r + row * p.r_row, p.C, tid, r);
    } else {
#pragma unroll
        for (int k = 0; k < CH; ++k)
#pragma unroll
            for (int j = 0; j < V; ++j) r[k][j] = 0.f;
    }
    if (p.gate) {
        float g[CH][V];
        ld_row<T, TPR, CH, V, WIDE>((const T*)p.gate + row * p.gate_row, p.C, tid, g);
#pragma unroll
        for (int k = 0; k < CH; ++k)
#pragma unroll
            for (int j = 0; j < V; ++j) m[k][j] *= silu(g[k][j]);
    }
    if (p.w_post) {
        to_unit<TPR, CH, V, WIDE>(m, p, tid, sum);
        scale_shift<TPR, CH, V, WIDE>(m, p.w_post, p.b_post, p.C, tid);
    }
    if (p.scale) scale_shift<TPR, CH, V, WIDE>(m, p.scale, nullptr, p.C, tid);
#pragma unroll
    for (int k = 0; k < CH; ++k)
#pragma unroll
        for (int j = 0; j < V; ++j) r[k][j] += m[k][j];
    st_row<R, TPR, CH, V, WIDE>((R*)p.r_out + row * p.C, p.C, tid, r);
    if (p.w_pre) {
        to_unit<TPR, CH, V, WIDE>(r, p, tid, sum);
        scale_shift<TPR, CH, V, WIDE>(r, p.w_pre, p.b_pre, p.C, tid);
        st_row<T, TPR, CH, V, WIDE>((T*)p.o + row * p.C, p.C, tid, r);
    }
}

// Backward of one norm: g = gradient of its normalised form (already times the weight) is taken in
// place to the gradient of its input: (g - unit mean(g unit) - mean(g)) / spread, the last mean only
// when centred.
template <int TPR, int CH, int V, bool WIDE>
__device__ __forceinline__ void unit_back(float (&g)[CH][V], const float (&unit)[CH][V], float rs, const NormArgs& p,
                                          int tid, RowSum<TPR>& sum) {
    float a = 0.f, b = 0.f;
#pragma unroll
    for (int k = 0; k < CH; ++k)
#pragma unroll
        for (int j = 0; j < V; ++j) {
            a = fmaf(g[k][j], unit[k][j], a);
            b += g[k][j];
        }
    const float2 s = sum(a, b);
    const float ma = s.x * p.inv_c, mb = p.center ? s.y * p.inv_c : 0.f;
#pragma unroll
    for (int k = 0; k < CH; ++k)
#pragma unroll
        for (int j = 0; j < V; ++j) g[k][j] = (g[k][j] - fmaf(unit[k][j], ma, mb)) * rs;
}

// Adds this row's share of a column sum. A thread's columns of `acc` are its own.
template <int TPR, int CH, int V, bool WIDE>
__device__ __forceinline__ void add_cols(float* acc, int slot, int C, int tid, const float (&v)[CH][V]) {
    if (slot < 0) return;
    float* a = acc + (long long)slot * C;
#pragma unroll
    for (int k = 0; k < CH; ++k) {
        if constexpr (WIDE) {
            const int c = col_of<TPR, V, true>(k, 0, tid);
            if (c < C) {
#pragma unroll
                for (int j = 0; j < V; j += 4) {
                    float4 f = *(float4*)(a + c + j);
                    f.x += v[k][j]; f.y += v[k][j + 1]; f.z += v[k][j + 2]; f.w += v[k][j + 3];
                    *(float4*)(a + c + j) = f;
                }
            }
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int c = col_of<TPR, V, false>(k, j, tid);
                if (c < C) a[c] += v[k][j];
            }
        }
    }
}

// One block takes rows blockIdx, blockIdx + grid, ... and keeps its column sums in shared memory, each
// column in the hands of one thread; narrow rows have one set of sums for each of the four warps,
// added in order at the end. k_norm_sum adds the blocks in order.
template <typename T, typename R, int TPR, int CH, bool WIDE>
__global__ void __launch_bounds__(TPR == 32 ? 128 : TPR) k_norm_bwd(const NormArgs p) {
    constexpr int V = Vec<T>::V, RPB = TPR == 32 ? 4 : 1;
    __shared__ float2 buf[3][TPR / 32];
    extern __shared__ __align__(16) float acc_all[];
    RowSum<TPR> sum{buf};
    const int tid = TPR == 32 ? threadIdx.x & 31 : threadIdx.x;
    const int grp = TPR == 32 ? threadIdx.x >> 5 : 0;
    const int n = p.slots * p.C;
    for (int i = threadIdx.x; i < RPB * n; i += blockDim.x) acc_all[i] = 0.f;
    __syncthreads();
    float* acc = acc_all + grp * n;
    for (long long row = (long long)blockIdx.x * RPB + grp; row < p.rows; row += (long long)gridDim.x * RPB) {
        float d[CH][V];                       // the gradient of r_out
        if (p.dr) {
            ld_row<R, TPR, CH, V, WIDE>((const R*)p.dr + row * p.C, p.C, tid, d);
        } else {
#pragma unroll
            for (int k = 0; k < CH; ++k)
#pragma unroll
                for (int j = 0; j < V; ++j) d[k][j] = 0.f;
        }
        float m[CH][V], g[CH][V], y[CH][V];
        ld_row<T, TPR, CH, V, WIDE>((const T*)p.y + row * p.y_row, p.C, tid, y);
        if (p.gate) ld_row<T, TPR, CH, V, WIDE>((const T*)p.gate + row * p.gate_row, p.C, tid, g);
        if (p.w_pre) {
            float u[CH][V], go[CH][V];
            ld_row<R, TPR, CH, V, WIDE>((const R*)p.r + row * p.r_row, p.C, tid, u);
            ld_row<T, TPR, CH, V, WIDE>((const T*)p.go + row * p.C, p.C, tid, go);
            const float rs = to_unit<TPR, CH, V, WIDE>(u, p, tid, sum);
            add_cols<TPR, CH, V, WIDE>(acc, p.slot[kDbPre], p.C, tid, go);
            float t[CH][V];
#pragma unroll
            for (int k = 0; k < CH; ++k)
#pragma unroll
                for (int j = 0; j < V; ++j) t[k][j] = go[k][j] * u[k][j];
            add_cols<TPR, CH, V, WIDE>(acc, p.slot[kDwPre], p.C, tid, t);
            scale_shift<TPR, CH, V, WIDE>(go, p.w_pre, nullptr, p.C, tid);
            unit_back<TPR, CH, V, WIDE>(go, u, rs, p, tid, sum);
#pragma unroll
            for (int k = 0; k < CH; ++k)
#pragma unroll
                for (int j = 0; j < V; ++j) d[k][j] += go[k][j];
        }
        if (p.dr_in) st_row<R, TPR, CH, V, WIDE>((R*)p.dr_in + row * p.C, p.C, tid, d);
#pragma unroll
        for (int k = 0; k < CH; ++k)
#pragma unroll
            for (int j = 0; j < V; ++j) m[k][j] = p.gate ? y[k][j] * silu(g[k][j]) : y[k][j];
        float rs = 1.f;
        if (p.w_post) rs = to_unit<TPR, CH, V, WIDE>(m, p, tid, sum);
        if (p.slot[kDscale] >= 0) {
            float v[CH][V];
#pragma unroll
            for (int k = 0; k < CH; ++k)
#pragma unroll
                for (int j = 0; j < V; ++j) v[k][j] = m[k][j];
            if (p.w_post) scale_shift<TPR, CH, V, WIDE>(v, p.w_post, p.b_post, p.C, tid);
#pragma unroll
            for (int k = 0; k < CH; ++k)
#pragma unroll
                for (int j = 0; j < V; ++j) v[k][j] *= d[k][j];
            add_cols<TPR, CH, V, WIDE>(acc, p.slot[kDscale], p.C, tid, v);
        }
        if (p.scale) scale_shift<TPR, CH, V, WIDE>(d, p.scale, nullptr, p.C, tid);
        if (p.w_post) {
            add_cols<TPR, CH, V, WIDE>(acc, p.slot[kDbPost], p.C, tid, d);
            if (p.slot[kDwPost] >= 0) {
                float t[CH][V];
#pragma unroll
                for (int k = 0; k < CH; ++k)
#pragma unroll
                    for (int j = 0; j < V; ++j) t[k][j] = d[k][j] * m[k][j];
                add_cols<TPR, CH, V, WIDE>(acc, p.slot[kDwPost], p.C, tid, t);
            }
            scale_shift<TPR, CH, V, WIDE>(d, p.w_post, nullptr, p.C, tid);
            unit_back<TPR, CH, V, WIDE>(d, m, rs, p, tid, sum);
        }
        if (p.gate) {
            if (p.dgate) {
                float t[CH][V];
#pragma unroll
                for (int k = 0; k < CH; ++k)
#pragma unroll
                    for (int j = 0; j < V; ++j) t[k][j] = d[k][j] * y[k][j] * silu_slope(g[k][j]);
                st_row<T, TPR, CH, V, WIDE>((T*)p.dgate + row * p.C, p.C, tid, t);
            }
#pragma unroll
            for (int k = 0; k < CH; ++k)
#pragma unroll
                for (int j = 0; j < V; ++j) d[k][j] *= silu(g[k][j]);
        }
        st_row<T, TPR, CH, V, WIDE>((T*)p.dy + row * p.C, p.C, tid, d);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += blockDim.x) {
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < RPB; ++w) s += acc_all[w * n + i];
        p.part[(long long)blockIdx.x * n + i] = s;
    }
}

struct SumOut {
    float* to[kSums];
};
// The blocks' column sums in order: 32 columns a block, 8 rows of threads share the blocks.
__global__ void k_norm_sum(const float* part, int blocks, int n, int C, SumOut out) {
    __shared__ float red[8][32];
    const int i = blockIdx.x * 32 + threadIdx.x;
    float s = 0.f;
    if (i < n)
        for (int b = threadIdx.y; b < blocks; b += 8) s += part[(long long)b * n + i];
    red[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.y == 0 && i < n) {
        s = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) s += red[k][threadIdx.x];
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

// How a row is held: threads and vectors for each.
struct Shape {
    int tpr, ch;
};
Shape shape_for(int C, int V) {
    const int n = (C + V - 1) / V;
    if (n <= 32) return {32, 1};
    if (n <= 64) return {32, 2};
    if (n <= 128) return {32, 4};
    if (n <= 256) return {128, 2};
    if (n <= 512) return {256, 2};
    if (n <= 1024) return {512, 2};
    if (n <= 2048) return {512, 4};
    return {1024, 4};
}
constexpr size_t kSumSmem = 200 * 1024;
int bwd_blocks(const gspn_norm_desc& d) {
    const Shape s = shape_for(d.C, d.dtype == GSPN_F32 ? 4 : 8);
    const int rpb = s.tpr == 32 ? 4 : 1;
    const long long groups = ((long long)d.rows + rpb - 1) / rpb;
    const long long most = 2LL * device_sm_count() * (s.tpr <= 128 ? 2 : 1);
    const long long n = groups < most ? groups : most;
    return n > 0 ? (int)n : 1;
}

template <bool FWD, typename T, typename R, int TPR, int CH>
cudaError_t launch(const NormArgs& p, bool wide, int blocks, cudaStream_t st) {
    constexpr int RPB = TPR == 32 ? 4 : 1, threads = TPR == 32 ? 128 : TPR;
    if constexpr (FWD) {
        if (wide) k_norm_fwd<T, R, TPR, CH, true><<<blocks, threads, 0, st>>>(p);
        else k_norm_fwd<T, R, TPR, CH, false><<<blocks, threads, 0, st>>>(p);
        return cudaSuccess;
    } else {
        const size_t smem = (size_t)RPB * p.slots * p.C * sizeof(float);
        auto go = [&](auto kernel) {
            cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
            if (e == cudaSuccess) kernel<<<blocks, threads, smem, st>>>(p);
            return e;
        };
        return wide ? go(k_norm_bwd<T, R, TPR, CH, true>) : go(k_norm_bwd<T, R, TPR, CH, false>);
    }
}
template <bool FWD, typename T, typename R>
cudaError_t by_shape(const NormArgs& p, bool wide, int blocks, cudaStream_t st) {
    const Shape s = shape_for(p.C, Vec<T>::V);
    if (s.tpr == 32) {
        if (s.ch == 1) return launch<FWD, T, R, 32, 1>(p, wide, blocks, st);
        if (s.ch == 2) return launch<FWD, T, R, 32, 2>(p, wide, blocks, st);
        return launch<FWD, T, R, 32, 4>(p, wide, blocks, st);
    }
    if (s.tpr == 128) return launch<FWD, T, R, 128, 2>(p, wide, blocks, st);
    if (s.tpr == 256) return launch<FWD, T, R, 256, 2>(p, wide, blocks, st);
    if (s.tpr == 512 && s.ch == 2) return launch<FWD, T, R, 512, 2>(p, wide, blocks, st);
    if (s.tpr == 512) return launch<FWD, T, R, 512, 4>(p, wide, blocks, st);
    if constexpr (sizeof(T) == 4) return launch<FWD, T, R, 1024, 4>(p, wide, blocks, st);   // bf16 rows end at 512 x 4
    return cudaErrorInvalidValue;
}
template <bool FWD>
cudaError_t by_type(const gspn_norm_desc& d, const NormArgs& p, bool wide, int blocks, cudaStream_t st) {
    if (d.dtype == GSPN_F32) return by_shape<FWD, float, float>(p, wide, blocks, st);
    if (d.res_dtype == GSPN_F32) return by_shape<FWD, __nv_bfloat16, float>(p, wide, blocks, st);
    return by_shape<FWD, __nv_bfloat16, __nv_bfloat16>(p, wide, blocks, st);
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
    return 256 + align256((size_t)bwd_blocks(*desc) * kSums * p.C * sizeof(float));
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
    bool wide = (p.C * es) % 16 == 0 && wide_ok(y, p.y_row, 0, es) && (!gate || wide_ok(gate, p.gate_row, 0, es)) &&
                (!r || wide_ok(r, p.r_row, 0, rs)) && aligned_to(r_out, 16) && aligned_to(o, 16);
    for (const float* q : {w_post, b_post, scale, w_pre, b_pre}) wide = wide && aligned_to(q, 16);
    const int rpb = shape_for(p.C, desc->dtype == GSPN_F32 ? 4 : 8).tpr == 32 ? 4 : 1;
    if (by_type<true>(*desc, p, wide, (p.rows + rpb - 1) / rpb, (cudaStream_t)stream) != cudaSuccess) return GSPN_ERR_CUDA;
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
    const int rpb = shape_for(p.C, desc->dtype == GSPN_F32 ? 4 : 8).tpr == 32 ? 4 : 1;
    // the column sums of a block live in shared memory
    if (p.C > kMaxC || (size_t)rpb * p.slots * p.C * sizeof(float) > kSumSmem) return GSPN_ERR_UNSUPPORTED;
    if (ws_bytes < gspn_norm_workspace_size(desc, 1)) return GSPN_ERR_WORKSPACE;
    p.y = y; p.gate = gate; p.r = r_out; p.w_post = w_post; p.b_post = b_post; p.scale = scale; p.w_pre = w_pre;
    p.dr = dr; p.go = go; p.dy = dy; p.dr_in = dr_in; p.dgate = dgate;
    p.part = (float*)((char*)ws + 256);
    bool wide = (p.C * es) % 16 == 0 && wide_ok(y, p.y_row, 0, es) && (!gate || wide_ok(gate, p.gate_row, 0, es)) &&
                (!w_pre || wide_ok(r_out, p.r_row, 0, rs)) && aligned_to(dr, 16) && aligned_to(go, 16) &&
                aligned_to(dy, 16) && aligned_to(dr_in, 16) && aligned_to(dgate, 16);
    for (const float* q : {w_post, b_post, scale, w_pre}) wide = wide && aligned_to(q, 16);
    const int blocks = bwd_blocks(*desc);
    cudaStream_t st = (cudaStream_t)stream;
    if (by_type<false>(*desc, p, wide, blocks, st) != cudaSuccess) return GSPN_ERR_CUDA;
    const int n = p.slots * p.C;
    if (n > 0) k_norm_sum<<<(n + 31) / 32, dim3(32, 8), 0, st>>>(p.part, blocks, n, p.C, to);
    return last_status();
}

}  // extern "C"
