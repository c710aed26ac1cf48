// k_ssm.cu -- selective state space scan over token sequences: prompts, gradients, single tokens.
//
//   h_t[c][n] = exp(d_t[c] A[c][n]) h_{t-1}[c][n] + d_t[c] x_t[c] B_t[g][n]
//   y_t[c]    = (sum_n C_t[g][n] h_t[c][n] + D[c] x_t[c]) silu(z_t[c]),   d = softplus(dt + bias)
//
// The recurrence is elementwise in (c, n), so it is no matrix product; what bounds it is one
// exponential for each (t, c, n), which the special-function unit makes at 16 a cycle and SM.
//
// Layout of a block: 32 channels of one sequence (64 bytes of a bf16 row: whole sectors) and
// NL = ceil(N / 4) rounded up to 2, 4, 8 or 16 lanes for each channel, four states in registers per
// lane. Tokens come in tiles of 32: each thread loads its part of the next tile into registers
// while the present one is scanned from shared memory, where the steps d and d x are formed once
// per (t, c). Sums over n stay in the NL lanes of a channel: four tokens at a time are reduced and
// scattered, so that each lane ends with one token's sum.
//
// Parallel over channels and sequences alone, a block walks its whole sequence. Where that leaves
// most of the chip idle, every sequence is cut into K equal pieces: a first pass finds each piece's
// own state from zero and its sum of steps (the decay over the piece is exp(A sum d)), and the main
// pass joins the pieces before its own. That makes every exponential twice.
#include "seq_common.cuh"

namespace gspn {
namespace seq {
namespace {

constexpr int kCh = 32;      // channels of a block
constexpr int kTile = 32;    // tokens staged at once
constexpr int kSub = 16;     // tokens between saved states
constexpr int kYS = 40;      // row stride of the per-token sums: four rows of eight channels miss each other's banks
constexpr int kMaxN = 64;

struct SsmArgs {
    int B, L, C, G, N, S;    // S: sequences (packed or rows)
    int Np;                  // N rounded up to 4
    int K;                   // pieces of a sequence
    int nb;                  // channel blocks of a group
    int softplus;
    bool wide;               // x, dt, z, y (and dy and the gradients) have 16-byte aligned vectors
    const void *x, *dt, *z, *Bm, *Cm;
    long long x_row, x_tok, dt_row, dt_tok, z_row, z_tok, b_row, b_tok, c_row, c_tok;
    const float *A, *D, *bias, *h0;
    const int* cu;
    void* y;
    float *h, *hsave;
    float *loc, *sdt;        // pieces: states (slot 0: the start) and sums of steps
    // backward
    const void* dy;
    const float* dh;
    void *dx, *ddt, *dz;
    float *dA_part, *dch_part, *dbc_part, *dh0;
};

// softplus(v) = max(v, 0) + log(1 + e), e = exp(-|v|), to a few 2^-24 relative: the exponential's
// argument keeps its rounding error, and log(1 + e) = 2 atanh(s) with s = e / (2 + e) <= 1/3, where
// atanh(s) / s is a polynomial of degree 4 in s^2 (least largest error on [0, 1/9]: 4e-9). A logarithm
// of 1 + e would lose the small steps.
__device__ __forceinline__ float softplus_of(float v) {
    const float w = -fminf(fabsf(v), 88.f);
    const float t = w * kLog2e;
    const float lo = fmaf(w, kLog2e, -t);
    float e = ex2(t);
    e = fmaf(e, lo * kLn2, e);
    const float s = e * rcp(2.f + e);
    const float q = s * s;
    float r = fmaf(q, 0.14089168f, 0.13980301f);
    r = fmaf(r, q, 0.20012455f);
    r = fmaf(r, q, 0.33333157f);
    r = fmaf(r, q, 1.f);
    const float out = fmaf(s + s, r, fmaxf(v, 0.f));
    return v != v ? v : out;
}

// Tokens of a piece: equal pieces, whole runs of kSub tokens so that saved states fall on borders.
__device__ __forceinline__ int piece_len(int len, int K) {
    return K == 1 ? len : ((len + K - 1) / K + kSub - 1) / kSub * kSub;
}
// First saved-state slot of a sequence: rows have ceil(L / kSub) slots each; packed sequences start
// at first / kSub + q, which never overlaps (a sequence of n tokens has at most n / kSub + 1).
__device__ __forceinline__ long long save_slot(const SsmArgs& p, const Span& sp, int q) {
    return p.cu ? (long long)(sp.first / kSub + q) : (long long)q * ((p.L + kSub - 1) / kSub);
}

// Where a block stands.
struct Place {
    int s, k, cb, g, c0, nc, lo, hi, last;   // sequence, piece, channel block; tokens [lo, hi) of the sequence
    Span sp;
};
__device__ __forceinline__ Place place_of(const SsmArgs& p, int pieces, int first_piece) {
    Place q;
    const int cblocks = p.nb * p.G;
    q.cb = blockIdx.x % cblocks;
    const int sk = blockIdx.x / cblocks;
    q.k = sk % pieces + first_piece;
    q.s = sk / pieces;
    q.g = q.cb / p.nb;
    const int Cg = p.C / p.G;
    q.c0 = q.g * Cg + (q.cb % p.nb) * kCh;
    q.nc = min(kCh, (q.g + 1) * Cg - q.c0);
    q.sp = span_of(p.cu, q.s, p.L);
    const int cl = piece_len(q.sp.len, p.K);
    q.lo = (int)min((long long)q.k * cl, (long long)q.sp.len);
    q.hi = min(q.lo + cl, q.sp.len);
    q.last = q.sp.len > 0 ? (q.sp.len - 1) / cl : 0;
    return q;
}

// Vectors of a tile of one input held by a thread.
template <typename T, int NL> struct Part {
    static constexpr int V = Vec<T>::V, VR = kCh / V, vecs = kTile * VR, threads = 32 * NL;
    static constexpr int NV = (vecs + threads - 1) / threads;
};

template <typename T, int NL>
__device__ __forceinline__ void ld_part(uint4 (&r)[Part<T, NL>::NV], const void* base, long long row, long long tok,
                                        const Place& q, int t0, bool wide) {
    using P = Part<T, NL>;
#pragma unroll
    for (int i = 0; i < P::NV; ++i) {
        const int v = i * P::threads + threadIdx.x;
        const int t = t0 + v / P::VR, c = v % P::VR * P::V;
        r[i] = make_uint4(0, 0, 0, 0);
        if (v < P::vecs && t < q.hi)
            r[i] = ld_raw<T>((const T*)base + q.sp.row * row + (q.sp.first + t) * tok + q.c0 + c, q.nc - c, wide);
    }
}

// The same for the kFeed threads that feed a forward block.
constexpr int kFeed = 128;
template <typename T> struct Feed {
    static constexpr int V = Vec<T>::V, VR = kCh / V, NV = kTile * VR / kFeed;
};
template <typename T>
__device__ __forceinline__ void ld_feed(uint4 (&r)[Feed<T>::NV], const void* base, long long row, long long tok,
                                        const Place& q, int t0, int tid, bool wide) {
    using P = Feed<T>;
#pragma unroll
    for (int i = 0; i < P::NV; ++i) {
        const int v = i * kFeed + tid;
        const int t = t0 + v / P::VR, c = v % P::VR * P::V;
        r[i] = make_uint4(0, 0, 0, 0);
        if (t < q.hi) r[i] = ld_raw<T>((const T*)base + q.sp.row * row + (q.sp.first + t) * tok + q.c0 + c, q.nc - c, wide);
    }
}

// A thread's elements of the tile's B (or C), as stored: conversions would wait for the loads here.
// Element e of the tile is token e / (4 NL), state e % (4 NL); `n` threads share it.
template <typename T, int NL, int E>
__device__ __forceinline__ void ld_states(T (&r)[E], const void* base, long long row, long long tok, const Place& q,
                                          int t0, int tid, int N) {
    constexpr int threads = kTile * 4 * NL / E;
#pragma unroll
    for (int i = 0; i < E; ++i) {
        const int e = i * threads + tid;
        const int t = t0 + e / (4 * NL), n = e % (4 * NL);
        r[i] = T(0.f);
        if (t < q.hi && n < N)
            r[i] = ((const T*)base)[q.sp.row * row + (q.sp.first + t) * tok + (long long)q.g * N + n];
    }
}

// Sums over the NL lanes of a channel for four tokens at once. NL >= 4: returns token (nl & 3)'s sum
// in r[0]; NL = 2: tokens 2 (nl & 1) and the next in r[0], r[1].
template <int NL>
__device__ __forceinline__ void reduce_tokens(const float (&v)[4], int nl, float (&r)[2]) {
    constexpr unsigned all = 0xffffffffu;
    if constexpr (NL == 2) {
        const bool up = nl & 1;
        r[0] = (up ? v[2] : v[0]) + __shfl_xor_sync(all, up ? v[0] : v[2], 1);
        r[1] = (up ? v[3] : v[1]) + __shfl_xor_sync(all, up ? v[1] : v[3], 1);
    } else {
        const bool hi = nl & 2, up = nl & 1;
        const float a = (hi ? v[2] : v[0]) + __shfl_xor_sync(all, hi ? v[0] : v[2], 2);
        const float b = (hi ? v[3] : v[1]) + __shfl_xor_sync(all, hi ? v[1] : v[3], 2);
        r[0] = (up ? b : a) + __shfl_xor_sync(all, up ? a : b, 1);
        if constexpr (NL >= 8) r[0] += __shfl_xor_sync(all, r[0], 4);
        if constexpr (NL >= 16) r[0] += __shfl_xor_sync(all, r[0], 8);
    }
}
template <int NL>
__device__ __forceinline__ void put_tokens(float* row0, int c, int nl, const float (&r)[2]) {
    if constexpr (NL == 2) {
        row0[(2 * (nl & 1)) * kYS + c] = r[0];
        row0[(2 * (nl & 1) + 1) * kYS + c] = r[1];
    } else {
        if (nl < 4) row0[nl * kYS + c] = r[0];
    }
}

// ------------------------------------------------------------------------------------- forward
// The block's first NL warps scan; four more feed them: they load the tokens, form d and d x, and turn
// the sums over n of the tile before into y. The two work on neighbouring tiles, with one barrier a
// tile, so the long latencies of the one side hide behind the other's arithmetic.
// A token's shares of the sums over n, NL for each channel, with four floats between the vectors of
// channels that one feeding thread adds up: its neighbours then start on other banks.
template <typename T, int NL> struct YRow {
    static constexpr int vec = Vec<T>::V * NL + 4, len = kCh / Vec<T>::V * vec;
    static __device__ __forceinline__ int at(int c, int nl) { return c / Vec<T>::V * vec + c % Vec<T>::V * NL + nl; }
    // the sum of channel c's shares; row is 16-byte aligned
    static __device__ __forceinline__ float sum(const float* row, int c) {
        const float* s = row + at(c, 0);
        if constexpr (NL == 2) {
            const float2 v = *(const float2*)s;
            return v.x + v.y;
        } else {
            float w = 0.f;
#pragma unroll
            for (int k = 0; k < NL; k += 4) {
                const float4 v = *(const float4*)(s + k);
                w += (v.x + v.y) + (v.z + v.w);
            }
            return w;
        }
    }
};

// Shared memory moves 128 bytes a cycle, and 16-byte loads of a whole warp take four cycles even where
// lanes read the same words, so what the scan loads for each token is kept small: d and d x as one
// pair, B and C of bf16 inputs as stored. Rows of d have 16 bytes between the vectors of channels
// that one feeding thread writes, which spreads its neighbours over the banks.
template <typename T> struct DRow {
    static constexpr int vec = Vec<T>::V + 2, len = kCh / Vec<T>::V * vec;     // in pairs
    static __device__ __forceinline__ int at(int c) { return c / Vec<T>::V * vec + c % Vec<T>::V; }
};
// B[4], C[4] of a lane side by side.
template <typename T> struct BC4 {
    T v[8];
};
__device__ __forceinline__ void get_b(const BC4<float>& s, float (&b)[4]) {
    const float4 q = *(const float4*)s.v;
    b[0] = q.x; b[1] = q.y; b[2] = q.z; b[3] = q.w;
}
__device__ __forceinline__ void get_bc(const BC4<float>& s, float (&b)[4], float (&c)[4]) {
    get_b(s, b);
    const float4 q = *(const float4*)(s.v + 4);
    c[0] = q.x; c[1] = q.y; c[2] = q.z; c[3] = q.w;
}
__device__ __forceinline__ void get_b(const BC4<__nv_bfloat16>& s, float (&b)[4]) {
    const uint2 q = *(const uint2*)s.v;
    b[0] = __uint_as_float(q.x << 16); b[1] = __uint_as_float(q.x & 0xffff0000u);
    b[2] = __uint_as_float(q.y << 16); b[3] = __uint_as_float(q.y & 0xffff0000u);
}
__device__ __forceinline__ void get_bc(const BC4<__nv_bfloat16>& s, float (&b)[4], float (&c)[4]) {
    float v[8];
    unpack_raw<__nv_bfloat16>(*(const uint4*)s.v, v);
#pragma unroll
    for (int j = 0; j < 4; ++j) { b[j] = v[j]; c[j] = v[4 + j]; }
}

template <typename T, int NL, bool LOCAL> struct FwdSmem {
    float2 dd[2][kTile][DRow<T>::len];                 // d, d x
    BC4<T> bc[2][kTile][NL];
    float y[LOCAL ? 1 : 2][LOCAL ? 1 : kTile][YRow<T, NL>::len];   // each lane's share of the sums over n
};

// LOCAL: the first pass over pieces (from a zero state, the last piece left out).
template <typename T, int NL, bool LOCAL>
__global__ void __launch_bounds__(32 * NL + kFeed) k_ssm_fwd(const SsmArgs p) {
    extern __shared__ __align__(16) unsigned char smem_raw[];
    FwdSmem<T, NL, LOCAL>& sm = *(FwdSmem<T, NL, LOCAL>*)smem_raw;

    const Place q = place_of(p, LOCAL ? p.K - 1 : p.K, 0);
    if (!LOCAL && q.k > 0 && q.lo >= q.hi) return;
    const int tiles = (q.hi - q.lo + kTile - 1) / kTile;

    if (threadIdx.x >= 32 * NL) {
        // ------------------------------------------------------------ feed
        using P = Feed<T>;
        constexpr int V = P::V, NS = NL;                          // elements of B (and of C) for each thread
        const int tid = threadIdx.x - 32 * NL;
        const int vc = tid % P::VR * V;
        float bias[V], Dv[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            bias[i] = (p.bias && vc + i < q.nc) ? p.bias[q.c0 + vc + i] : 0.f;
            Dv[i] = (!LOCAL && p.D && vc + i < q.nc) ? p.D[q.c0 + vc + i] : 0.f;
        }
        // x and z of the tile to be loaded, the one staged and the one before it
        uint4 rx[P::NV], rd[P::NV], rz[P::NV], x1[P::NV], z1[P::NV], x0[P::NV], z0[P::NV];
        T rB[NS], rC[NS];
        auto load = [&](int i) {
            const int t0 = q.lo + i * kTile;
            ld_feed<T>(rx, p.x, p.x_row, p.x_tok, q, t0, tid, p.wide);
            ld_feed<T>(rd, p.dt, p.dt_row, p.dt_tok, q, t0, tid, p.wide);
            ld_states<T, NL>(rB, p.Bm, p.b_row, p.b_tok, q, t0, tid, p.N);
            if constexpr (!LOCAL) {
                if (p.z) ld_feed<T>(rz, p.z, p.z_row, p.z_tok, q, t0, tid, p.wide);
                ld_states<T, NL>(rC, p.Cm, p.c_row, p.c_tok, q, t0, tid, p.N);
            }
        };
        auto stage = [&](int i) {
            const int t0 = q.lo + i * kTile, buf = i & 1;
#pragma unroll
            for (int k = 0; k < P::NV; ++k) {
                const int t = (k * kFeed + tid) / P::VR;
                x0[k] = x1[k];
                z0[k] = z1[k];
                x1[k] = rx[k];
                z1[k] = rz[k];
                float xv[V], dv[V];
                float2 dd[V];
                unpack_raw<T>(rx[k], xv);
                unpack_raw<T>(rd[k], dv);
                const bool ok = t0 + t < q.hi;
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    float d = dv[j] + bias[j];
                    if (p.softplus) d = softplus_of(d);
                    // a token behind the end makes no step, and the state stays; its x was read as zero, and so
                    // were those of channels behind the last, whose states are zero
                    dd[j] = make_float2(ok ? d : 0.f, ok ? d * xv[j] : 0.f);
                }
                float4* to = (float4*)&sm.dd[buf][t][DRow<T>::at(vc)];
#pragma unroll
                for (int j = 0; j < V; j += 2) to[j / 2] = make_float4(dd[j].x, dd[j].y, dd[j + 1].x, dd[j + 1].y);
            }
#pragma unroll
            for (int k = 0; k < NS; ++k) {
                const int e = k * kFeed + tid;
                T* to = (&sm.bc[buf][0][0])[e / 4].v + e % 4;
                to[0] = rB[k];
                if constexpr (!LOCAL) to[4] = rC[k];
            }
        };
        auto finish = [&](int i) {                                // i is the tile before the one staged last
            const int t0 = q.lo + i * kTile, buf = i & 1;
#pragma unroll
            for (int k = 0; k < P::NV; ++k) {
                const int t = (k * kFeed + tid) / P::VR;
                if (t0 + t < q.hi) {
                    float xv[V], zv[V], out[V];
                    unpack_raw<T>(x0[k], xv);
                    unpack_raw<T>(z0[k], zv);
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        out[j] = fmaf(Dv[j], xv[j], YRow<T, NL>::sum(sm.y[buf][t], vc + j));
                        if (p.z) out[j] *= silu(zv[j]);
                    }
                    st_vec<T>((T*)p.y + ((long long)q.sp.row * p.L + q.sp.first + t0 + t) * p.C + q.c0 + vc, out,
                              q.nc - vc, p.wide);
                }
            }
        };
        if (tiles > 0) {
            load(0);
            stage(0);
            if (tiles > 1) load(1);
        }
        __syncthreads();
        for (int i = 0; i < tiles; ++i) {
            if (i + 1 < tiles) {
                stage(i + 1);
                if (i + 2 < tiles) load(i + 2);
            } else {
#pragma unroll
                for (int k = 0; k < P::NV; ++k) { x0[k] = x1[k]; z0[k] = z1[k]; }
            }
            __syncthreads();
            // the sums of tile i are complete; its buffer is written again behind the next barrier only
            if constexpr (!LOCAL) finish(i);
        }
        return;
    }

    // ---------------------------------------------------------------- scan
    const int lane = threadIdx.x & 31, nl = lane % NL;
    const int cl = (threadIdx.x >> 5) * (32 / NL) + lane / NL;    // channel within the block
    const bool cok = cl < q.nc;
    const long long c = q.c0 + cl;
    const int n0 = 4 * nl;

    float A2[4], h[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const bool ok = cok && n0 + j < p.N;
        A2[j] = ok ? p.A[c * p.N + n0 + j] * kLog2e : 0.f;
        h[j] = (ok && p.h0 && (LOCAL || p.K == 1)) ? p.h0[((long long)q.s * p.C + c) * p.N + n0 + j] : 0.f;
    }
    const bool keeps = cok && n0 < p.Np;
    const long long piece0 = (long long)q.s * (p.K + 1);          // slots of this sequence's pieces
    if constexpr (LOCAL) {
        if (q.k == 0 && keeps) *(float4*)(p.loc + (piece0 * p.C + c) * p.Np + n0) = make_float4(h[0], h[1], h[2], h[3]);
#pragma unroll
        for (int j = 0; j < 4; ++j) h[j] = 0.f;
    } else if (p.K > 1) {
        if (keeps) {
            const float* l = p.loc + (piece0 * p.C + c) * p.Np + n0;
            const long long step = (long long)p.C * p.Np;
            const float4 f = *(const float4*)l;
            h[0] = f.x; h[1] = f.y; h[2] = f.z; h[3] = f.w;
            for (int k = 0; k < q.k; ++k) {
                const float sd = p.sdt[((long long)q.s * p.K + k) * p.C + c];
                const float4 m = *(const float4*)(l + (k + 1) * step);
                h[0] = fmaf(ex2(sd * A2[0]), h[0], m.x);
                h[1] = fmaf(ex2(sd * A2[1]), h[1], m.y);
                h[2] = fmaf(ex2(sd * A2[2]), h[2], m.z);
                h[3] = fmaf(ex2(sd * A2[3]), h[3], m.w);
            }
        }
    }
    f2 h01 = pack(h[0], h[1]), h23 = pack(h[2], h[3]);
    const long long save0 = LOCAL ? 0 : save_slot(p, q.sp, q.s);
    float sum_d = 0.f;
    __syncthreads();
    for (int i = 0; i < tiles; ++i) {
        const int t0 = q.lo + i * kTile, buf = i & 1;
        // Operands of four tokens are fetched while the four before are worked on; the stores below would
        // otherwise hold back the loads behind them.
        float2 dd[2][4];
        BC4<T> bc[2][4];
        auto fetch = [&](int t, int w) {
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                dd[w][u] = sm.dd[buf][t + u][DRow<T>::at(cl)];
                bc[w][u] = sm.bc[buf][t + u][nl];
            }
        };
        fetch(0, 0);
#pragma unroll
        for (int t = 0; t < kTile; t += 4) {
            const int w = t / 4 & 1;
            if (t + 4 < kTile) fetch(t + 4, w ^ 1);
            if constexpr (!LOCAL) {
                if (t % kSub == 0 && p.hsave && keeps && t0 + t < q.hi)
                    *(ulonglong2*)(p.hsave + ((save0 + (t0 + t) / kSub) * p.C + c) * p.Np + n0) = make_ulonglong2(h01, h23);
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const float d = dd[w][u].x, dx = dd[w][u].y;
                float b[4], cc[4];
                if constexpr (LOCAL) get_b(bc[w][u], b);
                else get_bc(bc[w][u], b, cc);
                const f2 a01 = pack(ex2(d * A2[0]), ex2(d * A2[1])), a23 = pack(ex2(d * A2[2]), ex2(d * A2[3]));
                h01 = fma2(a01, h01, pack(dx * b[0], dx * b[1]));
                h23 = fma2(a23, h23, pack(dx * b[2], dx * b[3]));
                if constexpr (LOCAL) {
                    sum_d += d;
                } else {
                    const float2 s = unpack(fma2(h01, pack(cc[0], cc[1]), mul2(h23, pack(cc[2], cc[3]))));
                    sm.y[buf][t + u][YRow<T, NL>::at(cl, nl)] = s.x + s.y;
                }
            }
        }
        __syncthreads();
    }
    if constexpr (LOCAL) {
        if (keeps) *(ulonglong2*)(p.loc + ((piece0 + q.k + 1) * p.C + c) * p.Np + n0) = make_ulonglong2(h01, h23);
        if (cok && nl == 0) p.sdt[((long long)q.s * p.K + q.k) * p.C + c] = sum_d;
    } else if (p.h && q.k == q.last) {
        const float2 u = unpack(h01), v = unpack(h23);
        const float f[4] = {u.x, u.y, v.x, v.y};
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (cok && n0 + j < p.N) p.h[((long long)q.s * p.C + c) * p.N + n0 + j] = f[j];
    }
}

// ------------------------------------------------------------------------------------ backward
// With g_t = dL/dh_t and r_t = dy_t silu(z_t):
//   g_t = C_t r_t + a_{t+1} g_{t+1}
//   dC_t = sum_c r_t h_t,  dB_t = sum_c g_t d_t x_t,  d(d x)_t = sum_n g_t B_t,
//   e_t = a_t g_t h_{t-1},  dA = sum_t e_t d_t,  dd_t = sum_n e_t A + x_t d(d x)_t
// The forward saved the state before every 16th token. From it 16 tokens are walked forward with
// every a_t and h_t kept in registers, then walked back, so each exponential is made once.
//
// Sums over the channels of a block: a lane's four states are held in an order that depends on the
// lane's channel (slot j holds state j xor the channel's low bits), so halving the four slots over
// the channel lanes needs no selects: what one lane gives away is what its partner keeps.
constexpr int perm_copies(int NL) { return 32 / NL < 4 ? 32 / NL : 4; }

__device__ __forceinline__ void permute4(float (&v)[4], int pm) {
    if (pm & 1) {
        const float a = v[0], b = v[2];
        v[0] = v[1]; v[1] = a; v[2] = v[3]; v[3] = b;
    }
    if (pm & 2) {
        const float a = v[0], b = v[1];
        v[0] = v[2]; v[2] = a; v[1] = v[3]; v[3] = b;
    }
}

template <typename T, int NL> struct BwdSmem {
    using P = Part<T, NL>;
    static constexpr int PC = perm_copies(NL);
    float2 dd[kTile][kCh];                 // d, d x
    float r[kTile][kCh];                   // dy silu(z)
    float B[kTile][PC][4 * NL], C[kTile][PC][4 * NL];
    float o[3][kTile][kYS];                // sums over n: C h, g B, e A
    float bc[NL][kSub][8 * NL];            // sums over a warp's channels: dB, dC
    uint4 raw[4][P::vecs];                 // x, dt, z, dy of the tile
    float acc[2][P::vecs < P::threads ? P::vecs : P::threads][P::V + 1];   // dD, d dt_bias of the thread's vector
};

// LOCAL: the first pass over pieces: what each piece passes back from a zero gradient behind it (all
// pieces but the first) and its sum of steps.
template <typename T, int NL>
__global__ void __launch_bounds__(32 * NL) k_ssm_bwd_local(const SsmArgs p) {
    using P = Part<T, NL>;
    constexpr int V = P::V;
    __shared__ __align__(16) float2 sdr[kTile][kCh];              // d, r
    __shared__ __align__(16) float sC[kTile][4 * NL];
    const Place q = place_of(p, p.K - 1, 1);
    const int lane = threadIdx.x & 31, nl = lane % NL;
    const int cl = (threadIdx.x >> 5) * (32 / NL) + lane / NL;
    const bool cok = cl < q.nc;
    const long long c = q.c0 + cl;
    const int n0 = 4 * nl;
    float A2[4], ag[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < 4; ++j) A2[j] = cok && n0 + j < p.N ? p.A[c * p.N + n0 + j] * kLog2e : 0.f;
    const int vc = threadIdx.x % P::VR * V;
    float bias[V];
#pragma unroll
    for (int i = 0; i < V; ++i) bias[i] = (p.bias && vc + i < q.nc) ? p.bias[q.c0 + vc + i] : 0.f;
    uint4 rd[P::NV], rz[P::NV], rg[P::NV];
    T rC[4];
    auto load = [&](int t0) {
        ld_part<T, NL>(rd, p.dt, p.dt_row, p.dt_tok, q, t0, p.wide);
        ld_part<T, NL>(rg, p.dy, (long long)p.L * p.C, p.C, q, t0, p.wide);
        if (p.z) ld_part<T, NL>(rz, p.z, p.z_row, p.z_tok, q, t0, p.wide);
        ld_states<T, NL>(rC, p.Cm, p.c_row, p.c_tok, q, t0, threadIdx.x, p.N);
    };
    float sum_d = 0.f;
    int t0 = q.lo + (q.hi - q.lo + kTile - 1) / kTile * kTile - kTile;
    if (t0 >= q.lo) load(t0);
    for (; t0 >= q.lo; t0 -= kTile) {
#pragma unroll
        for (int i = 0; i < P::NV; ++i) {
            const int v = i * P::threads + threadIdx.x;
            if (v < P::vecs) {
                const int t = v / P::VR;
                float dv[V], zv[V], gv[V];
                unpack_raw<T>(rd[i], dv);
                unpack_raw<T>(rz[i], zv);
                unpack_raw<T>(rg[i], gv);
                const bool ok = t0 + t < q.hi;
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    float d = dv[j] + bias[j];
                    if (p.softplus) d = softplus_of(d);
                    d = ok && vc + j < q.nc ? d : 0.f;
                    const float r = p.z ? gv[j] * silu(zv[j]) : gv[j];
                    sdr[t][vc + j] = make_float2(d, ok ? r : 0.f);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) (&sC[0][0])[i * P::threads + threadIdx.x] = Io<T>::ld(&rC[i]);
        __syncthreads();
        if (t0 - kTile >= q.lo) load(t0 - kTile);
#pragma unroll 8
        for (int t = kTile - 1; t >= 0; --t) {
            const float2 dr = sdr[t][cl];
            const float4 c4 = *(const float4*)&sC[t][n0];
            sum_d += dr.x;
            ag[0] = ex2(dr.x * A2[0]) * fmaf(c4.x, dr.y, ag[0]);
            ag[1] = ex2(dr.x * A2[1]) * fmaf(c4.y, dr.y, ag[1]);
            ag[2] = ex2(dr.x * A2[2]) * fmaf(c4.z, dr.y, ag[2]);
            ag[3] = ex2(dr.x * A2[3]) * fmaf(c4.w, dr.y, ag[3]);
        }
        __syncthreads();
    }
    const long long slot = (long long)q.s * p.K + q.k;
    if (cok && n0 < p.Np) *(float4*)(p.loc + (slot * p.C + c) * p.Np + n0) = make_float4(ag[0], ag[1], ag[2], ag[3]);
    if (cok && nl == 0) p.sdt[slot * p.C + c] = sum_d;
}

template <typename T, int NL>
__global__ void __launch_bounds__(32 * NL) k_ssm_bwd(const SsmArgs p) {
    using P = Part<T, NL>;
    constexpr int V = P::V, PC = perm_copies(NL);
    constexpr unsigned all = 0xffffffffu;
    extern __shared__ __align__(16) unsigned char smem_raw[];
    BwdSmem<T, NL>& sm = *(BwdSmem<T, NL>*)smem_raw;

    const Place q = place_of(p, p.K, 0);
    const int lane = threadIdx.x & 31, nl = lane % NL, warp = threadIdx.x >> 5;
    const int ql = lane / NL, pm = ql & (PC - 1);                 // channel lane, order of the states
    const int cl = warp * (32 / NL) + ql;
    const bool cok = cl < q.nc;
    const long long c = q.c0 + cl;
    const int n0 = 4 * nl;
    const bool keeps = cok && n0 < p.Np;

    float A2[4], ag[4], dA[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const bool ok = cok && n0 + j < p.N;
        A2[j] = ok ? p.A[c * p.N + n0 + j] * kLog2e : 0.f;
        ag[j] = ok && p.dh ? p.dh[((long long)q.s * p.C + c) * p.N + n0 + j] : 0.f;
    }
    if (keeps)
        for (int k = p.K - 1; k > q.k; --k) {                     // join the pieces behind this one
            const long long slot = (long long)q.s * p.K + k;
            const float sd = p.sdt[slot * p.C + c];
            const float4 m = *(const float4*)(p.loc + (slot * p.C + c) * p.Np + n0);
            ag[0] = fmaf(ex2(sd * A2[0]), ag[0], m.x);
            ag[1] = fmaf(ex2(sd * A2[1]), ag[1], m.y);
            ag[2] = fmaf(ex2(sd * A2[2]), ag[2], m.z);
            ag[3] = fmaf(ex2(sd * A2[3]), ag[3], m.w);
        }
    permute4(A2, pm);
    permute4(ag, pm);

    const int vc = threadIdx.x % P::VR * V;
    const bool stages = threadIdx.x < P::vecs;
    if (stages) {
#pragma unroll
        for (int j = 0; j < V; ++j) sm.acc[0][threadIdx.x][j] = sm.acc[1][threadIdx.x][j] = 0.f;
    }
    const long long save0 = save_slot(p, q.sp, q.s);
    const int cbk = q.cb % p.nb;

    uint4 rx[P::NV], rd[P::NV], rz[P::NV], rg[P::NV];
    T rB[4], rC[4];
    float4 rh[2];
    auto load = [&](int t0) {
        ld_part<T, NL>(rx, p.x, p.x_row, p.x_tok, q, t0, p.wide);
        ld_part<T, NL>(rd, p.dt, p.dt_row, p.dt_tok, q, t0, p.wide);
        ld_part<T, NL>(rg, p.dy, (long long)p.L * p.C, p.C, q, t0, p.wide);
        if (p.z) ld_part<T, NL>(rz, p.z, p.z_row, p.z_tok, q, t0, p.wide);
        ld_states<T, NL>(rB, p.Bm, p.b_row, p.b_tok, q, t0, threadIdx.x, p.N);
        ld_states<T, NL>(rC, p.Cm, p.c_row, p.c_tok, q, t0, threadIdx.x, p.N);
#pragma unroll
        for (int s = 0; s < 2; ++s)
            rh[s] = keeps && t0 + s * kSub < q.hi
                        ? *(const float4*)(p.hsave + ((save0 + t0 / kSub + s) * p.C + c) * p.Np + n0)
                        : make_float4(0.f, 0.f, 0.f, 0.f);
    };
    auto bias_of = [&](int j) { return p.bias && vc + j < q.nc ? __ldg(p.bias + q.c0 + vc + j) : 0.f; };

    int t0 = q.lo + (q.hi - q.lo + kTile - 1) / kTile * kTile - kTile;
    if (t0 >= q.lo) load(t0);
    for (; t0 >= q.lo; t0 -= kTile) {
#pragma unroll
        for (int i = 0; i < P::NV; ++i) {
            const int v = i * P::threads + threadIdx.x;
            if (v < P::vecs) {
                const int t = v / P::VR;
                float xv[V], dv[V], zv[V], gv[V];
                unpack_raw<T>(rx[i], xv);
                unpack_raw<T>(rd[i], dv);
                unpack_raw<T>(rz[i], zv);
                unpack_raw<T>(rg[i], gv);
                sm.raw[0][v] = rx[i];
                sm.raw[1][v] = rd[i];
                sm.raw[2][v] = rz[i];
                sm.raw[3][v] = rg[i];
                const bool ok = t0 + t < q.hi;
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    float d = dv[j] + bias_of(j);
                    if (p.softplus) d = softplus_of(d);
                    d = ok && vc + j < q.nc ? d : 0.f;
                    sm.dd[t][vc + j] = make_float2(d, ok ? d * xv[j] : 0.f);
                    const float r = p.z ? gv[j] * silu(zv[j]) : gv[j];
                    sm.r[t][vc + j] = ok ? r : 0.f;
                }
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int e = i * P::threads + threadIdx.x;
            const int t = e / (4 * NL), n = e % (4 * NL);
#pragma unroll
            for (int m = 0; m < PC; ++m) {
                sm.B[t][m][n ^ m] = Io<T>::ld(&rB[i]);
                sm.C[t][m][n ^ m] = Io<T>::ld(&rC[i]);
            }
        }
        const float4 hin[2] = {rh[0], rh[1]};
        __syncthreads();
        if (t0 - kTile >= q.lo) load(t0 - kTile);

#pragma unroll 1
        for (int s = 1; s >= 0; --s) {
            const int ts = s * kSub;
            const float4 hf = s ? hin[1] : hin[0];
            float hi4[4] = {hf.x, hf.y, hf.z, hf.w};
            permute4(hi4, pm);
            float a[kSub][4], h[kSub][4];
#pragma unroll
            for (int i = 0; i < kSub; ++i) {
                const float2 dd = sm.dd[ts + i][cl];
                const float4 b = *(const float4*)&sm.B[ts + i][pm][n0];
                const float bb[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    a[i][j] = ex2(dd.x * A2[j]);
                    h[i][j] = fmaf(a[i][j], i ? h[i - 1][j] : hi4[j], dd.y * bb[j]);
                }
            }
            float dAs[4] = {0.f, 0.f, 0.f, 0.f};                  // sums of 16 tokens join the long sum as one
#pragma unroll
            for (int i4 = kSub - 4; i4 >= 0; i4 -= 4) {
                float yv[4], gv[4], ev[4];
#pragma unroll
                for (int u = 3; u >= 0; --u) {
                    const int i = i4 + u;
                    const float2 dd = sm.dd[ts + i][cl];
                    const float r = sm.r[ts + i][cl];
                    const float4 b = *(const float4*)&sm.B[ts + i][pm][n0];
                    const float4 c4 = *(const float4*)&sm.C[ts + i][pm][n0];
                    const float bb[4] = {b.x, b.y, b.z, b.w}, cc[4] = {c4.x, c4.y, c4.z, c4.w};
                    float vB[4], vC[4];
                    yv[u] = gv[u] = ev[u] = 0.f;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float g = fmaf(cc[j], r, ag[j]);
                        vC[j] = r * h[i][j];
                        vB[j] = g * dd.y;
                        yv[u] = fmaf(cc[j], h[i][j], yv[u]);
                        gv[u] = fmaf(g, bb[j], gv[u]);
                        ag[j] = a[i][j] * g;
                        const float e = ag[j] * (i ? h[i - 1][j] : hi4[j]);
                        dAs[j] = fmaf(e, dd.x, dAs[j]);
                        ev[u] = fmaf(e, A2[j], ev[u]);
                    }
                    // sums over the warp's channels
                    vB[0] += __shfl_xor_sync(all, vB[1], NL);
                    vB[2] += __shfl_xor_sync(all, vB[3], NL);
                    vC[0] += __shfl_xor_sync(all, vC[1], NL);
                    vC[2] += __shfl_xor_sync(all, vC[3], NL);
                    float* out = sm.bc[warp][i];
                    if constexpr (NL == 16) {
                        out[n0 + pm] = vB[0];
                        out[n0 + (2 ^ pm)] = vB[2];
                        out[4 * NL + n0 + pm] = vC[0];
                        out[4 * NL + n0 + (2 ^ pm)] = vC[2];
                    } else {
                        vB[0] += __shfl_xor_sync(all, vB[2], 2 * NL);
                        vC[0] += __shfl_xor_sync(all, vC[2], 2 * NL);
                        if constexpr (NL == 8) {
                            out[n0 + pm] = vB[0];
                            out[4 * NL + n0 + pm] = vC[0];
                        } else {
                            const bool up = ql & 4;
                            float w = (up ? vC[0] : vB[0]) + __shfl_xor_sync(all, up ? vB[0] : vC[0], 4 * NL);
                            if constexpr (NL == 2) w += __shfl_xor_sync(all, w, 8 * NL);
                            if (NL != 2 || ql < 8) out[(up ? 4 * NL : 0) + n0 + pm] = w;
                        }
                    }
                }
                float w[2];
                reduce_tokens<NL>(yv, nl, w);
                put_tokens<NL>(&sm.o[0][ts + i4][0], cl, nl, w);
                reduce_tokens<NL>(gv, nl, w);
                put_tokens<NL>(&sm.o[1][ts + i4][0], cl, nl, w);
                reduce_tokens<NL>(ev, nl, w);
                put_tokens<NL>(&sm.o[2][ts + i4][0], cl, nl, w);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) dA[j] += dAs[j];
            __syncthreads();
            // sums over the warps, to this block's part of dB and dC
            for (int e = threadIdx.x; e < kSub * 8 * NL; e += P::threads) {
                const int i = e / (8 * NL), v = e % (8 * NL);
                float w = 0.f;
#pragma unroll
                for (int k = 0; k < NL; ++k) w += sm.bc[k][i][v];
                const int t = t0 + ts + i;
                if (t < q.hi)
                    p.dbc_part[(((long long)cbk * p.B * p.L + (long long)q.sp.row * p.L + q.sp.first + t) * p.G + q.g) *
                                   (8 * NL) + v] = w;
            }
            if (s == 1) __syncthreads();
        }
        // per (t, c): the gradients of x, dt, z
#pragma unroll
        for (int i = 0; i < P::NV; ++i) {
            const int v = i * P::threads + threadIdx.x;
            const int t = v / P::VR;
            if (v < P::vecs && t0 + t < q.hi) {
                float xv[V], dv[V], zv[V], gv[V], ox[V], od[V], oz[V];
                unpack_raw<T>(sm.raw[0][v], xv);
                unpack_raw<T>(sm.raw[1][v], dv);
                unpack_raw<T>(sm.raw[2][v], zv);
                unpack_raw<T>(sm.raw[3][v], gv);
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const float Dj = p.D && vc + j < q.nc ? __ldg(p.D + q.c0 + vc + j) : 0.f;
                    const float r = sm.r[t][vc + j], d = sm.dd[t][vc + j].x;
                    const float gB = sm.o[1][t][vc + j], eA = sm.o[2][t][vc + j] * kLn2;
                    ox[j] = fmaf(gB, d, Dj * r);
                    float w = fmaf(gB, xv[j], eA);
                    if (p.softplus) w *= sigmoid(dv[j] + bias_of(j));
                    od[j] = w;
                    if (p.z) oz[j] = gv[j] * fmaf(Dj, xv[j], sm.o[0][t][vc + j]) * silu_slope(zv[j]);
                    sm.acc[0][threadIdx.x][j] = fmaf(r, xv[j], sm.acc[0][threadIdx.x][j]);
                    sm.acc[1][threadIdx.x][j] += w;
                }
                const long long at = ((long long)q.sp.row * p.L + q.sp.first + t0 + t) * p.C + q.c0 + vc;
                st_vec<T>((T*)p.dx + at, ox, q.nc - vc, p.wide);
                st_vec<T>((T*)p.ddt + at, od, q.nc - vc, p.wide);
                if (p.z) st_vec<T>((T*)p.dz + at, oz, q.nc - vc, p.wide);
            }
        }
        // the staging of the next tile overwrites what other threads still read here: r and dd are read by
        // their own writer only, o by the epilogue above, B and C in the walks behind a barrier each
        __syncthreads();
    }

    permute4(ag, pm);
    permute4(dA, pm);
    const long long slot = (long long)q.s * p.K + q.k;
    if (keeps) *(float4*)(p.dA_part + (slot * p.C + c) * p.Np + n0) = make_float4(dA[0], dA[1], dA[2], dA[3]);
    if (p.dh0 && q.k == 0) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (cok && n0 + j < p.N) p.dh0[((long long)q.s * p.C + c) * p.N + n0 + j] = ag[j];
    }
    __syncthreads();
    constexpr int TL = (P::vecs < P::threads ? P::vecs : P::threads) / P::VR;   // threads that share a vector
    if (threadIdx.x < 2 * kCh) {
        const int which = threadIdx.x / kCh, cc = threadIdx.x % kCh;
        float w = 0.f;
#pragma unroll
        for (int i = 0; i < TL; ++i) w += sm.acc[which][i * P::VR + cc / V][cc % V];
        if (cc < q.nc) p.dch_part[(slot * 2 + which) * p.C + q.c0 + cc] = w;
    }
}

// dB and dC: the channel blocks of a group in order. Thread = (token, group, B or C, state).
template <typename T>
__global__ void k_ssm_sum_bc(const float* part, const int* cu, int S, int B, int L, int G, int N, int nb, int w8,
                             T* dBm, T* dCm) {
    const long long per = (long long)B * L * G * w8;
    const long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= per) return;
    const int v = (int)(i % w8);
    const long long tg = i / w8;                                   // token * G + group
    if (cu) {
        const long long t = tg / G;
        if (t < min(max(cu[0], 0), L) || t >= min(max(cu[S], 0), L)) return;
    }
    const int n = v % (w8 / 2);
    if (n >= N) return;
    float w = 0.f;
    for (int k = 0; k < nb; ++k) w += part[k * per + i];
    Io<T>::st((v < w8 / 2 ? dBm : dCm) + tg * N + n, w);
}

// dA, dD, d dt_bias: the sequences' pieces in order.
__global__ void k_ssm_sum_ac(const float* dA_part, const float* dch_part, int slots, int C, int N, int Np, float* dA,
                             float* dD, float* dbias) {
    const long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x;
    const long long na = (long long)C * Np;
    if (i < na) {
        const int n = (int)(i % Np);
        float w = 0.f;
        for (int k = 0; k < slots; ++k) w += dA_part[k * na + i];
        if (n < N) dA[i / Np * N + n] = w;
    } else if (i < na + 2 * C) {
        const long long c = i - na;
        float w = 0.f;
        for (int k = 0; k < slots; ++k) w += dch_part[(long long)k * 2 * C + c];
        float* out = c < C ? dD : dbias;
        if (out) out[c % C] = w;
    }
}

// ----------------------------------------------------------------------------------- one token
// A block takes one row and as many channels as its threads hold four states of. Rows that name the
// slot of an earlier row leave their token to that row, which walks them in order.
template <typename T>
__global__ void k_ssm_step(const SsmArgs p, const int* idx, int slots, int NL) {
    const int b0 = blockIdx.y;
    const int slot = idx ? idx[b0] : b0;
    if (slot < 0 || slot >= slots) return;
    int more = 0;
    if (idx) {
        bool earlier = false, later = false;
        for (int b = threadIdx.x; b < p.B; b += blockDim.x) {
            const bool same = b != b0 && idx[b] == slot;
            earlier |= same && b < b0;
            later |= same && b > b0;
        }
        if (__syncthreads_or(earlier)) return;
        more = __syncthreads_or(later);
    }
    const int nl = threadIdx.x % NL, n0 = 4 * nl;
    const long long c = (long long)blockIdx.x * (blockDim.x / NL) + threadIdx.x / NL;
    const bool cok = c < p.C;
    const int g = cok ? (int)(c / (p.C / p.G)) : 0;
    float h[4], A2[4];
    float* hp = p.h + ((long long)slot * p.C + c) * p.N + n0;
    const bool vec = (p.N & 3) == 0 && p.wide;
    if (vec && cok && n0 < p.N) {
        const float4 f = *(const float4*)hp, a = *(const float4*)(p.A + c * p.N + n0);
        h[0] = f.x; h[1] = f.y; h[2] = f.z; h[3] = f.w;
        A2[0] = a.x * kLog2e; A2[1] = a.y * kLog2e; A2[2] = a.z * kLog2e; A2[3] = a.w * kLog2e;
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const bool ok = cok && n0 + j < p.N;
            h[j] = ok ? hp[j] : 0.f;
            A2[j] = ok ? p.A[c * p.N + n0 + j] * kLog2e : 0.f;
        }
    }
    for (int b = b0; b < (more ? p.B : b0 + 1); ++b) {
        if (b != b0 && idx[b] != slot) continue;
        float x = 0.f, d = 0.f, z = 0.f;
        if (cok) {
            x = Io<T>::ld((const T*)p.x + b * p.x_row + c);
            d = Io<T>::ld((const T*)p.dt + b * p.dt_row + c) + (p.bias ? p.bias[c] : 0.f);
            if (p.z) z = Io<T>::ld((const T*)p.z + b * p.z_row + c);
        }
        if (p.softplus) d = softplus_of(d);
        float y = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (cok && n0 + j < p.N) {
                const float bv = Io<T>::ld((const T*)p.Bm + b * p.b_row + (long long)g * p.N + n0 + j);
                const float cv = Io<T>::ld((const T*)p.Cm + b * p.c_row + (long long)g * p.N + n0 + j);
                h[j] = fmaf(ex2(d * A2[j]), h[j], d * x * bv);
                y = fmaf(h[j], cv, y);
            }
        }
        for (int o = NL / 2; o; o >>= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
        if (cok && nl == 0) {
            if (p.D) y = fmaf(p.D[c], x, y);
            if (p.z) y *= silu(z);
            Io<T>::st((T*)p.y + (long long)b * p.C + c, y);
        }
    }
    if (vec && cok && n0 < p.N) {
        *(float4*)hp = make_float4(h[0], h[1], h[2], h[3]);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (cok && n0 + j < p.N) hp[j] = h[j];
    }
}

// ---------------------------------------------------------------------------------------- host
int lanes_for(int N) { return N <= 8 ? 2 : N <= 16 ? 4 : N <= 32 ? 8 : 16; }

bool make_args(const gspn_ssm_desc* d, SsmArgs* p) {
    if (!d) return false;
    if (d->B < 1 || d->L < 0 || d->C < 1 || d->G < 1 || d->N < 1 || d->S < 0) return false;
    if (d->C % d->G != 0 || !dtype_ok(d->dtype)) return false;
    if (d->softplus != 0 && d->softplus != 1) return false;
    if (d->S > 0 && d->B != 1) return false;
    for (long long s : {d->x_row, d->x_tok, d->dt_row, d->dt_tok, d->z_row, d->z_tok, d->b_row, d->b_tok, d->c_row,
                        d->c_tok})
        if (s < 0) return false;
    *p = SsmArgs{};
    p->B = d->B; p->L = d->L; p->C = d->C; p->G = d->G; p->N = d->N;
    p->S = d->S > 0 ? d->S : d->B;
    p->Np = (d->N + 3) / 4 * 4;
    p->nb = (d->C / d->G + kCh - 1) / kCh;
    p->softplus = d->softplus;
    p->x_row = d->x_row; p->x_tok = d->x_tok; p->dt_row = d->dt_row; p->dt_tok = d->dt_tok;
    p->z_row = d->z_row; p->z_tok = d->z_tok; p->b_row = d->b_row; p->b_tok = d->b_tok;
    p->c_row = d->c_row; p->c_tok = d->c_tok;
    return true;
}
// Sizes that the launches' 32-bit block counts and token arithmetic hold.
bool fits(const SsmArgs& p) {
    return p.N <= kMaxN && p.L <= (1 << 30) && (long long)p.B * p.L <= (1LL << 31) - 1 &&
           (long long)p.S * p.nb * p.G * 64 < (1LL << 31);
}

// Pieces of a sequence. Whole sequences are walked where their blocks fill half of the SMs: pieces
// make every exponential twice, so they have to bring more than twice the blocks.
int pieces_for(const SsmArgs& p, int sms) {
    const long long blocks = (long long)p.S * p.nb * p.G;
    const long long len = p.S > 0 && p.cu ? p.L / p.S : p.L;
    if (2 * blocks >= sms) return 1;
    long long K = (2LL * sms + blocks - 1) / blocks;
    K = K < 64 ? K : 64;
    const long long most = len / 64;
    K = K < most ? K : most;
    return K < 3 ? 1 : (int)K;
}

struct Carve {
    size_t loc, sdt, dA, dch, dbc, total;
};
Carve carve(const SsmArgs& p, bool bwd) {
    Carve w{};
    size_t off = 256;
    auto take = [&](size_t floats) {
        const size_t at = off;
        off += align256(floats * 4);
        return at;
    };
    const size_t CN = (size_t)p.C * p.Np;
    if (p.K > 1) {
        w.loc = take((size_t)p.S * (p.K + 1) * CN);
        w.sdt = take((size_t)p.S * p.K * p.C);
    }
    if (bwd) {
        w.dA = take((size_t)p.S * p.K * CN);
        w.dch = take((size_t)p.S * p.K * 2 * p.C);
        w.dbc = take((size_t)p.nb * p.B * p.L * p.G * 8 * lanes_for(p.N));
    }
    w.total = off;
    return w;
}

template <typename F>
void with_lanes(int dtype, int NL, F&& f) {
    auto by = [&](auto t) {
        using T = decltype(t);
        if (NL == 2) f(t, std::integral_constant<int, 2>());
        else if (NL == 4) f(t, std::integral_constant<int, 4>());
        else if (NL == 8) f(t, std::integral_constant<int, 8>());
        else f(t, std::integral_constant<int, 16>());
        (void)sizeof(T);
    };
    if (dtype == GSPN_F32) by(float{});
    else by(__nv_bfloat16{});
}

}  // namespace
}  // namespace seq
}  // namespace gspn

using namespace gspn;
using namespace gspn::seq;

extern "C" {

// The descriptor does not tell whether cu is given, S does: packed sequences have S > 0.
size_t gspn_ssm_workspace_size(const gspn_ssm_desc* desc, int for_backward) {
    SsmArgs p;
    if (!make_args(desc, &p) || !fits(p)) return 0;
    p.cu = desc->S > 0 ? (const int*)8 : nullptr;
    p.K = pieces_for(p, device_sm_count());
    return carve(p, for_backward != 0).total;
}

size_t gspn_ssm_hsave_size(const gspn_ssm_desc* desc) {
    SsmArgs p;
    if (!make_args(desc, &p) || !fits(p)) return 0;
    const size_t slots = desc->S > 0 ? (size_t)p.L / kSub + p.S : (size_t)p.B * ((p.L + kSub - 1) / kSub);
    return (slots > 0 ? slots : 1) * p.C * p.Np * sizeof(float);
}

gspn_status gspn_ssm_forward(const gspn_ssm_desc* desc, const void* x, const void* dt, const float* A, const void* Bm,
                             const void* Cm, const float* D, const void* z, const float* dt_bias, const int* cu,
                             const float* h0, void* y, float* h, float* hsave, void* ws, size_t ws_bytes,
                             void* stream) {
    SsmArgs p;
    if (!make_args(desc, &p)) return GSPN_ERR_INVALID_ARG;
    if ((desc->S > 0) != (cu != nullptr) || !A) return GSPN_ERR_INVALID_ARG;
    if (p.L > 0 && (!x || !dt || !Bm || !Cm || !y)) return GSPN_ERR_INVALID_ARG;
    if (!fits(p)) return GSPN_ERR_UNSUPPORTED;
    const size_t es = dtype_size(desc->dtype);
    for (const void* q : {x, dt, Bm, Cm, z, (const void*)y})
        if (!aligned_to(q, es)) return GSPN_ERR_ALIGNMENT;
    for (const void* q : {(const void*)A, (const void*)D, (const void*)dt_bias, (const void*)cu, (const void*)h0,
                          (const void*)h})
        if (!aligned_to(q, 4)) return GSPN_ERR_ALIGNMENT;
    if (!aligned_to(hsave, 16) || !aligned_to(ws, 16)) return GSPN_ERR_ALIGNMENT;
    p.x = x; p.dt = dt; p.z = z; p.Bm = Bm; p.Cm = Cm; p.A = A; p.D = D; p.bias = dt_bias; p.cu = cu; p.h0 = h0;
    p.y = y; p.h = h; p.hsave = hsave;
    p.K = pieces_for(p, device_sm_count());
    const Carve w = carve(p, false);
    if (p.K > 1 && !ws) return GSPN_ERR_INVALID_ARG;
    if (p.K > 1 && ws_bytes < w.total) return GSPN_ERR_WORKSPACE;
    p.loc = p.K > 1 ? (float*)((char*)ws + w.loc) : nullptr;
    p.sdt = p.K > 1 ? (float*)((char*)ws + w.sdt) : nullptr;
    p.wide = (p.C / p.G * es) % 16 == 0 && wide_ok(x, p.x_row, p.x_tok, es) && wide_ok(dt, p.dt_row, p.dt_tok, es) &&
             (!z || wide_ok(z, p.z_row, p.z_tok, es)) && aligned_to(y, 16);
    cudaStream_t st = (cudaStream_t)stream;
    cudaError_t e = cudaSuccess;
    with_lanes(desc->dtype, lanes_for(p.N), [&](auto t, auto nl) {
        using T = decltype(t);
        constexpr int NL = decltype(nl)::value;
        const unsigned cblocks = p.nb * p.G;
        auto go = [&](auto kernel, size_t smem, unsigned pieces) {
            if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
            if (e == cudaSuccess) kernel<<<cblocks * pieces * p.S, 32 * NL + kFeed, smem, st>>>(p);
        };
        if (p.K > 1) go(k_ssm_fwd<T, NL, true>, sizeof(FwdSmem<T, NL, true>), p.K - 1);
        go(k_ssm_fwd<T, NL, false>, sizeof(FwdSmem<T, NL, false>), p.K);
    });
    if (e != cudaSuccess) return GSPN_ERR_CUDA;
    return last_status();
}

gspn_status gspn_ssm_backward(const gspn_ssm_desc* desc, const void* x, const void* dt, const float* A, const void* Bm,
                              const void* Cm, const float* D, const void* z, const float* dt_bias, const int* cu,
                              const float* hsave, const void* dy, const float* dh, void* dx, void* ddt, float* dA,
                              void* dBm, void* dCm, float* dD, void* dz, float* ddt_bias, float* dh0, void* ws,
                              size_t ws_bytes, void* stream) {
    SsmArgs p;
    if (!make_args(desc, &p)) return GSPN_ERR_INVALID_ARG;
    if ((desc->S > 0) != (cu != nullptr) || !A || !hsave || !dA || !ws) return GSPN_ERR_INVALID_ARG;
    if ((z != nullptr) != (dz != nullptr) && p.L > 0) return GSPN_ERR_INVALID_ARG;
    if (p.L > 0 && (!x || !dt || !Bm || !Cm || !dy || !dx || !ddt || !dBm || !dCm)) return GSPN_ERR_INVALID_ARG;
    if (!fits(p)) return GSPN_ERR_UNSUPPORTED;
    const size_t es = dtype_size(desc->dtype);
    for (const void* q : {x, dt, Bm, Cm, z, dy, (const void*)dx, (const void*)ddt, (const void*)dBm, (const void*)dCm,
                          (const void*)dz})
        if (!aligned_to(q, es)) return GSPN_ERR_ALIGNMENT;
    for (const void* q : {(const void*)A, (const void*)D, (const void*)dt_bias, (const void*)cu, (const void*)dh,
                          (const void*)dA, (const void*)dD, (const void*)ddt_bias, (const void*)dh0})
        if (!aligned_to(q, 4)) return GSPN_ERR_ALIGNMENT;
    if (!aligned_to(hsave, 16) || !aligned_to(ws, 16)) return GSPN_ERR_ALIGNMENT;
    p.x = x; p.dt = dt; p.z = z; p.Bm = Bm; p.Cm = Cm; p.A = A; p.D = D; p.bias = dt_bias; p.cu = cu;
    p.hsave = const_cast<float*>(hsave); p.dy = dy; p.dh = dh; p.dx = dx; p.ddt = ddt; p.dz = dz; p.dh0 = dh0;
    p.K = pieces_for(p, device_sm_count());
    const Carve w = carve(p, true);
    if (ws_bytes < w.total) return GSPN_ERR_WORKSPACE;
    auto at = [&](size_t off) { return (float*)((char*)ws + off); };
    p.loc = at(w.loc); p.sdt = at(w.sdt); p.dA_part = at(w.dA); p.dch_part = at(w.dch); p.dbc_part = at(w.dbc);
    p.wide = (p.C / p.G * es) % 16 == 0 && wide_ok(x, p.x_row, p.x_tok, es) && wide_ok(dt, p.dt_row, p.dt_tok, es) &&
             (!z || wide_ok(z, p.z_row, p.z_tok, es)) && aligned_to(dy, 16) && aligned_to(dx, 16) &&
             aligned_to(ddt, 16) && aligned_to(dz, 16);
    cudaStream_t st = (cudaStream_t)stream;
    cudaError_t e = cudaSuccess;
    const int NLh = lanes_for(p.N);
    with_lanes(desc->dtype, NLh, [&](auto t, auto nl) {
        using T = decltype(t);
        constexpr int NL = decltype(nl)::value;
        const unsigned cblocks = p.nb * p.G;
        const size_t smem = sizeof(BwdSmem<T, NL>);
        e = cudaFuncSetAttribute(k_ssm_bwd<T, NL>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return;
        if (p.K > 1) k_ssm_bwd_local<T, NL><<<cblocks * (p.K - 1) * p.S, 32 * NL, 0, st>>>(p);
        k_ssm_bwd<T, NL><<<cblocks * p.K * p.S, 32 * NL, smem, st>>>(p);
        const long long per = (long long)p.B * p.L * p.G * 8 * NL;
        if (per > 0)
            k_ssm_sum_bc<T><<<(unsigned)((per + 255) / 256), 256, 0, st>>>(p.dbc_part, cu, p.S, p.B, p.L, p.G, p.N, p.nb,
                                                                         8 * NL, (T*)dBm, (T*)dCm);
        const long long na = (long long)p.C * p.Np + 2 * p.C;
        k_ssm_sum_ac<<<(unsigned)((na + 255) / 256), 256, 0, st>>>(p.dA_part, p.dch_part, p.S * p.K, p.C, p.N, p.Np, dA,
                                                                  dD, ddt_bias);
    });
    if (e != cudaSuccess) return GSPN_ERR_CUDA;
    return last_status();
}

gspn_status gspn_ssm_step(const gspn_ssm_desc* desc, const void* x, const void* dt, const float* A, const void* Bm,
                          const void* Cm, const float* D, const void* z, const float* dt_bias, const int* idx,
                          int slots, float* h, void* y, void* stream) {
    SsmArgs p;
    if (!make_args(desc, &p) || desc->L != 1 || desc->S != 0 || slots < 1) return GSPN_ERR_INVALID_ARG;
    if (!x || !dt || !A || !Bm || !Cm || !h || !y || (!idx && slots < p.B)) return GSPN_ERR_INVALID_ARG;
    if (p.N > kMaxN || p.B > 65535) return GSPN_ERR_UNSUPPORTED;
    const size_t es = dtype_size(desc->dtype);
    for (const void* q : {x, dt, Bm, Cm, z, (const void*)y})
        if (!aligned_to(q, es)) return GSPN_ERR_ALIGNMENT;
    for (const void* q : {(const void*)A, (const void*)D, (const void*)dt_bias, (const void*)idx, (const void*)h})
        if (!aligned_to(q, 4)) return GSPN_ERR_ALIGNMENT;
    p.x = x; p.dt = dt; p.z = z; p.Bm = Bm; p.Cm = Cm; p.A = A; p.D = D; p.bias = dt_bias; p.h = h; p.y = y;
    p.wide = aligned_to(h, 16) && aligned_to(A, 16);
    const int NL = lanes_for(p.N), threads = 128, ch = threads / NL;
    const dim3 grid((p.C + ch - 1) / ch, p.B);
    cudaStream_t st = (cudaStream_t)stream;
    if (desc->dtype == GSPN_F32) k_ssm_step<float><<<grid, threads, 0, st>>>(p, idx, slots, NL);
    else k_ssm_step<__nv_bfloat16><<<grid, threads, 0, st>>>(p, idx, slots, NL);
    return last_status();
}

}  // extern "C"
