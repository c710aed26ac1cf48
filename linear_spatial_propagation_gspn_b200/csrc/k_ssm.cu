// k_ssm.cu -- selective state space scan over token sequences: prompts, gradients, single tokens.
//
//   h_t[c][n] = exp(d_t[c] A[c][n]) h_{t-1}[c][n] + d_t[c] x_t[c] B_t[g][n]
//   y_t[c]    = (sum_n C_t[g][n] h_t[c][n] + D[c] x_t[c]) silu(z_t[c]),   d = softplus(dt + bias)
//
// The recurrence is elementwise in (c, n), so it is no matrix product; what bounds it is one
// exponential for each (t, c, n), which the special-function unit makes at 16 a cycle and SM.
//
// Layout of a block: 32 channels of one sequence (64 bytes of a bf16 row: whole sectors) and
// NL = ceil(N / 4) rounded up to 4, 8 or 16 lanes for each channel, four states in registers per
// lane. Some warps scan tiles of tokens from shared memory; others load the next tile, form the steps
// d and d x once per (t, c), add the lanes' shares of the sums over n and write y.
//
// Parallel over channels and sequences alone, a block walks its whole sequence. Where that leaves
// most of the chip idle, every sequence is cut into K equal pieces: a first pass finds each piece's
// own state from zero and its sum of steps (the decay over the piece is exp(A sum d)), and the main
// pass joins the pieces before its own. That makes every exponential twice.
//
// Measured (B200, bf16, N = 16, gate, D and bias), against the exponentials' time alone:
//   forward, 4 x 2048 tokens of 2048 channels, states saved   156 us   59 us   (two blocks an SM: 68 % of issue slots)
//   the same backward, sums included                          448 us   59 us   (54 % of issue slots, one block an SM)
//   forward, one sequence of 16384 tokens, 4096 channels      705 us  236 us   (128 blocks, 82 cycles a token)
//   a token of 256 rows of 4096 channels                       36 us   4.0 TB/s of states, A and inputs
// Issue slots and, with one block an SM, the scanning warp's latencies stand before the exponentials: a
// token costs a block 200 instructions forward, of which the four scanning warps take about half.
#include "seq_common.cuh"

namespace gspn {
namespace seq {
namespace {

constexpr int kCh = 32;      // channels of a block
constexpr int kTile = 32;    // tokens staged at once
constexpr int kSub = 16;     // tokens between saved states
constexpr int kMaxN = 64;

struct SsmArgs {
    int B, L, C, G, N, S;    // S: sequences (packed or rows)
    int Np;                  // N rounded up to 4
    int K;                   // pieces of a sequence
    int nb, nbb;             // channel blocks of a group; of a backward block's size
    int softplus;
    bool wide, wide_bc;      // x, dt, z, y (and dy and the gradients) have 16-byte aligned vectors; B and C have (a step's)
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
// Two at a time: issue slots are what the staging costs.
__device__ __forceinline__ float2 softplus_of(float2 v) {
    const f2 w = pack(-fminf(fabsf(v.x), 88.f), -fminf(fabsf(v.y), 88.f));
    const f2 t = mul2(w, both(kLog2e));
    const f2 lo = fma2(w, both(kLog2e), mul2(t, both(-1.f)));
    f2 e = ex2_2(t);
    e = fma2(e, mul2(lo, both(kLn2)), e);
    const float2 den = unpack(add2(e, both(2.f)));
    const f2 s = mul2(e, pack(rcp(den.x), rcp(den.y)));
    const f2 q = mul2(s, s);
    f2 r = fma2(q, both(0.14089168f), both(0.13980301f));
    r = fma2(r, q, both(0.20012455f));
    r = fma2(r, q, both(0.33333157f));
    r = fma2(r, q, both(1.f));
    return unpack(fma2(add2(s, s), r, pack(max_nan(v.x, 0.f), max_nan(v.y, 0.f))));
}
__device__ __forceinline__ float softplus_of(float v) { return softplus_of(make_float2(v, v)).x; }

// A token's decay 2^(d A2), A2 = A log2(e). The approximate exponential comes out low on average, and the states
// of a slow channel multiply as many decays as they remember tokens. Its mean relative error, in 1e-8, by -v:
// 0.5 to 0.9 below 2^-9, 0.7 to 2.2 up to 2^-7, 2.5 from there to 1/2 (0.6 to 3.1 by octave halves), 5 above 1. An
// addend to the exponent takes it up again, rounded once together with the product: `tilt_of` follows those
// figures to within 0.2 below 2^-9, where memory is longest. One addend for all, of 2.8e-8, left +1.4 there.
// It changes slowly with v, so a tile of tokens shares that of one step: forward of the token ahead of it, which is
// known before the tile begins (16384 x 4096: the addend costs 1.7 % of the pass, 2.0 with the tile's own first
// token); backward of its own first token (4 x 2048 x 2048: 2 %; renewed at the end of the tile before, registers
// ran out: 4 %). Single tokens have each their own (256 rows of 4096 channels: 34.0 -> 35.4 us).
// 2^tilt rounds to 1, so a step of zero still leaves its state as it was.
__device__ __forceinline__ float tilt_step(float v) { return __saturatef(fmaf(200.f, fabsf(v), -0.5f)); }
__device__ __forceinline__ float tilt_of(float v) { return fmaf(2.05e-8f, tilt_step(v), 0.95e-8f); }
__device__ __forceinline__ f2 tilt_of(f2 v) {
    const float2 s = unpack(v);
    return fma2(pack(tilt_step(s.x), tilt_step(s.y)), both(2.05e-8f), both(0.95e-8f));
}
__device__ __forceinline__ f2 decay2(f2 d, f2 A2, f2 tilt) { return ex2_2(fma2(d, A2, tilt)); }
__device__ __forceinline__ float decay(float d, float A2, float tilt) { return ex2(fmaf(d, A2, tilt)); }

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
// Packed sequences are taken longest first: a block walks its sequence alone, so the longest one decides the
// end, and begun last it ran on by itself (8192 x 2048, nine sequences, the longest of 2277 tokens the last one:
// forward 198 -> 144 us, backward 661 -> 498). Every thread compares one with all the others, which is paid by
// each block: with 128 sequences of 64 tokens 183 -> 242 us, so only up to kRanked, beyond which lengths even out.
// Not inlined: the scan that follows was compiled 3 % slower with it in place.
constexpr int kRanked = 32;
__device__ __noinline__ int nth_longest(const int* cu, int S, int n) {
    __shared__ int found;
    const int i = threadIdx.x;
    if (i < S) {
        const int len = cu[i + 1] - cu[i];
        int ahead = 0, lo = cu[0];
        for (int j = 0; j < S; ++j) {
            const int hi = cu[j + 1], other = hi - lo;
            ahead += other > len || (other == len && j < i);
            lo = hi;
        }
        if (ahead == n) found = i;
    }
    __syncthreads();
    return found;
}
__device__ __forceinline__ Place place_of(const SsmArgs& p, int pieces, int first_piece, int ch, int nb) {
    Place q;
    const int cblocks = nb * p.G;
    q.cb = blockIdx.x % cblocks;
    const int sk = blockIdx.x / cblocks;
    q.k = sk % pieces + first_piece;
    q.s = sk / pieces;
    if (p.cu && p.S > 1 && p.S <= kRanked) q.s = nth_longest(p.cu, p.S, q.s);
    q.g = q.cb / nb;
    const int Cg = p.C / p.G;
    q.c0 = q.g * Cg + (q.cb % nb) * ch;
    q.nc = min(ch, (q.g + 1) * Cg - q.c0);
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

// The same for the threads that feed a forward block: four channels each, NV times over. Eight warps:
// with four, one on each scheduler, their latencies took longer than the scan of a tile.
constexpr int kQ = 4, kVR = kCh / kQ;
template <int NL> struct Feed {
    static constexpr int threads = NL == 16 ? 128 : 256, NV = kTile * kVR / threads;
};
template <typename T, int NL>
__device__ __forceinline__ void ld_feed(typename Quad<T>::raw (&r)[Feed<NL>::NV], const void* base, long long row,
                                        long long tok, const Place& q, int t0, int tid, bool wide) {
#pragma unroll
    for (int i = 0; i < Feed<NL>::NV; ++i) {
        const int v = i * Feed<NL>::threads + tid;
        const int t = t0 + v / kVR, c = v % kVR * kQ;
        r[i] = typename Quad<T>::raw{};
        if (t < q.hi) r[i] = ld_quad((const T*)base + q.sp.row * row + (q.sp.first + t) * tok + q.c0 + c, q.nc - c, wide);
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

// ------------------------------------------------------------------------------------- forward
// The block's first NL warps scan; eight more (four for NL = 16) feed them: they load the tokens, form d and d x,
// and turn the sums over n of the tile before into y. The two work on neighbouring tiles, with one barrier a
// tile, so the long latencies of the one side hide behind the other's arithmetic (16384 x 4096: 1866 us with
// every warp doing both, 817 with four feeding warps, 690 with eight).
// A token's shares of the sums over n, NL for each channel, with four floats between the vectors of
// channels that one feeding thread adds up: its neighbours then start on other banks.
template <int NL> struct YRow {
    static constexpr int vec = kQ * NL + 4, len = kVR * vec;
    static __device__ __forceinline__ int at(int c, int nl) { return c / kQ * vec + c % kQ * NL + nl; }
    // the sum of channel c's shares; row is 16-byte aligned
    static __device__ __forceinline__ float sum(const float* row, int c) {
        const float* s = row + at(c, 0);
        float w = 0.f;
#pragma unroll
        for (int k = 0; k < NL; k += 4) {
            f2 a, b;
            ld_pairs(s + k, a, b);
            const float2 v = unpack(add2(a, b));
            w += v.x + v.y;
        }
        return w;
    }
};

// Shared memory moves 128 bytes a cycle, and 16-byte loads of a whole warp take four cycles even where
// lanes read the same words: a token costs a warp four of them for d, d, d x, d x (doubled, so that the
// two-wide products need no moves) and four for B and C of bf16 inputs, which stay as stored. Rows of
// d have 16 bytes between the vectors of channels that one feeding thread writes, which spreads its
// neighbours over the banks.
struct DRow {
    static constexpr int vec = kQ + 1, len = kVR * vec;     // in entries of 16 bytes
    static __device__ __forceinline__ int at(int c) { return c / kQ * vec + c % kQ; }
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

// Two blocks of NL = 4 fit an SM at 80 registers a thread; the scan needs more, the feed less.
constexpr int kScanRegs4 = 112, kFeedRegs4 = 64, kFwdThreads4 = 128 + Feed<4>::threads;
constexpr int kFwdRegs4 = 128 * kScanRegs4 + Feed<4>::threads * kFeedRegs4;

template <typename T, int NL, bool LOCAL> struct FwdSmem {
    float4 dd[2][kTile][DRow::len];                 // d, d, d x, d x
    BC4<T> bc[2][kTile][NL];
    float y[LOCAL ? 1 : 2][LOCAL ? 1 : kTile][YRow<NL>::len];   // each lane's share of the sums over n
};

// LOCAL: the first pass over pieces (from a zero state, the last piece left out).
template <typename T, int NL, bool LOCAL>
__global__ void __launch_bounds__(32 * NL + Feed<NL>::threads, NL == 4 ? 2 : 1) k_ssm_fwd(const SsmArgs p) {
    extern __shared__ __align__(16) unsigned char smem_raw[];
    FwdSmem<T, NL, LOCAL>& sm = *(FwdSmem<T, NL, LOCAL>*)smem_raw;

    const Place q = place_of(p, LOCAL ? p.K - 1 : p.K, 0, kCh, p.nb);
    if (!LOCAL && q.k > 0 && q.lo >= q.hi) return;
    const int tiles = (q.hi - q.lo + kTile - 1) / kTile;

    if (threadIdx.x >= 32 * NL) {
        // ------------------------------------------------------------ feed
        if constexpr (NL == 4) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kFeedRegs4));
        using P = Feed<NL>;
        typedef typename Quad<T>::raw Raw;
        constexpr int NS = kTile * 4 * NL / P::threads;           // elements of B (and of C) for each thread
        const int tid = threadIdx.x - 32 * NL;
        const int vc = tid % kVR * kQ;
        float bias[kQ], Dv[kQ];
#pragma unroll
        for (int i = 0; i < kQ; ++i) {
            bias[i] = (p.bias && vc + i < q.nc) ? p.bias[q.c0 + vc + i] : 0.f;
            Dv[i] = (!LOCAL && p.D && vc + i < q.nc) ? p.D[q.c0 + vc + i] : 0.f;
        }
        // x and z of the tile to be loaded, the one staged and the one before it
        Raw rx[P::NV], rd[P::NV], rz[P::NV], x1[P::NV], z1[P::NV], x0[P::NV], z0[P::NV];
        T rB[NS], rC[NS];
        auto load = [&](int i) {
            const int t0 = q.lo + i * kTile;
            ld_feed<T, NL>(rx, p.x, p.x_row, p.x_tok, q, t0, tid, p.wide);
            ld_feed<T, NL>(rd, p.dt, p.dt_row, p.dt_tok, q, t0, tid, p.wide);
            ld_states<T, NL>(rB, p.Bm, p.b_row, p.b_tok, q, t0, tid, p.N);
            if constexpr (!LOCAL) {
                if (p.z) ld_feed<T, NL>(rz, p.z, p.z_row, p.z_tok, q, t0, tid, p.wide);
                ld_states<T, NL>(rC, p.Cm, p.c_row, p.c_tok, q, t0, tid, p.N);
            }
        };
        auto stage = [&](int i) {
            const int t0 = q.lo + i * kTile, buf = i & 1;
#pragma unroll
            for (int k = 0; k < P::NV; ++k) {
                const int t = (k * P::threads + tid) / kVR;
                x0[k] = x1[k];
                z0[k] = z1[k];
                x1[k] = rx[k];
                z1[k] = rz[k];
                float xv[kQ], dv[kQ];
                unpack_quad(rx[k], xv);
                unpack_quad(rd[k], dv);
                // A token behind the end makes no step, and the state stays; its x was read as zero, and so were
                // those of channels behind the last, whose states are zero.
                const bool ok = t0 + t < q.hi;
                float4* to = &sm.dd[buf][t][DRow::at(vc)];
#pragma unroll
                for (int j = 0; j < kQ; j += 2) {
                    float2 d = make_float2(dv[j] + bias[j], dv[j + 1] + bias[j + 1]);
                    if (p.softplus) d = softplus_of(d);
                    if (!ok) d = make_float2(0.f, 0.f);
                    const float2 w = unpack(mul2(pack(d.x, d.y), pack(xv[j], xv[j + 1])));
                    to[j] = make_float4(d.x, d.x, w.x, w.x);
                    to[j + 1] = make_float4(d.y, d.y, w.y, w.y);
                }
            }
#pragma unroll
            for (int k = 0; k < NS; ++k) {
                const int e = k * P::threads + tid;
                T* to = (&sm.bc[buf][0][0])[e / 4].v + e % 4;
                to[0] = rB[k];
                if constexpr (!LOCAL) to[4] = rC[k];
            }
        };
        auto finish = [&](int i) {                                // i is the tile before the one staged last
            const int t0 = q.lo + i * kTile, buf = i & 1;
#pragma unroll
            for (int k = 0; k < P::NV; ++k) {
                const int t = (k * P::threads + tid) / kVR;
                if (t0 + t < q.hi) {
                    float xv[kQ], zv[kQ], out[kQ];
                    unpack_quad(x0[k], xv);
                    unpack_quad(z0[k], zv);
#pragma unroll
                    for (int j = 0; j < kQ; ++j) {
                        out[j] = fmaf(Dv[j], xv[j], YRow<NL>::sum(sm.y[buf][t], vc + j));
                        if (p.z) out[j] *= silu(zv[j]);
                    }
                    st_quad<T>((T*)p.y + ((long long)q.sp.row * p.L + q.sp.first + t0 + t) * p.C + q.c0 + vc, out,
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
    if constexpr (NL == 4) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kScanRegs4));
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
    const f2 A01 = pack(A2[0], A2[1]), A23 = pack(A2[2], A2[3]);
    f2 h01 = pack(h[0], h[1]), h23 = pack(h[2], h[3]);
    const long long save0 = LOCAL ? 0 : save_slot(p, q.sp, q.s);
    float sum_d = 0.f;
    __syncthreads();
    f2 t01 = 0, t23 = 0;                                          // see tilt_of
    if (tiles > 0) {
        const f2 d = both(sm.dd[0][0][DRow::at(cl)].x);
        t01 = tilt_of(mul2(d, A01));
        t23 = tilt_of(mul2(d, A23));
    }
    for (int i = 0; i < tiles; ++i) {
        const int t0 = q.lo + i * kTile, buf = i & 1;
        // Operands of four tokens are fetched while the four before are worked on; the stores below would
        // otherwise hold back the loads behind them.
        f2 dd[2][4], dx[2][4];
        BC4<T> bc[2][4];
        auto fetch = [&](int t, int w) {
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                ld_pairs((const float*)&sm.dd[buf][t + u][DRow::at(cl)], dd[w][u], dx[w][u]);
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
                float b[4], cc[4];
                if constexpr (LOCAL) get_b(bc[w][u], b);
                else get_bc(bc[w][u], b, cc);
                const f2 a01 = decay2(dd[w][u], A01, t01), a23 = decay2(dd[w][u], A23, t23);
                h01 = fma2(a01, h01, mul2(dx[w][u], pack(b[0], b[1])));
                h23 = fma2(a23, h23, mul2(dx[w][u], pack(b[2], b[3])));
                if constexpr (LOCAL) {
                    sum_d += unpack(dd[w][u]).x;
                } else {
                    const float2 s = unpack(fma2(h01, pack(cc[0], cc[1]), mul2(h23, pack(cc[2], cc[3]))));
                    sm.y[buf][t + u][YRow<NL>::at(cl, nl)] = s.x + s.y;
                }
            }
            if (t + 4 == kTile) {
                t01 = tilt_of(mul2(dd[w][3], A01));
                t23 = tilt_of(mul2(dd[w][3], A23));
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
// The forward saved the state before every 16th token. From it 16 tokens are walked forward with every
// h_t kept in registers, then walked back (their decays are formed again: kept too, they would leave
// no registers for a second channel in each lane).
//
// A block is four scanning warps and eight that feed them, as in the forward pass. A scanning lane has
// two channels x four states: B and C, and the sums over channels for dB and dC, are then shared by
// two. Those sums go over the warp's channel lanes by halving: what one lane gives away is what its
// partner keeps. No selects are needed, since a lane holds its states in an order of its own (slot j is
// state j xor the lane's low bits). The sums over n go the same way once (the two channels of
// neighbouring lanes are in opposite order), and the feeding warps add the rest. One channel a lane and
// eight scanning warps took 557 cycles a token of 64 channels against 464.
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

// LOCAL: the first pass over pieces: what each piece passes back from a zero gradient behind it (all
// pieces but the first) and its sum of steps.
template <typename T, int NL>
__global__ void __launch_bounds__(32 * NL) k_ssm_bwd_local(const SsmArgs p) {
    using P = Part<T, NL>;
    constexpr int V = P::V;
    __shared__ __align__(16) float2 sdr[kTile][kCh];              // d, r
    __shared__ __align__(16) float sC[kTile][4 * NL];
    const Place q = place_of(p, p.K - 1, 1, kCh, p.nb);
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
        float tilt[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) tilt[j] = tilt_of(sdr[0][cl].x * A2[j]);
#pragma unroll 8
        for (int t = kTile - 1; t >= 0; --t) {
            const float2 dr = sdr[t][cl];
            const float4 c4 = *(const float4*)&sC[t][n0];
            sum_d += dr.x;
            ag[0] = decay(dr.x, A2[0], tilt[0]) * fmaf(c4.x, dr.y, ag[0]);
            ag[1] = decay(dr.x, A2[1], tilt[1]) * fmaf(c4.y, dr.y, ag[1]);
            ag[2] = decay(dr.x, A2[2], tilt[2]) * fmaf(c4.z, dr.y, ag[2]);
            ag[3] = decay(dr.x, A2[3], tilt[3]) * fmaf(c4.w, dr.y, ag[3]);
        }
        __syncthreads();
    }
    const long long slot = (long long)q.s * p.K + q.k;
    if (cok && n0 < p.Np) *(float4*)(p.loc + (slot * p.C + c) * p.Np + n0) = make_float4(ag[0], ag[1], ag[2], ag[3]);
    if (cok && nl == 0) p.sdt[slot * p.C + c] = sum_d;
}

constexpr int kScan = 128, kFeedB = 256, kTB = kSub;              // threads, tokens of a backward block's tile
constexpr int kScanRegs = 248, kFeedRegs = 128;                   // 168 each at launch

template <int NL> struct Bwd {
    static constexpr int CH = 256 / NL;                           // channels of a block
    static constexpr int QR = CH / kQ;                            // vectors of four channels in a token
    static constexpr int quads = kTB * QR, active = quads;        // one for each feeding thread, at most
    static constexpr int states = kTB * 4 * NL, NS = (states + kFeedB - 1) / kFeedB;
    static constexpr int PC = perm_copies(NL), W = NL / 2;        // orders of B and C; shares of a sum over n
};
// Rows of pairs (d, d x), and of the shares of a sum over n: padded as in the forward pass.
template <int NL> struct PRow {
    static constexpr int vec = kQ + 1, len = Bwd<NL>::QR * vec;   // in entries of 16 bytes
    static __device__ __forceinline__ int at(int c) { return c / kQ * vec + c % kQ; }
};
template <int NL> struct ORow {
    static constexpr int W = Bwd<NL>::W, vec = kQ * W + 4, len = Bwd<NL>::QR * vec;
    static __device__ __forceinline__ int at(int c, int w) { return c / kQ * vec + c % kQ * W + w; }
    // the sums of the four channels from c on (a multiple of four)
    static __device__ __forceinline__ void sum(const float* row, int c, float (&o)[kQ]) {
        const float* s = row + at(c, 0);
        float f[kQ * W];
#pragma unroll
        for (int k = 0; k < kQ * W; k += 4) {
            const float4 v = *(const float4*)(s + k);
            f[k] = v.x; f[k + 1] = v.y; f[k + 2] = v.z; f[k + 3] = v.w;
        }
#pragma unroll
        for (int j = 0; j < kQ; ++j) {
            o[j] = f[j * W];
#pragma unroll
            for (int k = 1; k < W; ++k) o[j] += f[j * W + k];
        }
    }
};

template <typename T, int NL> struct BwdSmem {
    float4 dd[2][kTB][PRow<NL>::len];                             // d, d, d x, d x
    float2 r[2][kTB][Bwd<NL>::CH];                                // dy silu(z), twice
    float4 B[2][kTB][Bwd<NL>::PC][NL], C[2][kTB][Bwd<NL>::PC][NL];   // in fp32: unpacking costs the scan more than the loads
    float o[2][3][kTB][ORow<NL>::len];                            // C h, g B, e A: shares of the sums over n
    float sum[2][kScan / 32][kTB][8 * NL];                        // dB, dC: sums over a warp's channels
};

template <typename T, int NL>
__global__ void __launch_bounds__(kScan + kFeedB, 1) k_ssm_bwd(const SsmArgs p) {
    using W = Bwd<NL>;
    constexpr int PC = W::PC;
    constexpr unsigned all = 0xffffffffu;
    extern __shared__ __align__(16) unsigned char smem_raw[];
    BwdSmem<T, NL>& sm = *(BwdSmem<T, NL>*)smem_raw;
    const Place q = place_of(p, p.K, 0, W::CH, p.nbb);
    const int tiles = (q.hi - q.lo + kTB - 1) / kTB;
    const long long slot = (long long)q.s * p.K + q.k;

    if (threadIdx.x >= kScan) {
        // ------------------------------------------------------------ feed
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kFeedRegs));
        typedef typename Quad<T>::raw Raw;
        const int tid = threadIdx.x - kScan;
        const int vc = tid % W::QR * kQ;
        float bias[kQ], Dv[kQ], sD[kQ], sb[kQ];
#pragma unroll
        for (int j = 0; j < kQ; ++j) {
            bias[j] = (p.bias && vc + j < q.nc) ? p.bias[q.c0 + vc + j] : 0.f;
            Dv[j] = (p.D && vc + j < q.nc) ? p.D[q.c0 + vc + j] : 0.f;
            sD[j] = sb[j] = 0.f;
        }
        // x, dt, z, dy: of the tile in flight, of the one staged last and of the one staged before it
        Raw rr[4], k1[4], k0[4];
        T rB[W::NS], rC[W::NS];
        auto load = [&](int i) {
            if (i < 0) return;
            const int t0 = q.lo + i * kTB, t = t0 + tid / W::QR;
            const bool in = tid < W::quads && t < q.hi;
            auto one = [&](const void* base, long long row, long long tok) {
                return in ? ld_quad((const T*)base + q.sp.row * row + (q.sp.first + t) * tok + q.c0 + vc, q.nc - vc, p.wide) : Raw{};
            };
            rr[0] = one(p.x, p.x_row, p.x_tok);
            rr[1] = one(p.dt, p.dt_row, p.dt_tok);
            rr[2] = p.z ? one(p.z, p.z_row, p.z_tok) : Raw{};
            rr[3] = one(p.dy, (long long)p.L * p.C, p.C);
#pragma unroll
            for (int k = 0; k < W::NS; ++k) {
                const int e = k * kFeedB + tid, t = t0 + e / (4 * NL), n = e % (4 * NL);
                rB[k] = rC[k] = T(0.f);
                if (e < W::states && t < q.hi && n < p.N) {
                    rB[k] = ((const T*)p.Bm)[q.sp.row * p.b_row + (q.sp.first + t) * p.b_tok + (long long)q.g * p.N + n];
                    rC[k] = ((const T*)p.Cm)[q.sp.row * p.c_row + (q.sp.first + t) * p.c_tok + (long long)q.g * p.N + n];
                }
            }
        };
        auto stage = [&](int i) {
            const int t0 = q.lo + i * kTB, buf = i & 1;
            {
                const int t = tid / W::QR;
#pragma unroll
                for (int m = 0; m < 4; ++m) { k0[m] = k1[m]; k1[m] = rr[m]; }
                if (W::active == kFeedB || tid < W::quads) {
                    float xv[kQ], dv[kQ], zv[kQ], gv[kQ];
                    unpack_quad(rr[0], xv);
                    unpack_quad(rr[1], dv);
                    unpack_quad(rr[2], zv);
                    unpack_quad(rr[3], gv);
                    const bool ok = t0 + t < q.hi;                // behind the end: no step; x and dy were read as zero
                    float r[kQ];
#pragma unroll
                    for (int j = 0; j < kQ; j += 2) {
                        float2 d = make_float2(dv[j] + bias[j], dv[j + 1] + bias[j + 1]);
                        if (p.softplus) d = softplus_of(d);
                        if (!ok) d = make_float2(0.f, 0.f);
                        const float2 w = unpack(mul2(pack(d.x, d.y), pack(xv[j], xv[j + 1])));
                        sm.dd[buf][t][PRow<NL>::at(vc + j)] = make_float4(d.x, d.x, w.x, w.x);
                        sm.dd[buf][t][PRow<NL>::at(vc + j + 1)] = make_float4(d.y, d.y, w.y, w.y);
                        r[j] = p.z ? gv[j] * silu(zv[j]) : gv[j];
                        r[j + 1] = p.z ? gv[j + 1] * silu(zv[j + 1]) : gv[j + 1];
                    }
                    *(float4*)&sm.r[buf][t][vc] = make_float4(r[0], r[0], r[1], r[1]);
                    *(float4*)&sm.r[buf][t][vc + 2] = make_float4(r[2], r[2], r[3], r[3]);
                }
            }
#pragma unroll
            for (int k = 0; k < W::NS; ++k) {
                const int e = k * kFeedB + tid, t = e / (4 * NL), n = e % (4 * NL);
                if (W::states >= kFeedB || e < W::states) {
#pragma unroll
                    for (int m = 0; m < PC; ++m) {
                        ((float*)&sm.B[buf][t][m][n / 4])[n % 4 ^ m] = Io<T>::ld(&rB[k]);
                        ((float*)&sm.C[buf][t][m][n / 4])[n % 4 ^ m] = Io<T>::ld(&rC[k]);
                    }
                }
            }
        };
        // Gradients of tile i (the one staged before the last) from the complete sums.
        auto finish = [&](int i) {
            const int t0 = q.lo + i * kTB, buf = i & 1;
            {
                const int t = tid / W::QR;
                if (tid < W::quads && t0 + t < q.hi) {
                    float xv[kQ], dv[kQ], zv[kQ], gv[kQ], ox[kQ], od[kQ], oz[kQ], ys[kQ], gBs[kQ], eAs[kQ];
                    unpack_quad(k0[0], xv);
                    unpack_quad(k0[1], dv);
                    unpack_quad(k0[2], zv);
                    unpack_quad(k0[3], gv);
                    ORow<NL>::sum(sm.o[buf][0][t], vc, ys);
                    ORow<NL>::sum(sm.o[buf][1][t], vc, gBs);
                    ORow<NL>::sum(sm.o[buf][2][t], vc, eAs);
#pragma unroll
                    for (int j = 0; j < kQ; ++j) {
                        const float gB = gBs[j], eA = eAs[j] * kLn2;
                        const float d = sm.dd[buf][t][PRow<NL>::at(vc + j)].x;
                        float r = gv[j];
                        if (p.z) {
                            const float y = fmaf(Dv[j], xv[j], ys[j]);
                            const float s = sigmoid(zv[j]);
                            oz[j] = gv[j] * y * fmaf(zv[j] * s, 1.f - s, s);
                            r *= zv[j] * s;
                        }
                        ox[j] = fmaf(gB, d, Dv[j] * r);
                        float w = fmaf(gB, xv[j], eA);
                        if (p.softplus) w *= sigmoid(dv[j] + bias[j]);
                        od[j] = w;
                        sD[j] = fmaf(r, xv[j], sD[j]);
                        sb[j] += w;
                    }
                    const long long at = ((long long)q.sp.row * p.L + q.sp.first + t0 + t) * p.C + q.c0 + vc;
                    st_quad<T>((T*)p.dx + at, ox, q.nc - vc, p.wide);
                    st_quad<T>((T*)p.ddt + at, od, q.nc - vc, p.wide);
                    if (p.z) st_quad<T>((T*)p.dz + at, oz, q.nc - vc, p.wide);
                }
            }
            // the warps' sums in order, to this block's part of dB and dC
#pragma unroll
            for (int k = 0; k < kTB * 8 * NL / kFeedB; ++k) {
                const int e = k * kFeedB + tid, t = e / (8 * NL), v = e % (8 * NL);
                float w = 0.f;
#pragma unroll
                for (int m = 0; m < kScan / 32; ++m) w += sm.sum[buf][m][t][v];
                if (t0 + t < q.hi)
                    p.dbc_part[(((long long)(q.cb % p.nbb) * p.B * p.L + (long long)q.sp.row * p.L + q.sp.first + t0 + t) *
                                    p.G + q.g) * (8 * NL) + v] = w;
            }
        };
        if (tiles > 0) {
            load(tiles - 1);
            stage(tiles - 1);
            load(tiles - 2);
        }
        __syncthreads();
        for (int i = tiles - 1; i >= 0; --i) {
            if (i > 0) {
                stage(i - 1);
                load(i - 2);
            } else {
#pragma unroll
                for (int m = 0; m < 4; ++m) k0[m] = k1[m];
            }
            __syncthreads();
            // The shares and sums of tile i are written again behind the next barrier only. Its d is not: the next
            // stage() overwrites it before that, but each thread reads back only the entries that it staged itself.
            finish(i);
        }
        // dD and d dt_bias: the threads that share a vector of channels, in order
        asm volatile("bar.sync 1, 256;" ::: "memory");
        float* acc = &sm.o[0][0][0][0];
        static_assert(sizeof(sm.o) >= kFeedB * 2 * kQ * sizeof(float), "the sums fit where the shares were");
#pragma unroll
        for (int j = 0; j < kQ; ++j) {
            acc[tid * 2 * kQ + j] = sD[j];
            acc[tid * 2 * kQ + kQ + j] = sb[j];
        }
        asm volatile("bar.sync 1, 256;" ::: "memory");
        for (int e = tid; e < 2 * W::CH; e += kFeedB) {
            const int which = e / W::CH, cc = e % W::CH;
            float w = 0.f;
            for (int i = cc / kQ; i < W::active; i += W::QR) w += acc[i * 2 * kQ + which * kQ + cc % kQ];
            if (cc < q.nc) p.dch_part[(slot * 2 + which) * p.C + q.c0 + cc] = w;
        }
        return;
    }

    // ---------------------------------------------------------------- scan
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kScanRegs));
    const int lane = threadIdx.x & 31, nl = lane % NL, warp = threadIdx.x >> 5;
    const int ql = lane / NL, pm = ql & (PC - 1);                 // channel lane, order of the states
    const int b = nl & 1;
    // slot 0 is the channel whose sums over n this lane keeps, slot 1 the one it gives to its neighbour
    const int cl[2] = {warp * (64 / NL) + 2 * ql + b, warp * (64 / NL) + 2 * ql + 1 - b};
    const int n0 = 4 * nl;
    bool keeps[2];
    float A[2][4], ag4[2][4];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        const bool cok = cl[s] < q.nc;
        const long long c = q.c0 + cl[s];
        keeps[s] = cok && n0 < p.Np;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const bool ok = cok && n0 + j < p.N;
            A[s][j] = ok ? p.A[c * p.N + n0 + j] * kLog2e : 0.f;
            ag4[s][j] = ok && p.dh ? p.dh[((long long)q.s * p.C + c) * p.N + n0 + j] : 0.f;
        }
        if (keeps[s])
            for (int k = p.K - 1; k > q.k; --k) {                 // join the pieces behind this one
                const long long sl = (long long)q.s * p.K + k;
                const float sd = p.sdt[sl * p.C + c];
                const float4 m = *(const float4*)(p.loc + (sl * p.C + c) * p.Np + n0);
                ag4[s][0] = fmaf(ex2(sd * A[s][0]), ag4[s][0], m.x);
                ag4[s][1] = fmaf(ex2(sd * A[s][1]), ag4[s][1], m.y);
                ag4[s][2] = fmaf(ex2(sd * A[s][2]), ag4[s][2], m.z);
                ag4[s][3] = fmaf(ex2(sd * A[s][3]), ag4[s][3], m.w);
            }
        permute4(A[s], pm);
        permute4(ag4[s], pm);
    }
    f2 A2[2][2], ag[2][2], dA[2][2];
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            A2[s][m] = pack(A[s][2 * m], A[s][2 * m + 1]);
            ag[s][m] = pack(ag4[s][2 * m], ag4[s][2 * m + 1]);
            dA[s][m] = pack(0.f, 0.f);
        }
    const long long save0 = save_slot(p, q.sp, q.s);
    float4 rh[2];
    auto load_h = [&](int i) {
        if (i < 0) return;
#pragma unroll
        for (int s = 0; s < 2; ++s)
            rh[s] = keeps[s] ? *(const float4*)(p.hsave + ((save0 + q.lo / kSub + i) * p.C + q.c0 + cl[s]) * p.Np + n0)
                             : make_float4(0.f, 0.f, 0.f, 0.f);
    };
    load_h(tiles - 1);
    __syncthreads();
    for (int i = tiles - 1; i >= 0; --i) {
        const int buf = i & 1;
        f2 hin[2][2], h[kTB][2][2];
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            float f[4] = {rh[s].x, rh[s].y, rh[s].z, rh[s].w};
            permute4(f, pm);
            hin[s][0] = pack(f[0], f[1]);
            hin[s][1] = pack(f[2], f[3]);
        }
        load_h(i - 1);
        f2 tilt[2][2];
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const f2 d = both(sm.dd[buf][0][PRow<NL>::at(cl[s])].x);
            tilt[s][0] = tilt_of(mul2(d, A2[s][0]));
            tilt[s][1] = tilt_of(mul2(d, A2[s][1]));
        }
#pragma unroll
        for (int t = 0; t < kTB; ++t) {
            f2 b01, b23;
            ld_pairs((const float*)&sm.B[buf][t][pm][nl], b01, b23);
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                f2 d, dx;
                ld_pairs((const float*)&sm.dd[buf][t][PRow<NL>::at(cl[s])], d, dx);
                h[t][s][0] = fma2(decay2(d, A2[s][0], tilt[s][0]), t ? h[t - 1][s][0] : hin[s][0], mul2(dx, b01));
                h[t][s][1] = fma2(decay2(d, A2[s][1], tilt[s][1]), t ? h[t - 1][s][1] : hin[s][1], mul2(dx, b23));
            }
        }
        f2 dAs[2][2];                                             // sums of 16 tokens join the long sum as one
#pragma unroll
        for (int s = 0; s < 2; ++s) dAs[s][0] = dAs[s][1] = pack(0.f, 0.f);
        // A token's operands are fetched before the stores of the one ahead of it, which would hold them back.
        f2 od[2][2], odx[2][2], orr[2][2], ob[2][2], oc2[2][2];
        auto fetch = [&](int t) {
            const int w = t & 1;
            ld_pairs((const float*)&sm.B[buf][t][pm][nl], ob[w][0], ob[w][1]);
            ld_pairs((const float*)&sm.C[buf][t][pm][nl], oc2[w][0], oc2[w][1]);
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                ld_pairs((const float*)&sm.dd[buf][t][PRow<NL>::at(cl[s])], od[w][s], odx[w][s]);
                orr[w][s] = *(const f2*)&sm.r[buf][t][cl[s]];
            }
        };
        fetch(kTB - 1);
        // A token's sums over lanes take three exchanges in turn. They run beside the next token's arithmetic,
        // a level at a time: a scheduler has this one scanning warp, which issues in order and would
        // otherwise wait out each exchange.
        f2 pB[2], pC[2];                                          // of the token ahead: shares of dB and dC,
        float py[2], pg[2], pe[2];                                // and of the sums over n
#pragma unroll
        for (int t = kTB - 1; t >= -1; --t) {
            const bool work = t >= 0, sums = t < kTB - 1;
            float x0, x1, x2, x3, xy, xg, xe;                     // what comes back from the first exchange
            float vb = 0.f, vb2 = 0.f, vc = 0.f, vc2 = 0.f, y1 = 0.f, y2 = 0.f, z1 = 0.f;
            if (sums) {
                x0 = __shfl_xor_sync(all, unpack(pB[0]).y, NL);
                x1 = __shfl_xor_sync(all, unpack(pB[1]).y, NL);
                x2 = __shfl_xor_sync(all, unpack(pC[0]).y, NL);
                x3 = __shfl_xor_sync(all, unpack(pC[1]).y, NL);
                xy = __shfl_xor_sync(all, py[1], 1);              // slot 1 is the neighbour's slot 0
                xg = __shfl_xor_sync(all, pg[1], 1);
                xe = __shfl_xor_sync(all, pe[1], 1);
            }
            f2 vB[2], vC[2];
            float yv[2], gv[2], ev[2];
            auto slot = [&](auto which) {
                constexpr int s = decltype(which)::value;
                const f2 (&b2)[2] = ob[t & 1];
                const f2 (&c2)[2] = oc2[t & 1];
                const f2 d = od[t & 1][s], dx = odx[t & 1][s], r = orr[t & 1][s];
                f2 y, gb, ea;
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    const f2 hp = t > 0 ? h[t > 0 ? t - 1 : 0][s][m] : hin[s][m];
                    const f2 ht = h[t > 0 ? t : 0][s][m];
                    const f2 g = fma2(c2[m], r, ag[s][m]);
                    vC[m] = s ? fma2(r, ht, vC[m]) : mul2(r, ht);
                    vB[m] = s ? fma2(g, dx, vB[m]) : mul2(g, dx);
                    y = m ? fma2(c2[m], ht, y) : mul2(c2[m], ht);
                    gb = m ? fma2(g, b2[m], gb) : mul2(g, b2[m]);
                    ag[s][m] = mul2(decay2(d, A2[s][m], tilt[s][m]), g);
                    const f2 e = mul2(ag[s][m], hp);
                    dAs[s][m] = fma2(e, d, dAs[s][m]);
                    ea = m ? fma2(e, A2[s][m], ea) : mul2(e, A2[s][m]);
                }
                const float2 u = unpack(y), v = unpack(gb), w = unpack(ea);
                yv[s] = u.x + u.y;
                gv[s] = v.x + v.y;
                ev[s] = w.x + w.y;
            };
            if (work) {
                if (t > 0) fetch(t - 1);
                slot(std::integral_constant<int, 0>());
            }
            float* out = sm.sum[buf][warp][sums ? t + 1 : 0];
            if (sums) {
                vb = unpack(pB[0]).x + x0;
                vb2 = unpack(pB[1]).x + x1;
                vc = unpack(pC[0]).x + x2;
                vc2 = unpack(pC[1]).x + x3;
                if constexpr (NL < 16) {
                    y1 = __shfl_xor_sync(all, vb2, 2 * NL);
                    y2 = __shfl_xor_sync(all, vc2, 2 * NL);
                }
                const int oc = ORow<NL>::at(cl[0], nl >> 1);
                sm.o[buf][0][t + 1][oc] = py[0] + xy;
                sm.o[buf][1][t + 1][oc] = pg[0] + xg;
                sm.o[buf][2][t + 1][oc] = pe[0] + xe;
            }
            if (work) slot(std::integral_constant<int, 1>());
            if (sums) {
                if constexpr (NL == 16) {
                    out[n0 + pm] = vb;
                    out[n0 + (2 ^ pm)] = vb2;
                    out[4 * NL + n0 + pm] = vc;
                    out[4 * NL + n0 + (2 ^ pm)] = vc2;
                } else {
                    vb += y1;
                    vc += y2;
                    if constexpr (NL == 8) {
                        out[n0 + pm] = vb;
                        out[4 * NL + n0 + pm] = vc;
                    } else {
                        const bool up = ql & 4;
                        z1 = __shfl_xor_sync(all, up ? vb : vc, 4 * NL);
                        out[(up ? 4 * NL : 0) + n0 + pm] = (up ? vc : vb) + z1;
                    }
                }
            }
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                pB[m] = vB[m];
                pC[m] = vC[m];
                py[m] = yv[m];
                pg[m] = gv[m];
                pe[m] = ev[m];
            }
        }
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int m = 0; m < 2; ++m) dA[s][m] = add2(dA[s][m], dAs[s][m]);
        __syncthreads();
    }
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        const long long c = q.c0 + cl[s];
        const float2 u = unpack(ag[s][0]), v = unpack(ag[s][1]), x = unpack(dA[s][0]), y = unpack(dA[s][1]);
        float f[4] = {u.x, u.y, v.x, v.y}, a[4] = {x.x, x.y, y.x, y.y};
        permute4(f, pm);
        permute4(a, pm);
        if (keeps[s]) *(float4*)(p.dA_part + (slot * p.C + c) * p.Np + n0) = make_float4(a[0], a[1], a[2], a[3]);
        if (p.dh0 && q.k == 0) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (cl[s] < q.nc && n0 + j < p.N) p.dh0[((long long)q.s * p.C + c) * p.N + n0 + j] = f[j];
        }
    }
}

// dB and dC: the channel blocks of a group in order. Thread = four of a token's values (w4 such fours,
// B's before C's).
template <typename T>
__global__ void k_ssm_sum_bc(const float* part, const int* cu, int S, int B, int L, int G, int N, int nb, int w4,
                             T* dBm, T* dCm) {
    const long long per = (long long)B * L * G * w4;
    const long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= per) return;
    const int v = (int)(i % w4);
    const long long tg = i / w4;                                   // token * G + group
    if (cu) {
        const long long t = tg / G;
        if (t < min(max(cu[0], 0), L) || t >= min(max(cu[S], 0), L)) return;
    }
    const int n = v % (w4 / 2) * 4;
    if (n >= N) return;
    const float4* s = (const float4*)part + i;
    f2 a = pack(0.f, 0.f), b = a;
#pragma unroll 8
    for (int k = 0; k < nb; ++k) {
        const float4 f = s[k * per];
        a = add2(a, pack(f.x, f.y));
        b = add2(b, pack(f.z, f.w));
    }
    const float2 x = unpack(a), y = unpack(b);
    const float o[4] = {x.x, x.y, y.x, y.y};
    T* to = (v < w4 / 2 ? dBm : dCm) + tg * N + n;
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (n + j < N) Io<T>::st(to + j, o[j]);
}

// dA, dD, d dt_bias: the sequences' pieces in order.
__global__ void k_ssm_sum_ac(const float* dA_part, const float* dch_part, int slots, int C, int N, int Np, float* dA,
                             float* dD, float* dbias) {
    const long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x;
    const long long na = (long long)C * Np;
    if (i < na) {
        const int n = (int)(i % Np);
        float w = 0.f;
#pragma unroll 8
        for (int k = 0; k < slots; ++k) w += dA_part[k * na + i];
        if (n < N) dA[i / Np * N + n] = w;
    } else if (i < na + 2 * C) {
        const long long c = i - na;
        float w = 0.f;
#pragma unroll 8
        for (int k = 0; k < slots; ++k) w += dch_part[(long long)k * 2 * C + c];
        float* out = c < C ? dD : dbias;
        if (out) out[c % C] = w;
    }
}

// ----------------------------------------------------------------------------------- one token
// State traffic bounds it: 8 N bytes a row and channel. A lane holds four states of I channels. I = 4 (as
// far apart as the block is wide) puts four 16-byte loads of the state in flight, and each of a
// channel's lanes does the scalar work of one of the four channels (step size, gate, output) and hands
// the step to the others; I = 1 has more blocks for few rows. A, which is as large as a row's state, is
// read once for the block's `group` rows, and the next row's state is fetched ahead. Rows that name the
// slot of an earlier row leave their token to that row, which takes them in order.
constexpr int kStep = 128, kGroup = 8;

// PLAIN: full blocks of one group whose states fill their lanes with aligned vectors (N = 4 NL, C a multiple
// of the block's channels): without the general form's checks and 64-bit offsets, which were most of
// its instructions (256 rows of 4096 channels: 620 for each warp and row).
template <typename T, int NL, int I, bool PLAIN>
__global__ void __launch_bounds__(kStep) k_ssm_step(const SsmArgs p, const int* idx, int slots, int group) {
    constexpr unsigned all = 0xffffffffu;
    constexpr int CH = kStep / NL;                                // distance of a lane's channels
    __shared__ unsigned flags[2];                                 // rows of the group with an earlier, a later row of their slot
    const int b0 = blockIdx.y * group, rows = min(group, p.B - b0);
    const int lane = threadIdx.x & 31, nl = threadIdx.x % NL, n0 = 4 * nl, base = lane - nl;
    const long long c0 = (long long)blockIdx.x * I * CH + threadIdx.x / NL;
    const long long cm = c0 + (nl & (I - 1)) * CH;                // the channel of this lane's scalar work
    const bool mine = PLAIN || cm < p.C;
    const int Cg = p.C / p.G;
    const bool vec = PLAIN || p.wide;                             // N a multiple of four, h and A aligned
    const bool same_group = PLAIN || p.G == 1;

    // Offsets of the lane's states in a row's state (C N < 2^30).
    const unsigned N = PLAIN ? 4u * NL : (unsigned)p.N, at0 = (unsigned)c0 * N + n0, at_step = CH * N;
    bool in[I];
#pragma unroll
    for (int i = 0; i < I; ++i) in[i] = PLAIN || c0 + i * CH < p.C;
    auto read4 = [&](const float* s, f2 (&v)[2]) {                // four states of a channel
        v[0] = v[1] = both(0.f);
        if (vec) {
            if (PLAIN || n0 < p.N) ld_pairs(s, v[0], v[1]);
        } else {
            float f[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (n0 + j < p.N) f[j] = s[j];
            v[0] = pack(f[0], f[1]);
            v[1] = pack(f[2], f[3]);
        }
    };
    auto slot_of = [&](int r) { return r < rows ? (idx ? idx[b0 + r] : b0 + r) : -1; };
    f2 h[I][2], next[I][2];
    auto fetch = [&](int slot) {
        if (slot < 0 || slot >= slots) return;
        const float* hp = p.h + (long long)slot * p.C * p.N;
#pragma unroll
        for (int i = 0; i < I; ++i)
            if (in[i]) read4(hp + (at0 + i * at_step), next[i]);
    };
    int slot = slot_of(0);
    fetch(slot);
    f2 A2[I][2];
    int g[I];
#pragma unroll
    for (int i = 0; i < I; ++i) {
        A2[i][0] = A2[i][1] = both(0.f);
        if (in[i]) read4(p.A + (at0 + i * at_step), A2[i]);
        A2[i][0] = mul2(A2[i][0], both(kLog2e));
        A2[i][1] = mul2(A2[i][1], both(kLog2e));
        g[i] = in[i] && !same_group ? (int)((c0 + i * CH) / Cg) : 0;
    }
    const float D = mine && p.D ? p.D[cm] : 0.f, bias = mine && p.bias ? p.bias[cm] : 0.f;

    auto token = [&](int b) {
        float x = 0.f, d = 0.f, z = 0.f;
        if (mine) {
            x = Io<T>::ld((const T*)p.x + b * p.x_row + cm);
            d = Io<T>::ld((const T*)p.dt + b * p.dt_row + cm) + bias;
            if (p.z) z = Io<T>::ld((const T*)p.z + b * p.z_row + cm);
        }
        f2 bv[2], cv[2];
        auto states = [&](int gi) {
            const T* bp = (const T*)p.Bm + b * p.b_row + (long long)gi * p.N + n0;
            const T* cp = (const T*)p.Cm + b * p.c_row + (long long)gi * p.N + n0;
            float f[4];
            unpack_quad(ld_quad(bp, PLAIN ? 4 : p.N - n0, PLAIN || p.wide_bc), f);
            bv[0] = pack(f[0], f[1]);
            bv[1] = pack(f[2], f[3]);
            unpack_quad(ld_quad(cp, PLAIN ? 4 : p.N - n0, PLAIN || p.wide_bc), f);
            cv[0] = pack(f[0], f[1]);
            cv[1] = pack(f[2], f[3]);
        };
        if (same_group) states(0);
        if (p.softplus) d = softplus_of(d);
        const float dx = d * x;
        float y[I];
#pragma unroll
        for (int i = 0; i < I; ++i) {
            if (!same_group) states(g[i]);
            const f2 di = both(I == 1 ? d : __shfl_sync(all, d, base + i)), dxi = both(I == 1 ? dx : __shfl_sync(all, dx, base + i));
            h[i][0] = fma2(decay2(di, A2[i][0], tilt_of(mul2(di, A2[i][0]))), h[i][0], mul2(dxi, bv[0]));
            h[i][1] = fma2(decay2(di, A2[i][1], tilt_of(mul2(di, A2[i][1]))), h[i][1], mul2(dxi, bv[1]));
            const float2 s = unpack(fma2(h[i][0], cv[0], mul2(h[i][1], cv[1])));
            y[i] = s.x + s.y;
        }
        // sums over the channel's lanes; four channels are halved over the first four lanes
        float o;
        if constexpr (I == 4) {
            const bool hi = nl & 2, up = nl & 1;
            const float u = (hi ? y[2] : y[0]) + __shfl_xor_sync(all, hi ? y[0] : y[2], 2);
            const float v = (hi ? y[3] : y[1]) + __shfl_xor_sync(all, hi ? y[1] : y[3], 2);
            o = (up ? v : u) + __shfl_xor_sync(all, up ? u : v, 1);
        } else if constexpr (I == 2) {
            const bool up = nl & 1;
            o = (up ? y[1] : y[0]) + __shfl_xor_sync(all, up ? y[0] : y[1], 1);
            o += __shfl_xor_sync(all, o, 2);
        } else {
            o = y[0] + __shfl_xor_sync(all, y[0], 2);
            o += __shfl_xor_sync(all, o, 1);
        }
#pragma unroll
        for (int k = 4; k < NL; k *= 2) o += __shfl_xor_sync(all, o, k);
        if (mine && nl < I) {
            o = fmaf(D, x, o);
            if (p.z) o *= silu(z);
            Io<T>::st((T*)p.y + (long long)b * p.C + cm, o);
        }
    };

    unsigned earlier = 0, later = 0;
    if (idx) {
        if (threadIdx.x < 2) flags[threadIdx.x] = 0;
        __syncthreads();
        for (int b = threadIdx.x; b < p.B; b += kStep) {
            const int s = idx[b];
            for (int r = 0; r < rows; ++r)
                if (b != b0 + r && s == idx[b0 + r]) atomicOr(&flags[b > b0 + r], 1u << r);
        }
        __syncthreads();
        earlier = flags[0];
        later = flags[1];
    }
    for (int r = 0; r < rows; ++r) {
        const int now = slot;
#pragma unroll
        for (int i = 0; i < I; ++i) {
            h[i][0] = next[i][0];
            h[i][1] = next[i][1];
        }
        slot = slot_of(r + 1);
        fetch(slot);                                              // of no use to a row that leaves its token to another
        if (now < 0 || now >= slots || (earlier >> r & 1)) continue;
        token(b0 + r);
        if (later >> r & 1) {
            for (int b = b0 + r + 1; b < p.B; ++b)
                if (idx[b] == now) token(b);
        }
        float* hp = p.h + (long long)now * p.C * p.N;
#pragma unroll
        for (int i = 0; i < I; ++i) {
            if (!in[i]) continue;
            float* to = hp + (at0 + i * at_step);
            if (vec) {
                if (PLAIN || n0 < p.N) *(ulonglong2*)to = make_ulonglong2(h[i][0], h[i][1]);
            } else {
                const float2 u = unpack(h[i][0]), v = unpack(h[i][1]);
                const float f[4] = {u.x, u.y, v.x, v.y};
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (n0 + j < p.N) to[j] = f[j];
            }
        }
    }
}

// ---------------------------------------------------------------------------------------- host
// Two lanes for N <= 8 were no faster than four of which half idle (4 x 2048 x 4096: 324 us forward both).
int lanes_for(int N) { return N <= 16 ? 4 : N <= 32 ? 8 : 16; }

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
    p->nbb = (d->C / d->G + 256 / lanes_for(d->N) - 1) / (256 / lanes_for(d->N));
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

// Pieces of a sequence: as many (32 at most, of 64 tokens at least) as make the call shortest by this
// account, in units of one block's walk over a whole sequence. Blocks run in waves of one for each SM; two
// forward blocks of up to 16 states fit one and then take 1.63 times as long (132 cycles a token, not 81). The
// first pass over pieces costs 0.6 of the main one forward; backward a third, without waves, since its
// blocks are small; joining them takes about 24 tokens' time for each piece, backward 12. Measured at
// 4096 tokens, bf16, N = 16 (us whole, then for these numbers of pieces):
//   forward    64 blocks 178, 4: 144, 10: 135    80 blocks 177, 3: 184, 10: 161   100 blocks 180, 2: 223, 8: 194
//   backward   10 blocks 779, 6: 220, 12: 141    32 blocks 787, 4: 349, 12: 304    50 blocks 798, 2: 598, 8: 439
// Forward a larger number has to gain 3 %, since the account is no better than that.
int pieces_for(const SsmArgs& p, bool bwd, int sms) {
    const long long blocks = (long long)p.S * p.G * (bwd ? p.nbb : p.nb);
    const long long len = p.S > 0 && p.cu ? p.L / p.S : p.L;
    if (blocks >= sms || len < 128) return 1;
    const bool pairs = !bwd && p.N <= 16;
    auto waves = [&](long long n) {
        if (!pairs) return (double)((n + sms - 1) / sms);
        const long long rest = n % (2 * sms);
        return n / (2 * sms) * 1.63 + (rest == 0 ? 0.0 : rest <= sms ? 1.0 : 1.63);
    };
    const int most = (int)(len / 64 < 32 ? len / 64 : 32);
    int best = 1;
    double least = 0.97;
    for (int K = 2; K <= most; ++K) {
        const double all = (double)(K - 1) * blocks / sms;
        const double first = bwd ? 0.33 * (all > 1.0 ? all : 1.0) : 0.6 * waves((K - 1) * blocks);
        const double cost = (waves(K * blocks) + first) / K + (bwd ? 12.0 : 24.0) * K / len;
        if (cost < (bwd ? 0.995 : 0.97) * least) least = cost, best = K;
    }
    return best;
}

// The warps that scan take over registers of the ones that feed (setmaxnreg): the two shares have to be
// what the block was launched with, or the taking warps would wait for good.
template <typename K>
cudaError_t check_registers(K kernel, int threads, int needed) {
    cudaFuncAttributes a;
    const cudaError_t e = cudaFuncGetAttributes(&a, kernel);
    if (e != cudaSuccess) return e;
    return a.numRegs * threads >= needed ? cudaSuccess : cudaErrorInvalidKernelImage;
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
        w.dbc = take((size_t)p.nbb * p.B * p.L * p.G * 8 * lanes_for(p.N));
    }
    w.total = off;
    return w;
}

template <typename F>
void with_lanes(int dtype, int NL, F&& f) {
    auto by = [&](auto t) {
        using T = decltype(t);
        if (NL == 4) f(t, std::integral_constant<int, 4>());
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
    p.K = pieces_for(p, for_backward != 0, device_sm_count());
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
    p.K = pieces_for(p, false, device_sm_count());
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
            const unsigned blocks = cblocks * pieces * p.S;
            if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostSmem);
            if (e == cudaSuccess) kernel<<<blocks, 32 * NL + Feed<NL>::threads, smem, st>>>(p);
        };
        static_assert(sizeof(FwdSmem<T, NL, true>) <= kMostSmem && sizeof(FwdSmem<T, NL, false>) <= kMostSmem, "fits an SM");
        if constexpr (NL == 4) {
            static const cudaError_t first = check_registers(k_ssm_fwd<T, NL, true>, kFwdThreads4, kFwdRegs4);
            static const cudaError_t main = check_registers(k_ssm_fwd<T, NL, false>, kFwdThreads4, kFwdRegs4);
            e = first != cudaSuccess ? first : main;
        }
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
    p.K = pieces_for(p, true, device_sm_count());
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
        static_assert(sizeof(BwdSmem<T, NL>) <= kMostSmem, "fits an SM");
        static const cudaError_t regs = check_registers(k_ssm_bwd<T, NL>, kScan + kFeedB, kScan * kScanRegs + kFeedB * kFeedRegs);
        e = regs;
        if (e != cudaSuccess) return;
        e = cudaFuncSetAttribute(k_ssm_bwd<T, NL>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostSmem);
        if (e != cudaSuccess) return;
        if (p.K > 1) k_ssm_bwd_local<T, NL><<<cblocks * (p.K - 1) * p.S, 32 * NL, 0, st>>>(p);
        k_ssm_bwd<T, NL><<<(unsigned)(p.nbb * p.G) * p.K * p.S, kScan + kFeedB, smem, st>>>(p);
        const long long quads = (long long)p.B * p.L * p.G * 2 * NL;
        if (quads > 0)
            k_ssm_sum_bc<T><<<(unsigned)((quads + 127) / 128), 128, 0, st>>>(p.dbc_part, cu, p.S, p.B, p.L, p.G, p.N, p.nbb,
                                                                           2 * NL, (T*)dBm, (T*)dCm);
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
    if (p.N > kMaxN || p.B > 65535 || (long long)p.C * p.N >= (1 << 30)) return GSPN_ERR_UNSUPPORTED;
    const size_t es = dtype_size(desc->dtype);
    for (const void* q : {x, dt, Bm, Cm, z, (const void*)y})
        if (!aligned_to(q, es)) return GSPN_ERR_ALIGNMENT;
    for (const void* q : {(const void*)A, (const void*)D, (const void*)dt_bias, (const void*)idx, (const void*)h})
        if (!aligned_to(q, 4)) return GSPN_ERR_ALIGNMENT;
    p.x = x; p.dt = dt; p.z = z; p.Bm = Bm; p.Cm = Cm; p.A = A; p.D = D; p.bias = dt_bias; p.h = h; p.y = y;
    p.wide = p.N % 4 == 0 && aligned_to(h, 16) && aligned_to(A, 16);
    p.wide_bc = p.N % 4 == 0 && wide_ok(Bm, p.b_row, 0, es) && wide_ok(Cm, p.c_row, 0, es);
    // Four channels a lane in the plain form (against one: a row of 4096 channels 2.2 us either way, 12 rows 4.8 and
    // 6.2 us, 256 rows 34 and 43); in the general form only where that leaves four blocks for each SM (2000 channels
    // of 24 states: 4 rows 4.3 and 3.2 us, 32 rows 8.7 and 9.8, 256 rows 52 and 61). Rows share a block (and
    // its reading of A) as far as eight remain.
    const int NL = lanes_for(p.N);
    const long long sms = device_sm_count(), wide_blocks = (p.C + 4 * kStep / NL - 1) / (4 * kStep / NL);
    const bool plain = p.G == 1 && p.N == 4 * NL && p.wide && p.wide_bc && p.C % (4 * kStep / NL) == 0;
    const bool four = plain || wide_blocks * p.B >= 4 * sms;
    const long long gx = four ? wide_blocks : (p.C + kStep / NL - 1) / (kStep / NL);
    long long group = gx * p.B / (8 * sms);
    group = group < 1 ? 1 : group > kGroup ? kGroup : group;
    const dim3 grid((unsigned)gx, (unsigned)((p.B + group - 1) / group));
    cudaStream_t st = (cudaStream_t)stream;
    with_lanes(desc->dtype, NL, [&](auto t, auto nl) {
        using T = decltype(t);
        constexpr int N = decltype(nl)::value;
        auto go = [&](auto kernel) { kernel<<<grid, kStep, 0, st>>>(p, idx, slots, (int)group); };
        if (plain) go(k_ssm_step<T, N, 4, true>);
        else if (four) go(k_ssm_step<T, N, 4, false>);
        else go(k_ssm_step<T, N, 1, false>);
    });
    return last_status();
}

}  // extern "C"
