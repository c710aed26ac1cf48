// k_conv.cu -- short causal convolution over token sequences, one filter of K taps per channel:
//   u_t = bias + sum_{k<K} w_k x_{t-K+1+k},   y_t = u_t or u_t sigmoid(u_t).
//
// A few operations per element, so memory traffic should bound it: x read and y written once. A thread
// keeps four channels (eight of bf16 took registers that more warps use better) and walks a run of tokens
// with the K - 1 inputs before the present one in registers, so each input is loaded once per run; the
// K - 1 tokens that neighbouring runs share come from the caches.
//
// Measured (B200, bf16, K = 4, silu): forward 8192 x 4096 30.8 us, 4.4 TB/s; 4 x 2048 x 2048 18 us, 3.7 TB/s;
// backward of the latter 36 us, 2.8 TB/s, and 4.5 us for the sums of dw. A silu and its slope cost about as
// many instruction slots (45 % taken) as the traffic costs time.
#include "conv_runs.h"
#include "seq_common.cuh"

namespace gspn {
namespace seq {
namespace {

constexpr int kRunFwd = 32, kRunBwd = 64;   // most tokens of a thread's run, forward and backward
constexpr int kBatch = 4;       // tokens taken together
constexpr int kVB = 4;          // channels of a thread

struct ConvArgs : Tokens {      // cu, L; S: sequences, packed or rows
    int B, C, silu;
    bool wide, wide_w;          // 16-byte aligned vectors of channels; of filters
    const void* x;
    long long x_row, x_tok;
    const float *w, *bias;
    const void *state0, *dy, *dstate;
    void *y, *state, *dx, *dstate0;
    float* part;
    int nvec, run, runs;        // channel vectors; tokens of a run; runs of a row
};

// L consecutive elements (L * sizeof(T) = 8 or 16 bytes when wide), from floats.
template <typename T, int L>
__device__ __forceinline__ void st_ch(T* p, const float (&v)[L], int n, bool wide) {
    if (wide && n >= L) {
        st_lanes<T, L>(p, v);
    } else {
#pragma unroll
        for (int i = 0; i < L; ++i)
            if (i < n) Io<T>::st(p + i, v[i]);
    }
}

// Loads of `P` pairs of channels (n of them exist): as stored, and taken apart.
template <typename T, int P> struct Raw { typedef uint4 type; };
template <> struct Raw<__nv_bfloat16, 2> { typedef uint2 type; };
template <typename T, int P>
__device__ __forceinline__ typename Raw<T, P>::type ld_pairs_raw(const T* p, int n, bool wide) {
    if constexpr (2 * P == Vec<T>::V) return ld_raw<T>(p, n, wide);
    else return ld_quad(p, n, wide);
}
template <typename T, int P>
__device__ __forceinline__ void st_pairs(T* p, const f2 (&v)[P], int n, bool wide) {
    float f[2 * P];
    to_floats(v, f);
    st_ch<T, 2 * P>(p, f, n, wide);
}

// A thread's inputs on their way: tokens in batches of kBatch, S of them. WIDE: through places of its
// own in shared memory (asynchronous copies that hold no registers while they are under way; only the
// thread that copied them reads them, so there is no barrier); otherwise loaded when they are asked for.
template <typename T, int P, bool WIDE, int S> struct Ring {
    typedef typename Raw<T, P>::type R;
    R (*at)[kBatch][128];        // [S][kBatch][thread]
    const T* src;                // the next batch's tokens
    long long step;
    int left, n, put = 0, got = 0;
    const T* now;                // the batch to be taken next (not WIDE)
    __device__ __forceinline__ void issue() {
        if constexpr (WIDE) {
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                if (u < left) {
                    const unsigned to = (unsigned)__cvta_generic_to_shared(&at[put][u][threadIdx.x]);
                    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(to), "l"(src), "n"(sizeof(R)) : "memory");
                }
                src += step;
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
            put = put == S - 1 ? 0 : put + 1;
            left -= kBatch;
        }
    }
    __device__ __forceinline__ void begin(R (*smem)[kBatch][128], const T* p, long long tok, int tokens, int channels) {
        at = smem;
        src = now = p;
        step = tok;
        left = tokens;
        n = channels;
        put = got = 0;
    }
    // Waits for the copies of batches that nobody takes, before their places are filled anew.
    __device__ __forceinline__ void leave() {
        if constexpr (WIDE) asm volatile("cp.async.wait_all;" ::: "memory");
    }
    // Takes the next batch (of the `tokens` that still come) and sends for the one S - 1 behind it. The
    // groups of several rings of a thread have to be issued in turn.
    template <int RINGS> __device__ __forceinline__ void take(R (&r)[kBatch], int tokens) {
        if constexpr (WIDE) {
            asm volatile("cp.async.wait_group %0;" ::"n"((S - 2) * RINGS) : "memory");
#pragma unroll
            for (int u = 0; u < kBatch; ++u) r[u] = at[got][u][threadIdx.x];
            got = got == S - 1 ? 0 : got + 1;
        } else {
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                r[u] = R{};
                if (u < tokens) r[u] = ld_pairs_raw<T, P>(now, n, false);
                now += step;
            }
        }
    }
};

// The K - 1 inputs before token t of sequence s.
template <typename T, int K, int P>
__device__ __forceinline__ void window(const ConvArgs& p, const T* xr, const Seq& s, int t, int c, int n, f2 (&win)[K][P]) {
#pragma unroll
    for (int j = 0; j < K - 1; ++j) {
        const int at = t - (K - 1) + j;
        typename Raw<T, P>::type q{};
        if (at >= s.start) q = ld_pairs_raw<T, P>(xr + at * p.x_tok, n, p.wide);
        else if (p.state0)
            q = ld_pairs_raw<T, P>((const T*)p.state0 + ((long long)s.q * (K - 1) + (K - 1 + at - s.start)) * p.C + c, n, p.wide);
        to_pairs(q, win[j]);
    }
}

// A thread's filters: 2 P K consecutive floats.
template <int K, int P>
__device__ __forceinline__ void load_taps(const ConvArgs& p, int c, int n, f2 (&w)[K][P], f2 (&b)[P]) {
    float f[2 * P * K], bb[2 * P];
    const float* s = p.w + (long long)c * K;
    if (p.wide_w && n >= 2 * P) {
#pragma unroll
        for (int i = 0; i < 2 * P * K; i += 4) {
            const float4 v = *(const float4*)(s + i);
            f[i] = v.x; f[i + 1] = v.y; f[i + 2] = v.z; f[i + 3] = v.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 2 * P * K; ++i) f[i] = i / K < n ? s[i] : 0.f;
    }
#pragma unroll
    for (int i = 0; i < 2 * P; ++i) bb[i] = i < n && p.bias ? p.bias[c + i] : 0.f;
#pragma unroll
    for (int i = 0; i < P; ++i) {
        b[i] = pack(bb[2 * i], bb[2 * i + 1]);
#pragma unroll
        for (int k = 0; k < K; ++k) w[k][i] = pack(f[2 * i * K + k], f[(2 * i + 1) * K + k]);
    }
}

template <typename T, int K> __device__ void last_inputs(const ConvArgs& p, long long id);

// Blocks behind the first `blocks` take the states behind the sequences. Seven blocks an SM by registers for
// bf16 (32.9 -> 31.5 us at 8192 x 4096; eight spilled: 34.9), five for fp32 (seven spilled: 46 us against 27.5).
template <typename T, int K, bool WIDE>
__global__ void __launch_bounds__(128, sizeof(T) == 2 ? 7 : 5) k_conv_fwd(const ConvArgs p, long long blocks) {
    constexpr int P = kVB / 2;
    constexpr int S = 4;
    __shared__ __align__(16) typename Raw<T, P>::type smem[WIDE ? S : 1][kBatch][128];
    if (blockIdx.x >= blocks) {
        last_inputs<T, K>(p, (blockIdx.x - blocks) * (long long)blockDim.x + threadIdx.x);
        return;
    }
    const unsigned id = blockIdx.x * blockDim.x + threadIdx.x;    // under 2^31 (the host lengthens the runs for it)
    const unsigned rr = id / (unsigned)p.nvec, cv = id - rr * p.nvec;
    const int row = (int)(rr / (unsigned)p.runs);
    if (row >= p.B) return;
    const Run r = run_at(p, (int)(rr - row * (unsigned)p.runs) * p.run, p.run);
    int t = r.first;
    const int te = r.end, c = (int)cv * kVB, n = p.C - c;
    if (t >= te) return;
    const T* xr = (const T*)p.x + row * p.x_row + c;
    T* yr = (T*)p.y + (long long)row * p.L * p.C + c;
    typename Raw<T, P>::type raw[kBatch];
    T* py = yr + (long long)t * p.C;
    Ring<T, P, WIDE, S> ring;
    ring.begin(smem, xr + t * p.x_tok, p.x_tok, te - t, n);
#pragma unroll
    for (int k = 0; k < S - 1; ++k) ring.issue();
    f2 w[K][P], b[P], win[K][P];
    load_taps<K, P>(p, c, n, w, b);
    Seq s = find(p, row, t);
    window<T, K, P>(p, xr, s, t, c, n, win);
    auto one = [&](const typename Raw<T, P>::type& q) {
        to_pairs(q, win[K - 1]);
        f2 o[P];
#pragma unroll
        for (int i = 0; i < P; ++i) {
            f2 a = b[i];
#pragma unroll
            for (int k = 0; k < K; ++k) a = fma2(w[k][i], win[k][i], a);
            o[i] = p.silu ? silu2(a) : a;
#pragma unroll
            for (int k = 0; k < K - 1; ++k) win[k][i] = win[k + 1][i];
        }
        st_pairs<T, P>(py, o, WIDE ? 2 * P : n, WIDE || p.wide);
        py += p.C;
    };
    for (; t < te; t += kBatch) {
        ring.template take<1>(raw, te - t);
        ring.issue();
        if (t + kBatch <= te && (!p.cu || t + kBatch <= s.end)) {
#pragma unroll
            for (int u = 0; u < kBatch; ++u) one(raw[u]);
        } else {
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                if (t + u >= te) break;
                if (p.cu && t + u >= s.end) {
                    enter(p, s, t + u);
                    window<T, K, P>(p, xr, s, t + u, c, n, win);
                }
                one(raw[u]);
            }
        }
    }
}

// The last K - 1 inputs of every sequence. Thread = (sequence, channel); it reads all of its channel's
// rows before it writes them, so that state may be state0 (then in a launch of its own, behind the
// one that reads state0).
template <typename T, int K>
__device__ void last_inputs(const ConvArgs& p, long long id) {
    const int c = (int)(id % p.C);
    const long long q = id / p.C;
    if (q >= p.S) return;
    const Span sp = span_of(p.cu, (int)q, p.L);
    T v[K - 1];
#pragma unroll
    for (int j = 0; j < K - 1; ++j) {
        const int at = sp.len - (K - 1) + j;
        if (at >= 0) v[j] = ((const T*)p.x)[sp.row * p.x_row + (sp.first + at) * p.x_tok + c];
        else if (p.state0) v[j] = ((const T*)p.state0)[(q * (K - 1) + K - 1 + at) * p.C + c];
        else v[j] = T(0.f);
    }
#pragma unroll
    for (int j = 0; j < K - 1; ++j) ((T*)p.state)[(q * (K - 1) + j) * p.C + c] = v[j];
}

template <typename T, int K>
__global__ void k_conv_state(const ConvArgs p) {
    last_inputs<T, K>(p, (long long)blockIdx.x * blockDim.x + threadIdx.x);
}

// ------------------------------------------------------------------------------------ backward
//   du_t = dy_t (slope of silu at u_t);  dx_t = sum_k w_k du_{t+K-1-k};  dw_k = sum_t du_t x_{t-K+1+k}
// A thread walks a run forward, forming u_t again from the inputs, with the K sums of dx that du_t
// adds to in registers: after token t the one of t - K + 1 is complete. It goes K - 1 tokens past
// its run for its last sums. A block is 32 channel vectors (4 channels) x 4 runs; it takes several
// runs in turn and keeps its sums of dw and dbias until the end; k_conv_sum adds the blocks in order.
constexpr int kRows = 4;

template <typename T, int K, bool WIDE>
__global__ void __launch_bounds__(128) k_conv_bwd(const ConvArgs p) {
    constexpr int P = kVB / 2;
    typedef typename Raw<T, P>::type R;
    constexpr int S = sizeof(R) == 8 ? 4 : 2;                     // two rings of fp32 in 48 KB
    __shared__ __align__(16) R smem[2][WIDE ? S : 1][kBatch][128];
    __shared__ __align__(16) float red[kRows][K + 1][32 * kVB];
    const int lane = threadIdx.x & 31, grp = threadIdx.x >> 5;
    const int c = (blockIdx.x * 32 + lane) * kVB, n = p.C - c;
    const f2 zero = pack(0.f, 0.f);
    f2 w[K][P], b[P];
    // the thread's sums of dw and dbias over its runs: its own places, so no barrier is needed
    auto total = [&](int k) -> ulonglong2& { return *(ulonglong2*)&red[grp][k][lane * kVB]; };
#pragma unroll
    for (int k = 0; k <= K; ++k) total(k) = make_ulonglong2(zero, zero);
    if (n > 0) {
        load_taps<K, P>(p, c, n, w, b);
        const long long all = (long long)p.B * p.runs;
        for (long long rr = (long long)blockIdx.y * kRows + grp; rr < all; rr += (long long)gridDim.y * kRows) {
            const int row = (int)(rr / p.runs);
            // tb: where the next run begins (not run.end, which could not be formed anew and made the compiler spill)
            const int at = (int)(rr % p.runs) * p.run, tb = min(at + p.run, p.L);
            const Run run = run_at(p, at, p.run);
            const int ta = run.first;
            if (ta >= run.end) continue;
            const T* xr = (const T*)p.x + row * p.x_row + c;
            const T* gr = (const T*)p.dy + (long long)row * p.L * p.C + c;
            T* dr = (T*)p.dx + (long long)row * p.L * p.C + c;
            Seq s = find(p, row, ta);
            const int stop = min(tb + K - 1, p.cu ? border(p, p.S) : p.L);
            R xs[kBatch], gs[kBatch];
            T* pd = dr + (long long)(ta - (K - 1)) * p.C;         // where token t - (K - 1) goes
            Ring<T, P, WIDE, S> rx, rg;
            rx.begin(smem[0], xr + ta * p.x_tok, p.x_tok, stop - ta, n);
            rg.begin(smem[1], gr + (long long)ta * p.C, p.C, stop - ta, n);
#pragma unroll
            for (int k = 0; k < S - 1; ++k) {
                rx.issue();
                rg.issue();
            }
            f2 win[K][P], acc[K][P], run_dw[K][P], run_db[P];
            window<T, K, P>(p, xr, s, ta, c, n, win);
#pragma unroll
            for (int i = 0; i < P; ++i) {
                run_db[i] = zero;
#pragma unroll
                for (int k = 0; k < K; ++k) acc[k][i] = run_dw[k][i] = zero;
            }
            // writes token `at`'s sum, held in v, if the run owns it
            auto put = [&](int at, f2 (&v)[P]) {
                if (at < ta || at < s.start || at >= tb) return;
                const int m = at - s.end + K - 1;                 // its row in the state behind the sequence
                if (m >= 0 && p.dstate) {
                    f2 d[P];
                    to_pairs(ld_pairs_raw<T, P>((const T*)p.dstate + ((long long)s.q * (K - 1) + m) * p.C + c, n, p.wide), d);
#pragma unroll
                    for (int i = 0; i < P; ++i) v[i] = add2(v[i], d[i]);
                }
                st_pairs<T, P>(dr + (long long)at * p.C, v, n, p.wide);
            };
            // token t: its du into the sums of dx, and of dw if the run owns it
            auto one = [&](int u, bool own) {
                to_pairs(xs[u], win[K - 1]);
                f2 g[P];
                to_pairs(gs[u], g);
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    f2 du = g[i];
                    if (p.silu) {
                        f2 a = b[i];
#pragma unroll
                        for (int k = 0; k < K; ++k) a = fma2(w[k][i], win[k][i], a);
                        du = mul2(du, silu_slope2(a));
                    }
#pragma unroll
                    for (int k = 0; k < K; ++k) acc[k][i] = fma2(w[k][i], du, acc[k][i]);
                    if (own) {
                        run_db[i] = add2(run_db[i], du);
#pragma unroll
                        for (int k = 0; k < K; ++k) run_dw[k][i] = fma2(du, win[k][i], run_dw[k][i]);
                    }
                }
            };
            auto shift = [&] {
#pragma unroll
                for (int i = 0; i < P; ++i) {
#pragma unroll
                    for (int k = 0; k < K - 1; ++k) {
                        acc[k][i] = acc[k + 1][i];
                        win[k][i] = win[k + 1][i];
                    }
                    acc[K - 1][i] = zero;
                }
            };
            bool open = true;
            for (int t = ta; open && t < stop; t += kBatch) {
                rx.template take<2>(xs, stop - t);
                rg.template take<2>(gs, stop - t);
                rx.issue();
                rg.issue();
                if (t >= max(ta, s.start) + K - 1 && t + kBatch <= min(tb, s.end)) {
                    // all within the run and one sequence: every token completes one that the run owns
#pragma unroll
                    for (int u = 0; u < kBatch; ++u) {
                        one(u, true);
                        st_pairs<T, P>(pd, acc[0], WIDE ? 2 * P : n, WIDE || p.wide);
                        pd += p.C;
                        shift();
                    }
                    continue;
                }
                pd += (long long)kBatch * p.C;
#pragma unroll
                for (int u = 0; u < kBatch; ++u) {
                    const int tt = t + u;
                    if (!open || tt >= stop) break;
                    if (tt >= s.end) {                            // the sequence is over: its last sums are complete
#pragma unroll
                        for (int k = 0; k < K - 1; ++k) put(tt - (K - 1) + k, acc[k]);
                        if (tt >= tb) {
                            open = false;
                            break;
                        }
                        enter(p, s, tt);
                        window<T, K, P>(p, xr, s, tt, c, n, win);
#pragma unroll
                        for (int k = 0; k < K; ++k)
#pragma unroll
                            for (int i = 0; i < P; ++i) acc[k][i] = zero;
                    }
                    one(u, tt < tb);
                    put(tt - (K - 1), acc[0]);
                    shift();
                }
            }
            rx.leave();                                           // an early end leaves copies to places that the next run fills
            if (open && stop == s.end) {                          // ended with the sequence, inside the loop's last batch
#pragma unroll
                for (int k = 0; k < K - 1; ++k) put(stop - (K - 1) + k, acc[k]);
            }
#pragma unroll
            for (int k = 0; k <= K; ++k) {
                ulonglong2& s = total(k);
                s = make_ulonglong2(add2(s.x, k < K ? run_dw[k < K ? k : 0][0] : run_db[0]),
                                    add2(s.y, k < K ? run_dw[k < K ? k : 0][1] : run_db[1]));
            }
        }
    }
    __syncthreads();
    for (int e = threadIdx.x; e < (K + 1) * 32 * kVB; e += blockDim.x) {
        const int k = e / (32 * kVB), cc = e % (32 * kVB);
        float v = 0.f;
#pragma unroll
        for (int g = 0; g < kRows; ++g) v += red[g][k][cc];
        const int ch = blockIdx.x * 32 * kVB + cc;
        if (ch < p.C) p.part[((long long)blockIdx.y * (K + 1) + k) * p.C + ch] = v;
    }
}

// dw and dbias: the blocks' sums, 32 (tap or bias, channel) pairs a block, each by eight threads that take
// every eighth block; their sums are added in order.
__global__ void k_conv_sum(const float* part, int blocks, int C, int K, float* dw, float* dbias) {
    __shared__ float red[8][32];
    const int i = blockIdx.x * 32 + threadIdx.x, n = (K + 1) * C;
    float v = 0.f;
    if (i < n) {
#pragma unroll 4
        for (int g = threadIdx.y; g < blocks; g += 8) v += part[(long long)g * n + i];
    }
    red[threadIdx.y][threadIdx.x] = v;
    __syncthreads();
    if (threadIdx.y != 0 || i >= n) return;
    v = 0.f;
#pragma unroll
    for (int g = 0; g < 8; ++g) v += red[g][threadIdx.x];
    const int k = i / C, c = i % C;
    if (k < K) dw[(long long)c * K + k] = v;
    else if (dbias) dbias[c] = v;
}

// Gradient of state0: state row j stands K-1-j places before the sequence and meets u_i, i <= j,
// through tap j - i; rows that are still in the state behind a short sequence take dstate as well.
// Thread = (sequence, channel).
template <typename T, int K>
__global__ void k_conv_dstate(const ConvArgs p) {
    const long long id = (long long)blockIdx.x * blockDim.x + threadIdx.x;
    const int c = (int)(id % p.C);
    const long long q = id / p.C;
    if (q >= p.S) return;
    const Span sp = span_of(p.cu, (int)q, p.L);
    const T* xr = (const T*)p.x + sp.row * p.x_row + c;
    float w[K], line[2 * (K - 1)], out[K - 1];
#pragma unroll
    for (int k = 0; k < K; ++k) w[k] = p.w[(long long)c * K + k];
#pragma unroll
    for (int j = 0; j < K - 1; ++j) {
        line[j] = Io<T>::ld((const T*)p.state0 + (q * (K - 1) + j) * p.C + c);
        line[K - 1 + j] = j < sp.len ? Io<T>::ld(xr + (sp.first + j) * p.x_tok) : 0.f;
        out[j] = 0.f;
        const int m = j - sp.len;
        if (p.dstate && m >= 0) out[j] = Io<T>::ld((const T*)p.dstate + (q * (K - 1) + m) * p.C + c);
    }
#pragma unroll
    for (int i = 0; i < K - 1; ++i) {
        if (i < sp.len) {
            float du = Io<T>::ld((const T*)p.dy + ((long long)sp.row * p.L + sp.first + i) * p.C + c);
            if (p.silu) {
                float a = p.bias ? p.bias[c] : 0.f;
#pragma unroll
                for (int k = 0; k < K; ++k) a = fmaf(w[k], line[i + k], a);
                du *= silu_slope(a);
            }
#pragma unroll
            for (int j = i; j < K - 1; ++j) out[j] = fmaf(w[j - i], du, out[j]);
        }
    }
#pragma unroll
    for (int j = 0; j < K - 1; ++j) Io<T>::st((T*)p.dstate0 + (q * (K - 1) + j) * p.C + c, out[j]);
}

// ----------------------------------------------------------------------------------- one token
// Thread = four channels of the block's `group` rows, one after the other, with their filters read once
// and the next row's state fetched ahead. Rows that name the slot of an earlier row leave their token to
// that row, which takes them in order.
constexpr int kGroup = 8;

template <typename T, int K>
__global__ void __launch_bounds__(128) k_conv_step(const ConvArgs p, const int* idx, int slots, int group) {
    constexpr int P = kVB / 2;
    typedef typename Raw<T, P>::type R;
    __shared__ unsigned flags[2];                                 // rows of the group with an earlier, a later row of their slot
    const int b0 = blockIdx.y * group, rows = min(group, p.B - b0);
    const int c = (blockIdx.x * blockDim.x + threadIdx.x) * kVB, n = p.C - c;   // n <= 0: no channels, for the barriers only
    auto slot_of = [&](int r) { return r < rows ? (idx ? idx[b0 + r] : b0 + r) : -1; };
    R win[K], next[K];
    auto fetch = [&](int r, int slot) {
        if (slot < 0 || slot >= slots || n <= 0) return;
        const T* st = (const T*)p.state + (long long)slot * (K - 1) * p.C + c;
#pragma unroll
        for (int j = 0; j < K - 1; ++j) next[j] = ld_pairs_raw<T, P>(st + (long long)j * p.C, n, p.wide);
        next[K - 1] = ld_pairs_raw<T, P>((const T*)p.x + (b0 + r) * p.x_row + c, n, p.wide);
    };
    int slot = slot_of(0);
    fetch(0, slot);
    f2 w[K][P], bias[P];
    if (n > 0) load_taps<K, P>(p, c, n, w, bias);
    unsigned earlier = 0, later = 0;
    if (idx) {
        if (threadIdx.x < 2) flags[threadIdx.x] = 0;
        __syncthreads();
        for (int b = threadIdx.x; b < p.B; b += blockDim.x) {
            const int s = idx[b];
            for (int r = 0; r < rows; ++r)
                if (b != b0 + r && s == idx[b0 + r]) atomicOr(&flags[b > b0 + r], 1u << r);
        }
        __syncthreads();
        earlier = flags[0];
        later = flags[1];
    }
    if (n <= 0) return;
    auto token = [&](int b) {
        f2 o[P];
#pragma unroll
        for (int i = 0; i < P; ++i) o[i] = bias[i];
#pragma unroll
        for (int k = 0; k < K; ++k) {
            f2 v[P];
            to_pairs(win[k], v);
#pragma unroll
            for (int i = 0; i < P; ++i) o[i] = fma2(w[k][i], v[i], o[i]);
        }
        if (p.silu) {
#pragma unroll
            for (int i = 0; i < P; ++i) o[i] = silu2(o[i]);
        }
        st_pairs<T, P>((T*)p.y + (long long)b * p.C + c, o, n, p.wide);
    };
    for (int r = 0; r < rows; ++r) {
        const int now = slot;
#pragma unroll
        for (int k = 0; k < K; ++k) win[k] = next[k];
        slot = slot_of(r + 1);
        fetch(r + 1, slot);                                       // of no use to a row that leaves its token to another
        if (now < 0 || now >= slots || (earlier >> r & 1)) continue;
        token(b0 + r);
        if (later >> r & 1) {
            for (int b = b0 + r + 1; b < p.B; ++b) {
                if (idx[b] != now) continue;
#pragma unroll
                for (int k = 0; k < K - 1; ++k) win[k] = win[k + 1];
                win[K - 1] = ld_pairs_raw<T, P>((const T*)p.x + b * p.x_row + c, n, p.wide);
                token(b);
            }
        }
        T* st = (T*)p.state + (long long)now * (K - 1) * p.C + c;
#pragma unroll
        for (int j = 0; j < K - 1; ++j) {
            if (p.wide && n >= kVB) {
                *(R*)(st + (long long)j * p.C) = win[j + 1];
            } else {
                float f[kVB];
                unpack_quad(win[j + 1], f);
                st_quad<T>(st + (long long)j * p.C, f, n, false);
            }
        }
    }
}

// ---------------------------------------------------------------------------------------- host
bool make_args(const gspn_conv_desc* d, ConvArgs* p) {
    if (!d) return false;
    if (d->B < 1 || d->L < 0 || d->C < 1 || d->K < 2 || d->K > 4 || d->S < 0 || !dtype_ok(d->dtype)) return false;
    if (d->silu != 0 && d->silu != 1) return false;
    if (d->S > 0 && d->B != 1) return false;
    if (d->x_row < 0 || d->x_tok < 0) return false;
    *p = ConvArgs{};
    p->B = d->B; p->L = d->L; p->C = d->C; p->silu = d->silu;
    p->S = d->S > 0 ? d->S : d->B;
    p->x_row = d->x_row; p->x_tok = d->x_tok;
    return true;
}
bool fits(const gspn_conv_desc& d) {
    const long long seqs = d.S > 0 ? d.S : d.B;
    return d.L <= (1 << 30) && (long long)d.B * d.L <= (1LL << 31) - 1 && (long long)d.C * (d.K + 1) < (1LL << 30) &&
           (long long)d.B * d.L / 4 * d.C < (1LL << 36) && seqs * d.C < (1LL << 36);
}
// Tokens of a run: `most`, halved while fewer than 192 threads would be there for each SM (`lines` threads
// side by side). Short runs read K - 1 inputs and the filters more often: 2048 tokens of 1024 channels
// took 6.2 us in runs of 16 and 8.3 in runs of 4.
int run_for(long long lines, int L, int most) {
    int run = most;
    while (run > kBatch && lines * ((L + run - 1) / run) < 192LL * device_sm_count()) run /= 2;
    return run;
}
int run_bwd(const gspn_conv_desc& d) { return run_for((long long)d.B * ((d.C + kVB - 1) / kVB), d.L, kRunBwd); }
// Blocks along the tokens of the backward pass: enough to fill the SMs eight times, no more than there
// are groups of runs.
int bwd_blocks(const gspn_conv_desc& d) {
    const long long gx = (d.C + 32 * kVB - 1) / (32 * kVB);
    const int run = run_bwd(d);
    const long long groups = ((long long)d.B * ((d.L + run - 1) / run) + kRows - 1) / kRows;
    long long gy = (8LL * device_sm_count() + gx - 1) / gx;
    gy = gy < groups ? gy : groups;
    gy = gy < 65535 ? gy : 65535;
    return gy > 0 ? (int)gy : 1;
}

template <typename F>
void with_taps(int dtype, int K, F&& f) {
    auto by = [&](auto t) {
        if (K == 2) f(t, std::integral_constant<int, 2>());
        else if (K == 3) f(t, std::integral_constant<int, 3>());
        else f(t, std::integral_constant<int, 4>());
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

size_t gspn_conv_workspace_size(const gspn_conv_desc* desc, int for_backward) {
    ConvArgs p;
    if (!make_args(desc, &p) || !fits(*desc)) return 0;
    if (!for_backward) return 256;
    return 256 + align256((size_t)bwd_blocks(*desc) * (desc->K + 1) * desc->C * sizeof(float));
}

gspn_status gspn_conv_forward(const gspn_conv_desc* desc, const void* x, const float* w, const float* bias,
                              const int* cu, const void* state0, void* y, void* state, void* stream) {
    ConvArgs p;
    if (!make_args(desc, &p)) return GSPN_ERR_INVALID_ARG;
    if ((desc->S > 0) != (cu != nullptr) || !w || (p.L > 0 && (!x || !y))) return GSPN_ERR_INVALID_ARG;
    if (!fits(*desc)) return GSPN_ERR_UNSUPPORTED;
    const size_t es = dtype_size(desc->dtype);
    for (const void* q : {x, state0, (const void*)y, (const void*)state})
        if (!aligned_to(q, es)) return GSPN_ERR_ALIGNMENT;
    for (const void* q : {(const void*)w, (const void*)bias, (const void*)cu})
        if (!aligned_to(q, 4)) return GSPN_ERR_ALIGNMENT;
    p.x = x; p.w = w; p.bias = bias; p.cu = cu; p.state0 = state0; p.y = y; p.state = state;
    p.wide = (p.C * es) % 16 == 0 && wide_ok(x, p.x_row, p.x_tok, es) && aligned_to(y, 16) && aligned_to(state0, 16);
    p.wide_w = aligned_to(w, 16);
    p.nvec = (p.C + kVB - 1) / kVB;
    p.run = run_for((long long)p.B * p.nvec, p.L, kRunFwd);
    while ((long long)p.B * ((p.L + p.run - 1) / p.run) * p.nvec >= (1LL << 31) - 128 && p.run < p.L) p.run *= 2;
    p.runs = (p.L + p.run - 1) / p.run;
    const long long total = (long long)p.B * p.runs * p.nvec;
    if (total >= (1LL << 31) - 128) return GSPN_ERR_UNSUPPORTED;
    cudaStream_t st = (cudaStream_t)stream;
    with_taps(desc->dtype, desc->K, [&](auto t, auto k) {
        using T = decltype(t);
        constexpr int K = decltype(k)::value;
        const long long blocks = (total + 127) / 128, behind = state ? ((long long)p.S * p.C + 127) / 128 : 0;
        const bool apart = state == state0;                       // no thread of this launch may still read state0
        if (blocks + (apart ? 0 : behind) > 0)
            p.wide ? k_conv_fwd<T, K, true><<<(unsigned)(blocks + (apart ? 0 : behind)), 128, 0, st>>>(p, blocks)
                   : k_conv_fwd<T, K, false><<<(unsigned)(blocks + (apart ? 0 : behind)), 128, 0, st>>>(p, blocks);
        if (apart && behind > 0) k_conv_state<T, K><<<(unsigned)behind, 128, 0, st>>>(p);
    });
    return last_status();
}

gspn_status gspn_conv_backward(const gspn_conv_desc* desc, const void* x, const float* w, const float* bias,
                               const int* cu, const void* state0, const void* dy, const void* dstate, void* dx,
                               float* dw, float* dbias, void* dstate0, void* ws, size_t ws_bytes, void* stream) {
    ConvArgs p;
    if (!make_args(desc, &p)) return GSPN_ERR_INVALID_ARG;
    if ((desc->S > 0) != (cu != nullptr) || !w || !dw || !ws) return GSPN_ERR_INVALID_ARG;
    if (p.L > 0 && (!x || !dy || !dx)) return GSPN_ERR_INVALID_ARG;
    if (dstate0 && !state0) return GSPN_ERR_INVALID_ARG;
    if (!fits(*desc)) return GSPN_ERR_UNSUPPORTED;
    const size_t es = dtype_size(desc->dtype);
    for (const void* q : {x, state0, dy, dstate, (const void*)dx, (const void*)dstate0})
        if (!aligned_to(q, es)) return GSPN_ERR_ALIGNMENT;
    for (const void* q : {(const void*)w, (const void*)bias, (const void*)cu, (const void*)dw, (const void*)dbias})
        if (!aligned_to(q, 4)) return GSPN_ERR_ALIGNMENT;
    if (!aligned_to(ws, 16)) return GSPN_ERR_ALIGNMENT;
    if (ws_bytes < gspn_conv_workspace_size(desc, 1)) return GSPN_ERR_WORKSPACE;
    p.x = x; p.w = w; p.bias = bias; p.cu = cu; p.state0 = state0; p.dy = dy; p.dstate = dstate; p.dx = dx;
    p.dstate0 = dstate0;
    p.part = (float*)((char*)ws + 256);
    p.wide = (p.C * es) % 16 == 0 && wide_ok(x, p.x_row, p.x_tok, es) && aligned_to(dy, 16) && aligned_to(dx, 16) &&
             aligned_to(state0, 16) && aligned_to(dstate, 16);
    p.wide_w = aligned_to(w, 16);
    p.run = run_bwd(*desc);
    p.runs = (p.L + p.run - 1) / p.run;
    const int gy = bwd_blocks(*desc);
    cudaStream_t st = (cudaStream_t)stream;
    with_taps(desc->dtype, desc->K, [&](auto t, auto k) {
        using T = decltype(t);
        constexpr int K = decltype(k)::value;
        const dim3 grid((p.C + 32 * kVB - 1) / (32 * kVB), gy);
        p.wide ? k_conv_bwd<T, K, true><<<grid, 128, 0, st>>>(p) : k_conv_bwd<T, K, false><<<grid, 128, 0, st>>>(p);
        k_conv_sum<<<((K + 1) * p.C + 31) / 32, dim3(32, 8), 0, st>>>(p.part, gy, p.C, K, dw, dbias);
        if (dstate0) {
            const long long n = (long long)p.S * p.C;
            k_conv_dstate<T, K><<<(unsigned)((n + 127) / 128), 128, 0, st>>>(p);
        }
    });
    return last_status();
}

gspn_status gspn_conv_step(const gspn_conv_desc* desc, const void* x, const float* w, const float* bias,
                           const int* idx, int slots, void* state, void* y, void* stream) {
    ConvArgs p;
    if (!make_args(desc, &p) || desc->L != 1 || desc->S != 0 || slots < 1) return GSPN_ERR_INVALID_ARG;
    if (!x || !w || !state || !y || (!idx && slots < p.B)) return GSPN_ERR_INVALID_ARG;
    if (!fits(*desc) || p.B > 65535) return GSPN_ERR_UNSUPPORTED;
    const size_t es = dtype_size(desc->dtype);
    for (const void* q : {x, (const void*)state, (const void*)y})
        if (!aligned_to(q, es)) return GSPN_ERR_ALIGNMENT;
    for (const void* q : {(const void*)w, (const void*)bias, (const void*)idx})
        if (!aligned_to(q, 4)) return GSPN_ERR_ALIGNMENT;
    p.x = x; p.w = w; p.bias = bias; p.y = y; p.state = state;
    p.wide = (p.C * es) % 16 == 0 && wide_ok(x, p.x_row, 0, es) && aligned_to(y, 16) && aligned_to(state, 16);
    p.wide_w = aligned_to(w, 16);
    // rows share a block (and its filters) as far as four blocks remain for each SM
    const long long gx = (p.C + 128 * kVB - 1) / (128 * kVB);
    long long group = gx * p.B / (4LL * device_sm_count());
    group = group < 1 ? 1 : group > kGroup ? kGroup : group;
    const dim3 grid((unsigned)gx, (unsigned)((p.B + group - 1) / group));
    cudaStream_t st = (cudaStream_t)stream;
    with_taps(desc->dtype, desc->K, [&](auto t, auto k) {
        using T = decltype(t);
        constexpr int K = decltype(k)::value;
        k_conv_step<T, K><<<grid, 128, 0, st>>>(p, idx, slots, (int)group);
    });
    return last_status();
}

}  // extern "C"
