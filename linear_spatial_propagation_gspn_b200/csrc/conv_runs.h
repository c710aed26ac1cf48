// conv_runs.h -- the tokens of a convolution thread's run and the sequences that they lie in. Integer
// arithmetic alone, compiled for the host as well, where the tests walk it over every kind of borders.
#pragma once

#ifdef __CUDACC__
#define GSPN_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define GSPN_HOST_DEVICE inline
#endif

namespace gspn {
namespace seq {

GSPN_HOST_DEVICE int least(int a, int b) { return a < b ? a : b; }
GSPN_HOST_DEVICE int most(int a, int b) { return a < b ? b : a; }

// Rows of L tokens, or, with cu, one row of S sequences side by side.
struct Tokens {
    const int* cu;
    int S, L;
};
GSPN_HOST_DEVICE int border(const Tokens& p, int i) { return least(most(p.cu[i], 0), p.L); }

// A run's tokens [first, end): those from `at` on, `run` of them at most, that lie in a sequence. What lies before
// cu[0] or from cu[S] on belongs to none: no input there is read, nor a state, whose rows are those of the S
// sequences.
struct Run {
    int first, end;
};
GSPN_HOST_DEVICE Run run_at(const Tokens& p, int at, int run) {
    Run r{at, least(at + run, p.L)};
    if (p.cu) {
        r.first = most(r.first, border(p, 0));
        r.end = least(r.end, border(p, p.S));
    }
    return r;
}

// The sequence of a run's token and its bounds; 0 <= q < S whatever cu holds. A token of a run lies before
// cu[S], so the last sequence needs no comparison.
struct Seq {
    int q, start, end;
};
GSPN_HOST_DEVICE void enter(const Tokens& p, Seq& s, int t) {    // moves on to the sequence of t
    while (s.q < p.S - 1 && t >= border(p, s.q + 1)) ++s.q;
    s.start = least(border(p, s.q), t);
    s.end = border(p, s.q + 1);
}
GSPN_HOST_DEVICE Seq find(const Tokens& p, int row, int t) {
    if (!p.cu) return Seq{row, 0, p.L};
    int lo = 0, hi = p.S - 1;                    // first q with t < cu[q + 1]
    while (lo < hi) {
        const int mid = (lo + hi) / 2;
        if (t < border(p, mid + 1)) hi = mid;
        else lo = mid + 1;
    }
    Seq s{lo, 0, 0};
    enter(p, s, t);
    return s;
}

}  // namespace seq
}  // namespace gspn
