// win_geom.cuh -- which keys a row of the sliding-window attention sees, and
// the tile ranges that follow from it (device side).
#pragma once

#include <cuda_runtime.h>

namespace psa {
namespace win {

// n / d for 0 <= n < 2^31 by a multiplication (Granlund and Montgomery): with
// 2^(s-1) < d <= 2^s and m = ceil(2^(31+s) / d), n / d = floor(n m / 2^(31+s)).
// Every warp of a persistent kernel takes an item's number apart on its way to it.
struct FastDiv {
    unsigned d, m;
    int s;                                           // bits beyond 32
};
inline FastDiv fast_div(unsigned d) {
    int s = 0;
    while ((1ull << s) < d) ++s;
    if (s == 0) return FastDiv{1, 0, 0};
    return FastDiv{d, (unsigned)(((1ull << (31 + s)) + d - 1) / d), s - 1};
}
__device__ __forceinline__ int divide(int n, const FastDiv& f) {
    return f.d == 1 ? n : (int)(__umulhi((unsigned)n, f.m) >> f.s);
}

// Lengths of one sequence; row i sits at position i + off.
struct Seq {
    int ql, kl, off;
};
__device__ __forceinline__ Seq load_seq(const int* q_lens, const int* kv_lens, int b, int Nq, int Nk) {
    Seq s;
    s.ql = q_lens ? min(max(__ldcg(q_lens + b), 0), Nq) : Nq;
    s.kl = kv_lens ? min(max(__ldcg(kv_lens + b), 0), Nk) : Nk;
    s.off = s.kl - s.ql;
    return s;
}

// Key tiles of BK keys that rows [i0, i1) (i1 <= ql) see: tile indexes
// 0 .. n_sink-1 and lo .. hi (hi < lo: none), n_sink <= lo.
struct KeyTiles {
    int n_sink, lo, hi;
    __device__ __forceinline__ int count() const { return n_sink + (hi >= lo ? hi - lo + 1 : 0); }
    __device__ __forceinline__ int tile(int t) const { return t < n_sink ? t : lo + (t - n_sink); }
};
template <int BK>
__device__ __forceinline__ KeyTiles key_tiles(const Seq& s, int i0, int i1, int window, int sinks) {
    KeyTiles t{0, 0, -1};
    const int p1 = i1 - 1 + s.off;
    if (i1 <= i0 || p1 < 0) return t;
    const int low = max(i0 + s.off - window + 1, 0);
    t.lo = low / BK;
    t.hi = p1 / BK;
    t.n_sink = min((min(sinks, low) + BK - 1) / BK, t.lo);
    return t;
}

// Rows that see some key of the tile [j0, j0 + BK): positions p0 <= p < p1,
// clipped to existing rows.  `near_only`: only up to a window behind the tile
// (the rest are the far chunks).
struct RowRange {
    int i0, i1;
};
__device__ __forceinline__ RowRange rows_of_tile(const Seq& s, int j0, int BK, int window, int sinks, bool near_only) {
    const bool all = j0 < sinks && !near_only;
    const int p1 = all ? s.kl : min((long long)s.kl, (long long)j0 + BK + window - 1);
    RowRange r{max(j0 - s.off, 0), min(p1 - s.off, s.ql)};
    if (j0 >= s.kl || r.i1 < r.i0) r.i1 = r.i0;
    return r;
}
// Rows of far chunk c of a tile with sinks.
__device__ __forceinline__ RowRange rows_of_far(const Seq& s, int j0, int BK, int window, int far_rows, int c) {
    const long long p0 = (long long)j0 + BK + window - 1 + (long long)c * far_rows;
    RowRange r{0, 0};
    if (p0 >= s.kl || j0 >= s.kl) return r;
    r.i0 = max((int)p0 - s.off, 0);
    r.i1 = min((int)min((long long)s.kl, p0 + far_rows) - s.off, s.ql);
    if (r.i1 < r.i0) r.i1 = r.i0;
    return r;
}

}  // namespace win
}  // namespace psa
