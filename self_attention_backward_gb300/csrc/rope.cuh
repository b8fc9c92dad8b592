// rope.cuh -- what the rotation and the cache's writes share: a plan's angles, 16-byte
// units, groups of tokens and heads.
#pragma once

#include <cuda_bf16.h>

#include <algorithm>
#include <string>

#include "common.cuh"
#include "win_geom.cuh"
#include "win_internal.h"

namespace psa {
namespace win {
namespace {

constexpr int kT = 256;

// Layout of a rotation, in pairs and features.
struct Plan {
    int d, n, interleaved;                       // head_dim, pairs, pairing
    unsigned long long turn[PSA_ROPE_MAX_PAIRS];
    unsigned char axis[PSA_ROPE_MAX_PAIRS];
};

struct Pos {
    const int* p;
    long long axis, batch;
};

__device__ __forceinline__ float2 cos_sin(const Plan& pl, int i, int p, float sign) {
    const unsigned long long t = (unsigned long long)(long long)p * pl.turn[i] + 0x80000000ull;
    float s, c;
    sincospif((float)(int)(t >> 32) * 0x1p-31f, &s, &c);
    return make_float2(c, s * sign);
}
__device__ __forceinline__ int load_pos(const Plan& pl, const Pos& pos, int i, int b, long long n) {
    return __ldg(pos.p + pl.axis[i] * pos.axis + b * pos.batch + n);
}

template <typename T>
constexpr int VEC = 16 / sizeof(T);

template <typename T>
__device__ __forceinline__ void unpack(const uint4& u, float (&x)[VEC<T>]) {
    if constexpr (sizeof(T) == 4) {
        x[0] = __uint_as_float(u.x), x[1] = __uint_as_float(u.y), x[2] = __uint_as_float(u.z), x[3] = __uint_as_float(u.w);
    } else {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w[e]));
            x[2 * e] = f.x, x[2 * e + 1] = f.y;
        }
    }
}
template <typename T>
__device__ __forceinline__ uint4 pack(const float (&x)[VEC<T>]) {
    if constexpr (sizeof(T) == 4) {
        return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
    } else {
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * e], x[2 * e + 1]);
            w[e] = *reinterpret_cast<const uint32_t*>(&h);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// Where a thread's row lies: strides of heads and rows in 32 bits (larger ones take
// the kernel for any strides).
template <typename T>
__device__ __forceinline__ T* row_at(const void* base, long long sB, long long sH, long long sN, int b, int h, int n) {
    return static_cast<T*>(const_cast<void*>(base)) + b * sB + (long long)h * (int)sH + (long long)n * (int)sN;
}

// The groups: TN tokens of a sequence and hper heads, one row per thread at most
// (TN * hper * units <= kT), one angle per thread at most (TN * pairs <= kT).
struct Work {
    int N, H, TN, hper, nb, ny, groups;           // nb, ny: token groups per sequence, head groups
    FastDiv by_nb, by_ny, by_h, by_last, by_u, by_tn;
};
struct Group {
    int b, n0, nt, hb, nh;
};
__device__ __forceinline__ Group group_of(const Work& w, int g) {
    const int x = divide(g, w.by_ny), y = g - x * w.ny;
    Group r;
    r.b = divide(x, w.by_nb);
    r.n0 = (x - r.b * w.nb) * w.TN;
    r.nt = min(w.TN, w.N - r.n0);
    r.hb = y * w.hper;
    r.nh = min(w.hper, w.H - r.hb);
    return r;
}

// The rows of an append that stay, of sequence b: x < early (the sinks among them) and those
// no newer row of the call overwrites; groups count through these.
struct Kept {
    int b = -1, st = 0, n = 0, early = 0, skip = 0;
    __device__ __forceinline__ void of(const int* start, const int* n_new, int to, int T, int sinks, int ring) {
        if (to == b) return;
        b = to;
        st = __ldg(start + b);
        n = n_new ? min(max(__ldg(n_new + b), 0), T) : T;
        if (st < 0 || st - 1 > 0x7fffffff - n) n = 0;
        early = min(max(sinks - st, 0), n);
        skip = max(n - ring - early, 0);
    }
    __device__ __forceinline__ int row(int x) const { return x < early ? x : x + skip; }
};
// The input rows that an append takes, by index; an index out of range takes none.
struct Picked {
    const int* rows;
    long long stride;
    int n;
    __device__ __forceinline__ bool row(int b, int& x) const {
        x = __ldg(rows + b * stride + x);
        return (unsigned)x < (unsigned)n;
    }
};

// ---------------------------------------------------------------- host
inline Plan dev_plan(const psa_rope_plan* p, int d) {
    Plan pl{};
    pl.d = d;
    if (!p) return pl;                           // no pairs: everything is copied
    pl.n = p->rot_dim / 2;
    pl.interleaved = p->interleaved;
    for (int i = 0; i < pl.n; ++i) pl.turn[i] = p->turn[i], pl.axis[i] = p->axis[i];
    return pl;
}

inline bool aligned(const void* p, int esize, long long a, long long b, long long c) {
    const long long w = 16 / esize;
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && a % w == 0 && b % w == 0 && c % w == 0;
}
// by 16-byte units: aligned, adjacent features, 32-bit head and row strides
inline bool view_ok(const View& v, int esize) {
    return v.sJ == 1 && v.sH <= 0x7fffffffll && v.sN <= 0x7fffffffll && aligned(v.base, esize, v.sB, v.sH, v.sN);
}

inline int launched(const char* what, std::string* err) {
    const cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) return PSA_OK;
    *err = std::string(what) + ": " + cudaGetErrorString(e);
    return PSA_ERR_CUDA;
}
inline int too_large(std::string* err) {
    *err = "grid too large";
    return PSA_ERR_UNSUPPORTED;
}

// Groups of H heads of N tokens in B sequences, `per` units a row, n pairs: as many
// heads as fit, then tokens (their angles serve all heads), but groups enough for two
// blocks on each of 152 SMs where there are rows enough for that.
inline bool work_for(int B, int N, int H, int per, int n, Work* out) {
    const int rows = kT / per;
    Work w{};
    w.N = N, w.H = H;
    long long parts = (H + rows - 1) / rows;
    const long long fit = rows / ((H + parts - 1) / parts), angles = n ? kT / n : kT;
    w.TN = (int)std::max(1ll, std::min({fit, angles, (long long)N, (long long)B * N / 304}));
    w.nb = (N + w.TN - 1) / w.TN;
    const long long x = (long long)B * w.nb;
    parts = std::max(parts, std::min<long long>(H, 304 / x));
    w.hper = (int)((H + parts - 1) / parts);
    w.ny = (H + w.hper - 1) / w.hper;
    if (x * w.ny > 0x3fffffffll) return false;
    w.groups = (int)(x * w.ny);
    w.by_nb = fast_div(w.nb), w.by_ny = fast_div(w.ny), w.by_h = fast_div(w.hper);
    w.by_last = fast_div(H - (w.ny - 1) * w.hper), w.by_u = fast_div(per), w.by_tn = fast_div(w.TN);
    *out = w;
    return true;
}
// Blocks: four on each of 152 SMs (what their registers allow), each with a group or more.
inline int blocks_for(const Work& w) { return std::min(w.groups, 608); }

}  // namespace
}  // namespace win
}  // namespace psa
