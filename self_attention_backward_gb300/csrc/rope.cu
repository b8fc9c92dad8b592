// rope.cu -- rotary positions with several axes, and the rolling cache's
// writes (which rotate the keys on the way).
//
//   y1 = x1 cos a - x2 sin a,  y2 = x2 cos a + x1 sin a,  a = 2 pi pos F / 2^64
// F is the pair's frequency as a 64-bit fraction of a turn, so pos * F modulo
// 2^64 is the angle modulo a turn, exactly, for every 32-bit position: no range
// reduction, and no 64-bit floating point, which this GPU has little of.  Its
// upper 32 bits, rounded, go to sincospif; the angle is then off by at most
// half an fp32 step (2^-26 turns).
//
// Bound by memory: every element is read and written once.  A block takes a few
// tokens, computes their cos / sin once for all heads of both tensors (shared
// memory), and streams the heads through in 16-byte units.
#include <cuda_bf16.h>

#include <cmath>
#include <string>

#include "common.cuh"
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

struct Tensor {                                  // one view to rotate
    const void* x;
    void* y;
    long long xB, xH, xN, xJ, yB, yH, yN, yJ;
};

struct Pos {
    const int* p;
    long long axis, batch;
};

__device__ __forceinline__ float2 cos_sin(const Plan& pl, const Pos& pos, int i, int b, long long n, float sign) {
    const long long p = __ldg(pos.p + pl.axis[i] * pos.axis + b * pos.batch + n);
    const unsigned long long t = (unsigned long long)p * pl.turn[i] + 0x80000000ull;
    float s, c;
    sincospif((float)(int)(t >> 32) * 0x1p-31f, &s, &c);
    return make_float2(c, s * sign);
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

// Units of 16 bytes of a head: with pairs in halves a unit is the 16 bytes at
// feature c and those at c + n; interleaved pairs lie inside a unit; units past
// the rotated features are copied.
struct Units {
    int rot, total;
};
template <typename T>
__host__ __device__ __forceinline__ Units units(int d, int n, int interleaved) {
    const int rot = interleaved ? 2 * n / VEC<T> : n / VEC<T>;
    return Units{rot, rot + (d - 2 * n) / VEC<T>};
}

template <typename T>
struct Loaded {
    uint4 a, b;
};
template <typename T>
__device__ __forceinline__ Loaded<T> load_unit(const T* x, int u, const Units& us, int n, int interleaved) {
    Loaded<T> l;
    if (u >= us.rot) {
        l.a = *reinterpret_cast<const uint4*>(x + 2 * n + (u - us.rot) * VEC<T>);
    } else {
        l.a = *reinterpret_cast<const uint4*>(x + u * VEC<T>);
        if (!interleaved) l.b = *reinterpret_cast<const uint4*>(x + n + u * VEC<T>);
    }
    return l;
}
// cs: the token's (cos, sin) of every pair
template <typename T>
__device__ __forceinline__ void store_unit(T* y, const Loaded<T>& l, int u, const Units& us, int n, int interleaved,
                                           const float2* cs) {
    constexpr int W = VEC<T>;
    if (u >= us.rot) {
        *reinterpret_cast<uint4*>(y + 2 * n + (u - us.rot) * W) = l.a;
        return;
    }
    float a[W], r[W];
    unpack<T>(l.a, a);
    if (interleaved) {
#pragma unroll
        for (int e = 0; e < W / 2; ++e) {
            const float2 w = cs[u * (W / 2) + e];
            r[2 * e] = a[2 * e] * w.x - a[2 * e + 1] * w.y;
            r[2 * e + 1] = a[2 * e + 1] * w.x + a[2 * e] * w.y;
        }
        *reinterpret_cast<uint4*>(y + u * W) = pack<T>(r);
    } else {
        float b[W], q[W];
        unpack<T>(l.b, b);
#pragma unroll
        for (int e = 0; e < W; ++e) {
            const float2 w = cs[u * W + e];
            r[e] = a[e] * w.x - b[e] * w.y;
            q[e] = b[e] * w.x + a[e] * w.y;
        }
        *reinterpret_cast<uint4*>(y + u * W) = pack<T>(r);
        *reinterpret_cast<uint4*>(y + n + u * W) = pack<T>(q);
    }
}

// One feature pair (or, i >= n, one copied feature), any strides.
template <typename T>
__device__ __forceinline__ void scalar_pair(const T* x, long long xJ, T* y, long long yJ, int i, int n, int interleaved,
                                            float2 w) {
    if (i >= n) {
        const int f = n + i;                     // features 2n ...
        y[f * yJ] = x[f * xJ];
        return;
    }
    const int f1 = interleaved ? 2 * i : i, f2 = interleaved ? 2 * i + 1 : i + n;
    const float a = to_f32(x[f1 * xJ]), b = to_f32(x[f2 * xJ]);
    y[f1 * yJ] = from_f32<T>(a * w.x - b * w.y);
    y[f2 * yJ] = from_f32<T>(b * w.x + a * w.y);
}

// ---------------------------------------------------------------- rope
// Block (token group, head group): TN tokens, heads [hb, he) of the heads of
// both tensors one behind the other.
template <typename T>
__global__ void __launch_bounds__(kT)
rope_kernel(const __grid_constant__ Plan pl, Tensor t0, Tensor t1, int H0, int H, Pos pos, int N, long long tokens, int TN,
            int hper, float sign) {
    extern __shared__ float2 cs[];               // [TN][n]
    const long long tok0 = (long long)blockIdx.x * TN;
    const int nt = (int)min((long long)TN, tokens - tok0);
    for (int idx = threadIdx.x; idx < nt * pl.n; idx += kT) {
        const int t = idx / pl.n, i = idx - t * pl.n;
        const long long tok = tok0 + t;
        cs[idx] = cos_sin(pl, pos, i, (int)(tok / N), tok % N, sign);
    }
    __syncthreads();
    const Units us = units<T>(pl.d, pl.n, pl.interleaved);
    const int hb = blockIdx.y * hper, nh = min(hper, H - hb);
    const int rows = kT / us.total, r0 = threadIdx.x / us.total, u = threadIdx.x - r0 * us.total;
    if (r0 >= rows) return;
    for (int r = r0; r < nt * nh; r += rows) {
        const int t = r / nh, h = hb + r - t * nh;
        const long long tok = tok0 + t;
        const long long b = tok / N, n = tok - b * N;
        const Tensor& v = h < H0 ? t0 : t1;
        const int hh = h < H0 ? h : h - H0;
        const T* x = static_cast<const T*>(v.x) + b * v.xB + hh * v.xH + n * v.xN;
        T* y = static_cast<T*>(v.y) + b * v.yB + hh * v.yH + n * v.yN;
        const Loaded<T> l = load_unit(x, u, us, pl.n, pl.interleaved);
        store_unit(y, l, u, us, pl.n, pl.interleaved, cs + t * pl.n);
    }
}

// Any strides: a thread per (token, pair), over all heads; neighbouring threads
// take neighbouring positions (pos_fast: channel-major tensors) or pairs.
template <typename T>
__global__ void __launch_bounds__(kT)
rope_scalar_kernel(const __grid_constant__ Plan pl, Tensor t0, Tensor t1, int H0, int H, Pos pos, int N, long long total,
                   int pos_fast, float sign) {
    const long long idx = (long long)blockIdx.x * kT + threadIdx.x;
    if (idx >= total) return;
    const int items = pl.d - pl.n;               // pairs and copied features
    long long b, n;
    int i;
    if (pos_fast) {
        n = idx % N;
        const long long r = idx / N;
        i = (int)(r % items), b = r / items;
    } else {
        i = (int)(idx % items);
        const long long r = idx / items;
        n = r % N, b = r / N;
    }
    const float2 w = i < pl.n ? cos_sin(pl, pos, i, (int)b, n, sign) : make_float2(1.f, 0.f);
    for (int h = 0; h < H; ++h) {
        const Tensor& v = h < H0 ? t0 : t1;
        const int hh = h < H0 ? h : h - H0;
        scalar_pair<T>(static_cast<const T*>(v.x) + b * v.xB + hh * v.xH + n * v.xN, v.xJ,
                       static_cast<T*>(v.y) + b * v.yB + hh * v.yH + n * v.yN, v.yJ, i, pl.n, pl.interleaved, w);
    }
}

// ---------------------------------------------------------------- cache append
struct Cache {
    void* k;
    void* v;
    long long sB, sH, sS;
    int cap, sinks;
};

// Slot of row t of sequence b, or -1: past n_new, or overwritten by a newer
// row of the same call (sinks never are).
__device__ __forceinline__ int slot_of(const Cache& c, const int* start, const int* n_new, int b, int t, int T) {
    const int st = __ldg(start + b);
    const int n = n_new ? min(max(__ldg(n_new + b), 0), T) : T;
    if (t >= n || st < 0 || st > 0x7fffffff - n) return -1;
    const int ring = c.cap - c.sinks, p = st + t;
    if (p < c.sinks) return p;
    if (t < n - ring) return -1;                 // p + ring is in this call too
    return c.sinks + (p - c.sinks) % ring;
}

template <typename T>
__global__ void __launch_bounds__(kT)
append_kernel(const __grid_constant__ Plan pl, Tensor kn, Tensor vn, Cache c, int Hkv, Pos pos, const int* __restrict__ start,
              const int* __restrict__ n_new, int Tn, long long tokens, int TN) {
    extern __shared__ float2 cs[];               // [TN][n], then the tokens' slots
    int* slots = reinterpret_cast<int*>(cs + TN * pl.n);
    const long long tok0 = (long long)blockIdx.x * TN;
    const int nt = (int)min((long long)TN, tokens - tok0);
    if (threadIdx.x < nt) {
        const long long tok = tok0 + threadIdx.x;
        slots[threadIdx.x] = slot_of(c, start, n_new, (int)(tok / Tn), (int)(tok % Tn), Tn);
    }
    __syncthreads();
    for (int idx = threadIdx.x; idx < nt * pl.n; idx += kT) {
        const int t = idx / pl.n, i = idx - t * pl.n;
        const long long tok = tok0 + t;
        if (slots[t] >= 0) cs[idx] = cos_sin(pl, pos, i, (int)(tok / Tn), tok % Tn, 1.f);
    }
    __syncthreads();
    // keys by rotation units, values as plain 16-byte pieces (n = 0: all are copied)
    const Units uk = units<T>(pl.d, pl.n, pl.interleaved), uv = units<T>(pl.d, 0, 0);
    const int per = uk.total + uv.total, rows = kT / per;
    const int r0 = threadIdx.x / per, w = threadIdx.x - r0 * per;
    if (r0 >= rows) return;
    for (int r = r0; r < nt * Hkv; r += rows) {
        const int t = r / Hkv, h = r - t * Hkv, slot = slots[t];
        if (slot < 0) continue;
        const long long tok = tok0 + t;
        const long long b = tok / Tn, n = tok - b * Tn;
        const long long to = b * c.sB + h * c.sH + slot * c.sS;
        if (w < uk.total) {
            const T* x = static_cast<const T*>(kn.x) + b * kn.xB + h * kn.xH + n * kn.xN;
            store_unit(static_cast<T*>(c.k) + to, load_unit(x, w, uk, pl.n, pl.interleaved), w, uk, pl.n, pl.interleaved,
                       cs + t * pl.n);
        } else {
            const T* x = static_cast<const T*>(vn.x) + b * vn.xB + h * vn.xH + n * vn.xN;
            store_unit(static_cast<T*>(c.v) + to, load_unit(x, w - uk.total, uv, 0, 0), w - uk.total, uv, 0, 0, cs);
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(kT)
append_scalar_kernel(const __grid_constant__ Plan pl, Tensor kn, Tensor vn, Cache c, int Hkv, Pos pos,
                     const int* __restrict__ start, const int* __restrict__ n_new, int Tn, long long total) {
    const long long idx = (long long)blockIdx.x * kT + threadIdx.x;
    if (idx >= total) return;
    const int items = pl.d - pl.n, i = (int)(idx % items);
    const long long tok = idx / items, b = tok / Tn, n = tok % Tn;
    const int slot = slot_of(c, start, n_new, (int)b, (int)n, Tn);
    if (slot < 0) return;
    const float2 w = i < pl.n ? cos_sin(pl, pos, i, (int)b, n, 1.f) : make_float2(1.f, 0.f);
    for (int h = 0; h < Hkv; ++h) {
        const long long to = b * c.sB + h * c.sH + slot * c.sS;
        scalar_pair<T>(static_cast<const T*>(kn.x) + b * kn.xB + h * kn.xH + n * kn.xN, kn.xJ,
                       static_cast<T*>(c.k) + to, 1, i, pl.n, pl.interleaved, w);
        const T* x = static_cast<const T*>(vn.x) + b * vn.xB + h * vn.xH + n * vn.xN;
        T* y = static_cast<T*>(c.v) + to;
        for (int f = i; f < pl.d; f += items) y[f] = x[f * vn.xJ];
    }
}

Plan dev_plan(const psa_rope_plan* p, int d) {
    Plan pl{};
    pl.d = d;
    if (!p) return pl;                           // no pairs: everything is copied
    pl.n = p->rot_dim / 2;
    pl.interleaved = p->interleaved;
    for (int i = 0; i < pl.n; ++i) pl.turn[i] = p->turn[i], pl.axis[i] = p->axis[i];
    return pl;
}

bool aligned(const void* p, int esize, long long a, long long b, long long c) {
    const long long w = 16 / esize;
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && a % w == 0 && b % w == 0 && c % w == 0;
}
bool view_ok(const View& v, int esize) { return v.sJ == 1 && aligned(v.base, esize, v.sB, v.sH, v.sN); }
// a rotation whose pairs and rest fill whole 16-byte units
bool plan_ok(const Plan& pl, int esize) {
    const int w = 16 / esize;
    return pl.interleaved ? 2 * pl.n % w == 0 : pl.n % w == 0 && (pl.d - 2 * pl.n) % w == 0;
}

int launched(const char* what, std::string* err) {
    const cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) return PSA_OK;
    *err = std::string(what) + ": " + cudaGetErrorString(e);
    return PSA_ERR_CUDA;
}
int too_large(std::string* err) {
    *err = "grid too large";
    return PSA_ERR_UNSUPPORTED;
}

Tensor tensor(const View& x, const View& y) {
    return Tensor{x.base, const_cast<void*>(y.base), x.sB, x.sH, x.sN, x.sJ, y.sB, y.sH, y.sN, y.sJ};
}

template <typename T>
int launch_rope(const RopeArgs& a, std::string* err) {
    const Plan pl = dev_plan(a.plan, a.plan->head_dim);
    const long long tokens = (long long)a.B * a.N;
    const int H0 = a.heads[0], H = H0 + (a.n > 1 ? a.heads[1] : 0);
    const Tensor t0 = tensor(a.x[0], a.y[0]), t1 = a.n > 1 ? tensor(a.x[1], a.y[1]) : t0;
    const Pos pos{a.pos, a.pos_axis, a.pos_batch};
    const float sign = a.inverse ? -1.f : 1.f;
    bool vec = plan_ok(pl, sizeof(T));
    for (int i = 0; i < a.n; ++i) vec = vec && view_ok(a.x[i], sizeof(T)) && view_ok(a.y[i], sizeof(T));
    if (!vec) {
        const long long total = tokens * (pl.d - pl.n), grid = (total + kT - 1) / kT;
        if (grid > 0x7fffffffll) return too_large(err);
        rope_scalar_kernel<T><<<(unsigned)grid, kT, 0, a.stream>>>(pl, t0, t1, H0, H, pos, a.N, total,
                                                                   a.x[0].sN == 1 && a.x[0].sJ != 1, sign);
        return launched("rope launch", err);
    }
    // a few tokens per block, so that their angles serve many heads, but at
    // least about four blocks per SM; with few tokens the heads are split too
    const Units us = units<T>(pl.d, pl.n, pl.interleaved);
    const int rows = kT / us.total, target = 608;
    int TN = (int)std::min<long long>(8, std::max<long long>(1, tokens / target));
    const long long gx = (tokens + TN - 1) / TN;
    long long gy = std::min<long long>((H + rows - 1) / rows, std::max<long long>(1, target / gx));
    const int hper = (int)((H + gy - 1) / gy);
    gy = (H + hper - 1) / hper;
    if (gx > 0x7fffffffll) return too_large(err);
    rope_kernel<T><<<dim3((unsigned)gx, (unsigned)gy), kT, (size_t)TN * pl.n * sizeof(float2), a.stream>>>(
        pl, t0, t1, H0, H, pos, a.N, tokens, TN, hper, sign);
    return launched("rope launch", err);
}

template <typename T>
int launch_append(const AppendArgs& a, std::string* err) {
    const Plan pl = dev_plan(a.plan, a.d);
    const long long tokens = (long long)a.B * a.T;
    const View none{};
    const Tensor kn = tensor(a.kn, none), vn = tensor(a.vn, none);
    const Cache c{a.k, a.v, a.sB, a.sH, a.sS, a.cap, a.sinks};
    const Pos pos{a.pos, a.pos_axis, a.pos_batch};
    const bool vec = plan_ok(pl, sizeof(T)) && view_ok(a.kn, sizeof(T)) && view_ok(a.vn, sizeof(T)) &&
                     aligned(a.k, sizeof(T), a.sB, a.sH, a.sS) && aligned(a.v, sizeof(T), 0, 0, 0);
    if (!vec) {
        const long long total = tokens * (pl.d - pl.n), grid = (total + kT - 1) / kT;
        if (grid > 0x7fffffffll) return too_large(err);
        append_scalar_kernel<T><<<(unsigned)grid, kT, 0, a.stream>>>(pl, kn, vn, c, a.Hkv, pos, a.start, a.n_new, a.T, total);
        return launched("cache append launch", err);
    }
    const int TN = (int)std::min<long long>(8, std::max<long long>(1, tokens / 608));
    const long long gx = (tokens + TN - 1) / TN;
    if (gx > 0x7fffffffll) return too_large(err);
    append_kernel<T><<<(unsigned)gx, kT, (size_t)TN * (pl.n * sizeof(float2) + sizeof(int)), a.stream>>>(
        pl, kn, vn, c, a.Hkv, pos, a.start, a.n_new, a.T, tokens, TN);
    return launched("cache append launch", err);
}

}  // namespace

int rope(const RopeArgs& a, std::string* err) {
    return a.dtype == PSA_F32 ? launch_rope<float>(a, err) : launch_rope<__nv_bfloat16>(a, err);
}
int append(const AppendArgs& a, std::string* err) {
    return a.dtype == PSA_F32 ? launch_append<float>(a, err) : launch_append<__nv_bfloat16>(a, err);
}

}  // namespace win
}  // namespace psa
