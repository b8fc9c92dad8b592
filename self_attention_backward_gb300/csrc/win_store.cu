// win_store.cu -- the rolling cache in 8 bits: rows quantised as they are written (keys
// rotated on the way), and caches of every type read back by position.
//
// A row x of d features becomes e4m3 codes and one scale s, the smallest power of two (from
// 2^-100 on) with max|x| <= 448 s: code = x / s rounded to e4m3.  A power of two because
// e4m3 is a floating format: a scale in between would move the codes' range, not their
// precision, and x / s as well as code * s are then exact in fp32, the latter in bf16 too.  So
// the code is the one rounding on the way (of the fp32 rotated key; there is no bf16 in
// between) and does not depend on how a division is done.  A row with an element that is
// not finite has the scale NaN and codes 0.
//
// Bound by memory: every row is read and written once.  A lane has 8 features, d / 8 lanes a
// row, whose largest element goes round by shuffles; a rotation's other feature comes from
// the lane that has it.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <string>

#include "rope.cuh"

namespace psa {
namespace win {
namespace {

constexpr int kF = 8;                             // features per lane

struct Rows {                                     // keys or values to be written
    const void* x;
    long long sB, sH, sN, sJ;
};
struct Cache8 {
    uint8_t* k;
    uint8_t* v;
    float* ks;
    float* vs;
    long long sB, sH, sS, cB, cH, cS;
    int cap, sinks, vec;
};

// 8 features as they lie in memory
template <typename T>
struct Raw {
    uint4 u[kF * sizeof(T) / 16];
};
template <typename T, bool VEC>
__device__ __forceinline__ Raw<T> load_raw(const T* p, long long sJ) {
    Raw<T> r;
    if constexpr (VEC) {
#pragma unroll
        for (int i = 0; i < (int)(kF * sizeof(T) / 16); ++i) r.u[i] = reinterpret_cast<const uint4*>(p)[i];
    } else {
        T* x = reinterpret_cast<T*>(r.u);
#pragma unroll
        for (int e = 0; e < kF; ++e) x[e] = p[e * sJ];
    }
    return r;
}
template <typename T>
__device__ __forceinline__ void to_f(const Raw<T>& r, float (&x)[kF]) {
    constexpr int W = 16 / (int)sizeof(T);
#pragma unroll
    for (int i = 0; i < kF / W; ++i) {
        float y[W];
        unpack<T>(r.u[i], y);
#pragma unroll
        for (int e = 0; e < W; ++e) x[i * W + e] = y[e];
    }
}
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// The codes of a row's 8 features in a lane (largest element first by all `lanes` of the row) to
// `to`, its scale by the row's first lane.  All lanes of a warp take part; `write`: this
// lane's row is there.
__device__ __forceinline__ void quantise(const float (&y)[kF], int lanes, bool write, uint8_t* to, bool vec, float* scale) {
    uint32_t top = 0;                             // as whole numbers: infinities and NaN are the largest
#pragma unroll
    for (int e = 0; e < kF; ++e) top = max(top, __float_as_uint(y[e]) & 0x7fffffffu);
    for (int i = 1; i < lanes; i <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, i));
    if (!write) return;
    // 448 = 1.75 2^8
    const int e2 = max((int)(top >> 23) - 127 - ((top & 0x7fffffu) <= 0x600000u ? 8 : 7), -100);
    const bool some = top < 0x7f800000u;
    const float up = __uint_as_float((uint32_t)(127 - e2) << 23);
    uint32_t code[2] = {0, 0};
    if (some) {
#pragma unroll
        for (int e = 0; e < kF; e += 2) code[e / 4] |= e4m3x2(y[e] * up, y[e + 1] * up) << (8 * (e % 4));
    }
    if (vec) {
        *reinterpret_cast<uint2*>(to) = make_uint2(code[0], code[1]);
    } else {
#pragma unroll
        for (int e = 0; e < kF; ++e) to[e] = (uint8_t)(code[e / 4] >> (8 * (e % 4)));
    }
    if (scale) *scale = __uint_as_float(some ? (uint32_t)(127 + e2) << 23 : 0x7fffffffu);
}

// A warp per token and `hper` heads, a half for keys and a half for values: its angles once (two
// a lane, through shared memory), then head after head, the next one's loads on their way.
// No barriers between warps.  16-byte loads; a rotation's partners are at the same place of
// another lane, or in the lane.
template <typename T, int D>
__global__ void __launch_bounds__(kT, 4)
append8_kernel(const __grid_constant__ Plan pl, const __grid_constant__ Rows kn, const __grid_constant__ Rows vn,
               const __grid_constant__ Cache8 c, Pos pos, const int* __restrict__ start, const int* __restrict__ n_new, int Tn,
               int N, int H, int hper, int parts, int tasks, FastDiv by_parts, FastDiv by_n, Picked from) {
    constexpr int LANES = D / kF, SUB = 32 / (2 * LANES);   // lanes of a row; heads at a time
    __shared__ __align__(16) float2 cs_all[kT / 32][PSA_ROPE_MAX_PAIRS];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, q = lane % (2 * LANES), sub = lane / (2 * LANES);
    const bool key = q < LANES;
    const int f0 = (key ? q : q - LANES) * kF, n = pl.n;
    const Rows& mine = key ? kn : vn;
    float2* cs = cs_all[warp];
    // the lane's first pair, and the lane that has its other features
    const bool turned = key && f0 < 2 * n, first = f0 < n;
    const int p0 = pl.interleaved ? f0 / 2 : first ? f0 : f0 - n;
    const int other = turned && !pl.interleaved ? lane + (first ? n / kF : -n / kF) : lane;
    Kept kept;
    const int task = blockIdx.x * (kT / 32) + warp;
    if (task < tasks) {
        const int tok = divide(task, by_parts), h0 = (task - tok * parts) * hper, b = divide(tok, by_n);
        const int ring = c.cap - c.sinks, h1 = min(h0 + hper, H);
        kept.of(start, n_new, b, Tn, c.sinks, ring);
        int x = kept.row(tok - b * N);
        const int at_pos = kept.st + x;
        if (x >= kept.n || (from.rows && !from.row(b, x))) return;        // the same for the whole warp
        const long long slot = at_pos < c.sinks ? at_pos : c.sinks + (at_pos - c.sinks) % ring;
        const T* src = static_cast<const T*>(mine.x) + b * mine.sB + (long long)x * mine.sN + f0;
        uint8_t* to = (key ? c.k : c.v) + b * c.sB + slot * c.sS + f0;
        float* scale = (key ? c.ks : c.vs) + b * c.cB + slot * c.cS;
        Raw<T> l{}, ln{};
        if (h0 + sub < h1) l = load_raw<T, true>(src + (h0 + sub) * mine.sH, 1);
        for (int i = lane; i < n; i += 32) cs[i] = cos_sin(pl, i, load_pos(pl, pos, i, b, x), 1.f);
        __syncwarp();
        float2 w[kF];
#pragma unroll
        for (int e = 0; e < kF; ++e) w[e] = turned && (e < 4 || !pl.interleaved) ? cs[p0 + e] : make_float2(1.f, 0.f);
        for (int hh = h0; hh < h1; hh += SUB) {
            const int h = hh + sub;
            if (h + SUB < h1) ln = load_raw<T, true>(src + (h + SUB) * mine.sH, 1);
            float y[kF];
            to_f(l, y);
            if (n > 0) {
                Raw<T> ro;                        // the partners as they lie in memory
#pragma unroll
                for (int i = 0; i < (int)(sizeof(ro) / 16); ++i)
                    ro.u[i] = make_uint4(__shfl_sync(0xffffffffu, l.u[i].x, other), __shfl_sync(0xffffffffu, l.u[i].y, other),
                                         __shfl_sync(0xffffffffu, l.u[i].z, other), __shfl_sync(0xffffffffu, l.u[i].w, other));
                if (turned) {
                    if (pl.interleaved) {
#pragma unroll
                        for (int e = 0; e < kF; e += 2)
                            if (f0 + e < 2 * n) {
                                const float a = y[e], z = y[e + 1];
                                y[e] = a * w[e / 2].x - z * w[e / 2].y;
                                y[e + 1] = z * w[e / 2].x + a * w[e / 2].y;
                            }
                    } else {
                        float o[kF];
                        to_f(ro, o);
#pragma unroll
                        for (int e = 0; e < kF; ++e) y[e] = first ? y[e] * w[e].x - o[e] * w[e].y : y[e] * w[e].x + o[e] * w[e].y;
                    }
                }
            }
            quantise(y, LANES, h < h1, to + h * c.sH, c.vec, f0 == 0 ? scale + h * c.cH : nullptr);
            l = ln;
        }
    }
}

// Any layout: a lane per 8 features, element by element; a partner is read again.
template <typename T>
__global__ void __launch_bounds__(kT)
append8_scalar_kernel(const __grid_constant__ Plan pl, const __grid_constant__ Rows kn, const __grid_constant__ Rows vn,
                      const __grid_constant__ Cache8 c, Pos pos, const int* __restrict__ start, const int* __restrict__ n_new,
                      int Tn, int N, int H, long long total, Picked from) {
    const int lanes = pl.d / kF, n = pl.n;
    const long long idx = (long long)blockIdx.x * kT + threadIdx.x, row = idx / (2 * lanes);   // (token, head)
    const int q = (int)(idx % (2 * lanes));
    const bool key = q < lanes;
    const int f0 = (key ? q : q - lanes) * kF;
    const Rows& mine = key ? kn : vn;
    bool write = row < total;
    float y[kF] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    uint8_t* to = nullptr;
    float* scale = nullptr;
    if (write) {
        const int h = (int)(row % H);
        const long long tok = row / H;
        const int b = (int)(tok / N), ring = c.cap - c.sinks;
        Kept kept;
        kept.of(start, n_new, b, Tn, c.sinks, ring);
        int x = kept.row((int)(tok % N));
        const int at_pos = kept.st + x;
        write = x < kept.n && (!from.rows || from.row(b, x));
        if (write) {
            const long long slot = at_pos < c.sinks ? at_pos : c.sinks + (at_pos - c.sinks) % ring;
            const T* src = static_cast<const T*>(mine.x) + b * mine.sB + h * mine.sH + (long long)x * mine.sN;
            for (int e = 0; e < kF; ++e) {
                const int f = f0 + e;
                y[e] = to_f32(src[f * mine.sJ]);
                if (key && f < 2 * n) {
                    const bool first = pl.interleaved ? f % 2 == 0 : f < n;
                    const int i = pl.interleaved ? f / 2 : first ? f : f - n;
                    const float z = to_f32(src[(pl.interleaved ? f ^ 1 : first ? f + n : f - n) * mine.sJ]);
                    const float2 w = cos_sin(pl, i, load_pos(pl, pos, i, b, x), 1.f);
                    y[e] = first ? y[e] * w.x - z * w.y : y[e] * w.x + z * w.y;
                }
            }
            to = (key ? c.k : c.v) + b * c.sB + h * c.sH + slot * c.sS + f0;
            if (f0 == 0) scale = (key ? c.ks : c.vs) + b * c.cB + h * c.cH + slot * c.cS;
        }
    }
    quantise(y, lanes, write, to, c.vec, scale);
}

template <typename T>
int launch_append8(const AppendArgs& a, std::string* err) {
    const Plan pl = dev_plan(a.plan, a.d);
    const Rows kn{a.kn.base, a.kn.sB, a.kn.sH, a.kn.sN, a.kn.sJ}, vn{a.vn.base, a.vn.sB, a.vn.sH, a.vn.sN, a.vn.sJ};
    const int by8 = a.sB % 8 == 0 && a.sH % 8 == 0 && a.sS % 8 == 0;
    const Cache8 c{static_cast<uint8_t*>(a.k), static_cast<uint8_t*>(a.v), a.ks, a.vs, a.sB, a.sH, a.sS, a.cB, a.cH, a.cS,
                   a.cap, a.sinks, by8};
    const Pos pos{a.pos, a.pos_axis, a.pos_batch};
    const Picked from{a.rows, a.rows_stride, a.n_rows};
    const bool vec = view_ok(a.kn, sizeof(T)) && view_ok(a.vn, sizeof(T)) && (pl.interleaved || pl.n % kF == 0);
    const int N = std::min(a.T, a.cap);               // rows of a sequence that can stay
    const long long tokens = (long long)a.B * N;
    if (!vec) {
        const long long total = tokens * a.Hkv, grid = (total * (2 * a.d / kF) + kT - 1) / kT;
        if (grid > 0x7fffffffll) return too_large(err);
        append8_scalar_kernel<T><<<(unsigned)grid, kT, 0, a.stream>>>(pl, kn, vn, c, pos, a.start, a.n_new, a.T, N, a.Hkv, total, from);
        return launched("8-bit cache append launch", err);
    }
    // all heads of a token to one warp (its angles serve them all), where that leaves 8 warps an SM
    const long long want = 152 * 8;
    const int parts0 = (int)std::min<long long>(a.Hkv, std::max(1ll, want / tokens));
    const int hper = (a.Hkv + parts0 - 1) / parts0, parts = (a.Hkv + hper - 1) / hper;
    if (tokens * parts > 0x3fffffffll) return too_large(err);
    const int tasks = (int)(tokens * parts), grid = (tasks + kT / 32 - 1) / (kT / 32);
    auto go = [&](auto kernel) {
        kernel<<<grid, kT, 0, a.stream>>>(pl, kn, vn, c, pos, a.start, a.n_new, a.T, N, a.Hkv, hper, parts, tasks, fast_div(parts),
                                          fast_div(N), from);
    };
    switch (a.d) {
        case 16: go(append8_kernel<T, 16>); break;
        case 32: go(append8_kernel<T, 32>); break;
        case 64: go(append8_kernel<T, 64>); break;
        default: go(append8_kernel<T, 128>);
    }
    return launched("8-bit cache append launch", err);
}

// ---------------------------------------------------------------- read
struct ReadP {
    const void* k;
    const void* v;
    const float* ks;
    const float* vs;
    long long sB, sH, sS, cB, cH, cS;
    View ko, vo;
    const int* first;
    const int* lens;
    int N, H, sinks, ring, vec_in, vec_out;
    FastDiv by_n, by_h;
};
struct Byte {
    uint8_t x;
};

constexpr int kR = 16;                            // features per thread

template <typename C>
__device__ __forceinline__ void load16(const C* p, bool vec, float (&x)[kR]) {
    uint4 u[kR * sizeof(C) / 16];
    if (vec) {
#pragma unroll
        for (int i = 0; i < (int)(kR * sizeof(C) / 16); ++i) u[i] = __ldg(reinterpret_cast<const uint4*>(p) + i);
    } else {
#pragma unroll
        for (int e = 0; e < kR; ++e) reinterpret_cast<C*>(u)[e] = p[e];
    }
    if constexpr (sizeof(C) == 1) {
        const uint32_t w[4] = {u[0].x, u[0].y, u[0].z, u[0].w};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            uint32_t h;
            const uint16_t two = (uint16_t)(w[i / 2] >> (16 * (i % 2)));
            asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(two));
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
            x[2 * i] = f.x, x[2 * i + 1] = f.y;
        }
    } else {
        constexpr int W = 16 / (int)sizeof(C);
#pragma unroll
        for (int i = 0; i < kR / W; ++i) {
            float y[W];
            unpack<C>(u[i], y);
#pragma unroll
            for (int e = 0; e < W; ++e) x[i * W + e] = y[e];
        }
    }
}
template <typename T>
__device__ __forceinline__ void store16(T* p, long long sJ, bool vec, const float (&x)[kR]) {
    if (vec) {
        constexpr int W = 16 / (int)sizeof(T);
#pragma unroll
        for (int i = 0; i < kR / W; ++i) {
            float y[W];
#pragma unroll
            for (int e = 0; e < W; ++e) y[e] = x[i * W + e];
            reinterpret_cast<uint4*>(p)[i] = pack<T>(y);
        }
    } else {
#pragma unroll
        for (int e = 0; e < kR; ++e) p[e * sJ] = from_f32<T>(x[e]);
    }
}

// A thread has 16 features of a position's key and value.
template <typename T, typename C, int D>
__global__ void __launch_bounds__(kT)
read_kernel(const __grid_constant__ ReadP a, int rows) {
    constexpr int U = D / kR;
    const long long idx = (long long)blockIdx.x * kT + threadIdx.x;
    if (idx >= (long long)rows * U) return;
    const int row = (int)(idx / U), f = (int)(idx % U) * kR;
    const int bh = divide(row, a.by_n), i = row - bh * a.N, b = divide(bh, a.by_h), h = bh - b * a.H;
    const int L = max(__ldg(a.lens + b), 0);
    const long long p = (long long)__ldg(a.first + b) + i;
    float k[kR], v[kR];
    if (p >= 0 && p < L && (p < a.sinks || p >= L - a.ring)) {
        const int at_pos = (int)p;
        const long long slot = at_pos < a.sinks ? at_pos : a.sinks + (at_pos - a.sinks) % a.ring;
        const long long at = b * a.sB + h * a.sH + slot * a.sS + f;
        float sk = 1.f, sv = 1.f;
        if constexpr (sizeof(C) == 1) {
            const long long sc = b * a.cB + h * a.cH + slot * a.cS;
            sk = __ldg(a.ks + sc), sv = __ldg(a.vs + sc);
        }
        load16<C>(static_cast<const C*>(a.k) + at, a.vec_in, k);
        load16<C>(static_cast<const C*>(a.v) + at, a.vec_in, v);
        if constexpr (sizeof(C) == 1) {
#pragma unroll
            for (int e = 0; e < kR; ++e) k[e] *= sk, v[e] *= sv;
        }
    } else {
#pragma unroll
        for (int e = 0; e < kR; ++e) k[e] = v[e] = 0.f;
    }
    store16<T>(static_cast<T*>(const_cast<void*>(a.ko.base)) + b * a.ko.sB + h * a.ko.sH + (long long)i * a.ko.sN + f * a.ko.sJ,
               a.ko.sJ, a.vec_out, k);
    store16<T>(static_cast<T*>(const_cast<void*>(a.vo.base)) + b * a.vo.sB + h * a.vo.sH + (long long)i * a.vo.sN + f * a.vo.sJ,
               a.vo.sJ, a.vec_out, v);
}

template <typename T, typename C>
int launch_read(const ReadArgs& a, std::string* err) {
    const long long rows = (long long)a.B * a.Hkv * a.N, grid = (rows * (a.d / kR) + kT - 1) / kT;
    if (rows > 0x7fffffffll || grid > 0x7fffffffll) return too_large(err);
    ReadP p{a.k, a.v, a.ks, a.vs, a.sB, a.sH, a.sS, a.cB, a.cH, a.cS, a.ko, a.vo, a.first, a.lens, a.N, a.Hkv, a.sinks,
            a.cap - a.sinks, 0, 0, fast_div(a.N), fast_div(a.Hkv)};
    constexpr long long W = 16 / sizeof(C);
    p.vec_in = a.sB % W == 0 && a.sH % W == 0 && a.sS % W == 0;
    p.vec_out = view_ok(a.ko, sizeof(T)) && view_ok(a.vo, sizeof(T));
    switch (a.d) {
        case 16: read_kernel<T, C, 16><<<(unsigned)grid, kT, 0, a.stream>>>(p, (int)rows); break;
        case 32: read_kernel<T, C, 32><<<(unsigned)grid, kT, 0, a.stream>>>(p, (int)rows); break;
        case 64: read_kernel<T, C, 64><<<(unsigned)grid, kT, 0, a.stream>>>(p, (int)rows); break;
        default: read_kernel<T, C, 128><<<(unsigned)grid, kT, 0, a.stream>>>(p, (int)rows);
    }
    return launched("cache read launch", err);
}
template <typename T>
int launch_read_of(const ReadArgs& a, std::string* err) {
    return a.cache_dtype == PSA_E4M3  ? launch_read<T, Byte>(a, err)
           : a.cache_dtype == PSA_F32 ? launch_read<T, float>(a, err)
                                      : launch_read<T, __nv_bfloat16>(a, err);
}

}  // namespace

int append_8(const AppendArgs& a, std::string* err) {
    return a.dtype == PSA_F32 ? launch_append8<float>(a, err) : launch_append8<__nv_bfloat16>(a, err);
}
int read(const ReadArgs& a, std::string* err) {
    return a.dtype == PSA_F32 ? launch_read_of<float>(a, err) : launch_read_of<__nv_bfloat16>(a, err);
}

}  // namespace win
}  // namespace psa
