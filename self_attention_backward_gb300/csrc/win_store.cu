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
// the lane that has it.  Groups of tokens and heads, angles in shared memory and the next
// group's loads on their way are as in rope.cu.
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

// VEC: 16-byte loads, a rotation whose partners are the same place of another lane or in the
// lane.  Else element by element, a partner read again from memory.
template <typename T, bool VEC>
__global__ void __launch_bounds__(kT)
append8_kernel(const __grid_constant__ Plan pl, const __grid_constant__ Rows kn, const __grid_constant__ Rows vn,
               const __grid_constant__ Cache8 c, Pos pos, const int* __restrict__ start, const int* __restrict__ n_new, int Tn,
               const __grid_constant__ Work w, Picked from) {
    extern __shared__ __align__(16) float2 cs_all[];   // [2][TN][n]
    // a row's key by d / 8 lanes, then its value
    const int lanes = pl.d / kF, row = threadIdx.x / (2 * lanes), q = threadIdx.x % (2 * lanes);
    const bool key = q < lanes;
    const int f0 = (key ? q : q - lanes) * kF, n = pl.n;
    const int ai = divide(threadIdx.x, w.by_tn), at = threadIdx.x - ai * w.TN;
    const Rows& mine = key ? kn : vn;
    Kept kept;
    // the lane's row of a group: its place in memory, token, head and slot (-1: none)
    auto load = [&](const Group& g, Raw<T>& l, const T*& src, int& p, int& t, int& h) {
        const int ring = c.cap - c.sinks;
        kept.of(start, n_new, g.b, Tn, c.sinks, ring);
        int slot = -1;
        if (row < g.nt * g.nh) {
            t = divide(row, g.nh == w.hper ? w.by_h : w.by_last);
            h = g.hb + row - t * g.nh;
            int x = kept.row(g.n0 + t);
            const int at_pos = kept.st + x;
            if (x < kept.n && (!from.rows || from.row(g.b, x))) {
                slot = at_pos < c.sinks ? at_pos : c.sinks + (at_pos - c.sinks) % ring;
                src = static_cast<const T*>(mine.x) + g.b * mine.sB + h * mine.sH + (long long)x * mine.sN;
                l = load_raw<T, VEC>(src + f0 * mine.sJ, mine.sJ);
            }
        }
        if (ai < n && at < g.nt) {
            int ax = kept.row(g.n0 + at);
            if (ax < kept.n && (!from.rows || from.row(g.b, ax))) p = load_pos(pl, pos, ai, g.b, ax);
        }
        return slot;
    };
    Group g = group_of(w, blockIdx.x), gn = g;
    Raw<T> l{}, ln{};
    const T *src = nullptr, *srcn = nullptr;
    int p = 0, pn = 0, t = 0, tn = 0, h = 0, hn = 0, buf = 0, slot_next = -1;
    int slot = load(g, l, src, p, t, h);
    for (int x = blockIdx.x; x < w.groups; x += gridDim.x) {
        if (x + (int)gridDim.x < w.groups) {
            gn = group_of(w, x + gridDim.x);
            slot_next = load(gn, ln, srcn, pn, tn, hn);
        }
        float2* cs = cs_all + buf * w.TN * n;     // a buffer is written again two barriers later
        buf ^= 1;
        if (ai < n && at < g.nt) cs[at * n + ai] = cos_sin(pl, ai, p, 1.f);
        __syncthreads();
        // all lanes take part: those without a row have anything in it, and do not write
        float y[kF];
        to_f(l, y);
        if (n > 0) {
            float o[kF];
            if (pl.interleaved) {
#pragma unroll
                for (int e = 0; e < kF; ++e) o[e] = y[e ^ 1];
            } else if (VEC) {
                const int by = n / kF, to = f0 < n ? by : -by;   // the partner's lane
                const int lane = threadIdx.x & 31, other = key && f0 < 2 * n ? lane + to : lane;
#pragma unroll
                for (int e = 0; e < kF; ++e) o[e] = __shfl_sync(0xffffffffu, y[e], other);
            } else {
#pragma unroll
                for (int e = 0; e < kF; ++e) {
                    const int f = f0 + e;
                    o[e] = key && slot >= 0 && f < 2 * n ? to_f32(src[(f < n ? f + n : f - n) * kn.sJ]) : 0.f;
                }
            }
            if (key && slot >= 0) {
#pragma unroll
                for (int e = 0; e < kF; ++e) {
                    const int f = f0 + e;
                    if (f < 2 * n) {
                        const bool first = pl.interleaved ? e % 2 == 0 : f < n;
                        const float2 a = cs[t * n + (pl.interleaved ? f / 2 : first ? f : f - n)];
                        y[e] = first ? y[e] * a.x - o[e] * a.y : y[e] * a.x + o[e] * a.y;
                    }
                }
            }
        }
        float top = 0.f;
        bool fine = true;
#pragma unroll
        for (int e = 0; e < kF; ++e) top = fmaxf(top, fabsf(y[e])), fine = fine && y[e] - y[e] == 0.f;
        if (!fine) top = INFINITY;
        for (int i = 1; i < lanes; i <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, i));
        if (slot >= 0) {
            const uint32_t u = __float_as_uint(top);
            // 448 = 1.75 2^8
            const int e2 = max((int)(u >> 23) - 127 - ((u & 0x7fffffu) <= 0x600000u ? 8 : 7), -100);
            const bool some = top < INFINITY;
            const float up = __uint_as_float((uint32_t)(127 - e2) << 23), s = __uint_as_float((uint32_t)(127 + e2) << 23);
            uint32_t code[2] = {0, 0};
            if (some) {
#pragma unroll
                for (int e = 0; e < kF; e += 2) code[e / 4] |= e4m3x2(y[e] * up, y[e + 1] * up) << (8 * (e % 4));
            }
            uint8_t* to = (key ? c.k : c.v) + g.b * c.sB + h * c.sH + (long long)slot * c.sS + f0;
            if (c.vec) {
                *reinterpret_cast<uint2*>(to) = make_uint2(code[0], code[1]);
            } else {
#pragma unroll
                for (int e = 0; e < kF; ++e) to[e] = (uint8_t)(code[e / 4] >> (8 * (e % 4)));
            }
            if (f0 == 0)
                (key ? c.ks : c.vs)[g.b * c.cB + h * c.cH + (long long)slot * c.cS] = some ? s : __uint_as_float(0x7fffffffu);
        }
        g = gn, l = ln, src = srcn, p = pn, t = tn, h = hn, slot = slot_next;
    }
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
    Work w;
    if (!work_for(a.B, std::min(a.T, a.cap), a.Hkv, 2 * a.d / kF, pl.n, &w)) return too_large(err);
    const size_t smem = 2 * (size_t)w.TN * pl.n * sizeof(float2);
    if (vec)
        append8_kernel<T, true><<<blocks_for(w), kT, smem, a.stream>>>(pl, kn, vn, c, pos, a.start, a.n_new, a.T, w, from);
    else
        append8_kernel<T, false><<<blocks_for(w), kT, smem, a.stream>>>(pl, kn, vn, c, pos, a.start, a.n_new, a.T, w, from);
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

template <typename C>
__device__ __forceinline__ void load8(const C* p, bool vec, float (&x)[kF]) {
    if constexpr (sizeof(C) == 1) {
        uint32_t w[2] = {0, 0};
        if (vec) {
            const uint2 u = *reinterpret_cast<const uint2*>(p);
            w[0] = u.x, w[1] = u.y;
        } else {
#pragma unroll
            for (int e = 0; e < kF; ++e) w[e / 4] |= (uint32_t)p[e].x << (8 * (e % 4));
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t h;
            const uint16_t two = (uint16_t)(w[i / 2] >> (16 * (i % 2)));
            asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(two));
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
            x[2 * i] = f.x, x[2 * i + 1] = f.y;
        }
    } else {
        to_f(vec ? load_raw<C, true>(p, 1) : load_raw<C, false>(p, 1), x);
    }
}
template <typename T>
__device__ __forceinline__ void store8(T* p, long long sJ, bool vec, const float (&x)[kF]) {
    if (vec) {
        constexpr int W = 16 / (int)sizeof(T);
#pragma unroll
        for (int i = 0; i < kF / W; ++i) {
            float y[W];
#pragma unroll
            for (int e = 0; e < W; ++e) y[e] = x[i * W + e];
            reinterpret_cast<uint4*>(p)[i] = pack<T>(y);
        }
    } else {
#pragma unroll
        for (int e = 0; e < kF; ++e) p[e * sJ] = from_f32<T>(x[e]);
    }
}

// A thread has 8 features of a position's key and value.
template <typename T, typename C, int D>
__global__ void __launch_bounds__(kT)
read_kernel(const __grid_constant__ ReadP a, int rows) {
    constexpr int U = D / kF;
    const long long idx = (long long)blockIdx.x * kT + threadIdx.x;
    if (idx >= (long long)rows * U) return;
    const int row = (int)(idx / U), f = (int)(idx % U) * kF;
    const int bh = divide(row, a.by_n), i = row - bh * a.N, b = divide(bh, a.by_h), h = bh - b * a.H;
    const long long L = max(__ldg(a.lens + b), 0), p = (long long)__ldg(a.first + b) + i;
    float k[kF], v[kF];
#pragma unroll
    for (int e = 0; e < kF; ++e) k[e] = v[e] = 0.f;
    if (p >= 0 && p < L && (p < a.sinks || p >= L - a.ring)) {
        const long long slot = p < a.sinks ? p : a.sinks + (int)(p - a.sinks) % a.ring;
        const long long at = b * a.sB + h * a.sH + slot * a.sS + f;
        float sk = 1.f, sv = 1.f;
        if constexpr (sizeof(C) == 1) {
            const long long sc = b * a.cB + h * a.cH + slot * a.cS;
            sk = __ldg(a.ks + sc), sv = __ldg(a.vs + sc);
        }
        load8<C>(static_cast<const C*>(a.k) + at, a.vec_in, k);
        load8<C>(static_cast<const C*>(a.v) + at, a.vec_in, v);
        if constexpr (sizeof(C) == 1) {
#pragma unroll
            for (int e = 0; e < kF; ++e) k[e] *= sk, v[e] *= sv;
        }
    }
    auto out = [&](const View& o, const float (&x)[kF]) {
        store8<T>(static_cast<T*>(const_cast<void*>(o.base)) + b * o.sB + h * o.sH + (long long)i * o.sN + f * o.sJ, o.sJ,
                  a.vec_out, x);
    };
    out(a.ko, k);
    out(a.vo, v);
}

template <typename T, typename C>
int launch_read(const ReadArgs& a, std::string* err) {
    const long long rows = (long long)a.B * a.Hkv * a.N, grid = (rows * (a.d / kF) + kT - 1) / kT;
    if (rows > 0x7fffffffll || grid > 0x7fffffffll) return too_large(err);
    ReadP p{a.k, a.v, a.ks, a.vs, a.sB, a.sH, a.sS, a.cB, a.cH, a.cS, a.ko, a.vo, a.first, a.lens, a.N, a.Hkv, a.sinks,
            a.cap - a.sinks, 0, 0, fast_div(a.N), fast_div(a.Hkv)};
    const long long W = sizeof(C) == 1 ? 8 : 16 / sizeof(C);
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
