// win_store.cu -- the rolling cache in 8 bits: rows quantised as they are written (keys
// rotated on the way), and caches of every type read back by position.
//
// A row x of d features becomes e4m3 codes and one scale s, the smallest power of two (from
// 2^-100 on) with max|x| <= 448 s: code = x / s rounded to e4m3.  A power of two because
// e4m3 is a floating format: a scale in between would move the codes' range, not their
// precision, and x / s as well as code * s are then exact in fp32, the latter in bf16 too.  So
// the code is the one rounding on the way (of the exact rotated key, but for 2^-27 of its pair)
// and does not depend on how a division is done.  A row with an element that is
// not finite has the scale NaN and codes 0.
//
// Every row is read and written once.  A lane has 8 features, d / 8 lanes a row, whose largest element
// goes round by shuffles; a rotation's other feature comes from the lane that has it.
// Bound by latency, not by memory (DRAM 13%): 4 prompts of 2048 tokens, 8 heads of 128, are written in
// 33 us from cold caches with issue active 59% and the ALU pipe 57% of the time; what the 24 warps an SM that their
// registers leave wait for most are shuffles and shared memory.
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
__device__ __forceinline__ uint32_t pack_lo(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// The exponent of a row's scale, of its largest element's bits: 448 = 1.75 2^8.  Elements that are
// not finite have one of their own.
__device__ __forceinline__ int scale_exponent(uint32_t top) {
    const int e = (int)(top >> 23) - 127 - ((top & 0x7fffffu) <= 0x600000u ? 8 : 7);
    return top >= 0x7f800000u ? 128 : max(e, -100);
}
// The codes of a row's 8 features in a lane (largest element first by all `lanes` of the row) to
// `to`, its scale by the row's first lane.  All lanes of a warp take part; `write`: this
// lane's row is there.  near: some y are off, those of this lane by at most `off` (0 or 2^-21) of the
// row's largest, and again() puts what is right to y; it is asked where that may decide a code or a scale.
template <typename Again>
__device__ __forceinline__ void quantise(float (&y)[kF], int lanes, bool write, uint8_t* to, bool vec, float* scale, bool near,
                                         float off, Again again) {
    auto largest = [&] {
        uint32_t top = 0;                         // as whole numbers: infinities and NaN are the largest
#pragma unroll
        for (int e = 0; e < kF; ++e) top = max(top, __float_as_uint(y[e]) & 0x7fffffffu);
        for (int i = 1; i < lanes; i <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, i));
        return top;
    };
    uint32_t top = largest();
    int e2 = scale_exponent(top);
    float up = __uint_as_float((uint32_t)(127 - min(e2, 120)) << 23);
    uint32_t code[2] = {0, 0};
    if (near) {
        // 8 steps of fp32, 2^-21 of the largest at least, from a border between scales or from infinity
        bool ask = off > 0.f && (((top - (0x600000u - 7)) & 0x7fffffu) < 16 || top >= 0x7f800000u - 8);
        uint32_t differ = 0;
        const float d = __uint_as_float(top) * up * off;
#pragma unroll
        for (int e = 0; e < kF; e += 2) {
            const uint32_t c = e4m3x2(fmaf(y[e], up, d), fmaf(y[e + 1], up, d));
            differ |= c ^ e4m3x2(fmaf(y[e], up, -d), fmaf(y[e + 1], up, -d));
            code[e / 4] |= c << (8 * (e % 4));
        }
        ask |= differ != 0;
        if (__any_sync(0xffffffffu, ask)) {
            again();
            top = largest(), e2 = scale_exponent(top);
            up = __uint_as_float((uint32_t)(127 - min(e2, 120)) << 23);
            near = false, code[0] = code[1] = 0;
        }
    }
    if (!near) {
#pragma unroll
        for (int e = 0; e < kF; e += 2) code[e / 4] |= e4m3x2(y[e] * up, y[e + 1] * up) << (8 * (e % 4));
    }
    const bool some = top < 0x7f800000u;
    if (!write) return;
    if (!some) code[0] = code[1] = 0;
    if (vec) {
        *reinterpret_cast<uint2*>(to) = make_uint2(code[0], code[1]);
    } else {
#pragma unroll
        for (int e = 0; e < kF; ++e) to[e] = (uint8_t)(code[e / 4] >> (8 * (e % 4)));
    }
    if (scale) *scale = __uint_as_float(some ? (uint32_t)(127 + e2) << 23 : 0x7fffffffu);
}

// Rotated keys: a code is what the exact product rounds to, over the scale of the exact row.  An fp32
// rotation is off by some 2^-23 of |x1| + |x2|, which takes one code in about 10^6 to its other neighbour
// and one row in some 10^6 to the next scale; where it can, the key is computed in two fp32 numbers (4 prompts of 2048 tokens, 8 heads of 128, written and read back: 39 us
// without, 44 this way, 62 with every key computed so).
struct Pair {
    float h, l;                                   // h + l, l small
};
__device__ __forceinline__ Pair mul(Pair a, Pair b) {
    const float h = __fmul_rn(a.h, b.h);
    return Pair{h, fmaf(a.h, b.l, fmaf(a.l, b.h, fmaf(a.h, b.h, -h)))};
}
__device__ __forceinline__ Pair sum(float a, float b) {   // |a| >= |b|
    const float h = __fadd_rn(a, b);
    return Pair{h, __fsub_rn(b, __fsub_rn(h, a))};
}
// Cosine and sine of p times pair i's turn, off by 2^-27 at most: of the rest of the nearest quarter
// turn, |x| <= pi / 4, by their Taylor series, the first two terms of each in pairs.
struct Turn {
    float c, s;
    uint32_t lo;                                  // what c and s leave, as bf16
};
__device__ __forceinline__ Turn turn_of(const Plan& pl, int i, int p) {
    const unsigned long long t = (unsigned long long)(long long)p * pl.turn[i], q = (t + (1ull << 61)) >> 62;
    const long long r = (long long)(t - (q << 62));
    const int top = (int)(r >> 32);
    const float rh = (float)top, rl = (float)(top - (int)rh) + (float)(uint32_t)r * 0x1p-32f;
    // 2 pi and 1 / 6 as pairs
    const Pair x = mul(Pair{rh * 0x1p-32f, rl * 0x1p-32f}, Pair{6.28318548f, -1.74845553e-7f});
    const Pair x2 = mul(x, x), x3 = mul(x, mul(x2, Pair{0.166666672f, -4.96705379e-9f}));
    const float y = x2.h;
    const float s5 = x.h * y * y * fmaf(y, fmaf(y, fmaf(y, -1.f / 39916800.f, 1.f / 362880.f), -1.f / 5040.f), 1.f / 120.f);
    const float c4 = y * y * fmaf(y, fmaf(y, fmaf(y, -1.f / 3628800.f, 1.f / 40320.f), -1.f / 720.f), 1.f / 24.f);
    Pair s = sum(x.h, -x3.h), c = sum(1.f, -0.5f * y);
    s = sum(s.h, s.l + (x.l - x3.l + s5));
    c = sum(c.h, c.l + (c4 - 0.5f * x2.l));
    if (q & 1) {
        const Pair z = c;
        c = Pair{-s.h, -s.l}, s = z;
    }
    if (q & 2) c = Pair{-c.h, -c.l}, s = Pair{-s.h, -s.l};
    return Turn{c.h, s.h, pack_lo(c.l, s.l)};
}
__device__ __forceinline__ Turn back(Turn w) { return Turn{w.c, -w.s, w.lo ^ 0x80000000u}; }
// a c - z s.  Where fp32 has it on a tie between codes, the rest decides.
__device__ __forceinline__ float turned(float a, float z, const Turn& w) {
    const float p = __fmul_rn(a, w.c), q = __fmul_rn(z, w.s), y = __fsub_rn(p, q), b = __fsub_rn(y, p);
    const float rest = __fsub_rn(__fsub_rn(p, __fsub_rn(y, b)), __fadd_rn(q, b)) + (fmaf(a, w.c, -p) - fmaf(z, w.s, -q)) +
                       fmaf(a, __uint_as_float(w.lo << 16), -(z * __uint_as_float(w.lo & 0xffff0000u)));
    const float r = __fadd_rn(y, rest), left = __fadd_rn(__fsub_rn(y, r), rest);
    uint32_t bits = __float_as_uint(r);
    if ((bits & 0x7ffffu) == 0 && left != 0.f && r != 0.f) bits += (left > 0.f) == (r > 0.f) ? 1u : ~0u;
    return __uint_as_float(bits);
}

// A warp per token and `hper` heads, a half for keys and a half for values: its angles once (two
// a lane, through shared memory), then head after head, the next one's loads on their way.
// No barriers between warps.  16-byte loads; a rotation's partners are at the same place of
// another lane, or in the lane.  Three blocks an SM, whose 80 registers a thread leave some 50 bytes in
// local memory (44 us); two keep all in registers (47), four leave 64 of them (50).
template <typename T, int D>
__global__ void __launch_bounds__(kT, 3)
append8_kernel(const __grid_constant__ Plan pl, const __grid_constant__ Rows kn, const __grid_constant__ Rows vn,
               const __grid_constant__ Cache8 c, Pos pos, const int* __restrict__ start, const int* __restrict__ n_new, int Tn,
               int N, int H, int hper, int parts, int tasks, FastDiv by_parts, FastDiv by_n, Picked from) {
    constexpr int LANES = D / kF, SUB = 32 / (2 * LANES);   // lanes of a row; heads at a time
    __shared__ Turn cs_all[kT / 32][PSA_ROPE_MAX_PAIRS];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, q = lane % (2 * LANES), sub = lane / (2 * LANES);
    const bool key = q < LANES;
    const int f0 = (key ? q : q - LANES) * kF, n = pl.n;
    const Rows& mine = key ? kn : vn;
    Turn* cs = cs_all[warp];
    // the lane's first pair, and the lane that has its other features
    const bool turns = key && f0 < 2 * n, first = f0 < n;
    const int p0 = pl.interleaved ? f0 / 2 : first ? f0 : f0 - n;
    const int other = turns && !pl.interleaved ? lane + (first ? n / kF : -n / kF) : lane;
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
        for (int i = lane; i < n; i += 32) cs[i] = turn_of(pl, i, load_pos(pl, pos, i, b, x));
        __syncwarp();
        float2 w[kF];
#pragma unroll
        for (int e = 0; e < kF; ++e) {
            w[e] = turns && (e < 4 || !pl.interleaved) ? make_float2(cs[p0 + e].c, cs[p0 + e].s) : make_float2(1.f, 0.f);
            if (!first && !pl.interleaved) w[e].y = -w[e].y;
        }
        // c, s, the products and the sum: (2^-25 + 2^-27 + 2^-24 + 2^-24) (|x1| + |x2|), which is at most
        // twice the row's largest
        const float off = turns ? 0x1p-21f : 0.f;
        for (int hh = h0; hh < h1; hh += SUB) {
            const int h = hh + sub;
            if (h + SUB < h1) ln = load_raw<T, true>(src + (h + SUB) * mine.sH, 1);
            float y[kF];
            to_f(l, y);
            auto partners = [&](float (&o)[kF]) {    // exchanged as they lie in memory
                Raw<T> ro;
#pragma unroll
                for (int i = 0; i < (int)(sizeof(ro) / 16); ++i)
                    ro.u[i] = make_uint4(__shfl_sync(0xffffffffu, l.u[i].x, other), __shfl_sync(0xffffffffu, l.u[i].y, other),
                                         __shfl_sync(0xffffffffu, l.u[i].z, other), __shfl_sync(0xffffffffu, l.u[i].w, other));
                to_f(ro, o);
            };
            auto interleaved = [&](auto&& turn) {     // turn(first of a pair, second, number of the pair)
#pragma unroll
                for (int e = 0; e < kF; e += 2)
                    if (f0 + e < 2 * n) turn(e, e + 1, e / 2);
            };
            if (n > 0) {
                float o[kF];
                if (!pl.interleaved) partners(o);
                if (turns && pl.interleaved) {
                    interleaved([&](int i, int j, int x) {
                        const float a = y[i], z = y[j];
                        y[i] = fmaf(a, w[x].x, -(z * w[x].y));
                        y[j] = fmaf(z, w[x].x, a * w[x].y);
                    });
                } else if (turns) {
#pragma unroll
                    for (int e = 0; e < kF; ++e) y[e] = fmaf(y[e], w[e].x, -(o[e] * w[e].y));
                }
            }
            quantise(y, LANES, h < h1, to + h * c.sH, c.vec, f0 == 0 ? scale + h * c.cH : nullptr, n > 0, off, [&] {
                to_f(l, y);
                float o[kF];
                if (!pl.interleaved) partners(o);
                if (turns && pl.interleaved) {
                    interleaved([&](int i, int j, int x) {
                        const float a = y[i], z = y[j];
                        y[i] = turned(a, z, cs[p0 + x]);
                        y[j] = turned(z, a, back(cs[p0 + x]));
                    });
                } else if (turns) {
#pragma unroll
                    for (int e = 0; e < kF; ++e) y[e] = turned(y[e], o[e], first ? cs[p0 + e] : back(cs[p0 + e]));
                }
            });
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
                    const Turn w = turn_of(pl, i, load_pos(pl, pos, i, b, x));
                    y[e] = turned(y[e], z, first ? w : back(w));
                }
            }
            to = (key ? c.k : c.v) + b * c.sB + h * c.sH + slot * c.sS + f0;
            if (f0 == 0) scale = (key ? c.ks : c.vs) + b * c.cB + h * c.cH + slot * c.cS;
        }
    }
    quantise(y, lanes, write, to, c.vec, scale, false, 0.f, [] {});
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
