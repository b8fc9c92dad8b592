// win_tree_warp.cuh -- attention of new tokens (a tree of drafts, a run of tokens,
// or a single token that is in the cache already) over the rolling key/value
// cache, on warp-level matrix products.
//
//   s_x = c sk_x q.k_x (log2 units), O = sum_x e_x sv_x v_x / sum_x e_x, e_x = exp2(s_x - m)
// over the cached positions x = 0 .. nv-1 that the row sees, in slot order of the
// sinks, then the window, and over the drafts that are its ancestors or itself;
// sk, sv: an 8-bit cache's scales (1 elsewhere).
//
// The query heads of a key head and the T new tokens are the rows of the products
// (row t G + g), so a cached key or value is read from memory once for all of them.
// A block of four warps takes a run of keys and 16, 32 or 64 rows (WR = 1, 2, 4; 8 rows, WR = 0,
// over an 8-bit cache, with the products turned round, see Cols): WR
// warps, 16 rows each, are a team and share tiles of keys, the 4 / WR teams take
// tiles of their own and are joined at the end.  A team keeps its tiles in flight in
// shared memory (cp.async) and waits for nobody else.
//
// Products by type of query and cache:
//   bf16, bf16   m16n8k16 on bf16; P is rounded to bf16 (its sum is not)
//   bf16, e4m3   m16n8k16 on fp16, which holds every e4m3 number; q exactly too, scaled by
//                a power of two per row (down to 2^-31 of the row's largest element).  O has a
//                reference u of its own, which follows s + log2 sv: exp2(s + log2 sv - u) <= 2^8
//                is rounded to fp16 at 11 bits, and a row's sum keeps to m whatever the values' sizes
//   fp32, fp32   m16n8k8 on tf32, each operand in two parts, three products; a few products at
//                a time, which the tensor cores add with truncation, the rest as fp32 sums
//   fp32, e4m3   the same with two products: an e4m3 number is one tf32 part
//
// The runs of one (sequence, key head, row group) are joined in a fixed order: up to
// 8 of them form a cluster and read each other's results through distributed shared
// memory; more leave partial results in the workspace for a second kernel.
//
// Bound, over 8-bit caches (64 tokens of 32 / 8 heads, d = 128, over 4100 slots: 108 us, 5150 GB/s of
// 6795): by latency; DRAM is busy 63%, issue 41%, the ALU pipe with the codes' conversion 38% (65 pairs a
// cycle and SM), with the 12 warps an SM that 168 registers leave.  fp32 (2 trees of 17
// drafts, 4 heads, d = 32, window 333: 13.0 us): by the chain of one block, whose code and tiles
// leave room for no second one an SM.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <string>
#include <type_traits>

#include "common.cuh"
#include "tc_ptx.cuh"
#include "tc_tmap.h"
#include "win_geom.cuh"
#include "win_internal.h"

namespace psa {
namespace win {
namespace tk {

using bf16 = __nv_bfloat16;
struct e4m3 {
    uint8_t x;
};

constexpr int kWarps = 4, kT = 32 * kWarps, kCluster = 8;
constexpr float kMove = 8.f;                      // a stale maximum stays while the new one is at most 2^8 larger

struct P {
    const void* k;
    const void* v;
    const float* ks;                              // e4m3: scales
    const float* vs;
    long long sB, sH, sS, cB, cH, cS;             // cache strides, scale strides
    View q, o, kn, vn;
    float* lse;                                   // [B, Hq, T] or NULL
    const int* lens;
    const int* n_new;                             // NULL: T
    const int* parents;                           // NULL: each token's parent is the one before it
    long long par_stride;
    float* part;                                  // more than kCluster splits: [groups][splits][rows][d + 2]
    int Hq, Hkv, G, T, rgroups, cap, window, sinks, splits, vec, vec_new, drafts;
    float c;
    FastDiv by_g;
};

// Rows of CT in shared memory.
template <typename CT, int D>
struct Lay {
    static constexpr bool is8 = std::is_same<CT, e4m3>::value;
    static constexpr int E = (int)sizeof(CT), CH = D * E / 16, ROWB = D * E;
    // Chunk ch (16 bytes) of row r.  Eight rows' chunks at one ch lie in different banks
    // (ldmatrix), and so do four neighbouring chunks of rows 2i and 2i + 1 (16-byte reads
    // of e4m3 and fp32 keys).
    static __device__ __forceinline__ int at(int r, int ch) {
        const int s = E == 2 ? r & 7 : ((r & 1) << 2) | ((r >> 1) & 3);
        return 16 * (CH >= 8 ? r * CH + (ch ^ s) : r * CH + (ch ^ ((r / (8 / CH)) & (CH - 1))));
    }
    // fp32 values: rows 2t of two neighbouring chunks in different banks
    static __device__ __forceinline__ int at_v(int r, int ch) {
        return E == 4 && CH >= 8 ? 16 * (r * CH + (ch ^ ((r & 6) ^ ((r & 1) << 2)))) : at(r, ch);
    }
};
template <typename QT, typename CT, int D, int WR>
struct Cfg : Lay<CT, D> {
    using L = Lay<CT, D>;
    static constexpr int KS = sizeof(QT) == 2 ? 32 : 16;   // keys of a step of a warp
    static constexpr int TW = WR ? WR : 1;        // warps of a team
    static constexpr int KT = 16 * WR > KS ? 16 * WR : KS, WK = kWarps / TW, ROWS = WR ? 16 * WR : 8;
    static constexpr int TILE = KT * L::ROWB, STAGE = 2 * TILE + (L::is8 ? 8 * KT : 0);
    static constexpr int NST = L::is8 ? (sizeof(QT) == 2 ? (WR <= 1 ? 2 : 3) : 6) : 3;
    static constexpr int TEAM = NST * STAGE, PIPE = WK * TEAM;
    static constexpr bool TWO = L::is8 && sizeof(QT) == 2;   // O has a reference of its own
    static constexpr int RN = ROWS * (D + 2);     // floats of a result: O [ROWS][D] (TWO: over its l), m, l
    static constexpr int ALL = WK * RN * 4, OFF_RES = WK > 1 ? ALL : 0;
    static constexpr int USED = OFF_RES + RN * 4;
    static constexpr int MAIN = ((PIPE > USED ? PIPE : USED) + 15) / 16 * 16;
    // blocks per SM that registers are kept for (their tiles leave room for as many)
    static constexpr int BLOCKS = sizeof(QT) == 2 && MAIN <= 74 * 1024 ? 3 : 1;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool full) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(full ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, bool full) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(full ? 4 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm_x4(uint32_t (&r)[4], uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(a)
                 : "memory");
}
__device__ __forceinline__ void ldsm_x4_t(uint32_t (&r)[4], uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(a)
                 : "memory");
}
__device__ __forceinline__ void ldsm_x2_t(uint32_t& r0, uint32_t& r1, uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x2.trans.shared.b16 {%0, %1}, [%2];" : "=r"(r0), "=r"(r1) : "r"(a) : "memory");
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_tf32(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void add4(float (&d)[4], const float (&x)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) d[i] += x[i];
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// A row's factor times a key's scale, which may pass fp32's range where a score does not: 0 times an
// infinity is no 0.
__device__ __forceinline__ float factor(float c, float sk) {
    float f;
    asm("min.NaN.xorsign.abs.f32 %0, %1, %2;" : "=f"(f) : "f"(c * sk), "f"(0x1.fffffep127f));
    return f;
}
// A reference that follows a row's largest x; what was weighed against it is scaled by `by`.
__device__ __forceinline__ bool follow(float x, float& ref, float& by) {
    const bool move = x > ref + kMove;
    by = move ? ex2(ref - x) : 1.f;
    if (move) ref = x;
    return move;
}
__device__ __forceinline__ float finite_ref(float m) { return m == -INFINITY ? 0.f : m; }
// 2^((u - m) / 2), twice a factor of O: 2^(u - m) itself may pass fp32's range.  Without keys u = m.
__device__ __forceinline__ float half_unit(float u, float m) { return u == m ? 1.f : ex2(0.5f * (u - m)); }
__device__ __forceinline__ float inverse_or_0(float l) { return l != 0.f ? 1.f / l : 0.f; }
// Two e4m3 numbers (the lower byte first) as fp16.
__device__ __forceinline__ uint32_t f16_of_e4m3(uint32_t lo16) {
    uint32_t y;
    asm("{\n\t.reg .b16 t, u;\n\tmov.b32 {t, u}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}" : "=r"(y) : "r"(lo16));
    return y;
}
__device__ __forceinline__ uint32_t f16_of_e4m3_hi(uint32_t hi16) {
    uint32_t y;
    asm("{\n\t.reg .b16 t, u;\n\tmov.b32 {t, u}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, u;\n\t}" : "=r"(y) : "r"(hi16));
    return y;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float2 f32_of_f16x2(uint32_t x) { return __half22float2(*reinterpret_cast<const __half2*>(&x)); }
// x as the sum of two tf32 numbers, the first rounded (the largest finite fp32 numbers would
// round to an infinity, so it is held below it; PROB: not that large), the rest to 2^-22 of x.
template <bool PROB = false>
__device__ __forceinline__ void split_tf32(float x, uint32_t& hi, uint32_t& lo) {
    float y = x;
    if (!PROB) asm("min.xorsign.abs.f32 %0, %1, %2;" : "=f"(y) : "f"(x), "f"(0x1.ffdffep127f));
    hi = (__float_as_uint(y) + 0x1000u) & 0xffffe000u;
    lo = __float_as_uint(x - __uint_as_float(hi)) & 0xffffe000u;
}

// Visible position x of a sequence -> its slot.
struct Slots {
    int nv, sinks, r0, ring;
    __device__ __forceinline__ int of(int x) const {
        if (x < sinks) return x;
        const int r = r0 + x - sinks;             // < 2 ring
        return sinks + (r >= ring ? r - ring : r);
    }
};
// drafts = 1: the rows come behind position L - 1, so that they see at most window - 1 cached
// positions besides the sinks
__device__ __forceinline__ Slots load_slots(const P& a, int L) {
    Slots s;
    s.sinks = a.sinks;
    s.ring = a.cap - a.sinks;
    s.nv = (int)min((long long)L, (long long)a.sinks + a.window - a.drafts);   // <= capacity
    s.r0 = (L - s.nv) % s.ring;
    return s;
}

// ------------------------------------------------------------------ ancestors
// Bits of every node's ancestors and itself, nw words a node, by doubling: jump[t] is the
// nearest ancestor whose bit is not set yet.  A parent that is not below its node counts
// as none.  All kT threads; n <= PSA_TREE_MAX.
__device__ __forceinline__ void ancestors(const int* __restrict__ par, int n, int nw, uint32_t* anc, int* jump) {
    constexpr int MAXI = PSA_TREE_MAX * (PSA_TREE_MAX / 32) / kT, MAXN = PSA_TREE_MAX / kT;
    for (int t = threadIdx.x; t < n; t += kT) {
        const int p = __ldg(par + t);
        jump[t] = p >= 0 && p < t ? p : -1;
    }
    for (int i = threadIdx.x; i < n * nw; i += kT) {
        const int t = i / nw, w = i - t * nw;
        anc[i] = t >> 5 == w ? 1u << (t & 31) : 0u;
    }
    __syncthreads();
    for (;;) {
        uint32_t a[MAXI];
        int j[MAXN];
        bool more = false;
#pragma unroll
        for (int u = 0; u < MAXI; ++u) {
            const int i = threadIdx.x + u * kT;
            a[u] = 0;
            if (i < n * nw) {
                const int t = i / nw, at = jump[t];
                if (at >= 0) a[u] = anc[at * nw + i - t * nw];
            }
        }
#pragma unroll
        for (int u = 0; u < MAXN; ++u) {
            const int t = threadIdx.x + u * kT;
            j[u] = -1;
            if (t < n && jump[t] >= 0) j[u] = jump[jump[t]];
            more |= j[u] >= 0;
        }
        __syncthreads();
#pragma unroll
        for (int u = 0; u < MAXI; ++u) {
            const int i = threadIdx.x + u * kT;
            if (i < n * nw) anc[i] |= a[u];
        }
#pragma unroll
        for (int u = 0; u < MAXN; ++u) {
            const int t = threadIdx.x + u * kT;
            if (t < n) jump[t] = j[u];
        }
        if (!__syncthreads_or(more)) return;
    }
}

// ------------------------------------------------------------------ loads
// Keys [x0, x0 + KT) and their values to a stage; rows past x1 are zero.
template <typename QT, typename CT, int D, int WR>
__device__ __forceinline__ void load_rows(const P& a, const Slots& s, long long head, long long shead, uint32_t st, uint8_t* stp,
                                          int x0, int x1, int tl) {
    using C = Cfg<QT, CT, D, WR>;
    const CT *K = static_cast<const CT*>(a.k) + head, *V = static_cast<const CT*>(a.v) + head;
    constexpr int LANES = 32 * C::TW, N = C::KT * C::CH;         // chunks of 16 bytes
    const int s0 = s.of(x0);
    // a whole tile in neighbouring slots
    const bool run = x0 + C::KT <= x1 && s.of(x0 + C::KT - 1) == s0 + C::KT - 1;
    if (a.vec && run && C::CH <= LANES && LANES % C::CH == 0) {
        constexpr int R = C::CH <= LANES ? LANES / C::CH : 1;    // rows at a time
        const int r = tl / C::CH, ch = tl % C::CH;
        const long long g = (long long)(s0 + r) * a.sS + ch * (16 / C::E), by = (long long)R * a.sS;
        const CT *k = K + g, *v = V + g;
#pragma unroll
        for (int i = 0; i < (N + LANES - 1) / LANES; ++i) {
            if (N % LANES && tl + i * LANES >= N) break;
            cp_async16(st + C::at(r + i * R, ch), k, true);
            cp_async16(st + C::TILE + C::at_v(r + i * R, ch), v, true);
            k += by, v += by;
        }
    } else if (a.vec) {
#pragma unroll 2
        for (int i = tl; i < N; i += LANES) {
            const int r = i / C::CH, ch = i % C::CH, x = x0 + r;
            const bool in = x < x1;
            const long long g = (long long)(in ? s.of(x) : s0) * a.sS + ch * (16 / C::E);
            cp_async16(st + C::at(r, ch), K + g, in);
            cp_async16(st + C::TILE + C::at_v(r, ch), V + g, in);
        }
    } else {                                      // rows that are not 16-byte aligned: element by element
        constexpr int E = 16 / C::E;
        for (int i = tl; i < C::KT * D; i += LANES) {
            const int r = i / D, e = i % D, x = x0 + r;
            CT kv{}, vv{};
            if (x < x1) {
                const long long g = (long long)s.of(x) * a.sS + e;
                kv = K[g], vv = V[g];
            }
            reinterpret_cast<CT*>(stp + C::at(r, e / E))[e % E] = kv;
            reinterpret_cast<CT*>(stp + C::TILE + C::at_v(r, e / E))[e % E] = vv;
        }
    }
    if constexpr (C::is8) {                       // K's scales, then V's
#pragma unroll
        for (int i = tl; i < 2 * C::KT; i += LANES) {
            const int r = i % C::KT, x = x0 + r;
            const long long at = shead + (long long)(run ? s0 + r : s.of(x < x1 ? x : x0)) * a.cS;
            cp_async4(st + 2 * C::TILE + 4 * i, (i < C::KT ? a.ks : a.vs) + at, x < x1);
        }
    }
}

// 16 new keys and values [j0, j0 + 16) of n to a tile of QT rows at `to` (V behind K); rows
// past n are zero.  PERM: values with a 16-feature block's even features before its odd ones.
template <typename QT, int D, bool PERM, int LANES>
__device__ __forceinline__ void load_new(const P& a, int b, int hk, uint8_t* to, int j0, int n, int tl) {
    using C = Lay<QT, D>;
    constexpr int TILE = 16 * C::ROWB;
    constexpr int E = (int)sizeof(QT), U = 16 * E / 16;          // 16-byte chunks of a unit of 16 features
#pragma unroll 1
    for (int i = tl; i < 2 * 16 * (D / 16); i += LANES) {
        const int u = i % (D / 16), r = i / (D / 16) % 16, which = i / (D / 16) / 16;
        const View& v = which ? a.vn : a.kn;
        const QT* p = static_cast<const QT*>(v.base) + b * v.sB + hk * v.sH + (long long)(j0 + r) * v.sN + 16 * u * v.sJ;
        union {
            QT x[16];
            uint4 w[U];
        } d;
#pragma unroll
        for (int e = 0; e < U; ++e) d.w[e] = make_uint4(0, 0, 0, 0);
        if (j0 + r < n) {
            if (a.vec_new) {
#pragma unroll
                for (int e = 0; e < U; ++e) d.w[e] = reinterpret_cast<const uint4*>(p)[e];
            } else {
#pragma unroll
                for (int e = 0; e < 16; ++e) d.x[e] = p[e * v.sJ];
            }
        }
        if (PERM && E == 2 && which) {
            uint32_t* w = reinterpret_cast<uint32_t*>(d.w);
            uint32_t ev[4], od[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) ev[e] = __byte_perm(w[2 * e], w[2 * e + 1], 0x5410), od[e] = __byte_perm(w[2 * e], w[2 * e + 1], 0x7632);
            d.w[0] = make_uint4(ev[0], ev[1], ev[2], ev[3]);
            d.w[U - 1] = make_uint4(od[0], od[1], od[2], od[3]);
        }
#pragma unroll
        for (int e = 0; e < U; ++e) {
            const int ch = u * U + e;
            *reinterpret_cast<uint4*>(to + (which ? TILE + C::at_v(r, ch) : C::at(r, ch))) = d.w[e];
        }
    }
}

// ------------------------------------------------------------------ a warp's 16 rows
// Row i of the pair a lane works on is row g + 8 i, g = lane / 4.
template <typename QT, typename CT, int D>
struct Rows {
    static constexpr bool is8 = std::is_same<CT, e4m3>::value, f32 = sizeof(QT) == 4;
    // O tiles of 8 features: features 8 n + col, or, PERM, the even (n even) and odd ones of
    // the 16-feature block n / 2
    static constexpr bool PERM = is8 || f32, TWO = is8 && !f32;
    static constexpr int QN = f32 ? D / 2 : D / 4;
    static constexpr int KS = f32 ? 16 : 32;      // cached keys of a step
    // the rows that a lane weighs, and those whose queries it has (the same ones)
    static __device__ __forceinline__ int row(int i, int lane) { return (lane >> 2) + 8 * i; }
    static __device__ __forceinline__ int query(int i, int lane) { return row(i, lane); }
    uint32_t q[QN];                               // bf16/fp16: [D / 16][4]; fp32: [D / 8][4]
    float o[D / 8][4], m[2], l[2], u[2], c[2];    // u: TWO, O's reference; c: the row's factor of q.k

    // feature of (k-step s, k index 0 or 1 of the lane's pair, or 0..3 of its four), fp32
    static __device__ __forceinline__ int feat32(int s, int t, int e) {
        constexpr int W = is8 ? (D >= 64 ? 16 : D / 4) : 4;      // neighbouring features per lane
        constexpr int PER = W / 2;                               // k-steps that they fill
        return s / PER * 4 * W + t * W + s % PER * 2 + e;
    }
    // e4m3 with fp16: the lane's four features of k-step s
    static __device__ __forceinline__ int feat8(int s, int t) {
        constexpr int W = D >= 64 ? 16 : D / 4;
        constexpr int PER = W / 4;
        return s / PER * 4 * W + t * W + s % PER * 4;
    }

    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int n = 0; n < D / 8; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[n][i] = 0.f;
        m[0] = m[1] = u[0] = u[1] = -INFINITY;
        l[0] = l[1] = 0.f;
    }
    // bf16 queries as operands of bf16 products
    __device__ __forceinline__ void load_bf16(const uint16_t* const (&row)[2], long long sJ, float cc, int lane) {
        const int t = lane & 3;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint16_t* p = row[i & 1];
                const int k = 16 * kk + 2 * t + 8 * (i >> 1);
                q[4 * kk + i] = p ? (uint32_t)p[k * sJ] | ((uint32_t)p[(k + 1) * sJ] << 16) : 0u;
            }
        c[0] = c[1] = cc;
    }
    __device__ __forceinline__ void load(const void* const (&rows)[2], long long sJ, float cc, int lane) {
        const int t = lane & 3;
        if constexpr (f32) {
#pragma unroll
            for (int s = 0; s < D / 8; ++s)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float* p = static_cast<const float*>(rows[i & 1]);
                    q[4 * s + i] = p ? __float_as_uint(p[feat32(s, t, i >> 1) * sJ]) : 0u;
                }
            c[0] = c[1] = cc;
        } else if constexpr (!is8) {
            const uint16_t* const r[2] = {static_cast<const uint16_t*>(rows[0]), static_cast<const uint16_t*>(rows[1])};
            load_bf16(r, sJ, cc, lane);
        } else {
            // to fp16, the row's largest element scaled to 2^7 .. 2^8
            float top[2] = {0.f, 0.f};
            uint32_t raw[QN];
#pragma unroll
            for (int s = 0; s < D / 16; ++s)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint16_t* p = static_cast<const uint16_t*>(rows[i & 1]);
                    const int k = feat8(s, t) + 2 * (i >> 1);
                    const uint32_t x = p ? (uint32_t)p[k * sJ] | ((uint32_t)p[(k + 1) * sJ] << 16) : 0u;
                    raw[4 * s + i] = x;
                    top[i & 1] = fmaxf(top[i & 1], fmaxf(fabsf(__uint_as_float(x << 16)), fabsf(__uint_as_float(x & 0xffff0000u))));
                }
            float up[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], 1));
                top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], 2));
                const int e = max((int)(__float_as_uint(top[i]) >> 23) - 127, -100);   // floor(log2 top)
                up[i] = __uint_as_float((uint32_t)(127 + 7 - e) << 23);
                c[i] = cc * __uint_as_float((uint32_t)(127 - 7 + e) << 23);
            }
#pragma unroll
            for (int s = 0; s < D / 16; ++s)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t x = raw[4 * s + i];
                    q[4 * s + i] = pack_f16x2(__uint_as_float(x << 16) * up[i & 1], __uint_as_float(x & 0xffff0000u) * up[i & 1]);
                }
        }
    }

    // Scores of KS keys at ks, from the cache: s[n][i], column 8 n + 2 t + (i & 1), row i >> 1.
    __device__ __forceinline__ void scores(float (&s)[KS / 8][4], uint32_t ks, const uint8_t* ksp, int r0, int lane) const {
        using C = Lay<CT, D>;
        const int g = lane >> 2, t = lane & 3;
        if constexpr (f32 && !is8) {
            scores_f32<CT>(s, ksp, r0, lane);
        } else if constexpr (!is8) {
            scores_bf16(s, ks, r0, lane);
        } else {
            constexpr int W = D >= 64 ? 16 : D / 4;              // bytes per lane and read
#pragma unroll
            for (int j = 0; j < D / (4 * W); ++j) {
#pragma unroll
                for (int n = 0; n < KS / 8; ++n) {
                    const int r = r0 + 8 * n + g, f = 4 * W * j + W * t;
                    const uint8_t* p = ksp + C::at(r, f / 16) + f % 16;
                    uint32_t w[W / 4];
                    if constexpr (W == 16) {
                        const uint4 x = *reinterpret_cast<const uint4*>(p);
                        w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
                    } else if constexpr (W == 8) {
                        const uint2 x = *reinterpret_cast<const uint2*>(p);
                        w[0] = x.x, w[1] = x.y;
                    } else {
                        w[0] = *reinterpret_cast<const uint32_t*>(p);
                    }
#pragma unroll
                    for (int e = 0; e < W / 4; ++e) {
                        const uint32_t b0 = f16_of_e4m3(w[e]), b1 = f16_of_e4m3_hi(w[e]);
                        if constexpr (!f32) {
                            uint32_t a[4];
#pragma unroll
                            for (int i = 0; i < 4; ++i) a[i] = q[4 * (j * (W / 4) + e) + i];
                            mma_f16(s[n], a, b0, b1);
                        } else {
                            const float2 x0 = f32_of_f16x2(b0), x1 = f32_of_f16x2(b1);
                            float part[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                uint32_t hi[4], lo[4];
#pragma unroll
                                for (int i = 0; i < 4; ++i)
                                    split_tf32(__uint_as_float(q[4 * (j * (W / 2) + 2 * e + h) + i]), hi[i], lo[i]);
                                const uint32_t y0 = __float_as_uint(h ? x1.x : x0.x), y1 = __float_as_uint(h ? x1.y : x0.y);
                                mma_tf32(part, lo, y0, y1);
                                mma_tf32(part, hi, y0, y1);
                            }
                            add4(s[n], part);
                        }
                    }
                }
            }
        }
    }
    template <int NT>
    __device__ __forceinline__ void scores_bf16(float (&s)[NT][4], uint32_t ks, int r0, int lane) const {
        using C = Lay<bf16, D>;
        const int kr = r0 + (lane & 7) + ((lane >> 4) << 3), kc = (lane >> 3) & 1;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
            uint32_t a[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) a[i] = q[4 * kk + i];
#pragma unroll
            for (int n = 0; n < NT; n += 2) {
                uint32_t b[4];
                ldsm_x4(b, ks + C::at(kr + 8 * n, 2 * kk + kc));
                mma_bf16(s[n], a, b[0], b[1]);
                mma_bf16(s[n + 1], a, b[2], b[3]);
            }
        }
    }
    // fp32 keys, by the features of the lane's queries (which are those of the cache's type)
    template <typename Map>
    __device__ __forceinline__ void scores_f32(float (&s)[2][4], const uint8_t* ksp, int r0, int lane) const {
        using C = Lay<float, D>;
        const int g = lane >> 2, t = lane & 3;
#pragma unroll
        for (int j = 0; j < D / 16; ++j) {                       // two k-steps: four neighbouring features
            const int f = feat32(2 * j, t, 0);
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                const float4 x = *reinterpret_cast<const float4*>(ksp + C::at(r0 + 8 * n + g, f / 4));
                float part[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t hi[4], lo[4], b0h, b0l, b1h, b1l;
#pragma unroll
                    for (int i = 0; i < 4; ++i) split_tf32(__uint_as_float(q[4 * (2 * j + h) + i]), hi[i], lo[i]);
                    split_tf32(h ? x.z : x.x, b0h, b0l);
                    split_tf32(h ? x.w : x.y, b1h, b1l);
                    mma_tf32(part, lo, b0h, b1h);
                    mma_tf32(part, hi, b0l, b1l);
                    mma_tf32(part, hi, b0h, b1h);
                }
                add4(s[n], part);
            }
        }
    }

    // Masked scores in log2 units to weights (in s: e_x sv_x, TWO: in units of 2^u); m, l, u and O
    // are moved along.  sv: the columns' scales (SV), by n and i & 1.  TWO: the scale's logarithm, off by
    // 2^-22 of itself, goes into the exponent: at most 2^-15 of a weight, of which fp16 keeps 2^-12; a
    // product e_x sv_x 2^(m - u) instead (106 us for 108) passes fp32's range on the way.
    template <bool SV, int NT>
    __device__ __forceinline__ void weights(float (&s)[NT][4], const float (&sv)[NT][2]) {
        float mx[2] = {-INFINITY, -INFINITY}, ux[2] = {-INFINITY, -INFINITY}, ls[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                ls[n][e] = SV && TWO ? __log2f(sv[n][e]) : 0.f;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    mx[i] = fmaxf(mx[i], s[n][2 * i + e]);
                    if (SV && TWO) ux[i] = fmaxf(ux[i], s[n][2 * i + e] + ls[n][e]);
                }
            }
        bool move = false;
        float al[2];                              // of O
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 1));
            mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 2));
            float by;
            const bool mv = follow(mx[i], m[i], by);
            l[i] *= by;
            if constexpr (TWO) {
                if (SV) {
                    ux[i] = fmaxf(ux[i], __shfl_xor_sync(0xffffffffu, ux[i], 1));
                    ux[i] = fmaxf(ux[i], __shfl_xor_sync(0xffffffffu, ux[i], 2));
                }
                move |= follow(SV ? ux[i] : mx[i], u[i], al[i]);
            } else {
                move |= mv;
                al[i] = by;
            }
        }
        if (__any_sync(0xffffffffu, move)) {
#pragma unroll
            for (int n = 0; n < D / 8; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[n][i] *= al[i >> 1];
        }
        const float mref[2] = {finite_ref(m[0]), finite_ref(m[1])}, uref[2] = {finite_ref(u[0]), finite_ref(u[1])};
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float e = ex2(s[n][i] - mref[i >> 1]);
                l[i >> 1] += e;
                if constexpr (TWO) s[n][i] = ex2(s[n][i] + ls[n][i & 1] - uref[i >> 1]);
                else s[n][i] = SV ? e * sv[n][i & 1] : e;
            }
    }

    // O += weights * values at vs (KS rows from r0), from the cache
    __device__ __forceinline__ void values(const float (&w)[KS / 8][4], uint32_t vs, const uint8_t* vsp, int r0, int lane) {
        using C = Lay<CT, D>;
        if constexpr (f32 && !is8) {
            values_f32(w, vsp, r0, lane);
        } else if constexpr (!is8) {
            values_bf16(w, vs, r0, lane);
        } else {
            const int vr = r0 + (lane & 15), vc = lane >> 4;
            uint32_t p[KS / 16][4], ph[2][4], pl[2][4];
            if constexpr (!f32) {
#pragma unroll
                for (int k = 0; k < KS / 16; ++k) {
                    p[k][0] = pack_f16x2(w[2 * k][0], w[2 * k][1]), p[k][1] = pack_f16x2(w[2 * k][2], w[2 * k][3]);
                    p[k][2] = pack_f16x2(w[2 * k + 1][0], w[2 * k + 1][1]), p[k][3] = pack_f16x2(w[2 * k + 1][2], w[2 * k + 1][3]);
                }
            } else {
                split_weights(w, ph, pl);
            }
#pragma unroll
            for (int n = 0; n < (D + 31) / 32; ++n)              // two 16-feature blocks (D = 16: one)
#pragma unroll
                for (int k = 0; k < KS / 16; ++k) {              // 16 keys
                    uint32_t b[4] = {0, 0, 0, 0};
                    if constexpr (D >= 32) ldsm_x4_t(b, vs + C::at(vr + 16 * k, 2 * n + vc));
                    else ldsm_x2_t(b[0], b[1], vs + C::at(vr + 16 * k, 0));
#pragma unroll
                    for (int h = 0; h < (D >= 32 ? 2 : 1); ++h) {
                        const int j = 2 * n + h;
                        const uint32_t x0 = __byte_perm(b[2 * h], 0, 0x3120), x1 = __byte_perm(b[2 * h + 1], 0, 0x3120);
                        const uint32_t e0 = f16_of_e4m3(x0), o0 = f16_of_e4m3_hi(x0), e1 = f16_of_e4m3(x1), o1 = f16_of_e4m3_hi(x1);
                        if constexpr (!f32) {
                            mma_f16(o[2 * j], p[k], e0, e1);
                            mma_f16(o[2 * j + 1], p[k], o0, o1);
                        } else {
                            const float2 f[2][2] = {{f32_of_f16x2(e0), f32_of_f16x2(e1)}, {f32_of_f16x2(o0), f32_of_f16x2(o1)}};
#pragma unroll
                            for (int y = 0; y < 2; ++y) {
                                float part[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                                for (int i = 0; i < 2; ++i) {
                                    const uint32_t b0 = __float_as_uint(f[y][i].x), b1 = __float_as_uint(f[y][i].y);
                                    mma_tf32(part, pl[i], b0, b1);
                                    mma_tf32(part, ph[i], b0, b1);
                                }
                                add4(o[2 * j + y], part);
                            }
                        }
                    }
                }
        }
    }
    // A operands of m16n8k8 over 8 keys, whose k index t is key 2t and t + 4 key 2t + 1
    static __device__ __forceinline__ void split_weights(const float (&w)[2][4], uint32_t (&hi)[2][4], uint32_t (&lo)[2][4]) {
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            split_tf32<true>(w[n][0], hi[n][0], lo[n][0]);
            split_tf32<true>(w[n][2], hi[n][1], lo[n][1]);
            split_tf32<true>(w[n][1], hi[n][2], lo[n][2]);
            split_tf32<true>(w[n][3], hi[n][3], lo[n][3]);
        }
    }
    template <int NT>
    __device__ __forceinline__ void values_bf16(const float (&w)[NT][4], uint32_t vs, int r0, int lane) {
        using C = Lay<bf16, D>;
        const int vr = r0 + (lane & 15), vc = lane >> 4;
        uint32_t p[NT / 2][4];
#pragma unroll
        for (int k = 0; k < NT / 2; ++k) {
            p[k][0] = tc::pack_bf16x2(w[2 * k][0], w[2 * k][1]), p[k][1] = tc::pack_bf16x2(w[2 * k][2], w[2 * k][3]);
            p[k][2] = tc::pack_bf16x2(w[2 * k + 1][0], w[2 * k + 1][1]), p[k][3] = tc::pack_bf16x2(w[2 * k + 1][2], w[2 * k + 1][3]);
        }
#pragma unroll
        for (int n = 0; n < D / 16; ++n)
#pragma unroll
            for (int k = 0; k < NT / 2; ++k) {
                uint32_t b[4];
                ldsm_x4_t(b, vs + C::at(vr + 16 * k, 2 * n + vc));
                mma_bf16(o[2 * n], p[k], b[0], b[1]);
                mma_bf16(o[2 * n + 1], p[k], b[2], b[3]);
            }
    }
    __device__ __forceinline__ void values_f32(const float (&w)[2][4], const uint8_t* vsp, int r0, int lane) {
        using C = Lay<float, D>;
        const int g = lane >> 2, t = lane & 3;
        uint32_t ph[2][4], pl[2][4];
        split_weights(w, ph, pl);
#pragma unroll
        for (int j = 0; j < D / 16; ++j) {
            float part[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int r = r0 + 8 * k + 2 * t, f = 16 * j + 2 * g;
                const float2 x0 = *reinterpret_cast<const float2*>(vsp + C::at_v(r, f / 4) + 4 * (f % 4));
                const float2 x1 = *reinterpret_cast<const float2*>(vsp + C::at_v(r + 1, f / 4) + 4 * (f % 4));
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    uint32_t b0h, b0l, b1h, b1l;
                    split_tf32(y ? x0.y : x0.x, b0h, b0l);
                    split_tf32(y ? x1.y : x1.x, b1h, b1l);
                    mma_tf32(part[y], pl[k], b0h, b1h);
                    mma_tf32(part[y], ph[k], b0l, b1l);
                    mma_tf32(part[y], ph[k], b0h, b1h);
                }
            }
            add4(o[2 * j], part[0]);
            add4(o[2 * j + 1], part[1]);
        }
    }

    // KS cached keys: the tile's row r0 is position x; nk of them exist.  Row i sees x < sinks
    // and x > low[i].
    template <int WR>
    __device__ __forceinline__ void step(uint32_t st, const uint8_t* stp, int r0, int x, int nk, int sinks, const int (&low)[2],
                                         bool edge, int lane) {
        using C = Cfg<QT, CT, D, WR>;
        constexpr int NT = KS / 8;
        const int t = lane & 3;
        float s[NT][4], sv[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
            sv[n][0] = sv[n][1] = 1.f;
        }
        scores(s, st, stp, r0, lane);
        if constexpr (is8) {
            const float* sc = reinterpret_cast<const float*>(stp + 2 * C::TILE) + r0;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const float2 sk = *reinterpret_cast<const float2*>(sc + 8 * n + 2 * t);
                const float2 v = *reinterpret_cast<const float2*>(sc + C::KT + 8 * n + 2 * t);
                sv[n][0] = v.x, sv[n][1] = v.y;
#pragma unroll
                for (int i = 0; i < 4; ++i) s[n][i] *= factor(c[i >> 1], i & 1 ? sk.y : sk.x);
            }
        } else {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) s[n][i] *= c[i >> 1];
        }
        if (edge || nk < KS) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int col = 8 * n + 2 * t + (i & 1);
                    if (col >= nk || (x + col >= sinks && x + col <= low[i >> 1])) s[n][i] = -INFINITY;
                }
        }
        weights<is8>(s, sv);
        values(s, st + C::TILE, stp + C::TILE, r0, lane);
    }
    // 16 new keys, of which row i sees the bits see[i]
    __device__ __forceinline__ void step_new(uint32_t st, const uint8_t* stp, const uint32_t (&see)[2], int lane) {
        constexpr int TILE = 16 * Lay<QT, D>::ROWB;
        const int t = lane & 3;
        float s[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
        const float one[2][2] = {{1.f, 1.f}, {1.f, 1.f}};
        if constexpr (f32) scores_f32<CT>(s, stp, 0, lane);
        else scores_bf16(s, st, 0, lane);
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                s[n][i] = see[i >> 1] >> (8 * n + 2 * t + (i & 1)) & 1 ? s[n][i] * c[i >> 1] : -INFINITY;
        weights<false>(s, one);
        if constexpr (f32) values_f32(s, stp + TILE, 0, lane);
        else values_bf16(s, st + TILE, 0, lane);
    }
    // Result rows r0 .. r0 + 15 of `rows`: O [rows][D] (TWO: over l), m [rows], l [rows]
    __device__ __forceinline__ void store(float* res, int rows, int r0, int lane) {
        const int g = lane >> 2, t = lane & 3;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
            l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
            const int r = r0 + g + 8 * i;
            if (t == 0) res[rows * D + r] = m[i], res[rows * (D + 1) + r] = l[i];
            if constexpr (TWO) {
                const float half = half_unit(u[i], m[i]), inv = inverse_or_0(l[i]) * half;
#pragma unroll
                for (int n = 0; n < D / 8; ++n) o[n][2 * i] *= inv, o[n][2 * i] *= half, o[n][2 * i + 1] *= inv, o[n][2 * i + 1] *= half;
            }
            if constexpr (PERM) {
#pragma unroll
                for (int j = 0; j < D / 16; ++j)
                    *reinterpret_cast<float4*>(res + r * D + 16 * j + 4 * t) =
                        make_float4(o[2 * j][2 * i], o[2 * j + 1][2 * i], o[2 * j][2 * i + 1], o[2 * j + 1][2 * i + 1]);
            } else {
#pragma unroll
                for (int n = 0; n < D / 8; ++n)
                    *reinterpret_cast<float2*>(res + r * D + 8 * n + 2 * t) = make_float2(o[n][2 * i], o[n][2 * i + 1]);
            }
        }
    }
};

// A warp's 8 rows over an 8-bit cache (bf16 queries), as columns: S^T = K Q^T and O^T = V^T P^T
// have the keys resp. the features as the 16 rows of a product and the 8 rows as its columns, where
// the other way round half of a product's rows would be empty: half the products and half the
// sums' registers, so that more warps fit.  S^T's sums become the next product's operand by
// transposing 8x8 blocks between lanes (movmatrix).
template <int D>
struct Cols {
    static constexpr bool f32 = false, PERM = true, TWO = true;
    static constexpr int KS = 32;
    // the rows that a lane weighs, and the one whose query it has a part of
    static __device__ __forceinline__ int row(int i, int lane) { return 2 * (lane & 3) + i; }
    static __device__ __forceinline__ int query(int, int lane) { return lane >> 2; }
    uint32_t q[D / 8];                            // [D / 16][2]
    float o[D / 16][4], m[2], l[2], u[2], c[2];   // o: feature 16 j + 2 g (0, 1) or + 1 (2, 3) of rows 2 t and 2 t + 1

    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int j = 0; j < D / 16; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[j][i] = 0.f;
        m[0] = m[1] = u[0] = u[1] = -INFINITY;
        l[0] = l[1] = 0.f;
    }
    __device__ __forceinline__ void load_bf16(const uint16_t* const (&rows)[2], long long sJ, float cc, int lane) {
        const int t = lane & 3;
        const uint16_t* p = rows[0];
#pragma unroll
        for (int s = 0; s < D / 16; ++s)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int k = 16 * s + 2 * t + 8 * i;
                q[2 * s + i] = p ? (uint32_t)p[k * sJ] | ((uint32_t)p[(k + 1) * sJ] << 16) : 0u;
            }
        c[0] = c[1] = cc;
    }
    __device__ __forceinline__ void load(const void* const (&rows)[2], long long sJ, float cc, int lane) {
        const int t = lane & 3;
        const uint16_t* p = static_cast<const uint16_t*>(rows[0]);
        float top = 0.f;
#pragma unroll
        for (int s = 0; s < D / 16; ++s)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int k = Rows<bf16, e4m3, D>::feat8(s, t) + 2 * i;
                const uint32_t x = p ? (uint32_t)p[k * sJ] | ((uint32_t)p[(k + 1) * sJ] << 16) : 0u;
                q[2 * s + i] = x;
                top = fmaxf(top, fmaxf(fabsf(__uint_as_float(x << 16)), fabsf(__uint_as_float(x & 0xffff0000u))));
            }
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int e = max((int)(__float_as_uint(top) >> 23) - 127, -100);
        const float up = __uint_as_float((uint32_t)(127 + 7 - e) << 23), mine = cc * __uint_as_float((uint32_t)(127 - 7 + e) << 23);
#pragma unroll
        for (int i = 0; i < D / 8; ++i)
            q[i] = pack_f16x2(__uint_as_float(q[i] << 16) * up, __uint_as_float(q[i] & 0xffff0000u) * up);
#pragma unroll
        for (int i = 0; i < 2; ++i) c[i] = __shfl_sync(0xffffffffu, mine, 4 * row(i, lane));
    }
    // Masked scores s[k][]: keys 16 k + g (0, 1) and + 8 (2, 3), rows 2 t and 2 t + 1; to weights
    // times the keys' scales sv (in units of 2^u), as operands p of the next product.  BF16: to
    // bf16, no scales.
    template <bool BF16, int NK>
    __device__ __forceinline__ void weights(float (&s)[NK][4], const float (&sv)[NK][2], uint32_t (&p)[NK][2]) {
        float mx[2] = {-INFINITY, -INFINITY}, ux[2] = {-INFINITY, -INFINITY}, ls[NK][2];
#pragma unroll
        for (int k = 0; k < NK; ++k)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                ls[k][i] = BF16 ? 0.f : __log2f(sv[k][i]);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    mx[e] = fmaxf(mx[e], s[k][2 * i + e]);
                    if (!BF16) ux[e] = fmaxf(ux[e], s[k][2 * i + e] + ls[k][i]);
                }
            }
        bool move = false;
        float al[2];                              // of O
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) {
                mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], x));
                if (!BF16) ux[i] = fmaxf(ux[i], __shfl_xor_sync(0xffffffffu, ux[i], x));
            }
            float by;
            follow(mx[i], m[i], by);
            l[i] *= by;
            move |= follow(BF16 ? mx[i] : ux[i], u[i], al[i]);
        }
        if (__any_sync(0xffffffffu, move)) {
#pragma unroll
            for (int j = 0; j < D / 16; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[j][i] *= al[i & 1];
        }
        const float mref[2] = {finite_ref(m[0]), finite_ref(m[1])}, uref[2] = {finite_ref(u[0]), finite_ref(u[1])};
#pragma unroll
        for (int k = 0; k < NK; ++k)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                l[0] += ex2(s[k][2 * i] - mref[0]), l[1] += ex2(s[k][2 * i + 1] - mref[1]);
                const float a = ex2(s[k][2 * i] + ls[k][i] - uref[0]), b = ex2(s[k][2 * i + 1] + ls[k][i] - uref[1]);
                const uint32_t x = BF16 ? tc::pack_bf16x2(a, b) : pack_f16x2(a, b);
                asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(p[k][i]) : "r"(x));
            }
    }
    template <int WR>
    __device__ __forceinline__ void step(uint32_t st, const uint8_t* stp, int r0, int x, int nk, int sinks, const int (&low)[2],
                                         bool edge, int lane) {
        using C = Cfg<bf16, e4m3, D, WR>;
        constexpr int NK = KS / 16, W = D >= 64 ? 16 : D / 4;   // bytes per lane and read
        const int g = lane >> 2, t = lane & 3;
        float s[NK][4], sv[NK][2];
        uint32_t p[NK][2];
        const float* sc = reinterpret_cast<const float*>(stp + 2 * C::TILE) + r0;
#pragma unroll
        for (int k = 0; k < NK; ++k) {
            s[k][0] = s[k][1] = s[k][2] = s[k][3] = 0.f;
#pragma unroll
            for (int j = 0; j < D / (4 * W); ++j) {
                uint32_t w[2][W / 4];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int f = 4 * W * j + W * t;
                    const uint8_t* a = stp + C::at(r0 + 16 * k + 8 * i + g, f / 16) + f % 16;
                    if constexpr (W == 16) {
                        const uint4 y = *reinterpret_cast<const uint4*>(a);
                        w[i][0] = y.x, w[i][1] = y.y, w[i][2] = y.z, w[i][3] = y.w;
                    } else if constexpr (W == 8) {
                        const uint2 y = *reinterpret_cast<const uint2*>(a);
                        w[i][0] = y.x, w[i][1] = y.y;
                    } else {
                        w[i][0] = *reinterpret_cast<const uint32_t*>(a);
                    }
                }
#pragma unroll
                for (int e = 0; e < W / 4; ++e) {
                    const uint32_t a[4] = {f16_of_e4m3(w[0][e]), f16_of_e4m3(w[1][e]), f16_of_e4m3_hi(w[0][e]),
                                           f16_of_e4m3_hi(w[1][e])};
                    const int y = 2 * (j * (W / 4) + e);
                    mma_f16(s[k], a, q[y], q[y + 1]);
                }
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float sk = sc[16 * k + 8 * i + g];
                sv[k][i] = sc[C::KT + 16 * k + 8 * i + g];
                s[k][2 * i] *= factor(c[0], sk);
                s[k][2 * i + 1] *= factor(c[1], sk);
            }
        }
        if (edge || nk < KS) {
#pragma unroll
            for (int k = 0; k < NK; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int key = 16 * k + 8 * (i >> 1) + g;
                    if (key >= nk || (x + key >= sinks && x + key <= low[i & 1])) s[k][i] = -INFINITY;
                }
        }
        weights<false>(s, sv, p);
        const int vr = r0 + (lane & 15), vc = lane >> 4;
        const uint32_t vs = st + C::TILE;
#pragma unroll
        for (int n = 0; n < (D + 31) / 32; ++n)
#pragma unroll
            for (int k = 0; k < NK; ++k) {
                uint32_t b[4] = {0, 0, 0, 0};
                if constexpr (D >= 32) ldsm_x4_t(b, vs + C::at(vr + 16 * k, 2 * n + vc));
                else ldsm_x2_t(b[0], b[1], vs + C::at(vr + 16 * k, 0));
#pragma unroll
                for (int h = 0; h < (D >= 32 ? 2 : 1); ++h) {
                    const uint32_t x0 = __byte_perm(b[2 * h], 0, 0x3120), x1 = __byte_perm(b[2 * h + 1], 0, 0x3120);
                    const uint32_t a[4] = {f16_of_e4m3(x0), f16_of_e4m3_hi(x0), f16_of_e4m3(x1), f16_of_e4m3_hi(x1)};
                    mma_f16(o[2 * n + h], a, p[k][0], p[k][1]);
                }
            }
    }
    // 16 new keys (values with even features first), of which row i of the lane sees the bits see[i]
    __device__ __forceinline__ void step_new(uint32_t st, const uint8_t*, const uint32_t (&see)[2], int lane) {
        using C = Lay<bf16, D>;
        const int g = lane >> 2, r = lane & 15, h = lane >> 4;
        float s[1][4] = {{0.f, 0.f, 0.f, 0.f}};
        const float one[1][2] = {{1.f, 1.f}};
        uint32_t p[1][2];
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
            uint32_t a[4];
            ldsm_x4(a, st + C::at(r, 2 * kk + h));
            mma_bf16(s[0], a, q[2 * kk], q[2 * kk + 1]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) s[0][i] = see[i & 1] >> (8 * (i >> 1) + g) & 1 ? s[0][i] * c[i & 1] : -INFINITY;
        weights<true>(s, one, p);
#pragma unroll
        for (int j = 0; j < D / 16; ++j) {
            uint32_t b[4];
            ldsm_x4_t(b, st + 16 * C::ROWB + C::at(r, 2 * j + h));
            const uint32_t a[4] = {b[0], b[2], b[1], b[3]};
            mma_bf16(o[j], a, p[0][0], p[0][1]);
        }
    }
    __device__ __forceinline__ void store(float* res, int rows, int, int lane) {
        const int g = lane >> 2, t = lane & 3;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], x);
            const int r = 2 * t + i;
            if (g == 0) res[rows * D + r] = m[i], res[rows * (D + 1) + r] = l[i];
            const float half = half_unit(u[i], m[i]), inv = inverse_or_0(l[i]) * half;
#pragma unroll
            for (int j = 0; j < D / 16; ++j)
                *reinterpret_cast<float2*>(res + r * D + 16 * j + 2 * g) = make_float2(o[j][i] * inv * half, o[j][2 + i] * inv * half);
        }
    }
};
template <typename QT, typename CT, int D, int WR>
struct EngineOf {
    using type = Rows<QT, CT, D>;
};
template <int D>
struct EngineOf<bf16, e4m3, D, 0> {
    using type = Cols<D>;
};

// ------------------------------------------------------------------ joins
// Element e of row r from n results, get(i, at) the i-th's (TWO: its O over its l): y, not over l.
struct Sum {
    float y, m, l;
};
template <int D, int ROWS, bool TWO, typename Get>
__device__ __forceinline__ Sum join(int n, int r, int e, const Get& get) {
    Sum s{0.f, -INFINITY, 0.f};
    for (int i = 0; i < n; ++i) s.m = fmaxf(s.m, get(i, ROWS * D + r));
    const float ref = finite_ref(s.m);
    for (int i = 0; i < n; ++i) {
        const float w = exp2f(get(i, ROWS * D + r) - ref), l = get(i, ROWS * (D + 1) + r);
        s.l = fmaf(l, w, s.l);
        s.y = fmaf(get(i, r * D + e), TWO ? l * w : w, s.y);
    }
    return s;
}
struct Where {                                    // a group: sequence, key head, its first row
    int b, hk, row0, n;                           // n: real new tokens
};
__device__ __forceinline__ Where where_of(const P& a, int group, int rows) {
    Where w;
    const int rg = group % a.rgroups, bk = group / a.rgroups;
    w.b = bk / a.Hkv, w.hk = bk % a.Hkv;
    w.row0 = rg * rows;
    w.n = a.n_new ? min(max(__ldg(a.n_new + w.b), 0), a.T) : a.T;
    return w;
}
// A row that sees nothing, and a padding row, is 0 with the log-sum-exp -inf.
template <typename QT>
__device__ __forceinline__ void write_out(const P& a, const Where& w, int r, int e, const Sum& s) {
    const int row = w.row0 + r, t = divide(row, a.by_g), h = w.hk * a.G + row - t * a.G;
    const bool some = t < w.n && s.l != 0.f;
    static_cast<QT*>(const_cast<void*>(a.o.base))[w.b * a.o.sB + h * a.o.sH + (long long)t * a.o.sN + e * a.o.sJ] =
        from_f32<QT>(some ? s.y / s.l : 0.f);
    if (a.lse && e == 0) a.lse[((size_t)w.b * a.Hq + h) * a.T + t] = some ? (s.m + log2f(s.l)) * kLn2 : -INFINITY;
}
__device__ __forceinline__ float ld_cluster(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

// ------------------------------------------------------------------ the kernel
// Block (group, split); group = (sequence, key head, row group).
template <typename QT, typename CT, int D, int WR>
__global__ void __launch_bounds__(kT, (Cfg<QT, CT, D, WR>::BLOCKS))
tree_kernel(const __grid_constant__ P a) {
    using C = Cfg<QT, CT, D, WR>;
    extern __shared__ __align__(128) uint8_t sm[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int team = warp / C::TW, wr = warp % C::TW, tl = threadIdx.x - team * 32 * C::TW;
    const int split = blockIdx.x % a.splits, group = blockIdx.x / a.splits;
    const Where w = where_of(a, group, C::ROWS);
    const int L = max(__ldg(a.lens + w.b), 0);
    const Slots s = load_slots(a, L);
    const int per = ((s.nv + a.splits - 1) / a.splits + C::KT - 1) / C::KT * C::KT;
    const long long first = (long long)split * per;
    const int x0 = (int)min((long long)s.nv, first), x1 = (int)min((long long)s.nv, first + per);
    const long long head = w.b * a.sB + w.hk * a.sH, shead = w.b * a.cB + w.hk * a.cH;
    uint8_t* mine = sm + team * C::TEAM;
    const uint32_t mine32 = tc::smem_u32(mine);
    auto team_sync = [&]() {
        if constexpr (C::TW == 1) __syncwarp();
        else tc::named_bar_sync(1 + team, 32 * C::TW);
    };

    // the first tiles are on their way before anything else is read
    constexpr int stride = C::WK * C::KT;
    int next = x0 + team * C::KT;
#pragma unroll
    for (int i = 0; i < C::NST - 1; ++i) {
        if (next < x1) load_rows<QT, CT, D, WR>(a, s, head, shead, mine32 + i * C::STAGE, mine + i * C::STAGE, next, x1, tl);
        cp_async_commit();
        next += stride;
    }
    // a row's depth counts where the window's first positions are, its ancestors where the drafts are
    const bool last = a.drafts && split == a.splits - 1, bound = a.drafts && x0 < s.nv && s.nv - a.window + a.T - 1 >= x0;
    const int nw = (a.T + 31) / 32;
    uint32_t* anc = reinterpret_cast<uint32_t*>(sm + C::MAIN);
    int* jump = reinterpret_cast<int*>(anc + a.T * nw);
    const bool table = a.parents && (last || bound);
    if (table) ancestors(a.parents + w.b * a.par_stride, a.T, nw, anc, jump);

    using Engine = typename EngineOf<QT, CT, D, WR>::type;
    Engine rows;
    const void* qrow[2];
    int low[2], node[2], depth[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int qr = w.row0 + 16 * wr + Engine::query(i, lane), qn = divide(qr, a.by_g), h = w.hk * a.G + qr - qn * a.G;
        qrow[i] = qn < a.T ? static_cast<const QT*>(a.q.base) + w.b * a.q.sB + h * a.q.sH + (long long)qn * a.q.sN : nullptr;
        node[i] = min(divide(w.row0 + 16 * wr + Engine::row(i, lane), a.by_g), a.T - 1);
        depth[i] = node[i];
        if (table) {
            depth[i] = -1;
            for (int x = 0; x < nw; ++x) depth[i] += __popc(anc[node[i] * nw + x]);
        }
        low[i] = s.nv - a.window + (a.drafts ? depth[i] : -1);
    }
    rows.load(qrow, a.q.sJ, a.c, lane);
    rows.clear();

    int stage = 0;
    for (int x = x0 + team * C::KT; x < x1; x += stride, next += stride) {
        const int to = stage == 0 ? C::NST - 1 : stage - 1;       // the stage read in the last step
        if (next < x1) load_rows<QT, CT, D, WR>(a, s, head, shead, mine32 + to * C::STAGE, mine + to * C::STAGE, next, x1, tl);
        cp_async_commit();
        cp_async_wait<C::NST - 1>();
        team_sync();
#pragma unroll 1
        for (int y = 0; y < C::KT && x + y < x1; y += C::KS) {
            const int xx = x + y;
            rows.template step<WR>(mine32 + stage * C::STAGE, mine + stage * C::STAGE, y, xx, x1 - xx, a.sinks, low,
                                   xx <= s.nv - a.window + a.T - 1, lane);
        }
        team_sync();
        stage = stage == C::NST - 1 ? 0 : stage + 1;
    }
    cp_async_wait<0>();
    team_sync();
    if (last) {
        if constexpr (!Engine::f32) {                             // operands of bf16 products
            const uint16_t* const r[2] = {static_cast<const uint16_t*>(qrow[0]), static_cast<const uint16_t*>(qrow[1])};
            rows.load_bf16(r, a.q.sJ, a.c, lane);
        }
        // new keys up to the group's last token
        const int until = min(w.n, divide(w.row0 + C::ROWS - 1, a.by_g) + 1);
        for (int j0 = 16 * team; j0 < until; j0 += 16 * C::WK) {
            load_new<QT, D, Engine::PERM, 32 * C::TW>(a, w.b, w.hk, mine, j0, w.n, tl);
            team_sync();
            uint32_t see[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                see[i] = table ? anc[node[i] * nw + (j0 >> 5)] >> (j0 & 31)
                               : (node[i] < j0 ? 0u : 0xffffffffu >> (31 - min(node[i] - j0, 31)));
                see[i] &= 0xffffu;
                // ancestors beyond the window
                if (a.window < a.T) {
                    for (int e = 0; e < 16; ++e) {
                        int d = j0 + e;
                        if (table) {
                            d = -1;
                            if (j0 + e < a.T)
                                for (int x = 0; x < nw; ++x) d += __popc(anc[(j0 + e) * nw + x]);
                        }
                        if (d <= depth[i] - a.window && (long long)L + d >= a.sinks) see[i] &= ~(1u << e);
                    }
                }
            }
            rows.step_new(mine32, mine, see, lane);
            team_sync();
        }
    }
    __syncthreads();                              // the results go over the tiles
    float* all = reinterpret_cast<float*>(sm);
    rows.store(all + team * C::RN, C::ROWS, 16 * wr, lane);
    __syncthreads();
    auto from_teams = [&](int i, int at) { return all[i * C::RN + at]; };
    const int nrows = min(C::ROWS, a.T * a.G - w.row0);
    if (a.splits == 1) {
        for (int i = threadIdx.x; i < nrows * D; i += kT)
            write_out<QT>(a, w, i / D, i % D, join<D, C::ROWS, C::TWO>(C::WK, i / D, i % D, from_teams));
        return;
    }
    const bool cluster = a.splits <= kCluster;
    float* res = cluster ? reinterpret_cast<float*>(sm + C::OFF_RES) : a.part + ((size_t)group * a.splits + split) * C::RN;
    if (C::WK > 1 || !cluster)
        for (int i = threadIdx.x; i < nrows * D; i += kT) {
            const Sum s = join<D, C::ROWS, C::TWO>(C::WK, i / D, i % D, from_teams);
            res[i] = C::TWO ? s.y * inverse_or_0(s.l) : s.y;
            if (i % D == 0) res[C::ROWS * D + i / D] = s.m, res[C::ROWS * (D + 1) + i / D] = s.l;
        }
    if (!cluster) return;
    __syncwarp();
    tc::cluster_sync_all();
    const uint32_t res32 = tc::smem_u32(res);
    auto from_ranks = [&](int r, int at) { return ld_cluster(tc::mapa_shared(res32, r) + 4 * at); };
    for (int i = split * kT + threadIdx.x; i < nrows * D; i += a.splits * kT)   // split = rank in the cluster
        write_out<QT>(a, w, i / D, i % D, join<D, C::ROWS, C::TWO>(a.splits, i / D, i % D, from_ranks));
    __syncwarp();
    tc::cluster_sync_all();                       // no block leaves while its result is read
}

// Joins the splits of a group: a thread per element.
template <typename QT, typename CT, int D, int WR>
__global__ void __launch_bounds__(128)
tree_join_kernel(const __grid_constant__ P a) {
    using C = Cfg<QT, CT, D, WR>;
    constexpr int ROWS = C::ROWS, RN = C::RN, PER = ROWS * D / 128;
    const int group = blockIdx.x / PER, i = blockIdx.x % PER * 128 + threadIdx.x;
    const Where w = where_of(a, group, ROWS);
    if (i >= min(ROWS, a.T * a.G - w.row0) * D) return;
    const float* p = a.part + (size_t)group * a.splits * RN;
    auto from_runs = [&](int r, int at) { return p[(size_t)r * RN + at]; };
    write_out<QT>(a, w, i / D, i % D, join<D, ROWS, C::TWO>(a.splits, i / D, i % D, from_runs));
}

// ------------------------------------------------------------------ host
template <typename QT, typename CT, int D, int WR>
int launch_rows(const TreeArgs& a, const TreeSplit& s, std::string* err) {
    using C = Cfg<QT, CT, D, WR>;
    const long long grid = s.groups * s.splits;
    if (grid > 0x7fffffffll || s.groups * C::ROWS * D / 128 > 0x7fffffffll) {
        *err = "grid too large";
        return PSA_ERR_UNSUPPORTED;
    }
    const int smem = C::MAIN + (a.parents ? a.T * ((a.T + 31) / 32 + 1) * 4 : 0);
    constexpr int most = C::MAIN + PSA_TREE_MAX * (PSA_TREE_MAX / 32 + 1) * 4;
    if (!set_max_dynamic_smem((const void*)tree_kernel<QT, CT, D, WR>, most, err)) return PSA_ERR_CUDA;
    auto vec_of = [](const void* p, int esize, long long x, long long y, long long z) {
        const long long n = 16 / esize;
        return reinterpret_cast<uintptr_t>(p) % 16 == 0 && x % n == 0 && y % n == 0 && z % n == 0;
    };
    const int vec = vec_of(a.k, sizeof(CT), a.sB, a.sH, a.sS) && vec_of(a.v, sizeof(CT), 0, 0, 0);
    const int vec_new = a.drafts && a.kn.sJ == 1 && a.vn.sJ == 1 && vec_of(a.kn.base, sizeof(QT), a.kn.sB, a.kn.sH, a.kn.sN) &&
                        vec_of(a.vn.base, sizeof(QT), a.vn.sB, a.vn.sH, a.vn.sN);
    P p{};
    p.k = a.k, p.v = a.v, p.ks = a.ks, p.vs = a.vs;
    p.sB = a.sB, p.sH = a.sH, p.sS = a.sS, p.cB = a.cB, p.cH = a.cH, p.cS = a.cS;
    p.q = a.q, p.o = a.o, p.kn = a.kn, p.vn = a.vn, p.lse = a.lse, p.lens = a.lens, p.n_new = a.n_new;
    p.parents = a.parents, p.par_stride = a.par_stride, p.part = static_cast<float*>(a.workspace);
    p.Hq = a.Hq, p.Hkv = a.Hkv, p.G = a.Hq / a.Hkv, p.T = a.T, p.rgroups = s.rgroups, p.cap = a.cap, p.window = a.window;
    p.sinks = a.sinks, p.splits = s.splits, p.vec = vec, p.vec_new = vec_new, p.drafts = a.drafts, p.c = a.scale * kLog2e;
    p.by_g = fast_div(p.G);
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(kT);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = a.stream;
    cudaLaunchAttribute at[1];
    if (s.splits > 1 && s.splits <= kCluster) {
        at[0].id = cudaLaunchAttributeClusterDimension;
        at[0].val.clusterDim = {(unsigned)s.splits, 1, 1};
        cfg.attrs = at;
        cfg.numAttrs = 1;
    }
    ProfScope prof(kSlotFwd, a.stream);
    cudaError_t e = cudaLaunchKernelEx(&cfg, tree_kernel<QT, CT, D, WR>, p);
    if (e == cudaSuccess && s.splits > kCluster) {
        tree_join_kernel<QT, CT, D, WR><<<(unsigned)(s.groups * (C::ROWS * D / 128)), 128, 0, a.stream>>>(p);
        e = cudaGetLastError();
    }
    if (e == cudaSuccess) return PSA_OK;
    *err = std::string("tree attention launch: ") + cudaGetErrorString(e);
    return PSA_ERR_CUDA;
}
template <typename QT, typename CT, int D>
int launch_dim(const TreeArgs& a, const TreeSplit& s, std::string* err) {
    if constexpr (std::is_same<QT, bf16>::value && std::is_same<CT, e4m3>::value)
        if (s.wr == 0) return launch_rows<QT, CT, D, 0>(a, s, err);
    return s.wr == 1   ? launch_rows<QT, CT, D, 1>(a, s, err)
           : s.wr == 2 ? launch_rows<QT, CT, D, 2>(a, s, err)
                       : launch_rows<QT, CT, D, 4>(a, s, err);
}
template <typename QT, typename CT>
int launch(const TreeArgs& a, const TreeSplit& s, std::string* err) {
    switch (a.d) {
        case 16: return launch_dim<QT, CT, 16>(a, s, err);
        case 32: return launch_dim<QT, CT, 32>(a, s, err);
        case 64: return launch_dim<QT, CT, 64>(a, s, err);
        default: return launch_dim<QT, CT, 128>(a, s, err);
    }
}

}  // namespace tk
}  // namespace win
}  // namespace psa
