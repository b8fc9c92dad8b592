// win_warp.cu -- sliding-window attention with sinks on warp-level matrix products
// (mma.sync): fp32 storage, and bf16 in layouts that the tcgen05 path does not take.
// Also the row statistics and the sink rows' sums that every backward uses.
//
//   forward : per 32-row tile, online softmax over the key tiles it sees
//   D       : D_i = <dO_i, O_i>
//   dK, dV  : per 32-key tile, over the rows that see it, all query heads of
//             the key head in turn:  P = exp(S - LSE), dS = P (dO V^T - D),
//             dV += P^T dO, dK += dS^T Q   (sums over heads need no atomics)
//   dQ      : per 32-row tile, over the keys it sees: dQ += dS K
//
// Products have fp32 accuracy: an operand x is hi + lo, two tf32 numbers that hold 23 of its
// 24 bits, and a product is hi hi' + hi lo' + lo hi' in fp32: what is left out is below
// 2^-21 of |x x'|.  bf16 values are tf32 numbers as they are: their products take one
// step, and those with P or dS two.
// m16n8k8 runs at 480 FMA a cycle and SM on this GPU, so three steps beat FFMA's 128,
// and one instruction replaces 32 of them: B=2, 4 heads, N=1600, window 333, d=32 in
// fp32 took 47 us forward and 141 us backward on FFMA and takes 24 and 67.  (tcgen05's
// tf32 has four times the rate; it would take 128-row tiles, both halves of Q, K, V and dO in
// shared memory and P's and dS's in TMEM, and each tile's product added up outside of its
// accumulator.  Not built.)
//
// A block takes 32 rows (dK, dV: keys) through tiles of 64 keys (rows) in shared memory, the
// next tile on its way (cp.async); its eight warps own 16 rows by a quarter of each tile,
// skip what none of their rows sees, and the quarters' sums are joined at the end in order.
// (Halves and four warps: 23 and 73 us where this took 24 and 65; numbers near 2^128, which
// `split` treats since, are the rest of 67.  64 rows by whole tiles: 14 and 34% more than 32 by halves.)  A score tile's accumulators are the next product's A operand as they
// lie in the registers, with the keys of every 8 taken in the order 0 2 4 6 1 3 5 7, which
// the B operand's reads follow.  The block's own rows are split once, the tiles' values
// as they are read.  Tile rows are padded by 4 floats: all operand reads are free of bank
// conflicts.
//
// Bound by instruction issue (56% of the cycles on average, 80% on the SMs with three
// blocks): a product step is 3 of some 15 instructions, the rest operand reads, splits,
// sums, softmax and loads.  Splitting every tile once per block, (hi, lo) pairs in shared
// memory, read twice as much and lost the overlap of the loads: 32 and 93 us where the
// same by halves took 27 and 84.  The same case at d=16, 64, 128: forward 16, 47, 83 us, backward 42,
// 130, 250 (three tf32 products for each at that rate: 2.9, 12, 23 and 7.3, 29, 58).
#include <cuda_bf16.h>

#include <string>

#include "common.cuh"
#include "psa_internal.h"
#include "tc_ptx.cuh"
#include "tc_tmap.h"
#include "win_geom.cuh"
#include "win_internal.h"

namespace psa {
namespace win {
namespace {

constexpr int kT = 256;         // threads of the sink rows' sums
constexpr int kPre = 128;       // threads of the row statistics
constexpr int kParts = 4, kW = 64 * kParts;      // parts of a tile's keys (rows), each two warps'
constexpr int BM = 32;          // rows (dK, dV: keys) per block: two warps' 16, twice

template <int D>
constexpr int LD = D + 4;       // row stride of the tiles
constexpr int BN = 64;          // keys (rows) per tile

// Blocks an SM that the registers leave room for.  Head sizes 16 and 32: three, at 80
// registers (d=32 24.5 us forward, 67.4 backward; two 27.1 and 75.2; without a limit 29.7 and 85.1).
// 64: one, without a limit (46.6 and 130.3; two 47.7 and 132.8).  128: shared memory holds one
// (dK, dV there spills 72 bytes a thread at 255 registers).
template <int D>
constexpr int kBlocks = D <= 32 ? 3 : 1;

struct V {                      // a view's element strides, and whether 16 bytes (4 features) load at once
    const void* base;
    long long sB, sH, sN, sJ;
    int vec;
};

// 16 bytes of a row at once.
bool view_16(const View& v, int esize) {
    const long long w = 16 / esize;
    return v.sJ == 1 && v.sB % w == 0 && v.sH % w == 0 && v.sN % w == 0 && reinterpret_cast<uintptr_t>(v.base) % 16 == 0;
}
V dev_view(const View& v, int esize) { return V{v.base, v.sB, v.sH, v.sN, v.sJ, view_16(v, esize) ? 1 : 0}; }

__device__ __forceinline__ void cp_async16(void* dst, const void* src, bool full) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src),
                 "r"(full ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Rows [r0, r0 + R) of head (b, h) to a shared tile as fp32; rows >= n are zero and are
// not read.  L2: loads of 16 bytes go past L1 (those of fp32 always do).
template <typename T, int D, int R, bool L2 = false>
__device__ __forceinline__ void load_tile(float* s, const V& v, int b, int h, int r0, int n) {
    const T* base = static_cast<const T*>(v.base) + b * v.sB + h * v.sH;
    constexpr int E = 16 / (int)sizeof(T), C = D / E, RP = kW / C;   // chunks a row, rows a pass
    if (v.vec) {
        const int c = E * (threadIdx.x % C);
        const T* p = base + (long long)(r0 + (int)threadIdx.x / C) * v.sN + c;
#pragma unroll
        for (int i = 0; i < R; i += RP, p += RP * v.sN) {
            const int r = i + threadIdx.x / C;
            if (RP > R && r >= R) break;
            const bool in = r0 + r < n;
            float* to = s + r * LD<D> + c;
            if constexpr (sizeof(T) == 4) {
                cp_async16(to, in ? p : base, in);
            } else {
                uint4 u = make_uint4(0, 0, 0, 0);
                if (in) u = L2 ? __ldcg(reinterpret_cast<const uint4*>(p)) : *reinterpret_cast<const uint4*>(p);
                const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                for (int e = 0; e < 4; e += 2)
                    *reinterpret_cast<float4*>(to + 2 * e) =
                        make_float4(__uint_as_float(w[e] << 16), __uint_as_float(w[e] & 0xffff0000u),
                                    __uint_as_float(w[e + 1] << 16), __uint_as_float(w[e + 1] & 0xffff0000u));
            }
        }
    } else {
        for (int i = threadIdx.x; i < R * D; i += kW) {
            const int r = i / D, c = i % D;
            s[r * LD<D> + c] = r0 + r < n ? to_f32(base[(long long)(r0 + r) * v.sN + c * v.sJ]) : 0.f;
        }
    }
}

// x as tf32 hi + lo: hi is x rounded to 11 bits, x - hi has 12 at most and lo loses the
// last of them (2^-23 of x).  In integer steps: the conversion instruction runs at a quarter
// of their rate.  Up to the last step below 2^128 hi is rounded from 2^128 - 2^116 less one
// step instead: it would become infinite (lo then loses 2^-22 of x).  Probabilities (PROB) are
// never that large.  NaN and infinities stay (in lo).  (Without that step, 3 and 4% less time.)
template <bool PROB = false>
__device__ __forceinline__ void split(float x, uint32_t& hi, uint32_t& lo) {
    float y = x;
    if (!PROB) asm("min.xorsign.abs.f32 %0, %1, %2;" : "=f"(y) : "f"(x), "f"(0x1.ffdffep127f));
    hi = (__float_as_uint(y) + 0x1000u) & 0xffffe000u;
    lo = __float_as_uint(x - __uint_as_float(hi)) & 0xffffe000u;
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// The block's own tile to hi, in place, and lo behind it.
template <typename T, int D>
__device__ __forceinline__ void split_tile(float* s) {
    if constexpr (sizeof(T) == 4)
        for (int i = threadIdx.x; i < BM * D; i += kW) {
            float* x = s + i / D * LD<D> + i % D;
            uint32_t hi, lo;
            split(*x, hi, lo);
            x[0] = __uint_as_float(hi), x[BM * LD<D>] = __uint_as_float(lo);
        }
}
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma_0(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {   // on zeros
    asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

// acc[n] += A B_n for C tiles of 8 columns, B_n's fragment at (x0(n), x1(n)): each step goes
// over all tiles before the next, so that no product waits for the one before it.  The
// instruction cuts its sums off below 24 bits where fp32 addition rounds: fp32 operands'
// products of 8 are added up by the latter (one accumulator through all steps took 25
// and 78 us instead of 27 and 88, with dQ after dK, dV, and left O off by 1e-6 of its
// norm and the gradients by 2e-6 instead of 1.8e-7 and 3.2e-7).
template <int C, bool EXA, bool EXB, typename X0, typename X1>
__device__ __forceinline__ void mma_row(float (*acc)[4], const uint32_t (&hi)[4], const uint32_t (&lo)[4], const X0& x0,
                                        const X1& x1) {
    uint32_t h0[C], h1[C], l0[C], l1[C];
#pragma unroll
    for (int n = 0; n < C; ++n) {
        if (EXB) {
            h0[n] = __float_as_uint(x0(n)), h1[n] = __float_as_uint(x1(n));
        } else {
            split(x0(n), h0[n], l0[n]);
            split(x1(n), h1[n], l1[n]);
        }
    }
    if (EXB) {
        if (!EXA)
#pragma unroll
            for (int n = 0; n < C; ++n) mma(acc[n], lo, h0[n], h1[n]);
#pragma unroll
        for (int n = 0; n < C; ++n) mma(acc[n], hi, h0[n], h1[n]);
        return;
    }
    float s[C][4];
#pragma unroll
    for (int n = 0; n < C; ++n) mma_0(s[n], lo, h0[n], h1[n]);
#pragma unroll
    for (int n = 0; n < C; ++n) mma(s[n], hi, l0[n], l1[n]);
#pragma unroll
    for (int n = 0; n < C; ++n) mma(s[n], hi, h0[n], h1[n]);
#pragma unroll
    for (int n = 0; n < C; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[n][i] += s[n][i];
}

// acc[n] = A (the warp's 16 rows) times rows 8n .. 8n+7 of B.  EX: both are tf32 numbers.
template <int D, int NT, bool EX>
__device__ __forceinline__ void mm_nt(float (&acc)[NT][4], const float* A, const float* B, int g, int t) {
    constexpr int C = NT < 4 ? NT : 4;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[n][i] = 0.f;
#pragma unroll 2
    for (int k = 0; k < D; k += 8) {
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float* a = A + (g + 8 * (i & 1)) * LD<D> + k + t + 4 * (i >> 1);
            hi[i] = __float_as_uint(a[0]);
            if (!EX) lo[i] = __float_as_uint(a[BM * LD<D>]);
        }
        const float* p = B + g * LD<D> + k + t;
#pragma unroll
        for (int n = 0; n < NT; n += C)
            mma_row<C, EX, EX>(
                acc + n, hi, lo, [&](int c) { return p[8 * (n + c) * LD<D>]; },
                [&](int c) { return p[8 * (n + c) * LD<D> + 4]; });
    }
}
// acc[.][f] += sum over the tile's rows j of p[.][j] B[j][f], p as accumulators of mm_nt (PROB:
// probabilities).
template <int D, int NT, bool EX, bool PROB>
__device__ __forceinline__ void mm_pn(float (&acc)[D / 8][4], const float (&p)[NT][4], const float* B, int g, int t) {
    constexpr int C = D / 8 < 4 ? D / 8 : 4;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        uint32_t hi[4], lo[4];
        split<PROB>(p[n][0], hi[0], lo[0]);            // A's column t is row 2t of the 8, t + 4 is row 2t + 1
        split<PROB>(p[n][2], hi[1], lo[1]);
        split<PROB>(p[n][1], hi[2], lo[2]);
        split<PROB>(p[n][3], hi[3], lo[3]);
        const float* q = B + (8 * n + 2 * t) * LD<D> + g;
#pragma unroll
        for (int f = 0; f < D / 8; f += C)
            mma_row<C, false, EX>(
                acc + f, hi, lo, [&](int c) { return q[8 * (f + c)]; }, [&](int c) { return q[LD<D> + 8 * (f + c)]; });
    }
}

// Accumulators to shared memory, and added to those of another warp, lane by lane.
template <int D>
__device__ __forceinline__ void put_acc(float* s, const float (&x)[D / 8][4]) {
#pragma unroll
    for (int f = 0; f < D / 8; ++f)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[64 * (4 * f + i)] = x[f][i];
}
template <int D>
__device__ __forceinline__ void add_acc(float (&x)[D / 8][4], const float* s) {
#pragma unroll
    for (int f = 0; f < D / 8; ++f)
#pragma unroll
        for (int i = 0; i < 4; ++i) x[f][i] += s[64 * (4 * f + i)];
}

// The warp's 16 rows of accumulators to rows n0 + g, n0 + g + 8 < n of head (b, h).
template <typename T, int D>
__device__ __forceinline__ void store_rows(const V& v, int b, int h, int n0, int n, const float (&x)[D / 8][4], const float (&mul)[2],
                                           int g, int t) {
    T* base = static_cast<T*>(const_cast<void*>(v.base)) + b * v.sB + h * v.sH;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int r = n0 + g + 8 * i;
        if (r >= n) continue;
        T* row = base + (long long)r * v.sN;
#pragma unroll
        for (int f = 0; f < D / 8; ++f) {
            const float a = x[f][2 * i] * mul[i], c = x[f][2 * i + 1] * mul[i];
            const int j = 8 * f + 2 * t;
            if (v.vec) {
                if constexpr (sizeof(T) == 4) *reinterpret_cast<float2*>(row + j) = make_float2(a, c);
                else *reinterpret_cast<__nv_bfloat162*>(row + j) = __floats2bfloat162_rn(a, c);
            } else {
                row[j * v.sJ] = from_f32<T>(a);
                row[(j + 1) * v.sJ] = from_f32<T>(c);
            }
        }
    }
}

struct Dims {
    int Hq, G, Nq, Nk, window, sinks, ntiles, npad;
    float scale, scale_log2;
};

template <int D>
constexpr int fwd_smem() {
    return (2 * BM + 4 * BN) * LD<D> * 4;
}
template <int D>
constexpr int bwd_smem() {
    return (4 * BM + 4 * BN) * LD<D> * 4 + 4 * BN * 4;
}

// Rows of 8n + 2t + (i & 1), i of accumulator i: row index of keys or rows in a tile.
template <typename T, int D>
__global__ void __launch_bounds__(kW, kBlocks<D>)
warp_fwd_kernel(V q, V k, V v, V o, float* __restrict__ lse, const int* __restrict__ q_lens,
                const int* __restrict__ kv_lens, Dims m) {
    constexpr int N = BN, H = N / kParts, NT = H / 8;
    constexpr bool EX = sizeof(T) == 2;
    extern __shared__ __align__(16) float sm[];
    float *Qs = sm, *Ks = Qs + 2 * BM * LD<D>, *Vs = Ks + 2 * N * LD<D>;
    const int bh = blockIdx.x / m.ntiles, i0 = (int)(blockIdx.x % m.ntiles) * BM;
    const int b = bh / m.Hq, h = bh % m.Hq, hk = h / m.G;
    const int warp = threadIdx.x >> 5 & 1, slice = threadIdx.x >> 6, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const Seq s = load_seq(q_lens, kv_lens, b, m.Nq, m.Nk);
    const int i1 = min(i0 + BM, s.ql);
    const KeyTiles kt = key_tiles<N>(s, i0, i1, m.window, m.sinks);
    const int nk = kt.count();
    const int r0 = i0 + 16 * warp;
    const int p[2] = {r0 + g < s.ql ? r0 + g + s.off : -1, r0 + g + 8 < s.ql ? r0 + g + 8 + s.off : -1};
    // of the warp's 16 rows, whether some see some and whether all see all of keys j .. j + H - 1
    const int pf = r0 + s.off, pl = min(r0 + 16, s.ql) - 1 + s.off;
    auto sees_some = [&](int j) { return r0 < s.ql && j <= pl && (j + H - 1 > pf - m.window || j < m.sinks); };
    auto sees_all = [&](int j) { return r0 + 16 <= s.ql && j + H - 1 <= pf && j > pl - m.window; };
    float mx[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f}, acc[D / 8][4];
#pragma unroll
    for (int f = 0; f < D / 8; ++f)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[f][i] = 0.f;
    auto fetch = [&](int u) {
        const int j0 = kt.tile(u) * N;
        load_tile<T, D, N>(Ks + (u & 1) * N * LD<D>, k, b, hk, j0, s.kl);
        load_tile<T, D, N>(Vs + (u & 1) * N * LD<D>, v, b, hk, j0, s.kl);
    };
    if (nk > 0) {
        load_tile<T, D, BM>(Qs, q, b, h, i0, s.ql);
        fetch(0);
        cp_async_commit();
        cp_async_wait<0>();
        __syncthreads();
        split_tile<T, D>(Qs);
    }
    for (int u = 0; u < nk; ++u) {
        cp_async_wait<0>();
        __syncthreads();                              // tile u is there, and tile u - 1 done with
        if (u + 1 < nk) fetch(u + 1);
        cp_async_commit();
        const int jh = kt.tile(u) * N + slice * H;
        if (sees_some(jh)) {
            float c[NT][4];
            mm_nt<D, NT, EX>(c, Qs + 16 * warp * LD<D>, Ks + ((u & 1) * N + slice * H) * LD<D>, g, t);
            const bool whole = sees_all(jh);
            const int at[2] = {p[0] - jh - 2 * t, p[1] - jh - 2 * t}, sink = m.sinks - jh - 2 * t;
            float mt[2] = {-INFINITY, -INFINITY};
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int x = 8 * n + (i & 1);
                    c[n][i] *= m.scale_log2;
                    if (!whole && !(x <= at[i >> 1] && (x > at[i >> 1] - m.window || x < sink))) c[n][i] = -INFINITY;
                    mt[i >> 1] = fmaxf(mt[i >> 1], c[n][i]);
                }
            float ref[2];
            bool moved = false;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                mt[i] = fmaxf(mt[i], __shfl_xor_sync(0xffffffffu, mt[i], 1));
                mt[i] = fmaxf(mt[i], __shfl_xor_sync(0xffffffffu, mt[i], 2));
                ref[i] = fmaxf(mx[i], mt[i]);
                moved |= ref[i] != mx[i];
            }
            if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float alpha = ref[i] == -INFINITY ? 1.f : ex2(mx[i] - ref[i]);
                    mx[i] = ref[i];
                    l[i] *= alpha;
#pragma unroll
                    for (int f = 0; f < D / 8; ++f) acc[f][2 * i] *= alpha, acc[f][2 * i + 1] *= alpha;
                }
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) ref[i] = ref[i] == -INFINITY ? 0.f : ref[i];   // nothing seen yet: exp2(-inf) = 0
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    c[n][i] = ex2(c[n][i] - ref[i >> 1]);
                    l[i >> 1] += c[n][i];
                }
            mm_pn<D, NT, EX, true>(acc, c, Vs + ((u & 1) * N + slice * H) * LD<D>, g, t);
        }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
        l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
    }
    float* other = Ks + threadIdx.x % 64;             // the other parts' sums, lane by lane
    constexpr int size = 64 * (4 + D / 2);
    if (slice) {
        float* o1 = other + (slice - 1) * size;
#pragma unroll
        for (int i = 0; i < 2; ++i) o1[64 * i] = mx[i], o1[64 * (2 + i)] = l[i];
        put_acc<D>(o1 + 64 * 4, acc);
    }
    __syncthreads();
    if (slice) return;
    float inv[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        float now = mx[i];
#pragma unroll
        for (int q = 0; q < kParts - 1; ++q) now = fmaxf(now, other[q * size + 64 * i]);
        const float ref = now == -INFINITY ? 0.f : now, a = exp2f(mx[i] - ref);
        mx[i] = now;
        l[i] *= a;
#pragma unroll
        for (int f = 0; f < D / 8; ++f) acc[f][2 * i] *= a, acc[f][2 * i + 1] *= a;
#pragma unroll
        for (int q = 0; q < kParts - 1; ++q) {
            const float* o1 = other + q * size;
            const float c = exp2f(o1[64 * i] - ref);
            l[i] = fmaf(o1[64 * (2 + i)], c, l[i]);
#pragma unroll
            for (int f = 0; f < D / 8; ++f)
#pragma unroll
                for (int e = 2 * i; e < 2 * i + 2; ++e) acc[f][e] = fmaf(o1[64 * (4 + 4 * f + e)], c, acc[f][e]);
        }
        const bool some = l[i] > 0.f || l[i] != l[i];
        inv[i] = some ? 1.f / l[i] : 0.f;
        const int r = r0 + g + 8 * i;
        if (t == 0 && r < m.Nq) lse[(size_t)bh * m.Nq + r] = some ? (mx[i] + log2f(l[i])) * kLn2 : -INFINITY;
    }
    store_rows<T, D>(o, b, h, r0, m.Nq, acc, inv, g, t);
}

// x as a sum of three bf16 numbers (24 bits).
__device__ __forceinline__ void split3(float x, __nv_bfloat16* to) {
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        to[i] = from_f32<__nv_bfloat16>(x);
        x -= to_f32(to[i]);
    }
}

// The backward's row statistics, for whole 128-row tiles: D = rowsum(dO o O), and
// -LSE log2(e), which is -inf for rows that see nothing and for padding: their P
// = exp2(x - inf) is 0.  The tensor-core kernel gets them as operands too: the
// three bf16 numbers of -LSE / scale (the lowest one instead of -inf: finite, and
// times c still far below any exponent) and of -D.
//
// Bound by memory: 16 bytes of O and dO a thread and row, up to four rows, all of a
// block's loads on their way at once (B=1, 16 heads, N=8192, d=128 in bf16, 67 MB: 18 us
// with its launch; blocks of 128 rows in two steps, which one wave of blocks barely
// holds, took 22).
template <typename T, int D>
struct Pre {
    static constexpr int E = 16 / (int)sizeof(T), TR = D / E, R = kPre / TR;   // features a thread, threads a row, rows a pass
    static constexpr int ROWS = 4 * R < 128 ? 4 * R : 128, U = ROWS / R;      // rows a block
};
template <typename T, int D>
__global__ void __launch_bounds__(kPre)
pre_d_kernel(V o, V dO, const float* __restrict__ lse, float* __restrict__ Drow, float* __restrict__ negl,
             __nv_bfloat16* __restrict__ aug, const int* __restrict__ q_lens, int Hq, int Nq, int npad, float inv_c) {
    using C = Pre<T, D>;
    constexpr int E = C::E, U = C::U;
    // neighbouring blocks take the heads of the same rows: in token-major memory those
    // are neighbours (heads one after the other read a 256-byte piece every few KB)
    const int nb = npad / C::ROWS, bt = blockIdx.x / Hq, h = blockIdx.x - (unsigned)bt * Hq;
    const int b = bt / nb, bh = b * Hq + h;
    const int ql = q_lens ? min(__ldg(q_lens + b), Nq) : Nq;
    const int n0 = (bt - b * nb) * C::ROWS + threadIdx.x / C::TR, g = E * (threadIdx.x % C::TR);
    const T* po = static_cast<const T*>(o.base) + b * o.sB + h * o.sH + g * o.sJ;
    const T* pd = static_cast<const T*>(dO.base) + b * dO.sB + h * dO.sH + g * dO.sJ;
    float s[U], ln[U];                               // (LSE is on its way with the rest)
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int n = n0 + u * C::R;
        ln[u] = g == 0 && n < ql ? lse[(size_t)bh * Nq + n] : -INFINITY;
    }
    if (o.vec && dO.vec) {
        uint4 x[U], y[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int n = n0 + u * C::R;
            x[u] = y[u] = make_uint4(0, 0, 0, 0);
            if (n < ql) {
                x[u] = *reinterpret_cast<const uint4*>(po + n * o.sN);
                y[u] = *reinterpret_cast<const uint4*>(pd + n * dO.sN);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const T *a = reinterpret_cast<const T*>(&x[u]), *c = reinterpret_cast<const T*>(&y[u]);
            s[u] = 0.f;
#pragma unroll
            for (int e = 0; e < E; ++e) s[u] = fmaf(to_f32(a[e]), to_f32(c[e]), s[u]);
        }
    } else {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int n = n0 + u * C::R;
            s[u] = 0.f;
            if (n < ql)
#pragma unroll
                for (int e = 0; e < E; ++e) s[u] = fmaf(to_f32(po[n * o.sN + e * o.sJ]), to_f32(pd[n * dO.sN + e * dO.sJ]), s[u]);
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
        for (int w = C::TR / 2; w; w >>= 1) s[u] += __shfl_xor_sync(0xffffffffu, s[u], w);
        if (g != 0) continue;
        const size_t row = (size_t)bh * npad + n0 + u * C::R;
        const float L = ln[u] == -INFINITY ? -INFINITY : -ln[u] * kLog2e;
        Drow[row] = s[u], negl[row] = L;
        if (aug) {
            const float low = -3.3895313892515355e38f;   // the lowest finite bf16
            __nv_bfloat16 q[8];
            split3(fminf(fmaxf(L * inv_c, low), -low), q);
            split3(-s[u], q + 3);
            q[6] = q[7] = from_f32<__nv_bfloat16>(0.f);
            *reinterpret_cast<uint4*>(aug + 8 * row) = *reinterpret_cast<const uint4*>(q);
        }
    }
}

// P and dS from the accumulators of S and dP: L (-LSE log2(e)) and D of the
// accumulator's row (COLS: of its column), `hidden` where nothing is seen.
template <int NT, bool COLS, typename Hidden>
__device__ __forceinline__ void score_grads(float (&c)[NT][4], float (&dp)[NT][4], const float* L, const float* Dr, float scale_log2,
                                            bool whole, const Hidden& hidden) {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int at = COLS ? 8 * n + (i & 1) : i >> 1;
            const bool gone = !whole && hidden(n, i);
            c[n][i] = gone ? 0.f : ex2(fmaf(c[n][i], scale_log2, L[at]));
            dp[n][i] = gone ? 0.f : c[n][i] * (dp[n][i] - Dr[at]);
        }
}

// One work item of a key head: a 32-key tile and the rows that see it (x < ntiles), or
// far chunk c of a tile with sinks.
template <typename T, int D>
__global__ void __launch_bounds__(kW, kBlocks<D>)
warp_dkdv_kernel(V q, V k, V v, V dO, V dk, V dv, const float* __restrict__ negl, const float* __restrict__ Drow,
                 float* __restrict__ part, const int* __restrict__ q_lens, const int* __restrict__ kv_lens, Dims m,
                 FarSplit f, int items, int Hkv) {
    constexpr int N = BN, H = N / kParts, NT = H / 8;
    constexpr bool EX = sizeof(T) == 2;
    extern __shared__ __align__(16) float sm[];
    tc::griddep_wait();                                   // the row statistics are there
    tc::griddep_launch_dependents();                      // and the dQ kernel may start beside this one
    float *Ks = sm, *Vs = Ks + 2 * BM * LD<D>, *Qs = Vs + 2 * BM * LD<D>, *Os = Qs + 2 * N * LD<D>, *Ls = Os + 2 * N * LD<D>,
          *Ds = Ls + 2 * N;
    const int bk = blockIdx.x / items, x = blockIdx.x % items;
    const int b = bk / Hkv, hk = bk % Hkv;
    const int warp = threadIdx.x >> 5 & 1, slice = threadIdx.x >> 6, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const Seq s = load_seq(q_lens, kv_lens, b, m.Nq, m.Nk);
    const bool far = x >= m.ntiles;
    const int tile = far ? (x - m.ntiles) / f.n_far : x, chunk = far ? (x - m.ntiles) % f.n_far : 0;
    const int j0 = tile * BM;
    const bool sink = f.n_far > 0 && j0 < m.sinks;   // rows j < sinks go to the partial sums
    const RowRange rr = far ? rows_of_far(s, j0, BM, m.window, f.far_rows, chunk)
                            : rows_of_tile(s, j0, BM, m.window, m.sinks, sink);
    const int nr = (rr.i1 - rr.i0 + N - 1) / N, n_all = nr * m.G;
    const int jw = j0 + 16 * warp;
    float ak[D / 8][4], av[D / 8][4];
#pragma unroll
    for (int e = 0; e < D / 8; ++e)
#pragma unroll
        for (int i = 0; i < 4; ++i) ak[e][i] = av[e][i] = 0.f;
    auto fetch = [&](int u) {
        const int h = hk * m.G + u / nr, i0 = rr.i0 + u % nr * N, at = (u & 1) * N;
        load_tile<T, D, N>(Qs + at * LD<D>, q, b, h, i0, rr.i1);
        load_tile<T, D, N>(Os + at * LD<D>, dO, b, h, i0, rr.i1);
        if (threadIdx.x < N) {                        // rows past the range: P = exp2(x - inf) = 0
            const int i = i0 + threadIdx.x;
            const size_t row = ((size_t)b * m.Hq + h) * m.npad + i;
            Ls[at + threadIdx.x] = i < rr.i1 ? __ldcg(negl + row) : -INFINITY;
            Ds[at + threadIdx.x] = i < rr.i1 ? __ldcg(Drow + row) : 0.f;
        }
    };
    if (n_all > 0) {
        load_tile<T, D, BM>(Ks, k, b, hk, j0, s.kl);
        load_tile<T, D, BM>(Vs, v, b, hk, j0, s.kl);
        fetch(0);
        cp_async_commit();
        cp_async_wait<0>();
        __syncthreads();
        split_tile<T, D>(Ks);
        split_tile<T, D>(Vs);
    }
    for (int u = 0; u < n_all; ++u) {
        cp_async_wait<0>();
        __syncthreads();                              // tile u is there, and tile u - 1 done with
        if (u + 1 < n_all) fetch(u + 1);
        cp_async_commit();
        const int at = (u & 1) * N + slice * H, p0 = rr.i0 + u % nr * N + slice * H + s.off;
        // (rows past the range are 0 and their P too)
        if (p0 + H - 1 >= jw && (p0 < jw + 15 + m.window || jw < m.sinks)) {
            const float *Q = Qs + at * LD<D>, *O = Os + at * LD<D>;
            float c[NT][4], dp[NT][4];
            mm_nt<D, NT, EX>(c, Ks + 16 * warp * LD<D>, Q, g, t);
            mm_nt<D, NT, EX>(dp, Vs + 16 * warp * LD<D>, O, g, t);
            const bool whole = p0 >= jw + 15 && p0 + H - 1 < jw + m.window;
            const int j[2] = {jw + g - p0 - 2 * t, jw + g + 8 - p0 - 2 * t};   // a row's place less a key's
            score_grads<NT, true>(c, dp, Ls + at + 2 * t, Ds + at + 2 * t, m.scale_log2, whole, [&](int n, int i) {
                const int x = 8 * n + (i & 1);
                return !(x >= j[i >> 1] && (x < j[i >> 1] + m.window || jw + g + 8 * (i >> 1) < m.sinks));
            });
            mm_pn<D, NT, EX, true>(av, c, O, g, t);
            mm_pn<D, NT, EX, false>(ak, dp, Q, g, t);
        }
    }
    __syncthreads();
    float* other = Qs + threadIdx.x % 64;
    if (slice) put_acc<D>(other + (slice - 1) * 64 * D, ak), put_acc<D>(other + (slice - 1) * 64 * D + 32 * D, av);
    __syncthreads();
    if (slice) return;
    for (int x = 0; x < kParts - 1; ++x) add_acc<D>(ak, other + x * 64 * D), add_acc<D>(av, other + x * 64 * D + 32 * D);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int j = jw + g + 8 * i;
        if (!sink || j >= m.sinks) continue;
        float* p = part + (((size_t)bk * (1 + f.n_far) + (far ? 1 + chunk : 0)) * 2 * m.sinks + j) * D;
#pragma unroll
        for (int e = 0; e < D / 8; ++e) {
            const int c = 8 * e + 2 * t;
            *reinterpret_cast<float2*>(p + c) = make_float2(ak[e][2 * i], ak[e][2 * i + 1]);
            *reinterpret_cast<float2*>(p + (size_t)m.sinks * D + c) = make_float2(av[e][2 * i], av[e][2 * i + 1]);
        }
    }
    if (far) return;
    // (the sinks among these rows are written again from the sums)
    const float mk[2] = {m.scale, m.scale}, mv[2] = {1.f, 1.f};
    store_rows<T, D>(dk, b, hk, jw, m.Nk, ak, mk, g, t);
    store_rows<T, D>(dv, b, hk, jw, m.Nk, av, mv, g, t);
}

// dK, dV of the sink rows: the partial sums in slot order, one thread per element.
template <typename T>
__global__ void __launch_bounds__(kT)
sum_far_kernel(V dk, V dv, const float* __restrict__ part, int slots, int Hkv, int sinks, int d, float scale, long long n) {
    const long long x = (long long)blockIdx.x * kT + threadIdx.x;
    if (x >= n) return;
    const int e = (int)(x % d), j = (int)(x / d % sinks);
    const long long r = x / d / sinks;
    const int which = (int)(r & 1);
    const long long bk = r >> 1;
    const int b = (int)(bk / Hkv), hk = (int)(bk % Hkv);
    const float* p = part + ((bk * slots * 2 + which) * sinks + j) * d + e;
    float acc = 0.f;
    for (int c = 0; c < slots; ++c) acc += p[(size_t)c * 2 * sinks * d];
    const V& o = which ? dv : dk;
    static_cast<T*>(const_cast<void*>(o.base))[b * o.sB + hk * o.sH + j * o.sN + e * o.sJ] =
        from_f32<T>(which ? acc : acc * scale);
}

// `beside`: starts while dK, dV runs, whose blocks have all waited for the statistics, but
// waits for nothing itself.  An early start orders no memory, so that what an SM's L1 holds
// from before may be older than what it reads: all of it is read past L1, from L2, where
// the finished kernels' writes are.
template <typename T, int D>
__global__ void __launch_bounds__(kW, kBlocks<D>)
warp_dq_kernel(V q, V k, V v, V dO, V dq, const float* __restrict__ negl, const float* __restrict__ Drow,
               const int* __restrict__ q_lens, const int* __restrict__ kv_lens, Dims m, bool beside) {
    constexpr int N = BN, H = N / kParts, NT = H / 8;
    constexpr bool EX = sizeof(T) == 2;
    extern __shared__ __align__(16) float sm[];
    if (!beside) tc::griddep_wait();
    float *Qs = sm, *Os = Qs + 2 * BM * LD<D>, *Ks = Os + 2 * BM * LD<D>, *Vs = Ks + 2 * N * LD<D>;
    const int bh = blockIdx.x / m.ntiles, i0 = (int)(blockIdx.x % m.ntiles) * BM;
    const int b = bh / m.Hq, h = bh % m.Hq, hk = h / m.G;
    const int warp = threadIdx.x >> 5 & 1, slice = threadIdx.x >> 6, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const Seq s = load_seq(q_lens, kv_lens, b, m.Nq, m.Nk);
    const int i1 = min(i0 + BM, s.ql);
    const KeyTiles kt = key_tiles<N>(s, i0, i1, m.window, m.sinks);
    const int nk = kt.count(), r0 = i0 + 16 * warp;
    const int p[2] = {r0 + g < s.ql ? r0 + g + s.off : -1, r0 + g + 8 < s.ql ? r0 + g + 8 + s.off : -1};
    // of the warp's 16 rows, whether some see some and whether all see all of keys j .. j + H - 1
    const int pf = r0 + s.off, pl = min(r0 + 16, s.ql) - 1 + s.off;
    auto sees_some = [&](int j) { return r0 < s.ql && j <= pl && (j + H - 1 > pf - m.window || j < m.sinks); };
    auto sees_all = [&](int j) { return r0 + 16 <= s.ql && j + H - 1 <= pf && j > pl - m.window; };
    const size_t row = (size_t)bh * m.npad + r0 + g;  // the arrays hold whole 128-row tiles
    const float L[2] = {__ldcg(negl + row), __ldcg(negl + row + 8)}, Dr[2] = {__ldcg(Drow + row), __ldcg(Drow + row + 8)};
    float acc[D / 8][4];
#pragma unroll
    for (int f = 0; f < D / 8; ++f)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[f][i] = 0.f;
    auto fetch = [&](int u) {
        const int j0 = kt.tile(u) * N;
        load_tile<T, D, N, true>(Ks + (u & 1) * N * LD<D>, k, b, hk, j0, s.kl);
        load_tile<T, D, N, true>(Vs + (u & 1) * N * LD<D>, v, b, hk, j0, s.kl);
    };
    if (nk > 0) {
        load_tile<T, D, BM, true>(Qs, q, b, h, i0, s.ql);
        load_tile<T, D, BM, true>(Os, dO, b, h, i0, s.ql);
        fetch(0);
        cp_async_commit();
        cp_async_wait<0>();
        __syncthreads();
        split_tile<T, D>(Qs);
        split_tile<T, D>(Os);
    }
    for (int u = 0; u < nk; ++u) {
        cp_async_wait<0>();
        __syncthreads();                              // tile u is there, and tile u - 1 done with
        if (u + 1 < nk) fetch(u + 1);
        cp_async_commit();
        const int jh = kt.tile(u) * N + slice * H;
        if (sees_some(jh)) {
            const float *K = Ks + ((u & 1) * N + slice * H) * LD<D>, *W = Vs + ((u & 1) * N + slice * H) * LD<D>;
            float c[NT][4], dp[NT][4];
            mm_nt<D, NT, EX>(c, Qs + 16 * warp * LD<D>, K, g, t);
            mm_nt<D, NT, EX>(dp, Os + 16 * warp * LD<D>, W, g, t);
            const int at[2] = {p[0] - jh - 2 * t, p[1] - jh - 2 * t}, sink = m.sinks - jh - 2 * t;
            score_grads<NT, false>(c, dp, L, Dr, m.scale_log2, sees_all(jh), [&](int n, int i) {
                const int x = 8 * n + (i & 1);
                return !(x <= at[i >> 1] && (x > at[i >> 1] - m.window || x < sink));
            });
            mm_pn<D, NT, EX, false>(acc, dp, K, g, t);
        }
    }
    __syncthreads();
    float* other = Ks + threadIdx.x % 64;
    if (slice) put_acc<D>(other + (slice - 1) * 32 * D, acc);
    __syncthreads();
    if (slice) return;
    for (int x = 0; x < kParts - 1; ++x) add_acc<D>(acc, other + x * 32 * D);
    const float mul[2] = {m.scale, m.scale};
    store_rows<T, D>(dq, b, h, r0, m.Nq, acc, mul, g, t);
    tc::griddep_wait();                                   // done only when the kernel before is
}

int launched(const char* what, std::string* err) {
    const cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) return PSA_OK;
    *err = std::string(what) + ": " + cudaGetErrorString(e);
    return PSA_ERR_CUDA;
}

bool grid_ok(long long g, std::string* err) {
    if (g <= 0x7fffffffll) return true;
    *err = "grid too large";
    return false;
}

Dims dims(const Args& a, int n) {
    return Dims{a.Hq, a.Hq / a.Hkv, a.Nq, a.Nk, a.window, a.sinks, (n + BM - 1) / BM, stat_rows(a.Nq), a.scale,
                a.scale * kLog2e};
}

template <typename T, int D>
int launch_fwd(const Args& a, std::string* err) {
    const Dims m = dims(a, a.Nq);
    const long long grid = (long long)a.B * a.Hq * m.ntiles;
    if (grid == 0) return PSA_OK;
    if (!grid_ok(grid, err)) return PSA_ERR_UNSUPPORTED;
    if (!set_max_dynamic_smem((const void*)warp_fwd_kernel<T, D>, fwd_smem<D>(), err)) return PSA_ERR_CUDA;
    ProfScope prof(kSlotFwd, a.stream);
    constexpr int e = sizeof(T);
    warp_fwd_kernel<T, D><<<(unsigned)grid, kW, fwd_smem<D>(), a.stream>>>(
        dev_view(a.q, e), dev_view(a.k, e), dev_view(a.v, e), dev_view(a.o, e), a.lse, a.q_lens, a.kv_lens, m);
    return launched("window attention forward launch", err);
}

template <typename T, int D>
int launch_pre(const Args& a, std::string* err) {
    const long long grid = (long long)a.B * a.Hq * (stat_rows(a.Nq) / Pre<T, D>::ROWS);
    if (grid == 0) return PSA_OK;
    if (!grid_ok(grid, err)) return PSA_ERR_UNSUPPORTED;
    const V o = dev_view(a.o, sizeof(T)), d = dev_view(a.dO, sizeof(T));
    ProfScope prof(kSlotPre, a.stream);
    pre_d_kernel<T, D><<<(unsigned)grid, kPre, 0, a.stream>>>(o, d, a.lse, a.Drow, a.negl, static_cast<__nv_bfloat16*>(a.aug),
                                                            a.q_lens, a.Hq, a.Nq, stat_rows(a.Nq),
                                                            1.f / (a.scale * kLog2e));
    return launched("window attention D launch", err);
}

template <typename T, int D>
int launch_bwd(const Args& a, std::string* err) {
    Args s = a;
    s.aug = nullptr;
    const FarSplit f = far_split(a.Nk, a.window, a.sinks);
    const Dims mk = dims(a, a.Nk), mq = dims(a, a.Nq);
    const int items = mk.ntiles + f.n_far * ((a.sinks + BM - 1) / BM);
    const long long gk = (long long)a.B * a.Hkv * items, gq = (long long)a.B * a.Hq * mq.ntiles;
    if (!grid_ok(gk, err) || !grid_ok(gq, err)) return PSA_ERR_UNSUPPORTED;
    if (!set_max_dynamic_smem((const void*)warp_dkdv_kernel<T, D>, bwd_smem<D>(), err) ||
        !set_max_dynamic_smem((const void*)warp_dq_kernel<T, D>, bwd_smem<D>(), err))
        return PSA_ERR_CUDA;
    const int rc = launch_pre<T, D>(s, err);
    if (rc) return rc;
    constexpr int e = sizeof(T);
    // dQ beside dK, dV where all its inputs load 16 bytes at a time (past L1); element by
    // element past L1 would fetch a sector for each, so those layouts wait
    const bool beside = gk > 0 && view_16(a.q, e) && view_16(a.k, e) && view_16(a.v, e) && view_16(a.dO, e);
    cudaError_t c = cudaSuccess;
    if (gk > 0) {
        ProfScope prof(kSlotMain, a.stream);
        c = launch_beside(warp_dkdv_kernel<T, D>, (unsigned)gk, kW, 1, bwd_smem<D>(), a.stream, dev_view(a.q, e), dev_view(a.k, e),
                          dev_view(a.v, e), dev_view(a.dO, e), dev_view(a.dk, e), dev_view(a.dv, e), a.negl, a.Drow, a.part,
                          a.q_lens, a.kv_lens, mk, f, items, a.Hkv);
    }
    if (c == cudaSuccess && gq > 0) {
        ProfScope prof(kSlotDq, a.stream);
        c = launch_beside(warp_dq_kernel<T, D>, (unsigned)gq, kW, 1, bwd_smem<D>(), a.stream, dev_view(a.q, e), dev_view(a.k, e),
                          dev_view(a.v, e), dev_view(a.dO, e), dev_view(a.dq, e), a.negl, a.Drow, a.q_lens, a.kv_lens, mq,
                          beside);
    }
    if (c != cudaSuccess) {
        *err = std::string("window attention backward launch: ") + cudaGetErrorString(c);
        return PSA_ERR_CUDA;
    }
    return f.n_far ? sum_far(a, f, err) : PSA_OK;
}

}  // namespace

#define WIN_DISPATCH(FN, a, err)                                                                              \
    switch ((a).d) {                                                                                          \
        case 16: return (a).dtype == PSA_F32 ? FN<float, 16>(a, err) : FN<__nv_bfloat16, 16>(a, err);         \
        case 32: return (a).dtype == PSA_F32 ? FN<float, 32>(a, err) : FN<__nv_bfloat16, 32>(a, err);         \
        case 64: return (a).dtype == PSA_F32 ? FN<float, 64>(a, err) : FN<__nv_bfloat16, 64>(a, err);         \
        default: return (a).dtype == PSA_F32 ? FN<float, 128>(a, err) : FN<__nv_bfloat16, 128>(a, err);       \
    }

int warp_fwd(const Args& a, std::string* err) { WIN_DISPATCH(launch_fwd, a, err) }
int warp_bwd(const Args& a, std::string* err) { WIN_DISPATCH(launch_bwd, a, err) }
int pre_d(const Args& a, std::string* err) { WIN_DISPATCH(launch_pre, a, err) }

int sum_far(const Args& a, const FarSplit& f, std::string* err) {
    const long long n = (long long)a.B * a.Hkv * 2 * a.sinks * a.d, grid = (n + kT - 1) / kT;
    if (!grid_ok(grid, err)) return PSA_ERR_UNSUPPORTED;
    ProfScope prof(kSlotMain, a.stream);
    if (a.dtype == PSA_F32)
        sum_far_kernel<float><<<(unsigned)grid, kT, 0, a.stream>>>(dev_view(a.dk, 4), dev_view(a.dv, 4), a.part,
                                                                   1 + f.n_far, a.Hkv, a.sinks, a.d, a.scale, n);
    else
        sum_far_kernel<__nv_bfloat16><<<(unsigned)grid, kT, 0, a.stream>>>(
            dev_view(a.dk, 2), dev_view(a.dv, 2), a.part, 1 + f.n_far, a.Hkv, a.sinks, a.d,
            a.scale, n);
    return launched("window attention sink rows launch", err);
}

}  // namespace win
}  // namespace psa
