// win_simt.cu -- sliding-window attention with sinks on the CUDA cores: the
// fp32 path (fp32 results need full fp32 products), and bf16 in layouts that
// the tensor-core path does not take.
//
//   forward : per 64-row tile, online softmax over the 64-key tiles it sees
//   D       : D_i = <dO_i, O_i>
//   dK, dV  : per 64-key tile, over the rows that see it, all query heads of
//             the key head in turn:  P = exp(S - LSE), dS = P (dO V^T - D),
//             dV += P^T dO, dK += dS^T Q   (sums over heads need no atomics)
//   dQ      : per 64-row tile, over the keys it sees: dQ += dS K
//
// 256 threads as 16 x 16; every product is a register-tiled outer product from
// shared memory (4 rows x 4 columns, or 4 rows x D/16 columns, per thread): at
// d = 64 twelve 16-byte shared reads feed 64 FFMAs, which keeps the FFMA pipe,
// not shared memory, the bound.  Rows are padded by 4 floats, so that the
// 16-byte reads of 8 neighbouring rows fall into distinct banks.
#include <cuda_bf16.h>

#include <string>

#include "common.cuh"
#include "psa_internal.h"
#include "tc_tmap.h"
#include "win_geom.cuh"
#include "win_internal.h"

namespace psa {
namespace win {
namespace {

constexpr int kT = 256;
constexpr int BM = 64;      // rows and keys per tile
constexpr int PS = BM + 4;  // row stride of the score tiles

template <int D>
constexpr int LD = D + 4;   // row stride of the operand tiles

struct V {                  // a view's element strides, and whether 4 features load at once
    const void* base;
    long long sB, sH, sN, sJ;
    int vec;
};

template <typename T>
bool view_vec(const View& v) {
    const size_t a = 4 * sizeof(T);
    return v.sJ == 1 && v.sB % 4 == 0 && v.sH % 4 == 0 && v.sN % 4 == 0 &&
           reinterpret_cast<uintptr_t>(v.base) % a == 0;
}
// 16 bytes of a row at once.
bool view_16(const View& v, int esize) {
    const long long w = 16 / esize;
    return v.sJ == 1 && v.sB % w == 0 && v.sH % w == 0 && v.sN % w == 0 && reinterpret_cast<uintptr_t>(v.base) % 16 == 0;
}
template <typename T>
V dev_view(const View& v) {
    return V{v.base, v.sB, v.sH, v.sN, v.sJ, view_vec<T>(v) ? 1 : 0};
}

// Rows [r0, r0 + 64) of head (b, h) to a shared tile; rows >= n are zero and
// are not read.
template <typename T, int D>
__device__ __forceinline__ void load_tile(float* s, const V& v, int b, int h, int r0, int n) {
    const T* base = static_cast<const T*>(v.base) + b * v.sB + h * v.sH;
    for (int idx = threadIdx.x; idx < BM * (D / 4); idx += kT) {
        const int r = idx / (D / 4), g = 4 * (idx % (D / 4));
        float x[4] = {0.f, 0.f, 0.f, 0.f};
        if (r0 + r < n) {
            const T* p = base + (long long)(r0 + r) * v.sN + (long long)g * v.sJ;
            if (v.vec) {
                load4(p, x);
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) x[e] = to_f32(p[e * v.sJ]);
            }
        }
        *reinterpret_cast<float4*>(s + r * LD<D> + g) = make_float4(x[0], x[1], x[2], x[3]);
    }
}

// c[r][q] = <A row 4ty + r, B row tx + 16q>
template <int D>
__device__ __forceinline__ void mm_nt(float (&c)[4][4], const float* A, const float* B, int ty, int tx) {
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int q = 0; q < 4; ++q) c[r][q] = 0.f;
#pragma unroll 4
    for (int k = 0; k < D; k += 4) {
        float4 a[4], b[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) a[r] = *reinterpret_cast<const float4*>(A + (4 * ty + r) * LD<D> + k);
#pragma unroll
        for (int q = 0; q < 4; ++q) b[q] = *reinterpret_cast<const float4*>(B + (tx + 16 * q) * LD<D> + k);
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                c[r][q] = fmaf(a[r].x, b[q].x, c[r][q]);
                c[r][q] = fmaf(a[r].y, b[q].y, c[r][q]);
                c[r][q] = fmaf(a[r].z, b[q].z, c[r][q]);
                c[r][q] = fmaf(a[r].w, b[q].w, c[r][q]);
            }
    }
}

// D / 16 features of a row per thread: in groups of W = min(4, D/16) at
// W tx + 16 W g.
template <int D>
struct Cols {
    static constexpr int N = D / 16, W = N < 4 ? N : 4, G = N / W;
};
template <int D>
__device__ __forceinline__ void load_cols(float (&x)[D / 16], const float* row, int tx) {
    constexpr int W = Cols<D>::W;
#pragma unroll
    for (int g = 0; g < Cols<D>::G; ++g) {
        const float* p = row + W * tx + 16 * W * g;
        if (W == 4) {
            const float4 v = *reinterpret_cast<const float4*>(p);
            x[4 * g] = v.x, x[4 * g + 1] = v.y, x[4 * g + 2] = v.z, x[4 * g + 3] = v.w;
        } else if (W == 2) {
            const float2 v = *reinterpret_cast<const float2*>(p);
            x[0] = v.x, x[1] = v.y;
        } else {
            x[0] = *p;
        }
    }
}

// acc[r][.] += sum_j P[4ty + r][j] * B[j][.]
template <int D>
__device__ __forceinline__ void mm_nn(float (&acc)[4][D / 16], const float* P, const float* B, int ty, int tx) {
#pragma unroll 2
    for (int j = 0; j < BM; j += 4) {
        float4 p[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) p[r] = *reinterpret_cast<const float4*>(P + (4 * ty + r) * PS + j);
#pragma unroll
        for (int jj = 0; jj < 4; ++jj) {
            float x[D / 16];
            load_cols<D>(x, B + (j + jj) * LD<D>, tx);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const float w = jj == 0 ? p[r].x : jj == 1 ? p[r].y : jj == 2 ? p[r].z : p[r].w;
#pragma unroll
                for (int e = 0; e < D / 16; ++e) acc[r][e] = fmaf(w, x[e], acc[r][e]);
            }
        }
    }
}

// acc[c][.] += sum_i P[i][4ty + c] * B[i][.]
template <int D>
__device__ __forceinline__ void mm_tn(float (&acc)[4][D / 16], const float* P, const float* B, int ty, int tx) {
#pragma unroll 4
    for (int i = 0; i < BM; ++i) {
        const float4 p = *reinterpret_cast<const float4*>(P + i * PS + 4 * ty);
        float x[D / 16];
        load_cols<D>(x, B + i * LD<D>, tx);
#pragma unroll
        for (int e = 0; e < D / 16; ++e) {
            acc[0][e] = fmaf(p.x, x[e], acc[0][e]);
            acc[1][e] = fmaf(p.y, x[e], acc[1][e]);
            acc[2][e] = fmaf(p.z, x[e], acc[2][e]);
            acc[3][e] = fmaf(p.w, x[e], acc[3][e]);
        }
    }
}

// One row's D / 16 features of this thread to row n of head (b, h).
template <typename T, int D>
__device__ __forceinline__ void store_cols(const V& v, int b, int h, int n, const float (&x)[D / 16], float mul, int tx) {
    constexpr int W = Cols<D>::W;
    T* row = static_cast<T*>(const_cast<void*>(v.base)) + b * v.sB + h * v.sH + (long long)n * v.sN;
#pragma unroll
    for (int g = 0; g < Cols<D>::G; ++g) {
        const int c = W * tx + 16 * W * g;
        if (W == 4 && v.vec) {
            const float y[4] = {x[4 * g] * mul, x[(4 * g + 1) % (D / 16)] * mul, x[(4 * g + 2) % (D / 16)] * mul,
                                x[(4 * g + 3) % (D / 16)] * mul};
            store4(row + c, y);
        } else {
#pragma unroll
            for (int e = 0; e < W; ++e) row[(long long)(c + e) * v.sJ] = from_f32<T>(x[W * g + e] * mul);
        }
    }
}

// Sum and maximum over the 16 threads of a row.
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
    for (int m = 1; m < 16; m <<= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
    return x;
}
__device__ __forceinline__ float row_max(float x) {
#pragma unroll
    for (int m = 1; m < 16; m <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, m));
    return x;
}

struct Dims {
    int Hq, G, Nq, Nk, window, sinks, ntiles, npad;
    float scale, scale_log2;
};

template <int D>
constexpr int fwd_smem() {
    return (3 * BM * LD<D> + BM * PS) * 4;
}
template <int D>
constexpr int bwd_smem(int scores) {
    return (4 * BM * LD<D> + scores * BM * PS + 2 * BM) * 4;
}

template <typename T, int D>
__global__ void __launch_bounds__(kT)
simt_fwd_kernel(V q, V k, V v, V o, float* __restrict__ lse, const int* __restrict__ q_lens,
                const int* __restrict__ kv_lens, Dims m) {
    extern __shared__ __align__(16) float sm[];
    float *Qs = sm, *Ks = Qs + BM * LD<D>, *Vs = Ks + BM * LD<D>, *Ps = Vs + BM * LD<D>;
    const int bh = blockIdx.x / m.ntiles, i0 = (int)(blockIdx.x % m.ntiles) * BM;
    const int b = bh / m.Hq, h = bh % m.Hq, hk = h / m.G;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const Seq s = load_seq(q_lens, kv_lens, b, m.Nq, m.Nk);
    const KeyTiles kt = key_tiles<BM>(s, i0, min(i0 + BM, s.ql), m.window, m.sinks);
    load_tile<T, D>(Qs, q, b, h, i0, s.ql);
    float mx[4], l[4], acc[4][D / 16];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        mx[r] = -INFINITY, l[r] = 0.f;
#pragma unroll
        for (int e = 0; e < D / 16; ++e) acc[r][e] = 0.f;
    }
    for (int t = 0; t < kt.count(); ++t) {
        const int j0 = kt.tile(t) * BM;
        __syncthreads();
        load_tile<T, D>(Ks, k, b, hk, j0, s.kl);
        load_tile<T, D>(Vs, v, b, hk, j0, s.kl);
        __syncthreads();
        float c[4][4];
        mm_nt<D>(c, Qs, Ks, ty, tx);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int i = i0 + 4 * ty + r, p = i < s.ql ? i + s.off : -1;
            float mt = -INFINITY;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                c[r][e] = sees(p, j0 + tx + 16 * e, m.window, m.sinks) ? c[r][e] * m.scale_log2 : -INFINITY;
                mt = fmaxf(mt, c[r][e]);
            }
            const float m_new = fmaxf(mx[r], row_max(mt));
            const float ref = m_new == -INFINITY ? 0.f : m_new;   // nothing seen yet: exp2(-inf) = 0
            const float alpha = exp2f(mx[r] - ref);
            float sum = 0.f;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float pr = exp2f(c[r][e] - ref);
                sum += pr;
                Ps[(4 * ty + r) * PS + tx + 16 * e] = pr;
            }
            l[r] = l[r] * alpha + row_sum(sum);
            mx[r] = m_new;
#pragma unroll
            for (int e = 0; e < D / 16; ++e) acc[r][e] *= alpha;
        }
        __syncwarp();   // a row's 16 threads share a half warp
        mm_nn<D>(acc, Ps, Vs, ty, tx);
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int i = i0 + 4 * ty + r;
        if (i >= m.Nq) break;
        const bool some = l[r] > 0.f || l[r] != l[r];
        store_cols<T, D>(o, b, h, i, acc[r], some ? 1.f / l[r] : 0.f, tx);
        if (tx == 0) lse[(size_t)bh * m.Nq + i] = some ? (mx[r] + log2f(l[r])) * kLn2 : -INFINITY;
    }
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
// Bound by memory: a block takes a 128-row tile of a head, 16 bytes a thread and
// four rows in flight (B=1, 16 heads, N=8192, d=128 in bf16: XX us, 67 MB).
template <typename T, int D>
__global__ void __launch_bounds__(kT)
pre_d_kernel(V o, V dO, const float* __restrict__ lse, float* __restrict__ Drow, float* __restrict__ negl,
             __nv_bfloat16* __restrict__ aug, const int* __restrict__ q_lens, int Hq, int Nq, int npad, float inv_c) {
    constexpr int E = 16 / (int)sizeof(T), TR = D / E, R = kT / TR;   // features a thread, threads a row, rows a pass
    constexpr int P = 128 / R, U = P < 4 ? P : 4;
    // neighbouring blocks take the heads of the same rows: in token-major memory those
    // are neighbours (heads one after the other read a 256-byte piece every few KB)
    const int nb = npad / 128, bt = blockIdx.x / Hq, h = blockIdx.x - (unsigned)bt * Hq;
    const int b = bt / nb, i0 = (bt - b * nb) * 128, bh = b * Hq + h;
    const int ql = q_lens ? min(__ldg(q_lens + b), Nq) : Nq;
    const int r0 = threadIdx.x / TR, g = E * (threadIdx.x % TR);
    const T* po = static_cast<const T*>(o.base) + b * o.sB + h * o.sH + g * o.sJ;
    const T* pd = static_cast<const T*>(dO.base) + b * dO.sB + h * dO.sH + g * dO.sJ;
    const bool vec = o.vec && dO.vec;
    for (int p = 0; p < P; p += U) {
        float s[U];
        if (vec) {
            uint4 x[U], y[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int n = i0 + (p + u) * R + r0;
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
                const int n = i0 + (p + u) * R + r0;
                s[u] = 0.f;
                if (n < ql)
#pragma unroll
                    for (int e = 0; e < E; ++e)
                        s[u] = fmaf(to_f32(po[n * o.sN + e * o.sJ]), to_f32(pd[n * dO.sN + e * dO.sJ]), s[u]);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
#pragma unroll
            for (int w = TR / 2; w; w >>= 1) s[u] += __shfl_xor_sync(0xffffffffu, s[u], w);
            const int n = i0 + (p + u) * R + r0;
            if (g != 0) continue;
            const size_t row = (size_t)bh * npad + n;
            float L = n < ql ? lse[(size_t)bh * Nq + n] : -INFINITY;
            L = L == -INFINITY ? L : -L * kLog2e;
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
}

// P and dS of the 64 x 64 tile (rows i0.., keys j0..): P to Ps (when given), dS to Ss.
template <int D, bool WANT_P>
__device__ __forceinline__ void score_grads(float* Ps, float* Ss, const float* Qs, const float* Ks, const float* dOs,
                                            const float* Vs, const float* Ls, const float* Ds, const Seq& s, int i0,
                                            int j0, const Dims& m, int ty, int tx) {
    float c[4][4], dp[4][4];
    mm_nt<D>(c, Qs, Ks, ty, tx);
    mm_nt<D>(dp, dOs, Vs, ty, tx);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int ii = 4 * ty + r, i = i0 + ii, p = i < s.ql ? i + s.off : -1;
        const float L = Ls[ii], Di = Ds[ii];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int j = j0 + tx + 16 * e;
            const float pr = sees(p, j, m.window, m.sinks) ? exp2f(fmaf(c[r][e], m.scale_log2, L)) : 0.f;
            if (WANT_P) Ps[ii * PS + tx + 16 * e] = pr;
            Ss[ii * PS + tx + 16 * e] = pr * (dp[r][e] - Di);
        }
    }
}

// Statistics of rows i0 .. to shared memory (rows behind the arrays' last tile are not there).
__device__ __forceinline__ void load_stats(float* Ls, float* Ds, const float* negl, const float* Drow, size_t row0,
                                           int i0, int npad) {
    if (threadIdx.x < BM) {
        const int i = i0 + threadIdx.x;
        Ls[threadIdx.x] = i < npad ? negl[row0 + i] : -INFINITY;
        Ds[threadIdx.x] = i < npad ? Drow[row0 + i] : 0.f;
    }
}

// One work item of a key head: a 64-key tile and the rows that see it (x <
// nkt), or far chunk c of a tile with sinks.
template <typename T, int D>
__global__ void __launch_bounds__(kT)
simt_dkdv_kernel(V q, V k, V v, V dO, V dk, V dv, const float* __restrict__ negl, const float* __restrict__ Drow,
                 float* __restrict__ part, const int* __restrict__ q_lens, const int* __restrict__ kv_lens, Dims m,
                 FarSplit f, int items, int Hkv) {
    extern __shared__ __align__(16) float sm[];
    float *Ks = sm, *Vs = Ks + BM * LD<D>, *Qs = Vs + BM * LD<D>, *Os = Qs + BM * LD<D>, *Ps = Os + BM * LD<D>,
          *Ss = Ps + BM * PS, *Ls = Ss + BM * PS, *Ds = Ls + BM;
    const int bk = blockIdx.x / items, x = blockIdx.x % items;
    const int b = bk / Hkv, hk = bk % Hkv;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const Seq s = load_seq(q_lens, kv_lens, b, m.Nq, m.Nk);
    const int nkt = m.ntiles;
    const bool far = x >= nkt;
    const int tile = far ? (x - nkt) / f.n_far : x, chunk = far ? (x - nkt) % f.n_far : 0;
    const int j0 = tile * BM;
    const bool sink = f.n_far > 0 && j0 < m.sinks;   // rows j < sinks go to the partial sums
    const RowRange rr = far ? rows_of_far(s, j0, BM, m.window, f.far_rows, chunk)
                            : rows_of_tile(s, j0, BM, m.window, m.sinks, sink);
    float ak[4][D / 16], av[4][D / 16];
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int e = 0; e < D / 16; ++e) ak[r][e] = av[r][e] = 0.f;
    if (rr.i1 > rr.i0) {
        load_tile<T, D>(Ks, k, b, hk, j0, s.kl);
        load_tile<T, D>(Vs, v, b, hk, j0, s.kl);
        // rows before and behind the range see none of its keys (or belong to
        // another item): the tile starts at i0 itself, and ql ends it
        Seq cut = s;
        cut.ql = rr.i1;
        for (int g = 0; g < m.G; ++g) {
            const int h = hk * m.G + g;
            const size_t row0 = ((size_t)b * m.Hq + h) * m.npad;
            for (int i0 = rr.i0; i0 < rr.i1; i0 += BM) {
                __syncthreads();
                load_tile<T, D>(Qs, q, b, h, i0, rr.i1);
                load_tile<T, D>(Os, dO, b, h, i0, rr.i1);
                load_stats(Ls, Ds, negl, Drow, row0, i0, m.npad);
                __syncthreads();
                score_grads<D, true>(Ps, Ss, Qs, Ks, Os, Vs, Ls, Ds, cut, i0, j0, m, ty, tx);
                __syncthreads();
                mm_tn<D>(av, Ps, Os, ty, tx);
                mm_tn<D>(ak, Ss, Qs, ty, tx);
            }
        }
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int j = j0 + 4 * ty + r;
        if (j >= m.Nk) break;
        if (sink && j < m.sinks) {
            float* p = part + (((size_t)bk * (1 + f.n_far) + (far ? 1 + chunk : 0)) * 2 * m.sinks + j) * D;
            constexpr int W = Cols<D>::W;
#pragma unroll
            for (int e = 0; e < D / 16; ++e) {
                const int c = W * tx + 16 * W * (e / W) + e % W;
                p[c] = ak[r][e];
                p[(size_t)m.sinks * D + c] = av[r][e];
            }
        } else if (!far) {
            store_cols<T, D>(dk, b, hk, j, ak[r], m.scale, tx);
            store_cols<T, D>(dv, b, hk, j, av[r], 1.f, tx);
        }
    }
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

template <typename T, int D>
__global__ void __launch_bounds__(kT)
simt_dq_kernel(V q, V k, V v, V dO, V dq, const float* __restrict__ negl, const float* __restrict__ Drow,
               const int* __restrict__ q_lens, const int* __restrict__ kv_lens, Dims m) {
    extern __shared__ __align__(16) float sm[];
    float *Qs = sm, *Os = Qs + BM * LD<D>, *Ks = Os + BM * LD<D>, *Vs = Ks + BM * LD<D>, *Ss = Vs + BM * LD<D>,
          *Ls = Ss + BM * PS, *Ds = Ls + BM;
    const int bh = blockIdx.x / m.ntiles, i0 = (int)(blockIdx.x % m.ntiles) * BM;
    const int b = bh / m.Hq, h = bh % m.Hq, hk = h / m.G;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const Seq s = load_seq(q_lens, kv_lens, b, m.Nq, m.Nk);
    const KeyTiles kt = key_tiles<BM>(s, i0, min(i0 + BM, s.ql), m.window, m.sinks);
    float acc[4][D / 16];
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int e = 0; e < D / 16; ++e) acc[r][e] = 0.f;
    if (kt.count() > 0) {
        load_tile<T, D>(Qs, q, b, h, i0, s.ql);
        load_tile<T, D>(Os, dO, b, h, i0, s.ql);
        load_stats(Ls, Ds, negl, Drow, (size_t)bh * m.npad, i0, m.npad);
    }
    for (int t = 0; t < kt.count(); ++t) {
        const int j0 = kt.tile(t) * BM;
        __syncthreads();
        load_tile<T, D>(Ks, k, b, hk, j0, s.kl);
        load_tile<T, D>(Vs, v, b, hk, j0, s.kl);
        __syncthreads();
        score_grads<D, false>(nullptr, Ss, Qs, Ks, Os, Vs, Ls, Ds, s, i0, j0, m, ty, tx);
        __syncwarp();
        mm_nn<D>(acc, Ss, Ks, ty, tx);
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int i = i0 + 4 * ty + r;
        if (i < m.Nq) store_cols<T, D>(dq, b, h, i, acc[r], m.scale, tx);
    }
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
    return Dims{a.Hq, a.Hq / a.Hkv, a.Nq, a.Nk, a.window, a.sinks, (n + BM - 1) / BM, stat_rows(a.Nq), a.scale, a.scale * kLog2e};
}

template <typename T, int D>
int launch_fwd(const Args& a, std::string* err) {
    const Dims m = dims(a, a.Nq);
    const long long grid = (long long)a.B * a.Hq * m.ntiles;
    if (grid == 0) return PSA_OK;
    if (!grid_ok(grid, err)) return PSA_ERR_UNSUPPORTED;
    if (!set_max_dynamic_smem((const void*)simt_fwd_kernel<T, D>, fwd_smem<D>(), err)) return PSA_ERR_CUDA;
    ProfScope prof(kSlotFwd, a.stream);
    simt_fwd_kernel<T, D><<<(unsigned)grid, kT, fwd_smem<D>(), a.stream>>>(
        dev_view<T>(a.q), dev_view<T>(a.k), dev_view<T>(a.v), dev_view<T>(a.o), a.lse, a.q_lens, a.kv_lens, m);
    return launched("window attention forward launch", err);
}

template <typename T, int D>
int launch_pre(const Args& a, std::string* err) {
    const long long grid = (long long)a.B * a.Hq * (stat_rows(a.Nq) / 128);
    if (grid == 0) return PSA_OK;
    if (!grid_ok(grid, err)) return PSA_ERR_UNSUPPORTED;
    V o = dev_view<T>(a.o), d = dev_view<T>(a.dO);
    o.vec = view_16(a.o, sizeof(T)), d.vec = view_16(a.dO, sizeof(T));
    ProfScope prof(kSlotPre, a.stream);
    pre_d_kernel<T, D><<<(unsigned)grid, kT, 0, a.stream>>>(o, d, a.lse, a.Drow, a.negl, static_cast<__nv_bfloat16*>(a.aug),
                                                            a.q_lens, a.Hq, a.Nq, stat_rows(a.Nq),
                                                            1.f / (a.scale * kLog2e));
    return launched("window attention D launch", err);
}

template <typename T, int D>
int launch_bwd(const Args& a, std::string* err) {
    Args b = a;
    b.aug = nullptr;
    int rc = launch_pre<T, D>(b, err);
    if (rc) return rc;
    const FarSplit f = far_split(a.Nk, a.window, a.sinks);
    const Dims mk = dims(a, a.Nk), mq = dims(a, a.Nq);
    const int items = mk.ntiles + f.n_far * ((a.sinks + BM - 1) / BM);
    const long long gk = (long long)a.B * a.Hkv * items, gq = (long long)a.B * a.Hq * mq.ntiles;
    if (!grid_ok(gk, err) || !grid_ok(gq, err)) return PSA_ERR_UNSUPPORTED;
    if (!set_max_dynamic_smem((const void*)simt_dkdv_kernel<T, D>, bwd_smem<D>(2), err) ||
        !set_max_dynamic_smem((const void*)simt_dq_kernel<T, D>, bwd_smem<D>(1), err))
        return PSA_ERR_CUDA;
    if (gk > 0) {
        ProfScope prof(kSlotMain, a.stream);
        simt_dkdv_kernel<T, D><<<(unsigned)gk, kT, bwd_smem<D>(2), a.stream>>>(
            dev_view<T>(a.q), dev_view<T>(a.k), dev_view<T>(a.v), dev_view<T>(a.dO), dev_view<T>(a.dk),
            dev_view<T>(a.dv), a.negl, a.Drow, a.part, a.q_lens, a.kv_lens, mk, f, items, a.Hkv);
        rc = launched("window attention dK/dV launch", err);
    }
    if (!rc && f.n_far) rc = sum_far(a, f, err);
    if (rc || gq == 0) return rc;
    ProfScope prof(kSlotDq, a.stream);
    simt_dq_kernel<T, D><<<(unsigned)gq, kT, bwd_smem<D>(1), a.stream>>>(
        dev_view<T>(a.q), dev_view<T>(a.k), dev_view<T>(a.v), dev_view<T>(a.dO), dev_view<T>(a.dq), a.negl, a.Drow,
        a.q_lens, a.kv_lens, mq);
    return launched("window attention dQ launch", err);
}

}  // namespace

#define WIN_DISPATCH(FN, a, err)                                                                              \
    switch ((a).d) {                                                                                          \
        case 16: return (a).dtype == PSA_F32 ? FN<float, 16>(a, err) : FN<__nv_bfloat16, 16>(a, err);         \
        case 32: return (a).dtype == PSA_F32 ? FN<float, 32>(a, err) : FN<__nv_bfloat16, 32>(a, err);         \
        case 64: return (a).dtype == PSA_F32 ? FN<float, 64>(a, err) : FN<__nv_bfloat16, 64>(a, err);         \
        default: return (a).dtype == PSA_F32 ? FN<float, 128>(a, err) : FN<__nv_bfloat16, 128>(a, err);       \
    }

int simt_fwd(const Args& a, std::string* err) { WIN_DISPATCH(launch_fwd, a, err) }
int simt_bwd(const Args& a, std::string* err) { WIN_DISPATCH(launch_bwd, a, err) }
int pre_d(const Args& a, std::string* err) { WIN_DISPATCH(launch_pre, a, err) }

int sum_far(const Args& a, const FarSplit& f, std::string* err) {
    const long long n = (long long)a.B * a.Hkv * 2 * a.sinks * a.d, grid = (n + kT - 1) / kT;
    if (!grid_ok(grid, err)) return PSA_ERR_UNSUPPORTED;
    ProfScope prof(kSlotMain, a.stream);
    if (a.dtype == PSA_F32)
        sum_far_kernel<float><<<(unsigned)grid, kT, 0, a.stream>>>(dev_view<float>(a.dk), dev_view<float>(a.dv), a.part,
                                                                   1 + f.n_far, a.Hkv, a.sinks, a.d, a.scale, n);
    else
        sum_far_kernel<__nv_bfloat16><<<(unsigned)grid, kT, 0, a.stream>>>(
            dev_view<__nv_bfloat16>(a.dk), dev_view<__nv_bfloat16>(a.dv), a.part, 1 + f.n_far, a.Hkv, a.sinks, a.d,
            a.scale, n);
    return launched("window attention sink rows launch", err);
}

}  // namespace win
}  // namespace psa
