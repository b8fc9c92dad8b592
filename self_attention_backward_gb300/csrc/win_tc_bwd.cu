// win_tc_bwd.cu -- sliding-window attention with sinks, backward, on the tensor
// cores (tcgen05 / TMEM / TMA), bf16 storage.  Two passes, so that nothing is
// added atomically and the same inputs give the same bits:
//
//   dK, dV  per 128-key tile, over the 128-row tiles that see it, all query heads
//           of the key head in turn (S^T: keys in the TMEM lanes)
//             S^T = K Q^T, P^T = exp2(c S^T - L), dV += P^T dO
//             dP^T = V dO^T, dS^T = P^T o (dP^T - D), dK += dS^T Q
//   dQ      per 128-row tile of a head, over the key tiles that it sees
//             S = Q K^T, dP = dO V^T, dS = P o (dP - D), dQ += dS K
// c = scale log2(e), L = LSE log2(e) and D = rowsum(dO o O) per row, from a small
// kernel before.  P and dS are rounded to bf16 for their products only (the
// operand type), each once, from fp32: P stays in registers while dP is waited for (dS
// from P and dP - D in bf16 takes half of them and 3% less time at N=8192, and leaves
// dQ and dK off by 0.0033 of their norm instead of 0.0024).  At the 168 registers that 320
// threads leave, P in fp32 makes dK, dV spill 76 bytes of stores and 144 of loads a thread
// (d=128; dQ 4 and 4).  The two passes
// cost 7 matrix products where a fused pass has 5, but that one would add fp32 dQ
// partials of every tile through L2 in an order that varies.
//
// In S^T the row statistics belong to columns: every thread of the softmax would
// read all of them from shared memory, which the products' operands keep full
// (a 16-byte read took some 400 cycles there).  So the tensor cores add them: a
// k-step more in S and in dP, of (1, 1, 1, 0, ..) against -LSE / scale and -D split
// into three bf16 numbers each (24 bits, as fp32).
//
// Both kernels keep the tensor pipe busy by the order in which one thread issues.
// Steady state of dK, dV (a quarter of the period each):
//     dV(i)  S(i+1)  dK(i)  dP(i+1)
// P(i+1) is made from S(i+1) while dK(i), dP(i+1) run, dS(i+1) from dP(i+1) while
// dV(i+1), S(i+2) run; P overwrites S and dS overwrites dP in TMEM, so at head
// size 128 the four 128-column regions fill it exactly.  Of dQ (a third each):
//     dQ(j)  dP(j+1)  S(j+2)
// with two S regions: P(j+1) is made while dQ(j), dP(j+1) run.
//
// 320 threads: warp 0 producer, warp 1 MMA issuer (one thread) and TMEM owner,
// warps 2-9 softmax: two warps per TMEM lane quarter, each half of the columns,
// and P, dS of a half stay in its half of the region.  Persistent CTAs, one per
// SM; tiles are numbered over all of a CTA's items, so that loads run ahead
// across item borders.  All waits are bounded (tc_sync.cuh).
//
// Bound by the product stream: 3000 cycles a tile of dK, dV where its products take 2720.
// B=1, 16 / 4 heads, N=8192, window 1024, d=128: 245 us for both, statistics and sink
// sums included (660 TFLOP/s of 10 d per visible pair).
#include <cuda.h>
#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>
#include <string>
#include <type_traits>

#include "common.cuh"
#include "psa_internal.h"
#include "tc_ptx.cuh"
#include "tc_sync.cuh"
#include "tc_tmap.h"
#include "win_geom.cuh"
#include "win_internal.h"
#include "win_tc.cuh"

namespace psa {
namespace win {
namespace {

using namespace psa::tc;

__device__ int g_err = 0;

constexpr int kThreads = 320;

struct Shape {
    int B, Hq, Hkv, G, Nq, Nk, window, sinks, npad, tiles, sink_tiles, items, split;
    FarSplit far;
    FastDiv by_bk, by_hkv, by_sink, by_tiles, by_hq, by_g;
    float scale, scale_log2;
};

// Columns of a region: half w of its k-step kk (16 keys or rows, 8 columns).
__device__ __forceinline__ uint32_t half_step(int kk) { return (uint32_t)(64 * (kk >> 2) + 8 * (kk & 3)); }

// P = exp2(c s + l) of 32 columns over s, and, PUT, as bf16 pairs (l: a row's, twice; or
// nothing where s has it already).
template <bool ADD, bool PUT>
__device__ __forceinline__ void probs(uint32_t (&x)[32], uint32_t (&b)[16], uint64_t c2, uint64_t l2) {
#pragma unroll
    for (int e = 0; e < 32; e += 2) {
        const uint64_t s2 = f2_pack(__uint_as_float(x[e]), __uint_as_float(x[e + 1]));
        float y, z;
        f2_unpack(ADD ? f2_fma(s2, c2, l2) : f2_mul(s2, c2), y, z);
        y = ex2(y), z = ex2(z);
        if (PUT) b[e / 2] = pack_bf16x2(y, z);
        x[e] = __float_as_uint(y), x[e + 1] = __float_as_uint(z);
    }
}
__device__ __forceinline__ float4 ld_cluster_v4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
    return v;
}
// dS = P (dP - D) of columns 16 h .. 16 h + 15 of 32 as bf16 pairs (SUB: dp still lacks
// the row's D).
template <bool SUB>
__device__ __forceinline__ void dscore(const uint32_t (&x)[16], const uint32_t (&p)[32], uint32_t (&ds)[16], int h, uint64_t d2) {
#pragma unroll
    for (int e = 0; e < 16; e += 2) {
        uint64_t t = f2_pack(__uint_as_float(x[e]), __uint_as_float(x[e + 1]));
        if (SUB) t = f2_sub(t, d2);
        float a, b;
        f2_unpack(f2_mul(f2_pack(__uint_as_float(p[16 * h + e]), __uint_as_float(p[16 * h + e + 1])), t), a, b);
        ds[8 * h + e / 2] = pack_bf16x2(a, b);
    }
}
// Hidden columns of 16 bf16 pairs to zero.  Of a tile at the edge of the window most
// groups of 32 columns are seen by all or none of a warp's rows, and of the far rows'
// tiles a row sees all or nothing: only what is left takes the bit by bit way.
__device__ __forceinline__ void hide(uint32_t (&p)[16], uint32_t see) {
    if (__all_sync(0xffffffffu, see == 0xffffffffu)) return;
    if (__all_sync(0xffffffffu, see == 0xffffffffu || see == 0u)) {
#pragma unroll
        for (int e = 0; e < 16; ++e) p[e] &= see;
        return;
    }
#pragma unroll
    for (int e = 0; e < 16; ++e) p[e] &= ((see >> (2 * e)) & 1 ? 0xffffu : 0u) | ((see >> (2 * e + 1)) & 1 ? 0xffff0000u : 0u);
}
// A warp's 64 columns of S in TMEM to P (kept in p0, p1 and, PUT, stored over S without
// what is hidden), and of dP to dS (from p0, p1, stored at `to`).
template <bool MASK, bool ADD, bool PUT>
__device__ __forceinline__ void make_p(uint32_t tS, uint32_t (&p0)[32], uint32_t (&p1)[32], uint64_t c2, uint64_t l2,
                                       uint32_t see0, uint32_t see1) {
    tmem_ld_32x32b_x32(tS, p0);
    tmem_ld_32x32b_x32(tS + 32, p1);
    tmem_wait_ld();
    uint32_t b[16];
    probs<ADD, PUT>(p0, b, c2, l2);
    if (MASK) hide(b, see0);
    if (PUT) tmem_st_32x32b_x16(tS, b);
    probs<ADD, PUT>(p1, b, c2, l2);
    if (MASK) hide(b, see1);
    if (PUT) {
        tmem_st_32x32b_x16(tS + 16, b);
        tmem_wait_st();
    }
}
template <bool MASK, bool SUB>
__device__ __forceinline__ void make_ds(uint32_t tP, uint32_t to, const uint32_t (&p0)[32], const uint32_t (&p1)[32],
                                        uint64_t d2, uint32_t see0, uint32_t see1) {
    uint32_t x[16], y[16], ds[16];
    tmem_ld_32x32b_x16(tP, x);
    tmem_ld_32x32b_x16(tP + 16, y);
    tmem_wait_ld();
    dscore<SUB>(x, p0, ds, 0, d2);
    tmem_ld_32x32b_x16(tP + 32, x);
    dscore<SUB>(y, p0, ds, 1, d2);
    tmem_ld_32x32b_x16(tP + 48, y);
    if (MASK) hide(ds, see0);
    tmem_st_32x32b_x16(to, ds);
    tmem_wait_ld();
    dscore<SUB>(x, p1, ds, 0, d2);
    dscore<SUB>(y, p1, ds, 1, d2);
    if (MASK) hide(ds, see1);
    tmem_st_32x32b_x16(to + 16, ds);
    tmem_wait_st();
}

// ---------------------------------------------------------------- dK, dV
template <int D>
struct KCfg {
    using O = Operand<D>;
    static constexpr int TILE = O::TILE;
    static constexpr int NQ = 2, NO = 2;             // stages of Q (with its rows' statistics) and of dO
    static constexpr int OFF_K = 0, OFF_V = TILE;
    static constexpr int OFF_Q = 2 * TILE;
    static constexpr int OFF_O = OFF_Q + NQ * TILE;
    static constexpr int OFF_ST = OFF_O + NO * TILE;     // per Q stage: the statistics' operand tile
    static constexpr int OFF_ONE = OFF_ST + NQ * Operand<16>::TILE;   // what they are multiplied with: L's, D's
    static constexpr int OFF_EPI = OFF_ONE + 2 * Operand<16>::TILE;   // 1 KB per softmax warp
    static constexpr int OFF_BAR = OFF_EPI + 8 * 1024;
    static constexpr int OFF_MISC = OFF_BAR + 256;
    static constexpr int USED = OFF_MISC + 64 + 1024;
    static constexpr int SMEM = USED > 118784 ? USED : 118784;   // one CTA per SM: each takes all of TMEM
    static constexpr uint32_t C_S = 0, C_P = 128, C_K = 256, C_V = 384;
};
enum { K_KF = 0, K_KE, K_VF, K_VE, K_SF, K_DF, K_PF, K_DSF, K_ACC, K_DRAIN, K_QF, K_QE = K_QF + 4, K_OF = K_QE + 4, K_OE = K_OF + 4 };

// One item of a key head: a key tile and the row tiles that see it, or a far
// chunk of a tile with sinks (those first).
struct KItem {
    int b, hk, bk, tile, chunk;
    bool far, sink;               // sink: rows j < sinks go to the partial sums
    Seq s;
    RowRange rr;
    int rt0, nrt, n;              // first row tile, row tiles per head, this CTA's tiles
    int h, rt;                    // the head and row tile of the first of them
};
__device__ __forceinline__ KItem load_kitem(const Shape& m, const int* q_lens, const int* kv_lens, int idx, int rank) {
    KItem t;
    const int x = divide(idx, m.by_bk), nf = m.far.n_far * m.sink_tiles;
    t.bk = idx - x * (m.B * m.Hkv);
    t.b = divide(t.bk, m.by_hkv), t.hk = t.bk - t.b * m.Hkv;
    t.s = load_seq(q_lens, kv_lens, t.b, m.Nq, m.Nk);
    t.far = x < nf;
    t.chunk = t.far ? divide(x, m.by_sink) : 0;
    t.tile = t.far ? x - t.chunk * m.sink_tiles : x - nf;
    t.sink = m.far.n_far > 0 && t.tile * 128 < m.sinks;
    t.rr = t.far ? rows_of_far(t.s, t.tile * 128, 128, m.window, m.far.far_rows, t.chunk)
                 : rows_of_tile(t.s, t.tile * 128, 128, m.window, m.sinks, t.sink);
    t.rt0 = t.rr.i0 / 128;
    t.nrt = t.rr.i1 > t.rr.i0 ? (t.rr.i1 - 1) / 128 - t.rt0 + 1 : 0;
    t.n = t.nrt * m.G;
    t.h = t.hk * m.G;
    t.rt = 0;
    if (m.split > 1 && t.n > 0) { // the CTAs of a cluster take a part of the tiles each
        const int all = t.n, first = all * rank / m.split;
        t.n = all * (rank + 1) / m.split - first;
        t.h += first / t.nrt;
        t.rt = first % t.nrt;
    }
    return t;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
win_dkdv_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                const __grid_constant__ CUtensorMap tv, const __grid_constant__ CUtensorMap tdo,
                const __grid_constant__ CUtensorMap tst, RowOut dk, RowOut dv, float* __restrict__ part,
                const int* __restrict__ q_lens, const int* __restrict__ kv_lens, const __grid_constant__ Shape m) {
    using C = KCfg<D>;
    using Op = Operand<D>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sb = smem_u32(smem);
    Sync sy{sb + C::OFF_BAR, reinterpret_cast<volatile int*>(smem + C::OFF_MISC), &g_err};
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC + 16);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // split CTAs (a cluster) share an item
    const int rank = m.split > 1 ? (int)cluster_ctarank() : 0, x_first = blockIdx.x / m.split, x_step = gridDim.x / m.split;

    if (threadIdx.x == 0) {
        for (int x : {K_KF, K_KE, K_VF, K_VE, K_SF, K_DF, K_ACC, K_DRAIN}) mbar_init(sy.bar(x), 1);
        mbar_init(sy.bar(K_PF), 8);
        mbar_init(sy.bar(K_DSF), 8);
        for (int s = 0; s < C::NQ; ++s) mbar_init(sy.bar(K_QF + s), 1), mbar_init(sy.bar(K_QE + s), 1);
        for (int s = 0; s < C::NO; ++s) mbar_init(sy.bar(K_OF + s), 1), mbar_init(sy.bar(K_OE + s), 1);
        *sy.abort = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tq);
        tma_prefetch_desc(&tk);
        tma_prefetch_desc(&tv);
        tma_prefetch_desc(&tdo);
        tma_prefetch_desc(&tst);
    }
    // rows of the constant operands: 1 at features 0-2 (L) or 3-5 (D); a row's two
    // 16-byte halves change places with bit 2 of its number (32-byte swizzle)
    for (int x = threadIdx.x; x < 256; x += kThreads) {
        const int r = x & 127;
        const uint32_t at = sb + C::OFF_ONE + (x >> 7) * Operand<16>::TILE + 32 * r, one = 0x3f80u;
        const int sw = 16 * ((r >> 2) & 1);
        if (x < 128) st_shared_v4(at + sw, one | one << 16, one, 0, 0);
        else st_shared_v4(at + sw, 0, one << 16, one | one << 16, 0);
        st_shared_v4(at + 16 - sw, 0, 0, 0, 0);
    }
    fence_proxy_async_smem();
    if (warp == 1) {
        tmem_alloc(smem_u32(tmem_slot), 512);
        tmem_relinquish();
    }
    griddep_wait();                                  // the row statistics are there
    griddep_launch_dependents();                     // and the dQ kernel may start beside this one
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    if (warp == 0) {
        // ------------------------------------------------------------ producer: lane 0 K and Q, lane 1 V and dO
        if (lane < 2) {
            const CUtensorMap *big = lane ? &tv : &tk, *map = lane ? &tdo : &tq;
            const int bf = lane ? K_VF : K_KF, be = lane ? K_VE : K_KE, full = lane ? K_OF : K_QF, empty = lane ? K_OE : K_QE;
            const uint32_t big_at = sb + (lane ? C::OFF_V : C::OFF_K), base = sb + (lane ? C::OFF_O : C::OFF_Q);
            const int NST = lane ? C::NO : C::NQ;
            int it = 0, nb = 0;                      // tiles, items loaded
            bool ok = true;
            for (int x = x_first; x < m.items && ok; x += x_step) {
                const KItem t = load_kitem(m, q_lens, kv_lens, x, rank);
                if (t.n == 0) continue;
                ok = wait_one(sy, sy.bar(be), (nb & 1) ^ 1, 0, x);
                if (!ok) break;
                Op::load(big_at, big, t.tile * 128, t.hk, t.b, sy.bar(bf));
                ++nb;
                int h = t.h, rt = t.rt;
                for (int u = 0; u < t.n; ++u, ++it) {
                    const int st = it % NST;
                    ok = wait_one(sy, sy.bar(empty + st), ((it / NST) & 1) ^ 1, 1, it);
                    if (!ok) break;
                    const int i0 = (t.rt0 + rt) * 128;
                    if (lane == 0) {
                        mbar_expect_tx(sy.bar(full + st), Operand<16>::TILE);
                        tma_load_4d(sb + C::OFF_ST + st * Operand<16>::TILE, &tst, 0, i0, h, t.b, sy.bar(full + st));
                    }
                    Op::load(base + st * C::TILE, map, i0, h, t.b, sy.bar(full + st));
                    if (++rt == t.nrt) rt = 0, ++h;
                }
            }
            if (*sy.abort) {                         // wait for the copies in flight
                if (nb > 0) wait_drain(sy.bar(bf), (nb - 1) & 1);
                for (int st = 0; st < NST; ++st) {
                    const int n = (it - st + NST - 1) / NST;
                    if (n > 0) wait_drain(sy.bar(full + st), (n - 1) & 1);
                }
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer
        {
            constexpr uint32_t ID_S = idesc_bf16(128, 128, 0, 0), ID_G = idesc_bf16(128, D, 0, 1);
            const uint64_t k_desc = Op::kmajor(sb + C::OFF_K), v_desc = Op::kmajor(sb + C::OFF_V);
            const uint64_t one_l = Operand<16>::kmajor(sb + C::OFF_ONE),
                           one_d = Operand<16>::kmajor(sb + C::OFF_ONE + Operand<16>::TILE);
            int it = 0;
            uint32_t items = 0;
            bool ok = true;
            auto wait_q = [&](int u) { ok = ok && wait_warp(sy, sy.bar(K_QF + u % C::NQ), (u / C::NQ) & 1, 2, u); };
            auto wait_o = [&](int u) { ok = ok && wait_warp(sy, sy.bar(K_OF + u % C::NO), (u / C::NO) & 1, 3, u); };
            auto issue_s = [&](int u) {
                const int st = u % C::NQ;
                if (!ok) return;
                tc_fence_after();
                const uint64_t q = Op::kmajor(sb + C::OFF_Q + st * C::TILE);
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk)
                    mma_ss(tmem + C::C_S, k_desc + Op::kstep(kk), q + Op::kstep(kk), ID_S, kk);
                mma_ss(tmem + C::C_S, one_l, Operand<16>::kmajor(sb + C::OFF_ST + st * Operand<16>::TILE), ID_S, 1);
                commit(sy.bar(K_SF));
            };
            auto issue_dp = [&](int u) {
                const int st = u % C::NO;
                if (!ok) return;
                tc_fence_after();
                const uint64_t o = Op::kmajor(sb + C::OFF_O + st * C::TILE);
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk)
                    mma_ss(tmem + C::C_P, v_desc + Op::kstep(kk), o + Op::kstep(kk), ID_S, kk);
                mma_ss(tmem + C::C_P, one_d, Operand<16>::kmajor(sb + C::OFF_ST + (u % C::NQ) * Operand<16>::TILE), ID_S, 1);
                commit(sy.bar(K_DF));
            };
            for (int x = x_first; x < m.items && ok; x += x_step) {
                const KItem t = load_kitem(m, q_lens, kv_lens, x, rank);
                if (t.n == 0) continue;
                ok = wait_warp(sy, sy.bar(K_KF), items & 1, 4, x);
                wait_q(it);
                issue_s(it);
                if (ok && t.n == 1) commit(sy.bar(K_KE));
                ok = ok && wait_warp(sy, sy.bar(K_VF), items & 1, 4, x);
                wait_o(it);
                issue_dp(it);
                if (ok && t.n == 1) commit(sy.bar(K_VE));
                ++items;
                for (int u = 0; u < t.n && ok; ++u) {
                    const int i = it + u, so = i % C::NO, sq = i % C::NQ;
                    ok = wait_warp(sy, sy.bar(K_PF), i & 1, 5, i);
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t o = Op::mnmajor(sb + C::OFF_O + so * C::TILE);
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk)
                        mma_ts(tmem + C::C_V, tmem + C::C_S + half_step(kk), o + Op::MN_KSTEP * kk, ID_G,
                                    (u > 0 || kk > 0) ? 1u : 0u);
                    commit(sy.bar(K_OE + so));
                    if (u + 1 < t.n) {
                        wait_q(i + 1);
                        issue_s(i + 1);              // over P(i): the pipe keeps issue order
                        if (ok && u + 2 == t.n) commit(sy.bar(K_KE));
                    }
                    ok = ok && wait_warp(sy, sy.bar(K_DSF), i & 1, 6, i);
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t q = Op::mnmajor(sb + C::OFF_Q + sq * C::TILE);
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk)
                        mma_ts(tmem + C::C_K, tmem + C::C_P + half_step(kk), q + Op::MN_KSTEP * kk, ID_G,
                                    (u > 0 || kk > 0) ? 1u : 0u);
                    commit(sy.bar(K_QE + sq));
                    if (u + 1 < t.n) {
                        wait_o(i + 1);
                        issue_dp(i + 1);
                        if (ok && u + 2 == t.n) commit(sy.bar(K_VE));
                    }
                }
                if (ok) commit(sy.bar(K_ACC));
                it += t.n;
            }
            if (!ok) {                               // let what was issued finish before TMEM is freed
                commit(sy.bar(K_DRAIN));
                wait_drain(sy.bar(K_DRAIN), 0);
            }
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------ softmax
        const int w = (warp - 2) >> 2, q4 = warp & 3, r = q4 * 32 + lane;   // column half, key row
        const uint32_t trow = tmem + ((uint32_t)(q4 * 32) << 16);
        const uint32_t tS = trow + C::C_S + 64u * w, tP = trow + C::C_P + 64u * w;
        const uint32_t stg = sb + C::OFF_EPI + 1024u * (warp - 2);
        const uint64_t c2 = f2_pack(m.scale_log2, m.scale_log2);
        int it = 0;
        uint32_t items = 0;
        bool ok = true;
        for (int x = x_first; x < m.items && ok; x += x_step) {
            const KItem t = load_kitem(m, q_lens, kv_lens, x, rank);
            const int j0 = t.tile * 128, j = j0 + r;
            int rt = t.rt;
            for (int u = 0; u < t.n; ++u) {
                const int i = it + u, sq = i % C::NQ, so = i % C::NO;
                const int i0 = (t.rt0 + rt) * 128;
                if (++rt == t.nrt) rt = 0;
                const int pf = i0 + t.s.off;
                const bool mask = i0 < t.rr.i0 || i0 + 128 > t.rr.i1 || pf < j0 + 127 ||
                                  (pf + 127 >= j0 + m.window && j0 + 128 > m.sinks);
                ok = wait_warp(sy, sy.bar(K_SF), i & 1, 8, i);
                if (!ok) break;
                tc_fence_after();
                uint32_t p0[32], p1[32], see0 = 0, see1 = 0;
                if (mask) {
                    // rows that key j sees lie at columns lo .. hi of the tile
                    const int lo = max(j - t.s.off, t.rr.i0) - i0;
                    const int hi = (j < m.sinks ? t.rr.i1 : min(t.rr.i1, j + m.window - t.s.off)) - 1 - i0;
                    see0 = col_mask(lo, hi, -(1 << 30), 64 * w);
                    see1 = col_mask(lo, hi, -(1 << 30), 64 * w + 32);
                    make_p<true, false, true>(tS, p0, p1, c2, 0, see0, see1);
                } else {
                    make_p<false, false, true>(tS, p0, p1, c2, 0, 0, 0);
                }
                // Rows behind the sequence's end hold anything in Q and dO: P, dS are 0
                // there, but 0 times NaN is not, so their rows are cleared before the
                // products that sum over rows (half 0 clears dO, half 1 clears Q).
                const bool tail = i0 + 128 > t.s.ql && t.s.ql < m.Nq;
                if (tail) {
                    ok = wait_warp(sy, sy.bar(K_OF + so), (i / C::NO) & 1, 9, i);
                    if (!ok) break;
                    if (i0 + r >= t.s.ql) Op::clear_row(sb + (w ? C::OFF_Q + sq * C::TILE : C::OFF_O + so * C::TILE), r);
                    fence_proxy_async_smem();
                }
                tc_fence_before();
                warp_arrive(sy.bar(K_PF), lane);
                ok = wait_warp(sy, sy.bar(K_DF), i & 1, 10, i);
                if (!ok) break;
                tc_fence_after();
                if (mask) make_ds<true, false>(tP, tP, p0, p1, 0, see0, see1);
                else make_ds<false, false>(tP, tP, p0, p1, 0, 0, 0);
                tc_fence_before();
                warp_arrive(sy.bar(K_DSF), lane);
            }
            if (!ok) break;
            it += t.n;
            if (t.n > 0) {
                ok = wait_warp(sy, sy.bar(K_ACC), items++ & 1, 12, it);
                if (!ok) break;
                tc_fence_after();
            }
            if (m.split > 1) {                       // to shared memory, to be joined below
                const uint32_t to = sb + 16u * (w * (D / 4) * 128 + r), tA = trow + (w ? C::C_V : C::C_K);
#pragma unroll
                for (int h = 0; h < D; h += 16) {
                    uint32_t v[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) v[e] = 0;
                    if (t.n > 0) {
                        tmem_ld_32x32b_x16(tA + h, v);
                        tmem_wait_ld();
                    }
#pragma unroll
                    for (int e = 0; e < 16; e += 4)
                        st_shared_v4(to + 2048u * ((h + e) / 4), v[e], v[e + 1], v[e + 2], v[e + 3]);
                }
                break;                               // a cluster has one item
            }
            // warps of half 0 write dK, of half 1 dV
            const bool some = t.n > 0 && j < t.s.kl;
            const float mul = w ? 1.f : m.scale;
            const uint32_t tA = trow + (w ? C::C_V : C::C_K);
            const int r0 = j0 + q4 * 32;
            uint16_t* row0 = (w ? dv : dk).row(t.b, t.hk, r0);
            float* prow = part + (((size_t)t.bk * (1 + m.far.n_far) + (t.far ? 1 + t.chunk : 0)) * 2 + w) * m.sinks * D +
                          (size_t)j * D;
            constexpr int W = D < 32 ? D : 32;
#pragma unroll
            for (int h = 0; h < D; h += W) {
                uint32_t v[W], o[W / 2];
                if (t.n > 0) {
                    tmem_ld_row<W>(tA + h, v);
                    tmem_wait_ld();
                }
                if (t.sink && j < m.sinks) {         // unscaled, summed and scaled afterwards
#pragma unroll
                    for (int e = 0; e < W; e += 4)
                        *reinterpret_cast<float4*>(prow + h + e) =
                            some ? make_float4(__uint_as_float(v[e]), __uint_as_float(v[e + 1]), __uint_as_float(v[e + 2]),
                                               __uint_as_float(v[e + 3]))
                                 : make_float4(0.f, 0.f, 0.f, 0.f);
                }
                if (!t.far) {
#pragma unroll
                    for (int e = 0; e < W / 2; ++e)
                        o[e] = some ? pack_bf16x2(__uint_as_float(v[2 * e]) * mul, __uint_as_float(v[2 * e + 1]) * mul) : 0u;
                    store_rows<W>(stg, o, row0 + h, (w ? dv : dk).sN, m.Nk - r0, lane);
                }
            }
            tc_fence_before();                       // read before the next item's first products
        }
    }

    if (m.split > 1) {
        // Join: 8 features of a row per thread, the CTAs' sums in rank order.  Nothing is
        // in flight into the tiles any more (every copy was used, every product is done).
        __syncwarp();
        cluster_sync_all();
        const KItem t = load_kitem(m, q_lens, kv_lens, x_first, rank);
        const int j0 = t.tile * 128, per = 32 * D / m.split;
        for (int i = rank * per + threadIdx.x; i < (rank + 1) * per; i += kThreads) {
            const int r = i & 127, c = i >> 7, is_v = c / (D / 8), f = c % (D / 8), j = j0 + r;
            if (j >= m.Nk) continue;
            float a[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
            if (j < t.s.kl)
                for (int q = 0; q < m.split; ++q) {
                    const uint32_t from = mapa_shared(sb + 16u * ((is_v * (D / 4) + 2 * f) * 128 + r), q);
                    const float4 x = ld_cluster_v4(from), y = ld_cluster_v4(from + 2048);
                    a[0] += x.x, a[1] += x.y, a[2] += x.z, a[3] += x.w;
                    a[4] += y.x, a[5] += y.y, a[6] += y.z, a[7] += y.w;
                }
            if (t.sink && j < m.sinks) {             // unscaled, summed and scaled afterwards
                float4* p = reinterpret_cast<float4*>(
                    part + ((((size_t)t.bk * (1 + m.far.n_far) + (t.far ? 1 + t.chunk : 0)) * 2 + is_v) * m.sinks + j) * D + 8 * f);
                p[0] = make_float4(a[0], a[1], a[2], a[3]);
                p[1] = make_float4(a[4], a[5], a[6], a[7]);
            } else if (!t.far) {
                const float mul = is_v ? 1.f : m.scale;
                *reinterpret_cast<uint4*>((is_v ? dv : dk).row(t.b, t.hk, j) + 8 * f) =
                    make_uint4(pack_bf16x2(a[0] * mul, a[1] * mul), pack_bf16x2(a[2] * mul, a[3] * mul),
                               pack_bf16x2(a[4] * mul, a[5] * mul), pack_bf16x2(a[6] * mul, a[7] * mul));
            }
        }
        __syncwarp();
        cluster_sync_all();                          // no CTA leaves while its sums are read
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, 512);
}

// ---------------------------------------------------------------- dQ
template <int D>
struct QCfg {
    using O = Operand<D>;
    static constexpr int TILE = O::TILE;
    // S(j+2) is issued right behind dQ(j): three K stages; V serves dP alone
    static constexpr int NK = 3, NV = 2;
    static constexpr int OFF_Q = 0, OFF_DO = TILE;
    static constexpr int OFF_K = 2 * TILE;
    static constexpr int OFF_V = OFF_K + NK * TILE;
    static constexpr int OFF_BAR = OFF_V + NV * TILE;
    static constexpr int OFF_MISC = OFF_BAR + 256;
    static constexpr int USED = OFF_MISC + 64 + 1024;
    static constexpr int SMEM = USED > 118784 ? USED : 118784;
    static constexpr uint32_t C_S = 0, C_P = 256, C_Q = 384;   // S(j) at 128 (j & 1)
};
enum { Q_QF = 0, Q_QE, Q_OF, Q_OE, Q_DF, Q_DSF, Q_ACC, Q_DRAIN, Q_SF, Q_KF = Q_SF + 2, Q_KE = Q_KF + 4, Q_VF = Q_KE + 4, Q_VE = Q_VF + 4 };

struct QItem {
    int b, h, hk, i0, i1;
    Seq s;
    KeyTiles kt;
    int n;
};
__device__ __forceinline__ QItem load_qitem(const Shape& m, const int* q_lens, const int* kv_lens, int idx) {
    QItem t;
    const int bh = divide(idx, m.by_tiles);
    t.b = divide(bh, m.by_hq), t.h = bh - t.b * m.Hq, t.hk = divide(t.h, m.by_g);
    t.i0 = (m.tiles - 1 - (idx - bh * m.tiles)) * 128;   // long rows first
    t.s = load_seq(q_lens, kv_lens, t.b, m.Nq, m.Nk);
    t.i1 = min(t.i0 + 128, t.s.ql);
    t.kt = key_tiles<128>(t.s, t.i0, t.i1, m.window, m.sinks);
    t.n = t.kt.count();
    return t;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
win_dq_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
              const __grid_constant__ CUtensorMap tv, const __grid_constant__ CUtensorMap tdo, RowOut dq,
              const float* __restrict__ negl, const float* __restrict__ drow, const int* __restrict__ q_lens,
              const int* __restrict__ kv_lens, const __grid_constant__ Shape m) {
    using C = QCfg<D>;
    using Op = Operand<D>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sb = smem_u32(smem);
    Sync sy{sb + C::OFF_BAR, reinterpret_cast<volatile int*>(smem + C::OFF_MISC), &g_err};
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC + 16);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int x = Q_QF; x < Q_KF; ++x) mbar_init(sy.bar(x), x == Q_DSF ? 8 : 1);
        for (int s = 0; s < C::NK; ++s) mbar_init(sy.bar(Q_KF + s), 1), mbar_init(sy.bar(Q_KE + s), 1);
        for (int s = 0; s < C::NV; ++s) mbar_init(sy.bar(Q_VF + s), 1), mbar_init(sy.bar(Q_VE + s), 1);
        *sy.abort = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tq);
        tma_prefetch_desc(&tk);
        tma_prefetch_desc(&tv);
        tma_prefetch_desc(&tdo);
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(tmem_slot), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    if (warp == 0) {
        // ------------------------------------------------------------ producer: lane 0 Q and K, lane 1 dO and V
        if (lane < 2) {
            const CUtensorMap *big = lane ? &tdo : &tq, *map = lane ? &tv : &tk;
            const int bf = lane ? Q_OF : Q_QF, be = lane ? Q_OE : Q_QE, full = lane ? Q_VF : Q_KF, empty = lane ? Q_VE : Q_KE;
            const uint32_t big_at = sb + (lane ? C::OFF_DO : C::OFF_Q), base = sb + (lane ? C::OFF_V : C::OFF_K);
            const int NST = lane ? C::NV : C::NK;
            int it = 0, nb = 0;
            bool ok = true;
            for (int x = blockIdx.x; x < m.items && ok; x += gridDim.x) {
                const QItem t = load_qitem(m, q_lens, kv_lens, x);
                if (t.n == 0) continue;
                ok = wait_one(sy, sy.bar(be), (nb & 1) ^ 1, 0, x);
                if (!ok) break;
                Op::load(big_at, big, t.i0, t.h, t.b, sy.bar(bf));
                ++nb;
                for (int u = 0; u < t.n; ++u, ++it) {
                    const int st = it % NST;
                    ok = wait_one(sy, sy.bar(empty + st), ((it / NST) & 1) ^ 1, 1, it);
                    if (!ok) break;
                    Op::load(base + st * C::TILE, map, t.kt.tile(u) * 128, t.hk, t.b, sy.bar(full + st));
                }
            }
            if (*sy.abort) {
                if (nb > 0) wait_drain(sy.bar(bf), (nb - 1) & 1);
                for (int st = 0; st < NST; ++st) {
                    const int n = (it - st + NST - 1) / NST;
                    if (n > 0) wait_drain(sy.bar(full + st), (n - 1) & 1);
                }
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer
        {
            constexpr uint32_t ID_S = idesc_bf16(128, 128, 0, 0), ID_G = idesc_bf16(128, D, 0, 1);
            const uint64_t q_desc = Op::kmajor(sb + C::OFF_Q), o_desc = Op::kmajor(sb + C::OFF_DO);
            int it = 0;
            uint32_t items = 0;
            bool ok = true;
            auto wait_k = [&](int j) { ok = ok && wait_warp(sy, sy.bar(Q_KF + j % C::NK), (j / C::NK) & 1, 2, j); };
            auto wait_v = [&](int j) { ok = ok && wait_warp(sy, sy.bar(Q_VF + j % C::NV), (j / C::NV) & 1, 3, j); };
            auto issue_s = [&](int j, bool last) {
                const int st = j % C::NK;
                if (!ok) return;
                tc_fence_after();
                const uint64_t k = Op::kmajor(sb + C::OFF_K + st * C::TILE);
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk)
                    mma_ss(tmem + C::C_S + 128u * (j & 1), q_desc + Op::kstep(kk), k + Op::kstep(kk), ID_S, kk);
                commit(sy.bar(Q_SF + (j & 1)));
                if (last) commit(sy.bar(Q_QE));
            };
            auto issue_dp = [&](int j, bool last) {
                const int st = j % C::NV;
                if (!ok) return;
                tc_fence_after();
                const uint64_t v = Op::kmajor(sb + C::OFF_V + st * C::TILE);
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk)
                    mma_ss(tmem + C::C_P, o_desc + Op::kstep(kk), v + Op::kstep(kk), ID_S, kk);
                commit(sy.bar(Q_DF));
                commit(sy.bar(Q_VE + st));
                if (last) commit(sy.bar(Q_OE));
            };
            for (int x = blockIdx.x; x < m.items && ok; x += gridDim.x) {
                const QItem t = load_qitem(m, q_lens, kv_lens, x);
                if (t.n == 0) continue;
                ok = wait_warp(sy, sy.bar(Q_QF), items & 1, 4, x);
                wait_k(it);
                issue_s(it, t.n == 1);
                ok = ok && wait_warp(sy, sy.bar(Q_OF), items & 1, 4, x);
                wait_v(it);
                issue_dp(it, t.n == 1);
                if (t.n > 1) {
                    wait_k(it + 1);
                    issue_s(it + 1, t.n == 2);
                }
                ++items;
                for (int u = 0; u < t.n && ok; ++u) {
                    const int j = it + u;
                    ok = wait_warp(sy, sy.bar(Q_DSF), j & 1, 5, j);
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t k = Op::mnmajor(sb + C::OFF_K + (j % C::NK) * C::TILE);
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk)
                        mma_ts(tmem + C::C_Q, tmem + C::C_S + 128u * (j & 1) + half_step(kk), k + Op::MN_KSTEP * kk, ID_G,
                                    (u > 0 || kk > 0) ? 1u : 0u);
                    commit(sy.bar(Q_KE + j % C::NK));
                    if (u + 1 == t.n) commit(sy.bar(Q_ACC));
                    if (u + 1 < t.n) {
                        wait_v(j + 1);
                        issue_dp(j + 1, u + 2 == t.n);
                    }
                    if (u + 2 < t.n) {
                        wait_k(j + 2);
                        issue_s(j + 2, u + 3 == t.n);   // over dS(j): the pipe keeps issue order
                    }
                }
                it += t.n;
            }
            if (!ok) {
                commit(sy.bar(Q_DRAIN));
                wait_drain(sy.bar(Q_DRAIN), 0);
            }
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------ softmax
        const int w = (warp - 2) >> 2, q4 = warp & 3, r = q4 * 32 + lane;   // column half, row
        const uint32_t trow = tmem + ((uint32_t)(q4 * 32) << 16);
        const uint64_t c2 = f2_pack(m.scale_log2, m.scale_log2);
        int it = 0;
        uint32_t items = 0;
        bool ok = true;
        for (int x = blockIdx.x; x < m.items && ok; x += gridDim.x) {
            const QItem t = load_qitem(m, q_lens, kv_lens, x);
            const int i = t.i0 + r, p0 = i < t.s.ql ? i + t.s.off : -1;
            const size_t row = ((size_t)t.b * m.Hq + t.h) * m.npad + i;   // the arrays are padded to whole tiles
            const float L = __ldcg(negl + row), Dr = __ldcg(drow + row);
            const uint64_t l2 = f2_pack(L, L), d2 = f2_pack(Dr, Dr);
            const int pf = t.i0 + t.s.off, pl = t.i1 - 1 + t.s.off;
            for (int u = 0; u < t.n; ++u) {
                const int j = it + u, j0 = t.kt.tile(u) * 128;
                const uint32_t tS = trow + C::C_S + 128u * (j & 1) + 64u * w, tP = trow + C::C_P + 64u * w;
                const int lo = p0 - m.window + 1 - j0, hi = p0 - j0, snk = m.sinks - j0;
                const bool mask = !(j0 + 127 <= pf && j0 > pl - m.window) || t.i1 < t.i0 + 128;
                ok = wait_warp(sy, sy.bar(Q_SF + (j & 1)), (j >> 1) & 1, 6, j);
                if (!ok) break;
                tc_fence_after();
                uint32_t p0[32], p1[32];
                make_p<false, true, false>(tS, p0, p1, c2, l2, 0, 0);   // masked with dS
                ok = wait_warp(sy, sy.bar(Q_DF), j & 1, 7, j);
                if (!ok) break;
                tc_fence_after();
                if (mask)
                    make_ds<true, true>(tP, tS, p0, p1, d2, col_mask(lo, hi, snk, 64 * w), col_mask(lo, hi, snk, 64 * w + 32));
                else
                    make_ds<false, true>(tP, tS, p0, p1, d2, 0, 0);
                // K rows behind the sequence's end hold anything: dS is 0 there, 0 times NaN is not
                if (j0 + 128 > t.s.kl && t.s.kl < m.Nk) {
                    ok = wait_warp(sy, sy.bar(Q_KF + j % C::NK), (j / C::NK) & 1, 8, j);
                    if (!ok) break;
                    if (w == 0 && j0 + r >= t.s.kl) Op::clear_row(sb + C::OFF_K + (j % C::NK) * C::TILE, r);
                    fence_proxy_async_smem();
                }
                tc_fence_before();
                warp_arrive(sy.bar(Q_DSF), lane);
            }
            if (!ok) break;
            it += t.n;
            if (t.n > 0) {
                ok = wait_warp(sy, sy.bar(Q_ACC), items++ & 1, 9, it);
                if (!ok) break;
                tc_fence_after();
            }
            const bool some = t.n > 0 && i < t.s.ql;
            uint16_t* out = dq.row(t.b, t.h, i);
            constexpr int W = D < 32 ? D : 32;
            // each half writes every other group of 32 features (head size 16 and 32: half 0 alone)
#pragma unroll
            for (int h = 0; h < D; h += W) {
                if ((h / W) % 2 != w) continue;
                uint32_t v[W];
                if (t.n > 0) {
                    tmem_ld_row<W>(trow + C::C_Q + h, v);
                    tmem_wait_ld();
                }
                if (i < m.Nq)
#pragma unroll
                    for (int e = 0; e < W; e += 8) {
                        uint4 o = make_uint4(0, 0, 0, 0);
                        if (some) {
                            o.x = pack_bf16x2(__uint_as_float(v[e]) * m.scale, __uint_as_float(v[e + 1]) * m.scale);
                            o.y = pack_bf16x2(__uint_as_float(v[e + 2]) * m.scale, __uint_as_float(v[e + 3]) * m.scale);
                            o.z = pack_bf16x2(__uint_as_float(v[e + 4]) * m.scale, __uint_as_float(v[e + 5]) * m.scale);
                            o.w = pack_bf16x2(__uint_as_float(v[e + 6]) * m.scale, __uint_as_float(v[e + 7]) * m.scale);
                        }
                        *reinterpret_cast<uint4*>(out + h + e) = o;
                    }
            }
            tc_fence_before();
        }
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, 512);
    griddep_wait();                                  // done only when the kernel before is
}

// CTAs per dK, dV item: a cluster of 2, 4 or 8 shares the tiles of an item where all
// items together would leave half of the SMs idle, down to two tiles each (a tile takes
// about 1.5 us, joining a cluster 2 us: a batch of 8 sequences of 400 tokens, 64 items on 152
// SMs: the whole backward 33.5 us with 1 and 27.3 us with 2).
int split_of(const Shape& m, long long items, int sms) {
    const int nqt = (m.Nq + 127) / 128;
    const bool whole = m.sinks > 0 && m.far.n_far == 0;   // a tile that all later rows see
    const long long tiles = (long long)m.G * (whole ? nqt : std::min(nqt, (m.window + 127) / 128 + 1));
    int s = 1;
    while (s < 8 && items * s * 2 <= sms && tiles >= 4 * s) s *= 2;
    return s;
}

template <int D>
int launch(const Args& a, std::string* err) {
    using Op = Operand<D>;
    const FarSplit f = far_split(a.Nk, a.window, a.sinks);
    Shape m{a.B, a.Hq, a.Hkv, a.Hq / a.Hkv, a.Nq, a.Nk, a.window, a.sinks, stat_rows(a.Nq), (a.Nk + 127) / 128,
            f.n_far ? (a.sinks + 127) / 128 : 0, 0, 1, f, {}, {}, {}, {}, {}, {}, a.scale, a.scale * kLog2e};
    const long long ki = (long long)a.B * a.Hkv * (m.tiles + f.n_far * m.sink_tiles);
    const long long qi = (long long)a.B * a.Hq * ((a.Nq + 127) / 128);
    if (ki > 0x3fffffffll || qi > 0x3fffffffll) {
        *err = "grid too large";
        return PSA_ERR_UNSUPPORTED;
    }
    m.by_bk = fast_div(m.B * m.Hkv), m.by_hkv = fast_div(m.Hkv), m.by_sink = fast_div(m.sink_tiles ? m.sink_tiles : 1);
    m.by_hq = fast_div(m.Hq), m.by_g = fast_div(m.G);
    CUtensorMap tq, tk, tv, tdo, tst;
    int sms = 0;
    const long long np = stat_rows(a.Nq);
    if (!Op::encode(&tq, a.q, a.B, a.Hq, a.Nq, 128, err) || !Op::encode(&tk, a.k, a.B, a.Hkv, a.Nk, 128, err) ||
        !Op::encode(&tv, a.v, a.B, a.Hkv, a.Nk, 128, err) || !Op::encode(&tdo, a.dO, a.B, a.Hq, a.Nq, 128, err) ||
        // 8 numbers per row; features 8-15 of the operand are past the extent and read as zero
        !encode_bf16_4d(&tst, a.aug, 8, np, a.Hq, a.B, 8, np * 8, a.Hq * np * 8, 16, 128, err) ||
        !set_max_dynamic_smem((const void*)win_dkdv_kernel<D>, KCfg<D>::SMEM, err) ||
        !set_max_dynamic_smem((const void*)win_dq_kernel<D>, QCfg<D>::SMEM, err) || !sm_count(&sms, err))
        return PSA_ERR_CUDA;
    const int rc = pre_d(a, err);
    if (rc) return rc;
    // dQ does not need dK, dV: its kernel starts once the statistics are there and takes
    // the SMs that the dK, dV kernel leaves or does not fill, but ends after it (so does
    // what follows).  It must not read what the kernel before the statistics may have left
    // in an SM's L1: they are read past it.
    cudaError_t e;
    {
        m.items = (int)ki;
        m.split = split_of(m, ki, sms);
        ProfScope prof(kSlotMain, a.stream);
        e = launch_beside(win_dkdv_kernel<D>, (unsigned)(ki < sms ? ki * m.split : sms), kThreads, m.split, KCfg<D>::SMEM, a.stream, tq, tk, tv, tdo, tst,
                          row_out(a.dk), row_out(a.dv), a.part, a.q_lens, a.kv_lens, m);
    }
    if (e == cudaSuccess) {
        m.items = (int)qi;
        m.tiles = (a.Nq + 127) / 128;
        m.by_tiles = fast_div(m.tiles);
        ProfScope prof(kSlotDq, a.stream);
        e = launch_beside(win_dq_kernel<D>, (unsigned)(qi < sms ? qi : sms), kThreads, 1, QCfg<D>::SMEM, a.stream, tq, tk, tv, tdo,
                          row_out(a.dq), a.negl, a.Drow, a.q_lens, a.kv_lens, m);
    }
    if (e != cudaSuccess) {
        *err = std::string("window attention backward launch: ") + cudaGetErrorString(e);
        return PSA_ERR_CUDA;
    }
    return f.n_far ? sum_far(a, f, err) : PSA_OK;
}

}  // namespace

int tc_bwd(const Args& a, std::string* err) {
    switch (a.d) {
        case 16: return launch<16>(a, err);
        case 32: return launch<32>(a, err);
        case 64: return launch<64>(a, err);
        default: return launch<128>(a, err);
    }
}

int tc_bwd_take_error(std::string* err) { return take_error(g_err, "window attention backward", err); }

}  // namespace win
}  // namespace psa
