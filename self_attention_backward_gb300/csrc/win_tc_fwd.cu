// win_tc_fwd.cu -- sliding-window attention with sinks, forward, on the tensor
// cores (tcgen05 / TMEM / TMA), bf16 storage.
//
// Per 128-row tile of a head, over the 128-key tiles it sees (win_geom.cuh),
// with an online softmax in log2 units, c = scale log2(e):
//   S = Q K_j^T;  m' = max(m, max S c) if that exceeds m by more than 8, else m
//   P = exp2(S c - m) (bf16, over S in TMEM),  l += sum P,  O += P V_j
// (a stale maximum keeps P <= 2^8; when it moves, l and O are scaled), and at the
// end O / l and LSE = (m + log2 l) ln 2.  P is rounded to bf16 for its product
// (the sum l is not), which is the operand type of the tensor cores: an error of
// at most 2^-8 of each term.
//
// A persistent CTA per SM runs two such tiles ("slots") at once against the same
// K and V tiles: two query heads that share a key head, else neighbouring row
// tiles.  The tensor cores work on one slot while the other slot's softmax
// runs, and a K or V tile is fetched once for 256 rows.  Tiles are numbered over
// all of a CTA's items, so that loads run ahead across item borders.
//
// 320 threads: warp 0 producer (lane 0 K, lane 1 V, lane 2 Q), warp 1 MMA issuer
// (one thread) and TMEM owner, warps 2-5 and 6-9 the softmax of the two slots (a
// row per thread, the warp's TMEM lane quarter).  The softmax reads S twice, for
// the maximum and for P, 32 columns at a time with the next ones on their way:
// keeping a row's 128 scores in registers takes over 220 of them, and TMEM reads
// are cheap.
// Issue order per tile and slot: P V of tile j, then S of tile j+1 over P's
// columns (the pipe keeps issue order), so "S ready" also says that P V has been
// added: a rescale needs no other wait.
// A tile of which at most 32 columns can be seen (sinks, a sequence's end) takes a
// quarter of the work.  All waits are bounded (tc_sync.cuh).
//
// Bound by the products and the shared memory that they and the loads share (2048 cycles
// each per tile of both slots, which takes some 3000 with the issuer's waits, 200 cycles
// each after its products have ended).  B=1, 16 / 4 heads, N=16384, window 1024, d=128: 132 us,
// 1.0 PFLOP/s.  Slower there: 16 softmax warps (144 us), the issuer's waits and commits
// given to other warps (132 to 142), CTA pairs (170: the tiles' signals between the CTAs
// take longer than two tiles cover).
#include <cuda.h>
#include <cuda_bf16.h>

#include <cmath>
#include <string>

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
using bf16 = __nv_bfloat16;

__device__ int g_err = 0;

constexpr int kThreads = 320;
constexpr float kMove = 8.f;      // keep a stale row maximum while the new one is at most 2^8 larger

template <int D>
struct Cfg {
    using O = Operand<D>;
    static constexpr int TILE = O::TILE;             // one [128, D] tile
    static constexpr int NST = D == 128 ? 2 : 4;     // K stages, V stages
    static constexpr int OFF_Q = 0;                  // two slots
    static constexpr int OFF_K = 2 * TILE;
    static constexpr int OFF_V = OFF_K + NST * TILE;
    static constexpr int OFF_EPI = OFF_V + NST * TILE;   // 2 KB per softmax warp
    static constexpr int OFF_BAR = OFF_EPI + 8 * 2048;
    static constexpr int OFF_MISC = OFF_BAR + 256;
    static constexpr int USED = OFF_MISC + 64 + 1024;
    static constexpr int SMEM = USED > 118784 ? USED : 118784;   // one CTA per SM: each takes all of TMEM
    static constexpr uint32_t C_S = 0, C_O = 256;    // S of slot s at 128 s, O at 256 + 128 s
};

// barriers (slot s or stage s behind each)
enum { W_QF = 0, W_QE = 2, W_SF = 4, W_PF = 6, W_OF = 8, W_KF = 10, W_KE = 14, W_VF = 18, W_VE = 22, W_DRAIN = 26 };

struct Shape {
    int B, Hq, Hkv, G, Nq, Nk, window, sinks, nqt, pairs, items;
    FastDiv by_pairs, by_hkv, by_g;
    float scale_log2;
};

// One item: two slots of a key head, and the key tiles that they see together.
struct Slot {
    int i0, h;
    bool exists, active;          // active: some of its rows see something
};
struct Item {
    int b, hk;
    Seq s;
    KeyTiles kt;
    int n, p1;                    // tiles; last position of the item
    Slot s0, s1;
    __device__ __forceinline__ Slot slot(int i) const { return i ? s1 : s0; }
};
__device__ __forceinline__ Item load_item(const Shape& m, const int* q_lens, const int* kv_lens, int idx) {
    Item t;
    const int bk = divide(idx, m.by_pairs), x = m.pairs - 1 - (idx - bk * m.pairs);   // long rows first
    t.b = divide(bk, m.by_hkv), t.hk = bk - t.b * m.Hkv;
    t.s = load_seq(q_lens, kv_lens, t.b, m.Nq, m.Nk);
    int first = 0, last = 0;
    bool any = false;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        const int q = 2 * x + s;
        Slot c;
        c.exists = q < m.G * m.nqt;
        const int tile = divide(q, m.by_g);
        c.i0 = tile * 128;
        c.h = t.hk * m.G + q - tile * m.G;
        const int i1 = min(c.i0 + 128, t.s.ql);
        c.active = c.exists && i1 > c.i0 && i1 - 1 + t.s.off >= 0;
        if (c.active) {
            if (!any) first = c.i0;
            last = i1;
            any = true;
        }
        (s ? t.s1 : t.s0) = c;
    }
    t.kt = key_tiles<128>(t.s, first, last, m.window, m.sinks);
    t.n = t.kt.count();
    t.p1 = last - 1 + t.s.off;
    return t;
}
// 32-column groups of tile t that can be seen: 1 or (treated as) 4.
__device__ __forceinline__ int tile_groups(const Item& it, const Shape& m, int t) {
    const int j0 = it.kt.tile(t) * 128;
    const int need = t < it.kt.n_sink ? m.sinks - j0 : it.p1 + 1 - j0;
    return need <= 32 ? 1 : 4;
}

// Hidden columns of a 32-column group to -inf.
__device__ __forceinline__ void hide(uint32_t (&x)[32], uint32_t see) {
#pragma unroll
    for (int e = 0; e < 32; ++e)
        if (!(see >> e & 1)) x[e] = 0xff800000u;
}
__device__ __forceinline__ void max_group(const uint32_t (&x)[32], float& ma, float& mb) {
#pragma unroll
    for (int e = 0; e < 32; e += 4) {
        ma = fmax3(ma, __uint_as_float(x[e]), __uint_as_float(x[e + 1]));
        mb = fmax3(mb, __uint_as_float(x[e + 2]), __uint_as_float(x[e + 3]));
    }
}
// P of a 32-column group as bf16 pairs to TMEM; its sums to la, lb.
__device__ __forceinline__ void prob_group(const uint32_t (&x)[32], uint64_t c2, uint64_t r2, uint64_t& la, uint64_t& lb,
                                           uint32_t to) {
    const uint64_t one2 = f2_pack(1.f, 1.f);
    uint32_t pk[16];
#pragma unroll
    for (int e = 0; e < 32; e += 4) {
        float p0, p1, p2, p3;
        f2_unpack(f2_fma(f2_pack(__uint_as_float(x[e]), __uint_as_float(x[e + 1])), c2, r2), p0, p1);
        f2_unpack(f2_fma(f2_pack(__uint_as_float(x[e + 2]), __uint_as_float(x[e + 3])), c2, r2), p2, p3);
        p0 = ex2(p0);
        p1 = ex2(p1);
        p2 = ex2(p2);
        p3 = ex2(p3);
        la = f2_fma(f2_pack(p0, p1), one2, la);
        lb = f2_fma(f2_pack(p2, p3), one2, lb);
        pk[e / 2] = pack_bf16x2(p0, p1);
        pk[e / 2 + 1] = pack_bf16x2(p2, p3);
    }
    tmem_st_32x32b_x16(to, pk);
}

// The row's maximum after a tile whose scores reach mt (log2 units): l, and O when a
// maximum of the warp's rows moves, are scaled; returns -m for the exponentials.
template <int D>
__device__ __forceinline__ float move_max(uint32_t tO, bool first, float mt, float& m, float& l) {
    const bool move = mt > m + kMove;                // m = -inf: any finite score moves it
    const float alpha = move ? ex2(m - mt) : 1.f;
    if (move) m = mt;
    l *= alpha;
    if (!first && __any_sync(0xffffffffu, move)) {
        tmem_wait_ld();
#pragma unroll 1
        for (int h = 0; h < D; h += 16) {            // O *= alpha (every lane takes part)
            uint32_t o[16];
            tmem_ld_32x32b_x16(tO + h, o);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
            tmem_st_32x32b_x16(tO + h, o);
        }
    }
    return m == -INFINITY ? 0.f : -m;
}
__device__ __forceinline__ float pair_sum(uint64_t la, uint64_t lb) {
    float a0, a1, b0, b1;
    f2_unpack(la, a0, a1);
    f2_unpack(lb, b0, b1);
    return (a0 + a1) + (b0 + b1);
}

// One tile that every row of the warp sees in full: m and l of this thread's row, P
// over S.  32 columns are worked on while the next ones are on their way.
template <int D>
__device__ __forceinline__ void softmax_tile(uint32_t tS, uint32_t tO, bool first, float c, float& m, float& l) {
    uint32_t xa[32], xb[32];
    float ma = -INFINITY, mb = -INFINITY;
    tmem_ld_32x32b_x32(tS, xa);
#pragma unroll
    for (int g = 0; g < 4; ++g) {                    // even groups in xa, odd ones in xb
        tmem_wait_ld();
        tmem_ld_32x32b_x32(tS + 32 * ((g + 1) & 3), g % 2 ? xa : xb);
        max_group(g % 2 ? xb : xa, ma, mb);
    }
    const float nm = move_max<D>(tO, first, fmaxf(ma, mb) * c, m, l);   // c > 0
    const uint64_t c2 = f2_pack(c, c), r2 = f2_pack(nm, nm);
    uint64_t la = f2_pack(0.f, 0.f), lb = la;
#pragma unroll
    for (int g = 0; g < 4; ++g) {
        tmem_wait_ld();
        if (g < 3) tmem_ld_32x32b_x32(tS + 32 * (g + 1), g % 2 ? xa : xb);
        prob_group(g % 2 ? xb : xa, c2, r2, la, lb, tS + 16 * g);
    }
    l += pair_sum(la, lb);
    tmem_wait_st();
}
// The same for a tile of nc 32-column groups with hidden columns.  Most groups of
// such a tile are seen by all of a warp's rows, or by none: those are left out (P = 0),
// and a group in between is masked once and put back.  A loop over the groups: written
// out, its code, read once per item, took longer to come than to run.
template <int D>
__device__ __forceinline__ void softmax_edge(uint32_t tS, uint32_t tO, bool first, float c, float& m, float& l, int nc, int lo,
                                             int hi, int snk) {
    uint32_t x[32];
    float ma = -INFINITY, mb = -INFINITY;
    uint32_t some = 0;                               // groups that a row of the warp sees
#pragma unroll 1
    for (int g = 0; g < nc; ++g) {
        const uint32_t see = col_mask(lo, hi, snk, 32 * g);
        if (!__any_sync(0xffffffffu, see != 0u)) continue;
        some |= 1u << g;
        tmem_ld_32x32b_x32(tS + 32 * g, x);
        tmem_wait_ld();
        if (!__all_sync(0xffffffffu, see == 0xffffffffu)) {
            hide(x, see);
            tmem_st_32x32b_x16(tS + 32 * g, x);
            tmem_st_32x32b_x16(tS + 32 * g + 16, x + 16);
        }
        max_group(x, ma, mb);
    }
    tmem_wait_st();
    const float nm = move_max<D>(tO, first, fmaxf(ma, mb) * c, m, l);
    const uint64_t c2 = f2_pack(c, c), r2 = f2_pack(nm, nm);
    uint64_t la = f2_pack(0.f, 0.f), lb = la;
#pragma unroll 1
    for (int g = 0; g < nc; ++g) {
        if (some >> g & 1) {
            tmem_ld_32x32b_x32(tS + 32 * g, x);
            tmem_wait_ld();
            prob_group(x, c2, r2, la, lb, tS + 16 * g);
        } else {
#pragma unroll
            for (int e = 0; e < 16; ++e) x[e] = 0;
            tmem_st_32x32b_x16(tS + 16 * g, x);
        }
    }
    l += pair_sum(la, lb);
    tmem_wait_st();
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
win_fwd_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
               const __grid_constant__ CUtensorMap tv, RowOut o, float* __restrict__ lse, const int* __restrict__ q_lens,
               const int* __restrict__ kv_lens, const __grid_constant__ Shape m) {
    using C = Cfg<D>;
    using Op = Operand<D>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sb = smem_u32(smem);
    Sync sy{sb + C::OFF_BAR, reinterpret_cast<volatile int*>(smem + C::OFF_MISC), &g_err};
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC + 16);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int s = 0; s < 2; ++s) {
            mbar_init(sy.bar(W_QF + s), 1);
            mbar_init(sy.bar(W_QE + s), 1);
            mbar_init(sy.bar(W_SF + s), 1);
            mbar_init(sy.bar(W_PF + s), 4);
            mbar_init(sy.bar(W_OF + s), 1);
        }
        for (int s = 0; s < C::NST; ++s)
            for (int x : {W_KF, W_KE, W_VF, W_VE}) mbar_init(sy.bar(x + s), 1);
        mbar_init(sy.bar(W_DRAIN), 1);
        *sy.abort = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tq);
        tma_prefetch_desc(&tk);
        tma_prefetch_desc(&tv);
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
        // ------------------------------------------------------------ producer
        if (lane < 2) {                              // K tiles (lane 0), V tiles (lane 1)
            const CUtensorMap* map = lane ? &tv : &tk;
            const int full = lane ? W_VF : W_KF, empty = lane ? W_VE : W_KE;
            const uint32_t base = sb + (lane ? C::OFF_V : C::OFF_K);
            int it = 0;
            bool ok = true;
            for (int x = blockIdx.x; x < m.items && ok; x += gridDim.x) {
                const Item t = load_item(m, q_lens, kv_lens, x);
                for (int j = 0; j < t.n && ok; ++j, ++it) {
                    const int st = it % C::NST;
                    ok = wait_one(sy, sy.bar(empty + st), ((it / C::NST) & 1) ^ 1, 0, it);
                    if (!ok) break;
                    Op::load(base + st * C::TILE, map, t.kt.tile(j) * 128, t.hk, t.b, sy.bar(full + st));
                }
            }
            if (*sy.abort)                           // wait for the last copy into every stage
                for (int st = 0; st < C::NST; ++st) {
                    const int n = (it - st + C::NST - 1) / C::NST;   // copies made into stage st
                    if (n > 0) wait_drain(sy.bar(full + st), (n - 1) & 1);
                }
        } else if (lane == 2) {                      // Q tiles
            int n[2] = {0, 0};
            bool ok = true;
            for (int x = blockIdx.x; x < m.items && ok; x += gridDim.x) {
                const Item t = load_item(m, q_lens, kv_lens, x);
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    const Slot c = t.slot(s);
                    if (!c.active || !ok) continue;
                    ok = wait_one(sy, sy.bar(W_QE + s), (n[s] & 1) ^ 1, 1, x);
                    if (!ok) continue;
                    Op::load(sb + C::OFF_Q + s * C::TILE, &tq, c.i0, c.h, t.b, sy.bar(W_QF + s));
                    ++n[s];
                }
            }
            if (*sy.abort)
#pragma unroll
                for (int s = 0; s < 2; ++s)
                    if (n[s] > 0) wait_drain(sy.bar(W_QF + s), (n[s] - 1) & 1);
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer
        {
            uint32_t sf[2] = {0, 0}, nq[2] = {0, 0};   // tiles and items begun per slot
            int it = 0;                                // tile number of the item's tile 0
            bool ok = true;
            // S of tile j (number jt) of item t in slot s; its last tile frees Q
            auto issue_s = [&](const Item& t, int s, int j, int jt) {
                if (j == 0) ok = ok && wait_warp(sy, sy.bar(W_QF + s), nq[s]++ & 1, 2, jt);
                if (!ok) return;
                tc_fence_after();
                const uint32_t id = idesc_bf16(128, 32 * tile_groups(t, m, j), 0, 0);
                const uint64_t dq = Op::kmajor(sb + C::OFF_Q + s * C::TILE);
                const uint64_t dk = Op::kmajor(sb + C::OFF_K + (jt % C::NST) * C::TILE);
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk)
                    mma_ss(tmem + C::C_S + 128u * s, dq + Op::kstep(kk), dk + Op::kstep(kk), id, kk);
                commit(sy.bar(W_SF + s));
                if (j == t.n - 1) commit(sy.bar(W_QE + s));
            };
            int x = blockIdx.x;
            Item t;
            bool have = false;
            // the next item with anything to do
            auto next = [&]() {
                for (have = false; x < m.items && !have; x += gridDim.x) {
                    t = load_item(m, q_lens, kv_lens, x);
                    have = t.n > 0;
                }
            };
            next();
            if (have) {
                ok = wait_warp(sy, sy.bar(W_KF), 0, 3, 0);
#pragma unroll
                for (int s = 0; s < 2; ++s)
                    if (t.slot(s).active) issue_s(t, s, 0, 0);
                if (ok) commit(sy.bar(W_KE));
            }
            while (have && ok) {
                const Item cur = t;
                const int n = cur.n;
                for (int j = 0; j < n && ok; ++j) {
                    const int jt = it + j, vs = jt % C::NST;
                    const bool end = j == n - 1;
                    if (end) next();                  // t: the item whose tile 0 comes next
                    const int k2 = 2 * tile_groups(cur, m, j);
                    // V of this tile and K of the next are waited for before P: a wait takes its
                    // time even when the barrier is through
                    ok = wait_warp(sy, sy.bar(W_VF + vs), (jt / C::NST) & 1, 5, jt);
                    if (ok && (!end || have))
                        ok = wait_warp(sy, sy.bar(W_KF + (jt + 1) % C::NST), ((jt + 1) / C::NST) & 1, 3, jt + 1);
#pragma unroll
                    for (int s = 0; s < 2; ++s) {
                        if (cur.slot(s).active && ok) {
                            ok = wait_warp(sy, sy.bar(W_PF + s), sf[s]++ & 1, 4, jt);
                            if (!ok) continue;
                            tc_fence_after();
                            const uint64_t dv = Op::mnmajor(sb + C::OFF_V + vs * C::TILE);
                            constexpr uint32_t ID_O = idesc_bf16(128, D, 0, 1);
                            for (int kk = 0; kk < k2; ++kk)
                                mma_ts(tmem + C::C_O + 128u * s, tmem + C::C_S + 128u * s + 8 * kk,
                                            dv + Op::MN_KSTEP * kk, ID_O, (j > 0 || kk > 0) ? 1u : 0u);
                            if (end) commit(sy.bar(W_OF + s));
                        }
                        if (!end) {
                            if (cur.slot(s).active) issue_s(cur, s, j + 1, jt + 1);
                        } else if (have && t.slot(s).active) {
                            issue_s(t, s, 0, jt + 1);
                        }
                    }
                    if (!ok) break;
                    commit(sy.bar(W_VE + vs));
                    if (!end || have) commit(sy.bar(W_KE + (jt + 1) % C::NST));
                }
                it += n;
            }
            if (!ok) {                                // let what was issued finish before TMEM is freed
                commit(sy.bar(W_DRAIN));
                wait_drain(sy.bar(W_DRAIN), 0);
            }
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------ softmax
        const int slot = (warp - 2) >> 2, q4 = warp & 3;
        const int r = q4 * 32 + lane;
        const uint32_t trow = tmem + ((uint32_t)(q4 * 32) << 16);
        const uint32_t tS = trow + C::C_S + 128u * slot, tO = trow + C::C_O + 128u * slot;
        const uint32_t stg = sb + C::OFF_EPI + 2048u * (warp - 2);
        int it = 0, nit = 0;                          // tile numbers; items done by this slot
        uint32_t sf = 0;
        bool ok = true;
        for (int x = blockIdx.x; x < m.items && ok; x += gridDim.x) {
            const Item t = load_item(m, q_lens, kv_lens, x);
            const Slot me = t.slot(slot);
            if (!me.exists) {
                it += t.n;
                continue;
            }
            const int i0 = me.i0, i = i0 + r;
            float mx = -INFINITY, l = 0.f;
            if (me.active) {
                const int pf = i0 + t.s.off, pl = min(i0 + 127, t.s.ql - 1) + t.s.off;   // first, last position
                const int p = i < t.s.ql ? i + t.s.off : -1;
                const bool zeroes = slot == 0 || !t.s0.active;
                for (int j = 0; j < t.n; ++j) {
                    const int jt = it + j, j0 = t.kt.tile(j) * 128;
                    ok = wait_warp(sy, sy.bar(W_SF + slot), sf++ & 1, 6, jt);
                    if (!ok) break;
                    tc_fence_after();
                    const int lo = p - m.window + 1 - j0, hi = p - j0, snk = m.sinks - j0;
                    const int nc = tile_groups(t, m, j);
                    if (nc == 4 && j0 + 127 <= pf && j0 > pl - m.window)
                        softmax_tile<D>(tS, tO, j == 0, m.scale_log2, mx, l);
                    else
                        softmax_edge<D>(tS, tO, j == 0, m.scale_log2, mx, l, nc, lo, hi, snk);
                    // V rows behind the sequence's end hold anything: P there is 0, but 0 times
                    // NaN is not, so the tile's first slot clears them
                    if (zeroes && j0 + 128 > t.s.kl && t.s.kl < m.Nk) {
                        ok = wait_warp(sy, sy.bar(W_VF + jt % C::NST), (jt / C::NST) & 1, 7, jt);
                        if (!ok) break;
                        if (j0 + r >= t.s.kl) Op::clear_row(sb + C::OFF_V + (jt % C::NST) * C::TILE, r);
                        fence_proxy_async_smem();
                    }
                    tc_fence_before();
                    warp_arrive(sy.bar(W_PF + slot), lane);
                }
                if (ok) ok = wait_warp(sy, sy.bar(W_OF + slot), nit++ & 1, 8, it);
                if (!ok) break;
                tc_fence_after();
            }
            it += t.n;
            // rows that saw nothing (and padding) come out as 0 and -inf
            const bool some = i < t.s.ql && (l > 0.f || l != l);
            const float inv = some ? 1.f / l : 0.f;
            if (i < m.Nq)
                lse[((size_t)t.b * m.Hq + me.h) * m.Nq + i] = some ? (mx + __log2f(l)) * kLn2 : -INFINITY;
            const int r0 = i0 + q4 * 32;
            uint16_t* row0 = o.row(t.b, me.h, r0);
            constexpr int W = D < 32 ? D : 32;        // features per store round
#pragma unroll
            for (int h = 0; h < D; h += W) {
                uint32_t v[W], w[W / 2];
                if (me.active) {
                    tmem_ld_row<W>(tO + h, v);
                    tmem_wait_ld();
                }
#pragma unroll
                for (int e = 0; e < W / 2; ++e)
                    w[e] = some ? pack_bf16x2(__uint_as_float(v[2 * e]) * inv, __uint_as_float(v[2 * e + 1]) * inv) : 0u;
                store_rows_staged<W>(stg, w, row0 + h, o.sN, m.Nq - r0, lane);
            }
            tc_fence_before();                        // O is read before the next item's first P V
        }
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, 512);
}

template <int D>
int launch(const Args& a, std::string* err) {
    using C = Cfg<D>;
    Shape m{a.B, a.Hq, a.Hkv, a.Hq / a.Hkv, a.Nq, a.Nk, a.window, a.sinks, (a.Nq + 127) / 128, 0, 0, {}, {}, {}, a.scale * kLog2e};
    m.pairs = (int)(((long long)m.G * m.nqt + 1) / 2);
    m.by_pairs = fast_div(m.pairs), m.by_hkv = fast_div(m.Hkv), m.by_g = fast_div(m.G);
    const long long items = (long long)a.B * a.Hkv * m.pairs;
    if (items > 0x3fffffffll) {
        *err = "grid too large";
        return PSA_ERR_UNSUPPORTED;
    }
    CUtensorMap tq, tk, tv;
    if (!Operand<D>::encode(&tq, a.q, a.B, a.Hq, a.Nq, 128, err) || !Operand<D>::encode(&tk, a.k, a.B, a.Hkv, a.Nk, 128, err) ||
        !Operand<D>::encode(&tv, a.v, a.B, a.Hkv, a.Nk, 128, err) ||
        !set_max_dynamic_smem((const void*)win_fwd_kernel<D>, C::SMEM, err))
        return PSA_ERR_CUDA;
    m.items = (int)items;
    int sms = 0;
    if (!sm_count(&sms, err)) return PSA_ERR_CUDA;
    ProfScope prof(kSlotFwd, a.stream);
    win_fwd_kernel<D><<<(unsigned)(items < sms ? items : sms), kThreads, C::SMEM, a.stream>>>(tq, tk, tv, row_out(a.o), a.lse,
                                                                                           a.q_lens, a.kv_lens, m);
    const cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) return PSA_OK;
    *err = std::string("window attention forward launch: ") + cudaGetErrorString(e);
    return PSA_ERR_CUDA;
}

}  // namespace

int tc_fwd(const Args& a, std::string* err) {
    switch (a.d) {
        case 16: return launch<16>(a, err);
        case 32: return launch<32>(a, err);
        case 64: return launch<64>(a, err);
        default: return launch<128>(a, err);
    }
}

int tc_fwd_take_error(std::string* err) { return take_error(g_err, "window attention forward", err); }

}  // namespace win
}  // namespace psa
