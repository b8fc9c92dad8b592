// win_tc_softmax.cuh -- a 128-key tile's online softmax between two products on the
// tensor cores, S in TMEM, P over it as bf16 pairs (win_tc_fwd.cu, win_tree_tc.cu).
#pragma once

#include "tc_ptx.cuh"
#include "win_tc.cuh"

namespace psa {
namespace win {
namespace {

using namespace psa::tc;

constexpr float kMove = 8.f;      // keep a stale row maximum while the new one is at most 2^8 larger

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

}  // namespace
}  // namespace win
}  // namespace psa
