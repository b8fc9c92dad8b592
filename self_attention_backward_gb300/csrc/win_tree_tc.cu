// win_tree_tc.cu -- attention of new tokens (a tree of drafts, a run of tokens) over
// the rolling cache on the tensor cores (tcgen05 / TMEM / TMA), bf16 queries over a bf16
// or an 8-bit cache.
//
// The softmax between the products is win_tc_fwd.cu's: per 128-row tile and 128-key tile
//   S = Q K^T;  m' = max(m, max S c) if that exceeds m by more than 8, else m
//   P = exp2(S c - m) (bf16, over S in TMEM),  l += sum P,  O += P V.
// A row is a (token, query head) of one key head, row = token G + head; a tile has the rows
// of 128 / G tokens (G heads share a key head), fetched by one TMA box over heads and tokens.
// Two tiles ("slots") of a key head go through the same K and V tiles.  Where there is one row tile
// (DUO) the two slots take its K and V tiles by turns, so that the products of one run during the
// softmax of the other, and the first slot adds both up at an item's end (32 trees of 16 drafts
// over 4100 cached slots, 4 rows a token: 125 us by one slot, 104 by two).  Not over an 8-bit
// cache, where the second slot's warps widen tiles.
//
// Keys.  A sequence's visible slots are one run of memory, or two: the sinks with the ring's
// front, and the rest of the ring.  Each is cut into 128-slot tiles wherever it starts;
// the order of keys does not matter to a softmax.  Then the new keys' tiles, whose columns a
// row sees by its ancestors (one walk up the parents per row).  Slots behind a run's end may
// hold anything: their columns are hidden and their V rows cleared, 0 times NaN is not 0.
//
// Work is split by tiles, not by sequences: the tiles of all (sequence, key head) items form
// one line, of which each CTA (one per SM) takes an equal run, whatever the lengths are; with
// more than one pair of row tiles, as many CTAs take the same run side by side, one for each
// pair, so that its keys come from L2 for all but one.  An item that lies within a run is
// written out; of the others every CTA leaves its O, m and l in the workspace, and a second
// kernel adds them up in the order of the tiles.
//
// An 8-bit cache's tiles come by TMA as they are; four more warps write them, each row times
// its scale, as bf16 into the operand's swizzled layout, a row per thread.  Draft tiles come by
// TMA as they are.  That rounding is none for the scales that the cache's writes choose, powers of two, and
// the one a bf16 cache has for others; the contract says so, the warps' kernel has none.  Without it
// here, that is with rows widened by their scale's power of two and the rest on the scores and on P
// in tiles that have such scales, every call pays for the look at its scales and for the code (32
// trees of 16 drafts: 147 us; 155 to 171 in five ways to do it).
//
// Warp 1 issues the products and owns TMEM, warps 2-5 and 6-9 are the softmax of the two
// slots, 0, 10 and 11 load K, V and Q tiles, 12-15 write the 8-bit ones (with one row tile 6-9
// too).  All waits are bounded (tc_sync.cuh).
//
// Measured and bound (d = 128): 256 tokens behind 30000, 4 sequences of 16 / 4 heads: 185 us, 1366
// TFLOP/s (a pair of slots takes some 2900 cycles a tile, of which 2048 are products); 16 trees of 64
// drafts, 32 / 8 heads, over 4100 slots: 77 us, 3700 GB/s (the same chain, half the rows); 32 trees of 16:
// 104 us, 5260 GB/s of 6795; the same over 8-bit caches: 146 us, 1950 GB/s (133 without
// any softmax: the tiles' widening).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <string>

#include "common.cuh"
#include "psa_internal.h"
#include "tc_ptx.cuh"
#include "tc_sync.cuh"
#include "tc_tmap.h"
#include "win_geom.cuh"
#include "win_internal.h"
#include "win_tc.cuh"
#include "win_tc_softmax.cuh"

namespace psa {
namespace win {
namespace {

using bf16 = __nv_bfloat16;

__device__ int g_err = 0;

// Warps: 0 K tiles (8-bit: the raw ones of K), 1 products, 2-9 softmax, 10 V tiles, 11 Q tiles, 12-15 8-bit tiles.
constexpr int kSoft = 384, kConv = 128;           // threads without the last four warps; theirs

template <int D, bool E8>
struct Cfg {
    using O = Operand<D>;
    static constexpr int TILE = O::TILE;
    static constexpr int NK = E8 ? (D == 128 ? 1 : 2) : D == 128 ? 2 : 4, NV = NK;   // K stages, V stages
    // 8-bit tiles as they lie in memory: their stages, the first ones K's
    static constexpr int RAW = 128 * D, NRK = 2, NRV = 3, NR = E8 ? NRK + NRV : 0;
    static constexpr int OFF_Q = 0;                  // two slots
    static constexpr int OFF_K = 2 * TILE;
    static constexpr int OFF_V = OFF_K + NK * TILE;
    static constexpr int OFF_RAW = OFF_V + NV * TILE;
    static constexpr int OFF_EPI = OFF_RAW + NR * RAW;   // 2 KB per softmax warp
    static constexpr int OFF_BAR = OFF_EPI + 8 * 2048;
    static constexpr int OFF_MISC = OFF_BAR + 384;
    static constexpr int OFF_OTHER = OFF_MISC + 256;     // DUO: the second slot's m and l
    static constexpr int USED = OFF_OTHER + 1024 + 1024;
    static constexpr int SMEM = USED > 118784 ? USED : 118784;   // one CTA per SM: each takes all of TMEM
    static constexpr uint32_t C_S = 0, C_O = 256;    // S of slot s at 128 s, O at 256 + 128 s
    static_assert(USED <= 232448, "shared memory");
};
template <int D>
constexpr int kPart = 128 * (D + 2);                 // floats of a slot's partial result: O [D / 4][128][4], m, l

// barriers (slot s or stage s behind each)
enum { W_QF = 0, W_QE = 2, W_SF = 4, W_PF = 6, W_OF = 8, W_KF = 10, W_KE = 14, W_VF = 18, W_VE = 22, W_DRAIN = 26, W_RF = 27,
       W_RE = 33, W_MX = 38, W_MD = 39 };

struct Shape {
    int B, Hq, Hkv, G, T, cap, window, sinks;
    int NT, ntile, pairs, slots;      // tokens per row tile, row tiles and pairs of them per key head; slots in use
    int parts;                        // runs that the tiles are cut into at most
    FastDiv by_pairs, by_g;
    float scale_log2;
    long long par_stride;
    const float* ks;                  // 8-bit caches: scales
    const float* vs;
    long long cB, cH, cS;
};

// A sequence: its new tokens, its visible cached positions x < nv and the runs of slots that
// hold them.  Slot s of a run (beyond the sinks) is position x = s + off.
struct Runs {
    int L, n, nv, a_len, a_off, b_slot, b_len, b_off;   // run a starts at slot 0
    int n1, n2, total;                                  // tiles of run a, of run b, with the drafts'
};
__device__ __forceinline__ Runs load_runs(const Shape& m, const int* lens, const int* n_new, int b) {
    Runs r;
    r.L = max(__ldg(lens + b), 0);
    r.n = n_new ? min(max(__ldg(n_new + b), 0), m.T) : m.T;
    const int ring = m.cap - m.sinks;
    r.nv = r.n ? (int)min((long long)r.L, (long long)m.sinks + m.window - 1) : 0;
    const int r0 = (r.L - r.nv) % ring;
    r.a_len = r.nv, r.a_off = 0, r.b_slot = 0, r.b_len = 0, r.b_off = 0;
    if (r.nv < r.L && r0 > 0 && r.n) {
        const int cnt = r.nv - m.sinks, len1 = min(cnt, ring - r0);
        r.a_len = m.sinks + cnt - len1, r.a_off = len1;
        r.b_slot = m.sinks + r0, r.b_len = len1, r.b_off = -r0;
    }
    r.n1 = (r.a_len + 127) / 128, r.n2 = (r.b_len + 127) / 128;
    r.total = r.n1 + r.n2 + max((r.n + 127) / 128, 1);
    return r;
}
// Tile t of an item: its first slot, or first draft; how many of its 128 keys are there.
struct Tile {
    bool draft;
    int row, valid, off;
    __device__ __forceinline__ int groups() const { return valid <= 32 ? 1 : 4; }   // of 32 columns
};
__device__ __forceinline__ Tile tile_of(const Runs& r, int t) {
    Tile x;
    x.draft = t >= r.n1 + r.n2;
    if (t < r.n1) {
        x.row = 128 * t, x.valid = r.a_len - x.row, x.off = r.a_off;
    } else if (!x.draft) {
        x.row = r.b_slot + 128 * (t - r.n1), x.valid = r.b_slot + r.b_len - x.row, x.off = r.b_off;
    } else {
        x.row = 128 * (t - r.n1 - r.n2), x.valid = max(r.n - x.row, 0), x.off = 0;
    }
    x.valid = min(x.valid, 128);
    return x;
}

struct Slot {
    int n0, q;                    // first token; row tile
    bool exists, active;          // active: some of its tokens are there
};
// A CTA's run of tiles, (sequence, key head) by (sequence, key head), for its pair of row tiles.
struct Line {
    int pos, end, base, b;        // next tile; end; first tile of sequence b
    Runs r;
};
struct Item {
    int b, hk, t0, t1;            // tiles t0 .. t1 - 1 of it
    Runs r;
    Slot s0, s1;
    __device__ __forceinline__ Slot slot(int i) const { return i ? s1 : s0; }
    __device__ __forceinline__ bool whole() const { return t0 == 0 && t1 == r.total; }
};
struct Start {                    // found once per CTA
    int pos, end, base, b;
    int q, rem, part, pair;       // this is run `part`; runs have q tiles, the first `rem` one more
};
__device__ __forceinline__ Line line_of(const Shape& m, const Start& s, const int* lens, const int* n_new) {
    Line l{s.pos, s.end, s.base, s.b, {}};
    if (l.pos < l.end) l.r = load_runs(m, lens, n_new, l.b);
    return l;
}
__device__ __forceinline__ bool next_item(Line& l, const Shape& m, int pair, const int* lens, const int* n_new, Item& t) {
    if (l.pos >= l.end) return false;
    while (l.pos >= l.base + l.r.total * m.Hkv) {
        l.base += l.r.total * m.Hkv;
        l.r = load_runs(m, lens, n_new, ++l.b);
    }
    const int rel = l.pos - l.base;
    t.hk = (int)((unsigned)rel / (unsigned)l.r.total);
    t.b = l.b, t.r = l.r;
    t.t0 = rel - t.hk * l.r.total;
    t.t1 = min(l.r.total, t.t0 + (l.end - l.pos));
    l.pos += t.t1 - t.t0;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        Slot c;
        c.q = 2 * pair + s;
        c.n0 = c.q * m.NT;
        c.exists = c.q < m.ntile;
        c.active = c.exists && c.n0 < t.r.n;
        (s ? t.s1 : t.s0) = c;
    }
    return true;
}

// This CTA's run: the tiles of all sequences are added up, and the sequence that its first
// tile lies in is looked for (each thread has a few neighbouring sequences).  Where there is a
// CTA for every item, and the longest item is at most kAlone tiles more than an equal run,
// the items stay whole: writing and adding up parts costs as much (16 trees of 64 drafts: 77 us, 82
// with every item cut; a limit of 20 tiles is no faster).
constexpr int kAlone = 6;
template <int THREADS>
__device__ __forceinline__ void find_start(const Shape& m, const int* lens, const int* n_new, Start* out, int2* sums) {
    const int per = (m.B + THREADS - 1) / THREADS, b0 = min((int)threadIdx.x * per, m.B), b1 = min(b0 + per, m.B);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int mine = 0, most = 0;
    for (int b = b0; b < b1; ++b) {
        const int n = load_runs(m, lens, n_new, b).total;
        mine += n * m.Hkv;
        most = max(most, n);
    }
    int upto = mine;
#pragma unroll
    for (int i = 1; i < 32; i <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, upto, i);
        if (lane >= i) upto += x;
    }
    most = __reduce_max_sync(0xffffffffu, most);
    if (lane == 31) sums[warp] = make_int2(upto, most);
    __syncthreads();
    int all = 0, before = upto - mine;
    for (int w = 0; w < THREADS / 32; ++w) {
        const int2 x = sums[w];
        if (w < warp) before += x.x;
        all += x.x;
        most = max(most, x.y);
    }
    const int part = divide(blockIdx.x, m.by_pairs), pair = blockIdx.x - part * m.pairs, runs = m.parts, items = m.B * m.Hkv;
    // two tiles a run at least, where items have many: half as many parts to add up (26 drafts over
    // 4100 slots, 4 key heads: 20.4 us by 136 runs, 17.7 by 68; 2 sequences of 1000, 8 key heads, 9
    // tiles an item: 16.4 by 144, 18.4 by 72)
    const int parts = min(runs, all > 16 * items ? (all + 1) / 2 : all), q = (int)((unsigned)all / (unsigned)parts), rem = all - q * parts;
    if (items <= runs && most <= q + kAlone) {
        const int b = part / m.Hkv;                   // item `part`, whole
        if (part >= items) {
            if (threadIdx.x == 0) *out = Start{0, 0, 0, 0, all, 0, part, pair};
        } else if (b >= b0 && b < b1) {
            const int n = load_runs(m, lens, n_new, b).total, at = (part - b * m.Hkv) * n;
            *out = Start{at, at + n, 0, b, all, 0, part, pair};
        }
        return;
    }
    const int pos = part * q + min(part, rem), end = part < parts ? pos + q + (part < rem) : pos;
    if (pos >= end) {
        if (threadIdx.x == 0) *out = Start{0, 0, 0, 0, q, rem, part, pair};
    } else if (mine > 0 && pos >= before && pos < before + mine) {
        int b = b0, base = before;
        for (;;) {
            const int n = load_runs(m, lens, n_new, b).total * m.Hkv;
            if (pos < base + n) break;
            base += n, ++b;
        }
        *out = Start{pos, end, base, b, q, rem, part, pair};
    }
}

// Number of ancestors of a node; par: its sequence's parents (shared memory), 0: a run.
__device__ __forceinline__ int parent_of(uint32_t par, int t) {
    int p;
    asm volatile("ld.shared.s32 %0, [%1];" : "=r"(p) : "r"(par + 4 * t) : "memory");
    return p < t ? p : -1;
}
__device__ __forceinline__ int depth_of(uint32_t par, int node) {
    if (!par) return node;
    int d = 0;
    for (int t = parent_of(par, node); t >= 0; t = parent_of(par, t)) ++d;
    return d;
}
// Which of the drafts j0 .. j0 + 127 a node sees: itself and its ancestors, those within the
// window or below the sinks.
__device__ __forceinline__ void drafts_seen(uint32_t par, int node, int depth, int j0, int L, const Shape& m, uint32_t (&see)[4]) {
    if (!par) {
        // sinks - L - j0: drafts whose position is below the sinks
        const int snk = (int)max((long long)m.sinks - L - j0, -1ll);
#pragma unroll
        for (int g = 0; g < 4; ++g) see[g] = col_mask(node - m.window + 1 - j0, node - j0, min(snk, node - j0 + 1), 32 * g);
        return;
    }
#pragma unroll
    for (int g = 0; g < 4; ++g) see[g] = 0;
    int k = 0;
    for (int t = node; t >= 0; t = parent_of(par, t), ++k) {
        if ((unsigned)(t - j0) < 128u && (k < m.window || (long long)L + depth - k < m.sinks)) {
#pragma unroll
            for (int g = 0; g < 4; ++g)
                if ((t - j0) >> 5 == g) see[g] |= 1u << (t & 31);
        }
    }
}

// softmax_tile of win_tc_softmax.cuh in half the code, two groups of 32 columns a round: the warps
// of this kernel run five different loops, which do not all stay in the instruction cache (16
// trees of 64 drafts: 82 us with softmax_tile, 78 with this).  Over an 8-bit cache, where a thread
// has 128 registers, its loops keep some in local memory, and softmax_tile is the faster one (32
// trees of 16: 173 us with this, 153).
template <int D>
__device__ __forceinline__ void softmax_full(uint32_t tS, uint32_t tO, bool first, float c, float& m, float& l) {
    uint32_t xa[32], xb[32];
    float ma = -INFINITY, mb = -INFINITY;
    tmem_ld_32x32b_x32(tS, xa);
#pragma unroll 1
    for (int g = 0; g < 128; g += 64) {
        tmem_wait_ld();
        tmem_ld_32x32b_x32(tS + g + 32, xb);
        max_group(xa, ma, mb);
        tmem_wait_ld();
        tmem_ld_32x32b_x32(tS + ((g + 64) & 127), xa);
        max_group(xb, ma, mb);
    }
    const float nm = move_max<D>(tO, first, fmaxf(ma, mb) * c, m, l);   // c > 0
    const uint64_t c2 = f2_pack(c, c), r2 = f2_pack(nm, nm);
    uint64_t la = f2_pack(0.f, 0.f), lb = la;
#pragma unroll 1
    for (int g = 0; g < 128; g += 64) {
        tmem_wait_ld();
        tmem_ld_32x32b_x32(tS + g + 32, xb);
        prob_group(xa, c2, r2, la, lb, tS + g / 2);
        tmem_wait_ld();
        if (g == 0) tmem_ld_32x32b_x32(tS + 64, xa);
        prob_group(xb, c2, r2, la, lb, tS + g / 2 + 16);
    }
    l += pair_sum(la, lb);
    tmem_wait_st();
}

// A tile of nc 32-column groups of which the row sees the bits `see` (as softmax_edge of
// win_tc_fwd.cu: groups that no row of the warp sees are left out, P = 0).
template <int D>
__device__ __forceinline__ void softmax_masked(uint32_t tS, uint32_t tO, bool first, float c, float& m, float& l, int nc,
                                               const uint32_t (&see)[4]) {
    uint32_t x[32];
    float ma = -INFINITY, mb = -INFINITY;
    uint32_t some = 0;
#pragma unroll 1
    for (int g = 0; g < nc; ++g) {
        const uint32_t w = g == 0 ? see[0] : g == 1 ? see[1] : g == 2 ? see[2] : see[3];
        if (!__any_sync(0xffffffffu, w != 0u)) continue;
        some |= 1u << g;
        tmem_ld_32x32b_x32(tS + 32 * g, x);
        tmem_wait_ld();
        if (!__all_sync(0xffffffffu, w == 0xffffffffu)) {
            hide(x, w);
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

// ------------------------------------------------------------------ 8-bit tiles
// 16 e4m3 numbers times s as 16 bf16.
__device__ __forceinline__ void widen16(const uint4& u, uint64_t s2, uint32_t (&w)[8]) {
    const uint32_t x[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        uint32_t h;
        if (i % 2)
            asm("{\n\t.reg .b16 t, u;\n\tmov.b32 {t, u}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, u;\n\t}" : "=r"(h) : "r"(x[i / 2]));
        else
            asm("{\n\t.reg .b16 t, u;\n\tmov.b32 {t, u}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}" : "=r"(h) : "r"(x[i / 2]));
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
        float a, b;
        f2_unpack(f2_mul(f2_pack(f.x, f.y), s2), a, b);
        w[i] = pack_bf16x2(a, b);
    }
}
// Row r of an 8-bit tile (swizzled over its row by TMA) to row r of an operand tile, times s;
// zeros where it is not there.  A short loop of two chunks, whose loads go first (32 trees of 16
// drafts: 146 us, 150 one after the other): written out, its code takes longer to come than to run
// (four at once 159, eight 178).
template <int D>
__device__ __forceinline__ void widen_row(uint32_t raw, float s, bool there, uint32_t tile, int r) {
    using O = Operand<D>;
    constexpr int CH = D / 16, C = O::ROWB / 16;     // chunks of a raw row, of a panel row: 8, 4 or 2
    const int rw = CH > 1 ? (r / (8 / CH)) & (CH - 1) : 0, sw = (r / (8 / C)) & (C - 1);
    const uint64_t s2 = f2_pack(s, s);
    raw += r * D;
    tile += r * O::ROWB;
    constexpr int AT = CH < 2 ? CH : 2;
#pragma unroll 1
    for (int c0 = 0; c0 < CH; c0 += AT) {
        uint4 u[AT];
#pragma unroll
        for (int i = 0; i < AT; ++i) u[i] = ld_shared_v4(raw + 16 * ((c0 + i) ^ rw));
#pragma unroll
        for (int i = 0; i < AT; ++i) {
            const int c = c0 + i;
            uint32_t w[8];
            widen16(u[i], s2, w);
            if (!there)
#pragma unroll
                for (int e = 0; e < 8; ++e) w[e] = 0;
            const uint32_t row = tile + 16 * c / O::W * O::PANEL;
            const int ch = 16 * c % O::W / 8;
            st_shared_v4(row + 16 * (ch ^ sw), w[0], w[1], w[2], w[3]);
            st_shared_v4(row + 16 * ((ch + 1) ^ sw), w[4], w[5], w[6], w[7]);
        }
    }
}

template <int D, bool E8, bool DUO>
__global__ void __launch_bounds__(kSoft + (E8 ? kConv : 0), 1)
tree_tc_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
               const __grid_constant__ CUtensorMap tkn, const __grid_constant__ CUtensorMap tvn, RowOut o, float* __restrict__ lse,
               const int* __restrict__ lens, const int* __restrict__ n_new, const int* __restrict__ parents,
               float* __restrict__ part, int2* __restrict__ desc, const __grid_constant__ Shape m) {
    using C = Cfg<D, E8>;
    using Op = Operand<D>;
    constexpr int THREADS = kSoft + (E8 ? kConv : 0);
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sb = smem_u32(smem);
    Sync sy{sb + C::OFF_BAR, reinterpret_cast<volatile int*>(smem + C::OFF_MISC), &g_err};
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC + 16);
    Start* start = reinterpret_cast<Start*>(smem + C::OFF_MISC + 32);
    int2* sums = reinterpret_cast<int2*>(smem + C::OFF_MISC + 96);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // warps that write 8-bit tiles, for K and for V each: the second slot's help where it has no rows
    const int nconv = m.slots == 1 ? 4 : 2;
    float* const other = reinterpret_cast<float*>(smem + C::OFF_OTHER);

    if (threadIdx.x == 0) {
        for (int s = 0; s < 2; ++s) {
            mbar_init(sy.bar(W_QF + s), 1);
            mbar_init(sy.bar(W_QE + s), 1);
            mbar_init(sy.bar(W_SF + s), 1);
            mbar_init(sy.bar(W_PF + s), 4);
            mbar_init(sy.bar(W_OF + s), 1);
        }
        for (int s = 0; s < C::NK; ++s) mbar_init(sy.bar(W_KF + s), E8 ? nconv : 1), mbar_init(sy.bar(W_KE + s), 1);
        for (int s = 0; s < C::NV; ++s) mbar_init(sy.bar(W_VF + s), E8 ? nconv : 1), mbar_init(sy.bar(W_VE + s), 1);
        for (int s = 0; s < C::NR; ++s) mbar_init(sy.bar(W_RF + s), 1), mbar_init(sy.bar(W_RE + s), nconv);
        mbar_init(sy.bar(W_DRAIN), 1);
        mbar_init(sy.bar(W_MX), 4);
        mbar_init(sy.bar(W_MD), 4);
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
    find_start<THREADS>(m, lens, n_new, start, sums);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    griddep_launch_dependents();
    const uint32_t tmem = *tmem_slot;
    const Start st0 = *start;
    const uint32_t q_bytes = (uint32_t)(m.NT * m.G) * Op::ROWB * (D / Op::W);

    if (warp == 0 || warp == 10) {
        // ------------------------------------------------------------ K tiles, V tiles
        if (lane == 0) {
            const bool v = warp == 10;
            const CUtensorMap *map = v ? &tv : &tk, *mapn = v ? &tvn : &tkn;
            const int nst = E8 ? (v ? C::NRV : C::NRK) : C::NK, off = E8 && v ? C::NRK : 0;
            const int full = (E8 ? W_RF : v ? W_VF : W_KF) + off, empty = (E8 ? W_RE : v ? W_VE : W_KE) + off;
            const uint32_t base = sb + (E8 ? C::OFF_RAW + off * C::RAW : v ? C::OFF_V : C::OFF_K);
            int it = 0, st = 0, ph = 0;               // stage and its round
            bool ok = true;
            Line l = line_of(m, st0, lens, n_new);
            Item t;
            while (ok && next_item(l, m, st0.pair, lens, n_new, t))
                for (int j = t.t0; j < t.t1; ++j) {
                    const Tile x = tile_of(t.r, j);
                    if (E8 && x.draft) break;         // the other warps bring it
                    ok = wait_one(sy, sy.bar(empty + st), (ph & 1) ^ 1, 0, it);
                    if (!ok) break;
                    if constexpr (E8) {
                        mbar_arrive_expect_tx(sy.bar(full + st), C::RAW);
                        tma_load_4d(base + st * C::RAW, map, 0, x.row, t.hk, t.b, sy.bar(full + st));
                    } else {
                        Op::load(base + st * C::TILE, x.draft ? mapn : map, x.row, t.hk, t.b, sy.bar(full + st));
                    }
                    ++it;
                    if (++st == nst) st = 0, ++ph;
                }
            if (*sy.abort)                           // wait for the last copy into every stage
                for (int i = 0; i < nst; ++i) {
                    const int n = (it - i + nst - 1) / nst;   // copies made into stage i
                    if (n > 0) wait_drain(sy.bar(full + i), (n - 1) & 1);
                }
        }
        __syncwarp();
    } else if (warp == 11) {
        // ------------------------------------------------------------ Q tiles
        if (lane == 0) {
            int n[2] = {0, 0};
            bool ok = true;
            Line l = line_of(m, st0, lens, n_new);
            Item t;
            while (ok && next_item(l, m, st0.pair, lens, n_new, t)) {
#pragma unroll
                for (int s = 0; s < (DUO ? 1 : 2); ++s) {
                    const Slot c = t.slot(s);
                    if (!c.active || !ok) continue;
                    ok = wait_one(sy, sy.bar(W_QE + s), (n[s] & 1) ^ 1, 1, n[s]);
                    if (!ok) continue;
                    mbar_arrive_expect_tx(sy.bar(W_QF + s), q_bytes);
#pragma unroll
                    for (int p = 0; p < D / Op::W; ++p)
                        tma_load_4d(sb + C::OFF_Q + s * C::TILE + p * Op::PANEL, &tq, p * Op::W, t.hk * m.G, c.n0, t.b,
                                    sy.bar(W_QF + s));
                    ++n[s];
                }
            }
            if (*sy.abort)
#pragma unroll
                for (int s = 0; s < 2; ++s)
                    if (n[s] > 0) wait_drain(sy.bar(W_QF + s), (n[s] - 1) & 1);
        }
        __syncwarp();
    } else if (warp == 1 && DUO) {
        // ------------------------------------------------------------ MMA issuer, slots by turns
        bool ok = true;
        // the tile whose S is next (two ahead of the products P V): its item, number, stage and round
        Line ls = line_of(m, st0, lens, n_new), lp = ls;
        Item ts, tp;
        bool hs = next_item(ls, m, st0.pair, lens, n_new, ts);
        int js = hs ? ts.t0 : 0, gs = 0, ks = 0, kr = 0;
        uint32_t nq = 0, sf[2] = {0, 0};
        auto issue_s = [&]() {
            if (!hs || !ok) return;
            ok = warp_wait(sy, sy.bar(W_KF + ks), kr & 1, 3, gs);
            if (ok && ts.s0.active) {
                if (js == ts.t0) ok = warp_wait(sy, sy.bar(W_QF), nq++ & 1, 2, gs);
                if (!ok) return;
                tc_fence_after();
                const int nk = 32 * tile_of(ts.r, js).groups();
                const uint32_t id = idesc_bf16(128, nk, 0, 0);
                const uint64_t dq = Op::kmajor(sb + C::OFF_Q), dk = Op::kmajor(sb + C::OFF_K + ks * C::TILE);
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk)
                    mma_ss(tmem + C::C_S + 128u * (gs & 1), dq + Op::kstep(kk), dk + Op::kstep(kk), id, kk);
                commit(sy.bar(W_SF + (gs & 1)));
                if (js == ts.t1 - 1) commit(sy.bar(W_QE));
            }
            if (ok) commit(sy.bar(W_KE + ks));
            if (++ks == C::NK) ks = 0, ++kr;
            ++gs;
            if (++js == ts.t1) {
                hs = next_item(ls, m, st0.pair, lens, n_new, ts);
                js = hs ? ts.t0 : 0;
            }
        };
        int gp = 0, vs = 0, vr = 0;
        auto ahead = [&]() {                          // S up to two tiles ahead of P V
#pragma unroll 1
            while (ok && hs && gs < gp + 2) issue_s();
        };
        ahead();
        while (ok && next_item(lp, m, st0.pair, lens, n_new, tp)) {
#pragma unroll 1
            for (int j = tp.t0; j < tp.t1 && ok; ++j) {
                const int s = gp & 1;
                ok = warp_wait(sy, sy.bar(W_VF + vs), vr & 1, 5, gp);
                if (ok && tp.s0.active) {
                    ok = warp_wait(sy, sy.bar(W_PF + s), (s ? sf[1]++ : sf[0]++) & 1, 4, gp);
                    if (!ok) break;
                    tc_fence_after();
                    const int k2 = 2 * tile_of(tp.r, j).groups();
                    const uint64_t dv = Op::mnmajor(sb + C::OFF_V + vs * C::TILE);
                    constexpr uint32_t ID_O = idesc_bf16(128, D, 0, 1);
                    for (int kk = 0; kk < k2; ++kk)
                        mma_ts(tmem + C::C_O + 128u * s, tmem + C::C_S + 128u * s + 8 * kk, dv + Op::MN_KSTEP * kk, ID_O,
                               (j - tp.t0 >= 2 || kk > 0) ? 1u : 0u);
                    if (j + 2 >= tp.t1) commit(sy.bar(W_OF + s));
                }
                if (!ok) break;
                commit(sy.bar(W_VE + vs));
                if (++vs == C::NK) vs = 0, ++vr;
                ++gp;
                ahead();
            }
        }
        if (!ok) {                                    // let what was issued finish before TMEM is freed
            commit(sy.bar(W_DRAIN));
            wait_drain(sy.bar(W_DRAIN), 0);
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer
        uint32_t sf[2] = {0, 0}, nq[2] = {0, 0};     // tiles and items begun per slot
        int it = 0;                                  // number of the item's first tile
        bool ok = true;
        // S of tile j (number jt) of item t in slot s; the item's last tile frees Q
        auto issue_s = [&](const Item& t, int s, int j, int jt) {
            if (j == t.t0) ok = ok && wait_warp(sy, sy.bar(W_QF + s), nq[s]++ & 1, 2, jt);
            if (!ok) return;
            tc_fence_after();
            const uint32_t id = idesc_bf16(128, 32 * tile_of(t.r, j).groups(), 0, 0);
            const uint64_t dq = Op::kmajor(sb + C::OFF_Q + s * C::TILE);
            const uint64_t dk = Op::kmajor(sb + C::OFF_K + (jt % C::NK) * C::TILE);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
                mma_ss(tmem + C::C_S + 128u * s, dq + Op::kstep(kk), dk + Op::kstep(kk), id, kk);
            commit(sy.bar(W_SF + s));
            if (j == t.t1 - 1) commit(sy.bar(W_QE + s));
        };
        Line l = line_of(m, st0, lens, n_new);
        Item t;
        // the next item (an item with no token there is a tile that is only read)
        bool have = next_item(l, m, st0.pair, lens, n_new, t);
        if (have) {
            ok = wait_warp(sy, sy.bar(W_KF), 0, 3, 0);
#pragma unroll
            for (int s = 0; s < 2; ++s)
                if (t.slot(s).active) issue_s(t, s, t.t0, 0);
            if (ok) commit(sy.bar(W_KE));
        }
        while (have && ok) {
            const Item cur = t;
            const int n = cur.t1 - cur.t0;
            for (int j = 0; j < n && ok; ++j) {
                const int jt = it + j, vs = jt % C::NV, kn = (jt + 1) % C::NK;
                const bool end = j == n - 1;
                if (end) have = next_item(l, m, st0.pair, lens, n_new, t);   // t: the item whose first tile comes next
                const int k2 = 2 * tile_of(cur.r, cur.t0 + j).groups();
                // V of this tile and K of the next are waited for before P: a wait takes its
                // time even when the barrier is through
                ok = wait_warp(sy, sy.bar(W_VF + vs), (jt / C::NV) & 1, 5, jt);
                if (ok && (!end || have)) ok = wait_warp(sy, sy.bar(W_KF + kn), ((jt + 1) / C::NK) & 1, 3, jt + 1);
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    if (cur.slot(s).active && ok) {
                        ok = wait_warp(sy, sy.bar(W_PF + s), sf[s]++ & 1, 4, jt);
                        if (!ok) continue;
                        tc_fence_after();
                        const uint64_t dv = Op::mnmajor(sb + C::OFF_V + vs * C::TILE);
                        constexpr uint32_t ID_O = idesc_bf16(128, D, 0, 1);
                        for (int kk = 0; kk < k2; ++kk)
                            mma_ts(tmem + C::C_O + 128u * s, tmem + C::C_S + 128u * s + 8 * kk, dv + Op::MN_KSTEP * kk, ID_O,
                                   (j > 0 || kk > 0) ? 1u : 0u);
                        if (end) commit(sy.bar(W_OF + s));
                    }
                    if (!end) {
                        if (cur.slot(s).active) issue_s(cur, s, cur.t0 + j + 1, jt + 1);
                    } else if (have && t.slot(s).active) {
                        issue_s(t, s, t.t0, jt + 1);
                    }
                }
                if (!ok) break;
                commit(sy.bar(W_VE + vs));
                if (!end || have) commit(sy.bar(W_KE + kn));
            }
            it += n;
        }
        if (!ok) {                                    // let what was issued finish before TMEM is freed
            commit(sy.bar(W_DRAIN));
            wait_drain(sy.bar(W_DRAIN), 0);
        }
        __syncwarp();
    } else if (warp < 10 && (warp < 6 || m.slots == 2 || !E8)) {
        // ------------------------------------------------------------ softmax
        const int slot = (warp - 2) >> 2, q4 = warp & 3;
        const int r = q4 * 32 + lane;
        const uint32_t trow = tmem + ((uint32_t)(q4 * 32) << 16);
        const uint32_t tS = trow + C::C_S + 128u * slot, tO = trow + C::C_O + 128u * slot;
        const uint32_t stg = sb + C::OFF_EPI + 2048u * (warp - 2);
        const int rt = divide(r, m.by_g);             // the row's token of its tile
        int it = 0, nit = 0, ni = 0;                  // tile numbers; items that this slot had tiles of; items
        uint32_t sf = 0, owed = 0;                    // DUO: whether the first slot still has to take this one's sums
        bool ok = true;
        Line l = line_of(m, st0, lens, n_new);
        Item t;
        while (ok && next_item(l, m, st0.pair, lens, n_new, t)) {
            const Slot me = DUO ? t.s0 : t.slot(slot);
            // which runs have the item, for all its pairs of row tiles
            if (t.t0 == 0 && st0.pair == 0 && warp == 2 && lane == 0) {
                int last = -1;                        // the run of the item's last tile
                if (!t.whole()) {
                    const unsigned p = l.pos - t.t1 + t.r.total - 1, longer = st0.rem * (st0.q + 1);
                    last = (int)(p < longer ? p / (st0.q + 1) : st0.rem + (p - longer) / st0.q);
                }
                desc[(long long)t.b * m.Hkv + t.hk] = make_int2(st0.part, last);
            }
            const int n = t.t1 - t.t0;
            if (!me.exists) {
                it += n;
                continue;
            }
            const int node = me.n0 + rt;
            const bool real = rt < m.NT && node < t.r.n;
            const bool idle = !__any_sync(0xffffffffu, real);   // what P and O hold in such a warp's rows is never read
            float mx = -INFINITY, lsum = 0.f;
            if (me.active) {
                // a row sees slot s of the ring when s > low - off; rows differ by their depths
                const int top = t.r.nv - m.window + t.r.n - 1;
                const bool deep = top >= m.sinks || t.t1 > t.r.n1 + t.r.n2;
                if (parents && deep) {                // to the warp's staging rows, which the item's end uses again
                    const int* from = parents + t.b * m.par_stride;
                    int p[PSA_TREE_MAX / 32];
#pragma unroll
                    for (int i = 0; i < PSA_TREE_MAX / 32; ++i) p[i] = lane + 32 * i < t.r.n ? __ldg(from + lane + 32 * i) : -1;
#pragma unroll
                    for (int i = 0; i < PSA_TREE_MAX / 32; ++i) st_shared_b32(stg + 4 * (lane + 32 * i), (uint32_t)p[i]);
                    __syncwarp();
                }
                const uint32_t par = parents ? stg : 0;
                int depth = 0;
                if (real && deep) depth = depth_of(par, node);
                const int low = t.r.nv - m.window + depth;
                const bool zeroes = DUO || slot == 0;   // (the first slot has tokens where the second has)
                const int j0 = DUO ? t.t0 + ((it & 1) != slot) : t.t0;
                for (int j = j0; j < t.t1; j += DUO ? 2 : 1) {
                    const int jt = it + j - t.t0;
                    const Tile x = tile_of(t.r, j);
                    const int nc = x.groups();
                    uint32_t see[4] = {0, 0, 0, 0};
                    bool full = false;
                    if (x.draft) {
                        if (real) drafts_seen(par, node, depth, x.row, t.r.L, m, see);
                    } else {
                        const int f = max(x.row, m.sinks);
                        full = x.valid == 128 && (f > x.row + 127 || f + x.off > top);
                        if (!full && real) {
#pragma unroll
                            for (int g = 0; g < 4; ++g)
                                see[g] = col_mask(low - x.off + 1 - x.row, x.valid - 1, m.sinks - x.row, 32 * g);
                        }
                    }
                    ok = wait_warp(sy, sy.bar(W_SF + slot), sf++ & 1, 6, jt);
                    if (!ok) break;
                    tc_fence_after();
                    if (!idle) {
                        if (full && E8)
                            softmax_tile<D>(tS, tO, j == j0, m.scale_log2, mx, lsum);
                        else if (full)
                            softmax_full<D>(tS, tO, j == j0, m.scale_log2, mx, lsum);
                        else
                            softmax_masked<D>(tS, tO, j == j0, m.scale_log2, mx, lsum, nc, see);
                    }
                    // V rows that are not there hold anything: the tile's first slot clears them (an
                    // 8-bit tile has zeros there)
                    if (zeroes && x.valid < 128 && (!E8 || x.draft)) {
                        ok = wait_warp(sy, sy.bar(W_VF + jt % C::NV), (jt / C::NV) & 1, 7, jt);
                        if (!ok) break;
                        if (r >= x.valid) Op::clear_row(sb + C::OFF_V + (jt % C::NV) * C::TILE, r);
                        fence_proxy_async_smem();
                    }
                    if (DUO && owed) {                // P V writes O, which the first slot has to have read
                        ok = wait_warp(sy, sy.bar(W_MD), (ni - 1) & 1, 14, jt);
                        if (!ok) break;
                        owed = 0;
                    }
                    tc_fence_before();
                    warp_arrive(sy.bar(W_PF + slot), lane);
                }
                if (ok && j0 < t.t1) ok = wait_warp(sy, sy.bar(W_OF + slot), nit++ & 1, 8, it);
                if (!ok) break;
                tc_fence_after();
            }
            const bool had = !DUO || n > 1 || (it & 1) == slot, other_had = DUO && (n > 1 || (it & 1) != slot);
            it += n;
            float a0 = 1.f, a1 = 0.f;                 // DUO: what the slots' sums are multiplied by
            if (DUO && me.active) {
                if (slot == 1) {
                    if (owed) ok = wait_warp(sy, sy.bar(W_MD), (ni - 1) & 1, 14, it);
                    if (!ok) break;
                    other[r] = mx, other[128 + r] = lsum;
                    tc_fence_before();
                    warp_arrive(sy.bar(W_MX), lane);
                    owed = 1, ++ni;
                    continue;
                }
                ok = wait_warp(sy, sy.bar(W_MX), ni & 1, 13, it);
                if (!ok) break;
                tc_fence_after();
                const float m1 = other[r], top = fmaxf(mx, m1);
                a0 = mx == -INFINITY ? 0.f : ex2(mx - top);
                a1 = m1 == -INFINITY ? 0.f : ex2(m1 - top);
                lsum = fmaf(lsum, a0, other[128 + r] * a1);
                mx = top;
            } else if (DUO && slot == 1) {
                continue;
            }
            if (me.active) ++ni;
            // the slot's sums of W features; DUO: both slots' as one
            constexpr int W = DUO || D < 32 ? 16 : 32;   // features per round
            auto sums = [&](int h, uint32_t (&v)[W]) {
                if (had) {
                    tmem_ld_row<W>(tO + h, v);
                    tmem_wait_ld();
                }
                if constexpr (DUO) {
#pragma unroll
                    for (int e = 0; e < W; ++e) v[e] = had ? __float_as_uint(__uint_as_float(v[e]) * a0) : 0u;
                    if (other_had) {
                        uint32_t u[16];
                        tmem_ld_32x32b_x16(tO + 128 + h, u);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 16; ++e) v[e] = __float_as_uint(fmaf(__uint_as_float(u[e]), a1, __uint_as_float(v[e])));
                    }
                }
            };
            if (t.whole() || (!me.active && t.t0 == 0)) {
                // rows that are not there come out as 0 and -inf
                const bool some = real && (lsum > 0.f || lsum != lsum);
                const float inv = some ? 1.f / lsum : 0.f;
                const int nrow = min(m.NT, m.T - me.n0) * m.G;    // rows of the output
                if (lse && r < nrow)
                    lse[((size_t)t.b * m.Hq + t.hk * m.G + r - rt * m.G) * m.T + node] =
                        some ? (mx + __log2f(lsum)) * kLn2 : -INFINITY;
                constexpr int CHW = W / 8;            // 16-byte pieces
#pragma unroll(E8 ? D / W : 1)
                for (int h = 0; h < D; h += W) {
                    uint32_t v[W], w[W / 2];
                    if (me.active) sums(h, v);
#pragma unroll
                    for (int e = 0; e < W / 2; ++e)
                        w[e] = some ? pack_bf16x2(__uint_as_float(v[2 * e]) * inv, __uint_as_float(v[2 * e + 1]) * inv) : 0u;
                    auto swz = [](uint32_t i) { return (i & ~7u) | ((i & 7u) ^ ((i >> 3) & 7u)); };
#pragma unroll
                    for (int c = 0; c < CHW; ++c)
                        st_shared_v4(stg + 16u * swz(lane * CHW + c), w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
                    __syncwarp();
#pragma unroll
                    for (int k = 0; k < CHW; ++k) {
                        const int i = lane + 32 * k, rr = q4 * 32 + i / CHW, c = i % CHW;
                        const uint4 y = ld_shared_v4(stg + 16u * swz(i));
                        if (rr < nrow) {
                            const int tt = divide(rr, m.by_g);
                            *reinterpret_cast<uint4*>(o.row(t.b, t.hk * m.G + rr - tt * m.G, me.n0 + tt) + h + 8 * c) = y;
                        }
                    }
                    __syncwarp();
                }
            } else if (me.active) {
                float* to = part + ((long long)(2 * blockIdx.x + (t.t0 == 0 ? 1 : 0)) * m.slots + slot) * kPart<D>;
#pragma unroll(E8 ? D / W : 1)
                for (int h = 0; h < D; h += W) {
                    uint32_t v[W];
                    sums(h, v);
#pragma unroll
                    for (int e = 0; e < W; e += 4)
                        *reinterpret_cast<uint4*>(to + ((h + e) / 4 * 128 + r) * 4) = make_uint4(v[e], v[e + 1], v[e + 2], v[e + 3]);
                }
                to[128 * D + r] = mx;
                to[128 * (D + 1) + r] = lsum;
            }
            tc_fence_before();                        // O is read before the next item's first P V
            if (DUO && me.active) warp_arrive(sy.bar(W_MD), lane);
        }
    } else {
        // ------------------------------------------------------------ 8-bit tiles
        if constexpr (E8) {
            // K: warps 12, 13 (and 6, 7), V: 14, 15 (and 8, 9), every nconv-th 32 rows of a tile each
            const int w = warp >= 12 ? warp - 12 : warp - 6, cw = (w & 1) + (warp >= 12 ? 0 : 2);
            const bool v = w >= 2;
            const int full0 = v ? W_VF : W_KF, empty0 = v ? W_VE : W_KE, raw0 = v ? C::NRK : 0, nr = v ? C::NRV : C::NRK;
            const uint32_t stages = sb + (v ? C::OFF_V : C::OFF_K), raws = sb + C::OFF_RAW + raw0 * C::RAW;
            const float* from = v ? m.vs : m.ks;
            int it = 0, st = 0, ph = 0, rs = 0, rph = 0;
            bool ok = true, drafts = false;
            Line l = line_of(m, st0, lens, n_new);
            Item t;
            bool have = next_item(l, m, st0.pair, lens, n_new, t);
            int j = have ? t.t0 : 0;
            float s[2] = {0.f, 0.f};                  // the rows' scales, a tile ahead
            auto scales = [&]() {
                const Tile x = tile_of(t.r, j);
                if (x.draft) return;
                const long long at = t.b * m.cB + t.hk * m.cH;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int r = 32 * (cw + i * nconv) + lane;
                    if (i * nconv < 4 && r < x.valid) s[i] = __ldg(from + at + (long long)(x.row + r) * m.cS);
                }
            };
            if (have) scales();
            while (have && ok) {
                const Tile x = tile_of(t.r, j);
                const int hk = t.hk, b = t.b;
                const float now[2] = {s[0], s[1]};
                if (++j == t.t1) {
                    have = next_item(l, m, st0.pair, lens, n_new, t);
                    j = have ? t.t0 : 0;
                }
                if (have) scales();
                const uint32_t tile = stages + st * C::TILE;
                if (x.draft) {
                    ok = wait_warp(sy, sy.bar(empty0 + st), (ph & 1) ^ 1, 9, it);
                    if (!ok) break;
                    drafts = true;
                    if (lane == 0) {
                        if (cw == 0) Op::load(tile, v ? &tvn : &tkn, x.row, hk, b, sy.bar(full0 + st));
                        else mbar_arrive(sy.bar(full0 + st));
                    }
                    __syncwarp();
                } else {
                    ok = wait_warp(sy, sy.bar(W_RF + raw0 + rs), rph & 1, 11, it);
                    ok = ok && wait_warp(sy, sy.bar(empty0 + st), (ph & 1) ^ 1, 9, it);
                    if (!ok) break;
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        if (i * nconv < 4) {
                            const int r = 32 * (cw + i * nconv) + lane;
                            widen_row<D>(raws + rs * C::RAW, now[i], r < x.valid, tile, r);
                        }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(sy.bar(full0 + st)), mbar_arrive(sy.bar(W_RE + raw0 + rs));
                    if (++rs == nr) rs = 0, ++rph;
                }
                ++it;
                if (++st == C::NK) st = 0, ++ph;
            }
            // an abort leaves no copy in flight: the last draft tile's gets its time
            if (*sy.abort && drafts && cw == 0) {
                const uint64_t t0 = globaltimer_ns();
                while (globaltimer_ns() - t0 < 1000000ull) {
                }
            }
        }
        __syncwarp();
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, 512);
}

// Adds up what several CTAs have of an item, in the order of its tiles.  A unit is 32 rows (a
// lane each) and 16 features.  JW warps share a unit's partial results, every JW-th each, and
// their sums are added up in the order of the warps: 8 where an item lies in many CTAs, 1
// where it lies in two or three.
constexpr int kJoin = 8;                             // warps of a block
template <int D, int JW>
__global__ void __launch_bounds__(32 * kJoin)
tree_tc_join_kernel(RowOut o, float* __restrict__ lse, const int* __restrict__ n_new, const float* __restrict__ part,
                    const int2* __restrict__ desc, const __grid_constant__ Shape m, int units) {
    constexpr int PER = 4 * (D / 16), PART = kPart<D>;
    __shared__ float sum[JW > 1 ? JW : 1][18][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, jw = JW > 1 ? warp : 0;
    const int unit = JW > 1 ? blockIdx.x : blockIdx.x * kJoin + warp;
    if (unit >= units) return;
    const int x = unit / PER, i = unit % PER;
    const int item = m.slots == 2 ? x >> 1 : x, slot = m.slots == 2 ? x & 1 : 0, r = 32 * (i & 3) + lane, f = i >> 2;
    const int bk = divide(item, m.by_pairs), pair = item - bk * m.pairs, b = bk / m.Hkv, hk = bk - b * m.Hkv, q = 2 * pair + slot;
    const int n = n_new ? min(max(__ldg(n_new + b), 0), m.T) : m.T;
    griddep_wait();
    if (q >= m.ntile || q * m.NT >= n) return;        // no row of it was there: written already
    const int2 d = __ldcg(desc + bk);
    if (d.y < 0) return;
    auto at = [&](int c) { return part + ((long long)(2 * (c * m.pairs + pair) + (c == d.x ? 1 : 0)) * m.slots + slot) * PART; };
    float mx = -INFINITY, l = 0.f, y[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) y[e] = 0.f;
#pragma unroll 4
    for (int c = d.x + jw; c <= d.y; c += JW) mx = fmaxf(mx, __ldcg(at(c) + 128 * D + r));
    const float ref = mx == -INFINITY ? 0.f : mx;
#pragma unroll 2
    for (int c = d.x + jw; c <= d.y; c += JW) {
        const float* p = at(c);
        float4 v[4];
#pragma unroll
        for (int h = 0; h < 4; ++h) v[h] = __ldcg(reinterpret_cast<const float4*>(p) + (4 * f + h) * 128 + r);
        const float w = exp2f(__ldcg(p + 128 * D + r) - ref);
        l = fmaf(__ldcg(p + 128 * (D + 1) + r), w, l);
#pragma unroll
        for (int h = 0; h < 4; ++h) {
            y[4 * h] = fmaf(v[h].x, w, y[4 * h]), y[4 * h + 1] = fmaf(v[h].y, w, y[4 * h + 1]);
            y[4 * h + 2] = fmaf(v[h].z, w, y[4 * h + 2]), y[4 * h + 3] = fmaf(v[h].w, w, y[4 * h + 3]);
        }
    }
    const int rt = divide(r, m.by_g), node = q * m.NT + rt, h = hk * m.G + r - rt * m.G;
    const bool out = rt < m.NT && node < m.T;
    auto finish = [&](const float* z, int n4, uint2* to) {   // 4 n4 features of the row
        const bool some = node < n && l != 0.f;
        const float inv = some ? 1.f / l : 0.f;
        for (int e = 0; e < n4; ++e)
            to[e] = some ? make_uint2(pack_bf16x2(z[4 * e] * inv, z[4 * e + 1] * inv), pack_bf16x2(z[4 * e + 2] * inv, z[4 * e + 3] * inv))
                         : make_uint2(0, 0);
        return some;
    };
    bool some;
    if constexpr (JW == 1) {
        uint2 w[4];
        some = finish(y, 4, w);
        if (out) {
            uint4* to = reinterpret_cast<uint4*>(o.row(b, h, node) + 16 * f);
            to[0] = make_uint4(w[0].x, w[0].y, w[1].x, w[1].y);
            to[1] = make_uint4(w[2].x, w[2].y, w[3].x, w[3].y);
        }
    } else {
#pragma unroll
        for (int e = 0; e < 16; ++e) sum[warp][e][lane] = y[e];
        sum[warp][16][lane] = mx, sum[warp][17][lane] = l;
        __syncthreads();
        if (warp >= 4) return;                        // four features of each row per warp
        mx = -INFINITY, l = 0.f;
#pragma unroll
        for (int w = 0; w < JW; ++w) mx = fmaxf(mx, sum[w][16][lane]);
        const float top = mx == -INFINITY ? 0.f : mx;
        float z[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < JW; ++w) {
            const float by = exp2f(sum[w][16][lane] - top);
            l = fmaf(sum[w][17][lane], by, l);
#pragma unroll
            for (int e = 0; e < 4; ++e) z[e] = fmaf(sum[w][4 * warp + e][lane], by, z[e]);
        }
        uint2 w[1];
        some = finish(z, 1, w);
        if (out) *reinterpret_cast<uint2*>(o.row(b, h, node) + 16 * f + 4 * warp) = w[0];
    }
    if (out && lse && f == 0 && jw == 0) lse[((size_t)b * m.Hq + h) * m.T + node] = some ? (mx + log2f(l)) * kLn2 : -INFINITY;
}

// Items (sequence, key head, pair of row tiles) of a call.
struct Cut {
    int NT, ntile, pairs, slots, ctas;
    long long items;
};
constexpr int kMaxCtas = 160;
Cut cut_of(const TreeArgs& a) {
    Cut c;
    const int G = a.Hq / a.Hkv;
    c.NT = std::min(128 / G, a.T);
    c.ntile = (a.T + c.NT - 1) / c.NT;
    c.pairs = (c.ntile + 1) / 2;
    c.slots = c.ntile > 1 ? 2 : 1;
    c.items = (long long)a.B * a.Hkv * c.pairs;
    // CTAs that can have something to do: at most one per SM, and one per tile
    const long long tiles = ((long long)a.sinks + a.window) / 128 + 2 + (a.T + 127) / 128;
    const long long runs = std::min((long long)std::max(kMaxCtas / c.pairs, 1), c.items / c.pairs * std::min(tiles, (long long)kMaxCtas));
    c.ctas = (int)runs * c.pairs;
    return c;
}

template <int D, bool E8>
int launch(const TreeArgs& a, std::string* err) {
    using C = Cfg<D, E8>;
    using Op = Operand<D>;
    const Cut c = cut_of(a);
    Shape m{};
    m.B = a.B, m.Hq = a.Hq, m.Hkv = a.Hkv, m.G = a.Hq / a.Hkv, m.T = a.T, m.cap = a.cap, m.window = a.window, m.sinks = a.sinks;
    m.NT = c.NT, m.ntile = c.ntile, m.pairs = c.pairs, m.slots = c.slots;
    m.by_pairs = fast_div(m.pairs), m.by_g = fast_div(m.G), m.scale_log2 = a.scale * kLog2e, m.par_stride = a.par_stride;
    m.ks = a.ks, m.vs = a.vs, m.cB = a.cB, m.cH = a.cH, m.cS = a.cS;
    constexpr int PER = 4 * (D / 16);
    if (c.items * c.slots * PER > 0x3fffffffll) {
        *err = "grid too large";
        return PSA_ERR_UNSUPPORTED;
    }
    CUtensorMap tq, tk, tv, tkn, tvn;
    constexpr int CE = E8 ? 1 : 2;                   // bytes of a cached element
    auto cache_map = [&](CUtensorMap* map, const void* base) {
        return encode_4d(map, CE, base, {D, a.cap, a.Hkv, a.B},
                         {a.cap > 1 ? a.sS : 16 / CE, a.Hkv > 1 ? a.sH : 16 / CE, a.B > 1 ? a.sB : 16 / CE},
                         {E8 ? D : Op::W, 128, 1, 1}, err);
    };
    // a dimension of length 1 gets a stride that the encoder takes
    if (!encode_4d(&tq, 2, a.q.base, {D, a.Hq, a.T, a.B}, {a.Hq > 1 ? a.q.sH : D, a.T > 1 ? a.q.sN : D, a.B > 1 ? a.q.sB : D},
                   {Op::W, m.G, m.NT, 1}, err) ||
        !cache_map(&tk, a.k) || !cache_map(&tv, a.v) ||
        !Op::encode(&tkn, a.kn, a.B, a.Hkv, a.T, 128, err) || !Op::encode(&tvn, a.vn, a.B, a.Hkv, a.T, 128, err) ||
        !set_max_dynamic_smem((const void*)tree_tc_kernel<D, E8, false>, C::SMEM, err) ||
        !set_max_dynamic_smem((const void*)tree_tc_kernel<D, E8, !E8>, C::SMEM, err))
        return PSA_ERR_CUDA;
    int sms = 0;
    if (!sm_count(&sms, err)) return PSA_ERR_CUDA;
    float* part = static_cast<float*>(a.workspace);
    int2* desc = reinterpret_cast<int2*>(part + (size_t)2 * c.ctas * c.slots * kPart<D>);
    ProfScope prof(kSlotFwd, a.stream);
    const int grid = std::min(std::max(sms / c.pairs, 1) * c.pairs, c.ctas);
    m.parts = grid / c.pairs;
    (c.slots == 1 ? tree_tc_kernel<D, E8, !E8> : tree_tc_kernel<D, E8, false>)<<<grid, kSoft + (E8 ? kConv : 0), C::SMEM, a.stream>>>(
        tq, tk, tv, tkn, tvn, row_out(a.o), a.lse, a.lens, a.n_new, a.parents, part, desc, m);
    cudaError_t e = cudaGetLastError();
    // an item of a (sequence, key head) lies in about grid / (B Hkv) CTAs
    const int units = (int)(c.items * c.slots * PER);
    if (e == cudaSuccess && grid / c.pairs >= 4ll * a.B * a.Hkv)
        e = launch_beside(tree_tc_join_kernel<D, kJoin>, (unsigned)units, 32 * kJoin, 1, 0, a.stream, row_out(a.o), a.lse, a.n_new,
                          part, desc, m, units);
    else if (e == cudaSuccess)
        e = launch_beside(tree_tc_join_kernel<D, 1>, (unsigned)((units + kJoin - 1) / kJoin), 32 * kJoin, 1, 0, a.stream,
                          row_out(a.o), a.lse, a.n_new, part, desc, m, units);
    if (e == cudaSuccess) return PSA_OK;
    *err = std::string("tree attention launch: ") + cudaGetErrorString(e);
    return PSA_ERR_CUDA;
}
template <bool E8>
int launch_dim(const TreeArgs& a, std::string* err) {
    switch (a.d) {
        case 16: return launch<16, E8>(a, err);
        case 32: return launch<32, E8>(a, err);
        case 64: return launch<64, E8>(a, err);
        default: return launch<128, E8>(a, err);
    }
}

}  // namespace

size_t tree_tc_workspace(const TreeArgs& a) {
    if (a.Hq / a.Hkv > 128) return 0;
    const Cut c = cut_of(a);
    return (size_t)2 * c.ctas * c.slots * 128 * (a.d + 2) * 4 + (size_t)c.items * sizeof(int2);
}
int tree_tc(const TreeArgs& a, std::string* err) {
    return a.cache_dtype == PSA_E4M3 ? launch_dim<true>(a, err) : launch_dim<false>(a, err);
}
int tree_tc_take_error(std::string* err) { return take_error(g_err, "tree attention", err); }

}  // namespace win
}  // namespace psa
