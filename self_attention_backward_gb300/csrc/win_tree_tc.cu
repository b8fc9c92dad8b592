// win_tree_tc.cu -- attention of new tokens (a tree of drafts, a run of tokens) over
// the rolling cache on the tensor cores (tcgen05 / TMEM / TMA), bf16 queries over a bf16
// or an 8-bit cache.
//
// The softmax between the products is win_tc_fwd.cu's: per 128-row tile and 128-key tile
//   S = Q K^T;  m' = max(m, max S c) if that exceeds m by more than 8, else m
//   P = exp2(S c - m) (bf16, over S in TMEM),  l += sum P,  O += P V.
// A row is a (token, query head) of one key head, row = token G + head; a tile has the rows
// of 128 / G tokens (G heads share a key head), fetched by one TMA box over heads and tokens.
// Two tiles ("slots") of a key head go through the same K and V tiles.
//
// Keys.  A sequence's visible slots are one run of memory, or two: the sinks with the ring's
// front, and the rest of the ring.  Each is cut into 128-slot tiles wherever it starts;
// the order of keys does not matter to a softmax.  Then the new keys' tiles, whose columns a
// row sees by its ancestors (one walk up the parents per row).  Slots behind a run's end may
// hold anything: their columns are hidden and their V rows cleared, 0 times NaN is not 0.
//
// Work is split by tiles, not by sequences: the tiles of all (sequence, key head, pair of
// row tiles) items form one line, of which each CTA (one per SM) takes an equal run,
// whatever the lengths are.  An item that lies within a run is written out; of the others
// every CTA leaves its O, m and l in the workspace, and a second kernel adds them up in
// the order of the tiles.
//
// An 8-bit cache's tiles are brought in by four more warps: 16-byte loads, each row
// times its scale to bf16 (exact for the scales that the cache's writes choose), 16-byte
// stores into the operand's swizzled layout.  Draft tiles come by TMA as they are.
//
// 320 (448) threads: warp 0 producer (lane 0 K, lane 1 V, lane 2 Q), warp 1 MMA issuer and
// TMEM owner, warps 2-5 and 6-9 the softmax of the two slots, warps 10-13 the 8-bit tiles.
// All waits are bounded (tc_sync.cuh).
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

constexpr int kSoft = 320, kConv = 4;             // threads without the 8-bit tiles' warps; those warps

template <int D>
struct Cfg {
    using O = Operand<D>;
    static constexpr int TILE = O::TILE;
    static constexpr int NST = D == 128 ? 2 : 4;     // K stages, V stages
    static constexpr int OFF_Q = 0;                  // two slots
    static constexpr int OFF_K = 2 * TILE;
    static constexpr int OFF_V = OFF_K + NST * TILE;
    static constexpr int OFF_EPI = OFF_V + NST * TILE;   // 2 KB per softmax warp
    static constexpr int OFF_BAR = OFF_EPI + 8 * 2048;
    static constexpr int OFF_MISC = OFF_BAR + 256;
    static constexpr int USED = OFF_MISC + 256 + 1024;
    static constexpr int SMEM = USED > 118784 ? USED : 118784;   // one CTA per SM: each takes all of TMEM
    static constexpr uint32_t C_S = 0, C_O = 256;    // S of slot s at 128 s, O at 256 + 128 s
    static constexpr int PART = 128 * (D + 2);       // floats of a slot's partial result: O [D / 4][128][4], m, l
};

// barriers (slot s or stage s behind each)
enum { W_QF = 0, W_QE = 2, W_SF = 4, W_PF = 6, W_OF = 8, W_KF = 10, W_KE = 14, W_VF = 18, W_VE = 22, W_DRAIN = 26 };

struct Shape {
    int B, Hq, Hkv, G, T, cap, window, sinks;
    int NT, ntile, pairs, slots;      // tokens per row tile, row tiles and pairs of them per key head; slots in use
    int grain;                        // tiles that a CTA takes at least
    FastDiv by_pairs, by_g;
    float scale_log2;
    long long par_stride;
    // 8-bit caches
    const uint8_t* k;
    const uint8_t* v;
    const float* ks;
    const float* vs;
    long long sB, sH, sS, cB, cH, cS;
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
// A CTA's run of tiles, item by item.
struct Line {
    long long pos, end, base;     // next tile; end; first tile of sequence b
    int b;
    Runs r;
};
struct Item {
    int b, hk, pair, t0, t1;      // tiles t0 .. t1 - 1 of it
    Runs r;
    Slot s0, s1;
    __device__ __forceinline__ Slot slot(int i) const { return i ? s1 : s0; }
    __device__ __forceinline__ bool whole() const { return t0 == 0 && t1 == r.total; }
};
struct Start {                    // found once per CTA
    long long pos, end, base, all;
    int b, ctas;
};
__device__ __forceinline__ Line line_of(const Shape& m, const Start& s, const int* lens, const int* n_new) {
    Line l{s.pos, s.end, s.base, s.b, {}};
    if (l.pos < l.end) l.r = load_runs(m, lens, n_new, l.b);
    return l;
}
__device__ __forceinline__ bool next_item(Line& l, const Shape& m, const int* lens, const int* n_new, Item& t) {
    if (l.pos >= l.end) return false;
    while (l.pos >= l.base + (long long)l.r.total * m.Hkv * m.pairs) {
        l.base += (long long)l.r.total * m.Hkv * m.pairs;
        l.r = load_runs(m, lens, n_new, ++l.b);
    }
    const long long rel = l.pos - l.base;
    const int item = (int)(rel / l.r.total);
    t.b = l.b, t.r = l.r;
    t.t0 = (int)(rel - (long long)item * l.r.total);
    t.t1 = (int)min((long long)l.r.total, t.t0 + (l.end - l.pos));
    l.pos += t.t1 - t.t0;
    t.hk = divide(item, m.by_pairs), t.pair = item - t.hk * m.pairs;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        Slot c;
        c.q = 2 * t.pair + s;
        c.n0 = c.q * m.NT;
        c.exists = c.q < m.ntile;
        c.active = c.exists && c.n0 < t.r.n;
        (s ? t.s1 : t.s0) = c;
    }
    return true;
}

// This CTA's run: the tiles of all sequences are added up, and the sequence that its first
// tile lies in is looked for (each thread has a few neighbouring sequences).
template <int THREADS>
__device__ __forceinline__ void find_start(const Shape& m, const int* lens, const int* n_new, Start* out, long long* sums) {
    const int per = (m.B + THREADS - 1) / THREADS, b0 = min((int)threadIdx.x * per, m.B), b1 = min(b0 + per, m.B);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    long long mine = 0;
    for (int b = b0; b < b1; ++b) mine += (long long)load_runs(m, lens, n_new, b).total * m.Hkv * m.pairs;
    long long upto = mine;
#pragma unroll
    for (int i = 1; i < 32; i <<= 1) {
        const long long x = __shfl_up_sync(0xffffffffu, upto, i);
        if (lane >= i) upto += x;
    }
    if (lane == 31) sums[warp] = upto;
    __syncthreads();
    long long all = 0, before = upto - mine;
    for (int w = 0; w < THREADS / 32; ++w) {
        if (w < warp) before += sums[w];
        all += sums[w];
    }
    const int ctas = (int)min((long long)gridDim.x, (all + m.grain - 1) / m.grain);
    const long long pos = (int)blockIdx.x < ctas ? blockIdx.x * all / ctas : all;
    const long long end = (int)blockIdx.x < ctas ? (blockIdx.x + 1) * all / ctas : all;
    if (pos >= end) {
        if (threadIdx.x == 0) *out = Start{0, 0, 0, all, 0, ctas};
    } else if (mine > 0 && pos >= before && pos < before + mine) {
        int b = b0;
        long long base = before;
        for (;;) {
            const long long n = (long long)load_runs(m, lens, n_new, b).total * m.Hkv * m.pairs;
            if (pos < base + n) break;
            base += n, ++b;
        }
        *out = Start{pos, end, base, all, b, ctas};
    }
}

// Number of ancestors of a node.
__device__ __forceinline__ int depth_of(const int* par, int node) {
    if (!par) return node;
    int d = 0;
    for (int t = node;;) {
        const int p = __ldg(par + t);
        if (p < 0 || p >= t) return d;
        t = p, ++d;
    }
}
// Which of the drafts j0 .. j0 + 127 a node sees: itself and its ancestors, those within the
// window or below the sinks.
__device__ __forceinline__ void drafts_seen(const int* par, int node, int depth, int j0, int L, const Shape& m, uint32_t (&see)[4]) {
    if (!par) {
        // sinks - L - j0: drafts whose position is below the sinks
        const int snk = (int)max((long long)m.sinks - L - j0, -1ll);
#pragma unroll
        for (int g = 0; g < 4; ++g) see[g] = col_mask(node - m.window + 1 - j0, node - j0, min(snk, node - j0 + 1), 32 * g);
        return;
    }
#pragma unroll
    for (int g = 0; g < 4; ++g) see[g] = 0;
    for (int t = node, k = 0;; ++k) {
        if ((unsigned)(t - j0) < 128u && (k < m.window || (long long)L + depth - k < m.sinks)) {
#pragma unroll
            for (int g = 0; g < 4; ++g)
                if ((t - j0) >> 5 == g) see[g] |= 1u << (t & 31);
        }
        const int p = __ldg(par + t);
        if (p < 0 || p >= t) return;
        t = p;
    }
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
__device__ __forceinline__ void widen16(const uint4& u, float s, uint32_t (&w)[8]) {
    const uint32_t x[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        uint32_t h;
        const uint16_t two = (uint16_t)(x[i / 2] >> (16 * (i % 2)));
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(two));
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
        w[i] = pack_bf16x2(f.x * s, f.y * s);
    }
}
// A thread's share of a tile: 16-byte pieces p of rows r, a row's pieces by neighbouring
// lanes.  N pieces each; the tensor-core layout of row r is Operand<D>'s.
template <int D>
struct Bytes {
    static constexpr int CH = D / 16, N = CH * 128 / (32 * kConv);   // pieces per row, per thread
    uint4 u[N];
    float s[N];
    __device__ __forceinline__ void load(const uint8_t* base, const float* scale, long long sS, long long cS, const Tile& t, int ct) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int x = ct + 32 * kConv * i, r = x / CH;
            u[i] = make_uint4(0, 0, 0, 0);
            s[i] = 0.f;
            if (r < t.valid) {
                const long long slot = t.row + r;
                u[i] = __ldg(reinterpret_cast<const uint4*>(base + slot * sS) + x % CH);
                s[i] = __ldg(scale + slot * cS);
            }
        }
    }
    __device__ __forceinline__ void store(uint32_t tile, int ct) const {
        using O = Operand<D>;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int x = ct + 32 * kConv * i, r = x / CH, f = x % CH * 16;      // 16 features: two 16-byte chunks
            uint32_t w[8];
            widen16(u[i], s[i], w);
            constexpr int C = O::ROWB / 16;                                      // chunks per panel row: 8, 4 or 2
            const uint32_t row = tile + f / O::W * O::PANEL + r * O::ROWB;
            const int ch = f % O::W / 8, sw = (r / (8 / C)) & (C - 1);
            const bool odd = f / O::W;                                           // the other panel's lanes take other banks
            st_shared_v4(row + 16 * ((ch + odd) ^ sw), odd ? w[4] : w[0], odd ? w[5] : w[1], odd ? w[6] : w[2], odd ? w[7] : w[3]);
            st_shared_v4(row + 16 * ((ch + !odd) ^ sw), odd ? w[0] : w[4], odd ? w[1] : w[5], odd ? w[2] : w[6], odd ? w[3] : w[7]);
        }
    }
};

template <int D, bool E8>
__global__ void __launch_bounds__(kSoft + (E8 ? 32 * kConv : 0), 1)
tree_tc_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
               const __grid_constant__ CUtensorMap tkn, const __grid_constant__ CUtensorMap tvn, RowOut o, float* __restrict__ lse,
               const int* __restrict__ lens, const int* __restrict__ n_new, const int* __restrict__ parents,
               float* __restrict__ part, int2* __restrict__ desc, const __grid_constant__ Shape m) {
    using C = Cfg<D>;
    using Op = Operand<D>;
    constexpr int THREADS = kSoft + (E8 ? 32 * kConv : 0);
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sb = smem_u32(smem);
    Sync sy{sb + C::OFF_BAR, reinterpret_cast<volatile int*>(smem + C::OFF_MISC), &g_err};
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC + 16);
    Start* start = reinterpret_cast<Start*>(smem + C::OFF_MISC + 32);
    long long* sums = reinterpret_cast<long long*>(smem + C::OFF_MISC + 96);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int s = 0; s < 2; ++s) {
            mbar_init(sy.bar(W_QF + s), 1);
            mbar_init(sy.bar(W_QE + s), 1);
            mbar_init(sy.bar(W_SF + s), 1);
            mbar_init(sy.bar(W_PF + s), 4);
            mbar_init(sy.bar(W_OF + s), 1);
        }
        for (int s = 0; s < C::NST; ++s) {
            for (int x : {W_KF, W_VF}) mbar_init(sy.bar(x + s), E8 ? kConv : 1);
            for (int x : {W_KE, W_VE}) mbar_init(sy.bar(x + s), 1);
        }
        mbar_init(sy.bar(W_DRAIN), 1);
        *sy.abort = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tq);
        if (!E8) tma_prefetch_desc(&tk), tma_prefetch_desc(&tv);
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

    if (warp == 0) {
        // ------------------------------------------------------------ producer
        if (lane < 2 && !E8) {                       // K tiles (lane 0), V tiles (lane 1)
            const CUtensorMap *map = lane ? &tv : &tk, *mapn = lane ? &tvn : &tkn;
            const int full = lane ? W_VF : W_KF, empty = lane ? W_VE : W_KE;
            const uint32_t base = sb + (lane ? C::OFF_V : C::OFF_K);
            int it = 0;
            bool ok = true;
            Line l = line_of(m, st0, lens, n_new);
            Item t;
            while (ok && next_item(l, m, lens, n_new, t))
                for (int j = t.t0; j < t.t1 && ok; ++j, ++it) {
                    const int st = it % C::NST;
                    ok = wait_one(sy, sy.bar(empty + st), ((it / C::NST) & 1) ^ 1, 0, it);
                    if (!ok) break;
                    const Tile x = tile_of(t.r, j);
                    Op::load(base + st * C::TILE, x.draft ? mapn : map, x.row, t.hk, t.b, sy.bar(full + st));
                }
            if (*sy.abort)                           // wait for the last copy into every stage
                for (int st = 0; st < C::NST; ++st) {
                    const int n = (it - st + C::NST - 1) / C::NST;   // copies made into stage st
                    if (n > 0) wait_drain(sy.bar(full + st), (n - 1) & 1);
                }
        } else if (lane == 2) {                      // Q tiles
            int n[2] = {0, 0};
            bool ok = true;
            Line l = line_of(m, st0, lens, n_new);
            Item t;
            while (ok && next_item(l, m, lens, n_new, t)) {
#pragma unroll
                for (int s = 0; s < 2; ++s) {
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
            const uint64_t dk = Op::kmajor(sb + C::OFF_K + (jt % C::NST) * C::TILE);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
                mma_ss(tmem + C::C_S + 128u * s, dq + Op::kstep(kk), dk + Op::kstep(kk), id, kk);
            commit(sy.bar(W_SF + s));
            if (j == t.t1 - 1) commit(sy.bar(W_QE + s));
        };
        Line l = line_of(m, st0, lens, n_new);
        Item t;
        // the next item (an item with no token there is a tile that is only read)
        bool have = next_item(l, m, lens, n_new, t);
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
                const int jt = it + j, vs = jt % C::NST;
                const bool end = j == n - 1;
                if (end) have = next_item(l, m, lens, n_new, t);   // t: the item whose first tile comes next
                const int k2 = 2 * tile_of(cur.r, cur.t0 + j).groups();
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
                if (!end || have) commit(sy.bar(W_KE + (jt + 1) % C::NST));
            }
            it += n;
        }
        if (!ok) {                                    // let what was issued finish before TMEM is freed
            commit(sy.bar(W_DRAIN));
            wait_drain(sy.bar(W_DRAIN), 0);
        }
        __syncwarp();
    } else if (warp < 10) {
        // ------------------------------------------------------------ softmax
        const int slot = (warp - 2) >> 2, q4 = warp & 3;
        const int r = q4 * 32 + lane;
        const uint32_t trow = tmem + ((uint32_t)(q4 * 32) << 16);
        const uint32_t tS = trow + C::C_S + 128u * slot, tO = trow + C::C_O + 128u * slot;
        const uint32_t stg = sb + C::OFF_EPI + 2048u * (warp - 2);
        const int rt = divide(r, m.by_g);             // the row's token of its tile
        int it = 0, nit = 0;                          // tile numbers; items done by this slot
        uint32_t sf = 0;
        bool ok = true;
        Line l = line_of(m, st0, lens, n_new);
        Item t;
        while (ok && next_item(l, m, lens, n_new, t)) {
            const Slot me = t.slot(slot);
            // an item that goes on in another CTA: which ones have it
            if (t.t0 == 0 && warp == 2 && lane == 0) {
                const long long p0 = l.pos - (t.t1 - t.t0), p1 = p0 + t.r.total - 1;
                const int c1 = (int)(((p1 + 1) * st0.ctas - 1) / st0.all);
                desc[((long long)t.b * m.Hkv + t.hk) * m.pairs + t.pair] = make_int2(blockIdx.x, t.whole() ? -1 : c1);
            }
            const int n = t.t1 - t.t0;
            if (!me.exists) {
                it += n;
                continue;
            }
            const int node = me.n0 + rt;
            const bool real = rt < m.NT && node < t.r.n;
            const int* par = parents ? parents + t.b * m.par_stride : nullptr;
            float mx = -INFINITY, lsum = 0.f;
            if (me.active) {
                // a row sees slot s of the ring when s > low - off; rows differ by their depths
                const int top = t.r.nv - m.window + t.r.n - 1;
                int depth = 0;
                if (real && (top >= m.sinks || t.t1 > t.r.n1 + t.r.n2)) depth = depth_of(par, node);
                const int low = t.r.nv - m.window + depth;
                const bool zeroes = slot == 0 || !t.s0.active;
                for (int j = t.t0; j < t.t1; ++j) {
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
                    if (full)
                        softmax_tile<D>(tS, tO, j == t.t0, m.scale_log2, mx, lsum);
                    else
                        softmax_masked<D>(tS, tO, j == t.t0, m.scale_log2, mx, lsum, nc, see);
                    // V rows that are not there hold anything: the tile's first slot clears them (an
                    // 8-bit tile has zeros there)
                    if (zeroes && x.valid < 128 && (!E8 || x.draft)) {
                        ok = wait_warp(sy, sy.bar(W_VF + jt % C::NST), (jt / C::NST) & 1, 7, jt);
                        if (!ok) break;
                        if (r >= x.valid) Op::clear_row(sb + C::OFF_V + (jt % C::NST) * C::TILE, r);
                        fence_proxy_async_smem();
                    }
                    tc_fence_before();
                    warp_arrive(sy.bar(W_PF + slot), lane);
                }
                if (ok) ok = wait_warp(sy, sy.bar(W_OF + slot), nit++ & 1, 8, it);
                if (!ok) break;
                tc_fence_after();
            }
            it += n;
            if (t.whole() || (!me.active && t.t0 == 0)) {
                // rows that are not there come out as 0 and -inf
                const bool some = real && (lsum > 0.f || lsum != lsum);
                const float inv = some ? 1.f / lsum : 0.f;
                const int nrow = min(m.NT, m.T - me.n0) * m.G;    // rows of the output
                if (lse && r < nrow)
                    lse[((size_t)t.b * m.Hq + t.hk * m.G + r - rt * m.G) * m.T + node] =
                        some ? (mx + __log2f(lsum)) * kLn2 : -INFINITY;
                constexpr int W = D < 32 ? D : 32, CHW = W / 8;   // features per round, 16-byte pieces
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
                float* to = part + ((long long)(2 * blockIdx.x + (t.t0 == 0 ? 1 : 0)) * m.slots + slot) * C::PART;
                constexpr int W = D < 32 ? D : 32;
#pragma unroll
                for (int h = 0; h < D; h += W) {
                    uint32_t v[W];
                    tmem_ld_row<W>(tO + h, v);
                    tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < W; e += 4)
                        *reinterpret_cast<uint4*>(to + ((h + e) / 4 * 128 + r) * 4) = make_uint4(v[e], v[e + 1], v[e + 2], v[e + 3]);
                }
                to[128 * D + r] = mx;
                to[128 * (D + 1) + r] = lsum;
            }
            tc_fence_before();                        // O is read before the next item's first P V
        }
    } else {
        // ------------------------------------------------------------ 8-bit tiles
        if constexpr (E8) {
            const int ct = threadIdx.x - kSoft, cw = warp - 10;
            int it = 0;
            bool ok = true;
            Line l = line_of(m, st0, lens, n_new);
            Item t;
            Bytes<D> kb, vb;
            bool have = next_item(l, m, lens, n_new, t);
            int j = have ? t.t0 : 0;
            auto fetch = [&]() {
                const Tile x = tile_of(t.r, j);
                if (x.draft) return;
                kb.load(m.k + t.b * m.sB + t.hk * m.sH, m.ks + t.b * m.cB + t.hk * m.cH, m.sS, m.cS, x, ct);
                vb.load(m.v + t.b * m.sB + t.hk * m.sH, m.vs + t.b * m.cB + t.hk * m.cH, m.sS, m.cS, x, ct);
            };
            if (have) fetch();
            while (have && ok) {
                const int st = it % C::NST;
                const Tile x = tile_of(t.r, j);
                const int hk = t.hk, b = t.b;
                ok = wait_warp(sy, sy.bar(W_KE + st), ((it / C::NST) & 1) ^ 1, 9, it);
                if (!ok) break;
                if (x.draft) {
                    if (cw == 0) {
                        if (lane == 0) Op::load(sb + C::OFF_K + st * C::TILE, &tkn, x.row, hk, b, sy.bar(W_KF + st));
                    } else if (lane == 0) {
                        mbar_arrive(sy.bar(W_KF + st));
                    }
                    __syncwarp();
                } else {
                    kb.store(sb + C::OFF_K + st * C::TILE, ct);
                    fence_proxy_async_smem();
                    warp_arrive(sy.bar(W_KF + st), lane);
                }
                ok = wait_warp(sy, sy.bar(W_VE + st), ((it / C::NST) & 1) ^ 1, 10, it);
                if (!ok) break;
                if (x.draft) {
                    if (cw == 0) {
                        if (lane == 0) Op::load(sb + C::OFF_V + st * C::TILE, &tvn, x.row, hk, b, sy.bar(W_VF + st));
                    } else if (lane == 0) {
                        mbar_arrive(sy.bar(W_VF + st));
                    }
                    __syncwarp();
                } else {
                    vb.store(sb + C::OFF_V + st * C::TILE, ct);
                    fence_proxy_async_smem();
                    warp_arrive(sy.bar(W_VF + st), lane);
                }
                ++it;
                if (++j == t.t1) {
                    have = next_item(l, m, lens, n_new, t);
                    j = have ? t.t0 : 0;
                }
                if (have) fetch();
            }
            // after an abort no copy may be in flight; a draft tile's is waited for through its
            // barrier, which another warp may not have arrived on any more: give the copy its time
            if (*sy.abort && cw == 0) {
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

// Adds up what several CTAs have of an item.  Block: item, slot, a part of its rows and features;
// a thread has 8 features of a row.
template <int D>
__global__ void __launch_bounds__(256)
tree_tc_join_kernel(RowOut o, float* __restrict__ lse, const int* __restrict__ n_new, const float* __restrict__ part,
                    const int2* __restrict__ desc, const __grid_constant__ Shape m) {
    constexpr int PER = 128 * (D / 8) / 256, PART = Cfg<D>::PART;
    const int x = blockIdx.x / PER, i = blockIdx.x % PER * 256 + threadIdx.x;
    const int item = m.slots == 2 ? x >> 1 : x, slot = m.slots == 2 ? x & 1 : 0, r = i & 127, f = i >> 7;   // features 8 f ..
    const int bk = divide(item, m.by_pairs), b = bk / m.Hkv, hk = bk - b * m.Hkv, q = 2 * (item - bk * m.pairs) + slot;
    const int rt = divide(r, m.by_g), node = q * m.NT + rt, n = n_new ? min(max(__ldg(n_new + b), 0), m.T) : m.T;
    griddep_wait();
    if (q >= m.ntile || q * m.NT >= n) return;        // no row of it was there: written already
    const int2 d = __ldcg(desc + item);
    if (d.y < 0 || rt >= m.NT || node >= m.T) return;
    auto at = [&](int c) { return part + ((long long)(2 * c + (c == d.x ? 1 : 0)) * m.slots + slot) * PART; };
    float mx = -INFINITY, l = 0.f, y[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int c = d.x; c <= d.y; ++c) mx = fmaxf(mx, __ldcg(at(c) + 128 * D + r));
    const float ref = mx == -INFINITY ? 0.f : mx;
#pragma unroll 4
    for (int c = d.x; c <= d.y; ++c) {
        const float* p = at(c);
        const float w = exp2f(__ldcg(p + 128 * D + r) - ref);
        l = fmaf(__ldcg(p + 128 * (D + 1) + r), w, l);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float4 v = __ldcg(reinterpret_cast<const float4*>(p) + (2 * f + h) * 128 + r);
            y[4 * h] = fmaf(v.x, w, y[4 * h]), y[4 * h + 1] = fmaf(v.y, w, y[4 * h + 1]);
            y[4 * h + 2] = fmaf(v.z, w, y[4 * h + 2]), y[4 * h + 3] = fmaf(v.w, w, y[4 * h + 3]);
        }
    }
    const bool some = node < n && l != 0.f;
    const int h = hk * m.G + r - rt * m.G;
    if (lse && f == 0) lse[((size_t)b * m.Hq + h) * m.T + node] = some ? (mx + log2f(l)) * kLn2 : -INFINITY;
    const float inv = some ? 1.f / l : 0.f;
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = some ? pack_bf16x2(y[2 * e] * inv, y[2 * e + 1] * inv) : 0u;
    *reinterpret_cast<uint4*>(o.row(b, h, node) + 8 * f) = make_uint4(w[0], w[1], w[2], w[3]);
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
    c.ctas = (int)std::min((long long)kMaxCtas, c.items * std::min(tiles, (long long)kMaxCtas));
    return c;
}

template <int D, bool E8>
int launch(const TreeArgs& a, std::string* err) {
    using C = Cfg<D>;
    using Op = Operand<D>;
    const Cut c = cut_of(a);
    Shape m{};
    m.B = a.B, m.Hq = a.Hq, m.Hkv = a.Hkv, m.G = a.Hq / a.Hkv, m.T = a.T, m.cap = a.cap, m.window = a.window, m.sinks = a.sinks;
    m.NT = c.NT, m.ntile = c.ntile, m.pairs = c.pairs, m.slots = c.slots, m.grain = 1;
    m.by_pairs = fast_div(m.pairs), m.by_g = fast_div(m.G), m.scale_log2 = a.scale * kLog2e, m.par_stride = a.par_stride;
    m.k = static_cast<const uint8_t*>(a.k), m.v = static_cast<const uint8_t*>(a.v), m.ks = a.ks, m.vs = a.vs;
    m.sB = a.sB, m.sH = a.sH, m.sS = a.sS, m.cB = a.cB, m.cH = a.cH, m.cS = a.cS;
    constexpr int PER = 128 * (D / 8) / 256;
    if (c.items * c.slots * PER > 0x3fffffffll) {
        *err = "grid too large";
        return PSA_ERR_UNSUPPORTED;
    }
    const View kc{a.k, a.sB, a.sH, a.sS, 1}, vc{a.v, a.sB, a.sH, a.sS, 1};
    CUtensorMap tq, tk{}, tv{}, tkn, tvn;
    // a dimension of length 1 gets a stride that the encoder takes
    if (!encode_4d(&tq, 2, a.q.base, {D, a.Hq, a.T, a.B}, {a.Hq > 1 ? a.q.sH : D, a.T > 1 ? a.q.sN : D, a.B > 1 ? a.q.sB : D},
                   {Op::W, m.G, m.NT, 1}, err) ||
        (!E8 && (!Op::encode(&tk, kc, a.B, a.Hkv, a.cap, 128, err) || !Op::encode(&tv, vc, a.B, a.Hkv, a.cap, 128, err))) ||
        !Op::encode(&tkn, a.kn, a.B, a.Hkv, a.T, 128, err) || !Op::encode(&tvn, a.vn, a.B, a.Hkv, a.T, 128, err) ||
        !set_max_dynamic_smem((const void*)tree_tc_kernel<D, E8>, C::SMEM, err))
        return PSA_ERR_CUDA;
    int sms = 0;
    if (!sm_count(&sms, err)) return PSA_ERR_CUDA;
    float* part = static_cast<float*>(a.workspace);
    int2* desc = reinterpret_cast<int2*>(part + (size_t)2 * c.ctas * c.slots * C::PART);
    ProfScope prof(kSlotFwd, a.stream);
    tree_tc_kernel<D, E8><<<std::min(sms, c.ctas), kSoft + (E8 ? 32 * kConv : 0), C::SMEM, a.stream>>>(
        tq, tk, tv, tkn, tvn, row_out(a.o), a.lse, a.lens, a.n_new, a.parents, part, desc, m);
    cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess)
        e = launch_beside(tree_tc_join_kernel<D>, (unsigned)(c.items * c.slots * PER), 256, 1, 0, a.stream, row_out(a.o), a.lse, a.n_new,
                          part, desc, m);
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
