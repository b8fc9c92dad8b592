// win_decode.cu -- attention of one query row per sequence over the rolling
// key/value cache.
//
//   s_x = c q.k_x (log2 units), O = sum_x exp2(s_x - m) v_x / sum_x exp2(s_x - m)
// over the visible positions x = 0 .. nv-1 in slot order of the sinks, then the
// window (a softmax does not care about the order).
//
// Bound by memory: every visible key and value is read once for all the query
// heads of its key head.  A block of four warps takes a run of keys of one (sequence,
// key head, up to HG query heads); each warp keeps kStages tiles of 16 keys in
// flight in shared memory of its own (cp.async, no block-wide waits), with an
// online softmax.  bf16: both products on mma.sync m16n8k16, the heads as its 16
// rows -- at 16 rows a tcgen05 tile of 128 would be seven eighths empty, and the
// tensor pipe is idle most of the time anyhow.  fp32: FFMA.  P is rounded to bf16
// for its product (the operand type), its sum is not.
//
// The runs of one group are joined in a fixed order.  Up to 8: one cluster, whose
// blocks read each other's results through distributed shared memory, so that a
// small call is a single launch.  More (long windows with few sequences): partial
// results in the workspace and a second kernel.
//
// 64 sequences, 32 / 8 heads, window 4096, d=128 in bf16, 1.08 GB: 164 us, 6.6 TB/s (0.97 of
// the measured copy rate).  One sequence, 16 / 4 heads, window 1024: 6.6 us, a launch and
// the chain of loads and joins.  In fp32 651 us (3.3 TB/s) and 13.6: a block's tiles
// fill 207 KB there, one block an SM and one warp a scheduler, whose latencies nothing covers
// (issue 27%, FMA 16%, DRAM 25% with 16 sequences).
#include <cuda_bf16.h>

#include <algorithm>
#include <string>

#include "common.cuh"
#include "tc_ptx.cuh"
#include "tc_tmap.h"
#include "win_internal.h"

namespace psa {
namespace win {
namespace {

constexpr int kWarps = 4, kT = 32 * kWarps, kKeys = 16, kStages = 3;
constexpr int kCluster = 8;

template <typename T>
constexpr int HG = sizeof(T) == 2 ? 16 : 8;      // query heads per block

struct P {
    const void* k;
    const void* v;
    long long sB, sH, sS;
    View q, o;
    float* lse;
    const int* lens;
    float* part;                                  // more than kCluster splits: [groups][splits][HG][d + 2]
    int Hq, Hkv, G, hgroups, cap, window, sinks, splits, vec;
    float c;
};

template <typename T, int D>
struct Cfg {
    static constexpr int CH = D * (int)sizeof(T) / 16;             // 16-byte chunks per row
    static constexpr int TILE = kKeys * D * (int)sizeof(T);        // one K or V tile
    static constexpr int WARP = kStages * 2 * TILE;
    static constexpr int PIPE = kWarps * WARP;
    static constexpr int OUT = kWarps * HG<T> * (D + 2) * 4;       // the warps' results, over the tiles
    static constexpr int MAIN = PIPE > OUT ? PIPE : OUT;
    static constexpr int RES = HG<T> * (D + 2) * 4;                // the block's result
    static constexpr int QS = sizeof(T) == 4 ? HG<T> * D * 4 + kWarps * HG<T> * kKeys * 4 : 0;
    static constexpr int SMEM = MAIN + RES + QS;
    // chunk c of row r: rows of 128 bytes and more are spread over the banks by their
    // number, shorter rows by that of their 128-byte line
    static __device__ __forceinline__ int at(int r, int ch) {
        return 16 * (CH >= 8 ? r * CH + (ch ^ (r & 7)) : r * CH + (ch ^ ((r / (8 / CH)) & (CH - 1))));
    }
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool full) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(full ? 16 : 0) : "memory");
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
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
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
__device__ __forceinline__ Slots load_slots(const P& a, int b) {
    Slots s;
    const int L = max(__ldg(a.lens + b), 0);
    s.sinks = a.sinks;
    s.ring = a.cap - a.sinks;
    s.nv = min(L, a.sinks + a.window);            // <= capacity
    s.r0 = (L - s.nv) % s.ring;                   // the window's first position, p - sinks = L - nv
    return s;
}

// Rows [x0, x0 + 16) of K and V to a stage; rows past x1 are zero.
template <typename T, int D>
__device__ __forceinline__ void load_rows(const P& a, const Slots& s, long long head, uint32_t ks, uint8_t* ksp, int x0, int x1,
                                          int lane) {
    using C = Cfg<T, D>;
    const T *K = static_cast<const T*>(a.k) + head, *V = static_cast<const T*>(a.v) + head;
    if (a.vec) {
#pragma unroll
        for (int i = lane; i < kKeys * C::CH; i += 32) {
            const int r = i / C::CH, ch = i % C::CH, x = x0 + r;
            const bool in = x < x1;
            const long long g = (long long)s.of(in ? x : x0) * a.sS + ch * (16 / (int)sizeof(T));
            const uint32_t to = ks + C::at(r, ch);
            cp_async16(to, K + g, in);
            cp_async16(to + C::TILE, V + g, in);
        }
    } else {                                      // rows that are not 16-byte aligned: element by element
        constexpr int E = 16 / (int)sizeof(T);
        for (int i = lane; i < kKeys * D; i += 32) {
            const int r = i / D, e = i % D, x = x0 + r;
            T kv = from_f32<T>(0.f), vv = kv;
            if (x < x1) {
                const long long g = (long long)s.of(x) * a.sS + e;
                kv = K[g], vv = V[g];
            }
            T* to = reinterpret_cast<T*>(ksp + C::at(r, e / E)) + e % E;
            to[0] = kv;
            to[C::TILE / (int)sizeof(T)] = vv;
        }
    }
}

// A block's or warp's result: O [HG][D] unnormalised, m and l [HG] behind it.
template <typename T, int D>
struct Res {
    float* p;
    __device__ __forceinline__ float* o(int h) const { return p + h * D; }
    __device__ __forceinline__ float& m(int h) const { return p[HG<T> * D + h]; }
    __device__ __forceinline__ float& l(int h) const { return p[HG<T> * (D + 1) + h]; }
};

// bf16: heads are the 16 rows of mma.sync.
template <int D>
struct WarpBf16 {
    uint32_t q[D / 16][4];
    float o[D / 8][4], m[2], l[2];

    __device__ __forceinline__ void init(const P& a, const __nv_bfloat16* qh, int nh, int lane) {
        const int g = lane >> 2, t = lane & 3;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int h = g + 8 * (i & 1), k = 16 * kk + 2 * t + 8 * (i >> 1);
                uint32_t x = 0;
                if (h < nh) {
                    const uint16_t* p = reinterpret_cast<const uint16_t*>(qh) + h * a.q.sH;
                    x = (uint32_t)p[k * a.q.sJ] | ((uint32_t)p[(k + 1) * a.q.sJ] << 16);
                }
                q[kk][i] = x;
            }
#pragma unroll
        for (int n = 0; n < D / 8; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[n][i] = 0.f;
        m[0] = m[1] = -INFINITY;
        l[0] = l[1] = 0.f;
    }
    __device__ __forceinline__ void step(uint32_t ks, int nk, float c, int lane) {
        using C = Cfg<__nv_bfloat16, D>;
        const int t = lane & 3;
        float s[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
        const int kr = (lane & 7) + ((lane >> 4) << 3), kc = (lane >> 3) & 1;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
            uint32_t b[4];
            ldsm_x4(b, ks + C::at(kr, 2 * kk + kc));
            mma16816(s[0], q[kk], b[0], b[1]);
            mma16816(s[1], q[kk], b[2], b[3]);
        }
        float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                s[n][i] = 8 * n + 2 * t + (i & 1) < nk ? s[n][i] * c : -INFINITY;
                mx[i >> 1] = fmaxf(mx[i >> 1], s[n][i]);
            }
        bool move = false;
        float al[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 1));
            mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 2));
            // a stale maximum stays while the new one is at most 2^8 larger
            const bool mv = mx[i] > m[i] + 8.f;
            al[i] = mv ? ex2(m[i] - mx[i]) : 1.f;
            if (mv) m[i] = mx[i];
            move |= mv;
            l[i] *= al[i];
        }
        if (__any_sync(0xffffffffu, move)) {
#pragma unroll
            for (int n = 0; n < D / 8; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[n][i] *= al[i >> 1];
        }
        const float ref[2] = {m[0] == -INFINITY ? 0.f : m[0], m[1] == -INFINITY ? 0.f : m[1]};
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                s[n][i] = ex2(s[n][i] - ref[i >> 1]);
                l[i >> 1] += s[n][i];
            }
        const uint32_t p[4] = {tc::pack_bf16x2(s[0][0], s[0][1]), tc::pack_bf16x2(s[0][2], s[0][3]),
                               tc::pack_bf16x2(s[1][0], s[1][1]), tc::pack_bf16x2(s[1][2], s[1][3])};
        const int vr = lane & 15, vc = lane >> 4;
#pragma unroll
        for (int n = 0; n < D / 16; ++n) {
            uint32_t b[4];
            ldsm_x4_t(b, ks + C::TILE + C::at(vr, 2 * n + vc));
            mma16816(o[2 * n], p, b[0], b[1]);
            mma16816(o[2 * n + 1], p, b[2], b[3]);
        }
    }
    __device__ __forceinline__ void store(const Res<__nv_bfloat16, D>& r, int lane) {
        const int g = lane >> 2, t = lane & 3;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
            l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
            if (t == 0) r.m(g + 8 * i) = m[i], r.l(g + 8 * i) = l[i];
#pragma unroll
            for (int n = 0; n < D / 8; ++n)
                *reinterpret_cast<float2*>(r.o(g + 8 * i) + 8 * n + 2 * t) = make_float2(o[n][2 * i], o[n][2 * i + 1]);
        }
    }
};

// fp32: a lane takes half a key's dot products, then D / 32 features of every head.
template <int D>
struct WarpF32 {
    static constexpr int H = HG<float>, E = D >= 32 ? D / 32 : 1;
    float o[H][E], m[H], l[H];

    __device__ __forceinline__ void init() {
#pragma unroll
        for (int h = 0; h < H; ++h) {
            m[h] = -INFINITY, l[h] = 0.f;
#pragma unroll
            for (int e = 0; e < E; ++e) o[h][e] = 0.f;
        }
    }
    // ks, vs: the tiles; qs [H][D] scaled by c; ps [H][16] this warp's own
    __device__ __forceinline__ void step(const uint8_t* ks, const float* qs, float* ps, int nk, int lane) {
        using C = Cfg<float, D>;
        const int key = lane & 15, half = lane >> 4;
        float s[H];
#pragma unroll
        for (int h = 0; h < H; ++h) s[h] = 0.f;
#pragma unroll 4
        for (int i = 0; i < C::CH / 2; ++i) {
            const int ch = half * (C::CH / 2) + i;
            const float4 k = *reinterpret_cast<const float4*>(ks + C::at(key, ch));
#pragma unroll
            for (int h = 0; h < H; ++h) {
                const float4 q = *reinterpret_cast<const float4*>(qs + h * D + 4 * ch);
                s[h] = fmaf(k.x, q.x, fmaf(k.y, q.y, fmaf(k.z, q.z, fmaf(k.w, q.w, s[h]))));
            }
        }
#pragma unroll
        for (int h = 0; h < H; ++h) {
            s[h] += __shfl_xor_sync(0xffffffffu, s[h], 16);
            if (key >= nk) s[h] = -INFINITY;
            float mx = s[h];
#pragma unroll
            for (int w = 1; w < 16; w <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
            if (mx > m[h]) {                      // the same in every lane
                const float al = exp2f(m[h] - mx);
                m[h] = mx;
                l[h] *= al;
#pragma unroll
                for (int e = 0; e < E; ++e) o[h][e] *= al;
            }
            const float p = m[h] == -INFINITY ? 0.f : exp2f(s[h] - m[h]);
            if (half == 0) ps[h * kKeys + key] = p, l[h] += p;
        }
        __syncwarp();
        const int f = lane * E;                   // its features (head size 16: lanes 0-15)
#pragma unroll
        for (int x = 0; x < kKeys; ++x) {
            float v[E];
            const float* row = reinterpret_cast<const float*>(ks + C::TILE + C::at(x, (f / 4) % C::CH)) + f % 4;
#pragma unroll
            for (int e = 0; e < E; ++e) v[e] = row[e];
#pragma unroll
            for (int h = 0; h < H; ++h) {
                const float p = ps[h * kKeys + x];
#pragma unroll
                for (int e = 0; e < E; ++e) o[h][e] = fmaf(p, v[e], o[h][e]);
            }
        }
    }
    __device__ __forceinline__ void store(const Res<float, D>& r, int lane) {
#pragma unroll
        for (int h = 0; h < H; ++h) {
#pragma unroll
            for (int w = 1; w < 16; w <<= 1) l[h] += __shfl_xor_sync(0xffffffffu, l[h], w);   // half 0 holds the sum
            if (lane == 0) r.m(h) = m[h], r.l(h) = l[h];
            if (lane * E < D)
#pragma unroll
                for (int e = 0; e < E; ++e) r.o(h)[lane * E + e] = o[h][e];
        }
    }
};

// One element of head h from n results, `get(i)` the i-th; *lse (natural log) on demand.
template <typename T, int D, typename Get>
__device__ __forceinline__ float join(int n, int h, int e, const Get& get, float* m_out, float* l_out) {
    float m = -INFINITY, l = 0.f, y = 0.f;
    for (int i = 0; i < n; ++i) m = fmaxf(m, get(i, HG<T> * D + h));
    const float ref = m == -INFINITY ? 0.f : m;
    for (int i = 0; i < n; ++i) {
        const float w = exp2f(get(i, HG<T> * D + h) - ref);
        l = fmaf(get(i, HG<T> * (D + 1) + h), w, l);
        y = fmaf(get(i, h * D + e), w, y);
    }
    *m_out = m;
    *l_out = l;
    return y;
}

template <typename T>
__device__ __forceinline__ void write_out(const P& a, int b, int h, int e, float y, float m, float l, bool some) {
    static_cast<T*>(const_cast<void*>(a.o.base))[b * a.o.sB + h * a.o.sH + e * a.o.sJ] = from_f32<T>(some ? y / l : 0.f);
    if (a.lse && e == 0) a.lse[(size_t)b * a.Hq + h] = some ? (m + log2f(l)) * kLn2 : -INFINITY;
}

__device__ __forceinline__ float ld_cluster(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

// Block (group, split); group = (sequence, key head, head group).
template <typename T, int D>
__global__ void __launch_bounds__(kT)
decode_kernel(const __grid_constant__ P a) {
    using C = Cfg<T, D>;
    extern __shared__ __align__(128) uint8_t sm[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int split = blockIdx.x % a.splits, group = blockIdx.x / a.splits;
    const int hg = group % a.hgroups, bk = group / a.hgroups, b = bk / a.Hkv, hk = bk % a.Hkv;
    const int h0 = hk * a.G + hg * HG<T>, nh = min(HG<T>, a.G - hg * HG<T>);
    const Slots s = load_slots(a, b);
    const int per = ((s.nv + a.splits - 1) / a.splits + kKeys - 1) / kKeys * kKeys;
    const long long first = (long long)split * per;
    const int x0 = (int)min((long long)s.nv, first), x1 = (int)min((long long)s.nv, first + per);
    const long long head = b * a.sB + hk * a.sH;
    uint8_t* mine = sm + warp * C::WARP;
    const uint32_t mine32 = tc::smem_u32(mine);

    // the first tiles are on their way before the queries are read
    const int stride = kWarps * kKeys;
    int next = x0 + warp * kKeys;
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) {
        if (next < x1) load_rows<T, D>(a, s, head, mine32 + i * 2 * C::TILE, mine + i * 2 * C::TILE, next, x1, lane);
        cp_async_commit();
        next += stride;
    }
    const T* qh = static_cast<const T*>(a.q.base) + b * a.q.sB + h0 * a.q.sH;
    float* qs = reinterpret_cast<float*>(sm + C::MAIN + C::RES);
    float* ps = qs + HG<T> * D + warp * HG<T> * kKeys;
    WarpBf16<D> wb;
    WarpF32<D> wf;
    if constexpr (sizeof(T) == 2) {
        wb.init(a, qh, nh, lane);
    } else {
        for (int i = threadIdx.x; i < HG<T> * D; i += kT) qs[i] = i / D < nh ? qh[i / D * a.q.sH + i % D * a.q.sJ] * a.c : 0.f;
        wf.init();
        __syncthreads();
    }
    int stage = 0;
    for (int x = x0 + warp * kKeys; x < x1; x += stride, next += stride) {
        const int to = stage == 0 ? kStages - 1 : stage - 1;      // the stage read in the last step
        if (next < x1) load_rows<T, D>(a, s, head, mine32 + to * 2 * C::TILE, mine + to * 2 * C::TILE, next, x1, lane);
        cp_async_commit();
        cp_async_wait<kStages - 1>();
        __syncwarp();
        if constexpr (sizeof(T) == 2) wb.step(mine32 + stage * 2 * C::TILE, x1 - x, a.c, lane);
        else wf.step(mine + stage * 2 * C::TILE, qs, ps, x1 - x, lane);
        __syncwarp();
        stage = stage == kStages - 1 ? 0 : stage + 1;
    }
    cp_async_wait<0>();
    __syncthreads();                              // the warps' results go over the tiles
    float* all = reinterpret_cast<float*>(sm);
    constexpr int RN = HG<T> * (D + 2);
    if constexpr (sizeof(T) == 2) wb.store(Res<T, D>{all + warp * RN}, lane);
    else wf.store(Res<T, D>{all + warp * RN}, lane);
    __syncthreads();
    auto from_warps = [&](int i, int at) { return all[i * RN + at]; };
    if (a.splits == 1) {
        for (int i = threadIdx.x; i < nh * D; i += kT) {
            float m, l;
            const float y = join<T, D>(kWarps, i / D, i % D, from_warps, &m, &l);
            write_out<T>(a, b, h0 + i / D, i % D, y, m, l, s.nv > 0);
        }
        return;
    }
    const bool cluster = a.splits <= kCluster;
    const Res<T, D> res{cluster ? reinterpret_cast<float*>(sm + C::MAIN) : a.part + ((size_t)group * a.splits + split) * RN};
    for (int i = threadIdx.x; i < nh * D; i += kT) {
        float m, l;
        res.o(i / D)[i % D] = join<T, D>(kWarps, i / D, i % D, from_warps, &m, &l);
        if (i % D == 0) res.m(i / D) = m, res.l(i / D) = l;
    }
    if (!cluster) return;
    __syncwarp();
    tc::cluster_sync_all();
    const uint32_t res32 = tc::smem_u32(sm + C::MAIN);
    for (int i = split * kT + threadIdx.x; i < nh * D; i += a.splits * kT) {   // split = rank in the cluster
        float m, l;
        const float y = join<T, D>(a.splits, i / D, i % D,
                                   [&](int r, int at) { return ld_cluster(tc::mapa_shared(res32, r) + 4 * at); }, &m, &l);
        write_out<T>(a, b, h0 + i / D, i % D, y, m, l, s.nv > 0);
    }
    __syncwarp();
    tc::cluster_sync_all();                       // no block leaves while its result is read
}

// Joins the splits of a group: one block per (group, 128 elements).
template <typename T, int D>
__global__ void __launch_bounds__(128)
decode_join_kernel(const __grid_constant__ P a) {
    constexpr int RN = HG<T> * (D + 2), PER = HG<T> * D / 128 > 0 ? HG<T> * D / 128 : 1;
    const int group = blockIdx.x / PER, i = blockIdx.x % PER * 128 + threadIdx.x;
    const int hg = group % a.hgroups, bk = group / a.hgroups, b = bk / a.Hkv, hk = bk % a.Hkv;
    const int h0 = hk * a.G + hg * HG<T>, nh = min(HG<T>, a.G - hg * HG<T>);
    if (i >= nh * D) return;
    const float* p = a.part + (size_t)group * a.splits * RN;
    float m, l;
    const float y = join<T, D>(a.splits, i / D, i % D, [&](int r, int at) { return p[(size_t)r * RN + at]; }, &m, &l);
    write_out<T>(a, b, h0 + i / D, i % D, y, m, l, __ldg(a.lens + b) > 0);
}

// How many runs the keys of a group are cut into.  About six blocks per SM's pair
// of slots even out unequal lengths (912 = 152 * 6), but a run has at least 128 keys
// (two tiles per warp); up to 16 are done as 8 at most, which a cluster joins.
struct Split {
    long long groups;
    int splits, hgroups;
};
Split split_of(int B, int Hq, int Hkv, int window, int sinks, int dtype) {
    Split s;
    const int hgm = dtype == PSA_BF16 ? HG<__nv_bfloat16> : HG<float>;
    s.hgroups = (Hq / Hkv + hgm - 1) / hgm;
    s.groups = (long long)B * Hkv * s.hgroups;
    const long long want = (912 + s.groups - 1) / s.groups, most = ((long long)sinks + window + 127) / 128;
    s.splits = (int)std::max(1ll, std::min(want, most));
    if (s.splits > kCluster && s.splits <= 16) s.splits = kCluster;
    return s;
}

template <typename T, int D>
int launch(const DecodeArgs& a, std::string* err) {
    using C = Cfg<T, D>;
    const Split s = split_of(a.B, a.Hq, a.Hkv, a.window, a.sinks, a.dtype);
    const long long grid = s.groups * s.splits;
    if (grid > 0x7fffffffll) {
        *err = "grid too large";
        return PSA_ERR_UNSUPPORTED;
    }
    if (!set_max_dynamic_smem((const void*)decode_kernel<T, D>, C::SMEM, err)) return PSA_ERR_CUDA;
    constexpr long long W = 16 / sizeof(T);
    const int vec = a.sB % W == 0 && a.sH % W == 0 && a.sS % W == 0;
    const P p{a.k, a.v, a.sB, a.sH, a.sS, a.q, a.o, a.lse, a.lens, static_cast<float*>(a.workspace), a.Hq, a.Hkv,
              a.Hq / a.Hkv, s.hgroups, a.cap, a.window, a.sinks, s.splits, vec, a.scale * kLog2e};
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(kT);
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.stream = a.stream;
    cudaLaunchAttribute at[1];
    if (s.splits > 1 && s.splits <= kCluster) {
        at[0].id = cudaLaunchAttributeClusterDimension;
        at[0].val.clusterDim = {(unsigned)s.splits, 1, 1};
        cfg.attrs = at;
        cfg.numAttrs = 1;
    }
    ProfScope prof(kSlotFwd, a.stream);
    cudaError_t e = cudaLaunchKernelEx(&cfg, decode_kernel<T, D>, p);
    if (e == cudaSuccess && s.splits > kCluster) {
        constexpr int PER = HG<T> * D / 128 > 0 ? HG<T> * D / 128 : 1;
        decode_join_kernel<T, D><<<(unsigned)(s.groups * PER), 128, 0, a.stream>>>(p);
        e = cudaGetLastError();
    }
    if (e == cudaSuccess) return PSA_OK;
    *err = std::string("window decode launch: ") + cudaGetErrorString(e);
    return PSA_ERR_CUDA;
}

}  // namespace

size_t decode_workspace(int B, int Hq, int Hkv, int d, int window, int sinks, int dtype) {
    const Split s = split_of(B, Hq, Hkv, window, sinks, dtype);
    const int hgm = dtype == PSA_BF16 ? HG<__nv_bfloat16> : HG<float>;
    return s.splits > kCluster ? (size_t)s.groups * s.splits * hgm * (d + 2) * 4 : 0;
}

int decode(const DecodeArgs& a, std::string* err) {
    const bool f = a.dtype == PSA_F32;
    switch (a.d) {
        case 16: return f ? launch<float, 16>(a, err) : launch<__nv_bfloat16, 16>(a, err);
        case 32: return f ? launch<float, 32>(a, err) : launch<__nv_bfloat16, 32>(a, err);
        case 64: return f ? launch<float, 64>(a, err) : launch<__nv_bfloat16, 64>(a, err);
        default: return f ? launch<float, 128>(a, err) : launch<__nv_bfloat16, 128>(a, err);
    }
}

}  // namespace win
}  // namespace psa
