// rope.cu -- rotary positions with several axes, and the rolling cache's
// writes (which rotate the keys on the way).
//
//   y1 = x1 cos a - x2 sin a,  y2 = x2 cos a + x1 sin a,  a = 2 pi pos F / 2^64
// F is the pair's frequency in units of 2^-64 turns, rounded, so pos * F modulo 2^64
// is the angle modulo a turn to 2^-34 turns for every 32-bit position: no range
// reduction, and no 64-bit floating point, which this GPU has little of.  Its
// upper 32 bits, rounded, go to sincospif as fp32: half a step there (2^-26 turns)
// is most of the angle's error, 2^-26 + 2^-33 + 2^-34 turns.
//
// Every element is read and written once: 0.75 of the copy rate, with DRAM at 29% (the
// results stay in L2 meanwhile) and issue at 67%.  What it waits for most is the barrier between
// a group's angles and its rows, every one to eight tokens.  A block works on groups
// of a few tokens and heads, a 16-byte unit of one row (token and head) per thread, the
// angles' cos / sin once per token for all heads of the group (shared memory).  It goes
// from group to group with the next one's loads on their way: one group per block
// spent most of its time on the chain position, angle, barrier, store.  B=2, 24 heads,
// 6400 tokens, d=64 in bf16, 79 MB: 15.4 us (one group per block 19 us), in fp32 31.0.  Cache
// writes, 4 prompts of 2048 tokens, 8 heads, d=128, of which the newest 1028 stay: 10.6 us (21),
// in fp32 18.2.
#include "rope.cuh"

namespace psa {
namespace win {
namespace {

struct Tensor {                                  // one view to rotate
    const void* x;
    void* y;
    long long xB, xH, xN, xJ, yB, yH, yN, yJ;
};

// Units of 16 bytes of a head: with pairs in halves a unit is the 16 bytes at
// feature c and those at c + n; interleaved pairs lie inside a unit; units past
// the rotated features are copied.
struct Units {
    int rot, total;
};
template <typename T>
__host__ __device__ __forceinline__ Units units(int d, int n, int interleaved) {
    const int rot = interleaved ? 2 * n / VEC<T> : n / VEC<T>;
    return Units{rot, rot + (d - 2 * n) / VEC<T>};
}

template <typename T>
struct Loaded {
    uint4 a, b;
};
template <typename T>
__device__ __forceinline__ Loaded<T> load_unit(const T* x, int u, const Units& us, int n, int interleaved) {
    Loaded<T> l;
    if (u >= us.rot) {
        l.a = *reinterpret_cast<const uint4*>(x + 2 * n + (u - us.rot) * VEC<T>);
    } else {
        l.a = *reinterpret_cast<const uint4*>(x + u * VEC<T>);
        if (!interleaved) l.b = *reinterpret_cast<const uint4*>(x + n + u * VEC<T>);
    }
    return l;
}
// cs: the token's (cos, sin) of every pair, 16-byte aligned (a rotation by units has an
// even number of pairs)
template <typename T>
__device__ __forceinline__ void store_unit(T* y, const Loaded<T>& l, int u, const Units& us, int n, int interleaved,
                                           const float2* cs) {
    constexpr int W = VEC<T>;
    if (u >= us.rot) {
        *reinterpret_cast<uint4*>(y + 2 * n + (u - us.rot) * W) = l.a;
        return;
    }
    float a[W], r[W];
    unpack<T>(l.a, a);
    if (interleaved) {
#pragma unroll
        for (int e = 0; e < W; e += 4) {
            const float4 w = *reinterpret_cast<const float4*>(cs + (u * W + e) / 2);
            r[e] = a[e] * w.x - a[e + 1] * w.y;
            r[e + 1] = a[e + 1] * w.x + a[e] * w.y;
            r[e + 2] = a[e + 2] * w.z - a[e + 3] * w.w;
            r[e + 3] = a[e + 3] * w.z + a[e + 2] * w.w;
        }
        *reinterpret_cast<uint4*>(y + u * W) = pack<T>(r);
    } else {
        float b[W], q[W];
        unpack<T>(l.b, b);
#pragma unroll
        for (int e = 0; e < W; e += 2) {          // (cos, sin) of two pairs at a time
            const float4 w = *reinterpret_cast<const float4*>(cs + u * W + e);
            r[e] = a[e] * w.x - b[e] * w.y;
            q[e] = b[e] * w.x + a[e] * w.y;
            r[e + 1] = a[e + 1] * w.z - b[e + 1] * w.w;
            q[e + 1] = b[e + 1] * w.z + a[e + 1] * w.w;
        }
        *reinterpret_cast<uint4*>(y + u * W) = pack<T>(r);
        *reinterpret_cast<uint4*>(y + n + u * W) = pack<T>(q);
    }
}

// One feature pair (or, i >= n, one copied feature), any strides.
template <typename T>
__device__ __forceinline__ void scalar_pair(const T* x, long long xJ, T* y, long long yJ, int i, int n, int interleaved,
                                            float2 w) {
    if (i >= n) {
        const int f = n + i;                     // features 2n ...
        y[f * yJ] = x[f * xJ];
        return;
    }
    const int f1 = interleaved ? 2 * i : i, f2 = interleaved ? 2 * i + 1 : i + n;
    const float a = to_f32(x[f1 * xJ]), b = to_f32(x[f2 * xJ]);
    y[f1 * yJ] = from_f32<T>(a * w.x - b * w.y);
    y[f2 * yJ] = from_f32<T>(b * w.x + a * w.y);
}

// ---------------------------------------------------------------- rope
// Heads 0 .. H0-1 are those of the first tensor, then those of the second.
template <typename T>
__global__ void __launch_bounds__(kT)
rope_kernel(const __grid_constant__ Plan pl, const __grid_constant__ Tensor t0, const __grid_constant__ Tensor t1, int H0,
            Pos pos, const __grid_constant__ Work w, float sign) {
    extern __shared__ __align__(16) float2 cs_all[];   // [2][TN][n]
    const Units us = units<T>(pl.d, pl.n, pl.interleaved);
    const int row = divide(threadIdx.x, w.by_u), u = threadIdx.x - row * us.total;
    // the thread's angle: neighbouring threads share a pair, whose frequency is a kernel
    // argument, and those are read one place at a time
    const int ai = divide(threadIdx.x, w.by_tn), at = threadIdx.x - ai * w.TN;
    auto mine = [&](const Group& g, int& t, int& h) {  // the thread's token and head of a group
        if (row >= g.nt * g.nh) return false;
        t = divide(row, g.nh == w.hper ? w.by_h : w.by_last);
        h = g.hb + row - t * g.nh;
        return true;
    };
    auto load = [&](const Group& g, Loaded<T>& l, int& p) {
        int t, h;
        if (mine(g, t, h)) {
            const bool first = h < H0;
            l = load_unit(first ? row_at<T>(t0.x, t0.xB, t0.xH, t0.xN, g.b, h, g.n0 + t)
                                : row_at<T>(t1.x, t1.xB, t1.xH, t1.xN, g.b, h - H0, g.n0 + t), u, us, pl.n, pl.interleaved);
        }
        if (ai < pl.n && at < g.nt) p = load_pos(pl, pos, ai, g.b, g.n0 + at);
    };
    Group g = group_of(w, blockIdx.x), gn = g;
    Loaded<T> l, ln;
    int p = 0, pn = 0, buf = 0;
    load(g, l, p);
    for (int x = blockIdx.x; x < w.groups; x += gridDim.x) {
        if (x + (int)gridDim.x < w.groups) {
            gn = group_of(w, x + gridDim.x);
            load(gn, ln, pn);
        }
        float2* cs = cs_all + buf * w.TN * pl.n;   // a buffer is written again two barriers later
        buf ^= 1;
        if (ai < pl.n && at < g.nt) cs[at * pl.n + ai] = cos_sin(pl, ai, p, sign);
        __syncthreads();
        int t, h;
        if (mine(g, t, h))
            store_unit(h < H0 ? row_at<T>(t0.y, t0.yB, t0.yH, t0.yN, g.b, h, g.n0 + t)
                              : row_at<T>(t1.y, t1.yB, t1.yH, t1.yN, g.b, h - H0, g.n0 + t),
                       l, u, us, pl.n, pl.interleaved, cs + t * pl.n);
        g = gn, l = ln, p = pn;
    }
}

// Any strides: a thread per (token, pair), over all heads; neighbouring threads
// take neighbouring positions (pos_fast: channel-major tensors) or pairs.
template <typename T>
__global__ void __launch_bounds__(kT)
rope_scalar_kernel(const __grid_constant__ Plan pl, Tensor t0, Tensor t1, int H0, int H, Pos pos, int N, long long total,
                   int pos_fast, float sign) {
    const long long idx = (long long)blockIdx.x * kT + threadIdx.x;
    if (idx >= total) return;
    const int items = pl.d - pl.n;               // pairs and copied features
    long long b, n;
    int i;
    if (pos_fast) {
        n = idx % N;
        const long long r = idx / N;
        i = (int)(r % items), b = r / items;
    } else {
        i = (int)(idx % items);
        const long long r = idx / items;
        n = r % N, b = r / N;
    }
    const float2 w = i < pl.n ? cos_sin(pl, i, load_pos(pl, pos, i, (int)b, n), sign) : make_float2(1.f, 0.f);
    for (int h = 0; h < H; ++h) {
        const Tensor& v = h < H0 ? t0 : t1;
        const int hh = h < H0 ? h : h - H0;
        scalar_pair<T>(static_cast<const T*>(v.x) + b * v.xB + hh * v.xH + n * v.xN, v.xJ,
                       static_cast<T*>(v.y) + b * v.yB + hh * v.yH + n * v.yN, v.yJ, i, pl.n, pl.interleaved, w);
    }
}

// ---------------------------------------------------------------- cache append
struct Cache {
    void* k;
    void* v;
    long long sB, sH, sS;
    int cap, sinks;
};

// Slot of row t of sequence b, or -1: past n_new, or overwritten by a newer
// row of the same call (sinks never are).
__device__ __forceinline__ int slot_of(const Cache& c, const int* start, const int* n_new, int b, int t, int T) {
    const int st = __ldg(start + b);
    const int n = n_new ? min(max(__ldg(n_new + b), 0), T) : T;
    if (t >= n || st < 0 || st - 1 > 0x7fffffff - n) return -1;
    const int ring = c.cap - c.sinks, p = st + t;
    if (p < c.sinks) return p;
    if (t < n - ring) return -1;                 // p + ring is in this call too
    return c.sinks + (p - c.sinks) % ring;
}

// PICK: position x takes row from.row(b, x), else row x.
template <typename T, bool PICK>
__global__ void __launch_bounds__(kT)
append_kernel(const __grid_constant__ Plan pl, const __grid_constant__ Tensor kn, const __grid_constant__ Tensor vn,
              const __grid_constant__ Cache c, Pos pos, const int* __restrict__ start, const int* __restrict__ n_new, int Tn,
              const __grid_constant__ Work w, Picked from) {
    extern __shared__ __align__(16) float2 cs_all[];   // [2][TN][n]
    // a row's key by rotation units, then its value by 32 bytes
    const Units uk = units<T>(pl.d, pl.n, pl.interleaved);
    constexpr int V2 = 2 * VEC<T>;
    const int per = uk.total + pl.d / V2, row = divide(threadIdx.x, w.by_u), q = threadIdx.x - row * per;
    const bool key = q < uk.total;
    const int ai = divide(threadIdx.x, w.by_tn), at = threadIdx.x - ai * w.TN;
    Kept kept;
    // the thread's row of a group: its token, head and slot (-1: none)
    auto load = [&](const Group& g, Loaded<T>& l, int& p, int& t, int& h) {
        const int ring = c.cap - c.sinks;
        kept.of(start, n_new, g.b, Tn, c.sinks, ring);
        int slot = -1;
        if (row < g.nt * g.nh) {
            t = divide(row, g.nh == w.hper ? w.by_h : w.by_last);
            h = g.hb + row - t * g.nh;
            int x = kept.row(g.n0 + t);
            const int at_pos = kept.st + x;
            const bool there = x < kept.n && (!PICK || from.row(g.b, x));
            if (there) {
                slot = at_pos < c.sinks ? at_pos : c.sinks + (at_pos - c.sinks) % ring;
                if (key) {
                    l = load_unit(row_at<T>(kn.x, kn.xB, kn.xH, kn.xN, g.b, h, x), q, uk, pl.n, pl.interleaved);
                } else {
                    const uint4* v = reinterpret_cast<const uint4*>(row_at<T>(vn.x, vn.xB, vn.xH, vn.xN, g.b, h, x) +
                                                                    (q - uk.total) * V2);
                    l.a = v[0], l.b = v[1];
                }
            }
        }
        if (ai < pl.n && at < g.nt) {
            int ax = kept.row(g.n0 + at);
            if (ax < kept.n && (!PICK || from.row(g.b, ax))) p = load_pos(pl, pos, ai, g.b, ax);
        }
        return slot;
    };
    Group g = group_of(w, blockIdx.x), gn = g;
    Loaded<T> l, ln;
    int p = 0, pn = 0, t = 0, tn = 0, h = 0, hn = 0, buf = 0, slot_next = -1;
    int slot = load(g, l, p, t, h);
    for (int x = blockIdx.x; x < w.groups; x += gridDim.x) {
        if (x + (int)gridDim.x < w.groups) {
            gn = group_of(w, x + gridDim.x);
            slot_next = load(gn, ln, pn, tn, hn);
        }
        float2* cs = cs_all + buf * w.TN * pl.n;   // a buffer is written again two barriers later
        buf ^= 1;
        if (ai < pl.n && at < g.nt) cs[at * pl.n + ai] = cos_sin(pl, ai, p, 1.f);
        __syncthreads();
        if (slot >= 0) {
            if (key) {
                store_unit(row_at<T>(c.k, c.sB, c.sH, c.sS, g.b, h, slot), l, q, uk, pl.n, pl.interleaved, cs + t * pl.n);
            } else {
                uint4* v = reinterpret_cast<uint4*>(row_at<T>(c.v, c.sB, c.sH, c.sS, g.b, h, slot) + (q - uk.total) * V2);
                v[0] = l.a, v[1] = l.b;
            }
        }
        g = gn, l = ln, p = pn, t = tn, h = hn, slot = slot_next;
    }
}

template <typename T>
__global__ void __launch_bounds__(kT)
append_scalar_kernel(const __grid_constant__ Plan pl, Tensor kn, Tensor vn, Cache c, int Hkv, Pos pos,
                     const int* __restrict__ start, const int* __restrict__ n_new, int Tn, long long total, Picked from) {
    const long long idx = (long long)blockIdx.x * kT + threadIdx.x;
    if (idx >= total) return;
    const int items = pl.d - pl.n, i = (int)(idx % items);
    const long long tok = idx / items, b = tok / Tn;
    int n = (int)(tok % Tn);
    const int slot = slot_of(c, start, n_new, (int)b, n, Tn);
    if (slot < 0 || (from.rows && !from.row((int)b, n))) return;
    const float2 w = i < pl.n ? cos_sin(pl, i, load_pos(pl, pos, i, (int)b, n), 1.f) : make_float2(1.f, 0.f);
    for (int h = 0; h < Hkv; ++h) {
        const long long to = b * c.sB + h * c.sH + slot * c.sS;
        scalar_pair<T>(static_cast<const T*>(kn.x) + b * kn.xB + h * kn.xH + n * kn.xN, kn.xJ,
                       static_cast<T*>(c.k) + to, 1, i, pl.n, pl.interleaved, w);
        const T* x = static_cast<const T*>(vn.x) + b * vn.xB + h * vn.xH + n * vn.xN;
        T* y = static_cast<T*>(c.v) + to;
        for (int f = i; f < pl.d; f += items) y[f] = x[f * vn.xJ];
    }
}

// a rotation whose pairs and rest fill whole 16-byte units
bool plan_ok(const Plan& pl, int esize) {
    const int w = 16 / esize;
    return pl.interleaved ? 2 * pl.n % w == 0 : pl.n % w == 0 && (pl.d - 2 * pl.n) % w == 0;
}

Tensor tensor(const View& x, const View& y) {
    return Tensor{x.base, const_cast<void*>(y.base), x.sB, x.sH, x.sN, x.sJ, y.sB, y.sH, y.sN, y.sJ};
}

template <typename T>
int launch_rope(const RopeArgs& a, std::string* err) {
    const Plan pl = dev_plan(a.plan, a.plan->head_dim);
    const long long tokens = (long long)a.B * a.N;
    const int H0 = a.heads[0], H = H0 + (a.n > 1 ? a.heads[1] : 0);
    const Tensor t0 = tensor(a.x[0], a.y[0]), t1 = a.n > 1 ? tensor(a.x[1], a.y[1]) : t0;
    const Pos pos{a.pos, a.pos_axis, a.pos_batch};
    const float sign = a.inverse ? -1.f : 1.f;
    bool vec = plan_ok(pl, sizeof(T));
    for (int i = 0; i < a.n; ++i) vec = vec && view_ok(a.x[i], sizeof(T)) && view_ok(a.y[i], sizeof(T));
    if (!vec) {
        const long long total = tokens * (pl.d - pl.n), grid = (total + kT - 1) / kT;
        if (grid > 0x7fffffffll) return too_large(err);
        rope_scalar_kernel<T><<<(unsigned)grid, kT, 0, a.stream>>>(pl, t0, t1, H0, H, pos, a.N, total,
                                                                   a.x[0].sN == 1 && a.x[0].sJ != 1, sign);
        return launched("rope launch", err);
    }
    const Units us = units<T>(pl.d, pl.n, pl.interleaved);
    Work w;
    if (!work_for(a.B, a.N, H, us.total, pl.n, &w)) return too_large(err);
    rope_kernel<T><<<blocks_for(w), kT, 2 * (size_t)w.TN * pl.n * sizeof(float2), a.stream>>>(pl, t0, t1, H0, pos, w, sign);
    return launched("rope launch", err);
}

template <typename T>
int launch_append(const AppendArgs& a, std::string* err) {
    const Plan pl = dev_plan(a.plan, a.d);
    const long long tokens = (long long)a.B * a.T;
    const View none{};
    const Tensor kn = tensor(a.kn, none), vn = tensor(a.vn, none);
    const Cache c{a.k, a.v, a.sB, a.sH, a.sS, a.cap, a.sinks};
    const Pos pos{a.pos, a.pos_axis, a.pos_batch};   // not read without a plan (no pairs)
    const Picked from{a.rows, a.rows_stride, a.n_rows};
    const bool vec = plan_ok(pl, sizeof(T)) && view_ok(a.kn, sizeof(T)) && view_ok(a.vn, sizeof(T)) &&
                     aligned(a.k, sizeof(T), a.sB, a.sH, a.sS) && aligned(a.v, sizeof(T), 0, 0, 0) && a.sH <= 0x7fffffffll &&
                     a.sS <= 0x7fffffffll;
    if (!vec) {
        const long long total = tokens * (pl.d - pl.n), grid = (total + kT - 1) / kT;
        if (grid > 0x7fffffffll) return too_large(err);
        append_scalar_kernel<T><<<(unsigned)grid, kT, 0, a.stream>>>(pl, kn, vn, c, a.Hkv, pos, a.start, a.n_new, a.T, total,
                                                                     from);
        return launched("cache append launch", err);
    }
    Work w;
    if (!work_for(a.B, std::min(a.T, a.cap), a.Hkv,
                  units<T>(pl.d, pl.n, pl.interleaved).total + pl.d / (2 * VEC<T>), pl.n, &w))
        return too_large(err);
    const size_t smem = 2 * (size_t)w.TN * pl.n * sizeof(float2);
    if (a.rows)
        append_kernel<T, true><<<blocks_for(w), kT, smem, a.stream>>>(pl, kn, vn, c, pos, a.start, a.n_new, a.T, w, from);
    else
        append_kernel<T, false><<<blocks_for(w), kT, smem, a.stream>>>(pl, kn, vn, c, pos, a.start, a.n_new, a.T, w, from);
    return launched("cache append launch", err);
}

}  // namespace

int rope(const RopeArgs& a, std::string* err) {
    return a.dtype == PSA_F32 ? launch_rope<float>(a, err) : launch_rope<__nv_bfloat16>(a, err);
}
int append(const AppendArgs& a, std::string* err) {
    return a.dtype == PSA_F32 ? launch_append<float>(a, err) : launch_append<__nv_bfloat16>(a, err);
}

}  // namespace win
}  // namespace psa
