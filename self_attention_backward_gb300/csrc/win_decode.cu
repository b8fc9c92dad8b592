// win_decode.cu -- attention of one query row per sequence over the rolling
// key/value cache.
//
// One block per (sequence, key head): all query heads of the key head share
// its reads.  A warp takes a key at a time, its lanes the features; an online
// softmax per warp, the warps joined at the end.
#include <cuda_bf16.h>

#include <string>

#include "common.cuh"
#include "win_internal.h"

namespace psa {
namespace win {
namespace {

constexpr int kT = 256, kWarps = kT / 32;

struct P {
    const void* k;
    const void* v;
    long long sB, sH, sS;
    View q, o;
    float* lse;
    const int* lens;
    int Hq, Hkv, cap, window, sinks;
    float scale_log2;
};

template <typename T, int D>
__global__ void __launch_bounds__(kT)
decode_kernel(P a) {
    constexpr int E = D >= 32 ? D / 32 : 1;       // features per lane
    __shared__ float qs[D], om[kWarps][D], ms[kWarps], ls[kWarps];
    const int b = blockIdx.x / a.Hq, h = blockIdx.x % a.Hq, hk = h / (a.Hq / a.Hkv);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int L = max(__ldg(a.lens + b), 0), ring = a.cap - a.sinks;
    const long long seen = (long long)a.sinks + a.window;
    const int nv = (int)min((long long)L, seen);
    const T* q = static_cast<const T*>(a.q.base) + b * a.q.sB + h * a.q.sH;
    for (int e = threadIdx.x; e < D; e += kT) qs[e] = to_f32(q[e * a.q.sJ]) * a.scale_log2;
    __syncthreads();
    const bool on = lane < D;
    float m = -INFINITY, l = 0.f, acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
    for (int x = warp; x < nv; x += kWarps) {
        const int p = x < a.sinks ? x : L - nv + x;
        const int slot = p < a.sinks ? p : a.sinks + (p - a.sinks) % ring;
        const long long at = b * a.sB + hk * a.sH + slot * a.sS;
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e)
            if (on) s = fmaf(qs[lane * E + e], to_f32(static_cast<const T*>(a.k)[at + lane * E + e]), s);
#pragma unroll
        for (int w = 16; w; w >>= 1) s += __shfl_xor_sync(0xffffffffu, s, w);
        const float mn = fmaxf(m, s), al = exp2f(m - mn), pr = exp2f(s - mn);
        l = l * al + pr;
        m = mn;
#pragma unroll
        for (int e = 0; e < E; ++e)
            acc[e] = acc[e] * al + (on ? pr * to_f32(static_cast<const T*>(a.v)[at + lane * E + e]) : 0.f);
    }
#pragma unroll
    for (int e = 0; e < E; ++e)
        if (on) om[warp][lane * E + e] = acc[e];
    if (lane == 0) ms[warp] = m, ls[warp] = l;
    __syncthreads();
    float mx = -INFINITY, lt = 0.f;
    for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, ms[w]);
    const float ref = mx == -INFINITY ? 0.f : mx;
    for (int w = 0; w < kWarps; ++w) lt += ls[w] * exp2f(ms[w] - ref);
    T* o = static_cast<T*>(const_cast<void*>(a.o.base)) + b * a.o.sB + h * a.o.sH;
    for (int e = threadIdx.x; e < D; e += kT) {
        float y = 0.f;
        for (int w = 0; w < kWarps; ++w) y += om[w][e] * exp2f(ms[w] - ref);
        o[e * a.o.sJ] = from_f32<T>(nv > 0 ? y / lt : 0.f);
    }
    if (a.lse && threadIdx.x == 0) a.lse[(size_t)b * a.Hq + h] = nv > 0 ? (mx + log2f(lt)) * kLn2 : -INFINITY;
}

template <typename T, int D>
int launch(const DecodeArgs& a, std::string* err) {
    const long long grid = (long long)a.B * a.Hq;
    if (grid > 0x7fffffffll) {
        *err = "grid too large";
        return PSA_ERR_UNSUPPORTED;
    }
    ProfScope prof(kSlotFwd, a.stream);
    decode_kernel<T, D><<<(unsigned)grid, kT, 0, a.stream>>>(P{a.k, a.v, a.sB, a.sH, a.sS, a.q, a.o, a.lse, a.lens, a.Hq,
                                                              a.Hkv, a.cap, a.window, a.sinks, a.scale * kLog2e});
    const cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) return PSA_OK;
    *err = std::string("window decode launch: ") + cudaGetErrorString(e);
    return PSA_ERR_CUDA;
}

}  // namespace

size_t decode_workspace(int, int, int, int, int, int, int) { return 0; }

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
