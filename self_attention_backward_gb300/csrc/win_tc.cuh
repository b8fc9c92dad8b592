// win_tc.cuh -- operand tiles, masks and output rows shared by the tensor-core
// kernels of the sliding-window attention.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <map>
#include <mutex>
#include <string>

#include "psa_internal.h"
#include "tc_ptx.cuh"
#include "tc_tmap.h"

namespace psa {
namespace win {

// A [ROWS, D] bf16 tile in shared memory as the tensor cores read it: panels of
// 64 features (all of them below 64), each ROWS rows of ROWB bytes, swizzled over
// ROWB.
template <int D, int ROWS = 128>
struct Operand {
    static constexpr int W = D < 64 ? D : 64;         // features per panel
    static constexpr int ROWB = 2 * W;
    static constexpr int PANEL = ROWS * ROWB;
    static constexpr int TILE = D / W * PANEL;
    static constexpr uint32_t SW = W == 64 ? 2u : W == 32 ? 4u : 6u;
    // Descriptors: features as the product's K (steps of 16 features), or rows as
    // its K (steps of 16 rows) with the features as N.
    static __device__ __forceinline__ uint64_t kmajor(uint32_t s) { return tc::smem_desc(s, 16, 8 * ROWB, SW); }
    static __device__ __forceinline__ uint64_t mnmajor(uint32_t s) { return tc::smem_desc(s, PANEL, 8 * ROWB, SW); }
    static constexpr __device__ __forceinline__ uint32_t kstep(int kk) {
        return (uint32_t)((kk / (W / 16)) * (PANEL >> 4) + 2 * (kk % (W / 16)));
    }
    static constexpr uint32_t MN_KSTEP = (16 * ROWB) >> 4;

    // Rows row.. of head (b, h) into the tile at dst, arriving on bar.  Rows past
    // the tensor's end read as zero.
    static __device__ __forceinline__ void load(uint32_t dst, const CUtensorMap* map, int row, int h, int b, uint32_t bar) {
        tc::mbar_arrive_expect_tx(bar, TILE);
#pragma unroll
        for (int p = 0; p < D / W; ++p) tc::tma_load_4d(dst + p * PANEL, map, p * W, row, h, b, bar);
    }
    static __device__ __forceinline__ void clear_row(uint32_t tile, int r) {
#pragma unroll
        for (int p = 0; p < D / W; ++p)
#pragma unroll
            for (int x = 0; x < ROWB; x += 16) tc::st_shared_v4(tile + p * PANEL + r * ROWB + x, 0, 0, 0, 0);
    }
    // Map over a view [B, heads, N, D]; a dimension of length 1 gets a stride that
    // the encoder takes.
    static bool encode(CUtensorMap* map, const View& v, int B, int heads, int N, int rows, std::string* err) {
        return encode_bf16_4d(map, v.base, D, N, heads, B, N > 1 ? v.sN : D, heads > 1 ? v.sH : D, B > 1 ? v.sB : D, W, rows,
                              err);
    }
};

// 2^x, free to be scheduled (exponentials of a row are independent).
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Bits e (columns c0 + e) that a row sees: c0 + e <= hi and (c0 + e >= lo or
// c0 + e < snk).
__device__ __forceinline__ uint32_t bits_below(int n) {   // the lowest n bits, n clamped to 0..32
    return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u;
}
__device__ __forceinline__ uint32_t col_mask(int lo, int hi, int snk, int c0) {
    return bits_below(hi + 1 - c0) & (~bits_below(lo - c0) | bits_below(snk - c0));
}

// Rows of an output view with adjacent features.
struct RowOut {
    uint16_t* base;
    long long sB, sH, sN;
    __device__ __forceinline__ uint16_t* row(int b, int h, int n) const { return base + b * sB + h * sH + n * sN; }
};
inline RowOut row_out(const View& v) {
    return RowOut{static_cast<uint16_t*>(const_cast<void*>(v.base)), v.sB, v.sH, v.sN};
}

// SMs of the current device (looked up once per device).
inline bool sm_count(int* n, std::string* err) {
    static std::mutex mu;
    static std::map<int, int> known;
    int dev = -1;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) {
        std::lock_guard<std::mutex> g(mu);
        auto it = known.find(dev);
        if (it != known.end()) {
            *n = it->second;
            return true;
        }
        e = cudaDeviceGetAttribute(n, cudaDevAttrMultiProcessorCount, dev);
        if (e == cudaSuccess) {
            known[dev] = *n;
            return true;
        }
    }
    *err = std::string("SM count: ") + cudaGetErrorString(e);
    return false;
}

// Reads and clears a translation unit's device error word (a bounded wait that
// gave up); 1 if it was set.
template <typename Symbol>
int take_error(Symbol& word, const char* what, std::string* err) {
    int v = 0;
    if (cudaMemcpyFromSymbol(&v, word, sizeof(int)) != cudaSuccess || v == 0) return 0;
    const int zero = 0;
    cudaMemcpyToSymbol(word, &zero, sizeof(int));
    *err = std::string(what) + ": a bounded wait gave up (role " + std::to_string(((v >> 24) & 0xff) - 1) + ", tile " +
           std::to_string(v & 0xFFFFFF) + ")";
    return 1;
}

}  // namespace win
}  // namespace psa
