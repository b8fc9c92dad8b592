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
#include "tc_sync.cuh"
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

// MMA and commit by one elected lane of a warp that runs converged (the same lane
// each time, so a commit covers the warp's MMAs): descriptors then stay in uniform
// registers, where a branch to one lane has to move them there for every MMA.
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\telect.sync _|q, 0xffffffff;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(id), "r"(acc)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t id, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\telect.sync _|q, 0xffffffff;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(id), "r"(acc)
        : "memory");
}
__device__ __forceinline__ void commit(uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar)
        : "memory");
}

// Bounded waits (as in tc_sync.cuh) that let the hardware suspend the thread for
// longer: a waiting warp that keeps asking takes issue slots from the warps of its
// scheduler that it waits for.
__device__ __forceinline__ bool try_wait_long(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity), "r"(100000u)
        : "memory");
    return ok != 0;
}
static __device__ __noinline__ bool wait_more(const tc::Sync& s, uint32_t bar, uint32_t parity, int role, int tile) {
    const uint64_t t0 = tc::globaltimer_ns();
    for (;;) {
        if (try_wait_long(bar, parity)) return true;
        if (*s.abort) return false;
        if (tc::globaltimer_ns() - t0 > tc::kTimeoutNs) {
            *s.abort = 1;
            atomicCAS(s.err, 0, ((1 + role) << 24) | (tile & 0xFFFFFF));
            return false;
        }
    }
}
__device__ __forceinline__ bool wait_one(const tc::Sync& s, uint32_t bar, uint32_t parity, int role, int tile) {
    return tc::mbar_try_wait(bar, parity) || wait_more(s, bar, parity, role, tile);
}
__device__ __forceinline__ bool wait_warp(const tc::Sync& s, uint32_t bar, uint32_t parity, int role, int tile) {
    return __all_sync(0xffffffffu, wait_one(s, bar, parity, role, tile));
}

// One arrival for the whole warp, behind everything its lanes did (32 arrivals of
// one instruction are done one by one).
__device__ __forceinline__ void warp_arrive(uint32_t bar, int lane) {
    __syncwarp();
    if (lane == 0) tc::mbar_arrive(bar);
}

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

// A warp's 32 rows of W <= 32 bf16 features (row r as W / 2 pairs in lane r) to
// row0 + r ld, rows r < nvalid: through 1 KB of staging per round, so that the
// lanes of a store share rows (a row per lane makes every store touch 32 lines).
// The 16-byte pieces are spread over the banks by their line's number.
template <int W>
__device__ __forceinline__ void store_rows(uint32_t stg, const uint32_t (&w)[W / 2], uint16_t* row0, long long ld, int nvalid,
                                           int lane) {
    constexpr int CH = W / 8, R = 1024 / (2 * W) < 32 ? 1024 / (2 * W) : 32;   // pieces per row, rows per round
    auto swz = [](uint32_t i) { return (i & ~7u) | ((i & 7u) ^ ((i >> 3) & 7u)); };
#pragma unroll
    for (int q = 0; q < 32 / R; ++q) {
        if (lane / R == q) {
#pragma unroll
            for (int c = 0; c < CH; ++c)
                tc::st_shared_v4(stg + 16u * swz((lane - q * R) * CH + c), w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
        }
        __syncwarp();
#pragma unroll
        for (int k = 0; k < R * CH / 32; ++k) {
            const uint32_t i = (uint32_t)lane + 32u * k;
            const int r = q * R + (int)(i / CH), c = (int)(i % CH);
            const uint4 v = tc::ld_shared_v4(stg + 16u * swz(i));
            if (r < nvalid) *reinterpret_cast<uint4*>(row0 + (long long)r * ld + 8 * c) = v;
        }
        __syncwarp();
    }
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
