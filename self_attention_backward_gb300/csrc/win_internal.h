// win_internal.h -- host-side interface of the sliding-window attention family
// (win_api.cu: argument checks and dispatch; win_warp.cu, win_tc_*.cu, rope.cu,
// win_decode.cu: kernels).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>

#include <string>
#include <type_traits>

#include "psa_attn.h"
#include "psa_internal.h"

namespace psa {
namespace win {

// One problem, sizes checked; window and sinks are clamped to Nk (a larger
// value means the same), so positions never leave 32 bits.
struct Args {
    int B, Hq, Hkv, Nq, Nk, d, window, sinks;
    float scale;
    int dtype;
    View q, k, v, o, dO, dq, dk, dv;
    float* lse;
    const int* q_lens;
    const int* kv_lens;
    float* Drow;          // backward: row statistics [B, Hq, stat_rows(Nq)]: D, and
    float* negl;          // -LSE log2(e) (-inf for rows that see nothing, padding);
    void* aug;            // both for the tensor cores: 8 bf16 per row, -LSE / scale and
                          // -D as sums of three each, then two zeros
    float* part;          // backward: partial sums of the sink rows (see FarSplit)
    cudaStream_t stream;
};

// The keys j < sinks are seen by every later row, all other keys by `window`
// rows only.  A key-outer pass would give the few tiles with sinks many times
// the work of the rest; so rows further than a window behind such a tile are
// cut into `n_far` chunks of `far_rows` positions, each a work item that makes
// partial dK, dV of the sink rows (fp32, slot 1 + chunk; the tile's own item
// writes slot 0), which are then summed in slot order.
// far_rows is at least what an ordinary tile visits (window + one tile) and 512,
// so an item costs about as much as an ordinary one; no split where the sinks
// fill more than two 128-key tiles (those give parallelism of their own, and the partial sums
// would not be small) or the far rows fit one chunk twice over.
struct FarSplit {
    int n_far, far_rows;
};
inline FarSplit far_split(int Nk, int window, int sinks) {
    FarSplit f{0, 0};
    if (sinks <= 0 || sinks > 256) return f;
    const long long far = (long long)Nk - window;
    int rows = window + 128 > 512 ? window + 128 : 512;
    if (far < 2ll * rows) return f;
    if ((far + rows - 1) / rows > 64) rows = (int)((far + 63) / 64);
    f.far_rows = (rows + 127) / 128 * 128;
    f.n_far = (int)((far + f.far_rows - 1) / f.far_rows);
    return f;
}
inline size_t part_floats(const Args& a, const FarSplit& f) {
    return f.n_far ? (size_t)a.B * a.Hkv * (1 + f.n_far) * 2 * a.sinks * a.d : 0;
}

// Rows of the statistics arrays: whole 128-row tiles.
inline int stat_rows(int Nq) { return (Nq + 127) / 128 * 128; }

// Kernel launches; 0 or a psa_status with *err set.
int warp_fwd(const Args& a, std::string* err);
int warp_bwd(const Args& a, std::string* err);
// a.Drow and a.negl (any layout, both dtypes)
int pre_d(const Args& a, std::string* err);
// Tensor-core kernels (bf16, every view in tc_view's layout, scale > 0).
int tc_fwd(const Args& a, std::string* err);
int tc_fwd_take_error(std::string* err);
int tc_bwd(const Args& a, std::string* err);
int tc_bwd_take_error(std::string* err);
// dK, dV rows j < sinks from the partial sums
int sum_far(const Args& a, const FarSplit& f, std::string* err);

// A launch that may start while the kernel before it still runs (programmatic
// dependent launch); a plain one while kernels are timed one by one.
template <typename... P>
cudaError_t launch_beside(void (*kernel)(P...), unsigned grid, int threads, int cluster, int smem, cudaStream_t st,
                          const std::common_type_t<P>&... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at[2];
    cfg.attrs = at;
    if (!prof_enabled()) {
        at[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        at[cfg.numAttrs++].val.programmaticStreamSerializationAllowed = 1;
    }
    if (cluster > 1) {
        at[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
        at[cfg.numAttrs++].val.clusterDim = {(unsigned)cluster, 1, 1};
    }
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

struct DecodeArgs {
    const void* k;
    const void* v;
    int B, Hq, Hkv, cap, d, window, sinks, dtype;
    long long sB, sH, sS;
    View q, o;
    float* lse;
    const int* lens;
    float scale;
    void* workspace;
    cudaStream_t stream;
};
size_t decode_workspace(int B, int Hq, int Hkv, int d, int window, int sinks, int dtype);
int decode(const DecodeArgs& a, std::string* err);

// New tokens over the cache (win_tree.cu): a tree or run of drafts (drafts = 1), or the
// cache's newest token (drafts = 0, T = 1).
struct TreeArgs {
    const void* k;
    const void* v;
    const float* ks;             // 8-bit caches: scales, else NULL
    const float* vs;
    int B, Hq, Hkv, cap, d, window, sinks, dtype, cache_dtype;
    long long sB, sH, sS, cB, cH, cS;
    View q, o, kn, vn;
    float* lse;
    int T, drafts;
    const int* lens;
    const int* n_new;
    const int* parents;
    long long par_stride;
    float scale;
    void* workspace;
    cudaStream_t stream;
};
// How a call's rows and keys are cut: groups (sequence, key head, 16 wr or, wr = 0, 8 rows), each in
// `splits` runs of keys.
struct TreeSplit {
    long long groups;
    int wr, rgroups, splits;
};
size_t tree_workspace(const TreeArgs& a);
int tree(const TreeArgs& a, std::string* err);
size_t tree_tc_workspace(const TreeArgs& a);                                   // win_tree_tc.cu
int tree_tc(const TreeArgs& a, std::string* err);
int tree_tc_take_error(std::string* err);
int tree_bf16(const TreeArgs& a, const TreeSplit& s, std::string* err);        // one per pair of types
int tree_f32(const TreeArgs& a, const TreeSplit& s, std::string* err);
int tree_bf16_8(const TreeArgs& a, const TreeSplit& s, std::string* err);
int tree_f32_8(const TreeArgs& a, const TreeSplit& s, std::string* err);

struct RopeArgs {
    const psa_rope_plan* plan;
    View x[2], y[2];
    int heads[2];
    int n;               // tensors: 1 or 2
    int B, N;
    const int* pos;
    long long pos_axis, pos_batch;
    bool inverse;
    int dtype;
    cudaStream_t stream;
};
int rope(const RopeArgs& a, std::string* err);

struct AppendArgs {
    const psa_rope_plan* plan;   // NULL: keys are copied
    void* k;
    void* v;
    int B, Hkv, cap, d, sinks, dtype;
    long long sB, sH, sS;
    View kn, vn;
    int T;                       // positions per sequence at most
    const int* start;
    const int* n_new;
    const int* rows;             // NULL, or the rows of kn, vn to take: [B, T] of 0 .. n_rows - 1
    long long rows_stride;
    int n_rows;
    const int* pos;
    long long pos_axis, pos_batch;
    float* ks;                   // 8-bit caches (win_store.cu): scales, their strides
    float* vs;
    long long cB, cH, cS;
    cudaStream_t stream;
};
int append(const AppendArgs& a, std::string* err);
int append_8(const AppendArgs& a, std::string* err);

struct ReadArgs {
    const void* k;
    const void* v;
    const float* ks;
    const float* vs;
    int B, Hkv, cap, d, sinks, dtype, cache_dtype;
    long long sB, sH, sS, cB, cH, cS;
    View ko, vo;
    int N;
    const int* first;
    const int* lens;
    cudaStream_t stream;
};
int read(const ReadArgs& a, std::string* err);

}  // namespace win
}  // namespace psa
