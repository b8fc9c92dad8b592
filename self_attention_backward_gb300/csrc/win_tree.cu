// win_tree.cu -- dispatch of the attention of new tokens over the rolling cache.
#include <algorithm>

#include "win_internal.h"

namespace psa {
namespace win {
namespace {

// 8 (over 8-bit caches), 16, 32 or 64 rows a block, whatever holds all of a key head's rows.
// Keys are cut so that six blocks per SM even out unequal lengths (912 = 152 * 6; 64 single tokens over
// 4100 8-bit slots: 108 us, with 456 115, with 1824 108), but a run has at least 128 keys (one token
// over 1024: 10.3 us, with 64 12.4), in fp32, whose products take longer, 64 (2 trees of 17 drafts over
// 333: 13.0 us, with 128 15.0).  9 to 16 runs are done as 8, which a cluster joins.
TreeSplit split_of(const TreeArgs& a) {
    TreeSplit s{};
    const long long rows = (long long)a.T * (a.Hq / a.Hkv);
    const bool cols = a.cache_dtype == PSA_E4M3 && a.dtype == PSA_BF16 && rows <= 8;
    s.wr = cols ? 0 : rows <= 16 ? 1 : rows <= 32 ? 2 : 4;
    s.rgroups = cols ? 1 : (int)((rows + 16 * s.wr - 1) / (16 * s.wr));
    s.groups = (long long)a.B * a.Hkv * s.rgroups;
    const int least = a.dtype == PSA_F32 ? 64 : 128;
    const long long want = (912 + s.groups - 1) / s.groups, most = ((long long)a.sinks + a.window + least - 1) / least;
    s.splits = (int)std::max(1ll, std::min(want, most));
    if (s.splits > 8 && s.splits <= 16) s.splits = 8;
    return s;
}

}  // namespace

size_t tree_workspace(const TreeArgs& a) {
    const TreeSplit s = split_of(a);
    return s.splits > 8 ? (size_t)s.groups * s.splits * (s.wr ? 16 * s.wr : 8) * (a.d + 2) * 4 : 0;
}

int tree(const TreeArgs& a, std::string* err) {
    const TreeSplit s = split_of(a);
    if (a.cache_dtype == PSA_E4M3) return a.dtype == PSA_F32 ? tree_f32_8(a, s, err) : tree_bf16_8(a, s, err);
    return a.dtype == PSA_F32 ? tree_f32(a, s, err) : tree_bf16(a, s, err);
}

}  // namespace win
}  // namespace psa
