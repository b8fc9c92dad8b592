// win_tree_bf16.cu -- tree attention, bf16 queries over a bf16 cache (win_tree_warp.cuh).
#include "win_tree_warp.cuh"

namespace psa {
namespace win {

int tree_bf16(const TreeArgs& a, const TreeSplit& s, std::string* err) { return tk::launch<tk::bf16, tk::bf16>(a, s, err); }

}  // namespace win
}  // namespace psa
