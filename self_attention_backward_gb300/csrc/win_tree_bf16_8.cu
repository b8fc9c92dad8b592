// win_tree_bf16_8.cu -- tree attention, bf16 queries over an e4m3 cache (win_tree_warp.cuh).
#include "win_tree_warp.cuh"

namespace psa {
namespace win {

int tree_bf16_8(const TreeArgs& a, const TreeSplit& s, std::string* err) { return tk::launch<tk::bf16, tk::e4m3>(a, s, err); }

}  // namespace win
}  // namespace psa
