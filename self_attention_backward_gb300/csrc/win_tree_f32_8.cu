// win_tree_f32_8.cu -- tree attention, fp32 queries over an e4m3 cache (win_tree_warp.cuh).
#include "win_tree_warp.cuh"

namespace psa {
namespace win {

int tree_f32_8(const TreeArgs& a, const TreeSplit& s, std::string* err) { return tk::launch<float, tk::e4m3>(a, s, err); }

}  // namespace win
}  // namespace psa
