// win_tree_f32.cu -- tree attention, fp32 queries over an fp32 cache (win_tree_warp.cuh).
#include "win_tree_warp.cuh"

namespace psa {
namespace win {

int tree_f32(const TreeArgs& a, const TreeSplit& s, std::string* err) { return tk::launch<float, float>(a, s, err); }

}  // namespace win
}  // namespace psa
