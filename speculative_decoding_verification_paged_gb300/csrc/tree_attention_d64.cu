// Instances of the tree attention's kernels for head dim 64.
#include "tree_attention_launch.cuh"

namespace specv {
namespace tattn {

template int settings<64>(int, int, bool, int, Launch*);
template int launch<64>(int, int, bool, const Launch&, const Call&);

}  // namespace tattn
}  // namespace specv
