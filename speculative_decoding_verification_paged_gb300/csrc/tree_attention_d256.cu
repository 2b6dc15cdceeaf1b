// Instances of the tree attention's kernels for head dim 256.
#include "tree_attention_launch.cuh"

namespace specv {
namespace tattn {

template int settings<256>(int, int, bool, int, Launch*);
template int launch<256>(int, int, bool, const Launch&, const Call&);

}  // namespace tattn
}  // namespace specv
