// Instances of the attention over a 4-bit cache for head dim 256.
#include "q4_attention_launch.h"

namespace specv {
namespace qattn {

template <>
int launch<256>(const spec_attn_desc* d, int all, const Params& p, cudaStream_t stream) {
  return with_rows<256>(all, [&](auto c) { return launch_of<decltype(c)>(d, p, stream); });
}
template <>
size_t workspace<256>(const spec_attn_desc* d, int rows, int all) {
  return with_rows<256>(all, [&](auto c) { return workspace_of<decltype(c)>(d, rows); });
}

}  // namespace qattn
}  // namespace specv
