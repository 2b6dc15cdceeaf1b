// Instances of the attention over a 4-bit cache for head dim 128.
#include "window_attention_launch.h"

namespace specv {
namespace wattn {

template <>
int settings_q4<128>(int packed, int batch, Launch* l) {
  return with_rows<128, true, true>(packed, [&](auto c) { return settings_of<decltype(c)>(batch, l); });
}
template <>
int launch_q4<128>(int packed, const Launch& l, const Call& call) {
  return with_rows<128, true, true>(packed, [&](auto c) { return launch_of<decltype(c)>(l, call); });
}

}  // namespace wattn
}  // namespace specv
