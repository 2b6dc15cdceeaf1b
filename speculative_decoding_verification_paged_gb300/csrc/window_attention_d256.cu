// Instances of the windowed attention over a 16-bit cache for head dim 256.
#include "window_attention_launch.h"

namespace specv {
namespace wattn {

template <>
int settings_16<256>(int packed, bool fp16, int batch, Launch* l) {
  auto fn = [&](auto c) { return settings_of<decltype(c)>(batch, l); };
  return fp16 ? with_rows<256, true>(packed, fn) : with_rows<256, false>(packed, fn);
}
template <>
int launch_16<256>(int packed, bool fp16, const Launch& l, const Call& call) {
  auto fn = [&](auto c) { return launch_of<decltype(c)>(l, call); };
  return fp16 ? with_rows<256, true>(packed, fn) : with_rows<256, false>(packed, fn);
}

}  // namespace wattn
}  // namespace specv
