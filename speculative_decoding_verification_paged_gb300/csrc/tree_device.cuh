// The tree of drafts shared by the tree calls: what makes a parent table valid
// and which nodes a node sees.
#pragma once

#include <stdint.h>

#include "common.cuh"

namespace specv {
namespace tree {

constexpr int kMaxNodes = 64;  // a node's ancestors fit one 64-bit word

// Whether two arrays share a byte (host).
inline bool overlap(const void* a, size_t a_bytes, const void* b, size_t b_bytes) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + b_bytes && y < x + a_bytes;
}

// Whether entry i of the parent table `par` (any readable pointer) is allowed: unused, without a
// parent, or the child of an earlier used node; node 0 has no parent.
template <typename T>
__device__ __forceinline__ bool parent_ok(const T* par, int i) {
  const int p = par[i];
  if (p == SPEC_TREE_UNUSED || p == SPEC_TREE_ROOT) return true;
  return p >= 0 && p < i && par[p] != SPEC_TREE_UNUSED;
}

// Bit j set: node i sees node j, i itself and its ancestors; 0 for an unused node. The walk goes to
// ever smaller indices, so it ends whatever the table holds.
template <typename T>
__device__ __forceinline__ uint64_t ancestors(const T* par, int i) {
  int p = par[i];
  if (p == SPEC_TREE_UNUSED) return 0;
  uint64_t m = 1ull << i;
  for (int at = i; p >= 0 && p < at;) {
    m |= 1ull << p;
    at = p;
    p = par[p];
  }
  return m;
}

}  // namespace tree
}  // namespace specv
