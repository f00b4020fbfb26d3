// Instances of the tree kernel for fp32 inputs.
#include "lsq_tree_impl.h"

namespace lsq {

hipError_t launch_tree_f32(const TreeArgs& a, int dk, int delta, int diag, hipStream_t s) {
  return launch_tree_type<IO_F32>(a, dk, delta, diag, s);
}

}  // namespace lsq
