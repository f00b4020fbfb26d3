// Instances of the tree kernel for binary16 inputs.
#include "lsq_tree_impl.h"

namespace lsq {

hipError_t launch_tree_f16(const TreeArgs& a, int dk, int delta, int diag, hipStream_t s) {
  return launch_tree_type<IO_F16>(a, dk, delta, diag, s);
}

}  // namespace lsq
