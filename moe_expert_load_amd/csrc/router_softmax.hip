// The router's forward kernels for softmax scores.
#include "router.hpp"

namespace moonep {
template int launch_forward<true>(const RouterArgs&, bool, bool, bool, int, hipStream_t);
}  // namespace moonep
