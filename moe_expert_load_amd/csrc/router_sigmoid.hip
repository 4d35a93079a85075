// The router's forward kernels for sigmoid scores.
#include "router.hpp"

namespace moonep {
template int launch_forward<false>(const RouterArgs&, bool, bool, bool, int, hipStream_t);
}  // namespace moonep
