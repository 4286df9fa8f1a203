// cbk_nn_fused.h for index width 10.
#include "cbk_nn_fused.h"

namespace cbk {
template cbk_status launch_fused<10>(const FusedArgs &, uint32_t, bool, hipStream_t);
}  // namespace cbk
