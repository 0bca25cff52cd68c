#include "serving.h"
namespace sa {
bool packed_tc_supported(const PackedArgs&) { return false; }
int launch_packed_tc(const PackedArgs&, cudaStream_t) { return -1; }
}  // namespace sa
