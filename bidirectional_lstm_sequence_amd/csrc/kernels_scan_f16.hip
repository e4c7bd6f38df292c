// The chunked state space scan for _Float16 tensors.
#include "scan_chunks.h"

namespace bl {
template hipError_t launch_scan_chunks<_Float16>(const ScanArgs &, int, hipStream_t);
}  // namespace bl
