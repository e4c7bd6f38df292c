// The chunked state space scan for float tensors.
#include "scan_chunks.h"

namespace bl {
template hipError_t launch_scan_chunks<float>(const ScanArgs &, int, hipStream_t);
}  // namespace bl
