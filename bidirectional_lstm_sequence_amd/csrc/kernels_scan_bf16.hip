// The chunked state space scan for __bf16 tensors.
#include "scan_chunks.h"

namespace bl {
template hipError_t launch_scan_chunks<__bf16>(const ScanArgs &, int, hipStream_t);
}  // namespace bl
