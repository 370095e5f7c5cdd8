// attention_fp8.cu -- attention of new tokens over a paged cache of e4m3 codes
// (paged_attention_fp8): attention.cuh's kernels for codes.
#include "attention.cuh"

namespace svw {

cudaError_t launch_attention_fp8(const AttendArgs &a, cudaStream_t st) { return launch_form<true>(a, st); }

}  // namespace svw
