// attention.cu -- attention of new tokens over a paged cache of bf16
// (paged_attention): attention.cuh's kernels for bf16.
#include "attention.cuh"

namespace svw {

size_t attention_workspace(int64_t T, int32_t G, int32_t D) {
  const size_t rows = all_part_rows(T, G);
  return kJointBytes + kMarkBytes + round256(rows * sizeof(float2)) + rows * D * sizeof(float);
}

cudaError_t launch_attention(const AttendArgs &a, cudaStream_t st) { return launch_form<false>(a, st); }

}  // namespace svw
