// The gradient of leave_enter (hcb_leave_bwd.cuh).
#include "hcb_leave_bwd.cuh"

namespace hcb {

cudaError_t leave_enter_backward(const Params& p, int x_bf16, int y_bf16, bool vec, int* rows, cudaStream_t s) {
  return by_streams(p.S, x_bf16, y_bf16, vec, Backward<true>{p, rows, s});
}

}  // namespace hcb
