// Expert selection from bf16 and fp16 logits.
#define MOE_SELECT_FP32 false
#include "select.cuh"

namespace moe {

cudaError_t launch_select_16(const Select& c, const void* logits, const float* bias, int32_t* idx, float* w,
                             cudaStream_t s) {
  return forward(c, logits, bias, idx, w, s);
}

cudaError_t launch_select_bwd_16(const Select& c, const void* logits, const int32_t* idx, const float* dw, void* dl,
                                 cudaStream_t s) {
  return backward(c, logits, idx, dw, dl, s);
}

}  // namespace moe
