// Expert selection from fp32 logits, and the choice between it and that from 16-bit ones.
#define MOE_SELECT_FP32 true
#include "select.cuh"

namespace moe {

cudaError_t launch_select(const Select& c, const void* logits, const float* bias, int32_t* idx, float* w, cudaStream_t s) {
  return c.dtype == MOE_FP32 ? forward(c, logits, bias, idx, w, s) : launch_select_16(c, logits, bias, idx, w, s);
}

cudaError_t launch_select_bwd(const Select& c, const void* logits, const int32_t* idx, const float* dw, void* dl,
                              cudaStream_t s) {
  return c.dtype == MOE_FP32 ? backward(c, logits, idx, dw, dl, s) : launch_select_bwd_16(c, logits, idx, dw, dl, s);
}

}  // namespace moe
