// linear_few_fp32.cu — the small matrix products in fp32: linear_few.cuh.
#include "linear_few.cuh"

namespace dr {

cudaError_t launch_linear_few_fp32(int tn, const lin::Operand& M, const lin::Operand& N, const lin::Epilogue& e, bool full,
                                 int split, cudaStream_t st) {
  return lin::few_by_tile<float>(tn, M, N, e, full, split, st);
}

}  // namespace dr
