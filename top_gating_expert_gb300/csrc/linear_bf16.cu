// The linear layer's tensor-core products (linear_bf16.cuh) with its epilogue.
#include "linear_bf16.cuh"

namespace moe {

int launch_linear_bf16(const LinearOperand& A, const LinearOperand& B, int rows, int cols, int K,
                       const LinearEpi& e, unsigned* status, cudaStream_t st) {
  return run_product<kProduct>(A, B, rows, cols, K, e, NoExtra{}, status, st);
}

}  // namespace moe
