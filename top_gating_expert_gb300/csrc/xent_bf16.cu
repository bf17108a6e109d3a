// The tensor-core products (linear_bf16.cuh) of the cross entropy of a linear head.
#include "linear_bf16.cuh"

namespace moe {

int launch_xent_bf16(ProductMode mode, const LinearOperand& A, const LinearOperand& B, int rows, int cols, int K,
                     const LinearEpi& e, const XentEpi& x, unsigned* status, cudaStream_t st) {
  switch (mode) {
    case kXentStats: return run_product<kXentStats>(A, B, rows, cols, K, e, x, status, st);
    case kXentGrad: return run_product<kXentGrad>(A, B, rows, cols, K, e, x, status, st);
    case kProductSum: return run_product<kProductSum>(A, B, rows, cols, K, e, x, status, st);
    case kProduct: break;
  }
  return MOE_ERR_INVALID_ARG;
}

}  // namespace moe
