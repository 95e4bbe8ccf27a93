// Cross entropy through an output matrix: bf16, and the choice of the type.
#include "token.hpp"

namespace externd {

size_t token_workspace_bytes(int x_type, long long rows, int n, int vocab, const void* W, long long ldw, bool loss, bool dX,
                             bool dW) {
  if (rows == 0) return 0;
  const int es = x_type == 0 ? 4 : 2;
  return token_plan(es, rows, n, vocab, token_aligned(W, ldw, n, es), loss, dX, dW).bytes;
}

hipError_t token_run(int x_type, const TokenLaunch& L, hipStream_t st) {
  switch (x_type) {
    case 0: return token_run_f32(L, st);
    case 1: return token_run_f16(L, st);
    case 2: return token_typed<__bf16>(L, st);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace externd
