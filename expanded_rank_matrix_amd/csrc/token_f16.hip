// Cross entropy through an output matrix: fp16.
#include "token.hpp"

namespace externd {

hipError_t token_run_f16(const TokenLaunch& L, hipStream_t st) { return token_typed<_Float16>(L, st); }

}  // namespace externd
