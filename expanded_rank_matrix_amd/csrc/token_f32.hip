// Cross entropy through an output matrix: fp32.
#include "token.hpp"

namespace externd {

hipError_t token_run_f32(const TokenLaunch& L, hipStream_t st) { return token_typed<float>(L, st); }

}  // namespace externd
