// Products with 4-bit weights: fp16 tokens.
#include "grouped.hpp"

namespace externd {

hipError_t grouped_run_f16(const GroupedLaunch& L, hipStream_t st) { return grouped_typed<_Float16>(L, st); }

}  // namespace externd
