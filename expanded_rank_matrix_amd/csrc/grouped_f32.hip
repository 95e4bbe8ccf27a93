// Products with 4-bit weights: fp32 tokens.
#include "grouped.hpp"

namespace externd {

hipError_t grouped_run_f32(const GroupedLaunch& L, hipStream_t st) { return grouped_typed<float>(L, st); }

}  // namespace externd
