// Weights in 4 bits with a scale, and an offset, for each group of a row: their quantisation, the products for bf16
// tokens, and the choice of the type.
//
//   w_oj = s_og c_oj + o_og,  c in -8 .. 7,  g = j / group
//   y_to = sum_j w_oj x_tj
#include "grouped.hpp"

namespace externd {

// ---- quantisation -------------------------------------------------------------------------------
// The codes are the whole numbers nearest to quotients q = 7 w / a or 15 (w - lo) / (hi - lo).  The fp32
// estimate is off by less than 2^-18, so only one that close to a border between two whole numbers can round to
// the wrong side; those within 2^-14 are redone in fp64.
__device__ __forceinline__ int group_code(float x, float inv, double num, double den) {
  const float r = x * inv;
  float q = rintf(r);
  if (!(fabsf(r - q) <= 0.5f - 0x1p-14f)) q = (float)rint(num / den);
  return (int)q;
}

// A thread makes one word of eight codes, GROUP / 8 threads together a group.
template <typename T, int GROUP>
__global__ void __launch_bounds__(256) quantize_groups_kernel(const T* __restrict__ W, long long ldw, int n, int words,
                                                              long long total, int* __restrict__ Q, void* scale, void* offset,
                                                              int s_type) {
  constexpr int L = GROUP / 8;
  const long long x = (long long)blockIdx.x * 256 + threadIdx.x;
  const bool mine = x < total;
  const long long row = mine ? x / words : 0;
  const int j = mine ? (int)(x - row * words) * 8 : n, left = n - j;
  const T* w = W + row * ldw + j;
  float v[8];
  if (left >= 8) load8(w, v);
  else load8_tail(w, left, v);
  float lo = __builtin_inff(), hi = -__builtin_inff();
  bool bad = false;
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (e < left) {
      lo = fminf(lo, v[e]);
      hi = fmaxf(hi, v[e]);
      bad = bad || !(fabsf(v[e]) <= __FLT_MAX__);
    }
  int any = bad;
#pragma unroll
  for (int d = 1; d < L; d <<= 1) {
    lo = fminf(lo, __shfl_xor(lo, d));
    hi = fmaxf(hi, __shfl_xor(hi, d));
    any |= __shfl_xor(any, d);
  }
  if (!mine) return;
  const float a = fmaxf(fabsf(lo), fabsf(hi));
  const double d = (double)hi - (double)lo;
  const float num = offset ? 15.0f : 7.0f;
  const double den = offset ? d : (double)a;
  // an inverse that overflows, or a range that does, sends every element to fp64
  const float df = (float)den, inv = df >= 0x1p-100f && df <= __FLT_MAX__ ? num / df : __builtin_nanf("");
  unsigned word = 0;
  if (!any && den != 0.0) {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < left) {
        const int c = offset ? group_code(v[e] - lo, inv, 15.0 * ((double)v[e] - (double)lo), d) - 8
                             : group_code(v[e], inv, 7.0 * (double)v[e], (double)a);
        word |= (unsigned)(c & 15) << (4 * e);
      }
  }
  Q[x] = (int)word;
  if ((threadIdx.x & (L - 1)) == 0) {
    const long long g = x / L;
    const float nan = __builtin_nanf("");
    put_scale(scale, s_type, g, any ? nan : offset ? (float)(d / 15.0) : a / 7.0f);
    if (offset) put_scale(offset, s_type, g, any ? nan : (float)((double)lo + 8.0 * (d / 15.0)));
  }
}

template <typename T>
static hipError_t quantize_groups_typed(const T* W, long long rows, int n, long long ldw, int group, int* Q, void* scale,
                                        void* offset, int s_type, hipStream_t st) {
  const int words = (n + group - 1) / group * (group / 8), per = group / 8, es = s_type == 0 ? 4 : 2;
  // runs of rows whose threads a launch holds
  const long long run = (1ll << 31) / words > 0 ? (1ll << 31) / words : 1;
  for (long long r = 0; r < rows; r += run) {
    const long long total = (rows - r < run ? rows - r : run) * words, s = r * (words / per) * es;
    auto go = [&](auto kernel) {
      hipLaunchKernelGGL(kernel, dim3((unsigned)((total + 255) / 256)), dim3(256), 0, st, W + r * ldw, ldw, n, words, total,
                         Q + r * words, static_cast<char*>(scale) + s, offset ? static_cast<char*>(offset) + s : nullptr, s_type);
    };
    if (group == 32) go(quantize_groups_kernel<T, 32>);
    else if (group == 64) go(quantize_groups_kernel<T, 64>);
    else go(quantize_groups_kernel<T, 128>);
  }
  return hipGetLastError();
}

hipError_t quantize_groups_run(const void* W, int type, long long rows, int n, long long ldw, int group, int* Q, void* scale,
                               void* offset, int s_type, hipStream_t st) {
  switch (type) {
    case 0: return quantize_groups_typed(static_cast<const float*>(W), rows, n, ldw, group, Q, scale, offset, s_type, st);
    case 1: return quantize_groups_typed(static_cast<const _Float16*>(W), rows, n, ldw, group, Q, scale, offset, s_type, st);
    case 2: return quantize_groups_typed(static_cast<const __bf16*>(W), rows, n, ldw, group, Q, scale, offset, s_type, st);
    default: return hipErrorInvalidValue;
  }
}

// ---- products -----------------------------------------------------------------------------------
size_t grouped_workspace_bytes(int x_type, long long tokens, int n, int m, int group) {
  return x_type == 0 ? grouped_bytes<float>(tokens, n, m, group) : grouped_bytes<__bf16>(tokens, n, m, group);
}

hipError_t grouped_run(const GroupedLaunch& L, hipStream_t st) {
  switch (L.x_type) {
    case 0: return grouped_run_f32(L, st);
    case 1: return grouped_run_f16(L, st);
    case 2: return grouped_typed<__bf16>(L, st);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace externd
