// Products in 8-bit integers with a scale for each token and each output channel, and the
// quantisation of rows that makes their operands.
//
//   quantise:  a_t = max_j |x_tj|,  s_t = fl32(a_t / 127),  q_tj = the whole number nearest to the
//              exact quotient 127 x_tj / a_t, ties to even
//   product:   y_to = s_t w_o sum_j q_tj W_oj
//
// The sum is exact in int32 (n <= 131071), so it does not depend on how it is split; it is converted
// to fp32 and multiplied by the two scales (three fp32 roundings), then rounded once to Y's type.
#include "common.hpp"
#include "externd_internal.hpp"
#include "igemm.hpp"
#include "types.hpp"

namespace externd {

// ---- quantisation of rows ---------------------------------------------------------------------
// q = rint(127 x / a) of the exact quotient.  The fp32 estimate x fl(127 / a) is off by less than
// 127 2^-22.9 < 2^-15: only an estimate that close to a border between two whole numbers can round
// to the wrong side, and those few are redone in fp64, whose rounded quotient is never on the wrong
// side: 254 x and (2 q + 1) a are 32-bit integers times a power of two, so a quotient that is no
// tie is at least 2^-25 from one.
__device__ __forceinline__ int quant1(float x, float inv, float a) {
  const float r = x * inv;
  float q = rintf(r);
  if (fabsf(r - q) > 0.5f - 0x1p-14f) q = (float)rint(127.0 * (double)x / (double)a);
  return (int)q;
}
// rows whose largest value is so small that 127 / a overflows (or nears it) take fp64 throughout
__device__ __forceinline__ int quant1_small(float x, float a) { return (int)rint(127.0 * (double)x / (double)a); }

__device__ __forceinline__ unsigned pack4(int a, int b, int c, int d) {
  return (unsigned)(a & 255) | (unsigned)(b & 255) << 8 | (unsigned)(c & 255) << 16 | (unsigned)d << 24;
}

// One row per TPR threads (64: a wave; 256: the workgroup), 8 elements per thread and step; the
// first CH steps of a row stay in registers between the search for its maximum and its rounding, a
// longer row's rest is read again.  np bytes of each Q row are written, zeros behind the first n.
// A row with a NaN or an infinity gets scale NaN and q = 0.
template <typename T, int TPR, int CH>
__global__ void __launch_bounds__(256) quantize_kernel(const T* __restrict__ X, long long rows, int n, long long ldx,
                                                       int8_t* __restrict__ Q, long long ldq, int np,
                                                       float* __restrict__ scale) {
  constexpr int RPW = 256 / TPR;
  __shared__ unsigned wmx[4];
  const int tid = threadIdx.x % TPR;
  const long long row = (long long)blockIdx.x * RPW + threadIdx.x / TPR;
  const long long rr = row < rows ? row : rows - 1;
  const T* x = X + rr * ldx;
  float v[CH][8];
  unsigned mx = 0u;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int j = (c * TPR + tid) * 8;
    if (j + 8 <= n) load8(x + j, v[c]);
    else load8_tail(x + j, (long long)n - j, v[c]);
  }
#pragma unroll
  for (int c = 0; c < CH; ++c)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const unsigned b = __float_as_uint(v[c][e]) & 0x7FFFFFFFu;
      mx = b > mx ? b : mx;
    }
  for (long long j = (long long)(CH * TPR + tid) * 8; j < n; j += TPR * 8) {
    float w[8];
    if (j + 8 <= n) load8(x + j, w);
    else load8_tail(x + j, n - j, w);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const unsigned b = __float_as_uint(w[e]) & 0x7FFFFFFFu;
      mx = b > mx ? b : mx;
    }
  }
  mx = wave_max_u32(mx);
  if (TPR == 256) {
    if ((threadIdx.x & 63) == 0) wmx[threadIdx.x >> 6] = mx;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 4; ++w) mx = wmx[w] > mx ? wmx[w] : mx;
  }
  if (row >= rows) return;
  const bool bad = mx >= 0x7F800000u;
  const float a = __uint_as_float(mx);
  const bool tiny = mx < 0x0D000000u;  // a < 2^-101
  const float inv = bad || mx == 0u ? 0.0f : 127.0f / a;
  if (tid == 0) scale[row] = bad ? __uint_as_float(0x7FC00000u) : a / 127.0f;
  int8_t* q = Q + row * ldq;
  auto emit = [&](long long j, const float (&w)[8]) {
    int k[8];
    if (bad || mx == 0u) {
#pragma unroll
      for (int e = 0; e < 8; ++e) k[e] = 0;
    } else if (tiny) {
#pragma unroll
      for (int e = 0; e < 8; ++e) k[e] = quant1_small(w[e], a);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) k[e] = quant1(w[e], inv, a);
    }
    if (j + 8 <= np) {
      iv2_any o;
      o[0] = (int)pack4(k[0], k[1], k[2], k[3]);
      o[1] = (int)pack4(k[4], k[5], k[6], k[7]);
      *reinterpret_cast<iv2_any*>(q + j) = o;
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (j + e < np) q[j + e] = (int8_t)k[e];
    }
  };
#pragma unroll
  for (int c = 0; c < CH; ++c) emit((long long)(c * TPR + tid) * 8, v[c]);
  for (long long j = (long long)(CH * TPR + tid) * 8; j < np; j += TPR * 8) {
    float w[8];
    if (j + 8 <= n) load8(x + j, w);
    else load8_tail(x + j, n - j, w);
    emit(j, w);
  }
}

template <typename T>
static hipError_t quantize_typed(const T* X, long long rows, int n, long long ldx, int8_t* Q, long long ldq, int np,
                                 float* scale, hipStream_t st) {
  if (n <= 64 * 8 * 2) {
    hipLaunchKernelGGL((quantize_kernel<T, 64, 2>), dim3((unsigned)((rows + 3) / 4)), dim3(256), 0, st, X, rows, n, ldx,
                       Q, ldq, np, scale);
  } else {
    hipLaunchKernelGGL((quantize_kernel<T, 256, 5>), dim3((unsigned)rows), dim3(256), 0, st, X, rows, n, ldx, Q, ldq,
                       np, scale);
  }
  return hipGetLastError();
}

hipError_t quantize_run(const void* X, int type, long long rows, int n, long long ldx, int8_t* Q, long long ldq, int np,
                        float* scale, hipStream_t st) {
  switch (type) {
    case 0: return quantize_typed(static_cast<const float*>(X), rows, n, ldx, Q, ldq, np, scale, st);
    case 1: return quantize_typed(static_cast<const _Float16*>(X), rows, n, ldx, Q, ldq, np, scale, st);
    case 2: return quantize_typed(static_cast<const __bf16*>(X), rows, n, ldx, Q, ldq, np, scale, st);
    default: return hipErrorInvalidValue;
  }
}

template <typename T>
__device__ __forceinline__ void store_y(T* p, float v) {
  *p = (T)v;
}

// ---- few tokens -------------------------------------------------------------------------------
// Workgroup: 16 output channels and 16 NT tokens, the row length split over eight waves
// in steps of 64 bytes.  MFMA D(16 x 16) += A(16 x 64) B(64 x 16): A row = channel, B column =
// token, lane l holding the 16 bytes at 16 (l / 16) of row (column) l % 16 of the step.  The waves'
// partial tiles add in LDS.
constexpr int kFewWaves = 8;
template <int NT, typename YT>
__global__ void __launch_bounds__(64 * kFewWaves) few_kernel(const int8_t* __restrict__ W, long long ldw, int m, int n,
                                                             const float* __restrict__ sw,
                                                             const int8_t* __restrict__ Xq, long long ldx, int tokens,
                                                             const float* __restrict__ sx, YT* __restrict__ Y,
                                                             long long ldy) {
  __shared__ int red[kFewWaves][NT * 256];
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6, lr = lane & 15, gg = lane >> 4;
  const int r0 = blockIdx.x * 16;
  const long long t0 = blockIdx.y * (16ll * NT);
  const int r = r0 + lr < m ? r0 + lr : m - 1;
  const int8_t* wr = W + (long long)r * ldw;
  const int8_t* xr[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const long long c = t0 + 16 * t + lr < tokens ? t0 + 16 * t + lr : tokens - 1;
    xr[t] = Xq + c * ldx;
  }
  iv4 acc[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) acc[t] = iv4{0, 0, 0, 0};
  const int full = n / 64;
  int s = wv;
  constexpr int U = 4;
  for (; s + (U - 1) * kFewWaves < full; s += U * kFewWaves) {
    iv4 a[U], b[U][NT];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = 64 * (s + u * kFewWaves) + 16 * gg;
      a[u] = *reinterpret_cast<const iv4_any*>(wr + k);
#pragma unroll
      for (int t = 0; t < NT; ++t) b[u][t] = *reinterpret_cast<const iv4_any*>(xr[t] + k);
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int t = 0; t < NT; ++t) acc[t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(a[u], b[u][t], acc[t], 0, 0, 0);
  }
  if (n >= 16) {
    for (; 64 * s < n; s += kFewWaves) {
      const int k = 64 * s + 16 * gg;
      const iv4 a = row16(wr, k, n);
#pragma unroll
      for (int t = 0; t < NT; ++t)
        acc[t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(a, row16(xr[t], k, n), acc[t], 0, 0, 0);
    }
  } else if (s == 0) {
    const iv4 a = row16_short(wr, 16 * gg, n);
#pragma unroll
    for (int t = 0; t < NT; ++t)
      acc[t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(a, row16_short(xr[t], 16 * gg, n), acc[t], 0, 0, 0);
  }
  // acc[t][q] = D(channel 4 gg + q, token lr): stored token-major
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int q = 0; q < 4; ++q) red[wv][t * 256 + lr * 16 + 4 * gg + q] = acc[t][q];
  __syncthreads();
  for (int x = tid; x < NT * 256; x += 64 * kFewWaves) {
    const long long tok = t0 + (x >> 4);
    const int o = r0 + (x & 15);
    if (tok < tokens && o < m) {
      int sum = 0;
#pragma unroll
      for (int w = 0; w < kFewWaves; ++w) sum += red[w][x];
      store_y(Y + tok * ldy + o, (float)sum * sx[tok] * sw[o]);
    }
  }
}

// ---- many tokens: the tiles of igemm.hpp ----------------------------------------------------
// y = sum s_t w_o: the lane holds rows row + 8 (i / 4) + i % 4 of column col
template <typename YT>
struct ScaledY {
  const float* sx;
  const float* sw;
  YT* Y;
  long long ldy;
  struct Row {
    float s[16];
  };
  typedef float Col;
  __device__ __forceinline__ Row row(long long r, int M) const {
    Row o;
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const long long x = r + 8 * (e >> 2) + (e & 3);
      o.s[e] = sx[x < M ? x : M - 1];
    }
    return o;
  }
  __device__ __forceinline__ Col col(long long c) const { return sw[c]; }
  template <bool WHOLE>
  __device__ __forceinline__ void put(long long r, long long c, int M, int N, const Row& s, Col w,
                                      const iv16& acc) const {
    YT* y = Y + r * ldy + c;
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const int d = 8 * (e >> 2) + (e & 3);
      if (WHOLE || (r + d < M && c < N)) store_y(y + d * ldy, (float)acc[e] * s.s[e] * w);
    }
  }
};

template <typename YT>
static hipError_t product_typed(const int8_t* W, const float* sw, int m, int n, long long ldw, const int8_t* Xq,
                                const float* sx, int tokens, long long ldx, YT* Y, long long ldy, hipStream_t st) {
  const unsigned few = (unsigned)((m + 15ll) / 16);
  if (tokens <= 16) {
    hipLaunchKernelGGL((few_kernel<1, YT>), dim3(few), dim3(64 * kFewWaves), 0, st, W, ldw, m, n, sw, Xq, ldx, tokens,
                       sx, Y, ldy);
  } else if (tokens <= 32 || n < 16) {  // rows too short for the tiles' loads come here whatever their number
    const long long groups = (tokens + 31ll) / 32;
    for (long long g = 0; g < groups; g += 65535) {  // the grid's limit; one launch below 2 million tokens
      const unsigned gy = (unsigned)(groups - g < 65535 ? groups - g : 65535);
      const long long t0 = 32 * g;
      hipLaunchKernelGGL((few_kernel<2, YT>), dim3(few, gy), dim3(64 * kFewWaves), 0, st, W, ldw, m, n, sw,
                         Xq + t0 * ldx, ldx, (int)(tokens - t0), sx + t0, Y + t0 * ldy, ldy);
    }
  } else {
    return tile_product(Xq, ldx, tokens, W, ldw, m, n, ScaledY<YT>{sx, sw, Y, ldy}, st);
  }
  return hipGetLastError();
}

// Workspace of a product whose tokens come as floating-point rows: their scales and their
// quantised rows, padded to a multiple of 16 bytes.
static size_t al256(size_t x) { return (x + 255) & ~(size_t)255; }
static long long pad16(long long n) { return (n + 15) & ~15ll; }
size_t product_workspace_bytes(int x_type, long long tokens, int n) {
  return x_type == 3 ? 0 : al256((size_t)tokens * 4) + al256((size_t)tokens * pad16(n));
}

hipError_t product_run(const int8_t* W, const float* sw, int m, int n, long long ldw, const void* X, int x_type,
                       const float* sx, int tokens, long long ldx, void* Y, int y_type, long long ldy, void* ws,
                       hipStream_t st) {
  const int8_t* Xq = static_cast<const int8_t*>(X);
  if (x_type != 3) {
    float* scale = static_cast<float*>(ws);
    int8_t* q = static_cast<int8_t*>(ws) + al256((size_t)tokens * 4);
    const long long np = pad16(n);
    const hipError_t e = quantize_run(X, x_type, tokens, n, ldx, q, np, (int)np, scale, st);
    if (e != hipSuccess) return e;
    Xq = q;
    sx = scale;
    ldx = np;
  }
  switch (y_type) {
    case 0: return product_typed(W, sw, m, n, ldw, Xq, sx, tokens, ldx, static_cast<float*>(Y), ldy, st);
    case 1: return product_typed(W, sw, m, n, ldw, Xq, sx, tokens, ldx, static_cast<_Float16*>(Y), ldy, st);
    case 2: return product_typed(W, sw, m, n, ldw, Xq, sx, tokens, ldx, static_cast<__bf16*>(Y), ldy, st);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace externd
