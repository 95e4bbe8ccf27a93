// Gradient of a layer held as packed ternary factors, y = B diag(D) C x, over a batch:
//   u_b = B^T dy_b,   t_b = C x_b,   dD_i = sum_b t_bi u_bi,   dx_b = C^T (D u_b)
//
// Few vectors go through the inference kernels (apply.hip).  A larger batch is three products of
// 8-bit integers (igemm.hpp): each vector enters as four rows of signed 8-bit digits of a
// fixed-point image with its own power-of-two scale, N = rint(x 2^(30 - E)), |x| < 2^E for the
// whole vector, N = d0 + 2^8 d1 + 2^16 d2 + 2^24 d3; the factors' codes are widened to bytes.  A
// digit's sum is exact in int32 (lengths below 2^24), the four are joined in int64, scaled and
// rounded once to fp32: the image's rounding, 2^-31 of the vector's largest power of two, is the
// only error of a product besides.  t u and its sum over the batch are fp64, in a fixed order.
#include <algorithm>

#include "common.hpp"
#include "externd_internal.hpp"
#include "igemm.hpp"
#include "types.hpp"

namespace externd {

constexpr int kGChunk = 4096;       // vectors per pass over the factors (bounds the workspace)
constexpr int kGFew = 16;           // batches up to this take the inference kernels
constexpr int kGParts = 32;         // partial sums of dD
constexpr int kGBad = 0x7FFFFFFF;   // exponent of a vector with a NaN or an infinity

static size_t al256(size_t x) { return (x + 255) & ~(size_t)255; }
static long long pad16(long long n) { return (n + 15) & ~15ll; }

// four 2-bit codes (0 -> 0, 1 -> 1, 3 -> -1) of the low byte as four signed bytes
__device__ __forceinline__ unsigned widen4(unsigned x) {
  x = (x | x << 12) & 0x000F000Fu;
  x = (x | x << 6) & 0x03030303u;
  return __builtin_amdgcn_perm(0u, 0xFF000100u, x);  // byte i of the result is byte x_i of 00 01 00 FF
}

// packed rows -> bytes: out[r][16 w .. 16 w + 15] = the codes of word w
__global__ void __launch_bounds__(256) widen_kernel(const uint32_t* __restrict__ P, long long words,
                                                    int8_t* __restrict__ out) {
  const long long x = (long long)blockIdx.x * 256 + threadIdx.x;
  if (x >= words) return;
  const unsigned w = P[x];
  const iv4 v = {(int)widen4(w & 255u), (int)widen4(w >> 8 & 255u), (int)widen4(w >> 16 & 255u), (int)widen4(w >> 24)};
  *reinterpret_cast<iv4*>(out + 16 * x) = v;
}

// packed rows -> bytes of the transpose: out[j][i] = code j of row i, i < kp (zeros from k on).
// Workgroup: 256 rows x 16 words; thread: 16 rows of one word.
__global__ void __launch_bounds__(256) widen_t_kernel(const uint32_t* __restrict__ P, int k, int words, int n,
                                                      int8_t* __restrict__ out, long long kp) {
  __shared__ unsigned tile[256 * 17];
  const int tid = threadIdx.x;
  const long long i0 = (long long)blockIdx.x * 256, w0 = (long long)blockIdx.y * 16;
#pragma unroll
  for (int u = 0; u < 16; ++u) {
    const int r = (tid >> 4) + 16 * u, c = tid & 15;
    tile[r * 17 + c] = i0 + r < k && w0 + c < words ? P[(i0 + r) * words + w0 + c] : 0u;
  }
  __syncthreads();
  const int g = tid & 15, c = tid >> 4;
  unsigned w[16];
#pragma unroll
  for (int r = 0; r < 16; ++r) w[r] = tile[(16 * g + r) * 17 + c];
  const long long i = i0 + 16 * g;
  if (i >= kp) return;
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    const long long j = 16 * (w0 + c) + e;
    iv4 v;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      unsigned x = (w[4 * q] >> 2 * e & 3u) | (w[4 * q + 1] >> 2 * e & 3u) << 8 | (w[4 * q + 2] >> 2 * e & 3u) << 16 |
                   (w[4 * q + 3] >> 2 * e & 3u) << 24;
      v[q] = (int)__builtin_amdgcn_perm(0u, 0xFF000100u, x);
    }
    if (j < n) *reinterpret_cast<iv4*>(out + j * kp + i) = v;
  }
}

// digits of four values: word q holds digit q of values 0..3 (bytes 0..3)
__device__ __forceinline__ void digits4(const float (&x)[4], int sh, unsigned (&w)[4]) {
  unsigned b[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) b[e] = ((unsigned)__float2int_rn(ldexpf(x[e], sh)) + 0x00808080u) ^ 0x00808080u;
  const unsigned l01 = __builtin_amdgcn_perm(b[1], b[0], 0x05010400u);  // b0.0 b1.0 b0.1 b1.1
  const unsigned h01 = __builtin_amdgcn_perm(b[1], b[0], 0x07030602u);  // b0.2 b1.2 b0.3 b1.3
  const unsigned l23 = __builtin_amdgcn_perm(b[3], b[2], 0x05010400u);
  const unsigned h23 = __builtin_amdgcn_perm(b[3], b[2], 0x07030602u);
  w[0] = __builtin_amdgcn_perm(l23, l01, 0x05040100u);
  w[1] = __builtin_amdgcn_perm(l23, l01, 0x07060302u);
  w[2] = __builtin_amdgcn_perm(h23, h01, 0x05040100u);
  w[3] = __builtin_amdgcn_perm(h23, h01, 0x07060302u);
}

// One vector a workgroup: x (times D where given) -> digit rows 4 b .. 4 b + 3 of np bytes, and the
// exponent E - 30 of its image's unit.
__global__ void __launch_bounds__(256) digits_kernel(const float* __restrict__ X, long long n,
                                                     const float* __restrict__ D, int8_t* __restrict__ out,
                                                     long long np, int* __restrict__ ex) {
  __shared__ unsigned wmx[4];
  const long long b = blockIdx.x;
  const float* x = X + b * n;
  auto get = [&](long long j, float (&v)[4]) {
    if (j + 4 <= n) {
      const iv4 a = *reinterpret_cast<const iv4_any*>(x + j);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = __int_as_float(a[e]);
      if (D) {
        const iv4 d = *reinterpret_cast<const iv4_any*>(D + j);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] *= __int_as_float(d[e]);
      }
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = j + e < n ? (D ? x[j + e] * D[j + e] : x[j + e]) : 0.0f;
    }
  };
  unsigned mx = 0u;
  for (long long j = 4 * threadIdx.x; j < n; j += 1024) {
    float v[4];
    get(j, v);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const unsigned a = __float_as_uint(v[e]) & 0x7FFFFFFFu;
      mx = a > mx ? a : mx;
    }
  }
  mx = wave_max_u32(mx);
  if ((threadIdx.x & 63) == 0) wmx[threadIdx.x >> 6] = mx;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 4; ++w) mx = wmx[w] > mx ? wmx[w] : mx;
  const bool bad = mx >= 0x7F800000u;
  const int E = mx >> 23 ? (int)(mx >> 23) - 126 : -126;  // |x| < 2^E
  const int sh = 30 - E;
  if (threadIdx.x == 0) ex[b] = bad ? kGBad : -sh;
  int8_t* o = out + 4 * b * np;
  for (long long j = 4 * threadIdx.x; j < np; j += 1024) {
    float v[4];
    unsigned w[4] = {0u, 0u, 0u, 0u};
    get(j, v);
    if (!bad) digits4(v, sh, w);
#pragma unroll
    for (int q = 0; q < 4; ++q) *reinterpret_cast<unsigned*>(o + q * np + j) = w[q];
  }
}

// rows 4 b .. 4 b + 3 of a product are one vector's digits: out[b][col] = 2^e sum_q 2^(8 q) row_q
struct JoinDigits {
  const int* ex;
  float* out;
  long long ld;
  static constexpr bool kLds = false;
  struct Row {
    int e[4];
  };
  __device__ __forceinline__ void at(long long m0, long long n0) {
    ex += m0 >> 2;
    out += (m0 >> 2) * ld + n0;
  }
  __device__ __forceinline__ Row row(int r, int mr) const {
    Row o;
#pragma unroll
    for (int i = 0; i < 4; ++i) o.e[i] = ex[(r + 8 * i < mr ? r + 8 * i : mr - 1) >> 2];
#pragma unroll
    for (int i = 0; i < 4; ++i) asm volatile("" : "+v"(o.e[i]));  // not loaded one by one inside the guarded stores
    return o;
  }
  static __device__ __forceinline__ float join(int a, int b, int c, int d, int e) {
    const long long v = (long long)a + ((long long)b << 8) + ((long long)c << 16) + ((long long)d << 24);
    return e == kGBad ? __builtin_nanf("") : (float)ldexp((double)v, e);
  }
  __device__ __forceinline__ void put(int r, int c, int mr, const Row& s, const iv16& acc) const {
    float* o = out + (r >> 2) * ld + c;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (r + 8 * i < mr) o[2 * i * ld] = join(acc[4 * i], acc[4 * i + 1], acc[4 * i + 2], acc[4 * i + 3], s.e[i]);
  }
  template <int FM, int FN>
  __device__ __forceinline__ void finish(const iv16 (&acc)[FM][FN], int r0, int c0, int mr, int nr, float*) const {
    finish_direct<FM, FN>(*this, acc, r0, c0, mr, nr);
  }
  __device__ __forceinline__ void put4(long long r, int c, int M, const iv4& s) const {
    out[(r >> 2) * ld + c] = join(s[0], s[1], s[2], s[3], ex[r >> 2]);
  }
};

// part[p][i] (+)= sum over the batch's rows of part p of t u
__global__ void __launch_bounds__(256) dsum_kernel(const float* __restrict__ Tm, const float* __restrict__ U, int k,
                                                   int batch, int first, double* __restrict__ part) {
  const int i = blockIdx.x * 256 + threadIdx.x;
  if (i >= k) return;
  const int per = (batch + kGParts - 1) / kGParts;
  const int b0 = blockIdx.y * per, b1 = b0 + per < batch ? b0 + per : batch;
  double s = first ? 0.0 : part[(size_t)blockIdx.y * k + i];
  for (int b = b0; b < b1; ++b) s += (double)Tm[(size_t)b * k + i] * (double)U[(size_t)b * k + i];
  part[(size_t)blockIdx.y * k + i] = s;
}

__global__ void __launch_bounds__(256) dfin_kernel(const double* __restrict__ part, int parts, int k,
                                                   float* __restrict__ dD) {
  const int i = blockIdx.x * 256 + threadIdx.x;
  if (i >= k) return;
  double s = 0.0;
  for (int p = 0; p < parts; ++p) s += part[(size_t)p * k + i];
  dD[i] = (float)s;
}

struct GradSpace {
  size_t be, ce, ct, xd, yd, sd, u, t, ex, part, split, bytes;
};
static GradSpace grad_space(int k, int m, int n, long long batch) {
  const size_t c = (size_t)(batch < kGChunk ? batch : kGChunk);
  const size_t kp = pad16(k), mp = pad16(m), np = pad16(n);
  GradSpace s;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off = al256(off + bytes);
    return o;
  };
  s.be = take(k * mp);
  s.ce = take(k * np);
  s.ct = take(n * kp);
  s.xd = take(4 * c * np);
  s.yd = take(4 * c * mp);
  s.sd = take(4 * c * kp);
  s.u = take(4 * c * k);
  s.t = take(4 * c * k);
  s.ex = take(3 * c * 4);
  s.part = take((size_t)kGParts * k * 8);
  // the parts of a split product, one product at a time; a last pass of fewer vectors may split where
  // the others do not
  size_t split = 0;
  for (long long b = batch < kGChunk ? batch : batch % kGChunk, once = 0; once < 2; b = (long long)c, ++once)
    if (b > 0) {
      split = std::max(split, tile_plan(4 * b, k, (int)mp).bytes);
      split = std::max(split, tile_plan(4 * b, k, (int)np).bytes);
      split = std::max(split, tile_plan(4 * b, n, (int)kp).bytes);
    }
  s.split = take(split);
  s.bytes = off;
  return s;
}

size_t grad_workspace_bytes(int k, int m, int n, long long batch) {
  if (batch == 0) return 0;
  if (batch <= kGFew) return infer_grad_workspace_bytes(k, n, (int)batch);
  return grad_space(k, m, n, batch).bytes;
}

static hipError_t join_product(const int8_t* A, long long K, int M, const int8_t* B, int N, const int* ex, float* out,
                               long long ld, void* split, hipStream_t st) {
  return tile_product(A, K, M, B, K, N, (int)K, JoinDigits{ex, out, ld}, split, st);
}

hipError_t grad_run(const uint32_t* B, const uint32_t* C, const float* D, int k, int m, int n, const float* X,
                    const float* dY, long long batch, float* dX, float* dD, void* ws, hipStream_t st) {
  if (batch == 0) {
    if (dD) hipLaunchKernelGGL(dfin_kernel, dim3((k + 255) / 256), dim3(256), 0, st, nullptr, 0, k, dD);
    return hipGetLastError();
  }
  if (batch <= kGFew) return infer_grad_run(B, C, D, k, m, n, X, dY, (int)batch, dX, dD, ws, st);
  const GradSpace s = grad_space(k, m, n, batch);
  char* base = static_cast<char*>(ws);
  int8_t* be = reinterpret_cast<int8_t*>(base + s.be);
  int8_t* ce = reinterpret_cast<int8_t*>(base + s.ce);
  int8_t* ct = reinterpret_cast<int8_t*>(base + s.ct);
  int8_t* xd = reinterpret_cast<int8_t*>(base + s.xd);
  int8_t* yd = reinterpret_cast<int8_t*>(base + s.yd);
  int8_t* sd = reinterpret_cast<int8_t*>(base + s.sd);
  float* u = reinterpret_cast<float*>(base + s.u);
  float* t = reinterpret_cast<float*>(base + s.t);
  int* ex = reinterpret_cast<int*>(base + s.ex);
  double* part = reinterpret_cast<double*>(base + s.part);
  const long long kp = pad16(k), mp = pad16(m), np = pad16(n);
  const long long wb = k * (mp / 16), wc = k * (np / 16);
  hipLaunchKernelGGL(widen_kernel, dim3((unsigned)((wb + 255) / 256)), dim3(256), 0, st, B, wb, be);
  if (dD) hipLaunchKernelGGL(widen_kernel, dim3((unsigned)((wc + 255) / 256)), dim3(256), 0, st, C, wc, ce);
  if (dX)
    hipLaunchKernelGGL(widen_t_kernel, dim3((k + 255) / 256, (unsigned)((np / 16 + 15) / 16)), dim3(256), 0, st, C, k,
                       (int)(np / 16), n, ct, kp);
  for (long long b0 = 0; b0 < batch; b0 += kGChunk) {
    const int c = (int)(batch - b0 < kGChunk ? batch - b0 : kGChunk);
    hipError_t e;
    hipLaunchKernelGGL(digits_kernel, dim3(c), dim3(256), 0, st, dY + b0 * m, (long long)m, nullptr, yd, mp, ex);
    e = join_product(yd, mp, 4 * c, be, k, ex, u, k, base + s.split, st);
    if (e != hipSuccess) return e;
    if (dD) {
      hipLaunchKernelGGL(digits_kernel, dim3(c), dim3(256), 0, st, X + b0 * n, (long long)n, nullptr, xd, np, ex + c);
      e = join_product(xd, np, 4 * c, ce, k, ex + c, t, k, base + s.split, st);
      if (e != hipSuccess) return e;
      hipLaunchKernelGGL(dsum_kernel, dim3((k + 255) / 256, kGParts), dim3(256), 0, st, t, u, k, c, b0 == 0, part);
    }
    if (dX) {
      hipLaunchKernelGGL(digits_kernel, dim3(c), dim3(256), 0, st, u, (long long)k, D, sd, kp, ex + 2 * c);
      e = join_product(sd, kp, 4 * c, ct, n, ex + 2 * c, dX + b0 * n, n, base + s.split, st);
      if (e != hipSuccess) return e;
    }
  }
  if (dD) hipLaunchKernelGGL(dfin_kernel, dim3((k + 255) / 256), dim3(256), 0, st, part, kGParts, k, dD);
  return hipGetLastError();
}

}  // namespace externd
