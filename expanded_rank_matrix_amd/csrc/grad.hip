// Gradient of a layer held as packed ternary factors, y = B diag(D) C x, over a batch:
//   u_b = B^T dy_b,   t_b = C x_b,   dD_i = sum_b t_bi u_bi,   dx_b = C^T (D u_b)
//
// Little work goes through the inference kernels (apply.hip).  A larger batch is three products of
// 8-bit integers (igemm.hpp): each vector enters as four rows of signed 8-bit digits of a
// fixed-point image with its own power-of-two scale, N = rint(x 2^(30 - E)), |x| < 2^E for the
// whole vector, N = d0 + 2^8 d1 + 2^16 d2 + 2^24 d3; the factors' codes are widened to bytes.  A
// digit's sum is exact in int32 (lengths below 2^24), the four are joined in int64, scaled and
// rounded once to fp32: the image's rounding, 2^-31 of the vector's largest power of two, is the
// only error of a product besides.  t u and its sum over the batch are fp64, in a fixed order: the
// product that makes t multiplies its tile by u's and adds over the tile's vectors, so t is never
// stored (split products, which have no whole tiles, store it).
//
// Bound by the products (2048 vectors, k = 7680, 2560 x 2560: 966 10^9 operations of digits in about
// 450 of 490 us, 2.1 10^15 a second).  Three digits would take a quarter less, but their 2^-23 of the
// vector's largest element is worse than fp32 wherever a few channels are large.
#include <algorithm>

#include "common.hpp"
#include "externd_internal.hpp"
#include "igemm.hpp"
#include "types.hpp"

namespace externd {

constexpr int kGChunk = 4096;       // vectors per pass over the factors (bounds the workspace)
constexpr int kGParts = 32;         // partial sums of dD where the products are split
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
__device__ __forceinline__ void widen(const uint32_t* __restrict__ P, long long words, long long block,
                                      int8_t* __restrict__ out) {
  const long long x = block * 256 + threadIdx.x;
  if (x >= words) return;
  const unsigned w = P[x];
  const iv4 v = {(int)widen4(w & 255u), (int)widen4(w >> 8 & 255u), (int)widen4(w >> 16 & 255u), (int)widen4(w >> 24)};
  *reinterpret_cast<iv4*>(out + 16 * x) = v;
}

// packed rows -> bytes of the transpose: out[j][i] = code j of row i, i < kp (zeros from k on).
// Workgroup (bx, by): rows 256 bx on, words 16 by on; thread: 16 rows of one word.
__device__ __forceinline__ void widen_t(const uint32_t* __restrict__ P, int k, int words, int n, long long bx,
                                        long long by, int8_t* __restrict__ out, long long kp, unsigned* tile) {
  const int tid = threadIdx.x;
  const long long i0 = bx * 256, w0 = by * 16;
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
__device__ __forceinline__ void digits(const float* __restrict__ X, long long n, const float* __restrict__ D, long long b,
                                       int8_t* __restrict__ out, long long np, int* __restrict__ ex, unsigned* wmx) {
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

__global__ void __launch_bounds__(256) digits_kernel(const float* __restrict__ X, long long n,
                                                     const float* __restrict__ D, int8_t* __restrict__ out,
                                                     long long np, int* __restrict__ ex) {
  __shared__ unsigned wmx[4];
  digits(X, n, D, blockIdx.x, out, np, ex, wmx);
}

// Everything the products need but D u, in one launch: digits of dY and X (the rows of one pass), the
// factors' bytes (on the first pass).  Workgroups in runs: count[q] of them for part q.
struct Prep {
  const float* dY;
  const float* X;
  const uint32_t* B;
  const uint32_t* C;
  int8_t* yd;
  int8_t* xd;
  int8_t* be;
  int8_t* ce;
  int8_t* ct;
  int* ex;
  int m, n, k, batch;
  unsigned count[5];
};
__global__ void __launch_bounds__(256) prep_kernel(Prep p) {
  __shared__ unsigned lds[256 * 17];
  const long long kp = (p.k + 15ll) & ~15ll, mp = (p.m + 15ll) & ~15ll, np = (p.n + 15ll) & ~15ll;
  unsigned b = blockIdx.x;
  if (b < p.count[0]) return digits(p.dY, p.m, nullptr, b, p.yd, mp, p.ex, lds);
  b -= p.count[0];
  if (b < p.count[1]) return digits(p.X, p.n, nullptr, b, p.xd, np, p.ex + p.batch, lds);
  b -= p.count[1];
  if (b < p.count[2]) {
    const unsigned across = (unsigned)((np / 16 + 15) / 16);
    return widen_t(p.C, p.k, (int)(np / 16), p.n, b / across, b % across, p.ct, kp, lds);
  }
  b -= p.count[2];
  if (b < p.count[3]) return widen(p.B, p.k * (mp / 16), b, p.be);
  b -= p.count[3];
  widen(p.C, p.k * (np / 16), b, p.ce);
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

// The product that makes t, with u at hand: part[rows / 64 (32 for a matrix of up to 64 rows)][col] =
// the sum of t u over the vectors of those rows.
struct DotDigits {
  const int* ex;
  const float* u;
  long long ld;
  double* part;
  long long row0;
  static constexpr bool kLds = false;
  __device__ __forceinline__ void at(long long m0, long long n0) {
    ex += m0 >> 2;
    u += (m0 >> 2) * ld + n0;
    part += n0;
    row0 = m0;
  }
  template <int FM, int FN>
  __device__ __forceinline__ void finish(const iv16 (&acc)[FM][FN], int r0, int c0, int mr, int nr, float*) const {
    const int lane = threadIdx.x & 63, lg = lane >> 5, lr = lane & 31;
    constexpr int G = FM > 1 ? 2 : 1;  // accumulators of one partial sum
#pragma unroll
    for (int g = 0; g < FM; g += G) {
      if (r0 + 32 * g >= mr) break;  // the same for the wave
      int e[G][4];
      float uv[G][FN][4];
#pragma unroll
      for (int i = 0; i < G; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int r = r0 + 32 * (g + i) + 4 * lg + 8 * q, v = (r < mr ? r : mr - 1) >> 2;
          e[i][q] = ex[v];
#pragma unroll
          for (int j = 0; j < FN; ++j) {
            const int c = c0 + 32 * j + lr;
            uv[i][j][q] = u[v * ld + (c < nr ? c : nr - 1)];
          }
        }
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        double s = 0.0;
#pragma unroll
        for (int i = 0; i < G; ++i)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const iv16& a = acc[g + i][j];
            const long long v = (long long)a[4 * q] + ((long long)a[4 * q + 1] << 8) + ((long long)a[4 * q + 2] << 16) +
                                ((long long)a[4 * q + 3] << 24);
            const double t = e[i][q] == kGBad ? (double)__builtin_nanf("") : ldexp((double)v, e[i][q]);
            if (r0 + 32 * (g + i) + 4 * lg + 8 * q < mr) s += t * (double)uv[i][j][q];
          }
        s += __shfl_xor(s, 32);
        const int c = c0 + 32 * j + lr;
        if (lg == 0 && c < nr) part[(row0 + r0 + 32 * g) / (32 * G) * ld + c] = s;
      }
    }
  }
};

// part[p][i] = sum over the batch's rows of part p of t u (split products)
__global__ void __launch_bounds__(256) dsum_kernel(const float* __restrict__ Tm, const float* __restrict__ U, int k,
                                                   int batch, double* __restrict__ part) {
  const int i = blockIdx.x * 256 + threadIdx.x;
  if (i >= k) return;
  const int per = (batch + kGParts - 1) / kGParts;
  const int b0 = blockIdx.y * per, b1 = b0 + per < batch ? b0 + per : batch;
  double s = 0.0;
#pragma unroll 4
  for (int b = b0; b < b1; ++b) s += (double)Tm[(size_t)b * k + i] * (double)U[(size_t)b * k + i];
  part[(size_t)blockIdx.y * k + i] = s;
}

// the parts of one pass added in order to what earlier passes left in sum; the last pass rounds.
// Workgroup: 64 components, the parts over its four waves.
__global__ void __launch_bounds__(256) dfin_kernel(const double* __restrict__ part, int parts, int k, int first, int last,
                                                   double* __restrict__ sum, float* __restrict__ dD) {
  __shared__ double ws[256];
  const int wv = threadIdx.x >> 6, i = blockIdx.x * 64 + (threadIdx.x & 63);
  double s = 0.0;
  if (i < k) {
#pragma unroll 8
    for (int p = wv; p < parts; p += 4) s += part[(size_t)p * k + i];
  }
  ws[threadIdx.x] = s;
  __syncthreads();
  if (wv != 0 || i >= k) return;
  for (int w = 1; w < 4; ++w) s += ws[64 * w + threadIdx.x];
  if (!first) s += sum[i];
  if (last) dD[i] = (float)s;
  else sum[i] = s;
}

// Batches that the inference kernels serve sooner: their two launches take about 11 us and, per vector
// and 32 components, 7.5 ns and 1.7 ps an element of the two vectors; the products take about 30 us and
// 0.5 ps an element of the factors to widen.  Measured, k, m, n and batch, inference kernels / products, us:
// 7680, 2560, 2560: 1 18.6 / 58.7, 8 44.8 / 62.8, 14 67.3 / 63.9, 64 228 / 75.6; 1203, 777, 1025: 37 29.6 /
// 41.3, 100 60.7 / 43.6; 300, 200, 200: 100 18.9 / 26.6, 1000 99.2 / 30.0; 5000, 5000, 500: 10 41.8 / 53.4, 20
// 72.5 / 55.0; 1536, 1024, 1024: 16 21.9 / 34.1, 64 45.4 / 42.0.
static bool grad_few(int k, int m, int n, long long batch) {
  const double few = 11.0 + (double)batch * ((k + 31) / 32) * (7.5e-3 + 1.7e-6 * ((double)m + n));
  return batch <= 4096 && few <= 30.0 + 5e-7 * k * ((double)m + 2.0 * n);
}

struct GradSpace {
  size_t be, ce, ct, xd, yd, sd, u, t, ex, part, sum, split, bytes;
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
  s.ex = take(3 * c * 4);
  s.part = take(std::max<size_t>(kGParts, 4 * c / 32 + 2) * k * 8);
  s.sum = take((size_t)k * 8);
  // t and the parts of split products, one product at a time; a last pass of fewer vectors may split
  // where the others do not
  size_t split = 0, t = 0;
  for (const long long b : {(long long)c, batch % kGChunk})
    if (b > 0) {
      const TilePlan pt = tile_plan(4 * b, k, (int)np);
      if (pt.parts > 1) t = std::max(t, (size_t)(4 * b * k));
      split = std::max({split, pt.bytes, tile_plan(4 * b, k, (int)mp).bytes, tile_plan(4 * b, n, (int)kp).bytes});
    }
  s.t = take(t);
  s.split = take(split);
  s.bytes = off;
  return s;
}

size_t grad_workspace_bytes(int k, int m, int n, long long batch) {
  if (batch == 0) return 0;
  if (grad_few(k, m, n, batch)) return infer_grad_workspace_bytes(k, n, (int)batch);
  return grad_space(k, m, n, batch).bytes;
}

hipError_t grad_run(const uint32_t* B, const uint32_t* C, const float* D, int k, int m, int n, const float* X,
                    const float* dY, long long batch, float* dX, float* dD, void* ws, hipStream_t st) {
  const dim3 gk((k + 63) / 64);
  if (batch == 0) {
    if (dD) hipLaunchKernelGGL(dfin_kernel, gk, dim3(256), 0, st, nullptr, 0, k, 1, 1, nullptr, dD);
    return hipGetLastError();
  }
  if (grad_few(k, m, n, batch)) return infer_grad_run(B, C, D, k, m, n, X, dY, (int)batch, dX, dD, ws, st);
  const GradSpace s = grad_space(k, m, n, batch);
  char* base = static_cast<char*>(ws);
  auto at = [&](size_t o) { return static_cast<void*>(base + o); };
  float* u = static_cast<float*>(at(s.u));
  float* t = static_cast<float*>(at(s.t));
  double* part = static_cast<double*>(at(s.part));
  double* sum = static_cast<double*>(at(s.sum));
  int* ex = static_cast<int*>(at(s.ex));
  int8_t* sd = static_cast<int8_t*>(at(s.sd));
  void* split = at(s.split);
  const long long kp = pad16(k), mp = pad16(m), np = pad16(n);
  Prep p{dY, X, B, C, static_cast<int8_t*>(at(s.yd)), static_cast<int8_t*>(at(s.xd)), static_cast<int8_t*>(at(s.be)),
         static_cast<int8_t*>(at(s.ce)), static_cast<int8_t*>(at(s.ct)), ex, m, n, k, 0, {}};
  for (long long b0 = 0; b0 < batch; b0 += kGChunk) {
    const int c = (int)(batch - b0 < kGChunk ? batch - b0 : kGChunk);
    const bool first = b0 == 0, last = b0 + c == batch;
    p.dY = dY + b0 * m;
    p.X = dD ? X + b0 * n : nullptr;
    p.batch = c;
    const long long count[5] = {c, dD ? c : 0, first && dX ? (k + 255ll) / 256 * ((np / 16 + 15) / 16) : 0,
                                first ? (k * (mp / 16) + 255) / 256 : 0, first && dD ? (k * (np / 16) + 255) / 256 : 0};
    long long all = 0;
    for (int q = 0; q < 5; ++q) {
      p.count[q] = (unsigned)count[q];
      all += count[q];
    }
    if (all > (1ll << 23)) return hipErrorInvalidValue;
    hipLaunchKernelGGL(prep_kernel, dim3((unsigned)all), dim3(256), 0, st, p);
    hipError_t e = tile_product(p.yd, mp, 4 * c, p.be, mp, k, (int)mp, JoinDigits{ex, u, k}, split, st);
    if (e != hipSuccess) return e;
    if (dD) {
      int parts = kGParts;
      if (tile_plan(4ll * c, k, (int)np).parts > 1) {
        e = tile_product(p.xd, np, 4 * c, p.ce, np, k, (int)np, JoinDigits{ex + c, t, k}, split, st);
        if (e != hipSuccess) return e;
        hipLaunchKernelGGL(dsum_kernel, dim3((k + 255) / 256, kGParts), dim3(256), 0, st, t, u, k, c, part);
      } else {
        const int rows = 4 * c <= 64 ? 32 : 64;
        parts = (4 * c + rows - 1) / rows;
        e = tile_whole(p.xd, np, 4 * c, p.ce, np, k, (int)np, DotDigits{ex + c, u, k, part, 0}, st);
        if (e != hipSuccess) return e;
      }
      hipLaunchKernelGGL(dfin_kernel, gk, dim3(256), 0, st, part, parts, k, (int)first, (int)last, sum, dD);
    }
    if (dX) {
      hipLaunchKernelGGL(digits_kernel, dim3(c), dim3(256), 0, st, u, (long long)k, D, sd, kp, ex + 2 * c);
      e = tile_product(sd, kp, 4 * c, p.ct, kp, n, (int)kp, JoinDigits{ex + 2 * c, dX + b0 * n, n}, split, st);
      if (e != hipSuccess) return e;
    }
  }
  return hipGetLastError();
}

}  // namespace externd
