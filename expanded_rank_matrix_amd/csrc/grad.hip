// Gradient of a layer held as packed ternary factors, y = B diag(D) C x, over a batch:
//   u_b = B^T dy_b,   t_b = C x_b,   dD_i = sum_b t_bi u_bi,   dx_b = C^T (D u_b)
//
// Little work goes through the inference kernels (apply.hip).  A larger batch is three products of
// 8-bit integers: each vector enters as four rows of signed 8-bit digits of a fixed-point image with
// its own power-of-two scale, N = rint(x 2^(30 - E)), |x| < 2^E for the whole vector,
// N = d0 + 2^8 d1 + 2^16 d2 + 2^24 d3.  A digit's sum is exact in int32 (lengths below 2^24), the four
// are joined in int64, scaled and rounded once to fp32: the image's rounding, 2^-31 of the vector's
// largest power of two, is the only error of a product besides.  t u and its sum over the batch are
// fp64, in a fixed order.
//
// Up to a few hundred vectors the codes are widened on their way into the products (codes_ut_kernel,
// codes_x_kernel); a batch beyond has them widened to bytes once for igemm.hpp's tiles: the product that
// makes t multiplies its tile by u's and adds over the tile's vectors, so t is never stored (split
// products, which have no whole tiles, store it).
//
// The large ones are bound by the products (2048 vectors, k = 7680, 2560 x 2560: 966 10^9 operations of digits in about
// 430 of 495 us, 2.2 10^15 a second).  Three digits would take a quarter less, but their 2^-23 of the
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
static long long pad_step(long long n) { return (n + 255) & ~255ll; }

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

// 256 rows from i0 on by 16 words from w0 on, through LDS (zeros outside); thread: 16 rows of one word,
// w[r] = word tid >> 4 of row 16 (tid & 15) + r
__device__ __forceinline__ void tile_words(const uint32_t* __restrict__ P, int k, int words, long long i0, long long w0,
                                           unsigned* tile, unsigned (&w)[16]) {
  const int tid = threadIdx.x, r0 = tid >> 4, c = tid & 15;
  const long long col = w0 + c < words ? w0 + c : words - 1;
#pragma unroll
  for (int u = 0; u < 16; ++u) {
    const long long row = i0 + r0 + 16 * u;
    w[u] = P[(row < k ? row : k - 1) * words + col];
  }
#pragma unroll
  for (int u = 0; u < 16; ++u) asm volatile("" : "+v"(w[u]));  // all in flight: not loaded one by one before its store
#pragma unroll
  for (int u = 0; u < 16; ++u) tile[(r0 + 16 * u) * 17 + c] = i0 + r0 + 16 * u < k && w0 + c < words ? w[u] : 0u;
  __syncthreads();
#pragma unroll
  for (int r = 0; r < 16; ++r) w[r] = tile[(16 * c + r) * 17 + r0];
}

// packed rows -> bytes of the transpose: out[j][i] = code j of row i, i < kp (zeros from k on).
// Workgroup (bx, by): rows 256 bx on, words 16 by on; thread: 16 rows of one word.
__device__ __forceinline__ void widen_t(const uint32_t* __restrict__ P, int k, int words, int n, long long bx,
                                        long long by, int8_t* __restrict__ out, long long kp, unsigned* tile) {
  const int tid = threadIdx.x;
  const long long i0 = bx * 256, w0 = by * 16;
  const int g = tid & 15, c = tid >> 4;
  unsigned w[16];
  tile_words(P, k, words, i0, w0, tile, w);
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

// 16 words of 16 codes: bits 2 i of word j <-> bits 2 j of word i.  Step S swaps the off-diagonal blocks of
// S words by S codes.
template <int S>
__device__ __forceinline__ void transpose_step(unsigned (&w)[16]) {
  constexpr unsigned mask = S == 8 ? 0x0000FFFFu : S == 4 ? 0x00FF00FFu : S == 2 ? 0x0F0F0F0Fu : 0x33333333u;
#pragma unroll
  for (int i = 0; i < 16; ++i)
    if (!(i & S)) {
      const unsigned x = (w[i] >> 2 * S ^ w[i + S]) & mask;
      w[i + S] ^= x;
      w[i] ^= x << 2 * S;
    }
}
__device__ __forceinline__ void transpose_codes(unsigned (&w)[16]) {
  transpose_step<8>(w);
  transpose_step<4>(w);
  transpose_step<2>(w);
  transpose_step<1>(w);
}

// packed rows -> the packed transpose: word i / 16 of row j of out (kw words) holds code j of 16 rows i,
// zeros from row k on.  Workgroups as for widen_t.
__device__ __forceinline__ void pack_t(const uint32_t* __restrict__ P, int k, int words, long long bx, long long by,
                                       uint32_t* __restrict__ out, int kw, unsigned* tile) {
  const int tid = threadIdx.x;
  const long long i0 = bx * 256, w0 = by * 16;
  const int g = tid & 15, c = tid >> 4;
  unsigned w[16];
  tile_words(P, k, words, i0, w0, tile, w);
  transpose_codes(w);
  if (w0 + c >= words) return;
  uint32_t* o = out + 16 * (w0 + c) * kw + i0 / 16 + g;
#pragma unroll
  for (int e = 0; e < 16; ++e) o[(long long)e * kw] = w[e];
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
// exponent E - 30 of its image's unit.  TILED: the rows of four vectors in the order in which a wave's
// MFMA operands take them, 1 KB a load (codes_sums): of 256 columns the 16-byte pieces
// [piece & 3][piece >> 2][row & 15].
template <int TH, bool TILED>
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
  for (long long j = 4 * threadIdx.x; j < n; j += 4 * TH) {
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
  for (int w = 0; w < TH / 64; ++w) mx = wmx[w] > mx ? wmx[w] : mx;
  const bool bad = mx >= 0x7F800000u;
  const int E = mx >> 23 ? (int)(mx >> 23) - 126 : -126;  // |x| < 2^E
  const int sh = 30 - E;
  if (threadIdx.x == 0) ex[b] = bad ? kGBad : -sh;
  if (TILED) {
    int8_t* o = out + 16 * (b >> 2) * np + 64 * (b & 3);
    for (long long j = 16 * threadIdx.x; j < np; j += 16 * TH) {
      iv4 w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float v[4];
        unsigned d[4] = {0u, 0u, 0u, 0u};
        get(j + 4 * e, v);
        if (!bad) digits4(v, sh, d);
#pragma unroll
        for (int q = 0; q < 4; ++q) w[q][e] = (int)d[q];
      }
      const long long piece = j >> 4;
      iv4* p = reinterpret_cast<iv4*>(o + (piece >> 4) * 4096 + (piece & 3) * 1024 + (piece >> 2 & 3) * 256);
#pragma unroll
      for (int q = 0; q < 4; ++q) p[q] = w[q];
    }
    return;
  }
  int8_t* o = out + 4 * b * np;
  for (long long j = 4 * threadIdx.x; j < np; j += 4 * TH) {
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
  digits<256, false>(X, n, D, blockIdx.x, out, np, ex, wmx);
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
  long long yp, xp;  // bytes of a row of yd and xd
  int m, n, k, batch;
  unsigned count[5];
};
template <bool TILED>
__global__ void __launch_bounds__(256) prep_kernel(Prep p) {
  __shared__ unsigned lds[256 * 17];
  const long long kp = (p.k + 15ll) & ~15ll, mp = (p.m + 15ll) & ~15ll, np = (p.n + 15ll) & ~15ll;
  unsigned b = blockIdx.x;
  if (b < p.count[0]) return digits<256, TILED>(p.dY, p.m, nullptr, b, p.yd, p.yp, p.ex, lds);
  b -= p.count[0];
  if (b < p.count[1]) return digits<256, TILED>(p.X, p.n, nullptr, b, p.xd, p.xp, p.ex + p.batch, lds);
  b -= p.count[1];
  if (b < p.count[2]) {
    const unsigned across = (unsigned)((np / 16 + 15) / 16);
    if (TILED)
      return pack_t(p.C, p.k, (int)(np / 16), b / across, b % across, reinterpret_cast<uint32_t*>(p.ct),
                    (int)((kp + 255) / 256 * 16), lds);
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
  static constexpr bool kLds = false, kAligned = true;  // rows padded to 16 bytes, in the workspace
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
  static constexpr bool kLds = false, kAligned = true;
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

// ---- small batches, from the packed codes ---------------------------------------------------------
// Workgroup: 16 NT packed rows by 16 vectors (64 digit rows).  A wave walks the columns in steps of 256: a
// lane takes the codes of its row at 64 consecutive columns (one 16-byte load), and its digit row's bytes
// there; the order of the columns within a step does not matter, only that both operands have the same.
// An accumulator's four registers are the four digits of one vector.  Bound by the digits' way from L2 (7680,
// 2560, 2560: u and t of 16 vectors 10.6 us, 328 KB a workgroup; with their rows as they lie, 64 bytes of
// each at a time, 23), small sizes by the four launches (1203, 777, 1025 with 37 vectors: 5.6 + 5.6 + 4.3 + 3.2).
constexpr int kCVec = 16, kCStep = 256;
template <int NT>
__device__ __forceinline__ void codes_sums(const uint32_t* __restrict__ P, int count, int w, int i0,
                                           const int8_t* __restrict__ dig, int pitch, int batch, int b0, int first,
                                           int stride, int steps, long long (&sum)[NT][4]) {
  const int lane = threadIdx.x & 63, lr = lane & 15, lg = lane >> 4;
  const uint32_t* codes[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int i = i0 + 16 * t + lr;
    codes[t] = P + (long long)(i < count ? i : count - 1) * w;
  }
  const int8_t* rows[4];
  const int tiles = (batch + 3) >> 2;
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int tile = (b0 >> 2) + r;
    rows[r] = dig + (tile < tiles ? tile : tiles - 1) * (16ll * pitch) + 16 * lane;
  }
  iv4 acc[NT][4];
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int r = 0; r < 4; ++r) acc[t][r] = iv4{0, 0, 0, 0};
  for (int c = first; c < steps; c += stride) {
    const int x = 16 * c + 4 * lg;  // the lane's first word
    iv4 v[NT], a[4][4];
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int r = 0; r < 4; ++r) a[r][q] = *reinterpret_cast<const iv4*>(rows[r] + 16ll * kCStep * c + 1024 * q);
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      if (x + 4 <= w) {
        v[t] = *reinterpret_cast<const iv4_any*>(codes[t] + x);
      } else {
#pragma unroll
        for (int q = 0; q < 4; ++q) v[t][q] = x + q < w ? (int)codes[t][x + q] : 0;
      }
    }
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const unsigned y = (unsigned)v[t][q];
        const iv4 b = {(int)widen4(y & 255u), (int)widen4(y >> 8 & 255u), (int)widen4(y >> 16 & 255u),
                       (int)widen4(y >> 24)};
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[t][r] = __builtin_amdgcn_mfma_i32_16x16x64_i8(a[r][q], b, acc[t][r], 0, 0, 0);
      }
  }
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int r = 0; r < 4; ++r)
      sum[t][r] = (long long)acc[t][r][0] + ((long long)acc[t][r][1] << 8) + ((long long)acc[t][r][2] << 16) +
                  ((long long)acc[t][r][3] << 24);
}
__device__ __forceinline__ double scaled(long long v, int e) {
  return e == kGBad ? (double)__builtin_nanf("") : ldexp((double)v, e);
}

// u (waves 0-3) and t (waves 4-7), each wave a quarter of the columns.  The quarters meet in LDS as int64,
// u and t of a pair in one thread, which adds t u over the workgroup's vectors.
template <int NT>
__global__ void __launch_bounds__(512) codes_ut_kernel(const uint32_t* __restrict__ B, int wm,
                                                       const uint32_t* __restrict__ C, int wn, int k,
                                                       const int8_t* __restrict__ yd, int yp,
                                                       const int8_t* __restrict__ xd, int xp, const int* __restrict__ ex,
                                                       int batch, float* __restrict__ U, double* __restrict__ part) {
  __shared__ long long sums[8][256 * NT];
  __shared__ double ds[8][16];
  const int tid = threadIdx.x, lane = tid & 63, lr = lane & 15, lg = lane >> 4;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);  // scalar: MFMA runs whatever the lane mask
  const int i0 = blockIdx.x * 16 * NT, b0 = blockIdx.y * kCVec;
  const bool fwd = wv >= 4;
  const int pitch = fwd ? xp : yp;
  long long own[NT][4];
  codes_sums<NT>(fwd ? C : B, k, fwd ? wn : wm, i0, fwd ? xd : yd, pitch, batch, b0, wv & 3, 4,
                 fwd && !part ? 0 : pitch / kCStep, own);
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int r = 0; r < 4; ++r) sums[wv][t * 256 + (4 * r + lg) * 16 + lr] = own[t][r];
  __syncthreads();
  const int t = tid >> 8, b = b0 + (tid >> 4 & 15), i = i0 + 16 * t + lr;
  if (t < NT) {
    double s = 0.0;
    if (b < batch) {
      const double u = scaled(sums[0][tid] + sums[1][tid] + sums[2][tid] + sums[3][tid], ex[b]);
      if (U && i < k) U[(size_t)b * k + i] = (float)u;
      if (part) s = u * scaled(sums[4][tid] + sums[5][tid] + sums[6][tid] + sums[7][tid], ex[batch + b]);
    }
    s += __shfl_xor(s, 16);
    s += __shfl_xor(s, 32);
    if (lg == 0) ds[wv][lr] = s;
  }
  __syncthreads();
  if (part && tid < 16 * NT && i0 + tid < k) {
    const int q = 4 * (tid >> 4);
    part[(size_t)blockIdx.y * k + i0 + tid] = ds[q][tid & 15] + ds[q + 1][tid & 15] + ds[q + 2][tid & 15] + ds[q + 3][tid & 15];
  }
}

// Between the products: the images of D u (nd workgroups, one a vector), and dD from its parts.
constexpr int kCJoin = 1024;
__global__ void __launch_bounds__(kCJoin) codes_join_kernel(int nd, const float* __restrict__ U, int k,
                                                            const float* __restrict__ D, int8_t* __restrict__ sd, int sp,
                                                            int* __restrict__ ex, const double* __restrict__ part,
                                                            int parts, float* __restrict__ dD) {
  __shared__ unsigned wmx[kCJoin / 64];
  if ((int)blockIdx.x < nd) return digits<kCJoin, true>(U, k, D, blockIdx.x, sd, sp, ex, wmx);
  const int i = ((int)blockIdx.x - nd) * kCJoin + (int)threadIdx.x;
  if (i >= k) return;
  double s = 0.0;
#pragma unroll 4
  for (int p = 0; p < parts; ++p) s += part[(size_t)p * k + i];
  dD[i] = (float)s;
}

// dX from C's transpose and the images of D u, all eight waves over the components
template <int NT>
__global__ void __launch_bounds__(512) codes_x_kernel(const uint32_t* __restrict__ Ct, int n, const int8_t* __restrict__ sd,
                                                      int sp, const int* __restrict__ ex, int batch,
                                                      float* __restrict__ dX) {
  __shared__ long long sums[8][256 * NT];
  const int tid = threadIdx.x, lane = tid & 63, lr = lane & 15, lg = lane >> 4;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int j0 = blockIdx.x * 16 * NT, b0 = blockIdx.y * kCVec;
  long long own[NT][4];
  codes_sums<NT>(Ct, n, sp / 16, j0, sd, sp, batch, b0, wv, 8, sp / kCStep, own);
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int r = 0; r < 4; ++r) sums[wv][t * 256 + (4 * r + lg) * 16 + lr] = own[t][r];
  __syncthreads();
  const int t = tid >> 8, b = b0 + (tid >> 4 & 15), j = j0 + 16 * t + lr;
  if (t < NT && b < batch && j < n) {
    long long s = 0;
#pragma unroll
    for (int w = 0; w < 8; ++w) s += sums[w][tid];
    dX[(long long)b * n + j] = (float)scaled(s, ex[b]);
  }
}

// Two tiles of rows a workgroup (the digits are read half as often) where that still leaves one for every
// CU.  Measured, one / two, us of a whole gradient: k, m, n = 7680, 2560, 2560, batch 32 44.9 / 37.3, 256
// 170 / 116; 4000, 9728, 2560, 16 32.9 / 36.0, 64 62.8 / 50.0; 1203, 777, 1025, 64 20.7 / 21.1, 250 37.4 / 33.8.
static bool codes_wide(int rows, int groups) { return (rows + 31) / 32 * (long long)groups >= 256; }
static unsigned codes_blocks(int rows, int groups) {
  return codes_wide(rows, groups) ? (rows + 31) / 32 : (rows + 15) / 16;
}

// Which kernels serve a batch: the least of their times in us, fitted to measurements of 75 sizes (1% lost
// on average to the best choice, 30% in the worst).  kFew: two launches of the inference kernels, two
// vectors a workgroup; its sums of t u are chains over the batch.  kCodes: four launches, from the packed
// codes, 16 vectors a workgroup.  kProducts: up to nine, the codes widened to bytes once.  Measured, k, m, n
// and batch, kFew / kCodes / kProducts, us: 7680, 2560, 2560: 1 18.4 / 29.2 / 56.6, 4 28.5 / 29.5 / 58.0, 16 72 /
// 33.0 / 61.3, 128 432 / 73 / 82, 256 850 / 120 / 103; 1203, 777, 1025: 1 14.3 / 17.3 / 33.2, 37 30.1 / 18.7 /
// 40.7, 250 128 / 33.9 / 46.7, 1000 - / 74 / 57; 96, 9728, 9728: 16 29.0 / 32.9 / 38.3, 256 116 / 62 / 57; 300,
// 200, 200: 2 13.1 / 14.7 / 19.7, 100 19.5 / 15.8 / 25.6, 1000 98 / 31.7 / 29.3; 9728, 100, 9728: 1 45.5 / 58 / 95,
// 64 - / 113 / 138, 256 - / 355 / 242.
enum class GradWay { kFew, kCodes, kProducts };
static GradWay grad_way(int k, int m, int n, long long batch) {
  if (batch > kGChunk) return GradWay::kProducts;
  const double l = std::max(m, n), s = (double)m + n, w = k * ((double)m + 2.0 * n);
  const double b = (double)batch, g = (double)((batch + kCVec - 1) / kCVec);
  const double few = 11.7 + 1.2e-3 * l + b * ((k + 31) / 32 * (7.1e-3 + 1.5e-6 * s) + 1.2e-5 * s);
  const double codes = 13.6 + 1.1e-3 * l + 6.6e-4 * k + 1.6e-7 * k * n + g * (0.13 + 2.7e-4 * k + 1.7e-4 * l + 5.4e-8 * w);
  const double products = 21.1 + 2.0e-3 * l + 2.2e-3 * k + 1.6e-7 * w + b * (3.3e-3 + 5e-6 * k + 5e-6 * l + 2.8e-9 * w);
  if (batch <= 512 && few <= codes && few <= products) return GradWay::kFew;
  return codes <= products ? GradWay::kCodes : GradWay::kProducts;
}

struct GradSpace {
  size_t be, ce, ct, xd, yd, sd, u, t, ex, part, sum, split, bytes;
};
static GradSpace grad_space(int k, int m, int n, long long batch) {
  const size_t c = (size_t)(batch < kGChunk ? batch : kGChunk);
  const bool codes = grad_way(k, m, n, batch) == GradWay::kCodes;
  const size_t kp = pad16(k), mp = codes ? pad_step(m) : pad16(m), np = codes ? pad_step(n) : pad16(n);
  const size_t np16 = pad16(n);
  GradSpace s;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off = al256(off + bytes);
    return o;
  };
  s.be = take(codes ? 0 : k * mp);
  s.ce = take(codes ? 0 : k * np);
  s.ct = take(codes ? np16 * pad_step(k) / 4 : n * kp);
  const size_t c4 = codes ? (c + 3) & ~(size_t)3 : c;  // whole tiles
  s.xd = take(4 * c4 * np);
  s.yd = take(4 * c4 * mp);
  s.sd = take(codes ? 4 * c4 * pad_step(k) : 4 * c * kp);
  s.u = take(4 * c * k);
  s.ex = take(3 * c * 4);
  s.part = take(std::max<size_t>(kGParts, 4 * c / 32 + 2) * k * 8);
  s.sum = take((size_t)k * 8);
  // t and the parts of split products, one product at a time; a last pass of fewer vectors may split
  // where the others do not
  size_t split = 0, t = 0;
  for (const long long b : {(long long)c, batch % kGChunk})
    if (b > 0 && !codes) {
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
  if (grad_way(k, m, n, batch) == GradWay::kFew) return infer_grad_workspace_bytes(k, n, (int)batch);
  return grad_space(k, m, n, batch).bytes;
}

hipError_t grad_run(const uint32_t* B, const uint32_t* C, const float* D, int k, int m, int n, const float* X,
                    const float* dY, long long batch, float* dX, float* dD, void* ws, hipStream_t st) {
  const dim3 gk((k + 63) / 64);
  if (batch == 0) {
    if (dD) hipLaunchKernelGGL(dfin_kernel, gk, dim3(256), 0, st, nullptr, 0, k, 1, 1, nullptr, dD);
    return hipGetLastError();
  }
  const GradWay way = grad_way(k, m, n, batch);
  if (way == GradWay::kFew) return infer_grad_run(B, C, D, k, m, n, X, dY, (int)batch, dX, dD, ws, st);
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
  const bool codes = way == GradWay::kCodes;
  const long long kp = pad16(k), mp = pad16(m), np = pad16(n);
  const long long yp = codes ? pad_step(m) : mp, xp = codes ? pad_step(n) : np;
  Prep p{dY, X, B, C, static_cast<int8_t*>(at(s.yd)), static_cast<int8_t*>(at(s.xd)), static_cast<int8_t*>(at(s.be)),
         static_cast<int8_t*>(at(s.ce)), static_cast<int8_t*>(at(s.ct)), ex, yp, xp, m, n, k, 0, {}};
  for (long long b0 = 0; b0 < batch; b0 += kGChunk) {
    const int c = (int)(batch - b0 < kGChunk ? batch - b0 : kGChunk);
    const bool first = b0 == 0, last = b0 + c == batch;
    p.dY = dY + b0 * m;
    p.X = dD ? X + b0 * n : nullptr;
    p.batch = c;
    const long long count[5] = {c, dD ? c : 0, first && dX ? (k + 255ll) / 256 * ((np / 16 + 15) / 16) : 0,
                                first && !codes ? (k * (mp / 16) + 255) / 256 : 0,
                                first && dD && !codes ? (k * (np / 16) + 255) / 256 : 0};
    long long all = 0;
    for (int q = 0; q < 5; ++q) {
      p.count[q] = (unsigned)count[q];
      all += count[q];
    }
    if (all > (1ll << 23)) return hipErrorInvalidValue;
    if (codes) hipLaunchKernelGGL(prep_kernel<true>, dim3((unsigned)all), dim3(256), 0, st, p);
    else hipLaunchKernelGGL(prep_kernel<false>, dim3((unsigned)all), dim3(256), 0, st, p);
    if (codes) {
      const int groups = (c + kCVec - 1) / kCVec, nd = dX ? c : 0, ns = dD ? (k + kCJoin - 1) / kCJoin : 0;
      const int sp = (int)pad_step(k), wm = (int)(mp / 16), wn = (int)(np / 16);
      const auto ut = codes_wide(k, groups) ? codes_ut_kernel<2> : codes_ut_kernel<1>;
      hipLaunchKernelGGL(ut, dim3(codes_blocks(k, groups), groups), dim3(512), 0, st, B, wm, C, wn, k, p.yd, (int)yp, p.xd,
                         (int)xp, ex, c, dX ? u : nullptr, dD ? part : nullptr);
      hipLaunchKernelGGL(codes_join_kernel, dim3(nd + ns), dim3(kCJoin), 0, st, nd, u, k, D, sd, sp, ex + 2 * c, part, groups,
                         dD);
      if (dX) {
        const auto xk = codes_wide(n, groups) ? codes_x_kernel<2> : codes_x_kernel<1>;
        hipLaunchKernelGGL(xk, dim3(codes_blocks(n, groups), groups), dim3(512), 0, st,
                           reinterpret_cast<const uint32_t*>(p.ct), n, sd, sp, ex + 2 * c, c, dX);
      }
      return hipGetLastError();
    }
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
