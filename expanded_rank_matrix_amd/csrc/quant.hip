// Products in 8-bit integers with a scale for each token and each output channel, and the
// quantisation of rows that makes their operands.
//
//   quantise:  a_t = max_j |x_tj|,  s_t = fl32(a_t / 127),  q_tj = the whole number nearest to the
//              exact quotient 127 x_tj / a_t, ties to even
//   product:   y_to = (sum_j q_tj W_oj) w_o s_t
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
// side: in units of x's last place 254 x and (2 q + 1) a are whole numbers, the first below 2^32, so a
// quotient that is no tie differs from the border by at least 2^-32 of it, and fp64's is good to 2^-53.
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

// a row's scale and rounding, from the fp32 bits of its largest |x|
struct RowScale {
  float a, inv;
  bool bad, tiny;
  __device__ __forceinline__ explicit RowScale(unsigned mx) {
    bad = mx >= 0x7F800000u;
    tiny = mx < 0x0D000000u;  // a < 2^-101
    a = __uint_as_float(mx);
    inv = bad || mx == 0u ? 0.0f : 127.0f / a;
  }
  __device__ __forceinline__ float scale() const { return bad ? __uint_as_float(0x7FC00000u) : a / 127.0f; }
  __device__ __forceinline__ void quantize(const float (&v)[8], int (&k)[8]) const {
    if (bad || a == 0.0f) {
#pragma unroll
      for (int e = 0; e < 8; ++e) k[e] = 0;
    } else if (tiny) {
#pragma unroll
      for (int e = 0; e < 8; ++e) k[e] = quant1_small(v[e], a);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) k[e] = quant1(v[e], inv, a);
    }
  }
};

__device__ __forceinline__ unsigned max_abs8(const float (&v)[8], unsigned mx) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const unsigned b = __float_as_uint(v[e]) & 0x7FFFFFFFu;
    mx = b > mx ? b : mx;
  }
  return mx;
}

// One row per TPR threads (64: a wave; 256: the workgroup), 8 elements per thread and step; the
// first CH steps of a row stay in registers between the search for its maximum and its rounding, a
// longer row's rest is read again.  The row's last elements, fewer than 8, are one a thread.  np bytes
// of each Q row are written, zeros behind the first n (np - n <= TPR).
// Bound by memory (4096 x 9728 bf16: 22 us, 5.4 TB/s; a large copy runs at 4.8).
template <typename T, int TPR, int CH>
__global__ void __launch_bounds__(256) quantize_kernel(const T* __restrict__ X, long long rows, int n, long long ldx,
                                                       int8_t* __restrict__ Q, long long ldq, int np,
                                                       float* __restrict__ scale) {
  constexpr int RPW = 256 / TPR;
  __shared__ unsigned wmx[4];
  const int tid = threadIdx.x % TPR;
  const long long row = (long long)blockIdx.x * RPW + threadIdx.x / TPR;
  const T* x = X + (row < rows ? row : rows - 1) * ldx;
  const int whole = n & ~7, rest = n - whole;
  iv4 held[CH][words8<T>()];  // all loads in flight together, those behind the row at its start
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int j = (c * TPR + tid) * 8;
#pragma unroll
    for (int h = 0; h < words8<T>(); ++h) held[c][h] = whole > 0 ? word8(x + (j < whole ? j : 0), h) : iv4{0, 0, 0, 0};
  }
  const float last = tid < rest ? (float)x[whole + tid] : 0.0f;
  unsigned mx = __float_as_uint(last) & 0x7FFFFFFFu;
  float v[CH][8];
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    unpack8<T>(held[c], v[c]);
    mx = max_abs8(v[c], mx);  // a repeat of the row's start changes nothing
  }
  for (long long j = (long long)(CH * TPR + tid) * 8; j < whole; j += TPR * 8) {
    float w[8];
    load8(x + j, w);
    mx = max_abs8(w, mx);
  }
  mx = wave_max_u32(mx);
  if (TPR == 256) {
    if ((threadIdx.x & 63) == 0) wmx[threadIdx.x >> 6] = mx;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 4; ++w) mx = wmx[w] > mx ? wmx[w] : mx;
  }
  if (row >= rows) return;
  const RowScale rs(mx);
  if (tid == 0) scale[row] = rs.scale();
  int8_t* q = Q + row * ldq;
  auto emit = [&](long long j, const float (&w)[8]) {
    int k[8];
    rs.quantize(w, k);
    iv2_any o;
    o[0] = (int)pack4(k[0], k[1], k[2], k[3]);
    o[1] = (int)pack4(k[4], k[5], k[6], k[7]);
    *reinterpret_cast<iv2_any*>(q + j) = o;
  };
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int j = (c * TPR + tid) * 8;
    if (j < whole) emit(j, v[c]);
  }
  for (long long j = (long long)(CH * TPR + tid) * 8; j < whole; j += TPR * 8) {
    float w[8];
    load8(x + j, w);
    emit(j, w);
  }
  if (tid < rest) {
    const float w[8] = {last, 0, 0, 0, 0, 0, 0, 0};
    int k[8];
    rs.quantize(w, k);
    q[whole + tid] = (int8_t)k[0];
  }
  if (tid < np - n) q[n + tid] = 0;
}

template <typename T>
static hipError_t quantize_typed(const T* X, long long rows, int n, long long ldx, int8_t* Q, long long ldq, int np,
                                 float* scale, hipStream_t st) {
  // runs of 2^23 rows: a launch holds below 2^32 threads
  for (long long r = 0; r < rows; r += 1ll << 23) {
    const long long c = rows - r < (1ll << 23) ? rows - r : 1ll << 23;
    auto go = [&](auto kernel, long long blocks) {
      hipLaunchKernelGGL(kernel, dim3((unsigned)blocks), dim3(256), 0, st, X + r * ldx, c, n, ldx, Q + r * ldq, ldq, np,
                         scale + r);
    };
    if (n <= 64 * 8 * 2) go(quantize_kernel<T, 64, 2>, (c + 3) / 4);
    else if (n <= 256 * 8 * 2) go(quantize_kernel<T, 256, 2>, c);
    else go(quantize_kernel<T, 256, 5>, c);
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
// Workgroup: 16 output channels and 16 NT tokens; the row length goes round eight waves in chunks of 128
// bytes, so that each wave reads whole cache lines of W and two chunks' loads are in flight.  (32
// channels a workgroup read X half as often and were slower wherever that left fewer workgroups than
// CUs, and no faster elsewhere.)
// MFMA D(16 x 16) += A(16 x 64) B(64 x 16): A row = channel, B column = token, lane l holding the
// 16 bytes at 16 (l / 16) of row (column) l % 16 of the step.  The waves' partial tiles add in LDS.
//
// XT int8_t: the tokens are 8-bit rows.  Else they are quantised here first, by every workgroup for
// itself into LDS while the first loads of W are on their way.
constexpr int kFewWaves = 8;
constexpr int kFewTokens = 16;        // one column tile; up to 32 take two
constexpr int kFewFused = 8;          // most tokens quantised on the way
constexpr int kFewLds = 48 * 1024;    // bytes of their rows

// distance of the quantised rows in LDS: 16 rows' pieces of one column in different banks
__host__ __device__ constexpr int few_pitch(int n) { return (n + 127) / 128 * 128 % 256 == 0 ? (n + 127) / 128 * 128 + 16
                                                                                           : (n + 127) / 128 * 128 + 144; }

// The tokens' rows quantised into LDS by the workgroup's eight waves, G = 8, 4, 2 or 1 of them to a
// token (tokens <= 8), and their scales; ends with a barrier.
template <typename T>
__device__ __forceinline__ void few_quantize(const T* __restrict__ X, long long ldx, int tokens, int n,
                                             int8_t* __restrict__ q, float* srow, unsigned* wmx) {
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int G = tokens == 1 ? 8 : tokens == 2 ? 4 : tokens <= 4 ? 2 : 1, t = wv / G, first = ((wv % G) * 64 + lane) * 8, step = 512 * G;
  const bool mine = t < tokens;
  const T* x = X + (mine ? t : 0) * ldx;
  constexpr int H = 2;  // steps kept in registers; a longer row's rest is read again
  float v[H][8];
  unsigned mx = 0u;
  auto get = [&](int j, float (&w)[8]) {
    if (j + 8 <= n) load8(x + j, w);
    else load8_tail(x + j, (long long)n - j, w);
  };
  auto top = [&](const float (&w)[8]) { mx = max_abs8(w, mx); };
#pragma unroll
  for (int h = 0; h < H; ++h) get(first + h * step, v[h]);
#pragma unroll
  for (int h = 0; h < H; ++h) top(v[h]);
  for (int j = first + H * step; j < n; j += step) {
    float w[8];
    get(j, w);
    top(w);
  }
  mx = wave_max_u32(mx);
  if (lane == 0) wmx[wv] = mx;
  __syncthreads();
  if (mine) {
    for (int g = 0; g < G; ++g) {
      const unsigned o = wmx[t * G + g];
      mx = o > mx ? o : mx;
    }
    const RowScale rs(mx);
    if (wv % G == 0 && lane == 0) srow[t] = rs.scale();
    const int np = (n + 127) / 128 * 128;
    int8_t* o = q + t * few_pitch(n);
    auto emit = [&](int j, const float (&w)[8]) {
      int k[8];
      rs.quantize(w, k);
      if (j < np) {
        *reinterpret_cast<unsigned*>(o + j) = pack4(k[0], k[1], k[2], k[3]);
        *reinterpret_cast<unsigned*>(o + j + 4) = pack4(k[4], k[5], k[6], k[7]);
      }
    };
#pragma unroll
    for (int h = 0; h < H; ++h) emit(first + h * step, v[h]);
    for (int j = first + H * step; j < np; j += step) {
      float w[8];
      get(j, w);
      emit(j, w);
    }
  }
  __syncthreads();
}

template <int NT, typename XT, typename YT>
__global__ void __launch_bounds__(64 * kFewWaves) few_kernel(const int8_t* __restrict__ W, long long ldw, int m, int n,
                                                             const float* __restrict__ sw, const XT* __restrict__ X,
                                                             long long ldx, int tokens, const float* __restrict__ sx,
                                                             YT* __restrict__ Y, long long ldy) {
  constexpr bool FUSED = !__is_same(XT, int8_t);
  static_assert(!FUSED || (NT == 1 && kFewFused <= 16), "quantised on the way: one column tile");
  extern __shared__ __attribute__((aligned(16))) int8_t rows[];
  __shared__ int red[kFewWaves][NT * 256];
  __shared__ float srow[16];
  __shared__ unsigned wmx[kFewWaves];
  // the wave's number in a scalar register: the branches on it must be jumps, since MFMA runs whatever
  // the lane mask
  const int tid = threadIdx.x, lane = tid & 63, wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lr = lane & 15, gg = lane >> 4;
  const int r0 = blockIdx.x * 16;
  const long long t0 = blockIdx.y * (16ll * NT);
  const int8_t* wr = W + (long long)(r0 + lr < m ? r0 + lr : m - 1) * ldw;
  const int8_t* xr[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const long long c = t0 + 16 * t + lr < tokens ? t0 + 16 * t + lr : tokens - 1;
    xr[t] = FUSED ? rows + c * few_pitch(n) : reinterpret_cast<const int8_t*>(X + c * ldx);
  }
  iv4 acc[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) acc[t] = iv4{0, 0, 0, 0};
  const int full = n / 128;
  iv4 a[4], b[4][NT];
  auto load_w = [&](int c, int u) {
#pragma unroll
    for (int h = 0; h < 2; ++h) a[2 * u + h] = *reinterpret_cast<const iv4_any*>(wr + 128 * c + 64 * h + 16 * gg);
  };
  auto load_x = [&](int c, int u) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const int8_t* p = xr[t] + 128 * c + 64 * h + 16 * gg;
        b[2 * u + h][t] = FUSED ? *reinterpret_cast<const iv4*>(p) : (iv4)*reinterpret_cast<const iv4_any*>(p);
      }
  };
  auto mul = [&](int u) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int t = 0; t < NT; ++t)
        acc[t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(a[2 * u + h], b[2 * u + h][t], acc[t], 0, 0, 0);
  };
  int c = wv;
  const bool two = c + kFewWaves < full;
  if constexpr (FUSED) {
    if (c < full) load_w(c, 0);
    if (two) load_w(c + kFewWaves, 1);
    few_quantize(X, ldx, tokens, n, rows, srow, wmx);
    if (c < full) {
      load_x(c, 0);
      if (two) load_x(c + kFewWaves, 1);
      mul(0);
      if (two) mul(1);
      c += two ? 2 * kFewWaves : kFewWaves;
    }
  }
  for (; c + kFewWaves < full; c += 2 * kFewWaves) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      load_w(c + u * kFewWaves, u);
      load_x(c + u * kFewWaves, u);
    }
    mul(0);
    mul(1);
  }
  if (c < full) {
    load_w(c, 0);
    load_x(c, 0);
    mul(0);
    c += kFewWaves;
  }
  if (c == full && n % 128 != 0) {  // the rows' end: one wave
    const int k = 128 * full + 16 * gg;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      a[h] = n >= 16 ? row_load(wr, k + 64 * h, n) : row_short(wr, k + 64 * h, n);
#pragma unroll
      for (int t = 0; t < NT; ++t)
        b[h][t] = FUSED ? *reinterpret_cast<const iv4*>(xr[t] + k + 64 * h)  // zeros behind the row there
                        : n >= 16 ? row_load(xr[t], k + 64 * h, n) : row_short(xr[t], k + 64 * h, n);
    }
    if (n >= 16) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        a[h] = row_end(a[h], k + 64 * h, n);
        if (!FUSED) {
#pragma unroll
          for (int t = 0; t < NT; ++t) b[h][t] = row_end(b[h][t], k + 64 * h, n);
        }
      }
    }
    mul(0);
  }
  // acc[q] = D(channel 4 gg + q, token lr): stored token-major
#pragma unroll
  for (int t = 0; t < NT; ++t) *reinterpret_cast<iv4*>(&red[wv][(t * 16 + lr) * 16 + 4 * gg]) = acc[t];
  __syncthreads();
  for (int x = tid; x < NT * 256; x += 64 * kFewWaves) {
    const long long tok = t0 + (x >> 4);
    const int o = r0 + (x & 15);
    if (tok < tokens && o < m) {
      int sum = 0;
#pragma unroll
      for (int w = 0; w < kFewWaves; ++w) sum += red[w][x];
      store_y(Y + tok * ldy + o, (float)sum * sw[o] * (FUSED ? srow[tok & 15] : sx[tok]));
    }
  }
}

// ---- many tokens: the tiles of igemm.hpp ----------------------------------------------------
// y = sum w_o s_t.  The accumulators times w_o pass through LDS, 32 rows of the wave's columns at a
// time, so that each lane stores 16 bytes of a row: four or eight times fewer stores than from the
// accumulators, whole cache lines, and one guard each.  (Code run once costs too: its instructions
// come from memory.)  The rows' distance in LDS, 32 FN + 8 words, puts the two rows that a wave
// writes at once in different banks.
template <typename YT>
struct ScaledY {
  const float* sx;
  const float* sw;
  YT* Y;
  long long ldy;
  static constexpr bool kLds = true, kAligned = false;
  __device__ __forceinline__ void at(long long m0, long long n0) {
    sx += m0;
    sw += n0;
    Y += m0 * ldy + n0;
  }
  template <int FM, int FN>
  __device__ __forceinline__ void finish(const iv16 (&acc)[FM][FN], int r0, int c0, int mr, int nr, float* l) const {
    constexpr int W = 32 * FN, P = W + 8, E = 16 / sizeof(YT), CH = W / E;  // columns, distance, a store's elements
    const int lane = threadIdx.x & 63, lr = lane & 31, lg = lane >> 5;
    float w[FN];
#pragma unroll
    for (int j = 0; j < FN; ++j) w[j] = sw[c0 + 32 * j + lr < nr ? c0 + 32 * j + lr : nr - 1];
#pragma unroll
    for (int i = 0; i < FM; ++i) {
#pragma unroll
      for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int e = 0; e < 16; ++e) l[(8 * (e >> 2) + (e & 3) + 4 * lg) * P + 32 * j + lr] = (float)acc[i][j][e] * w[j];
#pragma unroll
      for (int x0 = 0; x0 < 32 * CH; x0 += 64) {
        const int x = x0 + lane, row = x / CH, ch = x % CH * E, r = r0 + 32 * i + row, c = c0 + ch;
        const float s = sx[r < mr ? r : mr - 1];
        float v[E];
#pragma unroll
        for (int q = 0; q < E; q += 4) {
          const fv4 f = *reinterpret_cast<const fv4*>(l + row * P + ch + q);
#pragma unroll
          for (int e = 0; e < 4; ++e) v[q + e] = f[e] * s;
        }
        if (r < mr) {
          YT* y = Y + r * ldy + c;
          if (c + E <= nr) {
            typedef YT ev __attribute__((ext_vector_type(E)));
            ev o;
#pragma unroll
            for (int e = 0; e < E; ++e) o[e] = (YT)v[e];
            *reinterpret_cast<iv4_any*>(y) = __builtin_bit_cast(iv4, o);
          } else {
#pragma unroll
            for (int e = 0; e < E; ++e)
              if (c + e < nr) y[e] = (YT)v[e];
          }
        }
      }
    }
  }
  __device__ __forceinline__ void put4(long long r, int c, int M, const iv4& sum) const {
    const float w = sw[c];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (r + e < M) store_y(Y + (r + e) * ldy + c, (float)sum[e] * w * sx[r + e]);
  }
};

// 16 NT tokens a workgroup; the grid's limits are kept by taking the tokens in runs
template <int NT, typename YT>
static hipError_t few_launch(const int8_t* W, const float* sw, int m, int n, long long ldw, const int8_t* Xq,
                             const float* sx, int tokens, long long ldx, YT* Y, long long ldy, hipStream_t st) {
  const unsigned gx = (unsigned)((m + 15ll) / 16);
  const long long groups = (tokens + 16ll * NT - 1) / (16 * NT);
  for (long long g = 0; g < groups; g += 65535) {
    const unsigned gy = (unsigned)(groups - g < 65535 ? groups - g : 65535);
    const long long t0 = 16ll * NT * g;
    hipLaunchKernelGGL((few_kernel<NT, int8_t, YT>), dim3(gx, gy), dim3(64 * kFewWaves), 0, st, W, ldw, m, n, sw,
                       Xq + t0 * ldx, ldx, (int)(tokens - t0), sx + t0, Y + t0 * ldy, ldy);
  }
  return hipGetLastError();
}

template <typename YT>
static hipError_t product_typed(const int8_t* W, const float* sw, int m, int n, long long ldw, const int8_t* Xq,
                                const float* sx, int tokens, long long ldx, YT* Y, long long ldy, void* parts,
                                hipStream_t st) {
  if (tokens <= kFewTokens) return few_launch<1>(W, sw, m, n, ldw, Xq, sx, tokens, ldx, Y, ldy, st);
  // rows too short for the tiles' loads come here whatever their number
  if (tokens <= 32 || n < 16) return few_launch<2>(W, sw, m, n, ldw, Xq, sx, tokens, ldx, Y, ldy, st);
  const long long run = tile_run(m);
  if (tokens <= run) return tile_product(Xq, ldx, tokens, W, ldw, m, n, ScaledY<YT>{sx, sw, Y, ldy}, parts, st);
  // more tiles than a launch holds: the tokens in runs (never split, there are tiles enough)
  for (long long t = 0; t < tokens; t += run) {
    const int c = tokens - t < run ? (int)(tokens - t) : (int)run;
    const hipError_t e = tile_whole(Xq + t * ldx, ldx, c, W, ldw, m, n, ScaledY<YT>{sx + t, sw, Y + t * ldy, ldy}, st);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <typename XT, typename YT>
static hipError_t fused_typed(const int8_t* W, const float* sw, int m, int n, long long ldw, const XT* X, int tokens,
                              long long ldx, YT* Y, long long ldy, hipStream_t st) {
  hipLaunchKernelGGL((few_kernel<1, XT, YT>), dim3((unsigned)((m + 15ll) / 16)), dim3(64 * kFewWaves),
                     (size_t)tokens * few_pitch(n), st, W, ldw, m, n, sw, X, ldx, tokens, nullptr, Y, ldy);
  return hipGetLastError();
}

// Whether the tokens are quantised within the product's own launch: every workgroup does it for itself,
// which pays while that is less than a launch more.  Measured (kernels alone), m x n and tokens, fused /
// two launches, us: 2560 x 2560, 1 token 4.7 / 6.2, 4 5.8 / 6.6, 8 6.9 / 6.8; 9728 x 2560, 1 7.5 / 8.9, 4
// 9.8 / 9.7; 2560 x 9728, 1 8.3 / 11.5, 2 10.3 / 12.0, 3 12.2 / 12.3; 700 x 700, 8 4.5 / 5.7.
static bool fused(int x_type, long long tokens, int n, int m) {
  return x_type != 3 && tokens <= kFewFused && tokens * few_pitch(n) <= kFewLds &&
         (double)tokens * n * (m > 4096 ? m / 4096.0 : 1.0) <= 20000.0;
}

// Workspace: the scales and quantised rows (padded to a multiple of 16 bytes) of tokens that come as
// floating-point rows, and the parts of a split product.
static size_t al256(size_t x) { return (x + 255) & ~(size_t)255; }
static long long pad16(long long n) { return (n + 15) & ~15ll; }
static size_t rows_bytes(int x_type, long long tokens, int n, int m) {
  return x_type == 3 || fused(x_type, tokens, n, m) ? 0 : al256((size_t)tokens * 4) + al256((size_t)tokens * pad16(n));
}
size_t product_workspace_bytes(int x_type, long long tokens, int n, int m) {
  return rows_bytes(x_type, tokens, n, m) + (tokens > 32 && n >= 16 ? tile_plan(tokens, m, n).bytes : 0);
}

template <typename YT>
static hipError_t product_to(const int8_t* W, const float* sw, int m, int n, long long ldw, const void* X, int x_type,
                             const float* sx, int tokens, long long ldx, YT* Y, long long ldy, void* ws,
                             hipStream_t st) {
  if (fused(x_type, tokens, n, m)) {
    switch (x_type) {
      case 0: return fused_typed(W, sw, m, n, ldw, static_cast<const float*>(X), tokens, ldx, Y, ldy, st);
      case 1: return fused_typed(W, sw, m, n, ldw, static_cast<const _Float16*>(X), tokens, ldx, Y, ldy, st);
      default: return fused_typed(W, sw, m, n, ldw, static_cast<const __bf16*>(X), tokens, ldx, Y, ldy, st);
    }
  }
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
  return product_typed(W, sw, m, n, ldw, Xq, sx, tokens, ldx, Y, ldy,
                       static_cast<char*>(ws) + rows_bytes(x_type, tokens, n, m), st);
}

hipError_t product_run(const int8_t* W, const float* sw, int m, int n, long long ldw, const void* X, int x_type,
                       const float* sx, int tokens, long long ldx, void* Y, int y_type, long long ldy, void* ws,
                       hipStream_t st) {
  switch (y_type) {
    case 0: return product_to(W, sw, m, n, ldw, X, x_type, sx, tokens, ldx, static_cast<float*>(Y), ldy, ws, st);
    case 1: return product_to(W, sw, m, n, ldw, X, x_type, sx, tokens, ldx, static_cast<_Float16*>(Y), ldy, ws, st);
    case 2: return product_to(W, sw, m, n, ldw, X, x_type, sx, tokens, ldx, static_cast<__bf16*>(Y), ldy, ws, st);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace externd
