// Softmax cross entropy of tokens through a model's output matrix, and its gradient, without the logits
// kept.
//
//   z_tv = x_t . w_v
//   loss_t = g_t (log sum_v exp z_tv - z_t,target)
//   P_tv = g_t (exp(z_tv - m_t) / S_t - [v = target_t]),   m_t = max_v z_tv,  S_t = sum_v exp(z_tv - m_t)
//   dX = P W,   dW = P^T X
//
// The loss is one product whose tiles (columns: tokens, rows: words) reduce their logits to a maximum and a
// sum of exponentials for each token; a second launch joins the tiles.  The gradient takes the vocabulary in pieces: a
// piece's logits are formed again and leave as P, in X's type, which two products then read while it is in the cache.  dX is
// summed over the pieces in fp32.  So the work is four products for loss and both gradients, and the matrix cores bound it
// but for few tokens, where reading W does.
//
// Roundings: sums of products (fp32's in runs), exponentials and a tile's sum of them are fp32, the sums over tiles, log S and
// the loss fp64.  P is rounded once to X's type for the products that follow (as a gradient of logits held in that
// type would be); its errors are independent and each at most half a step, like those of the
// result's own rounding, and the largest of a row, the target's, is put back into dX.  fp16 P carries a power of two that
// brings the largest |g| to 2^14 .. 2^15, taken out of the sums in fp32, so that small probabilities stay above fp16's
// smallest numbers.
//
// Measured (bf16, 2048 x 2560, us a piece of 32768 words): logits and P 310, dX 301, dW 312; the loss alone 4096 x 2560 x
// 131072 2250; one row, 1024 x 32768: 14.5 (W at 4.6 TB/s) and 7 of the launches around.
//
// Rows that do not count (target outside the vocabulary, g = 0) are left out: the others' rows are gathered
// at the start, their number stays on the device and cuts the products.
#pragma once
#include <type_traits>

#include "common.hpp"
#include "externd_internal.hpp"
#include "fgemm.hpp"

namespace externd {

// what is kept of a counted row
struct TokenCoef {
  float m, gi, g;  // largest logit, g 2^scale / S, g 2^scale
  int target;
};

struct TokenMeta {
  int count;   // rows that count
  int scale;   // P carries 2^scale
};

// exp(d), d <= 0: log2 e in two numbers, the first cut towards zero, so that an exponent is off by its own
// rounding alone (one number shifts every exponential of a row the same way); 0 below 2^-126
__device__ __forceinline__ float exp_neg(float d) {
  constexpr double c = 1.4426950408889634;
  constexpr float hi = 1.44269502162933349609375f;  // fp32 just below log2 e
  constexpr float lo = (float)(c - (double)hi);
  return __builtin_amdgcn_exp2f(fmaf(d, hi, d * lo));
}

// |g| for the power of two that P carries: of the numbers among the weights, so that an infinity (whose row is lost in any
// case) leaves the other rows' P where it was
__device__ __forceinline__ float finite_size(float g) { return fabsf(g) <= __FLT_MAX__ ? fabsf(g) : 0.0f; }

// A row gathered into an aligned copy by `threads` threads: row r of X (zeros where that is -1), n elements and zeros up to nq.
template <typename T>
__device__ __forceinline__ void gather_row(const T* __restrict__ X, long long ldx, int n, long long r, T* __restrict__ out, int nq,
                                           int thread, int threads) {
  constexpr int E = 16 / sizeof(T);
  for (int j = thread * E; j < nq; j += threads * E) {
    iv4 v = {0, 0, 0, 0};
    if (r >= 0) {
      const T* x = X + r * ldx + j;
      if (j + E <= n) {
        v = *reinterpret_cast<const iv4_any*>(x);
      } else {
        typedef T ev __attribute__((ext_vector_type(E)));
        ev t;
#pragma unroll
        for (int e = 0; e < E; ++e) t[e] = j + e < n ? x[e] : (T)0.0f;
        v = __builtin_bit_cast(iv4, t);
      }
    }
    *reinterpret_cast<iv4*>(out + j) = v;
  }
}

// ---- rows that count ------------------------------------------------------------------------------
// One workgroup: list[i] = the i-th row that counts, place[r] its inverse (-1: does not count), and the
// rows' g and targets in the list's order, up to `padded` with g = 0.  loss and stats (may be null) of the others are 0.
constexpr int kTokenScan = 1024;
template <typename TI>
__global__ void __launch_bounds__(kTokenScan) token_rows_kernel(const TI* __restrict__ target, const float* __restrict__ weight,
                                                                int rows, int padded, int V, bool scaled, TokenMeta* meta,
                                                                int* __restrict__ list, int* __restrict__ place,
                                                                TokenCoef* __restrict__ coef, float* __restrict__ loss,
                                                                float* __restrict__ stats) {
  __shared__ int sums[kTokenScan / 64];
  __shared__ float tops[kTokenScan / 64];
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  int base = 0;
  float top = 0.0f;
  for (int r0 = 0; r0 < rows; r0 += kTokenScan) {
    const int r = r0 + (int)threadIdx.x;
    const long long tg = r < rows ? (long long)target[r] : -1;
    const float g = r < rows ? (weight ? weight[r] : 1.0f) : 0.0f;
    const bool counts = tg >= 0 && tg < V && g != 0.0f;
    const unsigned long long mask = __ballot(counts);
    if (lane == 0) sums[wv] = __popcll(mask);
    __syncthreads();
    int before = base, all = 0;
#pragma unroll
    for (int w = 0; w < kTokenScan / 64; ++w) {
      const int s = sums[w];
      before += w < wv ? s : 0;
      all += s;
    }
    const int at = before + __popcll(mask & ((1ull << lane) - 1));
    if (counts) {
      list[at] = r;
      coef[at] = TokenCoef{0.0f, 0.0f, g, (int)tg};
      top = fmaxf(top, finite_size(g));
    }
    if (r < rows) {
      place[r] = counts ? at : -1;
      if (!counts && loss) {
        loss[r] = 0.0f;
        stats[2ll * r] = 0.0f;
        stats[2ll * r + 1] = 0.0f;
      }
    }
    base += all;
    __syncthreads();
  }
  for (int i = base + (int)threadIdx.x; i < padded; i += kTokenScan) {
    list[i] = -1;
    coef[i] = TokenCoef{0.0f, 0.0f, 0.0f, -1};
  }
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) top = fmaxf(top, __shfl_xor(top, d));
  if (lane == 0) tops[wv] = top;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 0; w < kTokenScan / 64; ++w) top = fmaxf(top, tops[w]);
    int e = 0;
    if (scaled && top > 0.0f) e = 14 - ilogbf(top);
    *meta = TokenMeta{base, e};
  }
}

// Up to 1024 rows: the same and the gathering in one launch.  Workgroup i finds the i-th row that counts for itself (four
// rows a thread) and copies it; the first writes the lists too.
template <typename T, typename TI>
__global__ void __launch_bounds__(256) token_start_kernel(const TI* __restrict__ target, const float* __restrict__ weight, int rows,
                                                          int padded, int V, bool scaled, TokenMeta* meta, int* __restrict__ list,
                                                          int* __restrict__ place, TokenCoef* __restrict__ coef,
                                                          float* __restrict__ loss, float* __restrict__ stats,
                                                          const T* __restrict__ X, long long ldx, int n, T* __restrict__ out, int nq) {
  __shared__ int sums[4];
  __shared__ float tops[4];
  __shared__ int mine;
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  long long tg[4];
  float g[4], top = 0.0f;
  int counts[4], n4 = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int r = 4 * (int)threadIdx.x + e;
    tg[e] = r < rows ? (long long)target[r] : -1;
    g[e] = r < rows ? (weight ? weight[r] : 1.0f) : 0.0f;
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    counts[e] = tg[e] >= 0 && tg[e] < V && g[e] != 0.0f;
    n4 += counts[e];
    top = fmaxf(top, counts[e] ? finite_size(g[e]) : 0.0f);
  }
  int before = n4;  // the sum over the lanes up to this one
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(before, d);
    before += lane >= d ? o : 0;
    top = fmaxf(top, __shfl_xor(top, d));
  }
  if (lane == 63) sums[wv] = before;
  if (lane == 0) tops[wv] = top;
  if (threadIdx.x == 0) mine = -1;
  __syncthreads();
  before -= n4;
  int count = 0;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    before += w < wv ? sums[w] : 0;
    count += sums[w];
    top = fmaxf(top, tops[w]);
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int r = 4 * (int)threadIdx.x + e;
    if (counts[e] && before == (int)blockIdx.x) mine = r;
    if (blockIdx.x == 0 && r < rows) {
      place[r] = counts[e] ? before : -1;
      if (counts[e]) {
        list[before] = r;
        coef[before] = TokenCoef{0.0f, 0.0f, g[e], (int)tg[e]};
      } else if (loss) {
        loss[r] = 0.0f;
        stats[2ll * r] = 0.0f;
        stats[2ll * r + 1] = 0.0f;
      }
    }
    before += counts[e];
  }
  if (blockIdx.x == 0) {
    for (int i = count + (int)threadIdx.x; i < padded; i += 256) {
      list[i] = -1;
      coef[i] = TokenCoef{0.0f, 0.0f, 0.0f, -1};
    }
    if (threadIdx.x == 0) *meta = TokenMeta{count, scaled && top > 0.0f ? 14 - ilogbf(top) : 0};
  }
  __syncthreads();
  gather_row(X, ldx, n, mine, out + blockIdx.x * (long long)nq, nq, (int)threadIdx.x, 256);
}

// Row i of `out` is row list[i] of X (zeros where that is -1), or row i without a list.
template <typename T>
__global__ void __launch_bounds__(256) gather_kernel(const T* __restrict__ X, long long ldx, int n, const int* __restrict__ list,
                                                     T* __restrict__ out, int nq) {
  const long long i = blockIdx.x;
  gather_row(X, ldx, n, list ? list[i] : i, out + i * nq, nq, (int)(blockIdx.y * 256 + threadIdx.x), (int)gridDim.y * 256);
}

// ---- the tiles' epilogues ---------------------------------------------------------------------------
// Rows of D are words, columns tokens: a lane holds one token's logits, so most of a reduction over
// words stays in its registers.
struct TokenStats {
  const TokenCoef* coef;
  float2* parts;  // [word tiles][padded]
  float* zt;      // logits of the targets
  long long padded;
  int first;      // of the piece's words
  static constexpr bool kLds = true;
  template <typename T, int BM, int BN, int WR, int WC, int FM, int FN, int LDS>
  __device__ __forceinline__ void finish(fv16 (&acc)[FM][FN], long long m0, long long n0, int mr, int, int wr, int wc,
                                         int8_t* lds) const {
    const int lane = threadIdx.x & 63, lr = lane & 31, lg = lane >> 5;
    const int r0 = wr * (BM / WR), c0 = wc * (BN / WC);
    float2* red = reinterpret_cast<float2*>(lds);  // [WR][BN]
    static_assert(WR * BN * 8 <= LDS, "epilogue in LDS");
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      const long long t = n0 + c0 + 32 * j + lr;
      const long long d = (long long)coef[t].target - first - m0 - r0 - 4 * lg;  // of the target among this lane's words
      if (__any(d >= 0 && d < 32 * FM)) {
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
          for (int e = 0; e < 16; ++e)
            if (d == 32 * i + 8 * (e >> 2) + (e & 3)) zt[t] = acc[i][j][e];
      }
      if (mr < BM) {
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
          for (int e = 0; e < 16; ++e)
            if (r0 + 32 * i + 8 * (e >> 2) + 4 * lg + (e & 3) >= mr) acc[i][j][e] = -__builtin_inff();
      }
      float m = -__FLT_MAX__, s = 0.0f;  // words of -inf alone: s = 0
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int e = 0; e < 16; ++e) m = fmaxf(m, acc[i][j][e]);
      m = fmaxf(m, __shfl_xor(m, 32));
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int e = 0; e < 16; ++e) s += exp_neg(acc[i][j][e] - m);
      s += __shfl_xor(s, 32);
      if (lg == 0) red[wr * BN + c0 + 32 * j + lr] = make_float2(m, s);
    }
    __syncthreads();
    if ((int)threadIdx.x < BN) {
      float m = -__FLT_MAX__, s = 0.0f;
#pragma unroll
      for (int w = 0; w < WR; ++w) m = fmaxf(m, red[w * BN + threadIdx.x].x);
#pragma unroll
      for (int w = 0; w < WR; ++w) {
        const float2 p = red[w * BN + threadIdx.x];
        s += p.y * exp_neg(p.x - m);
      }
      parts[m0 / BM * padded + n0 + threadIdx.x] = make_float2(m, s);
    }
  }
};

// A tile stored with its columns as rows: the accumulators pass through LDS, 32 columns of up to 256 bytes at
// a time, so that each lane stores 16 bytes of a row.  A lane's four consecutive rows of D are one write there.
//   value(j, i, e) gives the OT to store, put(column, row, piece) stores 16 bytes from `row` on
template <typename OT, int BM, int BN, int WR, int WC, int FM, int FN, int LDS, typename V, typename P>
__device__ __forceinline__ void store_columns(int wr, int wc, int8_t* lds, const V& value, const P& put) {
  constexpr int ES = (int)sizeof(OT), IC = FM * 32 * ES <= 256 ? FM : 256 / (32 * ES), RB = IC * 32 * ES, PITCH = RB + 16;
  static_assert(FM % IC == 0, "whole chunks");
  constexpr int kBytes = 32 * PITCH;
  static_assert(kBytes * WR * WC <= LDS, "epilogue in LDS");
  const int lane = threadIdx.x & 63, lr = lane & 31, lg = lane >> 5, wv = wr * WC + wc;
  int8_t* l = lds + wv * kBytes;
  const int r0 = wr * (BM / WR), c0 = wc * (BN / WC);
#pragma unroll
  for (int j = 0; j < FN; ++j)
#pragma unroll
    for (int i0 = 0; i0 < FM; i0 += IC) {
#pragma unroll
      for (int i = 0; i < IC; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          typedef OT ov __attribute__((ext_vector_type(4)));
          ov v;
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = value(j, i0 + i, 4 * q + e);
          *reinterpret_cast<ov*>(l + lr * PITCH + (32 * i + 8 * q + 4 * lg) * ES) = v;
        }
      constexpr int PR = RB / 16;  // pieces of a row
#pragma unroll
      for (int x0 = 0; x0 < 32 * PR; x0 += 64) {
        const int x = x0 + lane, row = x / PR, c = x % PR;
        const iv4 v = *reinterpret_cast<const iv4*>(l + row * PITCH + c * 16);
        put(c0 + 32 * j + row, r0 + 32 * i0 + c * (16 / ES), v);
      }
    }
}

// P of a piece of the vocabulary, [token][word of the piece]; words behind the last are zeros
template <typename PT>
struct TokenP {
  const TokenCoef* coef;
  PT* P;
  float* lost;  // what the rounding of the target's P takes
  long long ldp;
  int first;    // of the piece's words
  static constexpr bool kLds = true;
  template <typename T, int BM, int BN, int WR, int WC, int FM, int FN, int LDS>
  __device__ __forceinline__ void finish(fv16 (&acc)[FM][FN], long long m0, long long n0, int mr, int, int wr, int wc,
                                         int8_t* lds) const {
    const int lane = threadIdx.x & 63, lr = lane & 31, lg = lane >> 5;
    const int r0 = wr * (BM / WR), c0 = wc * (BN / WC);
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      const TokenCoef c = coef[n0 + c0 + 32 * j + lr];
      const long long d64 = (long long)c.target - first - m0 - r0 - 4 * lg;
      const int d = d64 >= 0 && d64 < 32 * FM ? (int)d64 : -1;  // the target among this lane's words
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const float q = c.gi * exp_neg(acc[i][j][e] - c.m);
          acc[i][j][e] = d == 32 * i + 8 * (e >> 2) + (e & 3) ? q - c.g : q;
        }
      if (sizeof(PT) < 4 && __any(d >= 0)) {
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
          for (int e = 0; e < 16; ++e)
            if (d == 32 * i + 8 * (e >> 2) + (e & 3)) lost[n0 + c0 + 32 * j + lr] = acc[i][j][e] - (float)(PT)acc[i][j][e];
      }
    }
    if (mr < BM) {
#pragma unroll
      for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
          for (int e = 0; e < 16; ++e)
            acc[i][j][e] = r0 + 32 * i + 8 * (e >> 2) + 4 * lg + (e & 3) < mr ? acc[i][j][e] : 0.0f;
    }
    PT* p = P + n0 * ldp + m0;
    store_columns<PT, BM, BN, WR, WC, FM, FN, LDS>(
        wr, wc, lds, [&](int j, int i, int e) { return (PT)acc[i][j][e]; },
        [&](int c, int r, const iv4& v) { *reinterpret_cast<iv4*>(p + c * ldp + r) = v; });
  }
};

// dX's share of a piece, fp32 [token][padded row], added to the earlier pieces'; each part of the length has its own
struct TokenDX {
  float* sum;
  long long stride;  // of the parts
  int nq;
  bool first;
  static constexpr bool kLds = true;
  template <typename T, int BM, int BN, int WR, int WC, int FM, int FN, int LDS>
  __device__ __forceinline__ void finish(fv16 (&acc)[FM][FN], long long m0, long long n0, int mr, int, int wr, int wc,
                                         int8_t* lds) const {
    float* p = sum + blockIdx.y * stride + n0 * nq + m0;
    store_columns<float, BM, BN, WR, WC, FM, FN, LDS>(
        wr, wc, lds, [&](int j, int i, int e) { return acc[i][j][e]; },
        [&](int c, int r, const iv4& v) {
          if (r >= mr) return;
          fv4* o = reinterpret_cast<fv4*>(p + (long long)c * nq + r);
          const fv4 x = __builtin_bit_cast(fv4, v);
          *o = first ? x : *o + x;
        });
  }
};

// dW of a piece, [word][n]
template <typename OT>
struct TokenDW {
  const TokenMeta* meta;
  OT* dW;  // of the piece
  long long ldw;
  int n;
  static constexpr bool kLds = true;
  template <typename T, int BM, int BN, int WR, int WC, int FM, int FN, int LDS>
  __device__ __forceinline__ void finish(fv16 (&acc)[FM][FN], long long m0, long long n0, int, int nr, int wr, int wc,
                                         int8_t* lds) const {
    constexpr int E = 16 / (int)sizeof(OT);
    const int scale = -meta->scale;
    const int left = n - (int)m0;
    OT* p = dW + n0 * ldw + m0;
    store_columns<OT, BM, BN, WR, WC, FM, FN, LDS>(
        wr, wc, lds,
        [&](int j, int i, int e) { return (OT)(__is_same(OT, _Float16) ? ldexpf(acc[i][j][e], scale) : acc[i][j][e]); },
        [&](int c, int r, const iv4& v) {
          if (c >= nr || r >= left) return;
          OT* o = p + (long long)c * ldw + r;
          if (r + E <= left) {
            *reinterpret_cast<iv4_any*>(o) = v;
          } else {
            typedef OT ev __attribute__((ext_vector_type(E)));
            const ev t = __builtin_bit_cast(ev, v);
#pragma unroll
            for (int e = 0; e < E; ++e)
              if (r + e < left) o[e] = t[e];
          }
        });
  }
};

// ---- the launches between ------------------------------------------------------------------------------
// The tiles' maxima and sums of 16 tokens joined by 64 threads each, all their loads in flight at once for up to 512 tiles; loss,
// stats and what the gradient needs of them.  coef is written where the gradient follows.
template <bool GRAD>
__global__ void __launch_bounds__(1024) token_join_kernel(const float2* __restrict__ parts, int tiles, long long padded,
                                                          const float* __restrict__ zt, const TokenMeta* __restrict__ meta,
                                                          const int* __restrict__ list, TokenCoef* __restrict__ coef,
                                                          float* __restrict__ loss, float* __restrict__ stats) {
  __shared__ float sm[16][16];
  __shared__ double ss[16][16];
  const int t = threadIdx.x & 15, k = threadIdx.x >> 4, wv = threadIdx.x >> 6;
  const long long c = (long long)blockIdx.x * 16 + t;  // padded is a multiple of 32
  float m = -__FLT_MAX__;
  double s = 0.0;
  auto add = [&](float pm, double ps) {
    const float top = fmaxf(m, pm);
    s = s * (double)exp_neg(m - top) + ps * (double)exp_neg(pm - top);
    m = top;
  };
  const int r = list[c];  // on their way with the parts
  const TokenCoef k0 = coef[c];
  const float target = zt[c];
  const TokenMeta M = *meta;
  for (int i = k; i < tiles; i += 512) {
    float2 p[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) p[u] = i + 64 * u < tiles ? parts[(i + 64 * u) * padded + c] : make_float2(-__FLT_MAX__, 0.0f);
    float top = m;
#pragma unroll
    for (int u = 0; u < 8; ++u) top = fmaxf(top, p[u].x);
    s *= (double)exp_neg(m - top);
    m = top;
#pragma unroll
    for (int u = 0; u < 8; ++u) s += (double)p[u].y * (double)exp_neg(p[u].x - m);
  }
#pragma unroll
  for (int d = 16; d < 64; d <<= 1) add(__shfl_xor(m, d), __shfl_xor(s, d));
  if ((threadIdx.x & 63) < 16) {
    sm[wv][t] = m;
    ss[wv][t] = s;
  }
  __syncthreads();
  if (wv != 0) return;
  m = -__FLT_MAX__;
  s = 0.0;
#pragma unroll
  for (int i = 0; i < 4; ++i) add(sm[4 * k + i][t], ss[4 * k + i][t]);
#pragma unroll
  for (int d = 16; d < 64; d <<= 1) add(__shfl_xor(m, d), __shfl_xor(s, d));
  if (k != 0 || c >= M.count) return;
  loss[r] = (float)((double)k0.g * ((double)m - (double)target + log(s)));
  // the maxima pass over a NaN, the sum holds it
  stats[2ll * r] = s != s ? __builtin_nanf("") : s == 0.0 ? -__builtin_inff() : m;
  stats[2ll * r + 1] = (float)s;
  if (GRAD) {
    const float g = ldexpf(k0.g, M.scale);
    coef[c] = TokenCoef{m, g / (float)s, g, k0.target};  // as from the stats, to the bit
  }
}

// The same from given statistics.
static __global__ void __launch_bounds__(256) token_coef_kernel(const float* __restrict__ stats, const TokenMeta* __restrict__ meta,
                                                                const int* __restrict__ list, TokenCoef* __restrict__ coef) {
  const int c = blockIdx.x * 256 + threadIdx.x;
  if (c >= meta->count) return;
  const long long r = list[c];
  const TokenCoef k0 = coef[c];
  const float g = ldexpf(k0.g, meta->scale);
  coef[c] = TokenCoef{stats[2 * r], g / stats[2 * r + 1], g, k0.target};
}

// dX: the parts added and rounded, rows back in their places; rows that do not count are zeros.  The target's P is most of a
// row's, so what its rounding took comes back here: `lost` times its word.  (dW keeps it: its rows are the words'.)
template <typename T>
__global__ void __launch_bounds__(256) token_dx_kernel(const float* __restrict__ sum, int parts, long long stride, int nq,
                                                       const TokenMeta* __restrict__ meta, const int* __restrict__ place,
                                                       const TokenCoef* __restrict__ coef, const float* __restrict__ lost,
                                                       const T* __restrict__ W, long long ldw, T* __restrict__ dX, long long ldx,
                                                       int n) {
  const long long r = blockIdx.x;
  const int at = place[r], scale = -meta->scale;
  const float l = sizeof(T) < 4 && at >= 0 ? lost[at] : 0.0f;
  const T* w = W + (at >= 0 ? coef[at].target : 0) * ldw;
  for (int j = ((int)blockIdx.y * 256 + (int)threadIdx.x) * 4; j < nq; j += (int)gridDim.y * 1024) {
    fv4 s = {0, 0, 0, 0};
    if (at >= 0) {
      const float* q = sum + (long long)at * nq + j;
      int p = 0;
      for (; p + 8 <= parts; p += 8) {
        fv4 v[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) v[u] = *reinterpret_cast<const fv4*>(q + (p + u) * stride);
#pragma unroll
        for (int u = 0; u < 8; ++u) s += v[u];
      }
      for (; p < parts; ++p) s += *reinterpret_cast<const fv4*>(q + p * stride);
      if (sizeof(T) < 4) {
#pragma unroll
        for (int e = 0; e < 4; ++e) s[e] = fmaf(l, j + e < n ? (float)w[j + e] : 0.0f, s[e]);
      }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (j + e < n) dX[r * ldx + j + e] = (T)(__is_same(T, _Float16) ? ldexpf(s[e], scale) : s[e]);
  }
}

template <typename T>
__global__ void __launch_bounds__(256) zero_rows_kernel(T* __restrict__ p, long long ld, int rows, int n) {
  for (long long r = blockIdx.x; r < rows; r += gridDim.x)
    for (int j = (int)threadIdx.x; j < n; j += 256) p[r * ld + j] = (T)0.0f;
}

// ---- the plan ----------------------------------------------------------------------------------------------
static inline size_t token_al(size_t x) { return (x + 255) & ~(size_t)255; }

struct TokenPlan {
  int shape;          // of the tiles: words (or elements of a hidden row) by tokens, bm x bn
  int bm, bn;
  int nq;             // n up to a multiple of 16 bytes
  long long padded;   // rows up to a multiple of bn
  int piece;          // words of a piece
  int parts;          // of a piece's length in dX
  bool copy;          // W's rows are copied to aligned ones, a piece at a time
  size_t meta, list, place, coef, zt, lost, tiles, x, w, p, dx, bytes;  // offsets in the workspace, and its size
};

// Tile shapes, how many workgroups of each the card runs at a time with a product's rate, and their threads.
struct TokenShape {
  int bm, bn, slots, threads;
};
constexpr TokenShape kTokenShapes[] = {{64, 32, 512, 128}, {128, 32, 1024, 256}, {128, 64, 512, 256}, {128, 128, 512, 256}, {256, 256, 256, 512}};

// Parts of the length of dX's product, so that its few tiles fill the card; at least eight stages each.
static inline long long token_parts(const TokenShape& s, long long tiles, long long words, int es) {
  const long long parts = s.slots / tiles, longest = (words * es + 1023) / 1024;
  return parts > longest ? longest : parts < 1 ? 1 : parts;
}

// 16 bits: up to 128 tokens the narrowest tiles that hold them in one column (reading W is what counts there); more by
// rounds of 128 x 128 (512 at a time, 0.62 of a 256 x 256 round's time; a round of at most 256 of them 0.38) against
// 256 x 256.
// fp32, whose products are sixteen times slower, by the work of the busiest CU in the products with the words and, half as
// often, in dX's (rounds of tiles, 64 x 32 two a CU at a time, times what a CU has of each), of which 64 x 32 tiles do
// 15% more slowly.  Measured, us of the loss and its dX in tiles of 64 x 32, 128 x 64, 128 x 128, 256 x 256 (n 2560):
//   65 x 32768     518   491   504  1502        600 x 32768    2934  2474  2280  3309
//   128 x 32768    740   516   509  1499       1024 x 32768    4067  4384  3643  3647
//   300 x 32768   1842  1180  1471  1842       2048 x 32768    8180  7668  8570  7283
// Over 92 sizes (20 to 4096 rows of 64 to 4096, 1451 to 131072 words) the loss with dX is within 16% of the best shape's, 1% in
// the mean (64 x 32 throughout: 64%, 11%), without 256 x 256, which gained 5% at one size.
// A shape of which dX's product would not fit a launch is left out; 128 x 128 always does.
static inline int token_shape(int es, long long rows, int nq, int V) {
  auto tiles = [&](long long m, int s) {
    return (m + kTokenShapes[s].bm - 1) / kTokenShapes[s].bm * ((rows + kTokenShapes[s].bn - 1) / kTokenShapes[s].bn);
  };
  if (es == 2) {
    if (rows <= 32) return 1;
    if (rows <= 64) return 2;
    if (rows <= 128) return 3;
    const long long t3 = tiles(V, 3), rest = t3 % 512;
    const double c3 = 0.62 * (double)(t3 / 512) + (rest == 0 ? 0.0 : rest <= 256 ? 0.38 : 0.62), c4 = (double)((tiles(V, 4) + 255) / 256);
    return c3 < c4 ? 3 : 4;
  }
  int best = 3;
  double least = 1e300;
  for (int s : {3, 2, 0}) {
    const long long each = s == 0 ? 2 : 1, dx = tiles(nq, s), parts = token_parts(kTokenShapes[s], dx, V, es);
    auto rounds = [&](long long t) { return (double)((t + 256 * each - 1) / (256 * each) * each); };
    const double c = (s == 0 ? 1.15 : 1.0) * kTokenShapes[s].bm * kTokenShapes[s].bn *
                     (1.5 * rounds(tiles(V, s)) * nq + 0.5 * rounds(dx * parts) * V / (double)parts);
    if (c < least && ftile_fits(dx, kTokenShapes[s].threads)) {
      least = c;
      best = s;
    }
  }
  return best;
}

static inline TokenPlan token_plan(int es, long long rows, int n, int V, bool aligned, bool loss, bool dX, bool dW) {
  TokenPlan P{};
  const int q = 16 / es;
  P.nq = (n + q - 1) / q * q;
  P.shape = token_shape(es, rows, P.nq, V);
  P.bm = kTokenShapes[P.shape].bm;
  P.bn = kTokenShapes[P.shape].bn;
  P.padded = (rows + P.bn - 1) / P.bn * P.bn;
  P.copy = !aligned;
  const bool grad = dX || dW;
  const long long vr = (V + 255ll) / 256 * 256;
  // P of a piece, or its copied rows, at most 128 MiB (but 256 words at least: 1 GiB of P for 2^20 rows of fp32): they are
  // written and read again within the Infinity Cache's 256
  const long long row = (grad ? P.padded * es : 0) > (P.copy ? (long long)P.nq * es : 0) ? P.padded * es : (long long)P.nq * es;
  long long most = !grad && !P.copy ? vr : (128ll << 20) / row / 256 * 256;
  if (most < 256) most = 256;
  // and 2^21 tiles, which a launch holds: of words and tokens, and (dW) of words and elements of a hidden row
  const long long held = (1ll << 21) / (P.padded / P.bn) * P.bm / 256 * 256, wide = (1ll << 21) / ((P.nq + 127) / 128) * 128 / 256 * 256;
  if (most > held) most = held;
  if (most > wide) most = wide;
  if (most > 1 << 20) most = 1 << 20;
  P.piece = (int)(most < vr ? most : vr);
  P.parts = (int)token_parts(kTokenShapes[P.shape], (P.nq + P.bm - 1) / P.bm * (P.padded / P.bn), P.piece, es);
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t a = at;
    at += token_al(bytes);
    return a;
  };
  P.meta = take(sizeof(TokenMeta));
  P.list = take((size_t)P.padded * 4);
  P.place = take((size_t)rows * 4);
  P.coef = take((size_t)P.padded * sizeof(TokenCoef));
  P.zt = take(loss ? (size_t)P.padded * 4 : 0);
  P.lost = take(grad ? (size_t)P.padded * 4 : 0);
  P.tiles = take(loss ? (size_t)((V + P.bm - 1) / P.bm) * P.padded * 8 : 0);
  P.x = take((size_t)P.padded * P.nq * es);
  P.w = take(P.copy ? (size_t)P.piece * P.nq * es : 0);
  P.p = take(grad ? (size_t)P.padded * P.piece * es : 0);
  P.dx = take(dX ? (size_t)P.parts * P.padded * P.nq * 4 : 0);
  P.bytes = at;
  return P;
}

static inline bool token_aligned(const void* W, long long ldw, int n, int es) {
  return (reinterpret_cast<uintptr_t>(W) & 15) == 0 && ldw * es % 16 == 0 && (long long)n * es % 16 == 0 && ldw * es < (1ll << 24);
}

#define TOKEN_TRY(expr)               \
  do {                                \
    const hipError_t e_ = (expr);     \
    if (e_ != hipSuccess) return e_;  \
  } while (0)

// rows of D: words (first two products) or elements of a hidden row (dX); columns: tokens
template <typename T, bool AX, typename EPI>
static hipError_t token_product(const TokenPlan& P, FOperand A, long long M, FOperand B, long long N, long long K, int parts,
                                const TokenMeta* meta, const EPI& epi, hipStream_t st) {
  const int* c = &meta->count;
  switch (P.shape) {
    case 0:
      if constexpr (sizeof(T) == 4) return ftile_launch<T, 64, 32, 2, 1, 128, 2, AX, false, kRowsOfB>(A, M, B, N, K, parts, c, epi, st);
      else return hipErrorInvalidValue;
    case 1:
      if constexpr (sizeof(T) == 2) return ftile_launch<T, 128, 32, 4, 1, 128, 2, AX, false, kRowsOfB>(A, M, B, N, K, parts, c, epi, st);
      else return hipErrorInvalidValue;
    case 2: return ftile_launch<T, 128, 64, 2, 2, 128, 2, AX, false, kRowsOfB>(A, M, B, N, K, parts, c, epi, st);
    case 3: return ftile_launch<T, 128, 128, 2, 2, 128, 2, AX, false, kRowsOfB>(A, M, B, N, K, parts, c, epi, st);
    default:
      if constexpr (sizeof(T) == 2) return ftile_launch<T, 256, 256, 2, 4, 128, 2, AX, false, kRowsOfB>(A, M, B, N, K, parts, c, epi, st);
      else return hipErrorInvalidValue;
  }
}

// dW.  Measured, us of dW alone with its P, in tiles of 128 x 128 / 256 x 128 (n x words): bf16, 32 rows, 2560 x 32768 95 / 90, 512
// rows 207 / 187, 2048 rows 640 / 615, 776 x 10007 117 / 112; fp32, 65 rows, 776 x 10007 62 / 66, 512 rows 179 / 208, 2048 rows
// 633 / 757, 512 rows, 2560 x 32768 1241 / 1229.  So by the type alone, over 32 to 2048 rows.
template <typename T>
static hipError_t token_dw(FOperand A, long long M, FOperand B, long long N, long long K, const TokenMeta* meta,
                           const TokenDW<T>& epi, hipStream_t st) {
  const int* c = &meta->count;
  if constexpr (sizeof(T) == 4) return ftile_launch<T, 128, 128, 2, 2, 128, 2, true, true, kLength>(A, M, B, N, K, 1, c, epi, st);
  else return ftile_launch<T, 256, 128, 2, 2, 64, 3, true, true, kLength>(A, M, B, N, K, 1, c, epi, st);
}

// Blocks of a row beside `count` rows: a launch holds below 2^32 threads, the kernels go on from there.
static inline unsigned token_blocks(long long count, int wanted) {
  const long long most = (1ll << 23) / count;
  return (unsigned)(most < 1 ? 1 : wanted < most ? wanted : most);
}

template <typename T>
static hipError_t token_typed(const TokenLaunch& L, hipStream_t st) {
  constexpr int ES = (int)sizeof(T);
  if (L.rows == 0) {  // dW alone: zeros
    hipLaunchKernelGGL((zero_rows_kernel<T>), dim3((unsigned)(L.vocab < 1 << 20 ? L.vocab : 1 << 20)), dim3(256), 0, st,
                       static_cast<T*>(L.dW), L.lddw, L.vocab, L.n);
    return hipGetLastError();
  }
  const bool forward = L.loss != nullptr, grad = L.dX || L.dW;
  const TokenPlan P = token_plan(ES, L.rows, L.n, L.vocab, token_aligned(L.W, L.ldw, L.n, ES), forward, L.dX, L.dW);
  char* ws = static_cast<char*>(L.ws);
  TokenMeta* meta = reinterpret_cast<TokenMeta*>(ws + P.meta);
  int* list = reinterpret_cast<int*>(ws + P.list);
  int* place = reinterpret_cast<int*>(ws + P.place);
  TokenCoef* coef = reinterpret_cast<TokenCoef*>(ws + P.coef);
  float* zt = reinterpret_cast<float*>(ws + P.zt);
  float* lost = reinterpret_cast<float*>(ws + P.lost);
  float2* tiles = reinterpret_cast<float2*>(ws + P.tiles);
  T* x = reinterpret_cast<T*>(ws + P.x);
  T* wc = reinterpret_cast<T*>(ws + P.w);
  T* p = reinterpret_cast<T*>(ws + P.p);
  float* dx = reinterpret_cast<float*>(ws + P.dx);
  const T* W = static_cast<const T*>(L.W);
  const int rows = (int)L.rows, n = L.n, V = L.vocab, nq = P.nq;
  const bool scaled = grad && __is_same(T, _Float16);
  auto gather = [&](const T* src, long long ld, long long count, const int* l, T* dst) {
    hipLaunchKernelGGL((gather_kernel<T>), dim3((unsigned)count, token_blocks(count, (nq * ES / 16 + 255) / 256)), dim3(256), 0, st, src,
                       ld, n, l, dst, nq);
  };
  auto start = [&](auto* target) {
    using TI = std::remove_pointer_t<decltype(target)>;
    float* stats = forward ? L.stats : nullptr;
    if (rows <= 1024) {
      hipLaunchKernelGGL((token_start_kernel<T, std::remove_const_t<TI>>), dim3((unsigned)P.padded), dim3(256), 0, st, target, L.weight,
                         rows, (int)P.padded, V, scaled, meta, list, place, coef, L.loss, stats, static_cast<const T*>(L.X), L.ldx, n, x,
                         nq);
    } else {
      hipLaunchKernelGGL((token_rows_kernel<std::remove_const_t<TI>>), dim3(1), dim3(kTokenScan), 0, st, target, L.weight, rows,
                         (int)P.padded, V, scaled, meta, list, place, coef, L.loss, stats);
      gather(static_cast<const T*>(L.X), L.ldx, P.padded, list, x);
    }
  };
  if (L.target_bytes == 8) start(static_cast<const long long*>(L.target));
  else start(static_cast<const int*>(L.target));
  const FOperand X{x, nq};
  // words first .. first + c - 1, aligned
  int copied = -1;  // the piece whose copy is there
  auto words = [&](int first, int c) {
    const T* w = W + first * L.ldw;
    if (!P.copy) return FOperand{w, L.ldw};
    if (copied != first) gather(w, L.ldw, c, nullptr, wc);
    copied = first;
    return FOperand{wc, nq};
  };
  if (forward) {
    for (int v = 0; v < V; v += P.piece) {
      const int c = V - v < P.piece ? V - v : P.piece;
      TOKEN_TRY((token_product<T, false>(P, words(v, c), c, X, P.padded, nq, 1, meta,
                                         TokenStats{coef, tiles + (long long)(v / P.bm) * P.padded, zt, P.padded, v}, st)));
    }
    const dim3 g((unsigned)((P.padded + 15) / 16));
    const int nt = (V + P.bm - 1) / P.bm;
    if (grad)
      hipLaunchKernelGGL((token_join_kernel<true>), g, dim3(1024), 0, st, tiles, nt, P.padded, zt, meta, list, coef, L.loss, L.stats);
    else
      hipLaunchKernelGGL((token_join_kernel<false>), g, dim3(1024), 0, st, tiles, nt, P.padded, zt, meta, list, coef, L.loss, L.stats);
  } else {
    hipLaunchKernelGGL(token_coef_kernel, dim3((unsigned)((P.padded + 255) / 256)), dim3(256), 0, st, L.stats, meta, list, coef);
  }
  if (grad) {
    const long long stride = P.padded * nq;
    for (int v = 0; v < V; v += P.piece) {
      const int c = V - v < P.piece ? V - v : P.piece;
      const FOperand w = words(v, c), pp{p, P.piece};
      TOKEN_TRY((token_product<T, false>(P, w, c, X, P.padded, nq, 1, meta, TokenP<T>{coef, p, lost, P.piece, v}, st)));
      if (L.dX)
        TOKEN_TRY((token_product<T, true>(P, w, nq, pp, P.padded, c, P.parts, meta, TokenDX{dx, stride, nq, v == 0}, st)));
      if (L.dW)
        TOKEN_TRY((token_dw<T>(X, nq, pp, c, P.padded, meta, TokenDW<T>{meta, static_cast<T*>(L.dW) + v * L.lddw, L.lddw, n}, st)));
    }
    if (L.dX) {
      hipLaunchKernelGGL((token_dx_kernel<T>), dim3((unsigned)rows, token_blocks(rows, (nq + 1023) / 1024)), dim3(256), 0, st, dx, P.parts, stride, nq,
                         meta, place, coef, lost, W, L.ldw, static_cast<T*>(L.dX), L.lddx, n);
    }
  }
  return hipGetLastError();
}

}  // namespace externd
