// Products of 8-bit integer rows on the matrix cores: D[r][c] = sum_k A[r][k] B[c][k] in int32, handed
// to an epilogue.
#pragma once
#include "types.hpp"

namespace externd {

// ---- operand loads ----------------------------------------------------------------------------
// 16 bytes of a row at k, zeros from the row's end on
__device__ __forceinline__ iv4 row16(const int8_t* __restrict__ row, int k, int n) {
  if (k + 16 <= n) return *reinterpret_cast<const iv4_any*>(row + k);
  iv4 v = {0, 0, 0, 0};
#pragma unroll
  for (int e = 0; e < 16; ++e)
    if (k + e < n) v[e >> 2] |= (int)((unsigned)(unsigned char)row[k + e] << (8 * (e & 3)));
  return v;
}

// ---- tiles --------------------------------------------------------------------------------------
// Workgroup: a BM x BN tile of D = A B^T (A: M rows, B: N rows of K bytes), WR x WC waves, each with FM x FN accumulators
// of v_mfma_i32_32x32x32_i8 (A row and B column l % 32 of lane l, both with the 16 bytes
// at 16 (l / 32) of the step; accumulator element i of lane l is row 8 (i / 4) + 4 (l / 32) + i % 4,
// column l % 32).  The tiles' rows pass through LDS 128 bytes at a time, double buffered: the loads
// of the next 128 bytes go out before the products of these, and are stored to the other buffer
// after them.  The 16-byte piece c of row r sits at c ^ (r / 2 % 8), so that 16 consecutive rows'
// pieces of one column lie in different banks.
template <int BM, int BN, int WR, int WC, typename EPI>
__global__ void __launch_bounds__(64 * WR * WC) tile_kernel(const int8_t* __restrict__ A, long long lda, int M,
                                                            const int8_t* __restrict__ B, long long ldb, int N, int K,
                                                            int ntm, int ntn, EPI epi) {
  constexpr int NTHR = 64 * WR * WC, PA = BM * 8 / NTHR, PB = BN * 8 / NTHR;
  constexpr int FM = BM / WR / 32, FN = BN / WC / 32;
  __shared__ __attribute__((aligned(16))) int8_t la[2][BM * 128];
  __shared__ __attribute__((aligned(16))) int8_t lb[2][BN * 128];
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
  const int wr = wv / WC, wc = wv % WC;
  // workgroups go round the eight XCDs: each XCD gets a run of neighbouring tiles, so that its L2
  // holds the rows that they share
  const int total = ntm * ntn, per = (total + 7) / 8, rem = total % 8;
  const int xcd = blockIdx.x % 8, at = blockIdx.x / 8;
  const int tile = rem == 0 || xcd < rem ? xcd * per + at : rem * per + (xcd - rem) * (per - 1) + at;
  const int tm = tile % ntm, tn = tile / ntm;
  const long long m0 = (long long)tm * BM, n0 = (long long)tn * BN;
  const int8_t* ap[PA];
  const int8_t* bp[PB];
  int ao[PA], bo[PB];
#pragma unroll
  for (int p = 0; p < PA; ++p) {
    const int x = tid + NTHR * p, r = x >> 3, c = x & 7;
    const long long row = m0 + r < M ? m0 + r : M - 1;
    ap[p] = A + row * lda;
    ao[p] = r * 128 + ((c ^ ((r >> 1) & 7)) << 4);
  }
#pragma unroll
  for (int p = 0; p < PB; ++p) {
    const int x = tid + NTHR * p, r = x >> 3, c = x & 7;
    const long long row = n0 + r < N ? n0 + r : N - 1;
    bp[p] = B + row * ldb;
    bo[p] = r * 128 + ((c ^ ((r >> 1) & 7)) << 4);
  }
  const int kc = (tid & 7) * 16;  // this thread's piece within each 128 bytes
  iv4 sa[PA], sb[PB];
  auto fetch = [&](int k0) {
    if (k0 + 128 <= K) {
#pragma unroll
      for (int p = 0; p < PA; ++p) sa[p] = *reinterpret_cast<const iv4_any*>(ap[p] + k0 + kc);
#pragma unroll
      for (int p = 0; p < PB; ++p) sb[p] = *reinterpret_cast<const iv4_any*>(bp[p] + k0 + kc);
    } else {
#pragma unroll
      for (int p = 0; p < PA; ++p) sa[p] = row16(ap[p], k0 + kc, K);
#pragma unroll
      for (int p = 0; p < PB; ++p) sb[p] = row16(bp[p], k0 + kc, K);
    }
  };
  auto put = [&](int buf) {
#pragma unroll
    for (int p = 0; p < PA; ++p) *reinterpret_cast<iv4*>(la[buf] + ao[p]) = sa[p];
#pragma unroll
    for (int p = 0; p < PB; ++p) *reinterpret_cast<iv4*>(lb[buf] + bo[p]) = sb[p];
  };
  iv16 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0;
  const int nk = (K + 127) / 128;
  const int lr = lane & 31, lg = lane >> 5;
  const int ra = wr * (BM / WR) + lr, rb = wc * (BN / WC) + lr;  // rows r + 32 f share r / 2 % 8
  const int za = (ra >> 1) & 7, zb = (rb >> 1) & 7;
  fetch(0);
  put(0);
  __syncthreads();
  for (int t = 0; t < nk; ++t) {
    const int buf = t & 1;
    if (t + 1 < nk) fetch(128 * (t + 1));
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
      iv4 fa[FM], fb[FN];
#pragma unroll
      for (int i = 0; i < FM; ++i)
        fa[i] = *reinterpret_cast<const iv4*>(la[buf] + (ra + 32 * i) * 128 + (((2 * ks + lg) ^ za) << 4));
#pragma unroll
      for (int j = 0; j < FN; ++j)
        fb[j] = *reinterpret_cast<const iv4*>(lb[buf] + (rb + 32 * j) * 128 + (((2 * ks + lg) ^ zb) << 4));
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fa[i], fb[j], acc[i][j], 0, 0, 0);
    }
    if (t + 1 < nk) put(buf ^ 1);
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j)
      epi(m0 + wr * (BM / WR) + 32 * i + 4 * lg, n0 + wc * (BN / WC) + 32 * j + lr, M, N, acc[i][j]);
}

}  // namespace externd
