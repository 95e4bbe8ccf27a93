// Products of 8-bit integer rows on the matrix cores: D[r][c] = sum_k A[r][k] B[c][k] in int32, handed
// to an epilogue.
#pragma once
#include "types.hpp"

namespace externd {

// ---- operand loads ----------------------------------------------------------------------------
// 16 bytes of a row of n >= 16 at k, zeros from the row's end on.  A piece that crosses the end is
// read from 16 bytes before it and shifted down, so that every load is inside the row and
// unconditional.
__device__ __forceinline__ iv4 row16(const int8_t* __restrict__ row, int k, int n) {
  const int at = k < n - 16 ? k : n - 16, drop = k - at;  // bytes to shift out; 16 or more: none left
  const iv4 v = *reinterpret_cast<const iv4_any*>(row + at);
  unsigned __int128 x = __builtin_bit_cast(unsigned __int128, v);
  x = drop < 16 ? x >> (8 * (drop & 15)) : (unsigned __int128)0;
  return __builtin_bit_cast(iv4, x);
}
// the same for a row of n < 16
__device__ __forceinline__ iv4 row16_short(const int8_t* __restrict__ row, int k, int n) {
  iv4 v = {0, 0, 0, 0};
#pragma unroll
  for (int e = 0; e < 15; ++e)
    if (k + e < n) v[e >> 2] |= (int)((unsigned)(unsigned char)row[k + e] << (8 * (e & 3)));
  return v;
}

// ---- tiles --------------------------------------------------------------------------------------
// Workgroup: a BM x BN tile of D, WR x WC waves, each with FM x FN accumulators of
// v_mfma_i32_32x32x32_i8 (A row and B column l % 32 of lane l, both with the 16 bytes at 16 (l / 32)
// of the step; accumulator element i of lane l is row 8 (i / 4) + 4 (l / 32) + i % 4, column l % 32).
//
// The tile's rows pass through LDS in stages of 128 bytes, two stages in turn.  In LDS, row r is 128
// bytes and its 16-byte piece c sits at c ^ (r / 2 % 8): 16 consecutive rows' pieces of one column lie
// in different banks (measured: no bank conflicts), and a wave's 1024 bytes of eight rows are
// contiguous, as the direct load to LDS wants them.
//   DMA: rows go to LDS directly (16 bytes a lane); K, the rows' distances and bases are multiples of
//        16 and the distances below 2^24, so that a row's offset in a tile fits 32 bits
//   else: through registers, loaded one stage earlier, at any alignment (K >= 16)
// The fragments of the next 32 bytes are read from LDS while the products of these run, two reads
// between four products (the scheduling groups), and the barrier that hands the stage over comes
// before the last of a stage's four steps, whose products cover the reads behind it.
// Measured (256 x 256, 8 waves, 8192^3): 2.36 10^15 operations a second, the matrix cores busy 62% of
// the time at 1.8 GHz (the card's clock falls under this load; 2.4 GHz in calls of some 100 us).  A
// tile bound by LDS reads would gain from larger tiles per wave, but four waves of 128 x 128 were
// slower (2.30) for want of a second wave to cover the barrier.
//
// Workgroups go round the eight XCDs: each XCD gets a run of neighbouring tiles, in groups of kGroup
// tile rows, so that the tiles it holds at one time share rows in its L2 (8192 x 7680 x 2560 in
// 128 x 128 tiles: 202 us, 265 us with all tile rows in one group).
constexpr int kGroup = 4;
static __device__ const int kZeros[4] = {0, 0, 0, 0};  // what a direct load reads behind a row's end

template <int BM, int BN, int WR, int WC, bool DMA, typename EPI>
__global__ void __launch_bounds__(64 * WR * WC, 1) tile_kernel(const int8_t* __restrict__ A, long long lda, int M,
                                                               const int8_t* __restrict__ B, long long ldb, int N,
                                                               int K, int ntm, int ntn, EPI epi) {
  typedef const __attribute__((address_space(1))) void gptr;
  typedef __attribute__((address_space(3))) void lptr;
  constexpr int NW = WR * WC, PA = BM / 8 / NW, PB = BN / 8 / NW;
  constexpr int FM = BM / WR / 32, FN = BN / WC / 32;
  static_assert(PA * 8 * NW == BM && PB * 8 * NW == BN && FM * 32 * WR == BM && FN * 32 * WC == BN, "tile shape");
  __shared__ __attribute__((aligned(1024))) int8_t l0[(BM + BN) * 128];
  __shared__ __attribute__((aligned(1024))) int8_t l1[(BM + BN) * 128];
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wr = wv / WC, wc = wv % WC;
  const int total = ntm * ntn, per = (total + 7) / 8, rem = total % 8;
  const int xcd = blockIdx.x % 8, at = blockIdx.x / 8;
  const int tile = rem == 0 || xcd < rem ? xcd * per + at : rem * per + (xcd - rem) * (per - 1) + at;
  const int grp = tile / (kGroup * ntn), g0 = grp * kGroup, gs = ntm - g0 < kGroup ? ntm - g0 : kGroup;
  const int in = tile - g0 * ntn;
  const long long m0 = (long long)(g0 + in % gs) * BM, n0 = (long long)(in / gs) * BN;
  const int8_t* ab = A + m0 * lda;
  const int8_t* bb = B + n0 * ldb;
  // this lane's piece of each of the wave's loads: row (p NW + wv) 8 + lane / 8, rows behind the last
  // repeat it
  const int lrow = lane >> 3;
  unsigned ao[PA], bo[PB];
  const int8_t* ap[PA];
  const int8_t* bp[PB];
  int ca[PA], cb[PB];  // piece's first byte within the stage
#pragma unroll
  for (int p = 0; p < PA; ++p) {
    const int r = (p * NW + wv) * 8 + lrow;
    const long long row = m0 + r < M ? r : M - 1 - m0;
    ca[p] = ((lane & 7) ^ ((r >> 1) & 7)) * 16;
    if (DMA) ao[p] = (unsigned)row * (unsigned)lda + ca[p];
    else ap[p] = ab + row * lda;
  }
#pragma unroll
  for (int p = 0; p < PB; ++p) {
    const int r = (p * NW + wv) * 8 + lrow;
    const long long row = n0 + r < N ? r : N - 1 - n0;
    cb[p] = ((lane & 7) ^ ((r >> 1) & 7)) * 16;
    if (DMA) bo[p] = (unsigned)row * (unsigned)ldb + cb[p];
    else bp[p] = bb + row * ldb;
  }
  const int nk = (K + 127) / 128;
  iv4 sa[PA], sb[PB];
  auto load = [&](int t) {  // a stage into registers
    const int k0 = 128 * t;
    if (k0 + 128 <= K) {
#pragma unroll
      for (int p = 0; p < PA; ++p) sa[p] = *reinterpret_cast<const iv4_any*>(ap[p] + k0 + ca[p]);
#pragma unroll
      for (int p = 0; p < PB; ++p) sb[p] = *reinterpret_cast<const iv4_any*>(bp[p] + k0 + cb[p]);
    } else {
#pragma unroll
      for (int p = 0; p < PA; ++p) sa[p] = row16(ap[p], k0 + ca[p], K);
#pragma unroll
      for (int p = 0; p < PB; ++p) sb[p] = row16(bp[p], k0 + cb[p], K);
    }
  };
  // stage t into l; every direct load issued is waited for by a barrier before the kernel's end
  auto fetch = [&](int8_t* l, int t) {
    if (DMA) {
      const int k0 = 128 * t;
      if (k0 + 128 <= K) {
#pragma unroll
        for (int p = 0; p < PA; ++p)
          __builtin_amdgcn_global_load_lds((gptr*)(ab + k0 + ao[p]), (lptr*)(l + (p * NW + wv) * 1024), 16, 0, 0);
#pragma unroll
        for (int p = 0; p < PB; ++p)
          __builtin_amdgcn_global_load_lds((gptr*)(bb + k0 + bo[p]), (lptr*)(l + BM * 128 + (p * NW + wv) * 1024), 16,
                                           0, 0);
      } else {
        // pieces behind the rows' end: zeros for A, so that B's may be anything (its row's first piece)
#pragma unroll
        for (int p = 0; p < PA; ++p) {
          const int8_t* s = k0 + ca[p] < K ? ab + k0 + ao[p] : reinterpret_cast<const int8_t*>(kZeros);
          __builtin_amdgcn_global_load_lds((gptr*)s, (lptr*)(l + (p * NW + wv) * 1024), 16, 0, 0);
        }
#pragma unroll
        for (int p = 0; p < PB; ++p) {
          const int8_t* s = k0 + cb[p] < K ? bb + k0 + bo[p] : bb + (bo[p] - cb[p]);
          __builtin_amdgcn_global_load_lds((gptr*)s, (lptr*)(l + BM * 128 + (p * NW + wv) * 1024), 16, 0, 0);
        }
      }
    } else {
#pragma unroll
      for (int p = 0; p < PA; ++p) *reinterpret_cast<iv4*>(l + (p * NW + wv) * 1024 + lane * 16) = sa[p];
#pragma unroll
      for (int p = 0; p < PB; ++p) *reinterpret_cast<iv4*>(l + BM * 128 + (p * NW + wv) * 1024 + lane * 16) = sb[p];
      if (t + 1 < nk) load(t + 1);
    }
  };
  iv16 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0;
  const int lr = lane & 31, lg = lane >> 5;
  const int ra = wr * (BM / WR) + lr, rb = wc * (BN / WC) + lr;  // rows r + 32 f share r / 2 % 8
  const int za = (ra >> 1) & 7, zb = (rb >> 1) & 7;
  iv4 fa[2][FM], fb[2][FN];
  auto read = [&](int f, const int8_t* l, int ks) {  // fragments of step ks of the stage in l
#pragma unroll
    for (int i = 0; i < FM; ++i)
      fa[f][i] = *reinterpret_cast<const iv4*>(l + (ra + 32 * i) * 128 + (((2 * ks + lg) ^ za) << 4));
#pragma unroll
    for (int j = 0; j < FN; ++j)
      fb[f][j] = *reinterpret_cast<const iv4*>(l + BM * 128 + (rb + 32 * j) * 128 + (((2 * ks + lg) ^ zb) << 4));
  };
  auto mul = [&](int f) {
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fa[f][i], fb[f][j], acc[i][j], 0, 0, 0);
  };
  auto step = [&](int f, const int8_t* l, int ks) {  // products of fragments f under the reads of the next
    read(f ^ 1, l, ks);
    mul(f);
    constexpr int reads = FM + FN, each = FM * FN / reads > 0 ? FM * FN / reads : 1;
#pragma unroll
    for (int i = 0; i < reads; ++i) {
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x008, each, 0);
    }
    if (FM * FN > each * reads) __builtin_amdgcn_sched_group_barrier(0x008, FM * FN - each * reads, 0);
    __builtin_amdgcn_sched_barrier(0);
  };
  if (!DMA) load(0);
  fetch(l0, 0);
  __syncthreads();
  if (nk > 1) fetch(l1, 1);
  read(0, l0, 0);
  __builtin_amdgcn_sched_barrier(0);
  int t = 0;
  for (; t + 2 < nk; t += 2) {  // stage t in l0, its first fragments read; stage t + 1 on its way to l1
    step(0, l0, 1);
    step(1, l0, 2);
    step(0, l0, 3);
    __syncthreads();
    fetch(l0, t + 2);
    __builtin_amdgcn_sched_barrier(0);
    step(1, l1, 0);
    step(0, l1, 1);
    step(1, l1, 2);
    step(0, l1, 3);
    __syncthreads();
    if (t + 3 < nk) fetch(l1, t + 3);
    __builtin_amdgcn_sched_barrier(0);
    step(1, l0, 0);
  }
  step(0, l0, 1);
  step(1, l0, 2);
  step(0, l0, 3);
  if (t + 1 < nk) {
    __syncthreads();
    step(1, l1, 0);
    step(0, l1, 1);
    step(1, l1, 2);
    step(0, l1, 3);
  }
  mul(1);
  // the epilogue's own operands first, all in flight together (clamped indexes, no branches), then
  // the stores; a tile inside the matrix needs no guards
  typename EPI::Row er[FM];
  typename EPI::Col ec[FN];
  const long long r0 = m0 + wr * (BM / WR) + 4 * lg, c0 = n0 + wc * (BN / WC) + lr;
#pragma unroll
  for (int i = 0; i < FM; ++i) er[i] = epi.row(r0 + 32 * i, M);
#pragma unroll
  for (int j = 0; j < FN; ++j) ec[j] = epi.col(c0 + 32 * j < N ? c0 + 32 * j : N - 1);
  if (m0 + BM <= M && n0 + BN <= N) {
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j) epi.template put<true>(r0 + 32 * i, c0 + 32 * j, M, N, er[i], ec[j], acc[i][j]);
  } else {
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j) epi.template put<false>(r0 + 32 * i, c0 + 32 * j, M, N, er[i], ec[j], acc[i][j]);
  }
}

// Whether rows can go to LDS directly.
static inline bool tile_dma(const void* p, long long ld, int K) {
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && ld % 16 == 0 && K % 16 == 0 && ld < (1ll << 24);
}

template <int BM, int BN, int WR, int WC, typename EPI>
static hipError_t tile_launch(const int8_t* A, long long lda, int M, const int8_t* B, long long ldb, int N, int K,
                              const EPI& epi, hipStream_t st) {
  const long long ntm = (M + BM - 1ll) / BM, ntn = (N + BN - 1ll) / BN;
  if (ntm * ntn > 2147483647ll) return hipErrorInvalidValue;
  if (tile_dma(A, lda, K) && tile_dma(B, ldb, K))
    hipLaunchKernelGGL((tile_kernel<BM, BN, WR, WC, true, EPI>), dim3((unsigned)(ntm * ntn)), dim3(64 * WR * WC), 0, st,
                       A, lda, M, B, ldb, N, K, (int)ntm, (int)ntn, epi);
  else
    hipLaunchKernelGGL((tile_kernel<BM, BN, WR, WC, false, EPI>), dim3((unsigned)(ntm * ntn)), dim3(64 * WR * WC), 0, st,
                       A, lda, M, B, ldb, N, K, (int)ntm, (int)ntn, epi);
  return hipGetLastError();
}

// The tile shape by what its rounds over 256 CUs would cost: a tile's time at K = 2560 is about 36 us
// (256 x 256), 29.5 us (256 x 192) and, for 128 x 128, 15 us alone on its CU and 25 us for two (its two
// stages take 64 KB of LDS, so two workgroups share a CU).
template <typename EPI>
static hipError_t tile_product(const int8_t* A, long long lda, int M, const int8_t* B, long long ldb, int N, int K,
                               const EPI& epi, hipStream_t st) {
  auto tiles = [&](int bm, int bn) { return ((M + bm - 1ll) / bm) * ((N + bn - 1ll) / bn); };
  const long long t1 = tiles(256, 256), t2 = tiles(256, 192), t3 = tiles(128, 128);
  const double c1 = 36.0 * ((t1 + 255) / 256), c2 = 29.5 * ((t2 + 255) / 256);
  const double c3 = t3 <= 256 ? 15.0 : 25.0 * ((t3 + 511) / 512);
  if (c3 <= c1 && c3 <= c2) return tile_launch<128, 128, 2, 2>(A, lda, M, B, ldb, N, K, epi, st);
  if (c2 <= c1) return tile_launch<256, 192, 4, 2>(A, lda, M, B, ldb, N, K, epi, st);
  return tile_launch<256, 256, 2, 4>(A, lda, M, B, ldb, N, K, epi, st);
}

}  // namespace externd
