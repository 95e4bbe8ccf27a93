// Products of 8-bit integer rows on the matrix cores: D[r][c] = sum_k A[r][k] B[c][k] in int32, handed
// to an epilogue.
#pragma once
#include "types.hpp"

namespace externd {

// ---- operand loads ----------------------------------------------------------------------------
// 16 bytes of a row of n >= 16 at k, zeros from the row's end on.  A piece that crosses the end is
// read from 16 bytes before it and shifted down, so that every load is inside the row and
// unconditional; row_end shifts what row_load read.
__device__ __forceinline__ iv4 row_load(const int8_t* __restrict__ row, int k, int n) {
  return *reinterpret_cast<const iv4_any*>(row + (k < n - 16 ? k : n - 16));
}
__device__ __forceinline__ iv4 row_end(iv4 v, int k, int n) {
  asm volatile("" : "+v"(v));  // else the load moves into a branch of its own, with its own wait
  const int drop = k < n - 16 ? 0 : k - (n - 16);  // bytes to shift out; 16 or more: none left
  unsigned __int128 x = __builtin_bit_cast(unsigned __int128, v);
  x = drop < 16 ? x >> (8 * (drop & 15)) : (unsigned __int128)0;
  return __builtin_bit_cast(iv4, x);
}
// the same for a row of n < 16
__device__ __forceinline__ iv4 row_short(const int8_t* __restrict__ row, int k, int n) {
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
// The fragments of the next 32 bytes are read from LDS while the products of these run, one read
// before each of the first products (the scheduling groups), and the barrier that hands the stage over
// comes before the last of a stage's four steps, whose products cover the reads behind it.
// Measured (256 x 256, 8 waves, 8192^3): 2.0 to 2.4 10^15 operations a second by the card's clock, which
// falls to 1.8 GHz under this load; the matrix cores are busy 62% of the time.  Four waves of 128 x 128
// each read less from LDS but were slower (2.2 to 2.3) for want of a second wave to cover the barrier;
// more stages in smaller tiles, and a raised wave priority around the products, lost 2 to 5%.
//
// Workgroups go round the eight XCDs: each XCD gets a run of neighbouring tiles, in groups of kGroup
// tile rows, so that the tiles it holds at one time share rows in its L2 (8192 x 7680 x 2560 in
// 128 x 128 tiles: 202 us, 265 us with all tile rows in one group).
constexpr int kGroup = 4;
static __device__ const int kZeros[4] = {0, 0, 0, 0};  // what a direct load reads behind a row's end

template <int BM, int BN, int WR, int WC, bool DMA, typename EPI>
__global__ void __launch_bounds__(64 * WR * WC, 1) tile_kernel(const int8_t* __restrict__ A, long long lda, int M,
                                                               const int8_t* __restrict__ B, long long ldb, int N,
                                                               int Kall, int kper, int ntm, int ntn, EPI epi) {
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
  const int kbeg = blockIdx.y * kper, K = Kall - kbeg < kper ? Kall - kbeg : kper;
  const int8_t* ab = A + m0 * lda + kbeg;
  const int8_t* bb = B + n0 * ldb + kbeg;
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
  // Stage 0 is the rows' last 128 bytes or what is left of them, stage t > 0 bytes 128 (t - 1) on: what
  // a row's end needs is in one place before the loop.
  const int nk = (K + 127) / 128, kl = 128 * (nk - 1);
  iv4 sa[PA], sb[PB];
  auto load = [&](int t) {  // stage t > 0 into registers
    const int k0 = 128 * (t - 1);
#pragma unroll
    for (int p = 0; p < PA; ++p) sa[p] = *reinterpret_cast<const iv4_any*>(ap[p] + k0 + ca[p]);
#pragma unroll
    for (int p = 0; p < PB; ++p) sb[p] = *reinterpret_cast<const iv4_any*>(bp[p] + k0 + cb[p]);
  };
  auto put = [&](int8_t* l, const iv4 (&va)[PA], const iv4 (&vb)[PB]) {  // registers to LDS
#pragma unroll
    for (int p = 0; p < PA; ++p) *reinterpret_cast<iv4*>(l + (p * NW + wv) * 1024 + lane * 16) = va[p];
#pragma unroll
    for (int p = 0; p < PB; ++p) *reinterpret_cast<iv4*>(l + BM * 128 + (p * NW + wv) * 1024 + lane * 16) = vb[p];
  };
  auto direct = [&](int8_t* l, int p, const int8_t* s) {
    __builtin_amdgcn_global_load_lds((gptr*)s, (lptr*)(l + (p * NW + wv) * 1024), 16, 0, 0);
  };
  // a third of stage t > 0 into l: three of the four steps between two barriers issue one each, so that
  // the loads do not come in one burst (1 to 3% over issuing them together).  Through registers, the
  // first does all (and loads stage t + 1).  Every direct load issued is waited for by a barrier
  // before the kernel's end.
  auto fetch = [&](int8_t* l, int t, int third) {
    if (DMA) {
      const int k0 = 128 * (t - 1);
      constexpr int all = PA + PB, each = (all + 2) / 3;
#pragma unroll
      for (int p = 0; p < all; ++p)
        if (p / each == third) {
          if (p < PA) direct(l, p, ab + k0 + ao[p < PA ? p : 0]);
          else direct(l + BM * 128, p - PA, bb + k0 + bo[p < PA ? 0 : p - PA]);
        }
    } else if (third == 0) {
      put(l, sa, sb);
      if (t + 1 < nk) load(t + 1);
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  if (DMA) {
    // pieces behind the rows' end: zeros for A, so that B's may be anything (its row's first piece)
#pragma unroll
    for (int p = 0; p < PA; ++p)
      direct(l0, p, kl + ca[p] < K ? ab + kl + ao[p] : reinterpret_cast<const int8_t*>(kZeros));
#pragma unroll
    for (int p = 0; p < PB; ++p) direct(l0 + BM * 128, p, bb + (kl + cb[p] < K ? kl + bo[p] : bo[p] - cb[p]));
  } else {
    iv4 ta[PA], tb[PB];  // stages 0 and 1 on their way together
#pragma unroll
    for (int p = 0; p < PA; ++p) ta[p] = row_load(ap[p], kl + ca[p], K);
#pragma unroll
    for (int p = 0; p < PB; ++p) tb[p] = row_load(bp[p], kl + cb[p], K);
    if (nk > 1) load(1);
    if (kl + 128 > K) {
#pragma unroll
      for (int p = 0; p < PA; ++p) ta[p] = row_end(ta[p], kl + ca[p], K);
#pragma unroll
      for (int p = 0; p < PB; ++p) tb[p] = row_end(tb[p], kl + cb[p], K);
    }
    put(l0, ta, tb);
  }
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
  __syncthreads();
  if (nk > 1) {
    fetch(l1, 1, 0);
    fetch(l1, 1, 1);
    fetch(l1, 1, 2);
  }
  read(0, l0, 0);
  __builtin_amdgcn_sched_barrier(0);
  int t = 0;
  for (; t + 2 < nk; t += 2) {  // stage t in l0, its first fragments read; stage t + 1 on its way to l1
    step(0, l0, 1);
    step(1, l0, 2);
    step(0, l0, 3);
    __syncthreads();
    fetch(l0, t + 2, 0);
    step(1, l1, 0);
    fetch(l0, t + 2, 1);
    step(0, l1, 1);
    fetch(l0, t + 2, 2);
    step(1, l1, 2);
    step(0, l1, 3);
    __syncthreads();
    const bool more = t + 3 < nk;
    if (more) fetch(l1, t + 3, 0);
    step(1, l0, 0);
    if (more) {
      fetch(l1, t + 3, 1);
      fetch(l1, t + 3, 2);
    }
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
  // the wave's share of D: rows wr BM / WR on, columns wc BN / WC on of the tile; mr x nr of the tile
  // lie in the matrix
  epi.at(m0, n0);
  const int mr = M - m0 < BM ? (int)(M - m0) : BM, nr = N - n0 < BN ? (int)(N - n0) : BN;
  if (EPI::kLds) __syncthreads();  // the stages are read: LDS is free
  constexpr int kBytes = EPI::kLds ? 32 * (32 * FN + 8) * 4 : 0;  // of one wave
  static_assert(kBytes * ((NW + 1) / 2) <= (BM + BN) * 128, "epilogue in LDS");
  epi.template finish<FM, FN>(acc, wr * (BM / WR), wc * (BN / WC), mr, nr,
                              reinterpret_cast<float*>((wv & 1 ? l1 : l0) + (wv >> 1) * kBytes));
}

// An epilogue that stores from the accumulators: put() gets the first row and the column of 16 values.
template <int FM, int FN, typename EPI>
__device__ __forceinline__ void finish_direct(const EPI& epi, const iv16 (&acc)[FM][FN], int r0, int c0, int mr, int nr) {
  const int lane = threadIdx.x & 63, r = r0 + 4 * (lane >> 5), c = c0 + (lane & 31);
#pragma unroll
  for (int i = 0; i < FM; ++i)
    if (r0 + 32 * i < mr) {  // the same for the wave
      const typename EPI::Row er = epi.row(r + 32 * i, mr);
#pragma unroll
      for (int j = 0; j < FN; ++j)
        if (c + 32 * j < nr) epi.put(r + 32 * i, c + 32 * j, mr, er, acc[i][j]);
    }
}

// ---- split row lengths --------------------------------------------------------------------------
// Where there are few tiles, the row length is split over blockIdx.y: each part writes its int32 tile,
// and a second launch adds the parts (exact, in any order) and applies the epilogue.
struct PartTile {
  int* part;  // [parts][rows of 4][N][4]: the four consecutive rows of an accumulator lie together
  long long N, stride;
  int* p;
  static constexpr bool kLds = false, kAligned = false;
  struct Row {};
  __device__ __forceinline__ void at(long long m0, long long n0) {
    p = part + blockIdx.y * stride + ((m0 >> 2) * N + n0) * 4;
  }
  __device__ __forceinline__ Row row(int, int) const { return {}; }
  __device__ __forceinline__ void put(int r, int c, int mr, Row, const iv16& acc) const {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (r + 8 * i < mr) {  // a last group of fewer than four rows is whole in the workspace
        iv4 v;
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = acc[4 * i + e];
        *reinterpret_cast<iv4*>(p + ((long long)((r >> 2) + 2 * i) * N + c) * 4) = v;
      }
  }
  template <int FM, int FN>
  __device__ __forceinline__ void finish(const iv16 (&acc)[FM][FN], int r0, int c0, int mr, int nr, float*) const {
    finish_direct<FM, FN>(*this, acc, r0, c0, mr, nr);
  }
};

template <typename EPI>
__global__ void __launch_bounds__(256) join_kernel(const int* __restrict__ part, int parts, long long stride, int M,
                                                   int N, EPI epi) {
  const long long groups = (M + 3ll) / 4, x = (long long)blockIdx.x * 256 + threadIdx.x;
  if (x >= groups * N) return;
  const long long g = x / N;
  const int c = (int)(x - g * N);
  iv4 s = {0, 0, 0, 0};
  for (int z = 0; z < parts; ++z) s += *reinterpret_cast<const iv4*>(part + z * stride + x * 4);
  epi.put4(4 * g, c, M, s);
}

// Whether rows can go to LDS directly.
static inline bool tile_dma(const void* p, long long ld, int K) {
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && ld % 16 == 0 && K % 16 == 0 && ld < (1ll << 24);
}

// Most tiles of a launch: its threads (up to 512 a tile) stay below 2^32.
constexpr long long kMaxTiles = 1ll << 22;
// Rows of one launch for a matrix of N columns: whole rows of every tile shape, at most kMaxTiles of the
// smallest tile of more than 64 rows, 128 x 128.  N is at most 2^26 (2^19 tiles across), so 1024 rows
// fit at the least.
constexpr long long tile_run(long long N) { return kMaxTiles / ((N + 127) / 128) * 128 / 256 * 256; }
constexpr bool tile_run_fits(long long N) {
  return tile_run(N) > 0 && tile_run(N) < (1ll << 31) && (tile_run(N) + 127) / 128 * ((N + 127) / 128) <= kMaxTiles;
}
static_assert(tile_run_fits(1) && tile_run_fits(128) && tile_run_fits(129) && tile_run_fits(1000003) &&
                  tile_run_fits(1ll << 26),
              "a run's tiles fit a launch");

// EPI::kAligned: the operands always can, so the other kernels are not built.
template <int BM, int BN, int WR, int WC, typename EPI>
static hipError_t tile_launch(const int8_t* A, long long lda, int M, const int8_t* B, long long ldb, int N, int K,
                              int parts, const EPI& epi, hipStream_t st) {
  const long long ntm = (M + BM - 1ll) / BM, ntn = (N + BN - 1ll) / BN;
  if (ntm * ntn > kMaxTiles) return hipErrorInvalidValue;
  const int kper = parts == 1 ? K : ((K + 127) / 128 + parts - 1) / parts * 128;
  const dim3 grid((unsigned)(ntm * ntn), (unsigned)parts);
  if (tile_dma(A, lda, K) && tile_dma(B, ldb, K)) {
    hipLaunchKernelGGL((tile_kernel<BM, BN, WR, WC, true, EPI>), grid, dim3(64 * WR * WC), 0, st, A, lda, M, B, ldb, N,
                       K, kper, (int)ntm, (int)ntn, epi);
  } else {
    if constexpr (EPI::kAligned) return hipErrorInvalidValue;
    else
      hipLaunchKernelGGL((tile_kernel<BM, BN, WR, WC, false, EPI>), grid, dim3(64 * WR * WC), 0, st, A, lda, M, B, ldb, N,
                         K, kper, (int)ntm, (int)ntn, epi);
  }
  return hipGetLastError();
}

// Parts of the row length for few tiles.  A stage of a tile with direct loads takes about 0.6 us however
// few workgroups run (the latency of its loads; 128 x 128 and 64 x 128), so a long row length on a card
// that is not full costs more than joining parts does: about 4 us and 8 bytes an element and part.  The
// rule counts a stage through registers the same, though it takes about 1.5 us (333 x 1021 x 2051: 12.5 us
// for eight), so rows at odd addresses are split later than they could be.
// At least three stages and sixteen bytes are left to every part.
struct TilePlan {
  bool small;  // 64 x 128 tiles (M <= 64)
  int parts;
  size_t bytes;  // of the parts
};
static inline TilePlan tile_plan(long long M, long long N, int K) {
  TilePlan p{M <= 64, 1, 0};
  const long long tiles = p.small ? (N + 127) / 128 : (M + 127) / 128 * ((N + 127) / 128);
  const int nk = (K + 127) / 128;
  const double bytes = 16.0 * (double)((M + 3) / 4) * (double)N;
  double best = 0.6 * nk;
  for (int s = 2; s <= 16 && tiles * s <= 512 && nk >= 3 * s; ++s) {
    const int per = (nk + s - 1) / s;
    if ((nk + per - 1) / per != s || K - (s - 1) * per * 128 < 16) continue;
    const double t = 0.6 * per + 4.0 + 2.0 * s * bytes / 4e6;
    if (t < best) {
      best = t;
      p.parts = s;
    }
  }
  if (p.parts > 1) p.bytes = (size_t)p.parts * (size_t)((M + 3) / 4) * (size_t)N * 16;
  return p;
}

// The tile shape by what its rounds over 256 CUs cost, in us at K = 2560: 38 for 256 x 256, 30 for
// 256 x 192, 22 for 512 tiles of 128 x 128 (its stages take 64 KB of LDS: two workgroups share a CU) and
// 13.5 for up to 256 of them.  Measured, 256 x 256 / 256 x 192 / 128 x 128: 8192 x 7680 x 2560 178 / 165 /
// 181 us, 2048 x 9728 x 2560 66 / 57 / 58, 1024 x 9728 x 2560 34 / 29 / 36, 4096 x 2560 x 9728 111 / 98 / 120.
template <typename EPI>
static hipError_t tile_whole(const int8_t* A, long long lda, int M, const int8_t* B, long long ldb, int N, int K,
                             const EPI& epi, hipStream_t st) {
  if (M <= 64) return tile_launch<64, 128, 2, 2>(A, lda, M, B, ldb, N, K, 1, epi, st);
  auto tiles = [&](int bm, int bn) { return ((M + bm - 1ll) / bm) * ((N + bn - 1ll) / bn); };
  const long long t1 = tiles(256, 256), t2 = tiles(256, 192), t3 = tiles(128, 128);
  const double c1 = 38.0 * ((t1 + 255) / 256), c2 = 30.0 * ((t2 + 255) / 256);
  const double c3 = 22.0 * (t3 / 512) + (t3 % 512 == 0 ? 0.0 : t3 % 512 <= 256 ? 13.5 : 22.0);
  if (c3 <= c1 && c3 <= c2) return tile_launch<128, 128, 2, 2>(A, lda, M, B, ldb, N, K, 1, epi, st);
  if (c2 <= c1) return tile_launch<256, 192, 4, 2>(A, lda, M, B, ldb, N, K, 1, epi, st);
  return tile_launch<256, 256, 2, 4>(A, lda, M, B, ldb, N, K, 1, epi, st);
}

// The product in whole or split tiles.  ws: tile_plan(M, N, K).bytes.
template <typename EPI>
static hipError_t tile_product(const int8_t* A, long long lda, int M, const int8_t* B, long long ldb, int N, int K,
                               const EPI& epi, void* ws, hipStream_t st) {
  const TilePlan p = tile_plan(M, N, K);
  if (p.parts == 1) return tile_whole(A, lda, M, B, ldb, N, K, epi, st);
  const long long groups = (M + 3ll) / 4, stride = groups * N * 4;
  int* part = static_cast<int*>(ws);
  const PartTile t{part, N, stride, nullptr};
  const hipError_t e = p.small ? tile_launch<64, 128, 2, 2>(A, lda, M, B, ldb, N, K, p.parts, t, st)
                               : tile_launch<128, 128, 2, 2>(A, lda, M, B, ldb, N, K, p.parts, t, st);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((join_kernel<EPI>), dim3((unsigned)((groups * N + 255) / 256)), dim3(256), 0, st, part, p.parts,
                     stride, M, N, epi);
  return hipGetLastError();
}

}  // namespace externd
