// Products of floating-point matrices on the matrix cores: D[r][c] = sum_k A(r, k) B(c, k), fp32 sums
// of fp32, fp16 or bf16 operands, handed to an epilogue.  Each operand lies either with k running
// along its rows, or with its rows along k ("across": element (r, k) at p[k ld + r]).
#pragma once
#include "common.hpp"
#include "types.hpp"

namespace externd {

typedef float fv16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf8 __attribute__((ext_vector_type(8)));
typedef _Float16 hf8 __attribute__((ext_vector_type(8)));

// Accumulators += the products of one step: 32 bytes of k a row, 16 in each half of the wave.
__device__ __forceinline__ fv16 fmul(__bf16, iv4 a, iv4 b, fv16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf8, a), __builtin_bit_cast(bf8, b), c, 0, 0, 0);
}
__device__ __forceinline__ fv16 fmul(_Float16, iv4 a, iv4 b, fv16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(hf8, a), __builtin_bit_cast(hf8, b), c, 0, 0, 0);
}
// fp32: four products of two k, one of each half's four
__device__ __forceinline__ fv16 fmul(float, iv4 a, iv4 b, fv16 c) {
#pragma unroll
  for (int e = 0; e < 4; ++e)
    c = __builtin_amdgcn_mfma_f32_32x32x2f32(__int_as_float(a[e]), __int_as_float(b[e]), c, 0, 0, 0);
  return c;
}

// An operand: bases and row distances are multiples of 16 bytes, distances below 2^24 bytes.
//   along:  rows of which `rows` exist, K elements each; a row behind the last repeats it
//   across: K rows of `rows` elements; elements behind a row's last are zeros
// `rows` (across) and K (along) are multiples of 16 bytes.
struct FOperand {
  const void* p;
  long long ld;  // elements
};

static __device__ const int kFZeros[4] = {0, 0, 0, 0};  // what a direct load reads behind an operand's end

// Whether a launch holds so many tiles of so many threads.
static inline bool ftile_fits(long long tiles, int threads) { return tiles * threads < 1ll << 32; }

// What the product's sizes may be cut to by a count that only the device knows.
enum FCount { kRowsOfB, kLength };

// Scheduling groups that spread a step's reads of LDS evenly over its products.
template <int READS, int MULS, int SLOTS>
__device__ __forceinline__ void interleave() {
  if constexpr (SLOTS > 0) {
    constexpr int r = (READS + SLOTS - 1) / SLOTS, m = (MULS + SLOTS - 1) / SLOTS;
    __builtin_amdgcn_sched_group_barrier(0x100, r, 0);
    __builtin_amdgcn_sched_group_barrier(0x008, m, 0);
    interleave<READS - r, MULS - m, SLOTS - 1>();
  }
}

// ---- tiles --------------------------------------------------------------------------------------
// Workgroup: a BM x BN tile of D, WR x WC waves, each with FM x FN accumulators of 32 x 32 (A row and B
// row l % 32 of lane l, with 16 bytes of k each at 16 (l / 32) of the step; accumulator element i of lane l
// is row 8 (i / 4) + 4 (l / 32) + i % 4, column l % 32).
//
// The operands pass through LDS in stages of KB bytes of k a row (64 or 128), NB stages in turn, by direct loads of 16
// bytes a lane, so that NB - 1 stages are on their way while one is used.
//   along:  row r is KB bytes and its 16-byte pieces change places with r (see place()), so that 16 consecutive
//           rows' pieces of one column lie in different banks
//   across: row k holds the tile's elements, 16-byte pieces.  fp16 and bf16 fragments are read by the
//           transposing load (16 lanes read four rows of 16 elements and get four k of an element each);
//           a wave's read takes 64 bytes of each of four rows at a time, so 64-byte chunk x of row k sits
//           at x ^ k % 4, all banks once.  fp32 fragments are four reads of one row each, the wave's halves four rows
//           apart, and the chunks of 128 bytes change places with k / 4.
// The fragments of the next step are read under the products of this one, and the barrier that hands a
// stage over comes before the last of its steps.
// Measured (bf16, K = 2560): 256 x 256, eight waves, stages of 128 bytes, 4096 x 131072: 1.21 10^15 operations a second, a
// library product 1.28; the matrix cores are busy 54 to 58% of the time at 2.0 GHz, LDS as long as they would be if
// fed (reads of the fragments and the loads' writes).  Both operands across, 256 x 128, four waves, two workgroups a CU,
// three stages of 64 bytes: 1.11 10^15, 0.97 for 256 x 256 in two stages; along rows, 64 bytes are half a cache line and lost 25%.
constexpr int kFGroup = 4;  // 2, 8 and 16 measured the same
// Stages of a run of fp32 sums.  300 x 2560 x 32768, loss and dX: S 4.3e-6 off without runs, 7.0e-7 with, dX 1.7e-6 and 3.3e-7, for
// 1% more time (1181 and 1190 us; 65 x 777 x 10007 109 and 111); runs of four 5.8e-7, 2.7e-7 and 1203 us.
constexpr int kFRun = 8;

template <typename T, int ROWS, bool ACROSS, int KB>
struct FStage {  // where an operand's pieces lie in a stage
  static constexpr int PPR = ACROSS ? ROWS * (int)sizeof(T) / 16 : KB / 16;  // pieces of a row in LDS
  static_assert(ACROSS || KB == 128, "64 bytes of a row are half a cache line: slower where k runs along rows");
  // what row r's pieces are moved by (xor)
  __device__ __forceinline__ static int place(int r) {
    if (!ACROSS) return (r >> 1) & 7;
    if (sizeof(T) == 4) return PPR >= 16 ? ((r >> 2) & 1) << 3 : 0;
    return PPR >= 16 ? (r & 3) << 2 : PPR == 8 ? ((r >> 1) & 1) << 2 : 0;
  }
};

template <typename T, int BM, int BN, int WR, int WC, int KB, int NB, bool AX, bool BX, FCount CUT, typename EPI>
__global__ void __launch_bounds__(64 * WR * WC, WR * WC >= 8 ? 1 : 2) ftile_kernel(FOperand A, int M, FOperand B, int N, int Kall,
                                                                                   int kper, int ntm, int ntn,
                                                                                   const int* __restrict__ count, EPI epi) {
  constexpr int NW = WR * WC, PA = BM * KB / 1024 / NW, PB = BN * KB / 1024 / NW, ES = (int)sizeof(T), KS = KB / ES;
  constexpr int FM = BM / WR / 32, FN = BN / WC / 32, S = KB / 32, kStage = (BM + BN) * KB;
  static_assert(PA * 1024 * NW == BM * KB && PB * 1024 * NW == BN * KB && FM * 32 * WR == BM && FN * 32 * WC == BN, "tile shape");
  using SA = FStage<T, BM, AX, KB>;
  using SB = FStage<T, BN, BX, KB>;
  __shared__ __attribute__((aligned(1024))) int8_t lds[NB * kStage];
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wr = wv / WC, wc = wv % WC;
  // workgroups go round the eight XCDs: each gets a run of neighbouring tiles, in groups of kFGroup tile rows
  const int total = ntm * ntn, per = (total + 7) / 8, rem = total % 8;
  const int xcd = blockIdx.x % 8, at = blockIdx.x / 8;
  const int tile = rem == 0 || xcd < rem ? xcd * per + at : rem * per + (xcd - rem) * (per - 1) + at;
  const int grp = tile / (kFGroup * ntn), g0 = grp * kFGroup, gs = ntm - g0 < kFGroup ? ntm - g0 : kFGroup;
  const int in = tile - g0 * ntn;
  const long long m0 = (long long)(g0 + in % gs) * BM, n0 = (long long)(in / gs) * BN;
  const int counted = *count;
  if (CUT == kRowsOfB && n0 >= counted) return;
  if (CUT == kLength) Kall = (counted + 31) / 32 * 32;  // rows behind the count are zeros up to there
  const int kbeg = blockIdx.y * kper;
  const int K = Kall - kbeg < kper ? Kall - kbeg : kper;
  fv16 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;
  if (K > 0) {
    const int8_t* ab = static_cast<const int8_t*>(A.p) + (AX ? kbeg * A.ld + m0 : m0 * A.ld + kbeg) * ES;
    const int8_t* bb = static_cast<const int8_t*>(B.p) + (BX ? kbeg * B.ld + n0 : n0 * B.ld + kbeg) * ES;
    const unsigned lda = (unsigned)(A.ld * ES), ldb = (unsigned)(B.ld * ES);
    // this lane's piece of each of the wave's loads: its offset from the stage's base, the k (along: byte of
    // k, across: row) at which it starts, and whether it lies in the matrix at all
    unsigned ao[PA], bo[PB];
    int ka[PA], kb[PB];
    bool oka[PA], okb[PB];
#pragma unroll
    for (int p = 0; p < PA; ++p) {
      const int q = (p * NW + wv) * 64 + lane, r = q / SA::PPR, c = q % SA::PPR;
      const int x = (c ^ SA::place(r)) * 16;
      ka[p] = AX ? r : x;
      oka[p] = !AX || m0 + x / ES < M;
      ao[p] = AX ? (unsigned)r * lda + x : (unsigned)(m0 + r < M ? r : M - 1 - m0) * lda + x;
    }
#pragma unroll
    for (int p = 0; p < PB; ++p) {
      const int q = (p * NW + wv) * 64 + lane, r = q / SB::PPR, c = q % SB::PPR;
      const int x = (c ^ SB::place(r)) * 16;
      kb[p] = BX ? r : x;
      okb[p] = !BX || n0 + x / ES < N;
      bo[p] = BX ? (unsigned)r * ldb + x : (unsigned)(n0 + r < N ? r : N - 1 - n0) * ldb + x;
    }
    const int8_t* zeros = reinterpret_cast<const int8_t*>(kFZeros);
    // Stage 0 is the last of k, of which some may be missing; stage t > 0 the whole one from KS (t - 1) on.
    const int nk = (K + KS - 1) / KS, kl = KS * (nk - 1);
    const long long sta = AX ? (long long)lda * KS : KB, stb = BX ? (long long)ldb * KS : KB;
    const bool wa = !AX || m0 + BM <= M, wb = !BX || n0 + BN <= N;  // no row of the operand ends in the tile
    auto fetch = [&](int8_t* l, int t) {
      const int8_t* a = ab + (t - 1) * sta;
      const int8_t* b = bb + (t - 1) * stb;
      if (wa) {
#pragma unroll
        for (int p = 0; p < PA; ++p) lds_load16(l + (p * NW + wv) * 1024, a, ao[p]);
      } else {
#pragma unroll
        for (int p = 0; p < PA; ++p) lds_load16(l + (p * NW + wv) * 1024, oka[p] ? a + ao[p] : zeros);
      }
      if (wb) {
#pragma unroll
        for (int p = 0; p < PB; ++p) lds_load16(l + BM * KB + (p * NW + wv) * 1024, b, bo[p]);
      } else {
#pragma unroll
        for (int p = 0; p < PB; ++p) lds_load16(l + BM * KB + (p * NW + wv) * 1024, okb[p] ? b + bo[p] : zeros);
      }
      __builtin_amdgcn_sched_barrier(0);
    };
    {
      const int left = K - kl;
      const int8_t* a = ab + (nk - 1) * sta;
      const int8_t* b = bb + (nk - 1) * stb;
#pragma unroll
      for (int p = 0; p < PA; ++p)
        lds_load16(lds + (p * NW + wv) * 1024, oka[p] && ka[p] < (AX ? left : left * ES) ? a + ao[p] : zeros);
#pragma unroll
      for (int p = 0; p < PB; ++p)
        lds_load16(lds + BM * KB + (p * NW + wv) * 1024, okb[p] && kb[p] < (BX ? left : left * ES) ? b + bo[p] : zeros);
    }
    const int lr = lane & 31, lg = lane >> 5;
    // along: the rows' offsets and their pieces' change of place (the same for rows 32 apart)
    const int ra = wr * (BM / WR) + lr, rb = wc * (BN / WC) + lr, za = SA::place(ra), zb = SB::place(rb);
    // across, 16 bits: of the transposing read, lane i of sixteen reads row 8 (l / 32) + i / 4, elements
    // 16 (l / 16 % 2) + 4 (i % 4) on of the fragment's 32
    const int xk = 8 * lg + ((lane >> 2) & 3), xm = 16 * ((lane >> 4) & 1) + 4 * (lane & 3);
    iv4 fa[2][FM], fb[2][FN];
    auto across = [&](const int8_t* l, int row0, int ks, auto which) -> iv4 {
      using ST = decltype(which);
      constexpr int pitch = ST::PPR * 16;
      iv4 v;
      if constexpr (ES == 2) {
        typedef short s4 __attribute__((ext_vector_type(4)));
        typedef __attribute__((address_space(3))) s4 ls4;
        const int b = (row0 + xm) * 2;
        // what the rows change by does not change with ks or between the two reads (multiples of 4)
        const int8_t* p = l + xk * pitch + (((b >> 4) ^ ST::place(xk)) << 4) + (b & 15);
        const s4 u0 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((ls4*)(p + 16 * ks * pitch));
        const s4 u1 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((ls4*)(p + (16 * ks + 4) * pitch));
        typedef int i2 __attribute__((ext_vector_type(2)));
        const i2 w0 = __builtin_bit_cast(i2, u0), w1 = __builtin_bit_cast(i2, u1);
        v = iv4{w0[0], w0[1], w1[0], w1[1]};
      } else {
        const int b = (row0 + lr) * 4;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int k = 8 * ks + 4 * lg + e;
          v[e] = *reinterpret_cast<const int*>(l + k * pitch + (((b >> 4) ^ ST::place(k)) << 4) + (b & 15));
        }
      }
      return v;
    };
    auto read = [&](int f, const int8_t* l, int ks) {  // fragments of step ks of the stage in l
#pragma unroll
      for (int i = 0; i < FM; ++i) {
        if constexpr (AX) fa[f][i] = across(l, wr * (BM / WR) + 32 * i, ks, SA{});
        else fa[f][i] = *reinterpret_cast<const iv4*>(l + (ra + 32 * i) * KB + (((2 * ks + lg) ^ za) << 4));
      }
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        if constexpr (BX) fb[f][j] = across(l + BM * KB, wc * (BN / WC) + 32 * j, ks, SB{});
        else fb[f][j] = *reinterpret_cast<const iv4*>(l + BM * KB + (rb + 32 * j) * KB + (((2 * ks + lg) ^ zb) << 4));
      }
    };
    auto mul = [&](int f) {
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) acc[i][j] = fmul(T{}, fa[f][i], fb[f][j], acc[i][j]);
    };
    constexpr int each = ES == 2 ? 2 : 4, reads = FM * (AX ? each : 1) + FN * (BX ? each : 1), muls = FM * FN * (ES == 2 ? 1 : 4);
    auto spread = [&]() {
      interleave<reads, muls, reads < muls ? reads : muls>();
      __builtin_amdgcn_sched_barrier(0);
    };
    // The stage behind t is in LDS (of this wave's loads at most those of NB - 2 stages behind that are on their way), and
    // the reads of t are done, so that its place may be filled.
    constexpr int kLoads = PA + PB;
    auto handover = [&](int t) {
      if (t + NB - 1 < nk) asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"((NB - 2) * kLoads) : "memory");
      else asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
      asm volatile("s_barrier" ::: "memory");
    };
#pragma unroll
    for (int i = 1; i < NB; ++i)
      if (i < nk) fetch(lds + i * kStage, i);
    if (nk >= NB) asm volatile("s_waitcnt vmcnt(%0)" ::"n"((NB - 1) * kLoads) : "memory");
    else asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    asm volatile("s_barrier" ::: "memory");
    read(0, lds, 0);
    __builtin_amdgcn_sched_barrier(0);
    // fp32 operands hold what fp32 sums lose: these go in runs of kFRun stages (256 k), added up apart, so that a sum of K
    // terms rounds like one of 256 + K / 256.
    constexpr bool kRuns = ES == 4;
    fv16 runs[kRuns ? FM : 1][kRuns ? FN : 1];
    auto run = [&](bool first) {
      if constexpr (kRuns) {
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
          for (int j = 0; j < FN; ++j)
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              runs[i][j][e] = first ? 0.0f : runs[i][j][e] + acc[i][j][e];
              acc[i][j][e] = 0.0f;
            }
      }
    };
    run(true);
    int here = 0;  // of the stage's place
    for (int t = 0; t < nk - 1; ++t) {
      if (kRuns && t > 0 && t % kFRun == 0) run(false);
      int8_t* l = lds + here;
      here = here == (NB - 1) * kStage ? 0 : here + kStage;
#pragma unroll
      for (int k = 0; k < S; ++k) {
        if (k < S - 1) {
          read((k + 1) & 1, l, k + 1);
        } else {
          handover(t);
          if (t + NB < nk) fetch(l, t + NB);
          read(0, lds + here, 0);
        }
        mul(k & 1);
        spread();
      }
    }
#pragma unroll
    for (int k = 0; k < S; ++k) {
      if (k < S - 1) read((k + 1) & 1, lds + here, k + 1);
      mul(k & 1);
      if (k < S - 1) spread();
    }
    if constexpr (kRuns) {
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
          for (int e = 0; e < 16; ++e) acc[i][j][e] += runs[i][j][e];
    }
    if (EPI::kLds) __syncthreads();  // the stages are read: LDS is free
  }
  const int mr = M - m0 < BM ? (int)(M - m0) : BM, nr = N - n0 < BN ? (int)(N - n0) : BN;
  epi.template finish<T, BM, BN, WR, WC, FM, FN, NB * kStage>(acc, m0, n0, mr, nr, wr, wc, lds);
}

template <typename T, int BM, int BN, int WR, int WC, int KB, int NB, bool AX, bool BX, FCount CUT, typename EPI>
static hipError_t ftile_launch(FOperand A, long long M, FOperand B, long long N, long long K, int parts, const int* count,
                               const EPI& epi, hipStream_t st) {
  const long long ntm = (M + BM - 1) / BM, ntn = (N + BN - 1) / BN;
  if (!ftile_fits(ntm * ntn * parts, 64 * WR * WC) || M >= (1ll << 31) - 256 || N >= (1ll << 31) - 256 || K >= (1ll << 30)) return hipErrorInvalidValue;
  constexpr int KS = KB / (int)sizeof(T);
  const long long kper = ((K + KS - 1) / KS + parts - 1) / parts * KS;
  hipLaunchKernelGGL((ftile_kernel<T, BM, BN, WR, WC, KB, NB, AX, BX, CUT, EPI>), dim3((unsigned)(ntm * ntn), (unsigned)parts),
                     dim3(64 * WR * WC), 0, st, A, (int)M, B, (int)N, (int)K, (int)kper, (int)ntm, (int)ntn, count, epi);
  return hipGetLastError();
}

}  // namespace externd
