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

// What the product's sizes may be cut to by a count that only the device knows.
enum FCount { kAll, kRowsOfA, kRowsOfB, kLength };

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
// The operands pass through LDS in stages of 128 bytes of k a row (64 or 32 elements), two stages in turn,
// by direct loads of 16 bytes a lane.
//   along:  row r is 128 bytes and its 16-byte piece c sits at c ^ (r / 2 % 8), so that 16 consecutive
//           rows' pieces of one column lie in different banks
//   across: row k holds the tile's elements, 16-byte pieces.  fp16 and bf16 fragments are read by the
//           transposing load (16 lanes read four rows of 16 elements and get four k of an element each);
//           a wave's read takes 64 bytes of each of four rows at a time, so 64-byte chunk x of row k sits
//           at x ^ k % 4, all banks once.  fp32 fragments are four reads of one row each, the wave's halves four rows apart, and
//           the chunks of 128 bytes change places with k / 4.
// The fragments of the next step are read under the products of this one, and the barrier that hands a
// stage over comes before the last of its four steps.
constexpr int kFGroup = 4;

template <typename T, int ROWS, bool ACROSS>
struct FStage {  // where an operand's piece lies in a stage
  static constexpr int PPR = ACROSS ? ROWS * (int)sizeof(T) / 16 : 8;  // pieces of a row in LDS
  // across: what row k's pieces are moved by (xor)
  __device__ __forceinline__ static int swap(int k) {
    if (sizeof(T) == 4) return PPR >= 16 ? ((k >> 2) & 1) << 3 : 0;
    return PPR >= 16 ? (k & 3) << 2 : PPR == 8 ? ((k >> 1) & 1) << 2 : 0;
  }
};

template <typename T, int BM, int BN, int WR, int WC, bool AX, bool BX, FCount CUT, typename EPI>
__global__ void __launch_bounds__(64 * WR * WC, 1) ftile_kernel(FOperand A, int M, FOperand B, int N, int Kall, int kper,
                                                                int ntm, int ntn, const int* __restrict__ count, EPI epi) {
  typedef const __attribute__((address_space(1))) void gptr;
  typedef __attribute__((address_space(3))) void lptr;
  constexpr int NW = WR * WC, PA = BM / 8 / NW, PB = BN / 8 / NW, KS = 128 / (int)sizeof(T), ES = (int)sizeof(T);
  constexpr int FM = BM / WR / 32, FN = BN / WC / 32;
  static_assert(PA * 8 * NW == BM && PB * 8 * NW == BN && FM * 32 * WR == BM && FN * 32 * WC == BN, "tile shape");
  using SA = FStage<T, BM, AX>;
  using SB = FStage<T, BN, BX>;
  __shared__ __attribute__((aligned(1024))) int8_t l0[(BM + BN) * 128];
  __shared__ __attribute__((aligned(1024))) int8_t l1[(BM + BN) * 128];
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wr = wv / WC, wc = wv % WC;
  // workgroups go round the eight XCDs: each gets a run of neighbouring tiles, in groups of kFGroup tile rows
  const int total = ntm * ntn, per = (total + 7) / 8, rem = total % 8;
  const int xcd = blockIdx.x % 8, at = blockIdx.x / 8;
  const int tile = rem == 0 || xcd < rem ? xcd * per + at : rem * per + (xcd - rem) * (per - 1) + at;
  const int grp = tile / (kFGroup * ntn), g0 = grp * kFGroup, gs = ntm - g0 < kFGroup ? ntm - g0 : kFGroup;
  const int in = tile - g0 * ntn;
  const long long m0 = (long long)(g0 + in % gs) * BM, n0 = (long long)(in / gs) * BN;
  if (CUT != kAll) {
    const int c = *count;
    if (CUT == kRowsOfA && m0 >= c) return;
    if (CUT == kRowsOfB && n0 >= c) return;
    if (CUT == kLength) Kall = (c + 31) / 32 * 32;  // rows behind the count are zeros up to there
  }
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
      if (AX) {
        ka[p] = r;
        const int x = (c ^ SA::swap(r)) * 16;
        oka[p] = m0 + x / ES < M;
        ao[p] = (unsigned)r * lda + x;
      } else {
        ka[p] = (c ^ ((r >> 1) & 7)) * 16;
        oka[p] = true;
        ao[p] = (unsigned)(m0 + r < M ? r : M - 1 - m0) * lda + ka[p];
      }
    }
#pragma unroll
    for (int p = 0; p < PB; ++p) {
      const int q = (p * NW + wv) * 64 + lane, r = q / SB::PPR, c = q % SB::PPR;
      if (BX) {
        kb[p] = r;
        const int x = (c ^ SB::swap(r)) * 16;
        okb[p] = n0 + x / ES < N;
        bo[p] = (unsigned)r * ldb + x;
      } else {
        kb[p] = (c ^ ((r >> 1) & 7)) * 16;
        okb[p] = true;
        bo[p] = (unsigned)(n0 + r < N ? r : N - 1 - n0) * ldb + kb[p];
      }
    }
    const int8_t* zeros = reinterpret_cast<const int8_t*>(kFZeros);
    auto direct = [&](int8_t* l, int p, const int8_t* s) {
      __builtin_amdgcn_global_load_lds((gptr*)s, (lptr*)(l + (p * NW + wv) * 1024), 16, 0, 0);
    };
    // Stage 0 is the last of k, of which some may be missing; stage t > 0 the whole one from KS (t - 1) on.
    const int nk = (K + KS - 1) / KS, kl = KS * (nk - 1);
    const long long sta = AX ? (long long)lda * KS : 128, stb = BX ? (long long)ldb * KS : 128;
    // a third of stage t > 0 into l: three of the four steps between two barriers issue one each.  Every
    // direct load issued is waited for by a barrier before the kernel's end.
    auto fetch = [&](int8_t* l, int t, int third) {
      const int8_t* a = ab + (t - 1) * sta;
      const int8_t* b = bb + (t - 1) * stb;
      constexpr int all = PA + PB, each = (all + 2) / 3;
#pragma unroll
      for (int p = 0; p < all; ++p)
        if (p / each == third) {
          if (p < PA) {
            const int8_t* s = a + ao[p < PA ? p : 0];
            direct(l, p, AX && !oka[p < PA ? p : 0] ? zeros : s);
          } else {
            const int8_t* s = b + bo[p < PA ? 0 : p - PA];
            direct(l + BM * 128, p - PA, BX && !okb[p < PA ? 0 : p - PA] ? zeros : s);
          }
        }
      __builtin_amdgcn_sched_barrier(0);
    };
    {
      const int left = K - kl;
      const int8_t* a = ab + (nk - 1) * sta;
      const int8_t* b = bb + (nk - 1) * stb;
#pragma unroll
      for (int p = 0; p < PA; ++p) direct(l0, p, oka[p] && ka[p] < (AX ? left : left * ES) ? a + ao[p] : zeros);
#pragma unroll
      for (int p = 0; p < PB; ++p) direct(l0 + BM * 128, p, okb[p] && kb[p] < (BX ? left : left * ES) ? b + bo[p] : zeros);
    }
    const int lr = lane & 31, lg = lane >> 5;
    // along: the rows' offsets and their pieces' change of place
    const int ra = wr * (BM / WR) + lr, rb = wc * (BN / WC) + lr;  // rows r + 32 f share r / 2 % 8
    const int za = (ra >> 1) & 7, zb = (rb >> 1) & 7;
    // across, 16 bits: of the transposing read, lane i of sixteen reads row 8 (l / 32) + i / 4, elements
    // 16 (l / 16 % 2) + 4 (i % 4) on of the fragment's 32
    const int xk = 8 * lg + ((lane >> 2) & 3), xm = 16 * ((lane >> 4) & 1) + 4 * (lane & 3);
    iv4 fa[2][FM], fb[2][FN];
    auto across = [&](const int8_t* l, int row0, int ks, auto S) -> iv4 {
      using ST = decltype(S);
      constexpr int pitch = ST::PPR * 16;
      iv4 v;
      if constexpr (ES == 2) {
        typedef short s4 __attribute__((ext_vector_type(4)));
        typedef __attribute__((address_space(3))) s4 ls4;
        const int b = (row0 + xm) * 2;
        // k % 4 and, where rows are short, k / 2 % 2 do not change with ks or the two reads (multiples of 4)
        const int8_t* p = l + xk * pitch + (((b >> 4) ^ ST::swap(xk)) << 4) + (b & 15);
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
          v[e] = *reinterpret_cast<const int*>(l + k * pitch + (((b >> 4) ^ ST::swap(k)) << 4) + (b & 15));
        }
      }
      return v;
    };
    auto read = [&](int f, const int8_t* l, int ks) {  // fragments of step ks of the stage in l
#pragma unroll
      for (int i = 0; i < FM; ++i) {
        if constexpr (AX) fa[f][i] = across(l, wr * (BM / WR) + 32 * i, ks, SA{});
        else fa[f][i] = *reinterpret_cast<const iv4*>(l + (ra + 32 * i) * 128 + (((2 * ks + lg) ^ za) << 4));
      }
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        if constexpr (BX) fb[f][j] = across(l + BM * 128, wc * (BN / WC) + 32 * j, ks, SB{});
        else fb[f][j] = *reinterpret_cast<const iv4*>(l + BM * 128 + (rb + 32 * j) * 128 + (((2 * ks + lg) ^ zb) << 4));
      }
    };
    auto mul = [&](int f) {
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) acc[i][j] = fmul(T{}, fa[f][i], fb[f][j], acc[i][j]);
    };
    auto step = [&](int f, const int8_t* l, int ks) {  // products of fragments f under the reads of the next
      read(f ^ 1, l, ks);
      mul(f);
      constexpr int per_x = ES == 2 ? 2 : 4;
      constexpr int reads = FM * (AX ? per_x : 1) + FN * (BX ? per_x : 1), muls = FM * FN * (ES == 2 ? 1 : 4);
      interleave<reads, muls, reads < muls ? reads : muls>();
      __builtin_amdgcn_sched_barrier(0);
    };
    stage_barrier();
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
      stage_barrier();
      fetch(l0, t + 2, 0);
      step(1, l1, 0);
      fetch(l0, t + 2, 1);
      step(0, l1, 1);
      fetch(l0, t + 2, 2);
      step(1, l1, 2);
      step(0, l1, 3);
      stage_barrier();
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
      stage_barrier();
      step(1, l1, 0);
      step(0, l1, 1);
      step(1, l1, 2);
      step(0, l1, 3);
    }
    mul(1);
    if (EPI::kLds) __syncthreads();  // the stages are read: LDS is free
  }
  const int mr = M - m0 < BM ? (int)(M - m0) : BM, nr = N - n0 < BN ? (int)(N - n0) : BN;
  epi.template finish<T, BM, BN, WR, WC, FM, FN>(acc, m0, n0, mr, nr, wr, wc, l0, l1);
}

template <typename T, int BM, int BN, int WR, int WC, bool AX, bool BX, FCount CUT, typename EPI>
static hipError_t ftile_launch(FOperand A, long long M, FOperand B, long long N, long long K, int parts, const int* count,
                               const EPI& epi, hipStream_t st) {
  const long long ntm = (M + BM - 1) / BM, ntn = (N + BN - 1) / BN;
  if (ntm * ntn >= (1ll << 22) || M >= (1ll << 31) - 256 || N >= (1ll << 31) - 256 || K >= (1ll << 30)) return hipErrorInvalidValue;
  constexpr int KS = 128 / (int)sizeof(T);
  const long long kper = ((K + KS - 1) / KS + parts - 1) / parts * KS;
  hipLaunchKernelGGL((ftile_kernel<T, BM, BN, WR, WC, AX, BX, CUT, EPI>), dim3((unsigned)(ntm * ntn), (unsigned)parts),
                     dim3(64 * WR * WC), 0, st, A, (int)M, B, (int)N, (int)K, (int)kper, (int)ntm, (int)ntn, count, epi);
  return hipGetLastError();
}

}  // namespace externd
