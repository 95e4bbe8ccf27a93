// What the kernels of the 4-bit products share: codes, tokens and scales as the matrix cores take them.
#pragma once
#include "common.hpp"
#include "externd_internal.hpp"
#include "types.hpp"

namespace externd {

// a number stored as fp32 (type 0), fp16 (1) or bf16 (2)
__device__ __forceinline__ void put_scale(void* p, int type, long long at, float v) {
  if (type == 0) static_cast<float*>(p)[at] = v;
  else if (type == 1) static_cast<_Float16*>(p)[at] = (_Float16)v;
  else static_cast<__bf16*>(p)[at] = (__bf16)v;
}
// A code enters the matrix cores as the number c + 8: its four bits, the sign turned, are an e4m3 number of 2^-9 (c + 8) as
// they are (the smallest exponents of e4m3 are one straight line), and one conversion widens two of them.  So eight
// codes cost nine instructions, and for each group
//   y += s sum (c + 8) x + (o - 8 s) sum x
// with sum x from the same x by products with ones.  The excess costs the sums one to two of fp32's bits.
template <typename T>
__device__ __forceinline__ iv4 widen(unsigned w) {  // eight codes, signs turned, in their order
  const unsigned even = w & 0x0F0F0F0Fu, odd = (w >> 4) & 0x0F0F0F0Fu;
  const unsigned p[2] = {__builtin_amdgcn_perm(odd, even, 0x05010400u), __builtin_amdgcn_perm(odd, even, 0x07030602u)};
  iv4 r;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if constexpr (__is_same(T, _Float16)) {
      r[2 * i] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(p[i], 512.0f, false));
      r[2 * i + 1] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(p[i], 512.0f, true));
    } else {
      r[2 * i] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(p[i], 512.0f, false));
      r[2 * i + 1] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(p[i], 512.0f, true));
    }
  }
  return r;
}
constexpr unsigned kSignTurn = 0x88888888u;

typedef __bf16 bf8 __attribute__((ext_vector_type(8)));
typedef _Float16 hf8 __attribute__((ext_vector_type(8)));
__device__ __forceinline__ fv4 gmul(__bf16, iv4 a, iv4 b, fv4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf8, a), __builtin_bit_cast(bf8, b), c, 0, 0, 0);
}
__device__ __forceinline__ fv4 gmul(_Float16, iv4 a, iv4 b, fv4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(hf8, a), __builtin_bit_cast(hf8, b), c, 0, 0, 0);
}

// Tokens as the matrix cores take them: fp16 and bf16 as they are; fp32 in three bf16 pieces of eight bits, cut off one
// after the other (exact: what is left of 24 bits fits the third).
template <typename XT>
struct Pieces {
  using type = XT;
  static constexpr int count = 1;
};
template <>
struct Pieces<float> {
  using type = __bf16;
  static constexpr int count = 3;
};
__device__ __forceinline__ void pieces8(const float (&v)[8], iv4 (&p)[3]) {
#pragma unroll
  for (int e = 0; e < 8; e += 2) {
    float a = v[e], b = v[e + 1];
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      const unsigned ua = __float_as_uint(a), ub = __float_as_uint(b);
      p[k][e / 2] = (int)__builtin_amdgcn_perm(ub, ua, 0x07060302u);  // both high halves
      a -= __uint_as_float(ua & 0xFFFF0000u);
      b -= __uint_as_float(ub & 0xFFFF0000u);
    }
  }
}
// 8 elements of a token at j, where TAIL zeros from n on
template <bool TAIL, typename XT>
__device__ __forceinline__ void token8(const XT* __restrict__ x, int j, int n, iv4 (&p)[1]) {
  if (!TAIL || j + 8 <= n) {
    p[0] = *reinterpret_cast<const iv4_any*>(x + j);
  } else {
    typedef XT v8 __attribute__((ext_vector_type(8)));
    v8 t;
#pragma unroll
    for (int e = 0; e < 8; ++e) t[e] = j + e < n ? x[j + e] : (XT)0.0f;
    p[0] = __builtin_bit_cast(iv4, t);
  }
}
template <bool TAIL>
__device__ __forceinline__ void token8(const float* __restrict__ x, int j, int n, iv4 (&p)[3]) {
  float v[8];
  if (!TAIL || j + 8 <= n) load8(x + j, v);
  else load8_tail(x + j, n - j, v);
  pieces8(v, p);
}

// the same from words already loaded
template <typename XT>
__device__ __forceinline__ void whole8(const iv4 (&h)[words8<XT>()], iv4 (&p)[Pieces<XT>::count]) {
  if constexpr (sizeof(XT) == 4) {
    float v[8];
    unpack8<XT>(h, v);
    pieces8(v, p);
  } else {
    p[0] = h[0];
  }
}

// Four registers of the wave's four groups of 16 lanes transposed: register j of group g becomes register g of group j.
__device__ __forceinline__ iv4 transpose4(iv4 v) {
  const auto a = __builtin_amdgcn_permlane32_swap(v[0], v[2], false, false);
  const auto b = __builtin_amdgcn_permlane32_swap(v[1], v[3], false, false);
  const auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
  const auto d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
  return iv4{(int)c[0], (int)c[1], (int)d[0], (int)d[1]};
}

// The scales of a wave's channels, one load a chunk of 128 codes: lane group g holds that of the chunk's g-th 32 codes,
// and spread() gives every lane all of them.
template <int SB>
__device__ __forceinline__ unsigned scale_bits(const void* p, long long at) {
  return SB == 4 ? static_cast<const unsigned*>(p)[at] : static_cast<const unsigned short*>(p)[at];
}
template <int SB>
__device__ __forceinline__ float scale_value(unsigned bits, bool half) {
  if (SB == 4) return __uint_as_float(bits);
  return half ? (float)__builtin_bit_cast(_Float16, (unsigned short)bits) : __uint_as_float(bits << 16);
}
template <int GROUP>
__device__ __forceinline__ void spread(float v, float (&o)[128 / GROUP]) {
  const unsigned u = __float_as_uint(v);
  if constexpr (GROUP == 128) {
    o[0] = v;
  } else {
    const auto h = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    if constexpr (GROUP == 64) {
      o[0] = __uint_as_float(h[0]);
      o[1] = __uint_as_float(h[1]);
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const auto q = __builtin_amdgcn_permlane16_swap(h[i], h[i], false, false);
        o[2 * i] = __uint_as_float(q[0]);
        o[2 * i + 1] = __uint_as_float(q[1]);
      }
    }
  }
}

// ---- few tokens: 16 CT output channels and 16 NT tokens a workgroup; the row goes round its waves in chunks of 128 codes.
// MFMA D(16 x 16) += A(16 x 32) B(32 x 16): A row = token, B column = channel, lane l holding the eight elements at
// 8 (l / 16) of row (column) l % 16; D's column l % 16, rows 4 (l / 16) on.  A lane loads 16 bytes of its channel's codes, and
// the transposition gives each product 32 consecutive ones, so that groups of 32 need nothing else.  The waves' partial
// sums add in LDS in their order.
constexpr int kGroupedWaves = 8;

template <typename XT, int NT, int CT, int GROUP, int SB>
__global__ void __launch_bounds__(64 * kGroupedWaves) grouped_few_kernel(GroupedLaunch L) {
  using T = typename Pieces<XT>::type;
  constexpr int NP = Pieces<XT>::count, G = 128 / GROUP;
  // chunks whose loads are in flight together, the tokens' among them where those fit the registers
  constexpr int U = NT * CT == 1 && sizeof(XT) == 2 ? 4 : 2;
  constexpr bool EARLY = NT == 1;
  __shared__ float red[kGroupedWaves][CT * NT * 256];
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lr = lane & 15, lg = lane >> 4;
  const int r0 = blockIdx.x * (16 * CT), n = L.n;
  const long long t0 = (long long)blockIdx.y * (16 * NT);
  const int groups = (n + GROUP - 1) / GROUP, words = groups * (GROUP / 8);
  const bool half = L.s_type == 1, offsets = L.offset != nullptr;
  const int* q[CT];
  long long sbase[CT];
#pragma unroll
  for (int i = 0; i < CT; ++i) {
    const int ch = r0 + 16 * i + lr < L.m ? r0 + 16 * i + lr : L.m - 1;
    q[i] = L.Q + (long long)ch * L.ldq;
    sbase[i] = (long long)ch * groups;
  }
  const XT* x[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const long long c = t0 + 16 * t + lr;
    x[t] = static_cast<const XT*>(L.X) + (c < L.tokens ? c : L.tokens - 1) * L.ldx + 8 * lg;
  }
  fv4 acc[CT][NT];
#pragma unroll
  for (int i = 0; i < CT; ++i)
#pragma unroll
    for (int t = 0; t < NT; ++t) acc[i][t] = fv4{0, 0, 0, 0};
  const int one = __is_same(T, _Float16) ? 0x3C003C00 : 0x3F803F80;
  const iv4 ones = {one, one, one, one};
  struct Chunk {
    iv4 w[CT];
    unsigned s[CT], o[CT];
  };
  auto load = [&](int c) {  // codes behind the row's end are its last, and meet zeros
    Chunk d;
    const int k = 16 * c + 4 * lg, g = G * c + lg * G / 4;
#pragma unroll
    for (int i = 0; i < CT; ++i) {
      d.w[i] = *reinterpret_cast<const iv4_any*>(q[i] + (k < words ? k : words - 4));
      const long long at = sbase[i] + (g < groups ? g : groups - 1);
      d.s[i] = scale_bits<SB>(L.scale, at);
      d.o[i] = offsets ? scale_bits<SB>(L.offset, at) : 0u;
    }
    return d;
  };
  auto chunk = [&](Chunk d, auto token) {
    float s[CT][G], b[CT][G];
#pragma unroll
    for (int i = 0; i < CT; ++i) {
      d.w[i] = transpose4(d.w[i] ^ (int)kSignTurn);
      const float sv = scale_value<SB>(d.s[i], half), bv = scale_value<SB>(d.o[i], half) - 8.0f * sv;
      spread<GROUP>(sv, s[i]);
      spread<GROUP>(bv, b[i]);
    }
#pragma unroll
    for (int g = 0; g < G; ++g) {
      fv4 part[CT][NT], sum[NT];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        sum[t] = fv4{0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < CT; ++i) part[i][t] = fv4{0, 0, 0, 0};
      }
#pragma unroll
      for (int k = g * (4 / G); k < (g + 1) * (4 / G); ++k) {
        iv4 wide[CT];
#pragma unroll
        for (int i = 0; i < CT; ++i) wide[i] = widen<T>((unsigned)d.w[i][k]);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          iv4 p[NP];
          token(k, t, p);
#pragma unroll
          for (int h = 0; h < NP; ++h) {
#pragma unroll
            for (int i = 0; i < CT; ++i) part[i][t] = gmul(T{}, p[h], wide[i], part[i][t]);
            sum[t] = gmul(T{}, p[h], ones, sum[t]);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < CT; ++i)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[i][t][e] += s[i][g] * part[i][t][e] + b[i][g] * sum[t][e];
      // one group after the other: left alone, the sums of all groups wait for one another, in twice the registers
#pragma unroll
      for (int i = 0; i < CT; ++i)
#pragma unroll
        for (int t = 0; t < NT; ++t) asm volatile("" : "+v"(acc[i][t]), "+v"(d.w[i]));
    }
  };
  const int full = n / 128;
  for (int c = wv; c < full; c += U * kGroupedWaves) {
    Chunk d[U];
    iv4 raw[EARLY ? U : 1][4][words8<XT>()];
    // the first chunk again where there are fewer: loads that depend on no branch
#pragma unroll
    for (int u = 0; u < U; ++u) d[u] = load(c + u * kGroupedWaves < full ? c + u * kGroupedWaves : c);
    if constexpr (EARLY) {
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
          for (int h = 0; h < words8<XT>(); ++h)
            raw[u][k][h] = word8(x[0] + 128 * (c + u * kGroupedWaves < full ? c + u * kGroupedWaves : c) + 32 * k, h);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int at = c + u * kGroupedWaves;
      if (at < full)
        chunk(d[u], [&](int k, int t, iv4 (&p)[NP]) {
          if constexpr (EARLY) whole8<XT>(raw[u][k], p);
          else token8<false>(x[t], 128 * at + 32 * k, n, p);
        });
    }
  }
  if (full % kGroupedWaves == wv && n % 128 != 0)  // the rows' end: one wave
    chunk(load(full), [&](int k, int t, iv4 (&p)[NP]) { token8<true>(x[t], 128 * full + 32 * k, n - 8 * lg, p); });
#pragma unroll
  for (int i = 0; i < CT; ++i)
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) red[wv][(16 * t + 4 * lg + e) * (16 * CT) + 16 * i + lr] = acc[i][t][e];
  __syncthreads();
  for (int i = threadIdx.x; i < CT * NT * 256; i += 64 * kGroupedWaves) {
    const long long t = t0 + i / (16 * CT);
    const int o = r0 + i % (16 * CT);
    if (t < L.tokens && o < L.m) {
      float v = 0.0f;
#pragma unroll
      for (int w = 0; w < kGroupedWaves; ++w) v += red[w][i];
      put_scale(L.Y, L.y_type, t * L.ldy + o, v);
    }
  }
}

template <typename XT, int NT, int CT, int GROUP, int SB>
static hipError_t few_launch(const GroupedLaunch& all, hipStream_t st) {
  GroupedLaunch L = all;
  const long long step = 65535ll * 16 * NT;
  for (long long t = 0; t < all.tokens; t += step) {
    L.tokens = all.tokens - t < step ? all.tokens - t : step;
    L.X = static_cast<const XT*>(all.X) + t * L.ldx;
    L.Y = static_cast<char*>(all.Y) + t * L.ldy * (L.y_type == 0 ? 4 : 2);
    hipLaunchKernelGGL((grouped_few_kernel<XT, NT, CT, GROUP, SB>), dim3((unsigned)((L.m + 16ll * CT - 1) / (16 * CT)), (unsigned)((L.tokens + 16 * NT - 1) / (16 * NT))),
                       dim3(64 * kGroupedWaves), 0, st, L);
  }
  return hipGetLastError();
}


// ---- many tokens --------------------------------------------------------------------------------------
// The tokens are laid out first: aligned rows of whole chunks of 128, fp32 as three planes of pieces, zeros behind a
// row's end, and beside them -8 times each group's sum.  So the tiles need no other path for odd sizes or addresses, and
// a group's partial sum starts from the excess it has to lose:
//   part = -8 sum x + sum (c + 8) x,   y += s part + o sum x
struct GroupedX {
  const void* x;      // [plane][padded][np]
  const float* sums;  // [group][padded]
  long long padded;
  int np, groups;     // groups of np
};

template <typename XT, int GROUP>
__global__ void __launch_bounds__(256) grouped_tokens_kernel(const XT* __restrict__ X, long long ldx, long long tokens, int n, int np,
                                                             long long padded, iv4* __restrict__ out, float* __restrict__ sums) {
  constexpr int NP = Pieces<XT>::count, L = GROUP / 8;
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x;  // of eight elements
  const int row8 = np / 8;
  const long long t = i / row8;
  if (t >= tokens) return;  // np / 8 is a multiple of 16: a group's threads end together
  const int j = (int)(i - t * row8) * 8;
  iv4 p[NP];
  float v[8], s = 0.0f;
  const XT* x = X + t * ldx;
  if (j + 8 <= n) load8(x + j, v);
  else load8_tail(x + j, (long long)n - j, v);
  if constexpr (NP == 3) {
    pieces8(v, p);
  } else {
    typedef XT v8 __attribute__((ext_vector_type(8)));
    v8 o;
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = (XT)v[e];  // as it was
    p[0] = __builtin_bit_cast(iv4, o);
  }
#pragma unroll
  for (int h = 0; h < NP; ++h) out[(h * padded + t) * row8 + j / 8] = p[h];
#pragma unroll
  for (int e = 0; e < 8; ++e) s += v[e];
#pragma unroll
  for (int d = 1; d < L; d <<= 1) s += __shfl_xor(s, d);
  if ((threadIdx.x & (L - 1)) == 0) sums[(long long)(j / GROUP) * padded + t] = -8.0f * s;
}

typedef float fv16 __attribute__((ext_vector_type(16)));
__device__ __forceinline__ fv16 gmul32(__bf16, iv4 a, iv4 b, fv16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf8, a), __builtin_bit_cast(bf8, b), c, 0, 0, 0);
}
__device__ __forceinline__ fv16 gmul32(_Float16, iv4 a, iv4 b, fv16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(hf8, a), __builtin_bit_cast(hf8, b), c, 0, 0, 0);
}

// Workgroup: BM tokens and 64 WC channels (32 FN each of WC waves across), WR waves down.  The tokens go through LDS in stages of 128
// elements a row, two in turn, by direct loads; row r's 16-byte piece c sits at c ^ r % 16, so that 32 rows' pieces of one column take every
// bank twice.  The codes go from memory to registers, 16 bytes a lane, one stage ahead, and every wave widens its
// own (the waves down the tile repeat that: it is vector work under the others' products).  A register swap between the
// wave's halves puts the words where a product of 16 elements wants them.
// MFMA D(32 x 32) += A(32 x 16) B(16 x 32): A row = token l % 32, B column = channel l % 32, both with the eight
// elements at 8 (l / 32) of the step.
template <typename XT, int BM, int WR, int WC, int FN, int GROUP, int SB>
__global__ void __launch_bounds__(64 * WR * WC, 1) grouped_tile_kernel(GroupedLaunch L, GroupedX X, int ntm, int ntn, int sper,
                                                                       float* __restrict__ partial) {
  using T = typename Pieces<XT>::type;
  constexpr int NP = Pieces<XT>::count, G = 128 / GROUP, FM = BM / WR / 32, NW = WR * WC, BN = 32 * FN * WC;
  constexpr int kRows = NP * BM, PL = kRows / 4 / NW;  // direct loads of a wave and stage: four rows each
  constexpr int kSums = G * BM * 4 / 1024 > 0 ? G * BM * 4 / 1024 : 1;  // and of the group sums, in all
  static_assert(PL * 4 * NW == kRows && FM * 32 * WR == BM && kSums <= NW, "tile shape");
  typedef const __attribute__((address_space(1))) void gptr;
  typedef __attribute__((address_space(3))) void lptr;
  constexpr int kStage = kRows * 256 + kSums * 1024;
  __shared__ __attribute__((aligned(1024))) int8_t l0[kStage];
  __shared__ __attribute__((aligned(1024))) int8_t l1[kStage];
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wr = wv / WC, wc = wv % WC, lr = lane & 31, lg = lane >> 5;
  // workgroups go round the eight XCDs: each gets a run of neighbouring tiles, the tokens of one run of channels after each other
  const int total = ntm * ntn, per = (total + 7) / 8, rem = total % 8;
  const int xcd = blockIdx.x % 8, at = blockIdx.x / 8;
  const int tile = rem == 0 || xcd < rem ? xcd * per + at : rem * per + (xcd - rem) * (per - 1) + at;
  const long long m0 = (long long)(tile % ntm) * BM;
  const int n0 = tile / ntm * BN;
  const int stages = X.np / 128, s0 = blockIdx.y * sper, s1 = s0 + sper < stages ? s0 + sper : stages;
  const int groups = (L.n + GROUP - 1) / GROUP, words = groups * (GROUP / 8);
  const bool half = L.s_type == 1, offsets = L.offset != nullptr;
  const int8_t* xb = static_cast<const int8_t*>(X.x);
  const int pitch = X.np * 2;
  unsigned xo[PL];  // this lane's piece of each of the wave's loads, from the tile's first token of the plane
#pragma unroll
  for (int p = 0; p < PL; ++p) {
    const int r = (p * NW + wv) * 4 + (lane >> 4);
    const long long t = m0 + r % BM < L.tokens ? r % BM : L.tokens - 1 - m0;
    xo[p] = (unsigned)t * (unsigned)pitch + (((lane & 15) ^ (r & 15)) << 4);
  }
  const int* q[FN];
  long long sbase[FN];
#pragma unroll
  for (int j = 0; j < FN; ++j) {
    const int o = n0 + (wc * FN + j) * 32 + lr, ch = o < L.m ? o : L.m - 1;
    q[j] = L.Q + (long long)ch * L.ldq;
    sbase[j] = (long long)ch * groups;
  }
  struct Codes {
    iv4 w[FN][2];
    unsigned s[FN][G], o[FN][G];
  };
  auto codes = [&](int t) {  // words behind the row's end are its last, and meet zeros
    Codes d;
#pragma unroll
    for (int j = 0; j < FN; ++j) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int k = 16 * t + 8 * h + 4 * lg;
        d.w[j][h] = *reinterpret_cast<const iv4_any*>(q[j] + (k < words ? k : words - 4));
      }
#pragma unroll
      for (int g = 0; g < G; ++g) {
        const long long a = sbase[j] + (G * t + g < groups ? G * t + g : groups - 1);
        d.s[j][g] = scale_bits<SB>(L.scale, a);
        d.o[j][g] = offsets ? scale_bits<SB>(L.offset, a) : 0u;
      }
    }
    return d;
  };
  auto fetch = [&](int8_t* l, int t) {
#pragma unroll
    for (int p = 0; p < PL; ++p) {
      const int8_t* x = xb + ((p * NW + wv) * 4 / BM * X.padded + m0) * pitch + t * 256ll;  // the same for the wave
      __builtin_amdgcn_global_load_lds((gptr*)(x + xo[p]), (lptr*)(l + (p * NW + wv) * 1024), 16, 0, 0);
    }
    if (wv < kSums) {
      // group sums of the stage, [group][BM]: 256 of them a load; behind the last they repeat it
      const int e = wv * 256 + lane * 4;
      const int g = e / BM < G ? e / BM : G - 1;
      const float* s = X.sums + (long long)(G * t + g) * X.padded + m0 + e % BM;
      __builtin_amdgcn_global_load_lds((gptr*)s, (lptr*)(l + kRows * 256 + wv * 1024), 16, 0, 0);
    }
  };
  fv16 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;
  const int row = wr * (BM / WR) + lr;  // rows r + 32 f share r % 16
  auto excess = [&](const float* s) {  // of the 16 rows of an accumulator
    fv16 v;
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const fv4 u = *reinterpret_cast<const fv4*>(s + 8 * x);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[4 * x + e] = u[e];
    }
    return v;
  };
  auto compute = [&](const int8_t* l, Codes d) {
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const iv4 w = d.w[j][h] ^ (int)kSignTurn;
        const auto a = __builtin_amdgcn_permlane32_swap(w[0], w[1], false, false);
        const auto b = __builtin_amdgcn_permlane32_swap(w[2], w[3], false, false);
        d.w[j][h] = iv4{(int)a[0], (int)b[0], (int)a[1], (int)b[1]};
      }
    const float* sums = reinterpret_cast<const float*>(l + kRows * 256) + wr * (BM / WR) + 4 * lg;
#pragma unroll
    for (int g = 0; g < G; ++g) {
      fv16 part[FM][FN];
#pragma unroll
      for (int i = 0; i < FM; ++i) {
        const fv16 lose = excess(sums + g * BM + 32 * i);
#pragma unroll
        for (int j = 0; j < FN; ++j) part[i][j] = lose;
      }
#pragma unroll
      for (int k = g * (8 / G); k < (g + 1) * (8 / G); ++k) {
        iv4 b[FN];
#pragma unroll
        for (int j = 0; j < FN; ++j) b[j] = widen<T>((unsigned)d.w[j][k >> 2][k & 3]);
#pragma unroll
        for (int h = 0; h < NP; ++h)
#pragma unroll
          for (int i = 0; i < FM; ++i) {
            const iv4 a = *reinterpret_cast<const iv4*>(l + (h * BM + row + 32 * i) * 256 + (((2 * k + lg) ^ (lr & 15)) << 4));
#pragma unroll
            for (int j = 0; j < FN; ++j) part[i][j] = gmul32(T{}, a, b[j], part[i][j]);
          }
      }
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        const float s = scale_value<SB>(d.s[j][g], half);
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
          for (int e = 0; e < 16; ++e) acc[i][j][e] = fmaf(s, part[i][j][e], acc[i][j][e]);
      }
      if (offsets) {
#pragma unroll
        for (int i = 0; i < FM; ++i) {
          const fv16 lose = excess(sums + g * BM + 32 * i);
#pragma unroll
          for (int j = 0; j < FN; ++j) {
            const float o = -0.125f * scale_value<SB>(d.o[j][g], half);
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[i][j][e] = fmaf(o, lose[e], acc[i][j][e]);
          }
        }
      }
    }
  };
  if (s0 < s1) {
    fetch(l0, s0);
    Codes d = codes(s0);
    for (int t = s0; t < s1; t += 2) {
      __syncthreads();  // stage t is in l0, and l1 is read
      Codes e = d;
      if (t + 1 < s1) {
        fetch(l1, t + 1);
        e = codes(t + 1);
      }
      compute(l0, d);
      if (t + 1 >= s1) break;
      __syncthreads();
      if (t + 2 < s1) {
        fetch(l0, t + 2);
        d = codes(t + 2);
      }
      compute(l1, e);
    }
  }
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      const int o = n0 + (wc * FN + j) * 32 + lr;
      const long long t0 = m0 + wr * (BM / WR) + 32 * i + 4 * lg;
      if (o < L.m) {
        if (partial) {
          float* p = partial + blockIdx.y * (L.tokens * L.m) + o;
#pragma unroll
          for (int e = 0; e < 16; ++e)
            if (t0 + 8 * (e >> 2) + (e & 3) < L.tokens) p[(t0 + 8 * (e >> 2) + (e & 3)) * L.m] = acc[i][j][e];
        } else {
#pragma unroll
          for (int e = 0; e < 16; ++e)
            if (t0 + 8 * (e >> 2) + (e & 3) < L.tokens)
              put_scale(L.Y, L.y_type, (t0 + 8 * (e >> 2) + (e & 3)) * L.ldy + o, acc[i][j][e]);
        }
      }
    }
}

// the parts of a row length added in their order
static __global__ void __launch_bounds__(256) grouped_join_kernel(const float* __restrict__ partial, int parts, long long size, int m,
                                                                  void* Y, int y_type, long long ldy) {
  const long long x = (long long)blockIdx.x * 256 + threadIdx.x;
  if (x >= size) return;
  float v = 0.0f;
  for (int p = 0; p < parts; ++p) v += partial[p * size + x];
  const long long t = x / m;
  put_scale(Y, y_type, t * ldy + (x - t * m), v);
}

struct GroupedPlan {
  bool few, small;   // the kernel for few tokens; tiles of fewer tokens
  int np, parts, sper;
  long long padded;
  size_t sums, partial, bytes;  // offsets in the workspace, and its size
};
constexpr long long kGroupedRun = 1 << 16;  // tokens of one run

template <typename XT>
static GroupedPlan grouped_plan(long long tokens, int n, int m, int group) {
  constexpr int NP = Pieces<XT>::count;
  GroupedPlan P{};
  P.few = tokens <= 64;
  if (P.few) return P;
  if (tokens > kGroupedRun) tokens = kGroupedRun;
  P.np = (n + 127) / 128 * 128;
  P.padded = (tokens + 255) / 256 * 256;
  P.small = NP == 1 && tokens <= 128;
  const int bm = NP == 3 ? 64 : P.small ? 128 : 256, bn = P.small ? 64 : 128;
  const long long tiles = (tokens + bm - 1) / bm * ((m + bn - 1ll) / bn);
  const int stages = P.np / 128;
  long long parts = 512 / tiles;
  if (parts > stages / 2) parts = stages / 2;
  if (parts < 1) parts = 1;
  P.sper = (int)((stages + parts - 1) / parts);
  P.parts = (stages + P.sper - 1) / P.sper;
  auto al = [](size_t x) { return (x + 1023) / 1024 * 1024; };
  P.sums = al((size_t)NP * P.padded * P.np * 2);
  P.partial = P.sums + al((size_t)(P.np / group) * P.padded * 4);
  P.bytes = P.partial + (P.parts > 1 ? al((size_t)P.parts * tokens * m * 4) : 0);
  return P;
}
template <typename XT>
static size_t grouped_bytes(long long tokens, int n, int m, int group) {
  return grouped_plan<XT>(tokens, n, m, group).bytes;
}

template <typename XT, int GROUP, int SB>
static hipError_t grouped_tiles(const GroupedLaunch& all, hipStream_t st) {
  GroupedLaunch L = all;
  for (long long t = 0; t < all.tokens; t += kGroupedRun) {
    L.tokens = all.tokens - t < kGroupedRun ? all.tokens - t : kGroupedRun;
    L.X = static_cast<const XT*>(all.X) + t * L.ldx;
    L.Y = static_cast<char*>(all.Y) + t * L.ldy * (L.y_type == 0 ? 4 : 2);
    const GroupedPlan P = grouped_plan<XT>(L.tokens < 65 ? 65 : L.tokens, L.n, L.m, GROUP);
    char* ws = static_cast<char*>(L.ws);
    float* sums = reinterpret_cast<float*>(ws + P.sums);
    float* partial = P.parts > 1 ? reinterpret_cast<float*>(ws + P.partial) : nullptr;
    const long long threads = L.tokens * (P.np / 8);
    hipLaunchKernelGGL((grouped_tokens_kernel<XT, GROUP>), dim3((unsigned)((threads + 255) / 256)), dim3(256), 0, st,
                       static_cast<const XT*>(L.X), L.ldx, L.tokens, L.n, P.np, P.padded, reinterpret_cast<iv4*>(ws), sums);
    const GroupedX X{ws, sums, P.padded, P.np, P.np / GROUP};
    auto go = [&](auto kernel, int bm, int bn, int threads) {
      const long long ntm = (L.tokens + bm - 1) / bm, ntn = (L.m + bn - 1ll) / bn;
      hipLaunchKernelGGL(kernel, dim3((unsigned)(ntm * ntn), (unsigned)P.parts), dim3(threads), 0, st, L, X, (int)ntm, (int)ntn, P.sper,
                         partial);
    };
    if constexpr (Pieces<XT>::count == 3) {
      go(grouped_tile_kernel<XT, 64, 2, 2, 2, GROUP, SB>, 64, 128, 256);
    } else {
      if (P.small) go(grouped_tile_kernel<XT, 128, 2, 2, 1, GROUP, SB>, 128, 64, 256);
      else go(grouped_tile_kernel<XT, 256, 4, 2, 2, GROUP, SB>, 256, 128, 512);
    }
    if (partial) {
      const long long size = L.tokens * L.m;
      hipLaunchKernelGGL(grouped_join_kernel, dim3((unsigned)((size + 255) / 256)), dim3(256), 0, st, partial, P.parts, size, L.m, L.Y,
                         L.y_type, L.ldy);
    }
  }
  return hipGetLastError();
}

template <typename XT, int GROUP, int SB>
static hipError_t grouped_sized(const GroupedLaunch& L, hipStream_t st) {
  if (!grouped_plan<XT>(L.tokens, L.n, L.m, GROUP).few) return grouped_tiles<XT, GROUP, SB>(L, st);
  const bool wide = L.m >= 6144;  // 32 channels a workgroup still fill the card
  if (L.tokens <= 16) return wide ? few_launch<XT, 1, 2, GROUP, SB>(L, st) : few_launch<XT, 1, 1, GROUP, SB>(L, st);
  if (L.tokens <= 32) return wide ? few_launch<XT, 2, 2, GROUP, SB>(L, st) : few_launch<XT, 2, 1, GROUP, SB>(L, st);
  return wide ? few_launch<XT, 4, 2, GROUP, SB>(L, st) : few_launch<XT, 4, 1, GROUP, SB>(L, st);
}

template <typename XT>
static hipError_t grouped_typed(const GroupedLaunch& L, hipStream_t st) {
  switch (L.group) {
    case 32: return L.s_type == 0 ? grouped_sized<XT, 32, 4>(L, st) : grouped_sized<XT, 32, 2>(L, st);
    case 64: return L.s_type == 0 ? grouped_sized<XT, 64, 4>(L, st) : grouped_sized<XT, 64, 2>(L, st);
    default: return L.s_type == 0 ? grouped_sized<XT, 128, 4>(L, st) : grouped_sized<XT, 128, 2>(L, st);
  }
}

}  // namespace externd
