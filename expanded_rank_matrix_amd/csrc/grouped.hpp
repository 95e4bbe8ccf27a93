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
__device__ __forceinline__ float get_scale(const void* p, int type, long long at) {
  if (type == 0) return static_cast<const float*>(p)[at];
  if (type == 1) return (float)static_cast<const _Float16*>(p)[at];
  return (float)static_cast<const __bf16*>(p)[at];
}

template <typename T>
__device__ __forceinline__ void put(T* p, float v) {
  *p = (T)v;
}

// A code enters the matrix cores as the number c + 8: its four bits, the sign turned, are an e4m3 number of 2^-9 (c + 8) as
// they are (the smallest exponents of e4m3 are one straight line), and one conversion widens two of them.  So eight
// codes cost nine instructions, and for each group
//   y += s sum (c + 8) x + (o / 8 - s) sum 8 x
// with sum 8 x from the same x by products with eights (8 s would leave fp32 for the largest scales).  The excess costs the
// sums one to two of fp32's bits.
template <typename T>
__device__ __forceinline__ iv4 widen_pairs(unsigned a, unsigned b) {  // four bytes each
  iv4 r;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const unsigned p = i == 0 ? a : b;
    if constexpr (__is_same(T, _Float16)) {
      r[2 * i] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(p, 512.0f, false));
      r[2 * i + 1] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(p, 512.0f, true));
    } else {
      r[2 * i] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(p, 512.0f, false));
      r[2 * i + 1] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(p, 512.0f, true));
    }
  }
  return r;
}
template <typename T>
__device__ __forceinline__ iv4 widen(unsigned w) {  // eight codes, signs turned, in their order
  const unsigned even = w & 0x0F0F0F0Fu, odd = (w >> 4) & 0x0F0F0F0Fu;
  return widen_pairs<T>(__builtin_amdgcn_perm(odd, even, 0x05010400u), __builtin_amdgcn_perm(odd, even, 0x07030602u));
}
// the even ones, then the odd: two instructions fewer, where the tokens are laid out the same
template <typename T>
__device__ __forceinline__ iv4 widen_apart(unsigned w) {
  return widen_pairs<T>(w & 0x0F0F0F0Fu, (w >> 4) & 0x0F0F0F0Fu);
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

constexpr int kGroupedWaves = 8;  // 2560 x 2560, one token: 4.1 us; 2560 x 9728, sixteen: 11.7 (1.1 TB/s of codes)

template <typename XT, int NT, int CT, int GROUP, int SB>
__global__ void __launch_bounds__(64 * kGroupedWaves) grouped_few_kernel(GroupedLaunch L) {
  using T = typename Pieces<XT>::type;
  constexpr int NP = Pieces<XT>::count, G = 128 / GROUP;
  // chunks whose loads are in flight together, the tokens' among them where those fit the registers
  constexpr int U = NT == 1 && sizeof(XT) == 2 ? 3 : 2;
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
  const int eight = __is_same(T, _Float16) ? 0x48004800 : 0x41004100;
  const iv4 eights = {eight, eight, eight, eight};
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
      const float sv = scale_value<SB>(d.s[i], half), bv = fmaf(0.125f, scale_value<SB>(d.o[i], half), -sv);
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
            sum[t] = gmul(T{}, p[h], eights, sum[t]);
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
  // runs of tokens whose threads a launch holds
  const long long wide = (all.m + 16ll * CT - 1) / (16 * CT), most = (1ll << 22) / wide;
  const long long step = (most < 1 ? 1 : most < 65535 ? most : 65535) * 16 * NT;
  for (long long t = 0; t < all.tokens; t += step) {
    L.tokens = all.tokens - t < step ? all.tokens - t : step;
    L.X = static_cast<const XT*>(all.X) + t * L.ldx;
    L.Y = static_cast<char*>(all.Y) + t * L.ldy * (L.y_type == 0 ? 4 : 2);
    hipLaunchKernelGGL((grouped_few_kernel<XT, NT, CT, GROUP, SB>), dim3((unsigned)wide, (unsigned)((L.tokens + 16 * NT - 1) / (16 * NT))),
                       dim3(64 * kGroupedWaves), 0, st, L);
  }
  return hipGetLastError();
}


// ---- many tokens --------------------------------------------------------------------------------------
// The tokens are laid out first: aligned rows of whole chunks of 128, fp32 as three planes of pieces, zeros behind a
// row's end, and beside them -8 times each group's sum; and the scales in fp32, a group's channels together.  So the tiles
// need no other path for odd sizes, addresses or types, and a group's partial sum starts from the excess it has to lose:
//   part = -8 sum x + sum (c + 8) x,   y += s part + o sum x
struct GroupedX {
  const void* x;        // [plane][padded][np]
  const float* sums;    // [group][padded]
  const float* scale;   // [group][channels]; groups behind the row's last are 0
  const float* offset;  // the same, or null
  long long padded;
  int np, channels;     // channels: m up to a multiple of 128
};

template <typename XT, int GROUP>
__global__ void __launch_bounds__(256) grouped_tokens_kernel(GroupedLaunch A, GroupedX P, unsigned token_blocks, iv4* __restrict__ out,
                                                             float* __restrict__ sums, float* __restrict__ scale,
                                                             float* __restrict__ offset) {
  constexpr int NP = Pieces<XT>::count, L = GROUP / 8;
  const XT* X = static_cast<const XT*>(A.X);
  const long long ldx = A.ldx, tokens = A.tokens, padded = P.padded;
  const int n = A.n, np = P.np;
  if (blockIdx.x >= token_blocks) {
    const int groups = (n + GROUP - 1) / GROUP;
    const long long i = (long long)(blockIdx.x - token_blocks) * 256 + threadIdx.x;
    if (i >= (long long)P.channels * (np / GROUP)) return;
    const int g = (int)(i / P.channels), ch = (int)(i - (long long)g * P.channels);
    const bool in = ch < A.m && g < groups;
    const long long at = (long long)ch * groups + g;
    scale[i] = in ? get_scale(A.scale, A.s_type, at) : 0.0f;
    if (offset) offset[i] = in ? -0.125f * get_scale(A.offset, A.s_type, at) : 0.0f;
    return;
  }
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
  float u[8];  // the even ones, then the odd, as the codes are widened
#pragma unroll
  for (int e = 0; e < 8; ++e) u[e] = v[e < 4 ? 2 * e : 2 * e - 7];
  if constexpr (NP == 3) {
    pieces8(u, p);
  } else {
    typedef XT v8 __attribute__((ext_vector_type(8)));
    v8 o;
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = (XT)u[e];  // as it was
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
struct Even {
  static constexpr bool value = true;
};
struct Odd {
  static constexpr bool value = false;
};
// Scheduling groups that spread a step's reads of LDS and vector work evenly over its products.
template <int READS, int MULS, int VEC>
__device__ __forceinline__ void interleave3() {
  if constexpr (MULS > 0) {
    constexpr int r = (READS + MULS - 1) / MULS, v = (VEC + MULS - 1) / MULS;
    if constexpr (r > 0) __builtin_amdgcn_sched_group_barrier(0x100, r, 0);
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    if constexpr (v > 0) __builtin_amdgcn_sched_group_barrier(0x002, v, 0);
    interleave3<READS - r, MULS - 1, VEC - v>();
  }
}
__device__ __forceinline__ fv16 gmul32(__bf16, iv4 a, iv4 b, fv16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf8, a), __builtin_bit_cast(bf8, b), c, 0, 0, 0);
}
__device__ __forceinline__ fv16 gmul32(_Float16, iv4 a, iv4 b, fv16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(hf8, a), __builtin_bit_cast(hf8, b), c, 0, 0, 0);
}

// A buffer and a direct load from it into LDS: 16 or 4 bytes a lane, from `at` (per lane) + `base` on, to `l` + the lane's
// place.  In assembly, since the compiler would wait for every load on its way before it reads LDS; the kernel's own
// waits see to it.  Its scalar operands are uniform by construction, written by scalar instructions (which need no wait
// before a load but m0's one).
struct Buffer {
  iv4 r;
  __device__ __forceinline__ explicit Buffer(const void* p) {
    const unsigned long long a = reinterpret_cast<unsigned long long>(p);
    r = iv4{(int)a, (int)(a >> 32) & 0xFFFF, -1, 0x00027000};
  }
  template <int BYTES>
  __device__ __forceinline__ void to_lds(int8_t* l, unsigned at, unsigned base) const {
    const unsigned m = lds_address(l);
    if constexpr (BYTES == 16)
      asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds" ::"s"(m), "v"(at), "s"(r), "s"(base) : "memory", "m0");
    else
      asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, %3 offen lds" ::"s"(m), "v"(at), "s"(r), "s"(base) : "memory", "m0");
  }
};

// Workgroup: BM tokens and 32 FN WC channels, WR waves down and WC across, two workgroups a CU, whose barriers leave each
// other's waves alone.  Tokens, codes, group sums and scales go through LDS in stages of 64 elements of a row, NB in turn,
// all by direct loads, so that NB - 1 stages are on their way while one is used.
//   tokens: row r is 128 bytes, its 16-byte piece c at c ^ r / 2 % 8 (16 rows' pieces of one column in different banks)
//   codes:  loaded a word a lane, so that any order costs nothing: a channel's eight words lie as the wave's halves take
//           them, 0 2 4 6 and 1 3 5 7
// Every wave widens its own fragments of codes (the waves down the tile repeat that: vector work under the others'
// products), one step ahead of the products that take them, and the barrier that hands a stage over comes before
// the last of its four steps.
// Measured (2048 x 2560 x 9728, groups of 128): 120 us; per wave and stage 16 products (512 cycles) beside about 130 vector
// instructions, of which 56 widen and 32 scale.  128 x 128 and two stages two workgroups a CU; 256 x 128 in one workgroup
// took 170 us with four waves and 177 with eight.
// MFMA D(32 x 32) += A(32 x 16) B(16 x 32): A row = token l % 32, B column = channel l % 32, both with the eight
// elements at 8 (l / 32) of the step.
template <typename XT, int BM, int WR, int WC, int FN, int NB, int GROUP>
__device__ __forceinline__ void grouped_tile(const GroupedLaunch& L, const GroupedX& X, int ntn, int whole, int parts, int sper,
                                             float* __restrict__ partial) {
  using T = typename Pieces<XT>::type;
  constexpr int NP = Pieces<XT>::count, FM = BM / WR / 32, NW = WR * WC, BN = 32 * FN * WC;
  constexpr int G = GROUP == 32 ? 2 : 1;               // groups of a stage (two stages to one of 128)
  constexpr int kRows = NP * BM, PL = kRows / 8 / NW;  // direct loads of a wave and stage: eight rows each
  constexpr int CL = BN / 8 / NW;                      // of codes: eight channels each
  constexpr int kSums = (G * BM * 4 + 1023) / 1024;    // of group sums, in all
  static_assert(PL * 8 * NW == kRows && CL * 8 * NW == BN && FM * 32 * WR == BM && kSums + 2 <= NW && PL % NP == 0, "tile shape");
  static_assert(G * BN * 4 <= 1024, "scales of a stage");
  constexpr int kCodes = kRows * 128, kSum = kCodes + BN * 32, kScale = kSum + kSums * 1024, kOffset = kScale + 1024;
  constexpr int kStage = kOffset + 1024;
  __shared__ __attribute__((aligned(1024))) int8_t lds[NB * kStage];
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wr = wv / WC, wc = wv % WC, lr = lane & 31, lg = lane >> 5;
  // The first `whole` tiles are each one workgroup's; the others' row lengths are cut into parts.  Workgroups go round the eight
  // XCDs: each gets a run of neighbouring tiles, the channels of one run of tokens after each other, so that its L2 holds
  // those tokens.
  const int stages = X.np / 64;
  int tile, s0 = 0, s1 = stages;
  long long place = -1;  // of the part's tile
  if ((int)blockIdx.x < whole) {
    tile = blockIdx.x % 8 * (whole / 8) + blockIdx.x / 8;  // whole is a multiple of 8
  } else {
    const int x = blockIdx.x - whole;
    tile = whole + x / parts;
    s0 = x % parts * sper;
    s1 = s0 + sper < stages ? s0 + sper : stages;
    if (parts > 1) place = x;
  }
  const long long m0 = (long long)(tile / ntn) * BM;
  const int n0 = tile % ntn * BN;
  const int groups = (L.n + GROUP - 1) / GROUP, words = groups * (GROUP / 8);
  const bool offsets = X.offset != nullptr;
  // Buffer loads: a lane keeps one offset a load, and what changes with the stage is a scalar.  Every offset stays inside
  // what it is given.
  const unsigned pitch = (unsigned)X.np * 2, ldq4 = (unsigned)(L.ldq * 4);  // the latter at most kGroupedPitch
  unsigned xo[PL / NP];  // this lane's piece of each of the wave's loads of a plane, from the tile's first token
#pragma unroll
  for (int p = 0; p < PL / NP; ++p) {
    const int r = (p * NW + wv) * 8 + (lane >> 3);
    const long long t = m0 + r < L.tokens ? r : L.tokens - 1 - m0;
    xo[p] = (unsigned)t * pitch + (((lane & 7) ^ ((r >> 1) & 7)) << 4);
  }
  const int word = (lane & 3) * 2 + ((lane >> 2) & 1);  // of the channel's eight, as above
  const int8_t* xb = static_cast<const int8_t*>(X.x) + m0 * pitch;
  const int* qb = L.Q + (long long)n0 * L.ldq;
  unsigned co[CL];
#pragma unroll
  for (int p = 0; p < CL; ++p) {
    const int o = (p * NW + wv) * 8 + (lane >> 3);
    co[p] = (unsigned)(n0 + o < L.m ? o : L.m - 1 - n0) * ldq4;
  }
  const Buffer bq(qb), bsum(X.sums + m0), bs(X.scale + n0), bo((offsets ? X.offset : X.scale) + n0);
  // group sums [group][BM], 256 of them a load (behind the last they repeat it), and scales and offsets [group][BN] likewise
  const int es = wv * 256 + lane * 4, ec = lane * 4;
  const unsigned so = (unsigned)(es / BM < G ? es / BM : G - 1) * (unsigned)X.padded * 4 + es % BM * 4;
  const unsigned cs = (unsigned)(ec / BN < G ? ec / BN : G - 1) * (unsigned)X.channels * 4 + ec % BN * 4;
  auto fetch = [&](int8_t* l, int t) {
#pragma unroll
    for (int h = 0; h < NP; ++h) {
      const Buffer bx(xb + h * X.padded * pitch);
#pragma unroll
      for (int p = 0; p < PL / NP; ++p) bx.to_lds<16>(l + ((h * (PL / NP) + p) * NW + wv) * 1024, xo[p], t * 128);
    }
    const int left = words - 8 * t;  // codes behind the row's end are its last word, and meet zeros
    const unsigned at = (unsigned)(word < left ? 8 * t + word : words - 1) * 4;
#pragma unroll
    for (int p = 0; p < CL; ++p) bq.to_lds<4>(l + kCodes + (p * NW + wv) * 256, co[p] + at, 0);
    const unsigned g0 = (unsigned)t * 64 / GROUP * 4;
    if (wv < kSums) bsum.to_lds<16>(l + kSum + wv * 1024, so, g0 * (unsigned)X.padded);
    else if (wv == kSums) bs.to_lds<16>(l + kScale, cs, g0 * (unsigned)X.channels);
    else if (wv == kSums + 1) bo.to_lds<16>(l + kOffset, cs, g0 * (unsigned)X.channels);
    __builtin_amdgcn_sched_barrier(0);
  };
  constexpr int kLeast = PL + CL;  // direct loads that every wave issues for a stage
  // The next stage is in LDS: of this wave's loads at most those of the NB - 2 stages behind it are on their way.  The
  // reads of this one are done, so that its place may be filled.
  auto handover = [&]() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"((NB - 2) * kLeast) : "memory");
  };
  fv16 acc[FM][FN], part[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;
  const int row = wr * (BM / WR) + lr, zx = (row >> 1) & 7;  // rows r + 32 f share r / 2 % 8
  iv4 w[2][FN];  // a stage's codes of this lane: the words of its half
  iv4 fa[2][NP * FM], fb[2][FN];
  float s[FN];
  auto take = [&](int b, const int8_t* l) {
#pragma unroll
    for (int j = 0; j < FN; ++j)
      w[b][j] = *reinterpret_cast<const iv4*>(l + kCodes + ((wc * FN + j) * 32 + lr) * 32 + lg * 16) ^ (int)kSignTurn;
  };
  auto read = [&](int f, const int8_t* l, int b, int k) {  // fragments of step k
#pragma unroll
    for (int h = 0; h < NP; ++h)
#pragma unroll
      for (int i = 0; i < FM; ++i)
        fa[f][h * FM + i] = *reinterpret_cast<const iv4*>(l + (h * BM + row + 32 * i) * 128 + (((2 * k + lg) ^ zx) << 4));
#pragma unroll
    for (int j = 0; j < FN; ++j) fb[f][j] = widen_apart<T>((unsigned)w[b][j][k]);
  };
  auto begin = [&](const int8_t* l, int g) {  // a group: its sums start from the excess
    const float* sums = reinterpret_cast<const float*>(l + kSum) + g * BM + wr * (BM / WR) + 4 * lg;
    const float* sc = reinterpret_cast<const float*>(l + kScale) + g * BN + wc * FN * 32 + lr;
    const float* of = reinterpret_cast<const float*>(l + kOffset) + g * BN + wc * FN * 32 + lr;
#pragma unroll
    for (int j = 0; j < FN; ++j) s[j] = sc[32 * j];
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      fv16 lose;
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const fv4 u = *reinterpret_cast<const fv4*>(sums + 32 * i + 8 * x);
#pragma unroll
        for (int e = 0; e < 4; ++e) lose[4 * x + e] = u[e];
      }
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        part[i][j] = lose;
        if (offsets) {
          const float o = of[32 * j];
#pragma unroll
          for (int e = 0; e < 16; ++e) acc[i][j][e] = fmaf(o, lose[e], acc[i][j][e]);
        }
      }
    }
  };
  auto end = [&]() {
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[i][j][e] = fmaf(s[j], part[i][j][e], acc[i][j][e]);
  };
  // stage t in l, its codes in w[b] and first fragments read; ln is the next one's place.  EVEN: t is.
  auto stage = [&](int t, int8_t* l, int8_t* ln, auto even) {
    constexpr bool EVEN = decltype(even)::value;
    constexpr int b = EVEN ? 0 : 1;
    if (GROUP != 128 || EVEN) begin(l, 0);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (GROUP == 32 && k == 2) {
        end();
        begin(l, 1);
      }
      if (k < 3) {
        read((k + 1) & 1, l, b, k + 1);
      } else {
        // behind the last stage it is loaded again, and read by no product: every path waits for the same number
        handover();
        fetch(l, t + NB < s1 ? t + NB : s1 - 1);
        take(b ^ 1, ln);
        read(0, ln, b ^ 1, 0);
      }
#pragma unroll
      for (int h = 0; h < NP; ++h)
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
          for (int j = 0; j < FN; ++j) part[i][j] = gmul32(T{}, fa[k & 1][h * FM + i], fb[k & 1][j], part[i][j]);
      interleave3<NP * FM, NP * FM * FN, 7 * FN>();
      __builtin_amdgcn_sched_barrier(0);
    }
    if (GROUP != 128 || !EVEN) end();
  };
  if (s0 < s1) {  // s0 and s1 are even
#pragma unroll
    for (int i = 0; i < NB; ++i) fetch(lds + i * kStage, s0 + i < s1 ? s0 + i : s1 - 1);
    asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"((NB - 1) * kLeast) : "memory");
    take(0, lds);
    read(0, lds, 0, 0);
    int at = 0;  // of the stage's place
    auto next = [](int a) { return a == (NB - 1) * kStage ? 0 : a + kStage; };
    for (int t = s0; t < s1; t += 2) {
      const int n1 = next(at), n2 = next(n1);
      stage(t, lds + at, lds + n1, Even{});
      stage(t + 1, lds + n1, lds + n2, Odd{});
      at = n2;
    }
    stage_barrier();  // no load is on its way into LDS when the workgroup ends
  }
  if (place >= 0) {
    float* p = partial + place * (BM * BN) + (wr * (BM / WR) + 4 * lg) * BN + wc * FN * 32 + lr;
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int e = 0; e < 16; ++e) p[(32 * i + 8 * (e >> 2) + (e & 3)) * BN + 32 * j] = acc[i][j][e];
    return;
  }
  auto store = [&](auto* y) {
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        const int o = n0 + (wc * FN + j) * 32 + lr;
        const long long t0 = m0 + wr * (BM / WR) + 32 * i + 4 * lg;
        if (o < L.m) {
#pragma unroll
          for (int e = 0; e < 16; ++e)
            if (t0 + 8 * (e >> 2) + (e & 3) < L.tokens) put(y + (t0 + 8 * (e >> 2) + (e & 3)) * L.ldy + o, acc[i][j][e]);
        }
      }
  };
  if (L.y_type == 0) store(static_cast<float*>(L.Y));
  else if (L.y_type == 1) store(static_cast<_Float16*>(L.Y));
  else store(static_cast<__bf16*>(L.Y));
}

template <typename XT, int BM, int WR, int WC, int FN, int NB, int GROUP>
__global__ void __launch_bounds__(64 * WR * WC, 2) grouped_tile_kernel(GroupedLaunch L, GroupedX X, int ntn, int whole, int parts,
                                                                       int sper, float* __restrict__ partial) {
  grouped_tile<XT, BM, WR, WC, FN, NB, GROUP>(L, X, ntn, whole, parts, sper, partial);
}

// The parts of the tiles behind the whole ones added in their order; a thread adds four channels.
template <int BM, int BN>
__global__ void __launch_bounds__(256) grouped_join_kernel(GroupedLaunch L, int ntn, int whole, int parts, const float* __restrict__ partial) {
  const int x = blockIdx.y * 1024 + threadIdx.x * 4, tile = whole + blockIdx.x;
  const long long t = (long long)(tile / ntn) * BM + x / BN;
  const int o = tile % ntn * BN + x % BN;
  if (t >= L.tokens || o >= L.m) return;
  const float* p = partial + (long long)blockIdx.x * parts * (BM * BN) + x;
  fv4 v = {0, 0, 0, 0};
  for (int i = 0; i < parts; ++i) v += *reinterpret_cast<const fv4*>(p + (long long)i * (BM * BN));
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (o + e < L.m) put_scale(L.Y, L.y_type, t * L.ldy + o + e, v[e]);
}

struct GroupedPlan {
  bool few, small;  // the kernel for few tokens; tiles of fewer channels
  int np, channels;
  int bm, bn, ntn, whole, rest, parts, sper;  // tiles whole and in parts, and stages of 64 elements of a part
  long long padded;
  size_t sums, scale, offset, partial, bytes;  // offsets in the workspace, and its size
};
constexpr long long kGroupedRun = 1 << 14;    // tokens of one run, so that the group sums' offsets fit 32 bits

template <typename XT>
static GroupedPlan grouped_plan(long long tokens, int n, int m, int group) {
  constexpr int NP = Pieces<XT>::count;
  GroupedPlan P{};
  // Few: up to 64 tokens of 16 bits, 32 of fp32, whose three pieces the kernel for few tokens makes again for each 16 or 32
  // channels.  Measured, few / tiles, us (n x m, groups of 128): bf16 2560 x 2560, 64 tokens 12.6 / 17.6, 65 15.7 / 17.6;
  // 2560 x 9728, 48 23.2 / 22.4, 65 26.0 / 23.1; 9728 x 2560, 32 21.8 / 25.6, 64 38.4 / 27.1; fp32 2560 x 2560, 32 12.8 /
  // 16.0, 48 19.4 / 17.1; 2560 x 9728, 32 24.2 / 23.5, 48 39.8 / 24.7; 9728 x 2560, 16 22.4 / 27.5, 32 39.1 / 30.0, 64 74.4 /
  // 31.3; 1021 x 2051, 48 9.2 / 13.3.  Over 118 sizes, 12 to 160 tokens, that costs 5 to 6% over the better of the two, the
  // worst on the longest rows.  Matrices whose offsets in a tile, or number of tiles, pass 32 bits take the kernel for few
  // tokens, whatever their number.
  const long long scales = (n + 127ll) / 128 * 128 / group * ((m + 127ll) / 128 * 128) * 4;
  P.few = tokens <= (NP == 3 ? 32 : 64) || scales >= 1ll << 32 || m > 1 << 22;
  if (P.few) return P;
  P.np = (n + 127) / 128 * 128;
  P.padded = (tokens + 255) / 256 * 256;
  P.small = NP == 1 && tokens <= 128;
  P.bm = NP == 3 ? 64 : 128;
  P.bn = P.small ? 64 : 128;
  P.ntn = (int)((m + P.bn - 1ll) / P.bn);
  const long long tiles = (tokens + P.bm - 1) / P.bm * P.ntn;
  // 512 workgroups run at a time.  Tiles behind the last whole round are cut along the row, into as many parts as fill
  // it, of at least two chunks of 128 elements each.
  const int chunks = P.np / 128;
  P.whole = (int)(tiles / 512 * 512);
  P.rest = (int)(tiles - P.whole);
  long long parts = P.rest ? 512 / P.rest : 1;
  if (parts > chunks / 2) parts = chunks / 2;
  if (parts < 1) parts = 1;
  const int each = (int)((chunks + parts - 1) / parts);
  P.sper = 2 * each;
  P.parts = (chunks + each - 1) / each;
  auto al = [](size_t x) { return (x + 1023) / 1024 * 1024; };
  P.sums = al((size_t)NP * P.padded * P.np * 2);
  P.channels = (m + 127) / 128 * 128;
  const size_t s = al((size_t)(P.np / group) * P.channels * 4);
  P.scale = P.sums + al((size_t)(P.np / group) * P.padded * 4);
  P.offset = P.scale + s;
  P.partial = P.offset + s;
  P.bytes = P.partial + (P.parts > 1 ? al((size_t)P.parts * P.rest * P.bm * P.bn * 4) : 0);
  return P;
}
template <typename XT>
static size_t grouped_bytes(long long tokens, int n, int m, int group) {
  const long long last = tokens % kGroupedRun;
  size_t a = grouped_plan<XT>(tokens < kGroupedRun ? tokens : kGroupedRun, n, m, group).bytes;
  const size_t b = tokens > kGroupedRun && last ? grouped_plan<XT>(last, n, m, group).bytes : 0;
  return a > b ? a : b;
}

// one run of tokens
template <typename XT, int GROUP>
static hipError_t grouped_tiles(const GroupedLaunch& L, const GroupedPlan& P, hipStream_t st) {
  char* ws = static_cast<char*>(L.ws);
  float* sums = reinterpret_cast<float*>(ws + P.sums);
  float* partial = P.parts > 1 ? reinterpret_cast<float*>(ws + P.partial) : nullptr;
  float* scale = reinterpret_cast<float*>(ws + P.scale);
  float* offset = L.offset ? reinterpret_cast<float*>(ws + P.offset) : nullptr;
  const GroupedX X{ws, sums, scale, offset, P.padded, P.np, P.channels};
  const unsigned tb = (unsigned)((L.tokens * (P.np / 8) + 255) / 256), sb = (unsigned)(((long long)P.channels * (P.np / GROUP) + 255) / 256);
  hipLaunchKernelGGL((grouped_tokens_kernel<XT, GROUP>), dim3(tb + sb), dim3(256), 0, st, L, X, tb, reinterpret_cast<iv4*>(ws), sums,
                     scale, offset);
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3((unsigned)(P.whole + P.rest * P.parts)), dim3(256), 0, st, L, X, P.ntn, P.whole, P.parts, P.sper, partial);
  };
  auto join = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3((unsigned)P.rest, (unsigned)(P.bm * P.bn / 1024)), dim3(256), 0, st, L, P.ntn, P.whole, P.parts, partial);
  };
  if constexpr (Pieces<XT>::count == 3) {
    go(grouped_tile_kernel<XT, 64, 2, 2, 2, 2, GROUP>);
    if (partial) join(grouped_join_kernel<64, 128>);
  } else if (P.small) {
    go(grouped_tile_kernel<XT, 128, 2, 2, 1, 3, GROUP>);
    if (partial) join(grouped_join_kernel<128, 64>);
  } else {
    go(grouped_tile_kernel<XT, 128, 2, 2, 2, 2, GROUP>);
    if (partial) join(grouped_join_kernel<128, 128>);
  }
  return hipGetLastError();
}

template <typename XT, int GROUP, int SB>
static hipError_t grouped_few(const GroupedLaunch& L, hipStream_t st) {
  // 32 channels a workgroup read the tokens half as often, but make half as many workgroups: taken where the busiest of the
  // 256 CUs has fewer of them by more than each costs more.  Measured, 16 / 32 channels, us (n x m, groups of 128): 2560 x
  // 2560, 1 token 4.3 / 5.4, 64 12.9 / 14.0; 2560 x 5120, 1 5.7 / 5.5, 64 22.6 / 14.1; 2560 x 9728, 1 7.2 / 8.7, 8 10.1 /
  // 10.4, 16 12.9 / 12.3, 64 31.9 / 26.3; 9728 x 5120, 1 14.0 / 12.2, 64 75 / 45; 9728 x 16384, 8 37 / 30; 2560 x 16400, 1
  // 9.9 / 11.5, 16 19.7 / 16.6.  (Sixteen waves instead of eight: 9728 x 2560, 1 token 8.4 against 8.0, 16 16.0 against
  // 14.6.)
  const long long narrow = (L.m + 4095ll) / 4096, half = (L.m + 8191ll) / 8192;  // workgroups of the busiest CU
  const bool wide = L.tokens > 8 ? narrow > half : 4 * narrow > 7 * half;
  if (L.tokens <= 16) return wide ? few_launch<XT, 1, 2, GROUP, SB>(L, st) : few_launch<XT, 1, 1, GROUP, SB>(L, st);
  if (L.tokens <= 32) return wide ? few_launch<XT, 2, 2, GROUP, SB>(L, st) : few_launch<XT, 2, 1, GROUP, SB>(L, st);
  return wide ? few_launch<XT, 4, 2, GROUP, SB>(L, st) : few_launch<XT, 4, 1, GROUP, SB>(L, st);
}

template <typename XT, int GROUP, int SB>
static hipError_t grouped_sized(const GroupedLaunch& all, hipStream_t st) {
  if (all.ldq * 4 > kGroupedPitch) return grouped_few<XT, GROUP, SB>(all, st);
  GroupedLaunch L = all;
  for (long long t = 0; t < all.tokens; t += kGroupedRun) {
    L.tokens = all.tokens - t < kGroupedRun ? all.tokens - t : kGroupedRun;
    L.X = static_cast<const XT*>(all.X) + t * L.ldx;
    L.Y = static_cast<char*>(all.Y) + t * L.ldy * (L.y_type == 0 ? 4 : 2);
    const GroupedPlan P = grouped_plan<XT>(L.tokens, L.n, L.m, GROUP);
    const hipError_t e = P.few ? grouped_few<XT, GROUP, SB>(L, st) : grouped_tiles<XT, GROUP>(L, P, st);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
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
