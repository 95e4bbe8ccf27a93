// Distillation from a teacher's top logits: the loss for each row (token) and its gradient.
//
//   p = softmax of a_k / T over the row's valid entries k (0 <= index_k < V, a_k > -inf)
//   q = softmax of z_v / T over the whole vocabulary
//   loss = w T^2 sum_k p_k (log p_k - log q_index(k))
//   dz_v = w T (q_v P - sum_{k: index(k) = v} p_k),  P = 1 with a valid entry, else 0
//
// One pass over z keeps the running maximum m and the sum S of exp((z - m) / T) (8 elements a step:
// one rescaling of the sum per step at most), so q_v = exp((z_v - m) / T) / S.  z is handled in
// fp32, each thread's sum too; the threads' sums, log S and the K terms of the loss are fp64, since
// log p - log q is a difference of numbers many times its size.  The gradient is a second pass: each element
// is read once more and written once, rounded once to z's type.  The corrections p sit in LDS lists
// by groups of 8 elements; equal indices of one row add in 64-bit fixed point (units of 2^-60), so
// their order does not matter.
#include "common.hpp"
#include "externd_internal.hpp"
#include "types.hpp"

namespace externd {

constexpr int kDThreads = 256;
constexpr int kDBuckets = 8192;          // lists of groups (group % kDBuckets)
constexpr unsigned short kDNone = 0xFFFF;
constexpr unsigned long long kDNaN = ~0ull;

__device__ __forceinline__ double block_sum_f64(double v, double* red) {  // red: kDThreads / 64
  v = wave_sum_f64(v);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  double s = 0.0;
#pragma unroll
  for (int w = 0; w < kDThreads / 64; ++w) s += red[w];
  return s;
}

__device__ __forceinline__ float wave_max_f32(float v) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) v = fmaxf(v, __shfl_xor(v, d));
  return v;
}
__device__ __forceinline__ float block_max_f32(float v, float* red) {
  v = wave_max_f32(v);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kDThreads / 64; ++w) v = fmaxf(v, red[w]);
  return v;
}

struct Teacher {
  const void* a;
  const void* index;
  int a_type, index_bytes, top;
};

__device__ __forceinline__ float teacher_value(const Teacher& t, long long at) {
  if (t.a_type == 0) return static_cast<const float*>(t.a)[at];
  if (t.a_type == 1) return (float)static_cast<const _Float16*>(t.a)[at];
  return (float)static_cast<const __bf16*>(t.a)[at];
}
// the entry's index, -1 if it is none of the vocabulary's
__device__ __forceinline__ int teacher_index(const Teacher& t, long long at, int V) {
  const long long v = t.index_bytes == 8 ? static_cast<const long long*>(t.index)[at]
                                         : (long long)static_cast<const int*>(t.index)[at];
  return v >= 0 && v < V ? (int)v : -1;
}

// The row's teacher into LDS: index of every entry (-1 where there is none) and e = exp((a - max) / T)
// (0 there).  Returns 1 / sum e, so that p = e / sum e, and sum p log p; 0 where no entry is valid.
// A NaN or +inf among the valid entries makes every e NaN.
__device__ __forceinline__ double teacher_row(const Teacher& t, long long row, int V, double rT, int* idx, float* ex,
                                              float* redf, double* redd, double* plogp) {
  const long long base = row * t.top;
  float mx = -__builtin_inff();
  int nan = 0;
  for (int k = threadIdx.x; k < t.top; k += kDThreads) {
    const int i = teacher_index(t, base + k, V);
    const float a = i >= 0 ? teacher_value(t, base + k) : -__builtin_inff();
    idx[k] = a == -__builtin_inff() ? -1 : i;
    ex[k] = a;
    nan |= a != a;
    mx = fmaxf(mx, a);
  }
  nan = __syncthreads_or(nan);
  mx = block_max_f32(mx, redf);
  if (nan) mx = __builtin_nanf("");
  if (mx == -__builtin_inff()) {  // the same in every thread
    *plogp = 0.0;
    return 0.0;
  }
  double s = 0.0, sx = 0.0;  // sums of e^x and of x e^x, x = (a - max) / T
  for (int k = threadIdx.x; k < t.top; k += kDThreads) {
    float e = 0.0f;
    if (idx[k] >= 0) {
      const double x = ((double)ex[k] - (double)mx) * rT;
      e = expf((float)x);
      s += (double)e;
      if (e != 0.0f) sx += x * (double)e;
    }
    ex[k] = e;
  }
  s = block_sum_f64(s, redd);
  sx = block_sum_f64(sx, redd);
  *plogp = sx / s - log(s);
  return 1.0 / s;
}

// running maximum m and sum s of exp2((z - m) c)
__device__ __forceinline__ void stats8(const float (&z)[8], float c, float& m, float& s) {
  float cm = z[0];
#pragma unroll
  for (int e = 1; e < 8; ++e) cm = fmaxf(cm, z[e]);
  if (cm > m) {
    s *= __builtin_amdgcn_exp2f((m - cm) * c);
    m = cm;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) s += __builtin_amdgcn_exp2f((z[e] - m) * c);
}

template <typename T>
__device__ __forceinline__ void load8_inf(const T* p, long long count, float (&v)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = e < count ? (float)p[e] : -__builtin_inff();
}

// m and S over elements lo .. hi - 1 of a row, the same in every thread.  -FLT_MAX, not -inf, stands
// for no maximum yet, so that elements of -inf add exp2(-inf) = 0.
template <typename T>
__device__ __forceinline__ void slice_stats(const T* z, int lo, int hi, float c, float* redf, double* redd, float& M,
                                            double& S) {
  float m = -__FLT_MAX__, s = 0.0f;
  int j = lo + 8 * (int)threadIdx.x;
  constexpr int step = 8 * kDThreads, U = 4;
  for (; (long long)j + (U - 1) * step + 8 <= hi; j += U * step) {
    float v[U][8];
#pragma unroll
    for (int u = 0; u < U; ++u) load8(z + j + u * step, v[u]);
#pragma unroll
    for (int u = 0; u < U; ++u) stats8(v[u], c, m, s);
  }
  for (; j < hi; j += step) {
    float v[8];
    if (hi - j >= 8) load8(z + j, v);
    else load8_inf(z + j, hi - j, v);
    stats8(v, c, m, s);
  }
  M = block_max_f32(m, redf);
  // a thread without elements, or with -inf alone, has s = 0
  S = block_sum_f64(s == 0.0f ? 0.0 : (double)s * (double)__builtin_amdgcn_exp2f((m - M) * c), redd);
}

template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&v)[8]) {
  typedef T v8 __attribute__((ext_vector_type(8)));
  v8 o;
#pragma unroll
  for (int e = 0; e < 8; ++e) o[e] = (T)v[e];
  *reinterpret_cast<iv4_any*>(p) = __builtin_bit_cast(iv4, o);
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  iv4 a, b;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    a[e] = __float_as_int(v[e]);
    b[e] = __float_as_int(v[4 + e]);
  }
  *reinterpret_cast<iv4_any*>(p) = a;
  *reinterpret_cast<iv4_any*>(p + 4) = b;
}

// The lists of the gradient's corrections, by group of 8 elements.
__device__ __forceinline__ void lists_build(const int* idx, int top, unsigned* heads32, unsigned short* next) {
  for (int x = threadIdx.x; x < kDBuckets / 2; x += kDThreads) heads32[x] = 0xFFFFFFFFu;
  __syncthreads();
  for (int k = threadIdx.x; k < top; k += kDThreads)
    if (idx[k] >= 0) {
      const int b = (idx[k] >> 3) & (kDBuckets - 1), sh = 16 * (b & 1);
      unsigned old = heads32[b >> 1], seen;
      do {  // exchange of one half word
        seen = old;
        old = atomicCAS(&heads32[b >> 1], seen, (seen & ~(0xFFFFu << sh)) | (unsigned)k << sh);
      } while (old != seen);
      next[k] = (unsigned short)(seen >> sh);
    }
  __syncthreads();
}

// dz of elements lo .. hi - 1 (lo a multiple of 8): g (exp2((z - m) c) / S - p), p = e pinv
template <typename T>
__device__ __forceinline__ void slice_grad(const T* z, T* d, int lo, int hi, float c, float m, float inv, float g,
                                           const int* idx, const float* ex, double pinv, const unsigned* heads32,
                                           const unsigned short* next) {
  const unsigned short* heads = reinterpret_cast<const unsigned short*>(heads32);
  const float gi = g * inv;
  for (int j = lo + 8 * (int)threadIdx.x; j < hi; j += 8 * kDThreads) {
    float v[8], o[8];
    const bool whole = hi - j >= 8;
    if (whole) load8(z + j, v);
    else load8_inf(z + j, hi - j, v);
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = __builtin_amdgcn_exp2f((v[e] - m) * c) * gi;
    unsigned k = heads[(j >> 3) & (kDBuckets - 1)];
    if (k != kDNone) {
      unsigned long long sum[8] = {0, 0, 0, 0, 0, 0, 0, 0};
      for (; k != kDNone; k = next[k])
        if ((idx[k] >> 3) == (j >> 3)) {
          const double q = (double)ex[k] * pinv;  // all of a row's are NaN or none
          const unsigned long long u = q == q ? (unsigned long long)(q * 0x1p60) : kDNaN;
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if ((idx[k] & 7) == e) sum[e] = u == kDNaN ? kDNaN : sum[e] + u;
        }
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (sum[e]) o[e] -= sum[e] == kDNaN ? __builtin_nanf("") : g * (float)((double)sum[e] * 0x1p-60);
    }
    if (whole) {
      store8(d + j, o);
    } else {
      for (int e = 0; e < hi - j; ++e) d[j + e] = (T)o[e];
    }
  }
}

template <typename T>
__device__ __forceinline__ void slice_zero(T* d, int lo, int hi) {
  const float o[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  for (int j = lo + 8 * (int)threadIdx.x; j < hi; j += 8 * kDThreads) {
    if (hi - j >= 8) store8(d + j, o);
    else
      for (int e = 0; e < hi - j; ++e) d[j + e] = (T)0.0f;
  }
}

// sums over the teacher's entries in lo .. hi - 1 of e and of e (z - m): this thread's part.  Taken
// from m, since z itself may be near the type's lowest value throughout a row.
template <typename T>
__device__ __forceinline__ void cross_part(const T* z, int lo, int hi, const int* idx, const float* ex, int top,
                                           float m, double& mass, double& cross) {
  mass = cross = 0.0;
  for (int k = threadIdx.x; k < top; k += kDThreads)
    if (idx[k] >= lo && idx[k] < hi && ex[k] != 0.0f) {
      mass += (double)ex[k];
      cross += (double)ex[k] * ((double)(float)z[idx[k]] - (double)m);
    }
}

// a slice's share of a split row, in the workspace
struct Part {
  double s;      // sum of exp2((z - m) c)
  double mass;   // sums of e and of e (z - m) over the teacher's entries
  double cross;
  float m;
  float unused;
};

// MODE 0: statistics and loss of whole rows, and their gradient where D is given
// MODE 1: a slice's share of them (split rows, first launch)
// MODE 2: the shares joined: the first slice of a row writes statistics and loss, each its gradient
// MODE 3: gradient of a slice from given statistics
// Every thread of a workgroup takes the same branches around the barriers.
template <typename T, int MODE>
__global__ void __launch_bounds__(kDThreads) distill_kernel(const T* Z, int V, long long ldz, Teacher teach, float Tmp,
                                                            const float* __restrict__ weight, float* __restrict__ loss,
                                                            float* __restrict__ stats, T* D, long long ldd, int slices,
                                                            int slice, int gslices, Part* __restrict__ parts) {
  extern __shared__ __attribute__((aligned(16))) unsigned char lds[];
  __shared__ double redd[kDThreads / 64];
  __shared__ float redf[kDThreads / 64];
  int* idx = reinterpret_cast<int*>(lds);
  float* ex = reinterpret_cast<float*>(idx + teach.top);
  unsigned* heads = reinterpret_cast<unsigned*>(ex + teach.top);
  unsigned short* next = reinterpret_cast<unsigned short*>(heads + kDBuckets / 2);
  const long long row = blockIdx.x / gslices;
  const int sl = (int)(blockIdx.x % gslices);
  const long long lo64 = (long long)sl * slice;
  const int lo = lo64 < V ? (int)lo64 : V, hi = lo64 + slice < V ? (int)(lo64 + slice) : V;
  const T* z = Z + row * ldz;
  T* d = D + row * ldd;
  const float w = weight ? weight[row] : 1.0f;
  if (w == 0.0f) {
    if (MODE == 1) return;
    if (MODE != 3 && sl == 0 && threadIdx.x == 0) {
      loss[row] = 0.0f;
      stats[2 * row] = 0.0f;
      stats[2 * row + 1] = 0.0f;
    }
    if (D) slice_zero(d, lo, hi);
    return;
  }
  const float c = (float)(1.4426950408889634 / (double)Tmp);
  const double rT = 1.0 / (double)Tmp;
  double plogp;
  const double pinv = teacher_row(teach, row, V, rT, idx, ex, redf, redd, &plogp);
  __syncthreads();
  float m;
  double S, mass, cross = 0.0;
  if (MODE == 0 || MODE == 1) {
    slice_stats(z, lo, hi, c, redf, redd, m, S);
    cross_part(z, lo, hi, idx, ex, teach.top, m, mass, cross);
    cross = block_sum_f64(cross, redd);
    if (MODE == 1) mass = block_sum_f64(mass, redd);
  } else if (MODE == 2) {
    const Part* q = parts + row * slices;
    m = -__FLT_MAX__;
    for (int i = 0; i < slices; ++i) m = fmaxf(m, q[i].m);
    S = 0.0;
    for (int i = 0; i < slices; ++i) {
      if (q[i].s != 0.0) S += q[i].s * (double)__builtin_amdgcn_exp2f((q[i].m - m) * c);
      if (q[i].mass != 0.0) cross += q[i].cross + q[i].mass * ((double)q[i].m - (double)m);
    }
  } else {
    m = stats[2 * row];
    S = (double)stats[2 * row + 1];
  }
  if (MODE == 1) {
    if (threadIdx.x == 0) {
      Part* o = parts + row * slices + sl;
      o->m = m;
      o->s = S;
      o->mass = mass;
      o->cross = cross;
    }
    return;
  }
  if (MODE != 3 && sl == 0 && threadIdx.x == 0) {
    const double kl = plogp - cross * pinv * rT + log(S);
    loss[row] = pinv != 0.0 ? (float)((double)w * (double)Tmp * (double)Tmp * kl) : 0.0f;
    stats[2 * row] = S == 0.0 ? -__builtin_inff() : m;
    stats[2 * row + 1] = (float)S;
  }
  if (!D) return;
  if (pinv == 0.0) {  // no teacher, no gradient
    slice_zero(d, lo, hi);
    return;
  }
  lists_build(idx, teach.top, heads, next);
  slice_grad(z, d, lo, hi, c, m, (float)(1.0 / S), w * Tmp, idx, ex, pinv, heads, next);
}

// Slices of a row, so that few rows fill the card: about four workgroups a CU, none with less than
// 4096 elements.
static void split(long long rows, int V, int* slices, int* slice) {
  long long s = (1024 + rows - 1) / rows;
  const long long most = (V + 4095) / 4096;
  if (s > most) s = most;
  long long len = (V + s - 1) / s;
  len = (len + 8 * kDThreads - 1) / (8 * kDThreads) * (8 * kDThreads);
  *slice = (int)len;
  *slices = (int)((V + len - 1) / len);
}

size_t distill_workspace_bytes(long long rows, int V) {
  int slices, slice;
  if (rows == 0) return 0;
  split(rows, V, &slices, &slice);
  return slices > 1 ? (size_t)rows * slices * sizeof(Part) : 0;
}

template <typename T>
static hipError_t distill_typed(const DistillLaunch& L, hipStream_t st) {
  const Teacher t{L.teacher, L.index, L.t_type, L.index_bytes, L.top};
  const T* Z = static_cast<const T*>(L.logits);
  T* D = static_cast<T*>(L.dlogits);
  Part* parts = static_cast<Part*>(L.ws);
  int slices, slice;
  split(L.rows, L.vocab, &slices, &slice);
  const size_t small = (size_t)L.top * 8, big = small + kDBuckets * 2 + (size_t)L.top * 2;
  const unsigned whole = (unsigned)L.rows, parted = (unsigned)(L.rows * slices);
#define EXTERND_DISTILL(MODE, GRID, GS, SMEM, LEN)                                                                     \
  hipLaunchKernelGGL((distill_kernel<T, MODE>), dim3(GRID), dim3(kDThreads), SMEM, st, Z, L.vocab, L.ldz, t,           \
                     L.temperature, L.weight, L.loss, L.stats, D, L.ldd, slices, LEN, GS, parts)
  if (!L.loss) {
    EXTERND_DISTILL(3, parted, slices, big, slice);
  } else if (slices == 1) {
    EXTERND_DISTILL(0, whole, 1, D ? big : small, slice);
  } else {
    EXTERND_DISTILL(1, parted, slices, small, slice);
    if (D) EXTERND_DISTILL(2, parted, slices, big, slice);
    else EXTERND_DISTILL(2, whole, 1, small, slice);
  }
#undef EXTERND_DISTILL
  return hipGetLastError();
}

hipError_t distill_run(const DistillLaunch& L, hipStream_t st) {
  switch (L.z_type) {
    case 0: return distill_typed<float>(L, st);
    case 1: return distill_typed<_Float16>(L, st);
    case 2: return distill_typed<__bf16>(L, st);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace externd
