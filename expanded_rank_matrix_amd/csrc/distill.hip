// Distillation from a teacher's top logits: the loss for each row (token) and its gradient.
//
//   p = softmax of a_k / T over the row's valid entries k (0 <= index_k < V, a_k > -inf)
//   q = softmax of z_v / T over the whole vocabulary
//   loss = w T^2 sum_k p_k (log p_k - log q_index(k))
//   dz_v = w T (q_v P - sum_{k: index(k) = v} p_k),  P = 1 with a valid entry, else 0
//
// One pass over z keeps the running maximum m and the sum S of exp((z - m) / T) (8 elements a step:
// one rescaling of the sum per step at most), so q_v = exp((z_v - m) / T) / S.  z is handled in
// fp32, each thread's sum too (about V / 256 terms or fewer, whose roundings average out to 10^-9 to
// 10^-8 of S; in fp64 every element would take a conversion and an fp64 addition more); the threads'
// sums, log S and the K terms of the loss are fp64, since log p - log q is a difference of numbers many
// times its size.  The gradient is a second pass: g q_v for every element, rounded once to z's type, and
// after it, behind a barrier, the teacher's at most K elements once more, with p in the difference before
// its rounding.  Equal indices of one row meet in hashed lists in LDS; their exponentials add as whole
// numbers of 2^-50 of the largest one's binade, so the order does not matter and each of them writes the
// same value.  p keeps fp32's relative precision however small it is: where the student gives less, it
// is the gradient.
#include "common.hpp"
#include "externd_internal.hpp"
#include "types.hpp"

namespace externd {

constexpr int kDThreads = 256;           // of streaming workgroups
constexpr int kDBuckets = 2048;          // lists of the teacher's indices
constexpr unsigned short kDNone = 0xFFFF;

__device__ __forceinline__ float wave_max_f32(float v) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) v = fmaxf(v, __shfl_xor(v, d));
  return v;
}

// log2 e / T in two fp32 numbers.  An exponent is d log2 e / T with d = z - m <= 0; with the constant in
// one fp32 number each exponential of a row would be off by the same 2^-24 |x| or so, which no sum averages
// out (S by 5 10^-8 at 50 021 logits).  The first part is cut towards zero and the second above it, so that
// d = -inf gives -inf.
struct Log2eT {
  float hi, lo, near;  // near: the nearest fp32 number alone
  __device__ __forceinline__ explicit Log2eT(float T) {
    const double c = 1.4426950408889634 / (double)T;
    near = hi = (float)c;
    if ((double)hi >= c) hi = __uint_as_float(__float_as_uint(hi) - 1u);
    lo = (float)(c - (double)hi);
  }
};
// e^(d / T).  0 below 2^-126, where the instruction flushes: an element's gradient loses at most w T 2^-126
// by it, and S, which is 1 or more, nothing.
__device__ __forceinline__ float exp_t(float d, const Log2eT& c) {
  return __builtin_amdgcn_exp2f(fmaf(d, c.hi, d * c.lo));
}
// The same for an element of T's gradient.  Of 16 bits, one constant will do: 2^-24 |x| is nothing beside
// their own rounding (2^-9 or 2^-12 at the least), and the product less is 2.5% of a step over 131072 logits.
template <typename T>
__device__ __forceinline__ float exp_grad(float d, const Log2eT& c) {
  return sizeof(T) == 4 ? exp_t(d, c) : __builtin_amdgcn_exp2f(d * c.near);
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

// What the row's teacher gives: 1 / sum e (0 without a valid entry) and sum p log p.
struct TeacherSums {
  double pinv, plogp;
};

// The row's teacher, by one wave, into LDS: index of every entry (-1 where there is none), e =
// exp((a - max) / T) (0 there) and the student's logit at it (0 outside lo .. hi - 1).  p = e / sum e.
// A NaN or +inf among the valid entries makes every e NaN.
template <typename T>
__device__ __forceinline__ TeacherSums teacher_row(const Teacher& t, long long row, int V, double rT, const T* z, int lo,
                                                   int hi, int* idx, float* ex, float* zk) {
  const int lane = threadIdx.x & 63;
  const long long base = row * t.top;
  float mx = -__builtin_inff();
  bool nan = false;
  for (int k = lane; k < t.top; k += 64) {
    const int i = teacher_index(t, base + k, V);
    const float a = teacher_value(t, base + k);
    const bool valid = i >= 0 && a != -__builtin_inff();
    idx[k] = valid ? i : -1;
    ex[k] = valid ? a : -__builtin_inff();
    zk[k] = valid && i >= lo && i < hi ? (float)z[i] : 0.0f;
    nan = nan || (valid && a != a);
    mx = fmaxf(mx, valid ? a : -__builtin_inff());
  }
  nan = __any(nan);
  mx = nan ? __builtin_nanf("") : wave_max_f32(mx);
  if (mx == -__builtin_inff()) return {0.0, 0.0};
  double s = 0.0, sx = 0.0;  // sums of e^x and of x e^x, x = (a - max) / T
  for (int k = lane; k < t.top; k += 64) {
    float e = 0.0f;
    if (idx[k] >= 0) {
      const double x = ((double)ex[k] - (double)mx) * rT;
      const float xf = (float)x;
      e = expf(xf);
      if (e != 0.0f) e = fmaf(e, (float)(x - (double)xf), e);  // what x lost by its rounding, up to 2^-24 |x| of e
      s += (double)e;
      if (e != 0.0f) sx += x * (double)e;
    }
    ex[k] = e;
  }
  s = wave_sum_f64(s);
  sx = wave_sum_f64(sx);
  return {1.0 / s, sx / s - log(s)};
}

// running maximum m and sum s of exp((z - m) / T)
__device__ __forceinline__ void stats8(const float (&z)[8], const Log2eT& c, float& m, float& s) {
  float cm = z[0];
#pragma unroll
  for (int e = 1; e < 8; ++e) cm = fmaxf(cm, z[e]);
  if (cm > m) {
    s *= exp_t(m - cm, c);
    m = cm;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) s += exp_t(z[e] - m, c);
}

__device__ __forceinline__ void stats1(float z, const Log2eT& c, float& m, float& s) {
  if (z > m) {
    s *= exp_t(m - z, c);
    m = z;
  }
  s += exp_t(z - m, c);
}

// The waves' (m, s) joined, in two steps around the caller's barrier; the result is the same in every
// thread.  A wave without elements, or with -inf alone, has s = 0 and m = -FLT_MAX (which, unlike
// -inf, lets elements of -inf add exp2(-inf) = 0).
__device__ __forceinline__ void stats_put(float m, float s, const Log2eT& c, float* wm, double* ws) {
  const float M = wave_max_f32(m);
  const double S = wave_sum_f64(s == 0.0f ? 0.0 : (double)s * (double)exp_t(m - M, c));
  if ((threadIdx.x & 63) == 0) {
    wm[threadIdx.x >> 6] = M;
    ws[threadIdx.x >> 6] = S;
  }
}
template <int TH>
__device__ __forceinline__ void stats_get(const Log2eT& c, const float* wm, const double* ws, float& M, double& S) {
  const int lane = threadIdx.x & 63;
  const float m = lane < TH / 64 ? wm[lane] : -__FLT_MAX__;
  const double s = lane < TH / 64 ? ws[lane] : 0.0;
  M = wave_max_f32(m);
  S = wave_sum_f64(s == 0.0 ? 0.0 : s * (double)exp_t(m - M, c));
}

// running (m, s) of this thread over elements lo .. hi - 1
template <typename T, int TH>
__device__ __forceinline__ void slice_stats(const T* z, int lo, int hi, const Log2eT& c, float& m, float& s) {
  m = -__FLT_MAX__;
  s = 0.0f;
  int j = lo + 8 * (int)threadIdx.x;
  constexpr int step = 8 * TH, U = 4;
  for (; (long long)j + (U - 1) * step + 8 <= hi; j += U * step) {
    float v[U][8];
#pragma unroll
    for (int u = 0; u < U; ++u) load8(z + j + u * step, v[u]);
#pragma unroll
    for (int u = 0; u < U; ++u) stats8(v[u], c, m, s);
  }
  for (; (long long)j + 8 <= hi; j += step) {
    float v[8];
    load8(z + j, v);
    stats8(v, c, m, s);
  }
  const int rest = hi & 7;  // the last, fewer than 8: one a thread
  if ((int)threadIdx.x < rest && hi > lo) stats1((float)z[hi - rest + (int)threadIdx.x], c, m, s);
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

template <typename T>
__device__ __forceinline__ iv4 inf_words() {  // -inf throughout
  const int x = sizeof(T) == 4 ? (int)0xFF800000 : __is_same(T, _Float16) ? (int)0xFC00FC00 : (int)0xFF80FF80;
  return iv4{x, x, x, x};
}

// Lists of the teacher's entries by a hash of their index; the caller's barrier lies between clearing
// and linking, another after linking.
__device__ __forceinline__ int bucket(int index) { return (int)((unsigned)index * 2654435769u >> 21); }
static_assert(kDBuckets == 1 << 11, "bucket()");
template <int TH>
__device__ __forceinline__ void lists_clear(unsigned* heads32) {
  for (int x = threadIdx.x; x < kDBuckets / 2; x += TH) heads32[x] = 0xFFFFFFFFu;
}
template <int TH>
__device__ __forceinline__ void lists_link(const int* idx, int top, unsigned* heads32, unsigned short* next) {
  for (int k = threadIdx.x; k < top; k += TH)
    if (idx[k] >= 0) {
      const int b = bucket(idx[k]), sh = 16 * (b & 1);
      unsigned old = heads32[b >> 1], seen;
      do {  // exchange of one half word
        seen = old;
        old = atomicCAS(&heads32[b >> 1], seen, (seen & ~(0xFFFFu << sh)) | (unsigned)k << sh);
      } while (old != seen);
      next[k] = (unsigned short)(seen >> sh);
    }
}

// g q of 8 elements
template <typename T>
__device__ __forceinline__ void grad8(const float (&v)[8], float m, const Log2eT& c, float gi, float (&o)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) o[e] = exp_grad<T>(v[e] - m, c) * gi;
}

// g q of elements lo .. hi - 1 (lo a multiple of 8)
template <typename T, int TH>
__device__ __forceinline__ void slice_grad(const T* z, T* d, int lo, int hi, float m, const Log2eT& c, float gi) {
  int j = lo + 8 * (int)threadIdx.x;
  constexpr int step = 8 * TH, U = 2;
  for (; (long long)j + (U - 1) * step + 8 <= hi; j += U * step) {
    float v[U][8], o[8];
#pragma unroll
    for (int u = 0; u < U; ++u) load8(z + j + u * step, v[u]);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      grad8<T>(v[u], m, c, gi, o);
      store8(d + j + u * step, o);
    }
  }
  if ((long long)j + 8 <= hi) {
    float v[8], o[8];
    load8(z + j, v);
    grad8<T>(v, m, c, gi, o);
    store8(d + j, o);
  }
  const int rest = hi & 7;
  if ((int)threadIdx.x < rest && hi > lo) {
    const int x = hi - rest + (int)threadIdx.x;
    d[x] = (T)(exp_grad<T>((float)z[x] - m, c) * gi);
  }
}

// the teacher's elements of lo .. hi - 1: g (q - p), p = pinv times the sum of e over equal indices
template <typename T, int TH>
__device__ __forceinline__ void teacher_grad(T* d, int lo, int hi, float m, const Log2eT& c, float g, float gi, double pinv,
                                             int top, const int* idx, const float* ex, const float* zk,
                                             const unsigned short* heads, const unsigned short* next) {
  for (int k = threadIdx.x; k < top; k += TH) {
    const int i = idx[k];
    if (i < lo || i >= hi) continue;
    float most = ex[k];  // all of a row's are NaN or none
    int same = 0;
    for (unsigned x = heads[bucket(i)]; x != kDNone; x = next[x])
      if (idx[x] == i) {
        most = fmaxf(most, ex[x]);
        ++same;
      }
    double sum = (double)ex[k];
    if (same > 1 && most > 0.0f) {
      const int sh = 50 + 127 - (int)(__float_as_uint(most) >> 23);  // most 2^sh < 2^51: 1024 of them fit
      unsigned long long whole = 0;
      for (unsigned x = heads[bucket(i)]; x != kDNone; x = next[x])
        if (idx[x] == i) whole += (unsigned long long)ldexp((double)ex[x], sh);
      sum = ldexp((double)whole, -sh);
    }
    const float p = (float)(sum * pinv);
    d[i] = (T)(exp_t(zk[k] - m, c) * gi - g * p);
  }
}

template <typename T, int TH>
__device__ __forceinline__ void slice_zero(T* d, int lo, int hi) {
  const float o[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  for (int j = lo + 8 * (int)threadIdx.x; (long long)j + 8 <= hi; j += 8 * TH) store8(d + j, o);
  const int rest = hi & 7;
  if ((int)threadIdx.x < rest && hi > lo) d[hi - rest + (int)threadIdx.x] = (T)0.0f;
}

// sums over the teacher's entries in lo .. hi - 1 of e and of e (z - m), by one wave.  Taken from m,
// since z itself may be near the type's lowest value throughout a row.
__device__ __forceinline__ void cross_sums(int lo, int hi, const int* idx, const float* ex, const float* zk, int top,
                                           float m, double& mass, double& cross) {
  mass = cross = 0.0;
  for (int k = threadIdx.x & 63; k < top; k += 64)
    if (idx[k] >= lo && idx[k] < hi && ex[k] != 0.0f) {
      mass += (double)ex[k];
      cross += (double)ex[k] * ((double)zk[k] - (double)m);
    }
  mass = wave_sum_f64(mass);
  cross = wave_sum_f64(cross);
}

// a slice's share of a split row, in the workspace
struct Part {
  double s;      // sum of exp((z - m) / T)
  double mass;   // sums of e and of e (z - m) over the slice's teacher entries
  double cross;
  TeacherSums t;
  float m;
  float unused;
};

__device__ __forceinline__ void write_loss(long long row, float w, float Tmp, const TeacherSums& t, double cross, float m,
                                           double S, float* loss, float* stats) {
  const double rT = 1.0 / (double)Tmp, kl = t.plogp - cross * t.pinv * rT + log(S);
  loss[row] = t.pinv != 0.0 ? (float)((double)w * (double)Tmp * (double)Tmp * kl) : 0.0f;
  stats[2 * row] = S == 0.0 ? -__builtin_inff() : m;
  stats[2 * row + 1] = (float)S;
}

// the parts of a row joined, the same in every lane of a wave
__device__ __forceinline__ void join_parts(const Part* q, int slices, const Log2eT& c, float& m, double& S, double& cross) {
  const int lane = threadIdx.x & 63;
  m = -__FLT_MAX__;
  for (int i = lane; i < slices; i += 64) m = fmaxf(m, q[i].m);
  m = wave_max_f32(m);
  S = cross = 0.0;
  for (int i = lane; i < slices; i += 64) {
    if (q[i].s != 0.0) S += q[i].s * (double)exp_t(q[i].m - m, c);
    if (q[i].mass != 0.0) cross += q[i].cross + q[i].mass * ((double)q[i].m - (double)m);
  }
  S = wave_sum_f64(S);
  cross = wave_sum_f64(cross);
}

// Split rows without a gradient: one wave joins a row's parts.
__global__ void __launch_bounds__(64) distill_join_kernel(const Part* __restrict__ parts, int slices, float Tmp,
                                                          const float* __restrict__ weight, float* __restrict__ loss,
                                                          float* __restrict__ stats) {
  const long long row = blockIdx.x;
  const float w = weight ? weight[row] : 1.0f;
  if (w == 0.0f) {
    if (threadIdx.x == 0) {
      loss[row] = 0.0f;
      stats[2 * row] = 0.0f;
      stats[2 * row + 1] = 0.0f;
    }
    return;
  }
  float m;
  double S, cross;
  join_parts(parts + row * slices, slices, Log2eT(Tmp), m, S, cross);
  if (threadIdx.x == 0) write_loss(row, w, Tmp, parts[row * slices].t, cross, m, S, loss, stats);
}

// MODE 0: statistics and loss of whole rows, and their gradient where D is given
// MODE 1: a slice's share of them (split rows, first launch)
// MODE 2: the shares joined: the first slice of a row writes statistics and loss, each its gradient
// MODE 3: gradient of a slice from given statistics
// CH > 0 (MODE 0 with a gradient): the row, at most 8 TH CH elements, stays in registers between the two
// passes; all its loads are in flight at once.  Wave 0 sees to the teacher meanwhile.
// Every thread of a workgroup takes the same branches around the barriers.
template <typename T, int MODE, int TH, int CH>
__global__ void __launch_bounds__(TH) distill_kernel(const T* Z, int V, long long ldz, Teacher teach, float Tmp,
                                                     const float* __restrict__ weight, float* __restrict__ loss,
                                                     float* __restrict__ stats, T* D, long long ldd, int slices,
                                                     int slice, Part* __restrict__ parts) {
  extern __shared__ __attribute__((aligned(16))) unsigned char lds[];
  __shared__ double ws[TH / 64];
  __shared__ float wm[TH / 64];
  __shared__ TeacherSums ts;
  int* idx = reinterpret_cast<int*>(lds);
  float* ex = reinterpret_cast<float*>(idx + teach.top);
  float* zk = ex + teach.top;
  unsigned* heads = reinterpret_cast<unsigned*>(zk + teach.top);
  unsigned short* next = reinterpret_cast<unsigned short*>(heads + kDBuckets / 2);
  const bool wave0 = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) == 0;
  const long long row = blockIdx.x / slices;
  const int sl = (int)(blockIdx.x % slices);
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
    if (D) slice_zero<T, TH>(d, lo, hi);
    return;
  }
  const Log2eT c(Tmp);
  const double rT = 1.0 / (double)Tmp;
  constexpr int W = words8<T>();
  iv4 held[CH > 0 ? CH : 1][W];
  const int rest = V & 7;  // the row's last elements, fewer than 8: one a thread
  float last = -__builtin_inff();
  if (CH > 0) {
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int j = 8 * (i * TH + (int)threadIdx.x);
#pragma unroll
      for (int q = 0; q < W; ++q) held[i][q] = j + 8 <= V ? word8(z + j, q) : inf_words<T>();
    }
    if ((int)threadIdx.x < rest) last = (float)z[V - rest + (int)threadIdx.x];
  }
  if (D) lists_clear<TH>(heads);
  if (wave0) {
    const TeacherSums t = teacher_row(teach, row, V, rT, z, lo, hi, idx, ex, zk);
    if (threadIdx.x == 0) ts = t;
  }
  float m;
  double S, mass, cross = 0.0;
  if (MODE == 0 || MODE == 1) {
    float tm = -__FLT_MAX__, tsum = 0.0f;
    if (CH > 0) {
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        // one chunk after the other, and unpacked anew in the second pass: with several chunks as fp32
        // at a time the row would take twice the registers, and half the waves
        asm volatile("" : "+v"(tm), "+v"(tsum));
#pragma unroll
        for (int q = 0; q < W; ++q) asm volatile("" : "+v"(held[i][q]));
        float v[8];
        unpack8<T>(held[i], v);
        stats8(v, c, tm, tsum);
      }
      stats1(last, c, tm, tsum);
    } else {
      slice_stats<T, TH>(z, lo, hi, c, tm, tsum);
    }
    stats_put(tm, tsum, c, wm, ws);
  }
  __syncthreads();  // the waves' statistics, the teacher, the cleared lists
  const TeacherSums t = ts;
  if (MODE == 0 || MODE == 1) {
    stats_get<TH>(c, wm, ws, m, S);
    if (wave0) cross_sums(lo, hi, idx, ex, zk, teach.top, m, mass, cross);
  } else if (MODE == 2) {
    join_parts(parts + row * slices, slices, c, m, S, cross);
  } else {
    m = stats[2 * row];
    S = (double)stats[2 * row + 1];
  }
  if (MODE == 1) {
    if (threadIdx.x == 0) parts[row * slices + sl] = Part{S, mass, cross, t, m, 0.0f};
    return;
  }
  if (MODE != 3 && sl == 0 && threadIdx.x == 0) write_loss(row, w, Tmp, t, cross, m, S, loss, stats);
  if (!D) return;
  if (t.pinv == 0.0) {  // no teacher, no gradient
    slice_zero<T, TH>(d, lo, hi);
    return;
  }
  lists_link<TH>(idx, teach.top, heads, next);
  const float g = w * Tmp, gi = g * (float)(1.0 / S);
  if (CH > 0) {
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int j = 8 * (i * TH + (int)threadIdx.x);
#pragma unroll
      for (int q = 0; q < W; ++q) asm volatile("" : "+v"(held[i][q]));
      float v[8], o[8];
      unpack8<T>(held[i], v);
      grad8<T>(v, m, c, gi, o);
      if (j + 8 <= V) store8(d + j, o);
    }
    if ((int)threadIdx.x < rest) d[V - rest + (int)threadIdx.x] = (T)(exp_grad<T>(last - m, c) * gi);
  } else {
    slice_grad<T, TH>(z, d, lo, hi, m, c, gi);
  }
  __syncthreads();  // the lists are linked, and the stores above come before those below
  teacher_grad<T, TH>(d, lo, hi, m, c, g, gi, t.pinv, teach.top, idx, ex, zk,
                      reinterpret_cast<const unsigned short*>(heads), next);
}

// Slices of a row, so that few rows fill the card: about four workgroups a CU, each of 4096 elements or
// more but the row's last, which takes what is left (4097 elements: 4096 and 1).
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

template <typename T, int MODE, int TH, int CH>
static void distill_launch(const DistillLaunch& L, bool lists, int slices, int slice, hipStream_t st) {
  const Teacher t{L.teacher, L.index, L.t_type, L.index_bytes, L.top};
  const size_t smem = (size_t)L.top * 12 + (lists ? kDBuckets * 2 + (size_t)L.top * 2 : 0);
  hipLaunchKernelGGL((distill_kernel<T, MODE, TH, CH>), dim3((unsigned)(L.rows * slices)), dim3(TH), smem, st,
                     static_cast<const T*>(L.logits), L.vocab, L.ldz, t, L.temperature, L.weight, L.loss, L.stats,
                     static_cast<T*>(L.dlogits), L.ldd, slices, slice, static_cast<Part*>(L.ws));
}

template <typename T>
static hipError_t distill_typed(const DistillLaunch& all, hipStream_t st) {
  int slices, slice;
  split(all.rows, all.vocab, &slices, &slice);
  DistillLaunch L = all;
  // runs of 2^21 rows: a launch holds below 2^32 threads (split rows are fewer than 1024)
  for (long long r0 = 0; r0 < all.rows; r0 += 1ll << 21) {
    L.rows = all.rows - r0 < (1ll << 21) ? all.rows - r0 : 1ll << 21;
    L.logits = static_cast<const T*>(all.logits) + r0 * L.ldz;
    L.teacher = static_cast<const char*>(all.teacher) + r0 * L.top * (L.t_type == 0 ? 4 : 2);
    L.index = static_cast<const char*>(all.index) + r0 * L.top * L.index_bytes;
    L.weight = all.weight ? all.weight + r0 : nullptr;
    L.loss = all.loss ? all.loss + r0 : nullptr;
    L.stats = all.stats + 2 * r0;
    L.dlogits = all.dlogits ? static_cast<T*>(all.dlogits) + r0 * L.ldd : nullptr;
    if (!L.loss) {
      distill_launch<T, 3, kDThreads, 0>(L, true, slices, slice, st);
    } else if (slices > 1) {
      L.dlogits = nullptr;
      distill_launch<T, 1, kDThreads, 0>(L, false, slices, slice, st);
      L.dlogits = all.dlogits;
      if (L.dlogits)
        distill_launch<T, 2, kDThreads, 0>(L, true, slices, slice, st);
      else
        hipLaunchKernelGGL(distill_join_kernel, dim3((unsigned)L.rows), dim3(64), 0, st, static_cast<const Part*>(L.ws),
                           slices, L.temperature, L.weight, L.loss, L.stats);
    } else if (!L.dlogits) {
      distill_launch<T, 0, kDThreads, 0>(L, false, 1, slice, st);
    } else {
      // The shape by the row's length: held where a thread has 8 or 16 chunks, with as few threads as
      // hold it (several rows share a CU, one's stores under another's loads).  Measured, 2048 rows of
      // bf16, step in us, held / 256 threads streaming / 1024 streaming: 8192: 19.5 / 18.7 / 29.5;
      // 32768: 52.7 / 64.5 / 62.2; 65536: 115 / 163 / 137; 131072: 235 / 334 / 267.
      constexpr bool f32 = sizeof(T) == 4;
      if (L.vocab <= 8 * 256 * 4) distill_launch<T, 0, kDThreads, 0>(L, true, 1, slice, st);
      else if (L.vocab <= 8 * 256 * 8) distill_launch<T, 0, 256, 8>(L, true, 1, slice, st);
      else if (L.vocab <= 8 * 512 * 8) distill_launch<T, 0, 512, 8>(L, true, 1, slice, st);
      else if (!f32 && L.vocab <= 8 * 512 * 16) distill_launch<T, 0, 512, f32 ? 8 : 16>(L, true, 1, slice, st);
      else if (f32 && L.vocab <= 8 * 1024 * 8) distill_launch<T, 0, 1024, 8>(L, true, 1, slice, st);
      else if (!f32 && L.vocab <= 8 * 1024 * 16) distill_launch<T, 0, 1024, f32 ? 8 : 16>(L, true, 1, slice, st);
      else distill_launch<T, 0, 1024, 0>(L, true, 1, slice, st);
    }
  }
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
