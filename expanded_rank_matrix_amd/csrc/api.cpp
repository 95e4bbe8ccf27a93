// C ABI of libexternd: argument validation, workspace, launch sequence, status codes.
#include <hip/hip_runtime.h>

#include <chrono>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <map>
#include <memory>
#include <mutex>
#include <string>
#include <utility>

#include "externd.h"
#include "externd_internal.hpp"

using namespace externd;

namespace {

thread_local std::string g_last_error;

int fail(int status, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  g_last_error = buf;
  return status;
}

#define HIP_OR_FAIL(expr)                                                                          \
  do {                                                                                             \
    hipError_t e_ = (expr);                                                                        \
    if (e_ != hipSuccess) return fail(EXTERND_EDEVICE, "%s failed: %s", #expr, hipGetErrorString(e_)); \
  } while (0)

int64_t rank_of(int64_t m, int64_t n, float mu) {
  if (m < 1 || n < 1 || !std::isfinite(mu) || !(mu > 0.0f)) return -1;
  const double k = std::floor((double)mu * (double)(m < n ? m : n) + 1e-9);
  if (!(k >= 1.0) || k > 2147483647.0) return -1;
  return (int64_t)k;
}

// Stream-ordered workspace that is always released.
struct Workspace {
  hipStream_t st;
  void* p = nullptr;
  explicit Workspace(hipStream_t s) : st(s) {}
  ~Workspace() {
    if (p) (void)hipFreeAsync(p, st);
  }
};

size_t al256(size_t x) { return (x + 255) & ~(size_t)255; }

unsigned spin_limit_from_env() {
  const char* s = std::getenv("EXTERND_SPIN_LIMIT");
  if (s && *s) {
    const long long v = std::atoll(s);
    if (v > 0) return (unsigned)v;
  }
  return 1u << 24;
}

int exp_bound_host(float x) {
  int e;
  std::frexp(x, &e);
  return e;
}

}  // namespace

extern "C" {

int64_t externd_rank(int64_t m, int64_t n, float mu) { return rank_of(m, n, mu); }

int64_t externd_packed_words(int64_t len) { return len < 0 ? -1 : (len + 15) / 16; }

const char* externd_status_string(int status) {
  switch (status) {
    case EXTERND_OK: return "EXTERND_OK";
    case EXTERND_EINVAL: return "EXTERND_EINVAL";
    case EXTERND_ENOMEM: return "EXTERND_ENOMEM";
    case EXTERND_EDEVICE: return "EXTERND_EDEVICE";
    case EXTERND_ENONFINITE: return "EXTERND_ENONFINITE";
    default: return "EXTERND_UNKNOWN";
  }
}

const char* externd_last_error(void) { return g_last_error.c_str(); }

int externd_decompose(const float* A, int64_t m, int64_t n, float mu, float tau, const float* h, int als_iters,
                      int block, uint32_t* B_packed, uint32_t* C_packed, float* D, double* energy, void* stream,
                      externd_stats* stats) {
  return externd_decompose_ex(A, m, n, mu, tau, h, als_iters, block, B_packed, C_packed, D, energy, nullptr, stream,
                              stats);
}

int externd_decompose_ex(const float* A, int64_t m, int64_t n, float mu, float tau, const float* h, int als_iters,
                         int block, uint32_t* B_packed, uint32_t* C_packed, float* D, double* energy,
                         const externd_options* options, void* stream, externd_stats* stats) {
  const auto t0 = std::chrono::steady_clock::now();
  g_last_error.clear();
  const double target = options ? options->energy_target : 0.0;
  const int safeguard = options ? options->safeguard : 0;
  const int sweeps = options ? options->sweeps : 0;
  const int ablation = options ? options->ablation : 0;
  const int residual_hbm = options ? options->residual_hbm : 0;
  if (ablation & ~3) return fail(EXTERND_EINVAL, "ablation must be a combination of 1 and 2");
  if (residual_hbm != 0 && residual_hbm != 1) return fail(EXTERND_EINVAL, "residual_hbm must be 0 or 1");
  if (sweeps < 0 || sweeps > 64) return fail(EXTERND_EINVAL, "sweeps must be in [0, 64]");
  if (!(target == 0.0 || (target > 0.0 && target <= 1.0)))
    return fail(EXTERND_EINVAL, "energy_target must be 0 (off) or in (0, 1]");
  if (safeguard != 0 && safeguard != 1) return fail(EXTERND_EINVAL, "safeguard must be 0 or 1");
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  if (!A || !B_packed || !C_packed || !D || !energy) return fail(EXTERND_EINVAL, "null pointer argument");
  if (m < 1 || n < 1) return fail(EXTERND_EINVAL, "m and n must be >= 1 (got %lld x %lld)", (long long)m, (long long)n);
  if (m > 16384 || n > 16384)
    return fail(EXTERND_EINVAL, "max(m, n) must be <= 16384 (got %lld x %lld)", (long long)m, (long long)n);
  if (!std::isfinite(tau) || tau < 0.0f || tau > 1.0f) return fail(EXTERND_EINVAL, "tau must be in [0, 1]");
  if (als_iters < 1) return fail(EXTERND_EINVAL, "als_iters must be >= 1");
  if (block < -1) return fail(EXTERND_EINVAL, "block must be >= -1");
  const int64_t k = rank_of(m, n, mu);
  if (k < 1) return fail(EXTERND_EINVAL, "mu must be finite and > 0 with k = floor(mu min(m,n)) >= 1");
  int64_t b = block == -1 ? std::max<int64_t>(1, std::min<int64_t>(256, std::min(m, n) / 8)) : (block <= 1 ? 1 : block);
  if (b > k) b = k;
  if (safeguard && b > 1) return fail(EXTERND_EINVAL, "the safeguard applies to the sequential path only (block resolved to %lld)", (long long)b);
  if ((ablation & 1) && b == 1)
    return fail(EXTERND_EINVAL, "ablation 1 (targets without decorrelation) applies to the block path only");
  const int mi = (int)m, ni = (int)n, ki = (int)k, bi = (int)b;
  const int ldr = (ni + 3) & ~3, ldt = (mi + 3) & ~3;

  // ---- workspace layout
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off = al256(off + bytes);
    return o;
  };
  const size_t o_flags = take(64);
  const size_t o_bar = take(sizeof(unsigned) * kBarWords);
  const size_t o_stats = take(8 * sizeof(u64));
  const size_t o_bytes = take(sizeof(double));
  const size_t o_R = take((size_t)mi * ldr * sizeof(float));
  const size_t o_rs = take((size_t)mi * sizeof(double));
  const size_t o_rowE = take((size_t)mi * sizeof(double));
  size_t o_RT = 0, o_xz = 0, o_xw = 0, o_xf = 0, o_rsg = 0, o_blk = 0;
  int grid = 0;
  bool rl = false, keys = true;
  if (b == 1) {
    o_RT = take((size_t)ni * ldt * sizeof(float));
    o_xz = take((size_t)mi * sizeof(double));
    o_xw = take((size_t)ni * sizeof(double));
    int dev = 0;
    HIP_OR_FAIL(hipGetDevice(&dev));
    int ncu = 0;
    HIP_OR_FAIL(hipDeviceGetAttribute(&ncu, hipDeviceAttributeMultiprocessorCount, dev));
    if (!seq_plan(mi, ni, h != nullptr, ncu, residual_hbm == 0, &grid, &rl, &keys))
      return fail(EXTERND_EINVAL, "problem too large for the sequential kernel's on-chip state (%d x %d)", mi, ni);
    o_xf = take((size_t)4 * grid * sizeof(double));
    o_rsg = take((size_t)grid * mi * sizeof(double));
  } else {
    o_RT = take((size_t)ni * ldt * sizeof(float));
    o_blk = take(block_workspace_bytes(mi, ni, bi, h != nullptr));
  }
  Workspace ws(st);
  if (hipMallocAsync(&ws.p, off, st) != hipSuccess) {
    (void)hipGetLastError();
    return fail(EXTERND_ENOMEM, "workspace allocation of %zu bytes failed", off);
  }
  char* base = static_cast<char*>(ws.p);
  unsigned* flags = reinterpret_cast<unsigned*>(base + o_flags);
  unsigned* bar = reinterpret_cast<unsigned*>(base + o_bar);
  u64* dstats = reinterpret_cast<u64*>(base + o_stats);
  double* dbytes = reinterpret_cast<double*>(base + o_bytes);
  float* R = reinterpret_cast<float*>(base + o_R);
  double* rs = reinterpret_cast<double*>(base + o_rs);
  double* rowE = reinterpret_cast<double*>(base + o_rowE);
  HIP_OR_FAIL(hipMemsetAsync(base, 0, o_R, st));  // flags, barrier words, counters

  // ---- input checks (one host round trip)
  HIP_OR_FAIL(check_inputs(A, mi, ni, h, flags, st));
  unsigned hflags[2] = {0u, 0u};
  HIP_OR_FAIL(hipMemcpyAsync(hflags, flags, sizeof(hflags), hipMemcpyDeviceToHost, st));
  HIP_OR_FAIL(hipStreamSynchronize(st));
  if (hflags[0] & 1u) return fail(EXTERND_ENONFINITE, "A contains NaN or Inf");
  if (hflags[0] & 2u) return fail(EXTERND_ENONFINITE, "importance_weights contain NaN or Inf");
  if (hflags[0] & 4u) return fail(EXTERND_EINVAL, "importance_weights must be > 0");
  int EHm = 0;
  if (h) {
    float hmax;
    std::memcpy(&hmax, &hflags[1], sizeof(float));
    EHm = exp_bound_host(hmax);
  }

  // ---- staging
  HIP_OR_FAIL(stage_rows(A, mi, ni, h, R, ldr, rs, rowE, st));
  hipEvent_t e0, e1;
  HIP_OR_FAIL(hipEventCreate(&e0));
  HIP_OR_FAIL(hipEventCreate(&e1));
  struct EvGuard {
    hipEvent_t a, b;
    ~EvGuard() {
      (void)hipEventDestroy(a);
      (void)hipEventDestroy(b);
    }
  } evg{e0, e1};
  double flops = 0.0, blk_bytes = -1.0;
  if (b == 1) {
    float* RT = reinterpret_cast<float*>(base + o_RT);
    HIP_OR_FAIL(stage_transpose(A, mi, ni, RT, ldt, st));
    SeqLaunch L;
    L.R = R;
    L.RT = RT;
    L.h = h;
    L.rs0 = rs;
    L.rowE = rowE;
    L.xz = reinterpret_cast<double*>(base + o_xz);
    L.xw = reinterpret_cast<double*>(base + o_xw);
    L.xf = reinterpret_cast<double*>(base + o_xf);
    L.rsg = reinterpret_cast<double*>(base + o_rsg);
    L.rl = rl;
    L.keys = keys;
    L.bar = bar;
    L.Bp = B_packed;
    L.Cp = C_packed;
    L.D = D;
    L.energy = energy;
    L.stats = dstats;
    L.bytes = dbytes;
    L.m = mi;
    L.n = ni;
    L.ldr = ldr;
    L.ldt = ldt;
    L.k = ki;
    L.T = als_iters;
    L.EHm = EHm;
    L.grid = grid;
    L.tau = tau;
    L.spin_limit = spin_limit_from_env();
    L.target = target;
    L.safeguard = safeguard;
    L.sweeps = sweeps;
    L.ablation = ablation;
    HIP_OR_FAIL(hipEventRecord(e0, st));
    HIP_OR_FAIL(seq_launch(L, st));
    HIP_OR_FAIL(hipEventRecord(e1, st));
  } else {
    float* RT = reinterpret_cast<float*>(base + o_RT);
    HIP_OR_FAIL(stage_transpose(A, mi, ni, RT, ldt, st));
    BlockLaunch L;
    L.R = R;
    L.RT = RT;
    L.m = mi;
    L.n = ni;
    L.ldr = ldr;
    L.ldt = ldt;
    L.k = ki;
    L.b = bi;
    L.T = als_iters;
    L.EHm = EHm;
    L.tau = tau;
    L.h = h;
    L.rowE = rowE;
    L.Bp = B_packed;
    L.Cp = C_packed;
    L.D = D;
    L.energy = energy;
    L.stats = dstats;
    L.ws = base + o_blk;
    L.target = target;
    L.sweeps = sweeps;
    L.ablation = ablation;
    HIP_OR_FAIL(hipEventRecord(e0, st));
    HIP_OR_FAIL(block_run(L, st, &flops, &blk_bytes));
    HIP_OR_FAIL(hipEventRecord(e1, st));
  }
  // final explicit energy from the residual
  HIP_OR_FAIL(row_energy(R, mi, ni, ldr, h, rs, st));
  u64 hst[8];
  unsigned hbar = 0;
  double hbytes = 0.0;
  HIP_OR_FAIL(hipMemcpyAsync(hst, dstats, sizeof(hst), hipMemcpyDeviceToHost, st));
  HIP_OR_FAIL(hipMemcpyAsync(&hbar, bar, sizeof(unsigned), hipMemcpyDeviceToHost, st));
  HIP_OR_FAIL(hipMemcpyAsync(&hbytes, dbytes, sizeof(double), hipMemcpyDeviceToHost, st));
  double* hrow = nullptr;
  if (stats) {
    hrow = static_cast<double*>(std::malloc(2 * sizeof(double) * (size_t)mi));
    if (!hrow) return fail(EXTERND_ENOMEM, "host allocation failed");
    HIP_OR_FAIL(hipMemcpyAsync(hrow, rs, sizeof(double) * mi, hipMemcpyDeviceToHost, st));
    HIP_OR_FAIL(hipMemcpyAsync(hrow + mi, rowE, sizeof(double) * mi, hipMemcpyDeviceToHost, st));
  }
  const hipError_t se = hipStreamSynchronize(st);
  if (se != hipSuccess) {
    std::free(hrow);
    return fail(EXTERND_EDEVICE, "decomposition failed on the device: %s", hipGetErrorString(se));
  }
  if (hbar != 0u) {
    std::free(hrow);
    return fail(EXTERND_EDEVICE, "grid barrier wait exceeded its limit (device-side failure)");
  }
  if (stats) {
    float ms = 0.0f;
    (void)hipEventElapsedTime(&ms, e0, e1);
    double er = 0.0, e0s = 0.0;
    for (int i = 0; i < mi; ++i) er += hrow[i];
    for (int i = 0; i < mi; ++i) e0s += hrow[mi + i];
    std::free(hrow);
    stats->k = k;
    stats->passes = (int64_t)hst[0];
    stats->early_exits = (int64_t)hst[1];
    stats->fallback_inits = (int64_t)hst[2];
    stats->zero_components = (int64_t)hst[3];
    stats->block = b;
    stats->energy_final_explicit = e0s > 0.0 ? 1.0 - er / e0s : 1.0;
    stats->kernel_ms = ms;
    stats->bytes_algorithmic = blk_bytes >= 0.0 ? blk_bytes : hbytes;
    stats->flops_algorithmic = flops;
    stats->components_used = hst[5] > 0 ? (int64_t)hst[5] : k;
    stats->safeguard_activations = (int64_t)hst[4];
    stats->sweep_reverts = (int64_t)hst[6];
    stats->residual_lds = rl ? 1 : 0;
    stats->seconds = std::chrono::duration<double>(std::chrono::steady_clock::now() - t0).count();
  }
  return EXTERND_OK;
}

int externd_project(const float* X, int64_t count, int64_t L, float tau, const float* h, int8_t* V, double* PHC,
                    void* stream) {
  g_last_error.clear();
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  if (!X || !V || !PHC) return fail(EXTERND_EINVAL, "null pointer argument");
  if (count < 1 || count > 2147483647 || L < 1 || L > 16384) return fail(EXTERND_EINVAL, "need count >= 1 and 1 <= L <= 16384");
  if (!std::isfinite(tau) || tau < 0.0f || tau > 1.0f) return fail(EXTERND_EINVAL, "tau must be in [0, 1]");
  int EHm = 0;
  unsigned* flags = nullptr;
  if (hipMallocAsync(reinterpret_cast<void**>(&flags), 64, st) != hipSuccess) {
    (void)hipGetLastError();
    return fail(EXTERND_ENOMEM, "workspace allocation failed");
  }
  struct F {
    unsigned* p;
    hipStream_t s;
    ~F() { (void)hipFreeAsync(p, s); }
  } fg{flags, st};
  HIP_OR_FAIL(hipMemsetAsync(flags, 0, 64, st));
  HIP_OR_FAIL(check_inputs(X, (int)count, (int)L, h, flags, st));
  unsigned hflags[2];
  HIP_OR_FAIL(hipMemcpyAsync(hflags, flags, sizeof(hflags), hipMemcpyDeviceToHost, st));
  HIP_OR_FAIL(hipStreamSynchronize(st));
  if (hflags[0] & 1u) return fail(EXTERND_ENONFINITE, "X contains NaN or Inf");
  if (hflags[0] & 2u) return fail(EXTERND_ENONFINITE, "h contains NaN or Inf");
  if (hflags[0] & 4u) return fail(EXTERND_EINVAL, "h must be > 0");
  if (h) {
    float hmax;
    std::memcpy(&hmax, &hflags[1], sizeof(float));
    EHm = exp_bound_host(hmax);
  }
  HIP_OR_FAIL(project_rows(X, (int)count, (int)L, tau, h, EHm, V, PHC, st));
  HIP_OR_FAIL(hipStreamSynchronize(st));
  return EXTERND_OK;
}

// Workspace of externd_apply_factors: one buffer per (device, stream), grown on demand and held
// until the process ends, so that a call after the first is its kernels alone.  Calls on one
// stream use its buffer in stream order; the lock keeps two threads from enqueueing on one stream
// at once.
struct InferBuffer {
  std::mutex mu;
  void* p = nullptr;
  size_t bytes = 0;
};

static InferBuffer& infer_buffer(int dev, hipStream_t st) {
  static std::mutex mu;
  static std::map<std::pair<int, hipStream_t>, std::unique_ptr<InferBuffer>> buffers;
  std::lock_guard<std::mutex> g(mu);
  std::unique_ptr<InferBuffer>& b = buffers[std::make_pair(dev, st)];
  if (!b) b.reset(new InferBuffer);
  return *b;
}

int externd_apply_factors(const uint32_t* B_packed, const uint32_t* C_packed, const float* D, int64_t k, int64_t m,
                          int64_t n, const float* X, int64_t batch, float* Y, void* stream) {
  g_last_error.clear();
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  if (!B_packed || !C_packed || !D || !X || !Y) return fail(EXTERND_EINVAL, "null pointer argument");
  if (k < 1 || k > 2147483647 || m < 1 || n < 1 || m > 2147483647 - 15 || n > 2147483647 - 15)
    return fail(EXTERND_EINVAL, "need k, m, n >= 1 (and below 2^31)");
  if (batch < 1 || batch > 65535) return fail(EXTERND_EINVAL, "need 1 <= batch <= 65535");
  const size_t wsb = infer_workspace_bytes((int)k, (int)m, (int)batch);
  int dev = 0;
  HIP_OR_FAIL(hipGetDevice(&dev));
  InferBuffer& buf = infer_buffer(dev, st);
  std::lock_guard<std::mutex> lock(buf.mu);
  if (buf.bytes < wsb) {
    if (buf.p) {  // earlier calls on this stream may still use the buffer
      HIP_OR_FAIL(hipStreamSynchronize(st));
      (void)hipFree(buf.p);
      buf.p = nullptr;
      buf.bytes = 0;
    }
    if (hipMalloc(&buf.p, wsb) != hipSuccess) {
      (void)hipGetLastError();
      buf.p = nullptr;
      return fail(EXTERND_ENOMEM, "workspace allocation failed");
    }
    buf.bytes = wsb;
  }
  HIP_OR_FAIL(infer_run(B_packed, C_packed, D, (int)k, (int)m, (int)n, X, (int)batch, Y, buf.p, st));
  return EXTERND_OK;
}

int externd_apply_factors_static(const uint32_t* B_packed, const uint32_t* C_packed, const float* D, int64_t k,
                                 int64_t m, int64_t n, const float* X, int64_t batch, float* Y, void* stream) {
  g_last_error.clear();
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  if (!B_packed || !C_packed || !D || !X || !Y) return fail(EXTERND_EINVAL, "null pointer argument");
  if (k < 1 || k > 2147483647 || m < 1 || n < 1 || m > 2147483647 - 15 || n > 2147483647 - 15)
    return fail(EXTERND_EINVAL, "need k, m, n >= 1 (and below 2^31)");
  if (batch < 1 || batch > 65535) return fail(EXTERND_EINVAL, "need 1 <= batch <= 65535");
  const size_t need = infer_workspace_bytes((int)k, (int)m, (int)batch);
  if (need > kInferStaticBytes)
    return fail(EXTERND_EINVAL,
                "batch x (k + m) too large for the fixed workspace: needs %zu bytes, the limit is %zu "
                "(8 batch (k + m) + 4 batch ceil(k / 32) + 4 ceil(batch / 2) ceil(m / 256) bytes, each part "
                "rounded up to 256)", need,
                kInferStaticBytes);
  void* ws = nullptr;
  HIP_OR_FAIL(infer_static_scratch(&ws));
  HIP_OR_FAIL(infer_run(B_packed, C_packed, D, (int)k, (int)m, (int)n, X, (int)batch, Y, ws, st));
  return EXTERND_OK;
}

int externd_matvec(const float* R, int64_t m, int64_t n, const int8_t* t, const float* h, int transpose, double* out,
                   void* stream) {
  g_last_error.clear();
  hipStream_t st = reinterpret_cast<hipStream_t>(stream);
  if (!R || !t || !out) return fail(EXTERND_EINVAL, "null pointer argument");
  if (m < 1 || n < 1 || m > 16384 || n > 16384) return fail(EXTERND_EINVAL, "need 1 <= m, n <= 16384");
  const int mi = (int)m, ni = (int)n;
  // stage the operand the way the decomposition kernel holds it: padded rows (R or R^T), the
  // ternary vector and the weights padded with zeros
  const int rows = transpose ? ni : mi, len = transpose ? mi : ni;
  const int ld = (len + 3) & ~3;
  const bool weighted = h && !transpose;
  void* p = nullptr;
  const size_t b_R = al256((size_t)rows * ld * 4), b_t = al256((size_t)ld), b_h = al256((size_t)ld * 4);
  const size_t b_s = al256((size_t)mi * 16);
  if (hipMallocAsync(&p, b_R + b_t + b_h + b_s, st) != hipSuccess) {
    (void)hipGetLastError();
    return fail(EXTERND_ENOMEM, "workspace allocation failed");
  }
  struct F {
    void* p;
    hipStream_t s;
    ~F() { (void)hipFreeAsync(p, s); }
  } fg{p, st};
  char* base = static_cast<char*>(p);
  float* Rs = reinterpret_cast<float*>(base);
  int8_t* tp = reinterpret_cast<int8_t*>(base + b_R);
  float* hp = reinterpret_cast<float*>(base + b_R + b_t);
  double* scratch = reinterpret_cast<double*>(base + b_R + b_t + b_h);
  if (transpose) HIP_OR_FAIL(stage_transpose(R, mi, ni, Rs, ld, st));
  else HIP_OR_FAIL(stage_rows(R, mi, ni, nullptr, Rs, ld, scratch, scratch + mi, st));
  HIP_OR_FAIL(hipMemsetAsync(tp, 0, (size_t)ld, st));
  HIP_OR_FAIL(hipMemcpyAsync(tp, t, (size_t)len, hipMemcpyDeviceToDevice, st));
  if (weighted) {
    HIP_OR_FAIL(hipMemsetAsync(hp, 0, (size_t)ld * 4, st));
    HIP_OR_FAIL(hipMemcpyAsync(hp, h, (size_t)len * 4, hipMemcpyDeviceToDevice, st));
  }
  HIP_OR_FAIL(matvec_rows(Rs, rows, ld / 4, ld, tp, weighted ? hp : nullptr, out, st));
  HIP_OR_FAIL(hipStreamSynchronize(st));
  return EXTERND_OK;
}

// ---- layers in 8-bit integers: enqueue only, the caller's workspace

static bool float_type(int t) { return t == EXTERND_F32 || t == EXTERND_F16 || t == EXTERND_BF16; }

constexpr int64_t kMaxCount = 2147483647;  // rows, tokens, channels
constexpr int64_t kMaxProductLen = 131071; // 128 128 n < 2^31: the sum of products of int8 fits int32
constexpr int64_t kMaxChannels = (int64_t)1 << 26;
constexpr int64_t kMaxLd = (int64_t)1 << 40;

// `rows` rows of `len` bytes, `pitch` bytes apart.
struct Rows {
  const void* p;
  int64_t rows, len, pitch;
};
static Rows dense(const void* p, int64_t bytes) { return {p, 1, bytes, bytes}; }
// Whether two arguments share memory: an output over an input is written by workgroups, or by a launch,
// that others of the call still read.  Rows of one pitch may lie side by side; of two pitches, any meeting
// of the whole counts.
static bool meet(const Rows& a, const Rows& b) {
  if (!a.p || !b.p || a.rows == 0 || a.len == 0 || b.rows == 0 || b.len == 0) return false;
  const __int128 x = (__int128)reinterpret_cast<uintptr_t>(a.p), y = (__int128)reinterpret_cast<uintptr_t>(b.p);
  const __int128 xe = x + (__int128)(a.rows - 1) * a.pitch + a.len, ye = y + (__int128)(b.rows - 1) * b.pitch + b.len;
  if (xe <= y || ye <= x) return false;
  if (a.rows == 1 ? b.rows == 1 : b.rows > 1 && a.pitch != b.pitch) return true;
  const int64_t pitch = a.rows > 1 ? a.pitch : b.pitch;
  const __int128 at = ((y - x) % pitch + pitch) % pitch;  // where a row of b starts among a's
  return at < a.len || at > pitch - b.len;
}

int externd_quantize_rows(const void* X, int x_type, int64_t rows, int64_t n, int64_t ldx, int8_t* Q, int64_t ldq,
                          float* scale, void* stream) {
  g_last_error.clear();
  if (!float_type(x_type)) return fail(EXTERND_EINVAL, "x_type must be EXTERND_F32, EXTERND_F16 or EXTERND_BF16");
  if (rows < 0 || rows > kMaxCount) return fail(EXTERND_EINVAL, "need 0 <= rows < 2^31");
  if (n < 1 || n > kMaxCount - 4096) return fail(EXTERND_EINVAL, "need 1 <= n < 2^31 - 4096");
  if (ldx < n || ldx > kMaxLd || ldq < n || ldq > kMaxLd)
    return fail(EXTERND_EINVAL, "ldx and ldq must be at least n (and at most 2^40)");
  if (rows == 0) return EXTERND_OK;
  if (!X || !Q || !scale) return fail(EXTERND_EINVAL, "null pointer argument");
  const int64_t es = x_type == EXTERND_F32 ? 4 : 2;
  const Rows in{X, rows, n * es, ldx * es}, out{Q, rows, n, ldq}, sc = dense(scale, rows * 4);
  if (meet(out, in) || meet(sc, in) || meet(sc, out)) return fail(EXTERND_EINVAL, "Q and scale must not overlap X or each other");
  HIP_OR_FAIL(quantize_run(X, x_type, rows, (int)n, ldx, Q, ldq, (int)n, scale, reinterpret_cast<hipStream_t>(stream)));
  return EXTERND_OK;
}

int64_t externd_apply_quantized_workspace(int x_type, int64_t tokens, int64_t n, int64_t m) {
  if (!(float_type(x_type) || x_type == EXTERND_I8) || tokens < 0 || tokens > kMaxCount || n < 1 ||
      n > kMaxProductLen || m < 1 || m > kMaxChannels)
    return -1;
  return (int64_t)product_workspace_bytes(x_type, tokens, (int)n, (int)m);
}

int externd_apply_quantized(const int8_t* W, const float* w_scale, int64_t m, int64_t n, int64_t ldw, const void* X,
                            int x_type, const float* x_scale, int64_t tokens, int64_t ldx, void* Y, int y_type,
                            int64_t ldy, void* workspace, void* stream) {
  g_last_error.clear();
  if (!float_type(x_type) && x_type != EXTERND_I8)
    return fail(EXTERND_EINVAL, "x_type must be EXTERND_F32, EXTERND_F16, EXTERND_BF16 or EXTERND_I8");
  if (!float_type(y_type)) return fail(EXTERND_EINVAL, "y_type must be EXTERND_F32, EXTERND_F16 or EXTERND_BF16");
  if (tokens < 0 || tokens > kMaxCount || m < 1 || m > kMaxChannels)
    return fail(EXTERND_EINVAL, "need 0 <= tokens < 2^31 and 1 <= m <= 2^26");
  if (n < 1 || n > kMaxProductLen)
    return fail(EXTERND_EINVAL, "need 1 <= n <= %lld (the sum of products must fit int32)", (long long)kMaxProductLen);
  if (ldw < n || ldw > kMaxLd || ldx < n || ldx > kMaxLd || ldy < m || ldy > kMaxLd)
    return fail(EXTERND_EINVAL, "ldw and ldx must be at least n and ldy at least m (and at most 2^40)");
  if (tokens == 0) return EXTERND_OK;
  if (!W || !w_scale || !X || !Y) return fail(EXTERND_EINVAL, "null pointer argument");
  if ((x_type == EXTERND_I8) != (x_scale != nullptr))
    return fail(EXTERND_EINVAL, "x_scale is given with x_type EXTERND_I8 and only then");
  if (product_workspace_bytes(x_type, tokens, (int)n, (int)m) > 0 && (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 15)))
    return fail(EXTERND_EINVAL, "workspace of externd_apply_quantized_workspace() bytes, 16-byte aligned, is needed");
  const int64_t xs = x_type == EXTERND_F32 ? 4 : x_type == EXTERND_I8 ? 1 : 2, ys = y_type == EXTERND_F32 ? 4 : 2;
  const Rows out{Y, tokens, m * ys, ldy * ys};
  if (meet(out, {X, tokens, n * xs, ldx * xs}) || meet(out, {W, m, n, ldw}) || meet(out, dense(w_scale, m * 4)) ||
      meet(out, dense(x_scale, x_scale ? tokens * 4 : 0)))
    return fail(EXTERND_EINVAL, "Y must not overlap the inputs");
  HIP_OR_FAIL(product_run(W, w_scale, (int)m, (int)n, ldw, X, x_type, x_scale, (int)tokens, ldx, Y, y_type, ldy,
                          workspace, reinterpret_cast<hipStream_t>(stream)));
  return EXTERND_OK;
}

// ---- distillation on a teacher's top logits

constexpr int64_t kMaxVocab = (int64_t)1 << 30;
constexpr int64_t kMaxTop = 1024;

int64_t externd_distill_workspace(int64_t rows, int64_t vocab) {
  if (rows < 0 || rows > kMaxCount || vocab < 1 || vocab > kMaxVocab) return -1;
  return (int64_t)distill_workspace_bytes(rows, (int)vocab);
}

// what both directions check; 1 where there is nothing to do
static int distill_checks(const void* logits, int z_type, int64_t rows, int64_t vocab, int64_t ldz, const void* teacher,
                          int t_type, const void* index, int index_bytes, int64_t top, float temperature) {
  if (!float_type(z_type) || !float_type(t_type))
    return fail(EXTERND_EINVAL, "z_type and t_type must be EXTERND_F32, EXTERND_F16 or EXTERND_BF16");
  if (index_bytes != 4 && index_bytes != 8) return fail(EXTERND_EINVAL, "index_bytes must be 4 or 8");
  if (rows < 0 || rows > kMaxCount) return fail(EXTERND_EINVAL, "need 0 <= rows < 2^31");
  if (vocab < 1 || vocab > kMaxVocab) return fail(EXTERND_EINVAL, "need 1 <= vocab <= 2^30");
  if (top < 1 || top > kMaxTop) return fail(EXTERND_EINVAL, "need 1 <= top <= %lld", (long long)kMaxTop);
  if (ldz < vocab || ldz > kMaxLd) return fail(EXTERND_EINVAL, "ldz must be at least vocab (and at most 2^40)");
  if (!std::isfinite(temperature) || temperature < 1e-3f || temperature > 1e3f)
    return fail(EXTERND_EINVAL, "temperature must be in [1e-3, 1e3]");
  if (rows == 0) return 1;
  if (!logits || !teacher || !index) return fail(EXTERND_EINVAL, "null pointer argument");
  return EXTERND_OK;
}

int externd_distill_loss(const void* logits, int z_type, int64_t rows, int64_t vocab, int64_t ldz, const void* teacher,
                         int t_type, const void* index, int index_bytes, int64_t top, float temperature,
                         const float* weight, float* loss, float* stats, void* dlogits, int64_t ldd, void* workspace,
                         void* stream) {
  g_last_error.clear();
  const int rc = distill_checks(logits, z_type, rows, vocab, ldz, teacher, t_type, index, index_bytes, top, temperature);
  if (rc < 0) return rc;
  if (dlogits && (ldd < vocab || ldd > kMaxLd)) return fail(EXTERND_EINVAL, "ldd must be at least vocab (and at most 2^40)");
  if (rc == 1) return EXTERND_OK;
  if (!loss || !stats) return fail(EXTERND_EINVAL, "null pointer argument");
  if (dlogits == logits && ldd != ldz) return fail(EXTERND_EINVAL, "a gradient in the logits' place needs ldd = ldz");
  const int64_t es = z_type == EXTERND_F32 ? 4 : 2;
  if (dlogits != logits && meet({logits, rows, vocab * es, ldz * es}, {dlogits, rows, vocab * es, ldd * es}))
    return fail(EXTERND_EINVAL, "the gradient must be apart from the logits or in their place");
  if (distill_workspace_bytes(rows, (int)vocab) > 0 && (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 15)))
    return fail(EXTERND_EINVAL, "workspace of externd_distill_workspace() bytes, 16-byte aligned, is needed");
  const DistillLaunch L{logits, teacher, index, weight, loss, stats, dlogits, workspace, rows, ldz, ldd,
                        (int)vocab, (int)top, z_type, t_type, index_bytes, temperature};
  HIP_OR_FAIL(distill_run(L, reinterpret_cast<hipStream_t>(stream)));
  return EXTERND_OK;
}

int externd_distill_grad(const void* logits, int z_type, int64_t rows, int64_t vocab, int64_t ldz, const float* stats,
                         const void* teacher, int t_type, const void* index, int index_bytes, int64_t top,
                         float temperature, const float* grad_loss, void* dlogits, int64_t ldd, void* stream) {
  g_last_error.clear();
  const int rc = distill_checks(logits, z_type, rows, vocab, ldz, teacher, t_type, index, index_bytes, top, temperature);
  if (rc < 0) return rc;
  if (ldd < vocab || ldd > kMaxLd) return fail(EXTERND_EINVAL, "ldd must be at least vocab (and at most 2^40)");
  if (rc == 1) return EXTERND_OK;
  if (!stats || !dlogits) return fail(EXTERND_EINVAL, "null pointer argument");
  if (dlogits == logits && ldd != ldz) return fail(EXTERND_EINVAL, "a gradient in the logits' place needs ldd = ldz");
  const int64_t es = z_type == EXTERND_F32 ? 4 : 2;
  if (dlogits != logits && meet({logits, rows, vocab * es, ldz * es}, {dlogits, rows, vocab * es, ldd * es}))
    return fail(EXTERND_EINVAL, "the gradient must be apart from the logits or in their place");
  const DistillLaunch L{logits, teacher, index, grad_loss, nullptr, const_cast<float*>(stats), dlogits, nullptr, rows, ldz,
                        ldd, (int)vocab, (int)top, z_type, t_type, index_bytes, temperature};
  HIP_OR_FAIL(distill_run(L, reinterpret_cast<hipStream_t>(stream)));
  return EXTERND_OK;
}

// ---- gradient of the factored layer

constexpr int64_t kMaxFactorSize = (int64_t)1 << 33;  // elements of a factor: a launch's threads
constexpr int64_t kMaxFactorLen = (int64_t)1 << 23;  // 128 len < 2^31: a digit's sum fits int32

int64_t externd_apply_factors_grad_workspace(int64_t k, int64_t m, int64_t n, int64_t batch) {
  if (k < 1 || m < 1 || n < 1 || k > kMaxFactorLen || m > kMaxFactorLen || n > kMaxFactorLen || batch < 0 ||
      batch > kMaxCount || k * m > kMaxFactorSize || k * n > kMaxFactorSize)
    return -1;
  return (int64_t)grad_workspace_bytes((int)k, (int)m, (int)n, batch);
}

int externd_apply_factors_grad(const uint32_t* B_packed, const uint32_t* C_packed, const float* D, int64_t k, int64_t m,
                               int64_t n, const float* X, const float* dY, int64_t batch, float* dX, float* dD,
                               void* workspace, void* stream) {
  g_last_error.clear();
  if (k < 1 || m < 1 || n < 1 || k > kMaxFactorLen || m > kMaxFactorLen || n > kMaxFactorLen)
    return fail(EXTERND_EINVAL, "need 1 <= k, m, n <= %lld", (long long)kMaxFactorLen);
  if (k * m > kMaxFactorSize || k * n > kMaxFactorSize)
    return fail(EXTERND_EINVAL, "need k m and k n <= 2^33");
  if (batch < 0 || batch > kMaxCount) return fail(EXTERND_EINVAL, "need 0 <= batch < 2^31");
  if (!dX && !dD) {
    if (batch == 0) return EXTERND_OK;
    return fail(EXTERND_EINVAL, "dX or dD must be given");
  }
  if (!B_packed || !C_packed || !D) return fail(EXTERND_EINVAL, "null pointer argument");
  if (batch > 0 && (!dY || (dD && !X))) return fail(EXTERND_EINVAL, "null pointer argument");
  if (batch > 0 && (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 15)))
    return fail(EXTERND_EINVAL, "workspace of externd_apply_factors_grad_workspace() bytes, 16-byte aligned, is needed");
  // An output over an input would be written by a launch that others of it still read.  dX in the place of
  // the vectors is none: every way reads a pass's vectors in a launch before the one that writes theirs.
  const Rows in[] = {dense(B_packed, k * ((m + 15) / 16) * 4), dense(C_packed, k * ((n + 15) / 16) * 4), dense(D, k * 4),
                     dense(X, batch * n * 4), dense(dY, batch * m * 4)};
  const Rows gx = dense(dX, batch * n * 4), gd = dense(dD, k * 4);
  const bool over_x = dX && dX == X, over_dy = dX && dX == dY && m == n;
  for (const Rows& s : in)
    if (meet(gd, s) || (meet(gx, s) && !(over_x && s.p == X) && !(over_dy && s.p == dY)))
      return fail(EXTERND_EINVAL, "dX and dD must not overlap the inputs");
  if (meet(gx, gd)) return fail(EXTERND_EINVAL, "dX and dD must not overlap");
  HIP_OR_FAIL(grad_run(B_packed, C_packed, D, (int)k, (int)m, (int)n, X, dY, batch, dX, dD, workspace,
                       reinterpret_cast<hipStream_t>(stream)));
  return EXTERND_OK;
}

}  // extern "C"
