// Log-probabilities of given tokens, the entropy of each row of logits and its
// likeliest ids.
//
// With m the row's largest logit, l = sum e^(x - m) and t = sum e^(x - m) (x - m):
//   log-probability of x = (x - m) - ln l;   entropy = ln l - t / l.
// Both terms of the entropy are of one sign, so nothing cancels, and a row with
// one candidate yields exactly 0 for both.
//
// Two launches.  The first reads the logits once: a workgroup takes a part of a
// row, each wave keeps m, l and t (rescaled when its maximum grows, about
// ln(vectors) times a row), and for the likeliest ids every 32 logits leave their
// largest.  The second takes a row to a workgroup: it joins the parts, and since
// n of the groups of 32 whose maxima are the n largest hold the n largest logits,
// it goes back for those alone.
#include <cmath>
#include <new>

#include "../../include/domino_verify.h"
#include "common.h"
#include "handle.h"
#include "vocab.h"

namespace {

constexpr int kThreads = 256;
constexpr int kChunk = kThreads * 8;  // logits of a step of a workgroup
constexpr int kGroup = 32;            // logits that leave one maximum
constexpr int kMaxTop = 64;
constexpr int kMaxParts = 128;
constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;

struct ScoreArgs {
  const void* logits;
  int64_t row_stride;
  int32_t rows, vocab, range, parts, top;
  const int32_t* tokens;
  float* part;    // [rows][parts][3]: m, l, t in powers of two
  float* maxima;  // [rows][groups]
  int32_t groups;
  float* logprob;
  float* entropy;
  int32_t* ids;    // [rows][top]
  float* values;
};

// Eight logits, every NaN made a quiet one: the maximum of a signaling NaN and a
// number is NaN, of a quiet one the number.
template <typename T>
__device__ __forceinline__ void load_logits(const T* p, int n, float (&x)[8]) {
  constexpr int V = Elem<T>::kVec;
#pragma unroll
  for (int i = 0; i < 8; i += V) unpack<T>(load_raw<T>(p + i, n - i), x + i);
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = __builtin_canonicalizef(x[i]);
}
template <typename T>
__device__ __forceinline__ float load_tame(const T* p) {
  return tame(__builtin_canonicalizef(load_one(p)));
}

struct Sums {
  float m, l, t;
};
// to the reference of the larger maximum
__device__ __forceinline__ Sums join(const Sums& a, const Sums& b) {
  const float m = fmaxf(a.m, b.m);
  if (m == -INFINITY) return a;
  Sums r{m, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const Sums& s = i ? b : a;
    if (s.m == -INFINITY) continue;
    const float d = fmaxf((s.m - m) * kLog2e, -200.f), f = exp2_fast(d);
    r.l += f * s.l;
    r.t += f * (s.t + d * s.l);
  }
  return r;
}

template <typename T, bool TOP>
__global__ __launch_bounds__(kThreads) void score_kernel(ScoreArgs a) {
  __shared__ Sums s_sums[kThreads / 64];
  const int row = blockIdx.y, part = blockIdx.x, tid = threadIdx.x;
  const int lo = part * a.range, hi = min(lo + a.range, a.vocab);
  const T* const p = (const T*)a.logits + row * a.row_stride;
  float m = -INFINITY, l = 0.f, t = 0.f;  // m is the wave's
  for (int v = lo + tid * 8; v - tid * 8 < hi; v += kChunk) {
    float x[8];
    load_logits<T>(p + v, hi - v, x);
    float top = x[0];
#pragma unroll
    for (int j = 1; j < 8; ++j) top = fmaxf(top, x[j]);
    if (__any(top > m)) {
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = tame(x[j]);
      top = tame(top);
      const float mn = fmaxf(m, wave_max(top));
      if (m != -INFINITY) {
        const float d = fmaxf((m - mn) * kLog2e, -200.f), f = exp2_fast(d);
        t = f * (t + d * l);
        l *= f;
      }
      m = mn;
    }
    if constexpr (TOP) {
      float g = fmaxf(top, __uint_as_float(other<0>(__float_as_uint(top))));
      g = fmaxf(g, __uint_as_float(other<1>(__float_as_uint(g))));
      if ((tid & 3) == 0 && v < hi) a.maxima[(int64_t)row * a.groups + v / kGroup] = tame(g);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      // -inf and NaN end at 2^-200, which is 0
      const float y = fmaxf((x[j] - m) * kLog2e, -200.f), e = exp2_fast(y);
      l += e;
      t = __builtin_fmaf(e, y, t);
    }
  }
  l = wave_sum(l);
  t = wave_sum(t);
  if ((tid & 63) == 0) s_sums[tid >> 6] = Sums{m, l, t};
  __syncthreads();
  if (tid == 0) {
    Sums s = s_sums[0];
#pragma unroll
    for (int i = 1; i < kThreads / 64; ++i) s = join(s, s_sums[i]);
    float* out = a.part + ((int64_t)row * a.parts + part) * 3;
    out[0] = s.m;
    out[1] = s.l;
    out[2] = s.t;
  }
}

// counts over a workgroup
__device__ __forceinline__ int count_all(int n, int* s_count) {
  __syncthreads();
  if (threadIdx.x == 0) *s_count = 0;
  __syncthreads();
  n = (int)wave_reduce((uint32_t)n, [](uint32_t a, uint32_t b) { return a + b; });
  if ((threadIdx.x & 63) == 0) atomicAdd(s_count, n);
  __syncthreads();
  return *s_count;
}

// f(logit, id) for each logit of the row above -inf
template <typename T, typename F>
__device__ __forceinline__ void each_logit(const T* p, int vocab, F f) {
  for (int v = threadIdx.x * 8; v < vocab; v += kChunk) {
    float x[8];
    load_logits<T>(p + v, vocab - v, x);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float y = tame(x[j]);
      if (y > -INFINITY) f(y, v + j);
    }
  }
}

template <typename T, bool TOP>
__global__ __launch_bounds__(kThreads) void score_join_kernel(ScoreArgs a) {
  constexpr int kGroups = 256, kKeys = 1024;  // what a row's lists hold
  __shared__ Sums s_sums;
  __shared__ float s_max[kThreads];
  __shared__ float s_bar;
  __shared__ int s_groups[kGroups], s_count, s_keys_n;
  __shared__ uint64_t s_keys[kKeys];
  const int row = blockIdx.x, tid = threadIdx.x;
  const T* const p = (const T*)a.logits + row * a.row_stride;

  if (tid < 64) {  // the parts, a lane to each
    Sums s{-INFINITY, 0.f, 0.f};
    for (int i = tid; i < a.parts; i += 64) {
      const float* in = a.part + ((int64_t)row * a.parts + i) * 3;
      s = join(s, Sums{in[0], in[1], in[2]});
    }
    const float m = wave_max(s.m);
    const float d = s.m == -INFINITY ? -200.f : fmaxf((s.m - m) * kLog2e, -200.f), f = exp2_fast(d);
    const float t = wave_sum(f * (s.t + d * s.l)), l = wave_sum(f * s.l);
    if (tid == 0) {
      const float norm = logf(l);
      if (a.entropy) a.entropy[row] = m == -INFINITY ? 0.f : norm - kLn2 * t / l;
      if (a.logprob) {
        const int token = a.tokens[row];
        const float x = token >= 0 && token < a.vocab ? load_tame(p + token) : -INFINITY;
        a.logprob[row] = x == -INFINITY ? -INFINITY : (x - m) - norm;
      }
      s_sums = Sums{m, norm, 0.f};
    }
  }
  if constexpr (TOP) {
    // A bar that at least `top` logits reach, where so many threads have met a
    // logit at all: the top-th largest of what the threads find largest.
    const float* const maxima = a.maxima + (int64_t)row * a.groups;
    float mine = -INFINITY;
    for (int g = tid; g < a.groups; g += kThreads) mine = fmaxf(mine, maxima[g]);
    s_max[tid] = mine;
    if (tid == 0) s_count = s_keys_n = 0;
    __syncthreads();
    int above = 0;
#pragma unroll 8
    for (int i = 0; i < kThreads; ++i) above += s_max[i] > mine || (s_max[i] == mine && i < tid);
    if (above == a.top - 1) s_bar = mine;
    __syncthreads();
    const float bar = s_bar;
    for (int g = tid; g < a.groups; g += kThreads) {
      const float x = maxima[g];
      if (x >= bar && x > -INFINITY) {
        const int at = atomicAdd(&s_count, 1);
        if (at < kGroups) s_groups[at] = g;
      }
    }
    __syncthreads();
    const int groups = s_count;
    if (groups <= kGroups) {
      for (int i = tid; i < groups * kGroup; i += kThreads) {
        const int id = s_groups[i / kGroup] * kGroup + i % kGroup;
        if (id >= a.vocab) continue;
        const float x = load_tame(p + id);
        if (x >= bar && x > -INFINITY) {
          const int at = atomicAdd(&s_keys_n, 1);
          if (at < kKeys) s_keys[at] = pack_key(x, id);
        }
      }
    }
    __syncthreads();
    if (groups > kGroups || s_keys_n > kKeys) {
      // Many equal logits, or few ids left in few groups.  The bar is found bit
      // by bit, and among the logits equal to it the last id, each by a pass
      // over the row.
      uint32_t at_least = 0;
      for (int bit = 31; bit >= 0; --bit) {
        const uint32_t next = at_least | 1u << bit;
        int n = 0;
        each_logit(p, a.vocab, [&](float x, int) { n += orderable(x) >= next; });
        if (count_all(n, &s_count) >= a.top) at_least = next;
      }
      int n = 0;
      each_logit(p, a.vocab, [&](float x, int) { n += orderable(x) > at_least; });
      const int left = a.top - count_all(n, &s_count);
      int ids = 0;  // the most of the lowest ids that hold fewer than `left` equal ones
      for (int step = 1 << 30; step; step >>= 1) {
        const int next = ids + step;
        if (next >= a.vocab || next < 0) continue;
        n = 0;
        each_logit(p, a.vocab, [&](float x, int id) { n += orderable(x) == at_least && id < next; });
        if (count_all(n, &s_count) < left) ids = next;
      }
      __syncthreads();
      if (tid == 0) s_keys_n = 0;
      __syncthreads();
      each_logit(p, a.vocab, [&](float x, int id) {
        if (orderable(x) > at_least || (orderable(x) == at_least && id <= ids)) {
          const int at = atomicAdd(&s_keys_n, 1);
          if (at < kKeys) s_keys[at] = pack_key(x, id);
        }
      });
      __syncthreads();
    }
    // each key to the place of its rank
    const int n = min(s_keys_n, kKeys);
    const float m = s_sums.m, norm = s_sums.l;
    for (int i = tid; i < n; i += kThreads) {
      const uint64_t key = s_keys[i];
      int rank = 0;
      for (int j = 0; j < n; ++j) rank += s_keys[j] > key;
      if (rank < a.top) {
        a.ids[(int64_t)row * a.top + rank] = key_id(key);
        a.values[(int64_t)row * a.top + rank] = (key_value(key) - m) - norm;
      }
    }
    for (int i = n + tid; i < a.top; i += kThreads) {
      a.ids[(int64_t)row * a.top + i] = -1;
      a.values[(int64_t)row * a.top + i] = -INFINITY;
    }
  }
}

int groups_of(int vocab) { return (int)(((int64_t)vocab + kGroup - 1) / kGroup); }

// parts of a row: what gives each CU eight workgroups, of at least a step each
int parts_of(int rows, int vocab, int cus) {
  const int64_t most = ((int64_t)vocab + kChunk - 1) / kChunk;
  int64_t n = ((int64_t)8 * cus + rows - 1) / rows;
  if (n > most) n = most;
  return (int)(n > kMaxParts ? kMaxParts : n);
}

}  // namespace

struct domino_scores : HandleBase {
  domino_scores_config_t cfg;
  int cus = 256;
  float* part = nullptr;
  float* maxima = nullptr;
};

static thread_local char t_err[256] = "";

extern "C" domino_status_t domino_scores_create(const domino_scores_config_t* cfg, domino_scores_t** out) {
  if (!out) return say(t_err, DOMINO_ERR_INVALID_ARG, "create: out is NULL");
  *out = nullptr;
  if (!cfg) return say(t_err, DOMINO_ERR_INVALID_ARG, "create: cfg is NULL");
  if (cfg->vocab < 1 || cfg->max_rows < 1)
    return say(t_err, DOMINO_ERR_INVALID_CONFIG, "create: vocab and max_rows must be positive");
  if (cfg->max_top < 0 || cfg->max_top > kMaxTop)
    return say(t_err, DOMINO_ERR_INVALID_CONFIG, "create: max_top must be in [0, %d]", kMaxTop);
  if (cfg->dtype != DOMINO_DTYPE_BF16 && cfg->dtype != DOMINO_DTYPE_FP32)
    return say(t_err, DOMINO_ERR_INVALID_CONFIG,
               "create: dtype must be DOMINO_DTYPE_BF16 or DOMINO_DTYPE_FP32");
  if (cfg->vocab > 1 << 24)
    return say(t_err, DOMINO_ERR_UNSUPPORTED, "create: vocab must be at most 2^24 (got %d)", cfg->vocab);
  if (cfg->max_rows > 65535)
    return say(t_err, DOMINO_ERR_UNSUPPORTED, "create: at most 65535 rows");
  int dev = 0;
  domino_status_t st = check_device(t_err, &dev);
  if (st != DOMINO_OK) return st;
  domino_scores* h = new (std::nothrow) domino_scores();
  if (!h) return say(t_err, DOMINO_ERR_OUT_OF_MEMORY, "create: out of host memory");
  h->cfg = *cfg;
  h->device = dev;
  if (hipDeviceGetAttribute(&h->cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess) {
    (void)hipGetLastError();
    h->cus = 256;
  }
  h->part = (float*)h->take(((size_t)8 * h->cus + cfg->max_rows) * 3 * sizeof(float));
  bool ok = h->part != nullptr;
  if (cfg->max_top) {
    h->maxima = (float*)h->take((size_t)cfg->max_rows * groups_of(cfg->vocab) * sizeof(float));
    ok = ok && h->maxima;
  }
  if (!ok || hipDeviceSynchronize() != hipSuccess) {
    (void)hipGetLastError();
    h->release();
    delete h;
    return say(t_err, DOMINO_ERR_OUT_OF_MEMORY, "create: workspace allocation failed");
  }
  *out = h;
  return DOMINO_OK;
}

extern "C" void domino_scores_destroy(domino_scores_t* h) {
  if (!h) return;
  h->release();
  delete h;
}

extern "C" const char* domino_scores_last_error(const domino_scores_t* h) { return h ? h->err : t_err; }

template <typename T>
static hipError_t launch_scores(const ScoreArgs& a, hipStream_t st) {
  const dim3 grid(a.parts, a.rows);
  if (a.top)
    hipLaunchKernelGGL((score_kernel<T, true>), grid, dim3(kThreads), 0, st, a);
  else
    hipLaunchKernelGGL((score_kernel<T, false>), grid, dim3(kThreads), 0, st, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;  // the join would follow the parts of an earlier call
  if (a.top)
    hipLaunchKernelGGL((score_join_kernel<T, true>), dim3(a.rows), dim3(kThreads), 0, st, a);
  else
    hipLaunchKernelGGL((score_join_kernel<T, false>), dim3(a.rows), dim3(64), 0, st, a);
  return hipGetLastError();
}

extern "C" domino_status_t domino_scores_run(domino_scores_t* h, const void* logits, int64_t row_stride, int32_t rows,
                                             const int32_t* tokens, int32_t top, float* logprob, float* entropy,
                                             int32_t* top_ids, float* top_logprob, void* stream) {
  if (!h) return DOMINO_ERR_INVALID_ARG;
  const domino_scores_config_t& f = h->cfg;
  const int elem = f.dtype == DOMINO_DTYPE_BF16 ? 2 : 4;
  if (rows < 0 || rows > f.max_rows)
    return say(h->err, DOMINO_ERR_INVALID_ARG, "run: rows %d outside [0, %d]", rows, f.max_rows);
  if (top < 0 || top > f.max_top)
    return say(h->err, DOMINO_ERR_INVALID_ARG, "run: top %d outside [0, %d]", top, f.max_top);
  if (row_stride < 0) return say(h->err, DOMINO_ERR_INVALID_ARG, "run: row_stride must be >= 0");
  if (rows == 0) return DOMINO_OK;
  if ((tokens == nullptr) != (logprob == nullptr))
    return say(h->err, DOMINO_ERR_INVALID_ARG, "run: tokens and logprob must be given together");
  if (top && (!top_ids || !top_logprob))
    return say(h->err, DOMINO_ERR_INVALID_ARG, "run: top needs top_ids and top_logprob");
  if (!logits || (uintptr_t)logits % elem)
    return say(h->err, DOMINO_ERR_INVALID_ARG, "run: logits must be non-NULL and aligned to their type");
  if (((uintptr_t)tokens | (uintptr_t)logprob | (uintptr_t)entropy | (uintptr_t)top_ids | (uintptr_t)top_logprob) & 3)
    return say(h->err, DOMINO_ERR_INVALID_ARG, "run: tokens and outputs must be 4-byte aligned");
  if (!logprob && !entropy && !top) return DOMINO_OK;
  ScoreArgs a{};
  a.logits = logits;
  a.row_stride = row_stride;
  a.rows = rows;
  a.vocab = f.vocab;
  const int parts = parts_of(rows, f.vocab, h->cus);
  a.range = ((f.vocab + parts - 1) / parts + kChunk - 1) / kChunk * kChunk;
  a.parts = (f.vocab + a.range - 1) / a.range;
  a.top = top;
  a.tokens = tokens;
  a.part = h->part;
  a.maxima = h->maxima;
  a.groups = groups_of(f.vocab);
  a.logprob = logprob;
  a.entropy = entropy;
  a.ids = top_ids;
  a.values = top_logprob;
  DeviceGuard dg(h->device);
  (void)hipGetLastError();
  const hipError_t e = f.dtype == DOMINO_DTYPE_BF16 ? launch_scores<bf16_t>(a, (hipStream_t)stream)
                                                    : launch_scores<float>(a, (hipStream_t)stream);
  if (e != hipSuccess)
    return say(h->err, DOMINO_ERR_HIP, "run: kernel launch failed: %s", hipGetErrorString(e));
  h->err[0] = 0;
  return DOMINO_OK;
}
