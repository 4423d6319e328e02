// Log-probabilities of given tokens, the entropy of each row of logits and its
// likeliest ids.
//
// With m the row's largest logit, n the logits equal to it, s = sum of e^(x - m) over
// the others, l = n + s and t = sum e^(x - m) (x - m):
//   log-probability of x = (x - m) - ln l;   entropy = ln l - t / l.
// Both terms of the entropy are of one sign, so nothing cancels, and a row with
// one candidate yields exactly 0 for both.  n is counted apart, since beside 1 a small s
// would lose its digits, and with them the log-probability of a near certain token,
// ln(1 + s): ln l = ln n + log1p(s / n).
//
// A workgroup takes a row, or a part of one where there are few: it reads the
// logits once, each wave keeps m, n, s and t (rescaled when its maximum grows, about
// ln(vectors) times a row), and for the likeliest ids every 128 logits leave their
// largest.  Then the row's last workgroup joins the parts, and since the n groups
// with the largest maxima hold n logits as large as any other group's, it goes back
// for the few groups that reach them.
//
// 1024 rows of 151936 bf16 logits with 5 ids each take 65 us, 4.8 TB/s (a large copy
// reaches 5.2; vector instructions are busy 75 % of the time).  777 rows of 50257 take 22.3 for
// 15.1 of bytes: a row is seven steps in parts of three, three and one, so a third of the
// workgroups start and join for a step that is mostly past the row's end.  One fp32 row
// of 151936 with 20 ids takes 11.5, near what the call takes on the host: 19 workgroups
// of a step each, then the last of them ranks maxima, goes back for the groups and
// ranks again.  Counting n apart takes 0.3 to 1.3 us of each.
#include <cmath>
#include <new>

#include "../../include/domino_verify.h"
#include "common.h"
#include "handle.h"
#include "parts.h"
#include "vocab.h"

namespace {

constexpr int kThreads = 256;
constexpr int kVectors = 4;           // of 8 logits, in flight to a lane
constexpr int kSpan = kThreads * 8;   // logits that a workgroup reads at once
constexpr int kChunk = kVectors * kSpan;  // logits of a step of a workgroup
// Four lanes' logits of a step leave one maximum: kVectors runs of 32, kSpan apart.
constexpr int kGroups = kThreads / 4;  // of a step
constexpr int kMaxTop = 64;
constexpr int kMaxParts = 128;
constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;

struct ScoreArgs {
  const void* logits;
  int64_t row_stride;
  int32_t rows, vocab, range, parts, top;
  const int32_t* tokens;
  float* part;       // [rows][parts][4]: m, s, t in powers of two, n
  float* maxima;     // [rows][groups]
  int32_t* arrived;  // [rows] parts there are, 0 between calls
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
  float m, s, t, n;
};
// to the reference of the larger maximum m
__device__ __forceinline__ Sums refer(const Sums& a, float m) {
  if (a.m == m || a.m == -INFINITY) return a;
  const float d = fmaxf((a.m - m) * kLog2e, -200.f), f = exp2_fast(d), all = a.s + a.n;
  return Sums{m, f * all, f * (a.t + d * all), 0.f};
}
__device__ __forceinline__ Sums join(const Sums& a, const Sums& b) {
  const float m = fmaxf(a.m, b.m);
  const Sums x = refer(a, m), y = refer(b, m);
  return Sums{m, x.s + y.s, x.t + y.t, x.n + y.n};
}

// ln(n + s): with r = s / n and u = 1 + r rounded, ln(1 + r) = ln u + (r - (u - 1)) / u
__device__ __forceinline__ float log_sum(float n, float s) {
  const float r = n == 1.f ? s : s / n, u = 1.f + r;
  const float x = logf(u) + (r - (u - 1.f)) * __builtin_amdgcn_rcpf(u);
  return n == 1.f ? x : logf(n) + x;
}

// A digit of a selection by a workgroup, a bin to each thread: in the order of the
// bins (UP: from 0, otherwise from 255) the bin that holds the `need`-th element,
// and the elements of earlier bins, in *found.  The bins hold at least `need`.
struct Found {
  int bin, before, here;
};
template <bool UP>
__device__ __forceinline__ void find_bin(const int* s_bins, int* s_waves, int need, Found* found) {
  const int tid = threadIdx.x, lane = tid & 63, bin = UP ? tid : kThreads - 1 - tid;
  __syncthreads();
  const int mine = s_bins[bin];
  int upto = mine;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int x = __shfl_up(upto, d, 64);
    if (lane >= d) upto += x;
  }
  if (lane == 63) s_waves[tid >> 6] = upto;
  __syncthreads();
  for (int i = 0; i < tid >> 6; ++i) upto += s_waves[i];
  if (upto >= need && upto - mine < need) *found = Found{bin, upto - mine, mine};
  __syncthreads();
}

// One to a bin by each active lane; equal logits meet in one, so the lanes that
// share the first lane's bin are counted for it.
__device__ __forceinline__ void count_in(int* s_bins, int bin) {
  const int first = __builtin_amdgcn_readfirstlane(bin);
  const uint64_t same = __ballot(bin == first);
  if (bin != first)
    atomicAdd(s_bins + bin, 1);
  else if ((threadIdx.x & 63) == __builtin_ctzll(same))
    atomicAdd(s_bins + bin, __builtin_popcountll(same));
}

// f(logit, id) for each logit of the row above -inf
template <typename T, typename F>
__device__ __forceinline__ void each_logit(const T* p, int vocab, F f) {
  for (int v = threadIdx.x * 8; v < vocab; v += kSpan) {
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
__global__ __launch_bounds__(kThreads) void score_kernel(ScoreArgs a) {
  constexpr int kList = 256, kKeys = 1024;  // what a row's lists hold
  constexpr int kKept = 8;                  // maxima of a thread in registers
  __shared__ Sums s_sums[kThreads / 64];
  __shared__ int s_last;
  __shared__ __align__(16) union {
    float maxima[kKept * kThreads];
    uint64_t keys[kKeys];
  } s_row;
  float* const s_maxima = s_row.maxima;
  const bool local = a.parts == 1 && a.groups <= kKept * kThreads;  // the maxima need not leave the workgroup
  const int row = blockIdx.y, part = blockIdx.x, tid = threadIdx.x;
  const int lo = part * a.range, hi = min(lo + a.range, a.vocab);
  const T* const p = (const T*)a.logits + row * a.row_stride;
  float m = -INFINITY, s = 0.f, t = 0.f;  // m is the wave's
  int n = 0;
  float* const maxima = TOP ? a.maxima + (int64_t)row * a.groups + tid / 4 : nullptr;
  u32x4 raw[kVectors][8 / Elem<T>::kVec], next[kVectors][8 / Elem<T>::kVec];
  auto load = [&](int at) {
    const bool whole = at + kChunk <= hi;
#pragma unroll
    for (int u = 0; u < kVectors; ++u)
#pragma unroll
      for (int i = 0; i < 8 / Elem<T>::kVec; ++i) {
        const int v = at + u * kSpan + tid * 8 + i * Elem<T>::kVec;
        if (whole)
          __builtin_memcpy(&next[u][i], p + v, 16);
        else
          next[u][i] = load_raw<T>(p + v, hi - v);
      }
  };
  load(lo);
  for (int at = lo; at < hi; at += kChunk) {
#pragma unroll
    for (int u = 0; u < kVectors; ++u)
#pragma unroll
      for (int i = 0; i < 8 / Elem<T>::kVec; ++i) raw[u][i] = next[u][i];
    if (at + kChunk < hi) load(at + kChunk);
    float group = -INFINITY;
#pragma unroll
    for (int u = 0; u < kVectors; ++u) {
      float x[8];
#pragma unroll
      for (int i = 0; i < 8 / Elem<T>::kVec; ++i) unpack<T>(raw[u][i], x + i * Elem<T>::kVec);
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = __builtin_canonicalizef(x[j]);
      float top = largest(x);
      if (__any(top >= m)) {
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = tame(x[j]);
        top = tame(top);
        const float mn = fmaxf(m, wave_max(top));
        if (mn > m) {
          if (m > -INFINITY) {
            const float d = fmaxf((m - mn) * kLog2e, -200.f), f = exp2_fast(d), all = s + (float)n;
            t = f * (t + d * all);
            s = f * all;
            n = 0;
          }
          m = mn;
        }
        if (m > -INFINITY) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const bool equal = x[j] == m;
            n += equal;
            x[j] = equal ? -INFINITY : x[j];
          }
        }
      }
      if (TOP) group = max3(group, top, top);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        // -inf and NaN end at 2^-200, which is 0
        const float y = fmaxf((x[j] - m) * kLog2e, -200.f), e = exp2_fast(y);
        s += e;
        t = __builtin_fmaf(e, y, t);
      }
    }
    if constexpr (TOP) {
      group = fmaxf(group, __uint_as_float(other<0>(__float_as_uint(group))));
      group = fmaxf(group, __uint_as_float(other<1>(__float_as_uint(group))));
      group = tame(group);
      if ((tid & 3) == 0) {
        if (local)
          s_maxima[at / kChunk * kGroups + tid / 4] = group;
        else
          __hip_atomic_store(maxima + at / kChunk * kGroups, group, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      }
    }
  }
  const Sums own{m, wave_sum(s), wave_sum(t), wave_sum((float)n)};
  if ((tid & 63) == 0) s_sums[tid >> 6] = own;
  __syncthreads();
  if (tid < 64) {
    Sums s = s_sums[0];
#pragma unroll
    for (int i = 1; i < kThreads / 64; ++i) s = join(s, s_sums[i]);
    if (tid == 0) s_sums[0] = s;
    if (a.parts > 1 && tid == 0) {
      float* const out = a.part + ((int64_t)row * a.parts + part) * 4;
      share2(out, s.m, s.s);
      share2(out + 2, s.t, s.n);
    }
  }
  if (a.parts > 1) {
    if (!last_of(a.arrived + row, a.parts, &s_last)) return;
    if (tid < 64) {  // the parts, a lane to each
      Sums s{-INFINITY, 0.f, 0.f, 0.f};
      for (int i = tid; i < a.parts; i += 64) {
        const float* const in = a.part + ((int64_t)row * a.parts + i) * 4;
        const float2 x = shared2(in), y = shared2(in + 2);
        s = join(s, Sums{x.x, x.y, y.x, y.y});
      }
      const float top = wave_max(s.m);
      s = refer(s, top);
      s = Sums{top, wave_sum(s.s), wave_sum(s.t), wave_sum(s.n)};
      if (tid == 0) s_sums[0] = s;
    }
  } else {
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // this wave's maxima are where all see them
  }
  __syncthreads();
  const Sums sums = s_sums[0];
  m = sums.m;
  const float norm = log_sum(sums.n, sums.s);
  if (tid == 0) {
    if (a.entropy) a.entropy[row] = m == -INFINITY ? 0.f : norm - kLn2 * sums.t / (sums.n + sums.s);
    if (a.logprob) {
      const int token = a.tokens[row];
      const float x = token >= 0 && token < a.vocab ? load_tame(p + token) : -INFINITY;
      a.logprob[row] = x == -INFINITY ? -INFINITY : (x - m) - norm;
    }
  }
  if constexpr (TOP) {
    __shared__ __align__(16) float s_max[kThreads];
    __shared__ float s_bar[kThreads / 64];
    __shared__ int s_groups[kList], s_count, s_keys_n, s_best_n, s_bins[kThreads], s_waves[kThreads / 64];
    __shared__ Found s_found;
    uint64_t* const s_keys = s_row.keys;
    const float* const all = a.maxima + (int64_t)row * a.groups;
    auto maximum = [&](int g) { return __hip_atomic_load(all + g, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); };
    float kept[kKept], mine = -INFINITY;
#pragma unroll
    for (int i = 0; i < kKept; ++i) {
      const int g = i * kThreads + tid;
      kept[i] = g >= a.groups ? -INFINITY : local ? s_maxima[g] : maximum(g);
    }
#pragma unroll
    for (int i = 0; i < kKept; ++i) mine = fmaxf(mine, kept[i]);
    for (int g = kKept * kThreads + tid; g < a.groups; g += kThreads) mine = fmaxf(mine, maximum(g));
    if (tid == 0) s_count = s_keys_n = 0;
    // A bar that at least `top` logits reach: the top-th largest of what the threads
    // find largest, -inf where fewer have met one at all.  Ranked within each wave
    // first: only its best can be among the best of all.
    auto bar_of = [&](float mine) {
      __syncthreads();
      s_max[tid] = -INFINITY;
      if (tid == 0) s_best_n = 0;
      __syncthreads();
      int above = 0;
#pragma unroll
      for (int i = 0; i < 64; ++i) above += __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(mine), i)) > mine;
      const bool best = above < a.top && mine > -INFINITY;
      if (best) s_max[atomicAdd(&s_best_n, 1)] = mine;
      __syncthreads();
      const int best_n = s_best_n;
      above = 0;
#pragma unroll 4
      for (int i = 0; i < best_n; i += 4) {
        const float4 x = *(const float4*)(s_max + i);
        above += (x.x > mine) + (x.y > mine) + (x.z > mine) + (x.w > mine);
      }
      const float least = -wave_max(best && above < a.top ? -mine : -INFINITY);
      if ((tid & 63) == 0) s_bar[tid >> 6] = least;
      __syncthreads();
      return best_n < a.top ? -INFINITY : fminf(fminf(s_bar[0], s_bar[1]), fminf(s_bar[2], s_bar[3]));
    };
    float bar = bar_of(mine);
    auto list = [&](float x, int g) {
      if (x >= bar && x > -INFINITY) {
        const int at = atomicAdd(&s_count, 1);
        if (at < kList) s_groups[at] = g;
      }
    };
#pragma unroll
    for (int i = 0; i < kKept; ++i) list(kept[i], i * kThreads + tid);
    for (int g = kKept * kThreads + tid; g < a.groups; g += kThreads) list(maximum(g), g);
    __syncthreads();
    const int groups = s_count;
    // the first id of piece i of the listed groups, 8 logits each
    auto piece_at = [&](int i) {
      const int g = s_groups[i / (4 * kVectors)];
      return g / kGroups * kChunk + i / 4 % kVectors * kSpan + g % kGroups * 32 + i % 4 * 8;
    };
    if (bar == -INFINITY && groups <= kList) {
      // Fewer groups than ids asked for (a small vocabulary, a mask that leaves ids
      // in few places): a bar from their pieces (100 rows of 1500 with 64 ids
      // 19.8 us, without it 25.4).
      mine = -INFINITY;
      for (int i = tid; i < groups * 4 * kVectors; i += kThreads) {
        const int id = piece_at(i);
        float x[8];
        load_logits<T>(p + id, a.vocab - id, x);
        mine = fmaxf(mine, tame(largest(x)));
      }
      bar = bar_of(mine);
    }
    if (groups <= kList) {
#pragma unroll 2
      for (int i = tid; i < groups * 4 * kVectors; i += kThreads) {
        const int id = piece_at(i);
        float x[8];
        load_logits<T>(p + id, a.vocab - id, x);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float y = tame(x[j]);
          if (y >= bar && y > -INFINITY) {
            const int at = atomicAdd(&s_keys_n, 1);
            if (at < kKeys) s_keys[at] = pack_key(y, id + j);
          }
        }
      }
    }
    __syncthreads();
    if (groups > kList || s_keys_n > kKeys) {
      // Many equal logits, or ids in fewer groups than asked for.  The value of
      // the top-th logit is found digit by digit, and among its equals the last id
      // in the same way, each digit by a pass over the row (a row of 151936 ids of
      // four values 648 us, 300 such rows 1268; bit by bit 2270 and 4250).
      uint32_t value = 0;  // of the last logit to take, and its number among its equals
      int left = a.top, equals = 0;
      bool all = false;
      for (int shift = 24; shift >= 0 && !all; shift -= 8) {
        __syncthreads();
        s_bins[tid] = 0;
        __syncthreads();
        int met = 0;
        each_logit<T>(p, a.vocab, [&](float x, int) {
          const uint32_t y = orderable(x);
          if (shift == 24 || y >> (shift + 8) == value >> (shift + 8)) {
            count_in(s_bins, y >> shift & 255);
            ++met;
          }
        });
        if (shift == 24) {
          met = (int)wave_reduce((uint32_t)met, [](uint32_t x, uint32_t y) { return x + y; });
          if ((tid & 63) == 0) s_waves[tid >> 6] = met;
          __syncthreads();
          all = s_waves[0] + s_waves[1] + s_waves[2] + s_waves[3] <= left;
          if (all) break;
        }
        find_bin<false>(s_bins, s_waves, left, &s_found);
        const Found f = s_found;
        value |= (uint32_t)f.bin << shift;
        left -= f.before;
        equals = f.here;
      }
      int last = 0;  // id of the last of the equals
      if (!all && equals > left) {
        for (int shift = 16; shift >= 0; shift -= 8) {
          if ((a.vocab - 1) >> shift == 0) continue;
          __syncthreads();
          s_bins[tid] = 0;
          __syncthreads();
          each_logit<T>(p, a.vocab, [&](float x, int id) {
            if (orderable(x) == value && id >> (shift + 8) == last >> (shift + 8)) count_in(s_bins, id >> shift & 255);
          });
          find_bin<true>(s_bins, s_waves, left, &s_found);
          const Found f = s_found;
          last |= f.bin << shift;
          left -= f.before;
        }
      } else {
        last = a.vocab;
      }
      __syncthreads();
      if (tid == 0) s_keys_n = 0;
      __syncthreads();
      each_logit<T>(p, a.vocab, [&](float x, int id) {
        if (all || orderable(x) > value || (orderable(x) == value && id <= last)) {
          const int at = atomicAdd(&s_keys_n, 1);
          if (at < kKeys) s_keys[at] = pack_key(x, id);
        }
      });
      __syncthreads();
    }
    int n = min(s_keys_n, kKeys);
    if (n > kThreads) {
      // Many for the ranking, which takes n^2: a bar from the threads' own largest
      // leaves few (500 rows of 5003 with masks and 64 ids 19.9 us, without it 42.8).
      uint64_t mine_keys[kKeys / kThreads];
      mine = -INFINITY;
#pragma unroll
      for (int i = 0; i < kKeys / kThreads; ++i) {
        mine_keys[i] = i * kThreads + tid < n ? s_keys[i * kThreads + tid] : 0;
        if (mine_keys[i]) mine = fmaxf(mine, key_value(mine_keys[i]));
      }
      bar = bar_of(mine);
      if (tid == 0) s_keys_n = 0;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kKeys / kThreads; ++i)
        if (mine_keys[i] && key_value(mine_keys[i]) >= bar) s_keys[atomicAdd(&s_keys_n, 1)] = mine_keys[i];
      __syncthreads();
      n = s_keys_n;
    }
    // each key to the place of its rank
    for (int i = tid; i < n; i += kThreads) {
      const uint64_t key = s_keys[i];
      int rank = 0;
#pragma unroll 8
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

int steps_of(int vocab) { return (vocab + kChunk - 1) / kChunk; }

}  // namespace

struct domino_scores : HandleBase {
  domino_scores_config_t cfg;
  int cus = 256;
  float* part = nullptr;
  float* maxima = nullptr;
  int32_t* arrived = nullptr;
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
  const int most_parts = steps_of(cfg->vocab) < kMaxParts ? steps_of(cfg->vocab) : kMaxParts;
  h->part = (float*)h->take((size_t)cfg->max_rows * most_parts * 4 * sizeof(float));
  h->arrived = (int32_t*)h->take((size_t)cfg->max_rows * sizeof(int32_t));
  bool ok = h->part && h->arrived &&
            hipMemset(h->arrived, 0, (size_t)cfg->max_rows * sizeof(int32_t)) == hipSuccess;
  if (cfg->max_top) {
    h->maxima = (float*)h->take((size_t)cfg->max_rows * steps_of(cfg->vocab) * kGroups * sizeof(float));
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
static void launch_scores(const ScoreArgs& a, hipStream_t st) {
  const dim3 grid(a.parts, a.rows);
  if (a.top)
    hipLaunchKernelGGL((score_kernel<T, true>), grid, dim3(kThreads), 0, st, a);
  else
    hipLaunchKernelGGL((score_kernel<T, false>), grid, dim3(kThreads), 0, st, a);
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
  // Parts of a row, of at least a step each: as many as give each CU eight
  // workgroups (777 rows of 50257 in 3 parts 22.3 us, in 2 25.2, undivided 23.7).  For the
  // likeliest ids four, and none from two rows to a CU on, where the maxima then
  // stay in LDS (1024 rows of 151936 undivided 65.5 us, in 2 parts 78; 256 rows in 4
  // parts 26.0, undivided 26.8; one fp32 row in 19 11.5, undivided 28).
  // Ranges are whole steps: those of a quarter of one balance better but run
  // steps half empty (777 rows of 50257 27.9).
  const int steps = steps_of(f.vocab);
  int parts = !top ? (8 * h->cus + rows - 1) / rows : rows >= 2 * h->cus ? 1 : (4 * h->cus + rows - 1) / rows;
  if (parts > steps) parts = steps;
  if (parts > kMaxParts) parts = kMaxParts;
  a.range = (steps + parts - 1) / parts * kChunk;
  a.parts = (f.vocab + a.range - 1) / a.range;
  a.groups = steps * kGroups;
  a.top = top;
  a.tokens = tokens;
  a.part = h->part;
  a.maxima = h->maxima;
  a.arrived = h->arrived;
  a.logprob = logprob;
  a.entropy = entropy;
  a.ids = top_ids;
  a.values = top_logprob;
  DeviceGuard dg(h->device);
  (void)hipGetLastError();
  if (f.dtype == DOMINO_DTYPE_BF16)
    launch_scores<bf16_t>(a, (hipStream_t)stream);
  else
    launch_scores<float>(a, (hipStream_t)stream);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess)
    return say(h->err, DOMINO_ERR_HIP, "run: kernel launch failed: %s", hipGetErrorString(e));
  h->err[0] = 0;
  return DOMINO_OK;
}
