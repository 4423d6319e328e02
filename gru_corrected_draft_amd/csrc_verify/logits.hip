// Rules on the target's logits (penalties, biases, grammar masks), alone and
// fused with the acceptance of a draft block.
//
// The vocabulary is cut into ranges; a workgroup takes one range of one
// request for all of the request's rows, so that what the rows share (the
// history's counts, the biases, the noise) is put into LDS once.
//
// Few ids of a range are touched by a penalty or a bias, and the division of the
// repetition penalty and the look-ups are paid for them alone.  A bitmap tells
// which they are.  Where logits are written (bound by memory), a lane takes the
// touched ones of its vector one by one while they are in registers: going back
// for them wrote their lines twice, and 64 blocks of 151936 ids with 4096 tokens
// of history took 212 us against 137.  Where they are not (bound by arithmetic),
// the pass leaves touched ids out and each row takes them afterwards from a list,
// a lane to each: taken in the pass, for a lane or two of a wave at a time, they
// made 64 greedy blocks with that history take 188 us against 137, which has
// since come to 113.  Counting uses
// integer atomics in LDS and the list is in the order of the ids, so nothing
// depends on the order of arrival.
#include <cmath>
#include <new>

#include "../../include/domino_verify.h"
#include "common.h"
#include "handle.h"

namespace {

constexpr int kThreads = 1024;
constexpr int kWaves = kThreads / 64;
constexpr int kMaxRows = 64;
constexpr uint32_t kPrompt = 0x80000000u;  // id stands in the prompt
constexpr uint32_t kDrafted = 0x40000000u;  // id is one of the proposals
constexpr uint32_t kCount = 0x3FFFFFFFu;

struct LogitsArgs {
  const void* logits;
  int64_t req_stride, row_stride;
  int32_t requests, rows, vocab;
  const int32_t* draft;
  int64_t draft_stride;
  const int32_t* draft_len;
  const int32_t* history;
  int64_t history_stride;
  int32_t history_width;
  const int32_t* history_len;
  const int32_t* prompt_len;
  const float* repetition;
  const float* frequency;
  const float* presence;
  const int32_t* bias_ids;
  const float* bias_values;
  int64_t bias_stride;
  int32_t bias_width;
  const int32_t* bias_len;
  const uint32_t* mask;
  int64_t mask_req, mask_row;
  int32_t range;     // ids of a range, a multiple of 64
  int32_t row_slots, parts;  // rows taken at once, waves to a row
  // process
  void* out;
  int64_t out_req, out_row;
  // verify
  const float* temperature;
  const float* accept_u;
  int64_t accept_stride;
  const float* noise;
  int64_t noise_stride;
  struct RowPart* partial;  // [requests][rows][ranges * parts]
  float* drafted;           // [requests][rows] processed logit of the row's proposal
  int32_t* out_tokens;
  int32_t* out_accepted;
  float* out_logprob;
};

// What one wave knows of a row: a reference m, the sum of e^((x - m) / T), and
// the best candidate: its score, its logit (a score less T ln E is not quite the
// logit, by an ulp over T of its log-probability) and its id (kNone: no candidate).
struct RowPart {
  float m, s, best, logit;
  int32_t id;
};
constexpr int32_t kNone = 0x7FFFFFFF;

__device__ __forceinline__ int clip_len(const int32_t* len, int b, int width) {
  if (!len) return width;
  const int n = len[b];
  return n < 0 ? 0 : (n > width ? width : n);
}

template <typename T>
struct Elem;
template <>
struct Elem<float> {
  static constexpr int kVec = 4;
};
template <>
struct Elem<bf16_t> {
  static constexpr int kVec = 8;
};

// kVec consecutive logits as they lie in memory.  Rows of an odd vocabulary are
// aligned to the element only; the copy still compiles to one 16-byte load,
// which the memory path takes at any alignment.  Past the n that there are, -inf.
template <typename T>
__device__ __forceinline__ u32x4 load_raw(const T* p, int n) {
  constexpr int V = Elem<T>::kVec;
  u32x4 raw;
  if (n >= V) {
    __builtin_memcpy(&raw, p, 16);
    return raw;
  }
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    if constexpr (sizeof(T) == 2) {
      const uint32_t lo = 2 * w < n ? p[2 * w] : 0xFF80u, hi = 2 * w + 1 < n ? p[2 * w + 1] : 0xFF80u;
      raw[w] = lo | hi << 16;
    } else {
      raw[w] = w < n ? __float_as_uint(p[w]) : 0xFF800000u;
    }
  }
  return raw;
}
template <typename T>
__device__ __forceinline__ void unpack(const u32x4& raw, float* x) {
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    if constexpr (sizeof(T) == 2) {
      x[2 * w] = __uint_as_float(raw[w] << 16);
      x[2 * w + 1] = __uint_as_float(raw[w] & 0xFFFF0000u);
    } else {
      x[w] = __uint_as_float(raw[w]);
    }
  }
}
__device__ __forceinline__ float load_one(const bf16_t* p) { return bf16_to_f32(*p); }
__device__ __forceinline__ float load_one(const float* p) { return *p; }

// element j of a vector that stays in registers
template <typename T>
__device__ __forceinline__ float element(const u32x4& raw, int j) {
  const int word = sizeof(T) == 2 ? j >> 1 : j;
  uint32_t r = raw[0];
#pragma unroll
  for (int w = 1; w < 4; ++w) r = word == w ? raw[w] : r;
  if constexpr (sizeof(T) == 2) r = j & 1 ? r & 0xFFFF0000u : r << 16;
  return __uint_as_float(r);
}

__device__ __forceinline__ bf16_t to_bf16(float x) {
  return __builtin_bit_cast(uint16_t, (__bf16)x);
}

template <typename T>
__device__ __forceinline__ void replace(u32x4& raw, int j, float x) {
  const int word = sizeof(T) == 2 ? j >> 1 : j;
  uint32_t keep = 0, put = __float_as_uint(x);
  if constexpr (sizeof(T) == 2) {
    keep = j & 1 ? 0x0000FFFFu : 0xFFFF0000u;
    put = (uint32_t)to_bf16(x) << (j & 1 ? 16 : 0);
  }
#pragma unroll
  for (int w = 0; w < 4; ++w) raw[w] = word == w ? (raw[w] & keep) | put : raw[w];
}


// the largest fp32 number for +inf, -inf for NaN
__device__ __forceinline__ float tame(float x) {
  return fminf(fmaxf(x, -INFINITY), 3.402823466e38f);
}

// all ones or none, as bit j of x.  Hidden from the compiler, which otherwise
// tests the bit once more for what the ones keep (five instructions for a masked
// logit in place of two).
__device__ __forceinline__ uint32_t spread(uint32_t x, int j) {
  uint32_t m = (uint32_t)__builtin_amdgcn_sbfe((int)x, j, 1);
  asm("" : "+v"(m));
  return m;
}

// -inf where bit j of `out` is set
__device__ __forceinline__ float masked(float x, uint32_t out, int j) {
  const uint32_t m = spread(out, j);
  return __uint_as_float((m & 0xFF800000u) | (~m & __float_as_uint(x)));
}

// e^x's power of two; results below 2^-126 become zero
__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

__device__ __forceinline__ float temperature_of(const LogitsArgs& a, int b) {
  const float t = a.temperature ? a.temperature[b] : 0.f;
  return t > 0.f ? fminf(fmaxf(t, 1e-30f), 1e30f) : 0.f;
}

// The largest of n; a quiet NaN is passed over, a signaling one takes its two
// neighbours with it.  Written out because fmaxf first makes each operand
// canonical, one more instruction apiece.
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("v_max3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "v"(c));
  return r;
}
template <int N>
__device__ __forceinline__ float largest(const float (&x)[N]) {
  float top = max3(x[0], x[1], x[2]);
#pragma unroll
  for (int j = 3; j + 1 < N; j += 2) top = max3(top, x[j], x[j + 1]);
  return max3(top, x[N - 1], x[N - 1]);
}

// Sum of the exponentials 2^((x - m) c).  From the difference: m c taken out of
// a fused product would be one instruction less apiece, but its rounding leaves
// the only candidate of a row a log-probability of not quite 0.
template <int N>
__device__ __forceinline__ float sum_exp(const float (&x)[N], float m, float c) {
  float e[N];
#pragma unroll
  for (int j = 0; j < N; ++j) e[j] = exp2_fast((x[j] - m) * c);
#pragma unroll
  for (int n = N / 2; n; n /= 2)
#pragma unroll
    for (int j = 0; j < n; ++j) e[j] += e[j + n];
  return e[0];
}

// Lane exchange for reductions over a wave: neighbours, pairs, halves of eight
// and sixteen by data-parallel moves, then halves of 32 and 64 by swaps.
template <int STEP>
__device__ __forceinline__ uint32_t other(uint32_t x) {
  if constexpr (STEP == 0) return __builtin_amdgcn_update_dpp(x, x, 0xB1, 0xF, 0xF, false);   // quad_perm 1 0 3 2
  if constexpr (STEP == 1) return __builtin_amdgcn_update_dpp(x, x, 0x4E, 0xF, 0xF, false);   // quad_perm 2 3 0 1
  if constexpr (STEP == 2) return __builtin_amdgcn_update_dpp(x, x, 0x141, 0xF, 0xF, false);  // row_half_mirror
  if constexpr (STEP == 3) return __builtin_amdgcn_update_dpp(x, x, 0x140, 0xF, 0xF, false);  // row_mirror
  return x;
}
template <typename F>
__device__ __forceinline__ uint32_t wave_reduce(uint32_t x, F f) {
  x = f(x, other<0>(x));
  x = f(x, other<1>(x));
  x = f(x, other<2>(x));
  x = f(x, other<3>(x));
  const auto a = __builtin_amdgcn_permlane16_swap(x, x, false, false);
  x = f(a[0], a[1]);
  const auto b = __builtin_amdgcn_permlane32_swap(x, x, false, false);
  return f(b[0], b[1]);
}
__device__ __forceinline__ float wave_max(float x) {
  return __uint_as_float(wave_reduce(__float_as_uint(x), [](uint32_t a, uint32_t b) {
    return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
  }));
}
__device__ __forceinline__ float wave_sum(float x) {
  return __uint_as_float(wave_reduce(__float_as_uint(x), [](uint32_t a, uint32_t b) {
    return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
  }));
}
__device__ __forceinline__ int wave_min(int x) {
  return (int)wave_reduce((uint32_t)x, [](uint32_t a, uint32_t b) { return (uint32_t)min((int)a, (int)b); });
}

// x of the first lane where `mine` holds (some lane's has to)
__device__ __forceinline__ float of_lane_with(float x, bool mine) {
  return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(x), __builtin_ctzll(__ballot(mine))));
}

// LDS of a workgroup: counts, last bias entry, list and bitmap of touched ids
struct Touched {
  uint32_t* count;   // [range]
  uint32_t* bias;    // [range] entry + 1
  uint32_t* bits;    // [range / 32]
  uint16_t* list;    // [range] offsets, ascending
  int n;
};

template <bool LIST>
__device__ __forceinline__ void build_touched(const LogitsArgs& a, int b, int lo, int ids,
                                              bool counts, bool biases, int n_draft,
                                              const int* s_draft, int* s_wave, Touched& t) {
  const int tid = threadIdx.x, lane = tid & 63, w = wave_index();
  for (int i = tid; i < a.range; i += kThreads) {
    t.count[i] = 0;
    if (biases) t.bias[i] = 0;
  }
  __syncthreads();
  if (counts && a.history) {
    const int len = clip_len(a.history_len, b, a.history_width);
    const int prompt = a.prompt_len ? clip_len(a.prompt_len, b, a.history_width) : 0;
    const int32_t* h = a.history + b * a.history_stride;
    for (int i0 = tid; i0 < len; i0 += 4 * kThreads) {
      uint32_t id[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) id[u] = i0 + u * kThreads < len ? (uint32_t)h[i0 + u * kThreads] : ~0u;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const uint32_t off = id[u] - (uint32_t)lo;
        if (i0 + u * kThreads < len && off < (uint32_t)ids) {
          if (i0 + u * kThreads < prompt)
            atomicOr(&t.count[off], kPrompt);
          else
            atomicAdd(&t.count[off], 1u);
        }
      }
    }
  }
  if (counts && tid < n_draft) {
    const uint32_t off = (uint32_t)s_draft[tid] - (uint32_t)lo;
    if (off < (uint32_t)ids) atomicOr(&t.count[off], kDrafted);
  }
  if (biases) {
    const int len = clip_len(a.bias_len, b, a.bias_width);
    const int32_t* h = a.bias_ids + b * a.bias_stride;
    for (int i = tid; i < len; i += kThreads) {
      const uint32_t off = (uint32_t)h[i] - (uint32_t)lo;
      if (off < (uint32_t)ids) atomicMax(&t.bias[off], (uint32_t)i + 1);
    }
  }
  __syncthreads();
  // each wave compacts a run of 64-id groups; the runs follow one another
  const int groups = a.range / 64, per = (groups + kWaves - 1) / kWaves;
  const int g0 = w * per, g1 = min(g0 + per, groups);
  int total = 0;
  for (int g = g0; g < g1; ++g) {
    const int i = g * 64 + lane;
    const uint64_t hit = __ballot(t.count[i] != 0 || (biases && t.bias[i] != 0));
    if (lane < 2) t.bits[2 * g + lane] = (uint32_t)(hit >> (32 * lane));
    total += __popcll(hit);
  }
  if (!LIST) {
    __syncthreads();
    return;
  }
  if (lane == 0) s_wave[w] = total;
  __syncthreads();
  int at = 0, all = 0;
  for (int i = 0; i < kWaves; ++i) {
    if (i < w) at += s_wave[i];
    all += s_wave[i];
  }
  for (int g = g0; g < g1; ++g) {
    const int i = g * 64 + lane;
    const bool hit = t.count[i] != 0 || (biases && t.bias[i] != 0);
    const uint64_t m = __ballot(hit);
    if (hit) t.list[at + __popcll(m & ((1ull << lane) - 1))] = (uint16_t)i;
    at += __popcll(m);
  }
  t.n = all;
  __syncthreads();
}

// the rules of one touched id on row t
struct Rules {
  float repetition, frequency, presence;
  bool has_repetition;
  const float* bias;
  const int* draft;
  int n_draft;
};

__device__ __forceinline__ float touched_logit(float x, uint32_t c, uint32_t entry, int id, int t,
                                               const Rules& r) {
  uint32_t n = c & kCount;
  if (c & kDrafted) {
    const int before = min(t, r.n_draft);
    for (int i = 0; i < before; ++i) n += r.draft[i] == id;
  }
  if (r.has_repetition && (n > 0 || (c & kPrompt))) x = x > 0.f ? x / r.repetition : __fmul_rn(x, r.repetition);
  x = __fsub_rn(x, __fmul_rn(r.frequency, (float)n));
  x = __fsub_rn(x, n > 0 ? r.presence : 0.f);
  if (entry) x = __fadd_rn(x, r.bias[entry - 1]);
  return x;
}

// Reads logits once; writes them (process) or keeps each row's statistics
// (verify): m and s = sum e^((x - m) / T), rescaled as m grows, and the largest
// x - T ln E with its id, which falls on id v with the probability e^(x_v / T) /
// sum e^(x / T).  Measured on 64 blocks of 16 rows of 151936 bf16 logits:
//   process, history, biases, masks   156 us, 643 MB, 4.1 TB/s (a large copy
//                                     5.2): memory
//   verify, greedy, no rules          71 us, 311 MB, 4.4 TB/s
//   verify, history, masks, T > 0     136 us: vector instructions, busy 82 % of
//                                     the time; touched ids read again bring the
//                                     bytes from 370 to 563 MB
// and on one block of fp32 logits, where starting and joining are most, 14.0.
template <typename T, bool VERIFY, bool TOUCH>
__global__ __launch_bounds__(kThreads, 8) void logits_kernel(LogitsArgs a) {
  constexpr int V = Elem<T>::kVec;
  extern __shared__ uint32_t dyn[];
  __shared__ int s_draft[kMaxRows];
  __shared__ int s_wave[kWaves];
  const int tid = threadIdx.x, lane = tid & 63, w = wave_index();
  // requests vary fastest: low ids are the frequent ones in most vocabularies,
  // so the ranges with the most touched ids start first
  const int b = blockIdx.x, lo = blockIdx.y * a.range;
  const int ids = min(a.range, a.vocab - lo);
  const bool counts = TOUCH && (a.repetition || a.frequency || a.presence);
  const bool biases = TOUCH && a.bias_ids;
  const int n_draft = a.draft ? clip_len(a.draft_len, b, a.rows - 1) : 0;
  if (tid < kMaxRows) s_draft[tid] = tid < n_draft ? a.draft[b * a.draft_stride + tid] : -1;
  const float temp = VERIFY ? temperature_of(a, b) : 0.f;

  Touched t;
  uint32_t* at = dyn;
  float* noise = nullptr;
  if (VERIFY && a.noise) {
    noise = (float*)at;
    at += a.range;
  }
  if (TOUCH) {
    t.count = at;
    at += a.range;
    t.bias = at;
    if (biases) at += a.range;
    t.bits = at;
    at += a.range / 32;
    t.list = (uint16_t*)at;
  }
  t.n = 0;
  if (VERIFY && temp > 0.f) {
    const float* e = a.noise + b * a.noise_stride + lo;
    for (int i = tid; i < ids; i += kThreads) noise[i] = temp * logf(e[i]);
  }
  __syncthreads();
  if (TOUCH) build_touched<VERIFY>(a, b, lo, ids, counts, biases, n_draft, s_draft, s_wave, t);

  Rules rules;
  rules.has_repetition = a.repetition != nullptr;
  rules.repetition = a.repetition ? a.repetition[b] : 1.f;
  rules.frequency = a.frequency ? a.frequency[b] : 0.f;
  rules.presence = a.presence ? a.presence[b] : 0.f;
  rules.bias = biases ? a.bias_values + b * a.bias_stride : nullptr;
  rules.draft = s_draft;
  rules.n_draft = n_draft;

  // A wave takes one row at a time, or one of `parts` contiguous pieces of it.
  const int slot = w / a.parts, part = w - slot * a.parts;
  const int rows = VERIFY ? n_draft + 1 : a.rows;
  const float c = VERIFY ? 1.44269504088896340736f / (temp > 0.f ? temp : 1.f) : 0.f;
  const bool sums = VERIFY && (temp > 0.f || a.out_logprob);
  if (slot >= a.row_slots) return;
  const int piece = ((ids + a.parts - 1) / a.parts + 63) / 64 * 64;
  const int begin = min(part * piece, ids), end = min(begin + piece, ids);
  // the piece's touched ids
  int e0 = 0, e1 = t.n;
  if (VERIFY && TOUCH && a.parts > 1) {
    for (int hi = t.n; e0 < hi;) {
      const int mid = (e0 + hi) >> 1;
      if (t.list[mid] < begin)
        e0 = mid + 1;
      else
        hi = mid;
    }
    e1 = e0;
    for (int hi = t.n; e1 < hi;) {
      const int mid = (e1 + hi) >> 1;
      if (t.list[mid] < end)
        e1 = mid + 1;
      else
        hi = mid;
    }
  }
  // Loads in flight for a lane.  With touched ids to look after, a fourth spills
  // registers, and 64 sampled blocks take 150 us against 131.
  constexpr int AHEAD = VERIFY && TOUCH ? 3 : 4;
  for (int row = slot; row < rows; row += a.row_slots) {
    const T* src = (const T*)a.logits + b * a.req_stride + row * a.row_stride + lo;
    const uint32_t* mask = a.mask ? a.mask + b * a.mask_req + row * a.mask_row + lo / 32 : nullptr;
    T* dst = VERIFY ? nullptr : (T*)a.out + b * a.out_req + row * a.out_row + lo;
    const int proposal = VERIFY && row < n_draft ? s_draft[row] : -1;
    const int own = proposal >= lo && proposal < lo + ids ? proposal - lo : -1;
    float* const own_logit = VERIFY ? a.drafted + b * a.rows + row : nullptr;
    // Reference of the exponents: a logit met, at most 16 powers of two below
    // the largest, so that the sum is seldom rescaled.
    float m = -INFINITY, s = 0.f, best = -INFINITY;
    int where = -1;  // vector of the best candidate
    for (int i0 = begin + lane * V; i0 < end; i0 += AHEAD * 64 * V) {
      u32x4 raw[AHEAD];
      uint32_t out[AHEAD];
      // the wave's last vector of this turn is whole: no lane needs a check
      if (i0 - lane * V + AHEAD * 64 * V <= min(end, ids)) {
#pragma unroll
        for (int u = 0; u < AHEAD; ++u) __builtin_memcpy(&raw[u], src + i0 + u * 64 * V, 16);
#pragma unroll
        for (int u = 0; u < AHEAD; ++u) {
          const int i = i0 + u * 64 * V;
          out[u] = mask ? ~(mask[(uint32_t)i >> 5] >> (i & 31)) : 0u;
        }
      } else {
#pragma unroll
        for (int u = 0; u < AHEAD; ++u) {
          const int i = i0 + u * 64 * V;
          if (i < end) {
            raw[u] = load_raw<T>(src + i, ids - i);
            out[u] = mask ? ~(mask[(uint32_t)i >> 5] >> (i & 31)) : 0u;
          }
        }
      }
#pragma unroll
      for (int u = 0; u < AHEAD; ++u) {
        const int i = i0 + u * 64 * V;
        if (i >= end) break;
        if constexpr (!VERIFY) {
          if (TOUCH) {
            uint32_t hit = t.bits[(uint32_t)i >> 5] >> (i & 31) & ~out[u] & ((1u << V) - 1);
            while (hit) {
              const int j = __builtin_ctz(hit), off = i + j;
              hit &= hit - 1;
              replace<T>(raw[u], j, touched_logit(element<T>(raw[u], j), t.count[off], biases ? t.bias[off] : 0u,
                                                  lo + off, row, rules));
            }
          }
          if (out[u] & ((1u << V) - 1)) {
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              if constexpr (sizeof(T) == 2) {
                const uint32_t lo_ = spread(out[u], 2 * w) & 0xFFFFu;
                const uint32_t hi_ = spread(out[u], 2 * w + 1) << 16;
                const uint32_t m = lo_ | hi_;
                raw[u][w] = (m & 0xFF80FF80u) | (~m & raw[u][w]);
              } else {
                raw[u][w] = __float_as_uint(masked(__uint_as_float(raw[u][w]), out[u], w));
              }
            }
          }
          if (i + V <= ids) {
            __builtin_memcpy(dst + i, &raw[u], 16);
          } else {
#pragma unroll
            for (int j = 0; j < V; ++j)
              if (i + j < ids) {
                if constexpr (sizeof(T) == 2)
                  dst[i + j] = (bf16_t)(raw[u][j / 2] >> (16 * (j & 1)));
                else
                  dst[i + j] = __uint_as_float(raw[u][j]);
              }
          }
        } else {
          uint32_t touched = 0;
          if (TOUCH) touched = t.bits[(uint32_t)i >> 5] >> (i & 31);
          float x[V];
          unpack<T>(raw[u], x);
          if ((out[u] | touched) & ((1u << V) - 1)) {
#pragma unroll
            for (int j = 0; j < V; ++j) x[j] = masked(x[j], out[u] | touched, j);
          }
          bool nan = false;
#pragma unroll
          for (int j = 0; j < V; j += 2) nan |= __builtin_isunordered(x[j], x[j + 1]);
          float top = largest<V>(x);
          if (nan || top == INFINITY) {
#pragma unroll
            for (int j = 0; j < V; ++j) x[j] = tame(x[j]);
            top = largest<V>(x);
          }
          if (sums) {
            if ((top - m) * c > 16.f) {  // also the first time, where m is -inf
              s *= exp2_fast((m - top) * c);
              m = top;
            }
            if (m > -INFINITY) s += sum_exp<V>(x, m, c);
          }
          if ((uint32_t)(own - i) < (uint32_t)V) {
#pragma unroll
            for (int j = 0; j < V; ++j)
              if (own - i == j) {
                // a touched proposal is written from the list below
                if (!((touched >> j) & 1)) *own_logit = x[j];
                x[j] = -INFINITY;
              }
            top = largest<V>(x);
          }
          if (temp > 0.f) {
            // -inf stays -inf, and a NaN is passed over by the maximum
#pragma unroll
            for (int j = 0; j < V; j += 4) {
              const float4 g = *reinterpret_cast<const float4*>(noise + i + j);
              x[j] -= g.x;
              x[j + 1] -= g.y;
              x[j + 2] -= g.z;
              x[j + 3] -= g.w;
            }
            top = largest<V>(x);
          }
          if (top > best) {
            best = top;
            where = i;
          }
        }
      }
    }
    int id = kNone;
    float logit = 0.f;
    if constexpr (VERIFY) {
      // exact id of this lane's best candidate: the first of its vector
      if (where >= 0) {
        float x[V];
        unpack<T>(load_raw<T>(src + where, ids - where), x);
        uint32_t gone = mask ? ~(mask[where / 32] >> (where % 32)) : 0u;
        if (TOUCH) gone |= t.bits[where / 32] >> (where % 32);
#pragma unroll
        for (int j = V - 1; j >= 0; --j) {
          float y = tame(x[j]);
          if (((gone >> j) & 1) || where + j == own) continue;
          const float l = y;
          if (temp > 0.f) y -= noise[where + j];
          if (y == best) {
            id = lo + where + j;
            logit = l;
          }
        }
      }
    }
    if (VERIFY && TOUCH) {
      for (int k0 = e0 + lane; k0 < e1; k0 += AHEAD * 64) {
        int off[AHEAD];
        float x[AHEAD];
        bool in[AHEAD];
#pragma unroll
        for (int u = 0; u < AHEAD; ++u) {
          in[u] = k0 + u * 64 < e1;
          if (in[u]) {
            off[u] = t.list[k0 + u * 64];
            x[u] = load_one(src + off[u]);
            if (mask) in[u] = (mask[off[u] / 32] >> (off[u] % 32)) & 1;
            if (!in[u] && off[u] == own) *own_logit = -INFINITY;
          }
        }
#pragma unroll
        for (int u = 0; u < AHEAD; ++u) {
          if (!in[u]) continue;
          float y = touched_logit(x[u], t.count[off[u]], biases ? t.bias[off[u]] : 0u, lo + off[u], row, rules);
          y = tame(y);
          if (off[u] == own) *own_logit = y;
          if (y == -INFINITY) continue;
          if (sums) {
            if ((y - m) * c > 16.f) {
              s *= exp2_fast((m - y) * c);
              m = y;
            }
            s += exp2_fast((y - m) * c);
          }
          if (off[u] == own) continue;
          const float l = y;
          if (temp > 0.f) y -= noise[off[u]];
          if (y > best || (y == best && lo + off[u] < id)) {
            best = y;
            id = lo + off[u];
            logit = l;
          }
        }
      }
    }
    if constexpr (VERIFY) {
      if (sums) {
        const float all = wave_max(m);
        if (all > -INFINITY) s = wave_sum(s * exp2_fast((m - all) * c));
        m = all;
      }
      const float most = wave_max(best);
      const int mine = best == most ? id : kNone;
      id = wave_min(mine);
      best = most;
      logit = of_lane_with(logit, mine == id);
      if (lane == 0)
        a.partial[((int64_t)b * a.rows + row) * ((int64_t)gridDim.y * a.parts) +
                  (int64_t)blockIdx.y * a.parts + part] = RowPart{m, s, best, logit, id};
    }
  }
}

// ln e^((x - m) / T) / s, above 0 only by roundings
__device__ __forceinline__ float log_probability(float x, float m, float scale, float ln_s) {
  return fminf((x - m) / scale - ln_s, 0.f);
}

// One workgroup per request joins the parts of its rows, walks the proposals
// and writes the outputs.  5 us, most of it the launch and two ways to memory
// and back; done by the last workgroup of the launch before instead, it took
// registers from the pass (64 blocks 155 us against 141, one block 15.0 against
// 13.5).
__global__ __launch_bounds__(1024) void accept_kernel(LogitsArgs a, int parts) {
  __shared__ float s_lse[kMaxRows], s_m[kMaxRows], s_logit[kMaxRows];
  __shared__ int s_id[kMaxRows], s_stands[kMaxRows];
  const int b = blockIdx.x, lane = threadIdx.x & 63, w = wave_index();
  const int n = a.draft ? clip_len(a.draft_len, b, a.rows - 1) : 0;
  const float temp = temperature_of(a, b);
  const float scale = temp > 0.f ? temp : 1.f, c = 1.44269504088896340736f / scale;
  for (int row = w; row <= n; row += (int)(blockDim.x >> 6)) {
    const RowPart* p = a.partial + ((int64_t)b * a.rows + row) * parts;
    float m = -INFINITY, s = 0.f, best = -INFINITY, logit = 0.f;
    int id = kNone;
    for (int i = lane; i < parts; i += 64) {
      const RowPart o = p[i];
      const float mn = fmaxf(m, o.m);
      if (mn > -INFINITY) s = s * exp2_fast((m - mn) * c) + o.s * exp2_fast((o.m - mn) * c);
      m = mn;
      if (o.best > best || (o.best == best && o.id < id)) {
        best = o.best;
        id = o.id;
        logit = o.logit;
      }
    }
    const float all = wave_max(m);
    if (all > -INFINITY) s = wave_sum(s * exp2_fast((m - all) * c));
    m = all;
    const float most = wave_max(best);
    const int mine = best == most ? id : kNone;
    id = wave_min(mine);
    best = most;
    logit = of_lane_with(logit, mine == id);
    if (lane == 0) {
      int stands = 0;
      float lp = -INFINITY;
      if (row < n) {
        const int d = a.draft[b * a.draft_stride + row];
        if (d >= 0 && d < a.vocab) {
          const float x = a.drafted[b * a.rows + row];
          if (x > -INFINITY) {
            lp = log_probability(x, m, scale, logf(s));
            stands = id == kNone || (temp > 0.f ? a.accept_u[b * a.accept_stride + row] < expf(lp)
                                                : x > best || (x == best && d < id));
          }
        }
      }
      s_stands[row] = stands;
      s_id[row] = id;
      s_m[row] = m;
      s_logit[row] = logit;
      // log-probability of the proposal where it stands; of the chosen id below
      s_lse[row] = stands ? lp : logf(s);
    }
  }
  __syncthreads();
  if (w == 0) {
    const bool ok = lane < n && s_stands[lane];
    const uint64_t stood = __ballot(ok);
    const int taken = min(n, stood == ~0ull ? 64 : __builtin_ctzll(~stood));
    if (lane == 0) a.out_accepted[b] = taken;
    if (lane < a.rows) {
      int tok = -1;
      float lp = 0.f;
      if (lane < taken) {
        tok = a.draft[b * a.draft_stride + lane];
        lp = s_lse[lane];
      } else if (lane == taken) {
        const int id = s_id[lane];
        if (id == kNone) {
          lp = -INFINITY;
        } else {
          tok = id;
          lp = log_probability(s_logit[lane], s_m[lane], scale, s_lse[lane]);
        }
      }
      a.out_tokens[b * a.rows + lane] = tok;
      if (a.out_logprob) a.out_logprob[b * a.rows + lane] = lp;
    }
  }
}

}  // namespace

// ---------------------------------------------------------------- handle
struct domino_verify : HandleBase {
  domino_verify_config_t cfg;
  RowPart* partial = nullptr;
  float* drafted = nullptr;
  int cus = 256;
};

static thread_local char t_err[256] = "";

constexpr int kMinRange = 512;
constexpr size_t kLdsBytes = 79 * 1024;  // two workgroups to a CU, beside their static LDS

struct Cut {
  int range, ranges, row_slots, parts;
  size_t lds;
};

static size_t lds_per_id(bool noise, bool touch, bool list, bool biases) {
  return (noise ? 4 : 0) + (touch ? 4 : 0) + (list ? 2 : 0) + (biases ? 4 : 0);
}

// longest range: what LDS for two workgroups to a CU holds, with a bit of the
// bitmap to each id
static int longest_range(size_t per_id) {
  const int fit = per_id ? (int)((kLdsBytes - 64) * 8 / (per_id * 8 + 1)) / 64 * 64 : 16384;
  return fit < 16384 ? fit : 16384;
}

// Ranges of a launch.  Workgroups run in rounds of two to a CU, and a range
// costs its ids plus what its start takes (about the time of 512 ids), so of
// the cuts that fill one to four rounds more than the longest ranges need,
// the one with the least rounds x (range + 512) is taken.  Where touched ids
// are taken in the pass, ranges differ in work and at least four rounds even
// it out: 64 blocks of 151936 ids with 4096 tokens of history, 300 biases and
// masks took 171 us in two rounds, 164 in three, 160 in four and six; the
// verification of 64 blocks, whose start takes longer, 144, 144, 151 and 170
// (136 since, in three).
// requests * ranges is at most requests * (ranges of the longest) + 8 rounds.
static Cut cut_vocab(int vocab, int cus, int requests, int rows, int vec, size_t per_id, bool touch, bool verify) {
  Cut k;
  const int most = longest_range(per_id), slots = 2 * cus;
  const int least = (vocab + most - 1) / most;
  int64_t best = -1;
  int64_t from = ((int64_t)least * requests + slots - 1) / slots;
  if (touch && !verify && from < 4) from = 4;
  k.range = most;
  for (int64_t rounds = from; rounds < from + 4; ++rounds) {
    int64_t r = rounds * slots / requests;
    if (r < least) r = least;
    int range = (int)(((vocab + r - 1) / r + 63) / 64 * 64);
    if (range < kMinRange) range = kMinRange;
    if (range > most) range = most;
    const int64_t ranges = (vocab + range - 1) / range;
    const int64_t cost = ((requests * ranges + slots - 1) / slots) * (range + 512);
    if (best < 0 || cost < best) {
      best = cost;
      k.range = range;
    }
  }
  k.ranges = (vocab + k.range - 1) / k.range;
  k.row_slots = rows < kWaves ? rows : kWaves;
  // waves to a row, each with at least one vector for most of its lanes
  const int pieces = (k.range + 64 * vec - 1) / (64 * vec);
  k.parts = kWaves / k.row_slots < pieces ? kWaves / k.row_slots : pieces;
  k.lds = per_id * k.range + (touch ? k.range / 8 : 0) + 64;
  return k;
}

// more dynamic LDS than the default 64 KB for every kernel of this type
template <typename T>
static hipError_t allow_lds() {
  const void* const kernels[] = {(const void*)&logits_kernel<T, false, false>, (const void*)&logits_kernel<T, false, true>,
                                 (const void*)&logits_kernel<T, true, false>, (const void*)&logits_kernel<T, true, true>};
  for (const void* k : kernels) {
    const hipError_t e = hipFuncSetAttribute(k, hipFuncAttributeMaxDynamicSharedMemorySize, (int)kLdsBytes);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

extern "C" domino_status_t domino_verify_create(const domino_verify_config_t* cfg, domino_verify_t** out) {
  if (!out) return say(t_err, DOMINO_ERR_INVALID_ARG, "create: out is NULL");
  *out = nullptr;
  if (!cfg) return say(t_err, DOMINO_ERR_INVALID_ARG, "create: cfg is NULL");
  if (cfg->vocab < 1) return say(t_err, DOMINO_ERR_INVALID_CONFIG, "create: vocab must be positive");
  if (cfg->max_requests < 1 || cfg->max_requests > 1024)
    return say(t_err, DOMINO_ERR_INVALID_CONFIG, "create: max_requests must be in [1, 1024]");
  if (cfg->max_rows < 1 || cfg->max_rows > kMaxRows)
    return say(t_err, DOMINO_ERR_INVALID_CONFIG, "create: max_rows must be in [1, %d]", kMaxRows);
  if (cfg->dtype != DOMINO_DTYPE_BF16 && cfg->dtype != DOMINO_DTYPE_FP32)
    return say(t_err, DOMINO_ERR_INVALID_CONFIG,
               "create: dtype must be DOMINO_DTYPE_BF16 or DOMINO_DTYPE_FP32");
  if (cfg->vocab > (1 << 24))
    return say(t_err, DOMINO_ERR_UNSUPPORTED, "create: vocab must be at most 2^24");
  int dev = 0;
  domino_status_t st = check_device(t_err, &dev);
  if (st != DOMINO_OK) return st;
  if ((cfg->dtype == DOMINO_DTYPE_BF16 ? allow_lds<bf16_t>() : allow_lds<float>()) != hipSuccess) {
    (void)hipGetLastError();
    return say(t_err, DOMINO_ERR_HIP, "create: the kernels' LDS limit could not be set");
  }
  domino_verify* h = new (std::nothrow) domino_verify();
  if (!h) return say(t_err, DOMINO_ERR_OUT_OF_MEMORY, "create: out of host memory");
  h->cfg = *cfg;
  h->device = dev;
  if (hipDeviceGetAttribute(&h->cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess) {
    (void)hipGetLastError();
    h->cus = 256;
  }
  // bound of cut_vocab's requests * ranges, times the waves of a row
  const int shortest = longest_range(lds_per_id(true, true, true, true));
  const size_t words = ((size_t)cfg->max_requests * ((cfg->vocab + shortest - 1) / shortest) + 8 * h->cus) *
                       (cfg->max_rows > kWaves ? cfg->max_rows : kWaves);
  h->partial = (RowPart*)h->take(words * sizeof(RowPart));
  h->drafted = (float*)h->take((size_t)cfg->max_requests * cfg->max_rows * 4);
  if (!h->partial || !h->drafted) {
    h->release();
    delete h;
    return say(t_err, DOMINO_ERR_OUT_OF_MEMORY, "create: workspace allocation failed");
  }
  *out = h;
  return DOMINO_OK;
}

extern "C" void domino_verify_destroy(domino_verify_t* h) {
  if (!h) return;
  h->release();
  delete h;
}

extern "C" const char* domino_verify_last_error(const domino_verify_t* h) { return h ? h->err : t_err; }

static domino_status_t take_logits(domino_verify_t* h, const char* who, const domino_logits_t* l,
                                   LogitsArgs& a) {
  if (!l) return say(h->err, DOMINO_ERR_INVALID_ARG, "%s: logits is NULL", who);
  const domino_verify_config_t& f = h->cfg;
  const int elem = f.dtype == DOMINO_DTYPE_BF16 ? 2 : 4;
  if (!l->logits || ((uintptr_t)l->logits & (elem - 1)))
    return say(h->err, DOMINO_ERR_INVALID_ARG, "%s: the logits pointer is NULL or misaligned", who);
  if (l->requests < 1 || l->requests > f.max_requests)
    return say(h->err, DOMINO_ERR_INVALID_ARG, "%s: requests %d outside [1, %d]", who, l->requests,
               f.max_requests);
  if (l->rows < 1 || l->rows > f.max_rows)
    return say(h->err, DOMINO_ERR_INVALID_ARG, "%s: rows %d outside [1, %d]", who, l->rows, f.max_rows);
  if (l->request_stride < 0 || l->row_stride < 0)
    return say(h->err, DOMINO_ERR_INVALID_ARG, "%s: strides must be >= 0", who);
  if (l->draft && l->rows > 1 && l->draft_stride < 0)
    return say(h->err, DOMINO_ERR_INVALID_ARG, "%s: strides must be >= 0", who);
  if (l->history && (l->history_width < 0 || l->history_stride < 0))
    return say(h->err, DOMINO_ERR_INVALID_ARG, "%s: history_width and history_stride must be >= 0", who);
  if ((l->bias_ids == nullptr) != (l->bias_values == nullptr))
    return say(h->err, DOMINO_ERR_INVALID_ARG, "%s: bias_ids and bias_values must be given together", who);
  if (l->bias_ids && (l->bias_width < 0 || l->bias_stride < 0))
    return say(h->err, DOMINO_ERR_INVALID_ARG, "%s: bias_width and bias_stride must be >= 0", who);
  if (l->mask && (l->mask_request_stride < 0 || l->mask_row_stride < 0))
    return say(h->err, DOMINO_ERR_INVALID_ARG, "%s: mask strides must be >= 0", who);
  const void* words[] = {l->draft, l->draft_len, l->history, l->history_len, l->prompt_len, l->repetition,
                         l->frequency, l->presence, l->bias_ids, l->bias_values, l->bias_len, l->mask};
  for (const void* p : words)
    if ((uintptr_t)p & 3)
      return say(h->err, DOMINO_ERR_INVALID_ARG, "%s: a list or mask pointer is not 4-byte aligned", who);
  a.logits = l->logits;
  a.req_stride = l->request_stride;
  a.row_stride = l->row_stride;
  a.requests = l->requests;
  a.rows = l->rows;
  a.vocab = f.vocab;
  a.draft = l->rows > 1 ? l->draft : nullptr;
  a.draft_stride = l->draft_stride;
  a.draft_len = l->draft_len;
  a.history = l->history_width > 0 ? l->history : nullptr;
  a.history_stride = l->history_stride;
  a.history_width = l->history_width;
  a.history_len = l->history_len;
  a.prompt_len = l->prompt_len;
  a.repetition = l->repetition;
  a.frequency = l->frequency;
  a.presence = l->presence;
  a.bias_ids = l->bias_width > 0 ? l->bias_ids : nullptr;
  a.bias_values = l->bias_values;
  a.bias_stride = l->bias_stride;
  a.bias_width = l->bias_width;
  a.bias_len = l->bias_len;
  a.mask = l->mask;
  a.mask_req = l->mask_request_stride;
  a.mask_row = l->mask_row_stride;
  return DOMINO_OK;
}

template <bool VERIFY>
static void launch_logits(const domino_verify_t* h, LogitsArgs& a, Cut& k, hipStream_t st) {
  const bool penalties = a.repetition || a.frequency || a.presence;
  const bool touch = penalties || a.bias_ids;
  k = cut_vocab(h->cfg.vocab, h->cus, a.requests, a.rows, h->cfg.dtype == DOMINO_DTYPE_BF16 ? 8 : 4,
                lds_per_id(VERIFY && a.noise, touch, VERIFY && touch, a.bias_ids != nullptr), touch, VERIFY);
  a.range = k.range;
  a.row_slots = k.row_slots;
  a.parts = k.parts;
  const dim3 grid(a.requests, k.ranges), block(kThreads);
  if (h->cfg.dtype == DOMINO_DTYPE_BF16) {
    if (touch)
      hipLaunchKernelGGL((logits_kernel<bf16_t, VERIFY, true>), grid, block, k.lds, st, a);
    else
      hipLaunchKernelGGL((logits_kernel<bf16_t, VERIFY, false>), grid, block, k.lds, st, a);
  } else {
    if (touch)
      hipLaunchKernelGGL((logits_kernel<float, VERIFY, true>), grid, block, k.lds, st, a);
    else
      hipLaunchKernelGGL((logits_kernel<float, VERIFY, false>), grid, block, k.lds, st, a);
  }
}

static domino_status_t launched(domino_verify_t* h, const char* who) {
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess)
    return say(h->err, DOMINO_ERR_HIP, "%s: kernel launch failed: %s", who, hipGetErrorString(e));
  h->err[0] = 0;
  return DOMINO_OK;
}

extern "C" domino_status_t domino_verify_process(domino_verify_t* h, const domino_logits_t* logits, void* out,
                                                 int64_t out_request_stride, int64_t out_row_stride,
                                                 void* stream) {
  if (!h) return DOMINO_ERR_INVALID_ARG;
  LogitsArgs a{};
  domino_status_t st = take_logits(h, "process", logits, a);
  if (st != DOMINO_OK) return st;
  const int elem = h->cfg.dtype == DOMINO_DTYPE_BF16 ? 2 : 4;
  if (!out || ((uintptr_t)out & (elem - 1)))
    return say(h->err, DOMINO_ERR_INVALID_ARG, "process: out is NULL or misaligned");
  if ((a.rows > 1 && out_row_stride < a.vocab) || (a.requests > 1 && out_request_stride < a.vocab))
    return say(h->err, DOMINO_ERR_INVALID_ARG, "process: rows of out overlap");
  a.out = out;
  a.out_req = out_request_stride;
  a.out_row = out_row_stride;
  DeviceGuard dg(h->device);
  (void)hipGetLastError();
  Cut k;
  launch_logits<false>(h, a, k, (hipStream_t)stream);
  return launched(h, "process");
}

extern "C" domino_status_t domino_verify_run(domino_verify_t* h, const domino_logits_t* logits,
                                             const float* temperature, const float* accept_u,
                                             int64_t accept_stride, const float* noise,
                                             int64_t noise_stride, int32_t* out_tokens,
                                             int32_t* out_accepted, float* out_logprob, void* stream) {
  if (!h) return DOMINO_ERR_INVALID_ARG;
  LogitsArgs a{};
  domino_status_t st = take_logits(h, "run", logits, a);
  if (st != DOMINO_OK) return st;
  if (!out_tokens || !out_accepted)
    return say(h->err, DOMINO_ERR_INVALID_ARG, "run: out_tokens and out_accepted must be non-NULL");
  if (temperature && (!noise || (a.draft && !accept_u)))
    return say(h->err, DOMINO_ERR_INVALID_ARG, "run: temperature needs noise, and accept_u where there are proposals");
  if (noise_stride < 0 || accept_stride < 0)
    return say(h->err, DOMINO_ERR_INVALID_ARG, "run: strides must be >= 0");
  const void* words[] = {temperature, accept_u, noise, out_tokens, out_accepted, out_logprob};
  for (const void* p : words)
    if ((uintptr_t)p & 3) return say(h->err, DOMINO_ERR_INVALID_ARG, "run: a pointer is not 4-byte aligned");
  a.temperature = temperature;
  a.accept_u = accept_u;
  a.accept_stride = accept_stride;
  a.noise = temperature ? noise : nullptr;
  a.noise_stride = noise_stride;
  a.partial = h->partial;
  a.drafted = h->drafted;
  a.out_tokens = out_tokens;
  a.out_accepted = out_accepted;
  a.out_logprob = out_logprob;
  DeviceGuard dg(h->device);
  (void)hipGetLastError();
  Cut k;
  launch_logits<true>(h, a, k, (hipStream_t)stream);
  if (hipPeekAtLastError() == hipSuccess)  // else it would join what an earlier call left
    hipLaunchKernelGGL(accept_kernel, dim3(a.requests), dim3(a.rows < 16 ? 64 * a.rows : 1024), 0, (hipStream_t)stream, a,
                       k.ranges * k.parts);
  return launched(h, "run");
}
