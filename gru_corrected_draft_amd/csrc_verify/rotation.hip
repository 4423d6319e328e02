// Norms of query and key heads and their rotation by position, in one pass.
//
// With x a head's D elements, w its weights, p the token's position, f_i the
// frequencies and g the magnitude:
//   y = x rsqrt(mean x^2 + eps) w          (y = x without weights)
//   a' = g (a cos p f_i - b sin p f_i), b' = g (b cos p f_i + a sin p f_i)
// for the pairs (a, b) = (y_i, y_(i + R/2)) or (y_2i, y_(2i+1)), i < R/2.
//
// A lane holds 16 elements of a head as two groups of 8 such that both numbers
// of a pair are its own: D / 16 lanes to a head, no exchange but the sum of
// squares.  The angles of a token are the same for all its heads: a workgroup
// forms cosines and sines of its tokens in LDS, once.  A frequency in revolutions is
// the sum of two 64-bit numbers; the whole turns are taken off the product with the
// first before it is rounded, so that with the second's the angle is good to 2^-53 of
// a turn at any position and frequency before it is rounded to 32 bits (one number and
// a rounded product were off by 5 x 2^-24 radians at position 2^31 of frequency 1, and
// by 7800 x 2^-24 of frequency 1000).
//
// Bound by memory: 8191 tokens of 48 heads of 128 take 43 us from call to call, 4.7
// TB/s (a large copy reaches 4.8 to 5.2), and 35 where the results fall into the same
// memory each time; a head's elements are loaded one ahead, the first before the
// angles are formed (46.5 and 41.5 without).  64 blocks of 16 tokens take 6.7 us
// on the GPU and one token 4.1, less than the call on the host, 9.5.  fp32: 4096 tokens
// of 48 heads 37 us for 39 of bytes (results in the same memory), 1024 of 40 heads 10.6 for 8.1.
#include <cmath>
#include <new>

#include "../../include/domino_verify.h"
#include "common.h"
#include "handle.h"

namespace {

constexpr int kMaxPairs = 128;

struct RotateArgs {
  const void* x[2];  // queries, keys
  void* y[2];
  const void* w[2];
  int64_t x_tok[2], x_head[2], y_tok[2], y_head[2];  // elements
  const int32_t* positions;
  const double2* turns;  // [rotary / 2] frequencies over 2 pi, x + y
  int32_t tokens, q_heads, heads, rotary;
  float eps, magnitude;
};

// eight elements as they lie in memory
template <typename T>
struct Raw {
  u32x4 x[sizeof(T) / 2];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) x[i] = *((const u32x4*)p + i);
  }
  __device__ __forceinline__ void unpack(float (&y)[8]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if constexpr (sizeof(T) == 4)
        y[i] = __uint_as_float(x[i / 4][i % 4]);
      else
        y[i] = __uint_as_float(i % 2 ? x[0][i / 2] & 0xFFFF0000u : x[0][i / 2] << 16);
    }
  }
};
__device__ __forceinline__ void store8(bf16_t* p, const float (&x)[8]) {
  typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
  v8bf v;
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = (__bf16)x[i];
  *(v8bf*)p = v;
}
__device__ __forceinline__ void store8(float* p, const float (&x)[8]) {
  *(float4*)p = make_float4(x[0], x[1], x[2], x[3]);
  *(float4*)(p + 4) = make_float4(x[4], x[5], x[6], x[7]);
}

// T: elements' type; D: of a head; PAIRS_NEXT: pairs are neighbours
template <typename T, int D, bool PAIRS_NEXT>
__global__ __launch_bounds__(256) void rotate_kernel(RotateArgs a, int tokens_each) {
  constexpr int LANES = D / 16;  // of a head
  __shared__ float2 s_turn[4][kMaxPairs];
  __shared__ int s_written[4];
  const int half = a.rotary / 2, t0 = blockIdx.x * tokens_each, tid = threadIdx.x;
  const int here = min(tokens_each, a.tokens - t0);
  const int lane = tid % LANES, rot_lanes = a.rotary / 16;
  // first elements of the lane's two groups
  int e0, e1;
  const bool turned = lane < rot_lanes;
  if (PAIRS_NEXT || !turned) {
    e0 = 16 * lane;
    e1 = e0 + 8;
  } else {
    e0 = 8 * lane;
    e1 = e0 + half;
  }
  // A head ahead of its use, the first on its way while the angles are formed.
  constexpr int STEP = 256 / LANES;
  const int step_t = STEP / a.heads, step_h = STEP % a.heads;
  int next_t = tid / LANES / a.heads, next_h = tid / LANES % a.heads;
  Raw<T> next_u, next_v;
  auto load = [&]() {
    if (next_t >= here) return;
    const int which = next_h >= a.q_heads, h = which ? next_h - a.q_heads : next_h;
    const T* x = (const T*)a.x[which] + (t0 + next_t) * a.x_tok[which] + h * a.x_head[which];
    next_u.load(x + e0);
    next_v.load(x + e1);
  };
  load();
  for (int i = tid; i < here * half; i += 256) {
    const int t = i / half, f = i - t * half;
    const double p = (double)a.positions[t0 + t];
    const double2 turn = a.turns[f];
    const double turns = fma(p, turn.y, fma(p, turn.x, -rint(p * turn.x)));
    float s, c;
    sincospif(2.f * (float)turns, &s, &c);
    s_turn[t][f] = make_float2(c * a.magnitude, s * a.magnitude);
  }
  if (tid < here) s_written[tid] = a.positions[t0 + tid] >= 0;
  __syncthreads();
  while (next_t < here) {
    const int t = next_t, which = next_h >= a.q_heads, h = which ? next_h - a.q_heads : next_h;
    float u[8], v[8];
    next_u.unpack(u);
    next_v.unpack(v);
    next_t += step_t;
    next_h += step_h;
    if (next_h >= a.heads) {
      next_h -= a.heads;
      ++next_t;
    }
    load();
    if (!s_written[t]) continue;
    if (a.w[0]) {
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) sum += u[i] * u[i] + v[i] * v[i];
#pragma unroll
      for (int m = 1; m < LANES; m <<= 1) sum += __shfl_xor(sum, m, 64);
      const float r = 1.f / sqrtf(sum * (1.f / D) + a.eps);
      float w[8];
      Raw<T> raw;
      const T* weight = (const T*)a.w[which];
      raw.load(weight + e0);
      raw.unpack(w);
#pragma unroll
      for (int i = 0; i < 8; ++i) u[i] = u[i] * r * w[i];
      raw.load(weight + e1);
      raw.unpack(w);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = v[i] * r * w[i];
    }
    if (turned) {
      const float2* turn = s_turn[t] + 8 * lane;
      if constexpr (PAIRS_NEXT) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float& p = i < 4 ? u[2 * i] : v[2 * i - 8];
          float& q = i < 4 ? u[2 * i + 1] : v[2 * i - 7];
          const float2 z = turn[i];
          const float p1 = p * z.x - q * z.y;
          q = q * z.x + p * z.y;
          p = p1;
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float2 z = turn[i];
          const float p1 = u[i] * z.x - v[i] * z.y;
          v[i] = v[i] * z.x + u[i] * z.y;
          u[i] = p1;
        }
      }
    }
    T* y = (T*)a.y[which] + (t0 + t) * a.y_tok[which] + h * a.y_head[which];
    store8(y + e0, u);
    store8(y + e1, v);
  }
}

struct Turns {
  double2 f[kMaxPairs];
};
__global__ void store_turns_kernel(Turns t, double2* out, int n) {
  if ((int)threadIdx.x < n) out[threadIdx.x] = t.f[threadIdx.x];
}

}  // namespace

struct domino_rotation : HandleBase {
  domino_rotation_config_t cfg;
  double2* turns = nullptr;
};

static thread_local char t_err[256] = "";

extern "C" domino_status_t domino_rotation_create(const domino_rotation_config_t* cfg, const double* inv_freq,
                                                  domino_rotation_t** out) {
  if (!out) return say(t_err, DOMINO_ERR_INVALID_ARG, "create: out is NULL");
  *out = nullptr;
  if (!cfg || !inv_freq) return say(t_err, DOMINO_ERR_INVALID_ARG, "create: cfg or inv_freq is NULL");
  if (cfg->q_heads < 1 || cfg->kv_heads < 1 || cfg->q_heads > 1024 || cfg->kv_heads > 1024)
    return say(t_err, DOMINO_ERR_INVALID_CONFIG, "create: q_heads and kv_heads must be in [1, 1024]");
  if (cfg->dtype != DOMINO_DTYPE_BF16 && cfg->dtype != DOMINO_DTYPE_FP32)
    return say(t_err, DOMINO_ERR_INVALID_CONFIG,
               "create: dtype must be DOMINO_DTYPE_BF16 or DOMINO_DTYPE_FP32");
  if (cfg->interleaved != 0 && cfg->interleaved != 1)
    return say(t_err, DOMINO_ERR_INVALID_CONFIG, "create: interleaved must be 0 or 1");
  if (!std::isfinite(cfg->magnitude))
    return say(t_err, DOMINO_ERR_INVALID_CONFIG, "create: magnitude must be finite");
  if (cfg->head_dim != 64 && cfg->head_dim != 128 && cfg->head_dim != 256)
    return say(t_err, DOMINO_ERR_UNSUPPORTED, "create: head_dim must be 64, 128 or 256 (got %d)", cfg->head_dim);
  if (cfg->rotary_dim < 16 || cfg->rotary_dim > cfg->head_dim || cfg->rotary_dim % 16)
    return say(t_err, DOMINO_ERR_UNSUPPORTED, "create: rotary_dim must be a multiple of 16 up to head_dim (got %d)",
               cfg->rotary_dim);
  Turns t{};
  for (int i = 0; i < cfg->rotary_dim / 2; ++i) {
    if (!std::isfinite(inv_freq[i]) || std::fabs(inv_freq[i]) > 1e3)
      return say(t_err, DOMINO_ERR_INVALID_CONFIG, "create: frequencies must be within 1000 of 0");
    // times 1 / (2 pi) = kTurn + kTurnRest, the product's rounding kept
    constexpr double kTurn = 0.15915494309189533577, kTurnRest = -9.839338337591243e-18;
    t.f[i].x = inv_freq[i] * kTurn;
    t.f[i].y = std::fma(inv_freq[i], kTurn, -t.f[i].x) + inv_freq[i] * kTurnRest;
  }
  int dev = 0;
  domino_status_t st = check_device(t_err, &dev);
  if (st != DOMINO_OK) return st;
  domino_rotation* h = new (std::nothrow) domino_rotation();
  if (!h) return say(t_err, DOMINO_ERR_OUT_OF_MEMORY, "create: out of host memory");
  h->cfg = *cfg;
  h->device = dev;
  h->turns = (double2*)h->take(sizeof(Turns));
  if (!h->turns) {
    delete h;
    return say(t_err, DOMINO_ERR_OUT_OF_MEMORY, "create: workspace allocation failed");
  }
  (void)hipGetLastError();
  hipLaunchKernelGGL(store_turns_kernel, dim3(1), dim3(kMaxPairs), 0, nullptr, t, h->turns, cfg->rotary_dim / 2);
  if (hipGetLastError() != hipSuccess || hipDeviceSynchronize() != hipSuccess) {
    (void)hipGetLastError();
    h->release();
    delete h;
    return say(t_err, DOMINO_ERR_HIP, "create: the frequencies could not be stored");
  }
  *out = h;
  return DOMINO_OK;
}

extern "C" void domino_rotation_destroy(domino_rotation_t* h) {
  if (!h) return;
  h->release();
  delete h;
}

extern "C" const char* domino_rotation_last_error(const domino_rotation_t* h) { return h ? h->err : t_err; }

template <typename T, int D>
static void launch_rotate(const domino_rotation* h, const RotateArgs& a, hipStream_t st) {
  // Several tokens to a workgroup save starts where a token is little for 256 lanes
  // and there are workgroups enough even so, one, two or four: 40 heads of 128 of
  // 2048 tokens 10.2, 10.1 and 10.2 us, of 4096 17.2, 14.9 and 15.0, of 8191 31.8, 30.1
  // and 28.9; 10 heads of 128 of 16000 21.8, 17.8 and 17.1; but 72 of 128 of 4096 27.6, 26.7
  // and 28.4, of 16000 109, 113 and 120.
  const int size = a.heads * D;  // of a token
  const int tokens_each = size > 8192 || a.tokens < 2560 ? 1 : a.tokens < 6000 ? 2 : 4;
  const dim3 grid((unsigned)((a.tokens + tokens_each - 1) / tokens_each));
  if (h->cfg.interleaved)
    hipLaunchKernelGGL((rotate_kernel<T, D, true>), grid, dim3(256), 0, st, a, tokens_each);
  else
    hipLaunchKernelGGL((rotate_kernel<T, D, false>), grid, dim3(256), 0, st, a, tokens_each);
}

template <typename T>
static void launch_rotate_dim(const domino_rotation* h, const RotateArgs& a, hipStream_t st) {
  if (h->cfg.head_dim == 64)
    launch_rotate<T, 64>(h, a, st);
  else if (h->cfg.head_dim == 128)
    launch_rotate<T, 128>(h, a, st);
  else
    launch_rotate<T, 256>(h, a, st);
}

extern "C" domino_status_t domino_rotation_run(domino_rotation_t* h, const domino_heads_t* q, const domino_heads_t* k,
                                               const int32_t* positions, int32_t tokens, float eps, void* stream) {
  if (!h) return DOMINO_ERR_INVALID_ARG;
  const domino_rotation_config_t& f = h->cfg;
  const int unit = f.dtype == DOMINO_DTYPE_BF16 ? 8 : 4;
  if (!q || !k) return say(h->err, DOMINO_ERR_INVALID_ARG, "run: q or k is NULL");
  if (tokens < 0) return say(h->err, DOMINO_ERR_INVALID_ARG, "run: tokens must be >= 0");
  if ((q->weight == nullptr) != (k->weight == nullptr))
    return say(h->err, DOMINO_ERR_INVALID_ARG, "run: weights of q and k must be given together");
  if (!(eps >= 0.f) || !std::isfinite(eps))
    return say(h->err, DOMINO_ERR_INVALID_ARG, "run: eps must be finite and >= 0");
  if (tokens == 0) return DOMINO_OK;
  if (!positions || ((uintptr_t)positions & 3))
    return say(h->err, DOMINO_ERR_INVALID_ARG, "run: positions must be non-NULL and 4-byte aligned");
  RotateArgs a{};
  for (int i = 0; i < 2; ++i) {
    const domino_heads_t* x = i ? k : q;
    const int heads = i ? f.kv_heads : f.q_heads;
    if (!x->in || !x->out) return say(h->err, DOMINO_ERR_INVALID_ARG, "run: in and out must be non-NULL");
    if (((uintptr_t)x->in | (uintptr_t)x->out | (uintptr_t)x->weight) & 15 || x->token_stride < 0 || x->head_stride < 0 ||
        x->out_token_stride < 0 || x->out_head_stride < 0 || x->token_stride % unit || x->head_stride % unit ||
        x->out_token_stride % unit || x->out_head_stride % unit)
      return say(h->err, DOMINO_ERR_INVALID_ARG,
                 "run: arrays must be 16-byte aligned, their strides multiples of 16 bytes");
    if ((tokens > 1 && x->out_token_stride < f.head_dim) || (heads > 1 && x->out_head_stride < f.head_dim))
      return say(h->err, DOMINO_ERR_INVALID_ARG, "run: rows of out overlap");
    a.x[i] = x->in;
    a.y[i] = x->out;
    a.w[i] = x->weight;
    a.x_tok[i] = x->token_stride;
    a.x_head[i] = x->head_stride;
    a.y_tok[i] = x->out_token_stride;
    a.y_head[i] = x->out_head_stride;
  }
  a.positions = positions;
  a.turns = h->turns;
  a.tokens = tokens;
  a.q_heads = f.q_heads;
  a.heads = f.q_heads + f.kv_heads;
  a.rotary = f.rotary_dim;
  a.eps = eps;
  a.magnitude = f.magnitude;
  DeviceGuard dg(h->device);
  (void)hipGetLastError();
  if (f.dtype == DOMINO_DTYPE_BF16)
    launch_rotate_dim<bf16_t>(h, a, (hipStream_t)stream);
  else
    launch_rotate_dim<float>(h, a, (hipStream_t)stream);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess)
    return say(h->err, DOMINO_ERR_HIP, "run: kernel launch failed: %s", hipGetErrorString(e));
  h->err[0] = 0;
  return DOMINO_OK;
}
