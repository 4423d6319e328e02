// Paged attention of new tokens over a key-value cache, and the append that
// fills it.  See attention.h for rows, key tiles and helpers.
#include <cmath>
#include <new>

#include "../../include/domino_verify.h"
#include "attention_bf16.h"
#include "fp4.h"
#include "handle.h"
#include "parts.h"

// ---------------------------------------------------------------- append
// A copy: one 16-byte piece per thread, keys in the first half of the grid's
// y, values in the second.  Bound by the launch for a decoding step (2.1 us on
// the GPU, 7 us from call to call) and by memory for a prompt: 8 requests of up
// to 1024 tokens, 51.6 MB read and written, take 10.9 us, 4.7 TB/s of a large
// copy's 5.2.  Rows of a head are contiguous on both sides.
struct AppendArgs {
  const void* src[2];
  void* dst[2];
  int64_t tok[2], headi[2];
  int64_t page, head;
  int32_t row, num_pages, pieces;  // pieces: 16-byte pieces of a row
  const int32_t* table;
  int64_t table_stride;
  int32_t page_shift, elem;
  const int32_t* kv_len;
  const int32_t* q_start;
  int32_t tokens, max_new, max_kv, kv_heads;
};

__global__ __launch_bounds__(256) void append_kernel(AppendArgs a) {
  const int which = blockIdx.y & 1, b = blockIdx.y >> 1;
  const Request r = request_of(a.q_start, a.kv_len, b, a.tokens, a.max_new, a.max_kv);
  if (r.bad) return;
  const int per_token = a.kv_heads * a.pieces;
  const int64_t total = (int64_t)r.n * per_token;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    const int t = (int)(i / per_token), rest = (int)(i - (int64_t)t * per_token);
    const int h = rest / a.pieces, piece = rest - h * a.pieces;
    const int pos = r.kv - r.n + t;
    if (pos < 0) continue;
    const int page = a.table[b * a.table_stride + (pos >> a.page_shift)];
    if (page < 0 || page >= a.num_pages) continue;
    const int row = pos & ((1 << a.page_shift) - 1);
    const char* s = (const char*)a.src[which] +
                    ((r.q0 + t) * a.tok[which] + h * a.headi[which]) * a.elem + piece * 16;
    char* d = (char*)a.dst[which] +
              (page * a.page + h * a.head + (int64_t)row * a.row) * a.elem + piece * 16;
    *(u32x4*)d = *(const u32x4*)s;
  }
}

// ---------------------------------------------------------------- fp32 attention
// Four waves share a tile of 16 rows and take 16-key tiles in turn, each with
// its own running maximum and sum; the four are joined in LDS at the end.
// Where few row tiles would leave the chip idle, the keys of each are dealt to
// several workgroups, the last of which joins their outputs: fp32 calls are
// small checks, bound by the time from load to use (blocks of 7 tokens of 3
// requests over up to 1001 keys 22 us undivided, 12.6 with a second launch, 10.8).
// The scores are computed transposed (keys x rows), so the row's maximum and
// sum stay in the row's lanes and the accumulator registers of the scores are
// the second product's operand as they are: lane (n = l % 16, q = l / 16)
// holds the scores of row n and keys 4 q .. 4 q + 3, and the product over keys
// takes key 4 q + i in its i-th step.  The head dimension is dealt to the
// lanes so that every load is 16 bytes: step i of the first product takes
// element 16 c + 4 q + i, and output row m of accumulator (blk, j) is element
// 64 blk + 4 m + j.
__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }

template <int D>
__global__ __launch_bounds__(256) void attend_f32_kernel(AttendArgs a, int splits) {
  constexpr int KT = 16, ROWS = 16, C = D / 16, NB = D / 64;
  __shared__ float s_o[4][ROWS][D + 4];
  __shared__ float s_m[4][ROWS], s_l[4][ROWS];
  __shared__ int s_bad[4];
  const int b = blockIdx.z, h = blockIdx.y, split = blockIdx.x % splits, r0 = blockIdx.x / splits * ROWS;
  const Request req = request_of(a.q_start, a.kv_len, b, a.tokens, a.max_new, a.max_kv);
  const int rows = req.n * a.group;
  if (r0 >= rows) return;
  const int lane = threadIdx.x & 63, w = wave_index(), n = lane & 15, q4 = lane >> 4;
  const int last = min(r0 + ROWS, rows) - 1;
  const KeySpan span = key_span<KT>(req, r0 / a.group, last / a.group, a.window, a.sinks);
  const int row = min(r0 + n, last);
  const int tok = row / a.group, hq = h * a.group + row - tok * a.group;
  const int pos = req.kv - req.n + tok;
  const float* qp = (const float*)a.q + (req.q0 + tok) * a.q_tok + hq * a.q_head + 4 * q4;
  float4 Q[C];
#pragma unroll
  for (int c = 0; c < C; ++c) Q[c] = load4(qp + 16 * c);
  v4f O[NB][4];
#pragma unroll
  for (int i = 0; i < NB; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) O[i][j] = zero4();
  float m = -INFINITY, l = 0.f;
  bool bad = req.bad;
  for (int i = split * 4 + w; i < span.count; i += 4 * splits) {
    const int k0 = tile_of(span, i) * KT;
    int page = a.table[b * a.table_stride + (k0 >> a.page_shift)];
    if (page < 0 || page >= a.num_pages) {
      bad = true;
      break;
    }
    const int64_t base = page * a.page + h * a.head + (int64_t)(k0 & ((1 << a.page_shift) - 1)) * a.row;
    const float* kp = (const float*)a.k + base + (int64_t)n * a.row + 4 * q4;
    v4f s = zero4();
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const float4 k = load4(kp + 16 * c);
      s = mfma_f32(k.x, Q[c].x, s);
      s = mfma_f32(k.y, Q[c].y, s);
      s = mfma_f32(k.z, Q[c].z, s);
      s = mfma_f32(k.w, Q[c].w, s);
    }
    const bool edge = !all_visible(span, k0, KT, a.window, a.sinks);
    if (edge) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (!visible(k0 + 4 * q4 + j, pos, a.window, a.sinks)) s[j] = -INFINITY;
    }
    float top = fmaxf(fmaxf(s[0], s[1]), fmaxf(s[2], s[3]));
    top = fmaxf(top, __shfl_xor(top, 16, 64));
    top = fmaxf(top, __shfl_xor(top, 32, 64));
    const float mn = fmaxf(m, top);
    const float ref = mn == -INFINITY ? 0.f : mn * a.scale_log2;
    // From the difference, so that it is 1 while the maximum stays.  m c - ref
    // contracts to a fused product whose rest, half an ulp of the score, would
    // multiply the sums once a tile: 7 to 11 times the error over 6001 and 8192
    // keys (2 requests with 500 tokens over 2000 keys take 344 us against 338).
    const float alpha = mn == -INFINITY ? 1.f : exp2f((m - mn) * a.scale_log2);
    float p[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) p[j] = exp2f(__builtin_fmaf(s[j], a.scale_log2, -ref));
    l = l * alpha + ((p[0] + p[1]) + (p[2] + p[3]));
    m = mn;
#pragma unroll
    for (int x = 0; x < NB; ++x)
#pragma unroll
      for (int j = 0; j < 4; ++j) O[x][j] *= alpha;
    const float* vp = (const float*)a.v + base + (int64_t)(4 * q4) * a.row + 4 * n;
    float4 V[4][NB];
    bool odd = false;
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int x = 0; x < NB; ++x) {
        V[j][x] = load4(vp + (int64_t)j * a.row + 64 * x);
        odd |= nonfinite(V[j][x].x) || nonfinite(V[j][x].y) || nonfinite(V[j][x].z) ||
               nonfinite(V[j][x].w);
      }
    if (edge && __any(odd)) {
      // a product would multiply a row's zero weight by an infinity or NaN
      // that the row does not see: add key by key, to the rows that see it
      for (int kk = 0; kk < KT; ++kk) {
        const float mine = (kk & 2) ? ((kk & 1) ? p[3] : p[2]) : ((kk & 1) ? p[1] : p[0]);
        const float pk = __shfl(mine, (kk >> 2) * 16 + n, 64);
        if (!visible(k0 + kk, pos, a.window, a.sinks)) continue;
        const float* vk = (const float*)a.v + base + (int64_t)kk * a.row;
#pragma unroll
        for (int x = 0; x < NB; ++x)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float4 v = load4(vk + 64 * x + 16 * q4 + 4 * e);
            O[x][0][e] += pk * v.x;
            O[x][1][e] += pk * v.y;
            O[x][2][e] += pk * v.z;
            O[x][3][e] += pk * v.w;
          }
      }
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int x = 0; x < NB; ++x) {
          O[x][0] = mfma_f32(V[j][x].x, p[j], O[x][0]);
          O[x][1] = mfma_f32(V[j][x].y, p[j], O[x][1]);
          O[x][2] = mfma_f32(V[j][x].z, p[j], O[x][2]);
          O[x][3] = mfma_f32(V[j][x].w, p[j], O[x][3]);
        }
    }
  }
  l += __shfl_xor(l, 16, 64);
  l += __shfl_xor(l, 32, 64);
  if (lane < 16) {
    s_m[w][n] = m;
    s_l[w][n] = l;
  }
  if (lane == 0) s_bad[w] = bad;
#pragma unroll
  for (int x = 0; x < NB; ++x)
#pragma unroll
    for (int e = 0; e < 4; ++e)
      *reinterpret_cast<float4*>(&s_o[w][n][64 * x + 16 * q4 + 4 * e]) =
          make_float4(O[x][0][e], O[x][1][e], O[x][2][e], O[x][3][e]);
  __syncthreads();
  const bool spoilt = s_bad[0] | s_bad[1] | s_bad[2] | s_bad[3];
  const int64_t part = ((int64_t)b * a.kv_heads + h) * gridDim.x + blockIdx.x;
  for (int i = threadIdx.x; i < ROWS * D / 2; i += 256) {  // two elements of a row
    const int rr = i / (D / 2), d = 2 * (i - rr * (D / 2));
    if (r0 + rr > last) break;
    float top = -INFINITY;
#pragma unroll
    for (int x = 0; x < 4; ++x) top = fmaxf(top, s_m[x][rr]);
    const float ref = top == -INFINITY ? 0.f : top;
    float2 num = make_float2(0.f, 0.f);
    float den = 0.f;
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const float f = exp2f((s_m[x][rr] - ref) * a.scale_log2);
      den += f * s_l[x][rr];
      // a wave that saw no key of this row holds only zeros
      if (s_m[x][rr] != -INFINITY) {
        num.x += f * s_o[x][rr][d];
        num.y += f * s_o[x][rr][d + 1];
      }
    }
    if (spoilt) den = NAN;
    if (splits > 1) {
      share2(a.part_o + (part * ROWS + rr) * D + d, num.x, num.y);
      if (d == 0) share2(a.part_ml + (part * ROWS + rr) * 2, top, den);
      continue;
    }
    const bool none = den == 0.f && top == -INFINITY;
    const int tk = (r0 + rr) / a.group, hd = h * a.group + (r0 + rr) - tk * a.group;
    *(float2*)((float*)a.out + (req.q0 + tk) * a.o_tok + hd * a.o_head + d) =
        none ? make_float2(0.f, 0.f) : make_float2(num.x / den, num.y / den);
    if (d == 0 && a.lse)
      a.lse[(int64_t)(req.q0 + tk) * a.q_heads + hd] = none ? -INFINITY : top * a.scale + logf(den);
  }
  if (splits == 1) return;

  // the last of the row tile's workgroups joins its parts, in their order
  __shared__ int s_last;
  if (!last_of(a.arrived + (part - split) / splits, splits, &s_last)) return;
  for (int i = threadIdx.x; i < (last - r0 + 1) * (D / 4); i += 256) {
    const int rr = i / (D / 4), piece = i - rr * (D / 4);
    float top = -INFINITY, den = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int64_t g = part - split; g < part - split + splits; ++g) {
      const float2 ml = shared2(a.part_ml + (g * ROWS + rr) * 2);
      const float4 y = shared4(a.part_o + (g * ROWS + rr) * D + 4 * piece);
      const float mn = fmaxf(top, ml.x), ref = mn == -INFINITY ? 0.f : mn;
      const float fo = exp2f((top - ref) * a.scale_log2), fn = exp2f((ml.x - ref) * a.scale_log2);
      den = den * fo + ml.y * fn;
      o.x = scaled(o.x, fo) + scaled(y.x, fn);
      o.y = scaled(o.y, fo) + scaled(y.y, fn);
      o.z = scaled(o.z, fo) + scaled(y.z, fn);
      o.w = scaled(o.w, fo) + scaled(y.w, fn);
      top = mn;
    }
    const bool none = den == 0.f && top == -INFINITY;
    const int tk = (r0 + rr) / a.group, hd = h * a.group + (r0 + rr) - tk * a.group;
    *(float4*)((float*)a.out + (req.q0 + tk) * a.o_tok + hd * a.o_head + 4 * piece) =
        none ? make_float4(0.f, 0.f, 0.f, 0.f) : make_float4(o.x / den, o.y / den, o.z / den, o.w / den);
    if (piece == 0 && a.lse)
      a.lse[(int64_t)(req.q0 + tk) * a.q_heads + hd] = none ? -INFINITY : top * a.scale + logf(den);
  }
}

// workspace of split fp32 attention: 2 parts of 16 rows to a CU
static size_t attend_f32_floats(int head_dim, int cus) { return (size_t)2 * cus * 16 * (head_dim + 2); }

// ---------------------------------------------------------------- handle
struct domino_attention : HandleBase {
  domino_attention_config_t cfg;
  bool fp4 = false;  // the cache is held in 4 bits
  int cus = 256;
  float* part = nullptr;    // split segments: outputs, then (m, l)
  int32_t* plan = nullptr;     // bf16: running sum of the requests' steps, or of 64 row tiles' pieces
  int32_t* arrived = nullptr;  // fp32: parts there are of each row tile and key head, 0 between calls
};

static thread_local char t_err[256] = "";

static domino_status_t create(const domino_attention_config_t* cfg, bool fp4, domino_attention_t** out) {
  if (!out) return say(t_err, DOMINO_ERR_INVALID_ARG, "create: out is NULL");
  *out = nullptr;
  if (!cfg) return say(t_err, DOMINO_ERR_INVALID_ARG, "create: cfg is NULL");
  if (cfg->q_heads < 1 || cfg->kv_heads < 1 || cfg->q_heads % cfg->kv_heads)
    return say(t_err, DOMINO_ERR_INVALID_CONFIG,
               "create: q_heads must be a positive multiple of kv_heads (got %d and %d)",
               cfg->q_heads, cfg->kv_heads);
  if (cfg->max_requests < 1 || cfg->max_requests > 1024)
    return say(t_err, DOMINO_ERR_INVALID_CONFIG, "create: max_requests must be in [1, 1024]");
  if (cfg->dtype != DOMINO_DTYPE_BF16 && cfg->dtype != DOMINO_DTYPE_FP32)
    return say(t_err, DOMINO_ERR_INVALID_CONFIG,
               "create: dtype must be DOMINO_DTYPE_BF16 or DOMINO_DTYPE_FP32");
  if (fp4 && cfg->dtype != DOMINO_DTYPE_BF16)
    return say(t_err, DOMINO_ERR_UNSUPPORTED, "create: a cache in 4 bits takes DOMINO_DTYPE_BF16");
  if (cfg->head_dim != 64 && cfg->head_dim != 128 && cfg->head_dim != 256)
    return say(t_err, DOMINO_ERR_UNSUPPORTED, "create: head_dim must be 64, 128 or 256 (got %d)",
               cfg->head_dim);
  if (cfg->page_size < 16 || cfg->page_size > 4096 || (cfg->page_size & (cfg->page_size - 1)))
    return say(t_err, DOMINO_ERR_UNSUPPORTED,
               "create: page_size must be a power of two in [16, 4096] (got %d)", cfg->page_size);
  if (cfg->q_heads > 1024)
    return say(t_err, DOMINO_ERR_UNSUPPORTED, "create: at most 1024 query heads");
  int dev = 0;
  domino_status_t st = check_device(t_err, &dev);
  if (st != DOMINO_OK) return st;
  if (cfg->dtype == DOMINO_DTYPE_BF16 &&
      (fp4 ? attend_fp4_prepare(cfg->head_dim) : attend_split_prepare(cfg->head_dim)) != hipSuccess) {
    (void)hipGetLastError();
    return say(t_err, DOMINO_ERR_HIP, "create: the kernels' LDS limit could not be set");
  }
  domino_attention* h = new (std::nothrow) domino_attention();
  if (!h) return say(t_err, DOMINO_ERR_OUT_OF_MEMORY, "create: out of host memory");
  h->cfg = *cfg;
  h->fp4 = fp4;
  h->device = dev;
  if (hipDeviceGetAttribute(&h->cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess) {
    (void)hipGetLastError();
    h->cus = 256;
  }
  const size_t floats = cfg->dtype == DOMINO_DTYPE_BF16 ? attend_split_floats(cfg->head_dim, h->cus)
                                                        : attend_f32_floats(cfg->head_dim, h->cus);
  h->part = (float*)h->take(floats * sizeof(float));
  bool ok = h->part != nullptr;
  if (cfg->dtype == DOMINO_DTYPE_BF16) {
    h->plan = (int32_t*)h->take((size_t)((cfg->max_requests < 64 ? 64 : cfg->max_requests) + 1) * sizeof(int32_t));
    ok = ok && h->plan;
  } else {
    h->arrived = (int32_t*)h->take((size_t)h->cus * sizeof(int32_t));
    ok = ok && h->arrived && hipMemset(h->arrived, 0, (size_t)h->cus * sizeof(int32_t)) == hipSuccess;
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

extern "C" domino_status_t domino_attention_create(const domino_attention_config_t* cfg,
                                                   domino_attention_t** out) {
  return create(cfg, false, out);
}

extern "C" domino_status_t domino_attention_create_fp4(const domino_attention_config_t* cfg,
                                                       domino_attention_t** out) {
  return create(cfg, true, out);
}

extern "C" void domino_attention_destroy(domino_attention_t* h) {
  if (!h) return;
  h->release();
  delete h;
}

extern "C" const char* domino_attention_last_error(const domino_attention_t* h) {
  return h ? h->err : t_err;
}

static domino_status_t check_cache(domino_attention_t* h, const char* who, const domino_cache_t* c) {
  const domino_attention_config_t& f = h->cfg;
  // strides count elements; those of a cache in 4 bits bytes
  const int elem = h->fp4 ? 1 : f.dtype == DOMINO_DTYPE_BF16 ? 2 : 4, unit = 16 / elem;
  if (!c) return say(h->err, DOMINO_ERR_INVALID_ARG, "%s: cache is NULL", who);
  if (!c->k_cache || !c->v_cache || !c->page_table || !c->kv_len || !c->q_start)
    return say(h->err, DOMINO_ERR_INVALID_ARG, "%s: a pointer of the cache is NULL", who);
  if (((uintptr_t)c->k_cache | (uintptr_t)c->v_cache) & 15)
    return say(h->err, DOMINO_ERR_INVALID_ARG, "%s: caches must be 16-byte aligned", who);
  if (((uintptr_t)c->page_table | (uintptr_t)c->kv_len | (uintptr_t)c->q_start) & 3)
    return say(h->err, DOMINO_ERR_INVALID_ARG, "%s: page_table, kv_len and q_start must be 4-byte aligned", who);
  if (c->requests < 1 || c->requests > f.max_requests)
    return say(h->err, DOMINO_ERR_INVALID_ARG, "%s: requests %d outside [1, %d]", who, c->requests,
               f.max_requests);
  if (c->tokens < 0 || c->max_new < 0 || c->max_kv < 0)
    return say(h->err, DOMINO_ERR_INVALID_ARG, "%s: tokens, max_new and max_kv must be >= 0", who);
  if (c->num_pages < 1 || c->table_width < 1 || c->table_stride < 0)
    return say(h->err, DOMINO_ERR_INVALID_ARG,
               "%s: num_pages and table_width must be positive, table_stride >= 0", who);
  if (h->fp4 && c->row_stride != f.head_dim / 2)
    return say(h->err, DOMINO_ERR_INVALID_ARG, "%s: row_stride must be head_dim / 2 bytes", who);
  if (c->page_stride < 0 || c->head_stride < 0 || (!h->fp4 && c->row_stride < f.head_dim) ||
      c->page_stride % unit || c->head_stride % unit || c->row_stride % unit)
    return say(h->err, DOMINO_ERR_INVALID_ARG,
               "%s: cache strides must be multiples of 16 bytes, row_stride at least head_dim", who);
  const double page_rows = (double)f.page_size * (h->fp4 ? f.head_dim / 2 + f.head_dim / 32 : c->row_stride);
  if (((double)(f.kv_heads - 1) * c->head_stride + page_rows) * elem >= 2147483648.0)
    return say(h->err, DOMINO_ERR_INVALID_ARG, "%s: a page must span less than 2^31 bytes", who);
  return DOMINO_OK;
}

// token arrays: 16-byte aligned base and strides
static bool rows_ok(const void* p, int64_t tok, int64_t head, int unit) {
  return !((uintptr_t)p & 15) && tok >= 0 && head >= 0 && tok % unit == 0 && head % unit == 0;
}

// Also 2^30, so that sums of positions, windows and tiles stay in 32 bits: no
// cache in this memory holds so many keys of a request.
static int32_t clip_kv(const domino_cache_t* c, int page_size) {
  int64_t most = (int64_t)c->table_width * page_size;
  if (most > 1 << 30) most = 1 << 30;
  return (int32_t)(c->max_kv < most ? c->max_kv : most);
}

static domino_status_t launched(domino_attention_t* h, const char* who) {
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess)
    return say(h->err, DOMINO_ERR_HIP, "%s: kernel launch failed: %s", who, hipGetErrorString(e));
  h->err[0] = 0;
  return DOMINO_OK;
}

static RowsArgs4 rows_args(const domino_attention_t* h, const domino_cache_t* c, void* k, int64_t k_token_stride,
                           int64_t k_head_stride, void* v, int64_t v_token_stride, int64_t v_head_stride) {
  const domino_attention_config_t& f = h->cfg;
  RowsArgs4 a;
  a.tok[0] = k;
  a.tok[1] = v;
  a.cache[0] = c->k_cache;
  a.cache[1] = c->v_cache;
  a.tok_stride[0] = k_token_stride;
  a.tok_stride[1] = v_token_stride;
  a.head_stride[0] = k_head_stride;
  a.head_stride[1] = v_head_stride;
  a.page = c->page_stride;
  a.head = c->head_stride;
  a.num_pages = c->num_pages;
  a.head_dim = f.head_dim;
  a.table = c->page_table;
  a.table_stride = c->table_stride;
  a.page_shift = __builtin_ctz(f.page_size);
  a.kv_len = c->kv_len;
  a.q_start = c->q_start;
  a.requests = c->requests;
  a.tokens = c->tokens;
  a.max_new = c->max_new;
  a.max_kv = clip_kv(c, f.page_size);
  a.kv_heads = f.kv_heads;
  a.piece_shift = __builtin_ctz(f.head_dim / 8);
  const uint32_t per_token = (uint32_t)f.kv_heads << a.piece_shift;
  a.magic_shift = per_token > 1 ? 32 - __builtin_clz(per_token - 1) : 0;
  a.magic = (uint32_t)((((uint64_t)1 << 32) * (((uint64_t)1 << a.magic_shift) - per_token)) / per_token + 1);
  return a;
}

// pieces of a request's new tokens stay in 31 bits
static bool rows_fit(const domino_attention_t* h, const domino_cache_t* c) {
  const int most = c->max_new < c->tokens ? c->max_new : c->tokens;
  return (int64_t)most * h->cfg.kv_heads * (h->cfg.head_dim / 8) < (int64_t)1 << 30;
}

extern "C" domino_status_t domino_attention_append(domino_attention_t* h, const domino_cache_t* c,
                                                   const void* k, int64_t k_token_stride,
                                                   int64_t k_head_stride, const void* v,
                                                   int64_t v_token_stride, int64_t v_head_stride,
                                                   void* stream) {
  if (!h) return DOMINO_ERR_INVALID_ARG;
  domino_status_t st = check_cache(h, "append", c);
  if (st != DOMINO_OK) return st;
  const domino_attention_config_t& f = h->cfg;
  const int elem = f.dtype == DOMINO_DTYPE_BF16 ? 2 : 4, unit = 16 / elem;
  if (c->tokens == 0 || c->max_new == 0) return DOMINO_OK;
  if (!k || !v) return say(h->err, DOMINO_ERR_INVALID_ARG, "append: k and v must be non-NULL");
  if (!rows_ok(k, k_token_stride, k_head_stride, unit) || !rows_ok(v, v_token_stride, v_head_stride, unit))
    return say(h->err, DOMINO_ERR_INVALID_ARG,
               "append: k and v must be 16-byte aligned, their strides multiples of 16 bytes");
  if (h->fp4) {
    if (!rows_fit(h, c)) return say(h->err, DOMINO_ERR_UNSUPPORTED, "append: too many rows for a request");
    const RowsArgs4 a = rows_args(h, c, (void*)k, k_token_stride, k_head_stride, (void*)v, v_token_stride, v_head_stride);
    DeviceGuard dg(h->device);
    (void)hipGetLastError();
    launch_append_fp4(a, (hipStream_t)stream);
    return launched(h, "append");
  }
  AppendArgs a;
  a.src[0] = k;
  a.src[1] = v;
  a.dst[0] = c->k_cache;
  a.dst[1] = c->v_cache;
  a.tok[0] = k_token_stride;
  a.tok[1] = v_token_stride;
  a.headi[0] = k_head_stride;
  a.headi[1] = v_head_stride;
  a.page = c->page_stride;
  a.head = c->head_stride;
  a.row = (int32_t)c->row_stride;
  a.num_pages = c->num_pages;
  a.pieces = f.head_dim / unit;
  a.table = c->page_table;
  a.table_stride = c->table_stride;
  a.page_shift = __builtin_ctz(f.page_size);
  a.elem = elem;
  a.kv_len = c->kv_len;
  a.q_start = c->q_start;
  a.tokens = c->tokens;
  a.max_new = c->max_new;
  a.max_kv = clip_kv(c, f.page_size);
  a.kv_heads = f.kv_heads;
  const int most = c->max_new < c->tokens ? c->max_new : c->tokens;
  const int64_t blocks = ((int64_t)most * f.kv_heads * a.pieces + 255) / 256;
  DeviceGuard dg(h->device);
  (void)hipGetLastError();
  hipLaunchKernelGGL(append_kernel, dim3((unsigned)(blocks < 1024 ? blocks : 1024), 2 * c->requests),
                     dim3(256), 0, (hipStream_t)stream, a);
  return launched(h, "append");
}

extern "C" domino_status_t domino_attention_read(domino_attention_t* h, const domino_cache_t* c, void* k,
                                                 int64_t k_token_stride, int64_t k_head_stride, void* v,
                                                 int64_t v_token_stride, int64_t v_head_stride, void* stream) {
  if (!h) return DOMINO_ERR_INVALID_ARG;
  domino_status_t st = check_cache(h, "read", c);
  if (st != DOMINO_OK) return st;
  const int dim = h->cfg.head_dim;
  if (!h->fp4) return say(h->err, DOMINO_ERR_UNSUPPORTED, "read: for caches in 4 bits");
  if (c->tokens == 0 || c->max_new == 0) return DOMINO_OK;
  if (!k || !v) return say(h->err, DOMINO_ERR_INVALID_ARG, "read: k and v must be non-NULL");
  if (!rows_ok(k, k_token_stride, k_head_stride, 8) || !rows_ok(v, v_token_stride, v_head_stride, 8))
    return say(h->err, DOMINO_ERR_INVALID_ARG,
               "read: k and v must be 16-byte aligned, their strides multiples of 16 bytes");
  if ((c->tokens > 1 && (k_token_stride < dim || v_token_stride < dim)) ||
      (h->cfg.kv_heads > 1 && (k_head_stride < dim || v_head_stride < dim)))
    return say(h->err, DOMINO_ERR_INVALID_ARG, "read: rows of k or v overlap");
  if (!rows_fit(h, c)) return say(h->err, DOMINO_ERR_UNSUPPORTED, "read: too many rows for a request");
  const RowsArgs4 a = rows_args(h, c, k, k_token_stride, k_head_stride, v, v_token_stride, v_head_stride);
  DeviceGuard dg(h->device);
  (void)hipGetLastError();
  launch_read_fp4(a, (hipStream_t)stream);
  return launched(h, "read");
}

template <int D>
static void launch_attend_f32(const AttendArgs& a, int cus, hipStream_t st) {
  const int64_t rows = (int64_t)a.max_new * a.group, tiles = (rows + 15) / 16;
  const int64_t segments = tiles * a.kv_heads * a.requests, keys = (a.max_kv + 63) / 64;
  // a workgroup to each half of a CU, with at least 64 keys
  int64_t splits = 2 * cus / segments;
  if (splits > keys) splits = keys;
  if (splits < 1) splits = 1;
  hipLaunchKernelGGL((attend_f32_kernel<D>), dim3((unsigned)(tiles * splits), a.kv_heads, a.requests), dim3(256), 0, st,
                     a, (int)splits);
}

extern "C" domino_status_t domino_attention_run(domino_attention_t* h, const domino_cache_t* c,
                                                const void* q, int64_t q_token_stride,
                                                int64_t q_head_stride, int32_t window,
                                                int32_t sinks, float scale, void* out,
                                                int64_t out_token_stride, int64_t out_head_stride,
                                                float* lse, void* stream) {
  if (!h) return DOMINO_ERR_INVALID_ARG;
  domino_status_t st = check_cache(h, "run", c);
  if (st != DOMINO_OK) return st;
  const domino_attention_config_t& f = h->cfg;
  const int unit = f.dtype == DOMINO_DTYPE_BF16 ? 8 : 4;
  if (window < 0 || sinks < 0)
    return say(h->err, DOMINO_ERR_INVALID_ARG, "run: window and sinks must be >= 0");
  if (!(scale > 0.f) || !std::isfinite(scale))
    return say(h->err, DOMINO_ERR_INVALID_ARG, "run: scale must be finite and > 0");
  if (c->tokens == 0 || c->max_new == 0) return DOMINO_OK;
  if (!q || !out) return say(h->err, DOMINO_ERR_INVALID_ARG, "run: q and out must be non-NULL");
  if (!rows_ok(q, q_token_stride, q_head_stride, unit) || !rows_ok(out, out_token_stride, out_head_stride, unit))
    return say(h->err, DOMINO_ERR_INVALID_ARG,
               "run: q and out must be 16-byte aligned, their strides multiples of 16 bytes");
  if ((c->tokens > 1 && out_token_stride < f.head_dim) || (f.q_heads > 1 && out_head_stride < f.head_dim))
    return say(h->err, DOMINO_ERR_INVALID_ARG, "run: rows of out overlap");
  if ((uintptr_t)lse & 3) return say(h->err, DOMINO_ERR_INVALID_ARG, "run: lse must be 4-byte aligned");
  const int32_t max_new = c->max_new < c->tokens ? c->max_new : c->tokens;
  if ((int64_t)max_new * (f.q_heads / f.kv_heads) > (1 << 30))
    return say(h->err, DOMINO_ERR_UNSUPPORTED, "run: too many rows for a request");
  AttendArgs a{};
  a.q = q;
  a.out = out;
  a.lse = lse;
  a.k = c->k_cache;
  a.v = c->v_cache;
  a.q_tok = q_token_stride;
  a.q_head = q_head_stride;
  a.o_tok = out_token_stride;
  a.o_head = out_head_stride;
  a.page = c->page_stride;
  a.head = c->head_stride;
  a.row = (int32_t)c->row_stride;
  a.num_pages = c->num_pages;
  a.table = c->page_table;
  a.table_stride = c->table_stride;
  a.page_shift = __builtin_ctz(f.page_size);
  a.kv_len = c->kv_len;
  a.q_start = c->q_start;
  a.requests = c->requests;
  a.tokens = c->tokens;
  // a request can have no more tokens than there are, nor more keys than its
  // table holds
  a.max_new = max_new;
  a.max_kv = clip_kv(c, f.page_size);
  a.q_heads = f.q_heads;
  a.kv_heads = f.kv_heads;
  a.group = f.q_heads / f.kv_heads;
  // a window that no position reaches past hides nothing
  a.window = window >= a.max_kv ? 0 : window;
  a.sinks = sinks < a.max_kv ? sinks : a.max_kv;
  a.scale = scale;
  a.scale_log2 = scale * 1.44269504088896340736f;
  DeviceGuard dg(h->device);
  (void)hipGetLastError();
  if (f.dtype == DOMINO_DTYPE_BF16) {
    a.part_o = h->part;
    a.part_ml = h->part + attend_split_floats(f.head_dim, h->cus) / (f.head_dim + 2) * f.head_dim;
    a.plan = h->plan;
    if (h->fp4)
      launch_attend_fp4(f.head_dim, a, h->cus, (hipStream_t)stream);
    else
      launch_attend_split(f.head_dim, a, h->cus, (hipStream_t)stream);
  } else {
    a.part_o = h->part;
    a.part_ml = h->part + attend_f32_floats(f.head_dim, h->cus) / (f.head_dim + 2) * f.head_dim;
    a.arrived = h->arrived;
    if (f.head_dim == 64)
      launch_attend_f32<64>(a, h->cus, (hipStream_t)stream);
    else if (f.head_dim == 128)
      launch_attend_f32<128>(a, h->cus, (hipStream_t)stream);
    else
      launch_attend_f32<256>(a, h->cus, (hipStream_t)stream);
  }
  return launched(h, "run");
}
