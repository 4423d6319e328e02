// Arguments and device helpers shared by the paged-attention kernels.
//
// Rows.  The new tokens of a request and the query heads that share a key
// head form one list of rows per (request, key head): row r is token
// r / group, head r % group of the group, so a draft block of 16 positions
// with 4 heads to a key head is 64 rows that read the same keys.  A row tile
// is a run of consecutive rows handled together.
//
// Keys.  A row tile sees keys [0, sinks) and [lo, hi): hi is one past its
// last row's position, lo the first key in its first row's window (0 without
// a window).  They are walked in key tiles aligned to the tile size; tiles
// between the sinks and lo are never touched.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "common.h"

typedef float v16f __attribute__((ext_vector_type(16)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef const int32_t __attribute__((address_space(4))) const_i32;

struct AttendArgs {
  const void* q;
  void* out;
  float* lse;
  const void* k;
  const void* v;
  int64_t q_tok, q_head, o_tok, o_head;  // element strides
  int64_t page, head;
  int32_t row;
  int32_t num_pages;
  const int32_t* table;
  int64_t table_stride;
  int32_t page_shift;
  const int32_t* kv_len;
  const int32_t* q_start;
  int32_t requests, tokens, max_new, max_kv;
  int32_t q_heads, kv_heads, group;
  int32_t window, sinks;  // window 0: none
  float scale, scale_log2;
  // split attention
  float* part_o;   // [slots][rows][head_dim]
  float* part_ml;  // [slots][rows][2]
  int32_t* plan;   // bf16: [max(requests, 64) + 1]
  int32_t* arrived;  // fp32: [CUs] parts there are of a row tile and key head; 0 between calls
  int32_t row_tiles;  // of the longest request there can be
  bool pieces;  // segments cut for themselves
};

// A value that is the same in every lane, in a scalar register: branches and
// loads that follow from it stay scalar.
__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }

// rows of the token arrays and keys of request b
struct Request {
  int q0, n, kv;
  bool bad;
};

__device__ __forceinline__ Request request_of(const int32_t* q_start_, const int32_t* kv_len_, int b,
                                              int tokens, int max_new, int max_kv) {
  // constant memory: scalar loads where b is the same in every lane
  const_i32* const q_start = (const_i32*)q_start_;
  const_i32* const kv_len = (const_i32*)kv_len_;
  const int s0 = q_start[b], s1 = q_start[b + 1];
  Request r;
  r.kv = kv_len[b];
  const int64_t n = (int64_t)s1 - s0;
  r.bad = s0 < 0 || s1 > tokens || n < 0 || n > max_new || r.kv < 0 || r.kv > max_kv;
  r.q0 = s0 < 0 ? 0 : s0;
  const int end = s1 > tokens ? tokens : s1;
  r.n = end > r.q0 ? end - r.q0 : 0;
  if (r.n > max_new) r.n = max_new;
  if (r.bad) r.kv = 0;
  return r;
}

// key tiles of one row tile
struct KeySpan {
  int pmin, pmax;  // positions of the tile's first and last row's token
  int hi, lo;
  int sink_tiles, first, count;  // tile i: i < sink_tiles ? i : first + i - sink_tiles
};

template <int KT>
__device__ __forceinline__ KeySpan key_span(const Request& r, int t_first, int t_last, int window,
                                            int sinks) {
  KeySpan s;
  s.pmin = r.kv - r.n + t_first;
  s.pmax = r.kv - r.n + t_last;
  s.hi = s.pmax + 1;
  s.lo = 0;
  if (window > 0 && s.pmin - window + 1 > 0) s.lo = s.pmin - window + 1;
  s.sink_tiles = s.first = s.count = 0;
  if (s.hi <= 0) return s;
  s.first = s.lo / KT;
  const int st = (sinks + KT - 1) / KT;
  s.sink_tiles = st < s.first ? st : s.first;
  s.count = s.sink_tiles + (s.hi + KT - 1) / KT - s.first;
  return s;
}

__device__ __forceinline__ KeySpan uniform(const KeySpan& s) {
  return KeySpan{uniform(s.pmin),       uniform(s.pmax),  uniform(s.hi),   uniform(s.lo),
                 uniform(s.sink_tiles), uniform(s.first), uniform(s.count)};
}

__device__ __forceinline__ int tile_of(const KeySpan& s, int i) {
  return i < s.sink_tiles ? i : s.first + i - s.sink_tiles;
}

// whether every row of the tile sees all `n` keys from k0 on
__device__ __forceinline__ bool all_visible(const KeySpan& s, int k0, int n, int window, int sinks) {
  return k0 + n - 1 <= s.pmin && (window == 0 || k0 > s.pmax - window || k0 + n <= sinks);
}

// Ranges of tile indices: [whole_lo, whole_hi) are tiles that all rows see
// whole, and of those from sink_hi on, which hold no sink, some row sees a key
// of [some_lo, some_hi).
struct TileRange {
  int whole_lo, whole_hi, some_lo, some_hi, sink_hi;
};

__device__ __forceinline__ int floor_div(int a, int b) { return a >= 0 ? a / b : -((b - 1 - a) / b); }

template <int KT>
__device__ __forceinline__ TileRange tile_range(const KeySpan& s, int window, int sinks) {
  const int shift = s.sink_tiles - s.first;  // index of a tile past the sinks, less the tile
  TileRange r;
  r.whole_hi = floor_div(s.pmin + 1, KT) + shift;
  r.whole_lo = s.sink_tiles;
  r.some_hi = floor_div(s.pmax, KT) + 1 + shift;
  r.some_lo = s.sink_tiles;
  r.sink_hi = (sinks + KT - 1) / KT + shift;
  if (r.sink_hi < s.sink_tiles) r.sink_hi = s.sink_tiles;
  if (window > 0) {
    const int lo = floor_div(s.pmax - window, KT) + 1 + shift;      // first key > pmax - window
    if (lo > r.whole_lo) r.whole_lo = lo;
    const int some = floor_div(s.pmin - window + 1, KT) + shift;    // last key > pmin - window
    if (some > r.some_lo) r.some_lo = some;
  }
  return r;
}

__device__ __forceinline__ TileRange uniform(const TileRange& r) {
  return TileRange{uniform(r.whole_lo), uniform(r.whole_hi), uniform(r.some_lo), uniform(r.some_hi),
                   uniform(r.sink_hi)};
}

__device__ __forceinline__ bool visible(int key, int p, int window, int sinks) {
  return key <= p && (window == 0 || key > p - window || key < sinks);
}

// two floats rounded to bf16 (nearest even, NaN kept), lower one first
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
  const v2bf r = {(__bf16)a, (__bf16)b};
  return __builtin_bit_cast(uint32_t, r);
}
// x f, an infinity kept where f has underflowed
__device__ __forceinline__ float scaled(float x, float f) { return __builtin_isinf(x) ? x : x * f; }

__device__ __forceinline__ bool nonfinite(float x) {
  return (__float_as_uint(x) & 0x7F800000u) == 0x7F800000u;
}
