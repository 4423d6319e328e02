// bf16 attention over a cache in 4 bits, the append that fills it and the read
// that gives back what stands there.
#include "attention_few.h"
#include "attention_split.h"

namespace {

// Row tiles of 32 rows save conversions over 16 where there are so many; for
// heads of 256 their sums do not fit in registers.
template <int D>
constexpr int kRowGroups = D == 256 ? 1 : 2;
template <int D>
constexpr int kManyWaves = D == 256 ? 8 : 16;  // what a CU holds

template <int D>
hipError_t prepare_fp4() {
  hipError_t e = allow_few<D, 1, 4>();
  if (e == hipSuccess) e = allow_few<D, 1, kManyWaves<D>>();
  if (D < 256 && e == hipSuccess) e = allow_few<D, kRowGroups<D>, 4>();
  if constexpr (D < 256) {
    if (e == hipSuccess) e = allow_lds<D, 8, true>();
  }
  if (e == hipSuccess) e = allow_lds<D, 4, true>();
  return e;
}

template <int D>
void launch_fp4(const AttendArgs& a, int cus, hipStream_t st) {
  const int64_t rows = (int64_t)a.max_new * a.group;
  if (rows <= 64 || (rows <= 128 && a.max_kv <= 4096)) {
    if ((rows + 15) / 16 * a.requests * a.kv_heads <= cus) return launch_few<D, 1, kManyWaves<D>>(a, cus, cus, st);
    if (rows <= 16) return launch_few<D, 1, 4>(a, 2 * cus, cus, st);
    return launch_few<D, kRowGroups<D>, 4>(a, 2 * cus, cus, st);
  }
  if constexpr (D < 256) {
    if (rows > 128) return launch<D, 8, true>(a, cus, st);
  }
  launch<D, 4, true>(a, cus, st);
}

}  // namespace

hipError_t attend_fp4_prepare(int head_dim) {
  return head_dim == 64 ? prepare_fp4<64>() : head_dim == 128 ? prepare_fp4<128>() : prepare_fp4<256>();
}

void launch_attend_fp4(int head_dim, const AttendArgs& a, int cus, hipStream_t st) {
  if (head_dim == 64)
    launch_fp4<64>(a, cus, st);
  else if (head_dim == 128)
    launch_fp4<128>(a, cus, st);
  else
    launch_fp4<256>(a, cus, st);
}

namespace {

// where 8 elements of a token's row lie, or nowhere
struct Place {
  int64_t token;        // elements into the token array
  char* data;           // 4 bytes
  char* power;          // the block's
  bool there;
};

// Walks the rows of a request's new tokens, 8 elements to a lane (four lanes
// to a block of 32): grid.y is 2 x requests, keys and values.
template <class F>
__device__ __forceinline__ void each_piece(const RowsArgs4& a, const Request& r, int which, int b, F f) {
  const int pieces = a.head_dim / 8, per_token = a.kv_heads * pieces;
  const int64_t total = (int64_t)r.n * per_token;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    const int t = (int)(i / per_token), rest = (int)(i - (int64_t)t * per_token);
    const int h = rest / pieces, piece = rest - h * pieces;
    const int pos = r.kv - r.n + t;
    Place p;
    p.token = (r.q0 + t) * a.tok_stride[which] + h * a.head_stride[which] + 8 * piece;
    const int page = r.bad || pos < 0 ? -1 : a.table[b * a.table_stride + (pos >> a.page_shift)];
    p.there = page >= 0 && page < a.num_pages;
    const int row = pos & ((1 << a.page_shift) - 1);
    char* const at = (char*)a.cache[which] + (p.there ? page * a.page + h * a.head : 0);
    p.data = at + (int64_t)row * (a.head_dim / 2) + 4 * piece;
    p.power = at + ((int64_t)(a.head_dim / 2) << a.page_shift) + (int64_t)row * (a.head_dim / 32) + piece / 4;
    f(p, piece);
  }
}

// The largest magnitude of a block gives its power: the least with
// max <= 7 x 2^e.  Up to 6 a number is off by at most half a step, and from 6 to
// 7 by no more than the widest half step, 1, so nothing is gained by a larger
// power.  e stays in [-125, 125]: all products are then normal bf16 numbers.
__global__ __launch_bounds__(256) void append_fp4_kernel(RowsArgs4 a) {
  const int which = blockIdx.y & 1, b = blockIdx.y >> 1;
  const Request r = request_of(a.q_start, a.kv_len, b, a.tokens, a.max_new, a.max_kv);
  if (r.bad) return;
  each_piece(a, r, which, b, [&](const Place& p, int piece) {
    if (!p.there) return;
    const u32x4 x = *(const u32x4*)((const bf16_t*)a.tok[which] + p.token);
    // magnitudes as whole numbers order like the values, infinities and NaN last
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t lo = x[i] & 0x7FFF, hi = x[i] >> 16 & 0x7FFF;
      top = max(top, max(lo, hi));
    }
    top = max(top, __shfl_xor(top, 1, 64));
    top = max(top, __shfl_xor(top, 2, 64));
    // 7 x 2^e is 1.75 x 2^(e + 2): beyond a significand of 1.75 the next power
    int byte = (int)((top + 0x1F) >> 7) - 2;
    byte = byte < 2 ? 2 : byte > 252 ? 252 : byte;
    const bool odd = top >= 0x7F80;
    uint32_t y = 0;
    if (!odd) {
      v2bf two[4];
      __builtin_memcpy(two, &x, 16);
      const float power = power_of(byte);
      y = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(y, two[0], power, 0);
      y = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(y, two[1], power, 1);
      y = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(y, two[2], power, 2);
      y = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(y, two[3], power, 3);
    }
    *(uint32_t*)p.data = y;
    if ((piece & 3) == 0) *(uint8_t*)p.power = odd ? 255 : (uint8_t)byte;
  });
}

__global__ __launch_bounds__(256) void read_fp4_kernel(RowsArgs4 a) {
  const int which = blockIdx.y & 1, b = blockIdx.y >> 1;
  const Request r = request_of(a.q_start, a.kv_len, b, a.tokens, a.max_new, a.max_kv);
  each_piece(a, r, which, b, [&](const Place& p, int) {
    v8s y;
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = 0x7FC0;
    if (p.there) y = from_fp4(*(const uint32_t*)p.data, power_of(*(const uint8_t*)p.power));
    *(v8s*)((bf16_t*)a.tok[which] + p.token) = y;
  });
}

dim3 rows_grid(const RowsArgs4& a) {
  const int most = a.max_new < a.tokens ? a.max_new : a.tokens;
  const int64_t blocks = ((int64_t)most * a.kv_heads * (a.head_dim / 8) + 255) / 256;
  return dim3((unsigned)(blocks < 1024 ? blocks : 1024), 2 * a.requests);
}

}  // namespace

void launch_append_fp4(const RowsArgs4& a, hipStream_t st) {
  hipLaunchKernelGGL(append_fp4_kernel, rows_grid(a), dim3(256), 0, st, a);
}

void launch_read_fp4(const RowsArgs4& a, hipStream_t st) {
  hipLaunchKernelGGL(read_fp4_kernel, rows_grid(a), dim3(256), 0, st, a);
}
