// bf16 attention over a cache in 4 bits, the append that fills it and the read
// that gives back what stands there.
#include "attention_few.h"
#include "attention_split.h"

namespace {

// Row tiles of 32 rows save conversions over 16 where there are so many (32 blocks of 16
// tokens over 8 to 16 thousand keys 201 us against 285); for heads of 256 their sums do
// not fit in registers, and 64 rows of heads of 64 are no faster (16 prompts of 256
// tokens over 4096 keys 200 against 174).
template <int D>
constexpr int kRowGroups = D == 256 ? 1 : 2;
template <int D>
constexpr int kManyWaves = D == 256 ? 8 : 16;  // what a CU holds

template <int D, bool FINE>
hipError_t allow_few_d() {
  hipError_t e = allow_few<D, 1, kManyWaves<D>, FINE>();
  if (e == hipSuccess) e = allow_few<D, kRowGroups<D>, 4, FINE>();
  return e;
}

template <int D>
hipError_t prepare_fp4() {
  hipError_t e = allow_few_d<D, true>();
  if (e == hipSuccess) e = allow_few_d<D, false>();
  if constexpr (D < 256) {
    if (e == hipSuccess) e = allow_few<D, 1, 4, true>();
  }
  if constexpr (D == 128) {
    if (e == hipSuccess) e = allow_lds<D, 8, true>();
  }
  if constexpr (D > 64) {
    if (e == hipSuccess) e = allow_lds<D, 4, true>();
  }
  return e;
}

// Where row tiles of 16 do not fill the CUs, one workgroup of all the waves that a CU
// holds to each: 32 single tokens over 2 to 4 thousand keys 27.3 us against 33.8 with
// workgroups of 4 waves, 8 blocks 21.3 against 29.9.  A block's four row tiles convert
// the same keys each, but fewer of more rows with the keys cut into runs instead are
// slower: 8 blocks 25.3 us in tiles of 32 rows with 8 waves and two runs, 25.7 with 4
// waves, 31.6 in tiles of 64.  Beyond that 4 waves, two workgroups to a CU: they leave the
// wait at the end to others (32 blocks over 8 to 16 thousand keys 201 us, with 8 waves 212;
// 12 over 2 to 4 thousand 31.0 and 32.0, but 16 of them 38.9 and 32.1).
template <int D, bool FINE>
void launch_few_d(const AttendArgs& a, int cus, hipStream_t st) {
  const int64_t rows = (int64_t)a.max_new * a.group;
  if ((rows + 15) / 16 * a.requests * a.kv_heads <= cus) return launch_few<D, 1, kManyWaves<D>, FINE>(a, cus, cus, st);
  if constexpr (FINE) {
    if (rows <= 16) return launch_few<D, 1, 4, true>(a, 2 * cus, cus, st);
  }
  launch_few<D, kRowGroups<D>, 4, FINE>(a, 2 * cus, cus, st);
}

// The kernels of attention_split.h convert a tile once for all rows of a
// workgroup (128 or 256), but start, wait at barriers and join slowly.  They win from
// some work for each CU on, rows x keys:
//   heads of 64    never: 16 prompts of 512 tokens of 16 heads over up to 16384 keys
//                  took 612 us here (589 since) and 800 there, one over 1024 13 and 24
//   128, to 128 rows   at 2^20: 16 of 128 rows over 8192 keys (half of that) 105 and
//                  114, over 16384 201 and 206, 32 over 16384 (twice) 360 and 324
//   128, beyond    at 2^18: 256 tokens over 4096 keys (half) 40 and 47, over
//                  16384 (twice) 111 and 95
//   256            at 2^16: 32 tokens of 4 requests over 4096 keys 50 and 56, over
//                  8192 91 and 80
template <int D>
void launch_fp4(const AttendArgs& a, int cus, hipStream_t st) {
  const int64_t rows = (int64_t)a.max_new * a.group;
  if (rows <= 32) return launch_few_d<D, true>(a, cus, st);
  if constexpr (D > 64) {
    // rows times keys for each CU
    const double work = (double)a.requests * a.kv_heads * rows * few_keys(a) / cus;
    const int most = D == 256 ? 1 << 16 : rows <= 128 ? 1 << 20 : 1 << 18;
    if (rows > 64 && work > most) {
      if constexpr (D == 128) {
        if (rows > 128) return launch<D, 8, true>(a, cus, st);
      }
      return launch<D, 4, true>(a, cus, st);
    }
  }
  launch_few_d<D, false>(a, cus, st);
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

// Append and read: 8 elements to a lane, four lanes to a block of 32, grid.y is
// 2 x requests, keys and values.  Both are bound by the chain from the lengths over
// the page table to memory, so a lane takes kPieces at a time, their loads on their
// way together (prompts of 8 requests up to 1024 tokens, both after one another: 19.2 us,
// with one piece 19.9; 64 requests of 64 tokens 14.7 and 14.8, but one prompt of 512, whose
// lanes have a piece each either way, 7.2 and 6.1).
constexpr int kPieces = 4;

// where a piece lies, or nowhere
struct Place {
  int64_t token;  // elements into the token array
  int64_t data;   // bytes into the cache: 4 of elements,
  int64_t power;  // the block's
  int piece;
  bool mine, there;
};

__device__ __forceinline__ Place place_of(const RowsArgs4& a, const Request& r, int which, int b, uint32_t i) {
  const uint32_t per_token = (uint32_t)a.kv_heads << a.piece_shift;
  Place p;
  p.mine = i < (uint32_t)r.n * per_token;
  if (!p.mine) i = 0;
  const int t = (int)((__umulhi(a.magic, i) + i) >> a.magic_shift), rest = (int)(i - t * per_token);  // t = i / per_token
  const int h = rest >> a.piece_shift;
  p.piece = rest & ((1 << a.piece_shift) - 1);
  const int pos = r.kv - r.n + t;
  p.token = (r.q0 + t) * a.tok_stride[which] + h * a.head_stride[which] + 8 * p.piece;
  const int page = !p.mine || r.bad || pos < 0 ? -1 : a.table[b * a.table_stride + (pos >> a.page_shift)];
  p.there = page >= 0 && page < a.num_pages;
  const int row = pos & ((1 << a.page_shift) - 1);
  const int64_t at = p.there ? page * a.page + h * a.head : 0;
  p.data = at + (int64_t)row * (a.head_dim / 2) + 4 * p.piece;
  p.power = at + ((int64_t)(a.head_dim / 2) << a.page_shift) + (int64_t)row * (a.head_dim / 32) + p.piece / 4;
  return p;
}

// The largest magnitude of a block gives its power: the least with
// max <= 7 x 2^e.  Up to 6 a number is off by at most half a step, and from 6 to
// 7 by no more than the widest half step, 1, so nothing is gained by a larger
// power.  e stays in [-125, 125]: all products are then normal bf16 numbers.
__device__ __forceinline__ void store_fp4(const u32x4& x, const Place& p, char* cache) {
  // magnitudes as whole numbers order like the values, infinities and NaN last
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) top = max(top, max(x[i] & 0x7FFF, x[i] >> 16 & 0x7FFF));
  top = max(top, __shfl_xor(top, 1, 64));
  top = max(top, __shfl_xor(top, 2, 64));
  if (!p.there) return;
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
  *(uint32_t*)(cache + p.data) = y;
  if ((p.piece & 3) == 0) *(uint8_t*)(cache + p.power) = odd ? 255 : (uint8_t)byte;
}

__global__ __launch_bounds__(256) void append_fp4_kernel(RowsArgs4 a) {
  const int which = blockIdx.y & 1, b = blockIdx.y >> 1;
  const Request r = request_of(a.q_start, a.kv_len, b, a.tokens, a.max_new, a.max_kv);
  if (r.bad) return;
  const uint32_t total = ((uint32_t)r.n * a.kv_heads) << a.piece_shift, step = gridDim.x * 256;
  for (uint32_t i = blockIdx.x * 256 + threadIdx.x; i < total; i += kPieces * step) {
    Place p[kPieces];
    u32x4 x[kPieces];
#pragma unroll
    for (int u = 0; u < kPieces; ++u) {
      p[u] = place_of(a, r, which, b, i + u * step);
      x[u] = p[u].mine ? *(const u32x4*)((const bf16_t*)a.tok[which] + p[u].token) : u32x4{0, 0, 0, 0};
    }
#pragma unroll
    for (int u = 0; u < kPieces; ++u) store_fp4(x[u], p[u], (char*)a.cache[which]);
  }
}

__global__ __launch_bounds__(256) void read_fp4_kernel(RowsArgs4 a) {
  const int which = blockIdx.y & 1, b = blockIdx.y >> 1;
  const Request r = request_of(a.q_start, a.kv_len, b, a.tokens, a.max_new, a.max_kv);
  const uint32_t total = ((uint32_t)r.n * a.kv_heads) << a.piece_shift, step = gridDim.x * 256;
  const char* const cache = (const char*)a.cache[which];
  for (uint32_t i = blockIdx.x * 256 + threadIdx.x; i < total; i += kPieces * step) {
    Place p[kPieces];
    uint32_t x[kPieces], power[kPieces];
#pragma unroll
    for (int u = 0; u < kPieces; ++u) {
      p[u] = place_of(a, r, which, b, i + u * step);
      x[u] = p[u].there ? *(const uint32_t*)(cache + p[u].data) : 0;
      power[u] = p[u].there ? *(const uint8_t*)(cache + p[u].power) : 255;
    }
#pragma unroll
    for (int u = 0; u < kPieces; ++u)
      if (p[u].mine) *(v8s*)((bf16_t*)a.tok[which] + p[u].token) = from_fp4(x[u], power_of(power[u]));
  }
}

// A piece to a lane up to 1024 workgroups, then up to kPieces.
dim3 rows_grid(const RowsArgs4& a) {
  const int most = a.max_new < a.tokens ? a.max_new : a.tokens;
  const int64_t all = ((int64_t)most * a.kv_heads * (a.head_dim / 8) + 255) / 256;
  const int64_t few = 512 / a.requests > 0 ? 512 / a.requests : 1;
  int64_t blocks = all < few ? all : (all + kPieces - 1) / kPieces;
  if (all > few && blocks < few) blocks = few;
  return dim3((unsigned)(blocks < 1024 ? blocks : 1024), 2 * a.requests);
}

}  // namespace

void launch_append_fp4(const RowsArgs4& a, hipStream_t st) {
  hipLaunchKernelGGL(append_fp4_kernel, rows_grid(a), dim3(256), 0, st, a);
}

void launch_read_fp4(const RowsArgs4& a, hipStream_t st) {
  hipLaunchKernelGGL(read_fp4_kernel, rows_grid(a), dim3(256), 0, st, a);
}
