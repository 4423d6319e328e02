// What the bf16 attention kernels share: key tiles in LDS and the two products
// on 32 x 32 matrix-core tiles.
//
// Both products are computed transposed, so that a lane keeps one row of the
// row tile: S^T = K Q^T (keys x rows) and O^T = V^T P^T (elements x rows).
// With V_MFMA_F32_32X32X16_BF16 lane l (n = l % 32, h = l / 32) holds in
// accumulator register i row 8 (i / 4) + 4 h + i % 4 of column n.  The keys
// are dealt to the rows of S^T so that registers 8 c .. 8 c + 7 are the keys
// 16 c + 8 h .. + 7: exactly the slots of the second product's operand, so the
// weights go from one product to the next without leaving their lane.
//
// A key tile is 32 rows of K and 32 of V, copied from the pages straight into
// LDS as rows of 2 D bytes.  Within a row the 16-byte pieces are permuted by
// an exclusive or with a function of the row, chosen so that neither the
// fragments of K (16 rows at one piece) nor those of V (8 rows at four pieces,
// read through the transposing load) meet in a bank more than they must.  The
// copy writes LDS in lane order, so each lane picks the piece that belongs
// where it lands.
#pragma once
#include "attention.h"

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) unsigned char lds_byte;

__device__ __forceinline__ v16f mfma_32x32(v8s a, v8s b, v16f c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v8bf, a), __builtin_bit_cast(v8bf, b), c,
                                                 0, 0, 0);
}

// Copies 16 bytes per lane from base + off into LDS, lane l at dst + 16 l.
// Written out because the compiler, which knows what the builtin writes, waits
// for every copy in flight before each transposing read of LDS; no register is
// written, and wait_copies is what orders the copies.  m0 is free: the compiler
// sets it right before each use of its own.
__device__ __forceinline__ void copy_to_lds(const void* base, uint32_t off, const lds_byte* dst) {
  const uint32_t to = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(uintptr_t)dst);
  asm volatile(
      "s_mov_b32 m0, %2\n\t"
      "s_nop 0\n\t"
      "global_load_lds_dwordx4 %0, %1"
      :
      : "v"(off), "s"(base), "s"(to)
      : "memory");
}

template <int N>
__device__ __forceinline__ void wait_copies() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

template <int D>
struct KeyTile {
  static constexpr int kPieces = D / 8;            // 16-byte pieces of a row
  static constexpr int kRow = 2 * D;               // bytes
  static constexpr int kHalf = 32 * kRow;          // bytes of the K (or V) tile
  static constexpr int kBytes = 2 * kHalf;
  static constexpr int kChunkLoads = 16 * kRow / 1024;  // copies of 1 KB to 16 rows
  static constexpr int kLoads = 4 * kChunkLoads;   // copies of a tile

  static __device__ __forceinline__ int swizzle(int row) {
    if constexpr (D == 64) {
      const int r = (row >> 1) & 7;
      return ((r & 1) << 2) | (r & 2) | (r >> 2);
    } else {
      const int r = row & 15;
      return ((r & 3) << 2) | (r >> 2);
    }
  }

  // bytes from the start of a 16-row chunk in the cache to what lane `lane`
  // copies in the chunk's j-th copy
  static __device__ __forceinline__ uint32_t source(int j, int lane, int row_bytes) {
    const int piece = j * 64 + lane, row = piece / kPieces;
    return row * row_bytes + (((piece % kPieces) ^ swizzle(row)) << 4);
  }

  // LDS bytes (from the tile's start) of this lane's K fragment of step 0; step
  // kc is at k_step(that, kc)
  static __device__ __forceinline__ uint32_t k_first(int lane) {
    const int m = lane & 31, h = lane >> 5;
    const int key = 16 * (m >> 4) + 8 * ((m >> 2) & 1) + 4 * ((m >> 3) & 1) + (m & 3);
    return key * kRow + ((h ^ swizzle(key)) << 4);
  }
  static __device__ __forceinline__ uint32_t k_step(uint32_t first, int kc) {
    return (first ^ ((kc & 7) << 5)) + (kc >> 3) * 256;
  }
  // of the half e of this lane's V fragment of elements 0..31, keys 0..15
  static __device__ __forceinline__ uint32_t v_first(int lane, int e) {
    const int g = lane >> 4, j = lane & 15;
    const int key = 8 * (g >> 1) + 4 * e + (j >> 2), piece = 2 * (g & 1) + ((j & 3) >> 1);
    return kHalf + key * kRow + ((piece ^ swizzle(key)) << 4) + ((j & 1) << 3);
  }
  static __device__ __forceinline__ uint32_t v_step(uint32_t first, int block, int c) {
    return (first ^ ((block & 3) << 6)) + (block >> 2) * 256 + c * 16 * kRow;
  }
};

// 16 bytes of LDS per lane
__device__ __forceinline__ v8s lds_read16(const lds_byte* p) {
  return *(const __attribute__((address_space(3))) v8s*)p;
}
// Transposing read: of the 16 x 4 block that 16 lanes point at (4 rows of 16
// elements), lane j of them gets column j.
__device__ __forceinline__ v4s lds_read_tr(const lds_byte* p) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) v4s*)p);
}

__device__ __forceinline__ float max_halves(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float sum_halves(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

__device__ __forceinline__ int scan_lanes(int x, int lane) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int y = __shfl_up(x, d, 64);
    if (lane >= d) x += y;
  }
  return x;
}

__device__ __forceinline__ Request of_lane(const Request& r, int lane) {
  return Request{__builtin_amdgcn_readlane(r.q0, lane), __builtin_amdgcn_readlane(r.n, lane),
                 __builtin_amdgcn_readlane(r.kv, lane), (bool)__builtin_amdgcn_readlane((int)r.bad, lane)};
}

// One row tile's state in a wave: 32 rows, lane n = l % 32 holds row n in both
// halves (m in both, l as each half's part).  m is what the exponents are taken
// against: a score the row has met, at most kSlack (in powers of two) below its
// largest, so that the sums are rescaled only when a row's maximum has grown by
// more than that.  Weights stay below 2^kSlack, and neither fp32 sums nor bf16
// weights lose by a common factor.
template <int D>
struct RowState {
  v16f o[D / 32];
  float m, l;
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
#pragma unroll
      for (int j = 0; j < 16; ++j) o[i][j] = 0.f;
    m = -INFINITY;
    l = 0.f;
  }
};

constexpr float kSlack = 8.f;

// Scores of N tiles to weights: updates the running sum, first rescaling what
// there is where the maximum has outgrown m, and leaves the weights for the
// second product, whose operands are bf16.
//   FINE: as the sum of two bf16 numbers, p and rest, for a product each; off by
//   at most 2^-15, so the result's own rounding is all that shows (0.0017 of it
//   in the root mean square).  The first is cut off, not rounded, and the second
//   kept above 0, so that an infinite value meets two weights of one sign.  For
//   up to 32 rows, bound by bytes, this costs 0 to 2 % (64 requests with one
//   token each 285 us with it and without, 8 requests over 4096 keys 29.1 and
//   28.5).
//   Otherwise rounded to bf16 once (0.0023 of the result): a second product
//   would take a block of 8 requests from 34 us to 37, one with a window from 66
//   to 80 and a prompt from 237 to 318.
template <int D, int N, bool FINE>
__device__ __forceinline__ void softmax_step(v16f (&s)[N], RowState<D>& st, v8s (&p)[N][2], v8s (&rest)[N][2],
                                             float scale_log2) {
  float top = fmaxf(s[0][0], s[0][1]);
#pragma unroll
  for (int i = 2; i < 16 * N; ++i) top = fmaxf(top, s[i / 16][i % 16]);
  top = max_halves(top);
  // also true at a row's first visible score, where m is -inf
  if (__any(top * scale_log2 > st.m * scale_log2 + kSlack)) {
    const float mn = fmaxf(st.m, top);
    const float alpha = mn == -INFINITY ? 1.f : __builtin_amdgcn_exp2f((st.m - mn) * scale_log2);
    st.l *= alpha;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) st.o[i] *= alpha;
    st.m = mn;
  }
  const float ref = st.m == -INFINITY ? 0.f : st.m * scale_log2;
#pragma unroll
  for (int t = 0; t < N; ++t) {
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      s[t][i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[t][i], scale_log2, -ref));
      sum += s[t][i];
    }
    st.l += sum;
    uint32_t w[8], r[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if constexpr (FINE) {
        const uint32_t a = __float_as_uint(s[t][2 * i]) & 0xFFFF0000u, b = __float_as_uint(s[t][2 * i + 1]) & 0xFFFF0000u;
        w[i] = a >> 16 | b;
        r[i] = pack_bf16(fmaxf(s[t][2 * i] - __uint_as_float(a), s[t][2 * i] * 0x1p-20f),
                         fmaxf(s[t][2 * i + 1] - __uint_as_float(b), s[t][2 * i + 1] * 0x1p-20f));
      } else {
        w[i] = pack_bf16(s[t][2 * i], s[t][2 * i + 1]);
      }
    }
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      p[t][c] = __builtin_bit_cast(v8s, (u32x4{w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]}));
      if constexpr (FINE) rest[t][c] = __builtin_bit_cast(v8s, (u32x4{r[4 * c], r[4 * c + 1], r[4 * c + 2], r[4 * c + 3]}));
    }
  }
}

// S^T = K Q^T for one tile.  The fragments are all on their way before the
// first product: left to itself the compiler reads one at a time and waits.
template <int D>
__device__ __forceinline__ v16f scores(const lds_byte* tile, uint32_t k0, const v8s (&q)[D / 16]) {
  constexpr int STEP = D / 16 < 8 ? D / 16 : 8;
  v16f s;
#pragma unroll
  for (int i = 0; i < 16; ++i) s[i] = 0.f;
#pragma unroll
  for (int c0 = 0; c0 < D / 16; c0 += STEP) {
    v8s k[STEP];
#pragma unroll
    for (int c = 0; c < STEP; ++c) k[c] = lds_read16(tile + KeyTile<D>::k_step(k0, c0 + c));
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int c = 0; c < STEP; ++c) s = mfma_32x32(k[c], q[c0 + c], s);
  }
  return s;
}

// Fragments of V of 64 elements, and O^T += V^T P^T for them
struct ValueFrags {
  v4s v[2][2][2];
};
template <int D>
__device__ __forceinline__ ValueFrags read_values(const lds_byte* tile, const uint32_t (&v0)[2], int pair) {
  ValueFrags f;
#pragma unroll
  for (int b = 0; b < 2; ++b)
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int e = 0; e < 2; ++e) f.v[b][c][e] = lds_read_tr(tile + KeyTile<D>::v_step(v0[e], 2 * pair + b, c));
  return f;
}
template <int D>
__device__ __forceinline__ void add_values(const ValueFrags& f, int pair, RowState<D>& st, const v8s (&p)[2]) {
#pragma unroll
  for (int c = 0; c < 2; ++c)
#pragma unroll
    for (int b = 0; b < 2; ++b)
      st.o[2 * pair + b] = mfma_32x32(__builtin_shufflevector(f.v[b][c][0], f.v[b][c][1], 0, 1, 2, 3, 4, 5, 6, 7),
                                      p[c], st.o[2 * pair + b]);
}

// Values that are not finite, in tiles that some rows do not see whole: a
// product would multiply them by a weight of zero and spoil rows that do not
// see them.  In such a tile they are noted for the rows that do, and become
// zeros in LDS before its product.  A note is 2 bits for each row and element, +inf and -inf,
// both for NaN; the notes of a wave are [32 rows][D / 8] words of 8 elements.

// whether the tile's values hold an infinity or NaN
template <int D>
__device__ __forceinline__ bool odd_values(const lds_byte* tile, int lane) {
  int odd = 0;
#pragma unroll 1
  for (int i = 0; i < KeyTile<D>::kHalf / 1024; ++i) {
    const v8s v = lds_read16(tile + KeyTile<D>::kHalf + i * 1024 + lane * 16);
#pragma unroll
    for (int j = 0; j < 8; ++j) odd |= (v[j] & 0x7F80) == 0x7F80;
  }
  return __any(odd);
}

typedef __attribute__((address_space(3))) uint16_t lds_u16;

template <int D>
__device__ __forceinline__ void note_odd_values(const lds_byte* tile, lds_u16* notes, int first_key, int pos,
                                                int window, int sinks, int lane) {
  if (lane >= D / 8) return;  // a lane for each piece of a row
#pragma unroll 1
  for (int key = 0; key < 32; ++key) {
    const v8s v = lds_read16(tile + KeyTile<D>::kHalf + key * KeyTile<D>::kRow +
                             ((lane ^ KeyTile<D>::swizzle(key)) << 4));
    uint32_t note = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if ((v[j] & 0x7F80) == 0x7F80) note |= ((v[j] & 0x7F) ? 3 : v[j] < 0 ? 2 : 1) << (2 * j);
    if (!note) continue;
#pragma unroll 1
    for (int row = 0; row < 32; ++row)
      if (visible(first_key + key, __builtin_amdgcn_readlane(pos, row), window, sinks))
        notes[row * (D / 8) + lane] |= (uint16_t)note;
  }
}

// zeros in their place, in part `part` of `parts` of the tile
template <int D>
__device__ __forceinline__ void clear_odd_values(lds_byte* tile, int part, int parts, int lane) {
#pragma unroll 1
  for (int i = part; i < KeyTile<D>::kHalf / 1024; i += parts) {
    lds_byte* const at = tile + KeyTile<D>::kHalf + i * 1024 + lane * 16;
    v8s v = lds_read16(at);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = (v[j] & 0x7F80) == 0x7F80 ? (short)0 : v[j];
    *(__attribute__((address_space(3))) v8s*)at = v;
  }
}

// what a sum becomes by a note's 2 bits
__device__ __forceinline__ float noted(float x, uint32_t bits) {
  return bits == 0 ? x : x + (bits == 3 ? NAN : bits == 2 ? -INFINITY : INFINITY);
}

// once for a device, before the first launch there
hipError_t attend_split_prepare(int head_dim);
void launch_attend_split(int head_dim, const AttendArgs& a, int cus, hipStream_t st);
size_t attend_split_floats(int head_dim, int cus);
