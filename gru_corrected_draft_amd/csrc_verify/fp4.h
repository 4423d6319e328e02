// A key-value cache in 4 bits: its numbers, and tiles of it in LDS.
//
// 32 elements of a row (a token and key head) share a power of two, the byte
// e + 127 with 255 for NaN; an element is a sign and one of 0, 0.5, 1, 1.5, 2,
// 3, 4, 6.  In a page of a head lie the elements of all rows, D / 2 bytes each
// with the lower element in the low bits, then the powers, D / 32 bytes a row.
//
// Every such number times its power is a bf16 number, and the hardware converts
// two of them in an instruction that takes the power along.
#pragma once
#include "attention_bf16.h"

typedef __bf16 v2bf __attribute__((ext_vector_type(2)));

// the scale operand of the conversions: a float whose exponent counts
__device__ __forceinline__ float power_of(uint32_t byte) { return __uint_as_float(byte << 23); }

// eight elements
__device__ __forceinline__ v8s from_fp4(uint32_t x, float power) {
  u32x4 r;
  r[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(x, power, 0));
  r[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(x, power, 1));
  r[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(x, power, 2));
  r[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(x, power, 3));
  return __builtin_bit_cast(v8s, r);
}

// A tile of 32 keys as it lies in the cache, for heads of 128 and 256: four chunks of 16 rows, two of K
// and two of V, then their powers.  A piece is the 16 bytes of a block of 32
// elements.
template <int D>
struct RawTile {
  static constexpr int kBlocks = D / 32;       // of a row
  static constexpr int kChunk = 8 * D;         // bytes of 16 rows
  static constexpr int kPowers = 4 * kChunk;   // where the powers begin
  static constexpr int kBytes = kPowers + 2 * D;
  static constexpr int kData = D < 128 ? 1 : D / 128;   // copies of a chunk's elements
  static constexpr int kLoads = 4 * (kData + 1);        // copies of a tile

  // Row and block that a lane copies and converts in a chunk's copy j.  The 16
  // lanes that write to LDS together then write 16 different pieces of the
  // bf16 tile's 256 bytes of banks, whose swizzle goes by these bits of the row.
  static __device__ __forceinline__ int row_of(int lane) { return (lane >> 2 & 3) << 2 | lane >> 4; }
  static __device__ __forceinline__ int block_of(int lane, int j) { return (lane & 3) + 4 * j; }
  static __device__ __forceinline__ uint32_t source(int lane, int j) {
    return row_of(lane) * (D / 2) + block_of(lane, j) * 16;
  }

  // chunk c of the tile at `slot`, from its elements and powers in the cache
  static __device__ __forceinline__ void copy(const char* data, const char* powers, const uint32_t (&src)[kData],
                                              const lds_byte* slot, int c, int lane) {
#pragma unroll
    for (int j = 0; j < kData; ++j) copy_to_lds(data, src[j], slot + c * kChunk + j * 1024);
    if (lane < D / 32) copy_to_lds(powers, 16 * lane, slot + kPowers + c * (D / 2));
  }

  // chunk c, by the wave that copied it (as source says), into a bf16 tile
  static __device__ __forceinline__ void convert(const lds_byte* slot, int c, lds_byte* tile, int lane) {
    using T = KeyTile<D>;
    const int row = row_of(lane), swizzle = T::swizzle(row);
    lds_byte* const to = tile + (c >> 1) * T::kHalf + ((c & 1) * 16 + row) * T::kRow;
#pragma unroll
    for (int j = 0; j < kData; ++j) {
      const int block = block_of(lane, j);
      const u32x4 x = __builtin_bit_cast(u32x4, lds_read16(slot + c * kChunk + j * 1024 + lane * 16));
      const float power = power_of(slot[kPowers + c * (D / 2) + row * kBlocks + block]);
#pragma unroll
      for (int q = 0; q < 4; ++q)
        *(__attribute__((address_space(3))) v8s*)(to + (((4 * block + q) ^ swizzle) << 4)) = from_fp4(x[q], power);
    }
  }
};

// what is done to a row, 8 elements to a lane
struct RowsArgs4 {
  void* tok[2];  // [tokens][heads][D] bf16, keys and values
  void* cache[2];
  int64_t tok_stride[2], head_stride[2];
  int64_t page, head;  // bytes
  int32_t num_pages, head_dim;
  const int32_t* table;
  int64_t table_stride;
  int32_t page_shift;
  const int32_t* kv_len;
  const int32_t* q_start;
  int32_t requests, tokens, max_new, max_kv, kv_heads;
  int32_t piece_shift;  // 2^that pieces of 8 elements in a row
  uint32_t magic;       // i / pieces of a token = (high half of magic i, + i) >> magic_shift, i < 2^31
  int32_t magic_shift;
};

hipError_t attend_fp4_prepare(int head_dim);
void launch_attend_fp4(int head_dim, const AttendArgs& a, int cus, hipStream_t st);
void launch_append_fp4(const RowsArgs4& a, hipStream_t st);
void launch_read_fp4(const RowsArgs4& a, hipStream_t st);
