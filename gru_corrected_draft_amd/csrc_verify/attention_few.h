// Attention over a cache in 4 bits where a wave converts what it reads: tokens,
// draft blocks, short prompts, and all calls with heads of 64.
//
// A workgroup takes 16 G rows (a row tile) of a request and key head and a run of
// the tiles of 32 keys that they see; each of its S waves works alone on every S-th
// of them, reads K and V straight into registers, a tile ahead of their use, and
// keeps its own maximum, sum and output.  A wave waits for no other before the end:
// with barriers and V shared by row tiles 8 blocks took 1.4 times as long.
// Products are 16 x 16 x 32, with both results transposed: S^T = K Q^T (keys x
// rows) and O^T = V^T P^T.  Lane l (n = l % 16, q = l / 16) holds row n, of S the keys
// 4 q .. 4 q + 3 of both halves of the tile, which are its slots of the second
// product's operand, and of O the elements 16 x + 4 q .. + 3 of block x.
//   K: lane l converts elements q D / 4 .. of key n of a half: fragments as they
//      are, with the queries' elements dealt alike.
//   V: bf16 rows go through 64 D bytes of LDS of the wave's own for the transposing
//      read, swizzled as in KeyTile.
// FINE keeps each weight as the sum of two bf16 numbers (15 bits), otherwise they
// are rounded once, as over a bf16 cache by the same rule of rows: beyond 32 rows the
// second product is no longer hidden (32 blocks over 8 to 16 thousand keys 234 us
// against 201, 8 blocks over 2 to 4 thousand 23.0 against 21.3, 16 prompts of 512 tokens of
// 32 heads of 64 over 8 to 16 thousand 1505 against 1223; 0.0017 of the result in the root
// mean square, most of it the result's own rounding, against 0.0023).
//
// Units.  A unit is a (request, key head, run of its tiles).  Where the requests
// fill the chip by themselves or are short a run is all of a request's tiles,
// otherwise each request is cut into as many equal runs as workgroups allow and a
// second launch joins them.  Every workgroup finds the division by itself, a lane
// to each request.
//
// What bounds it.  64 single tokens over 4 to 8 thousand keys take 88 us, 4.9 TB/s
// of the cache's bytes (a large copy reaches 5.2, reads alone more).  8 blocks of 16
// tokens over 2 to 4 thousand keys take 21 us for 5 us of bytes: start, queries and
// the joining of streams take about 8, then a wave takes 2 us to a tile, of which
// vector instructions (conversions a third of them) fill 60 % and products 20 %.
// 32-row tiles share each conversion between two products; the scaled products
// that take 4-bit keys as they are were left: their sums lose up to 1e-4 of the
// magnitudes they add.
#pragma once
#include "fp4.h"

namespace {

__device__ __forceinline__ v4f mfma_16x16(v8s a, v8s b, v4f c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, a), __builtin_bit_cast(v8bf, b), c, 0, 0, 0);
}

// over the four lanes that hold a row
__device__ __forceinline__ float max_quarters(float x) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return max_halves(fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1])));
}
__device__ __forceinline__ float sum_quarters(float x) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return sum_halves(__uint_as_float(r[0]) + __uint_as_float(r[1]));
}

// a quarter of a row: D / 4 elements and their powers
template <int D>
struct Quarter {
  static constexpr int kWords = D / 32;
  static constexpr int kPowers = D == 256 ? 2 : 1;
  uint32_t x[kWords];
  // The four bytes among which the powers are: a byte alone would be widened
  // where it lands, a wait for memory in every tile.
  uint32_t powers;
  static __device__ __forceinline__ uint32_t data_at(int row, int part) { return row * (D / 2) + part * (D / 8); }
  static __device__ __forceinline__ int block_of(int part) { return D == 64 ? part >> 1 : part * (D / 128); }
  static __device__ __forceinline__ uint32_t power_at(int row, int part) { return row * (D / 32) + block_of(part); }
  __device__ __forceinline__ void load(const char* data, const char* power) {
    powers = *(const uint32_t*)power;
    if constexpr (D == 64) {
      const u32x2 v = *(const u32x2*)data;
      x[0] = v[0];
      x[1] = v[1];
    } else {
#pragma unroll
      for (int i = 0; i < kWords / 4; ++i) {
        const u32x4 v = *(const u32x4*)(data + 16 * i);
#pragma unroll
        for (int j = 0; j < 4; ++j) x[4 * i + j] = v[j];
      }
    }
  }
  // power e, the first `shift` bits up
  __device__ __forceinline__ uint32_t byte(int e, uint32_t shift) const {
    return __builtin_amdgcn_ubfe(powers, shift + 8 * e, 8);
  }
  // that of word i
  __device__ __forceinline__ float power(int i, uint32_t shift) const { return power_of(byte(D == 256 ? i / 4 : 0, shift)); }
};

template <int D, int G, int S>
struct FewShape {
  static constexpr int kRows = 16 * G;
  static constexpr int kThreads = 64 * S;
  static constexpr int kTile = 64 * D;  // V of a tile in bf16; also 16 rows of sums
  static constexpr int kLds = S * kTile;
};

// What a workgroup does: tiles [first, stop) of request b and key head h, which
// is cut into `runs`.
struct Unit {
  int b, h, first, stop, runs;
};

__device__ __forceinline__ int quotient_up(int x, int y, float inv) {  // about x / y, at least 1
  const int q = (int)((float)(x + y - 1) * inv);
  return q < 1 ? 1 : q;
}

struct FewArgs {
  int32_t units;     // workgroups there are for units; 0: a run is all of a request's tiles
  int32_t per, most; // beyond 64 requests: tiles to a run, and runs to a request, of the longest one
  int32_t least;     // tiles of a run that are worth a workgroup: one to a wave
};

__device__ __forceinline__ int few_tiles(const AttendArgs& a, const Request& r) {
  return r.n > 0 ? key_span<32>(r, 0, r.n - 1, a.window, a.sinks).count : -1;
}

// Runs of each request, by a wave: a lane to each, 0 for requests without rows.
__device__ __forceinline__ int few_runs(const AttendArgs& a, const FewArgs& f, int tiles, int lane) {
  int all = tiles < 0 ? 0 : tiles;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) all += __shfl_xor(all, d, 64);
  // The shortest run for which there are workgroups, each lane trying one
  // between an even share and twice that.
  int even = (int)(((int64_t)all * a.kv_heads + f.units - 1) / f.units);
  if (even < f.least) even = f.least;
  const int size = even + (int)((int64_t)even * lane / 63);
  const float inv = 1.f / (float)size;
  int need = 0;
#pragma unroll 1
  for (int i = 0; i < a.requests; ++i) {
    const int t = __builtin_amdgcn_readlane(tiles, i);
    if (t >= 0) need += quotient_up(t, size, inv);
  }
  const uint64_t fits = __ballot((int64_t)need * a.kv_heads <= f.units);
  const int pick = fits ? __builtin_ctzll(fits) : 63;
  return tiles < 0 ? 0 : quotient_up(tiles, __builtin_amdgcn_readlane(size, pick), __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(inv), pick)));
}

template <int D, int G, int S, bool FINE>
__global__ __launch_bounds__((FewShape<D, G, S>::kThreads), (D * G <= 128 ? 4 : D * G <= 256 ? 2 : 1)) void attend_few_kernel(AttendArgs a, FewArgs f) {
  using T = KeyTile<D>;
  using C = FewShape<D, G, S>;
  constexpr int DT = D / 16, KC = D / 32;
  extern __shared__ __align__(1024) unsigned char s_tiles[];
  __shared__ float s_m[S][16 * G], s_l[S][16 * G], s_f[S][16];
  __shared__ int s_bad;
  const int tid = threadIdx.x, lane = tid & 63, w = wave_index(), n = lane & 15, q = lane >> 4;
  const int unit = blockIdx.x;
  // the last row tiles see the most keys and go first
  const int row_tiles = gridDim.y * gridDim.z, row_tile = row_tiles - 1 - (blockIdx.z * gridDim.y + blockIdx.y);

  int b, h, run, runs;
  Request req;
  if (f.units == 0) {
    b = unit / a.kv_heads;
    h = unit - b * a.kv_heads;
    run = 0;
    runs = 1;
    req = request_of(a.q_start, a.kv_len, b, a.tokens, a.max_new, a.max_kv);
  } else if (a.requests > 64) {
    const int x = unit / a.kv_heads;
    h = unit - x * a.kv_heads;
    b = x / f.most;
    run = x - b * f.most;
    req = request_of(a.q_start, a.kv_len, b, a.tokens, a.max_new, a.max_kv);
    runs = min(quotient_up(few_tiles(a, req), f.per, 1.f / (float)f.per), f.most);
    if (run >= runs) return;
  } else {
    Request mine{0, 0, 0, false};
    if (lane < a.requests) mine = request_of(a.q_start, a.kv_len, lane, a.tokens, a.max_new, a.max_kv);
    const int own = few_runs(a, f, lane < a.requests ? few_tiles(a, mine) : -1, lane);
    const int upto = scan_lanes(own, lane) * a.kv_heads;
    if (unit == 0 && row_tile == 0 && w == 0) {  // for the join
      if (lane == 0) a.plan[0] = 0;
      a.plan[lane + 1] = upto;
    }
    const uint64_t past = __ballot(upto > unit);
    if (!past) return;
    b = __builtin_ctzll(past);
    const int off = unit - (b ? __builtin_amdgcn_readlane(upto, b - 1) : 0);
    runs = __builtin_amdgcn_readlane(own, b);
    run = off / a.kv_heads;
    h = off - run * a.kv_heads;
    req = of_lane(mine, b);
  }
  req = Request{uniform(req.q0), uniform(req.n), uniform(req.kv), (bool)uniform(req.bad)};
  const int rows = req.n * a.group, w0 = row_tile * C::kRows;
  if (w0 >= rows) return;
  const KeySpan span = uniform(key_span<32>(req, w0 / a.group, (min(w0 + C::kRows, rows) - 1) / a.group, a.window, a.sinks));
  const int first = uniform((int)((int64_t)span.count * run / runs)), stop = uniform((int)((int64_t)span.count * (run + 1) / runs));

  int pos[G];
  v8s Q[G][KC];
#pragma unroll
  for (int g = 0; g < G; ++g) {
    const int row = min(w0 + 16 * g + n, rows - 1), tok = row / a.group;
    pos[g] = req.kv - req.n + tok;
    const bf16_t* qp = (const bf16_t*)a.q + (req.q0 + tok) * a.q_tok + (h * a.group + row - tok * a.group) * a.q_head + q * (D / 4);
#pragma unroll
    for (int c = 0; c < KC; ++c) Q[g][c] = load_frag_bf16(qp + 8 * c);
  }

  v4f o[G][DT];
  float m[G], l[G];
  uint32_t note[G];  // blocks of a row's output that are NaN
#pragma unroll
  for (int g = 0; g < G; ++g) {
    m[g] = -INFINITY;
    l[g] = 0.f;
    note[g] = 0;
#pragma unroll
    for (int x = 0; x < DT; ++x) o[g][x] = zero4();
  }
  bool bad = req.bad;

  const_i32* const table = (const_i32*)(a.table + b * a.table_stride);
  const uint64_t head = (uint64_t)h * (uint64_t)a.head, page_bytes = (uint64_t)a.page;
  const int page_mask = (1 << a.page_shift) - 1;
  lds_byte* const tile = (lds_byte*)s_tiles + w * C::kTile;
  // V: rows that meet in different banks when they are written
  const int v_row = (lane >> 2 & 3) * 4 + (lane >> 4), v_part = lane & 3;
  using Q4 = Quarter<D>;
  const uint32_t k_data = Q4::data_at(n, q), k_power = Q4::power_at(n, q) & ~3u, k_shift = 8 * (Q4::power_at(n, q) & 3);
  const uint32_t v_data = Q4::data_at(v_row, v_part), v_power = Q4::power_at(v_row, v_part) & ~3u;
  const uint32_t v_shift = 8 * (Q4::power_at(v_row, v_part) & 3);

  Q4 K[2], V[2];
  int page[2] = {0, 0}, key = 0;
  auto look_up = [&](int i) {
    key = tile_of(span, i) * 32;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int k = key + 16 * t;
      const bool any = k < span.hi && (k + 15 >= span.lo || k < a.sinks);
      page[t] = table[(any ? k : key + 16 * (1 - t)) >> a.page_shift];
    }
  };
  auto load = [&]() {
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      int p = page[t];
      if ((uint32_t)p >= (uint32_t)a.num_pages) {
        bad = true;
        p = 0;
      }
      const uint32_t row = (uint32_t)(key + 16 * t) & page_mask;
      const uint64_t at = (uint32_t)p * page_bytes + head, data = at + row * (D / 2);
      const uint64_t power = at + ((uint64_t)(D / 2) << a.page_shift) + row * (D / 32);
      K[t].load((const char*)a.k + data + k_data, (const char*)a.k + power + k_power);
      V[t].load((const char*)a.v + data + v_data, (const char*)a.v + power + v_power);
    }
  };
  int i = first + w;
  if (i < stop) {
    look_up(i);
    load();
  }
#pragma unroll 1
  for (; i < stop; i += S) {
    const int at = key;  // of this tile
    if (i + S < stop) look_up(i + S);
    const bool whole = all_visible(span, at, 32, a.window, a.sinks);
    // scores, and V on its way through LDS
    v4f s[G][2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
#pragma unroll
      for (int g = 0; g < G; ++g) s[g][t] = zero4();
#pragma unroll
      for (int c = 0; c < KC; ++c) {
        const v8s k = from_fp4(K[t].x[c], K[t].power(c, k_shift));
#pragma unroll
        for (int g = 0; g < G; ++g) s[g][t] = mfma_16x16(k, Q[g][c], s[g][t]);
      }
    }
    if (!whole) {
      // Blocks of V that are not finite (or nearly: their elements may not be): a
      // product would spoil rows that do not see them.  They become zeros, and
      // the rows that do see them get NaN at the end.
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int e = 0; e < Q4::kPowers; ++e) {
          const bool odd = V[t].byte(e, v_shift) >= 253;
          uint64_t hit = __ballot(odd);
          while (hit) {
            const int from = __builtin_ctzll(hit);
            hit &= hit - 1;
            const int k = at + 16 * t + (from >> 2 & 3) * 4 + (from >> 4);
#pragma unroll
            for (int g = 0; g < G; ++g)
              if (visible(k, pos[g], a.window, a.sinks)) note[g] |= 1u << (Q4::block_of(from & 3) + e);
          }
          if (odd) {
            V[t].powers &= ~(255u << (v_shift + 8 * e));
#pragma unroll
            for (int x = 0; x < Q4::kWords; ++x)
              if (Q4::kPowers == 1 || x / 4 == e) V[t].x[x] = 0;
          }
        }
    }
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int x = 0; x < D / 32; ++x)
        *(__attribute__((address_space(3))) v8s*)(tile + (16 * t + v_row) * T::kRow + (((v_part * (D / 32) + x) ^ T::swizzle(v_row)) << 4)) =
            from_fp4(V[t].x[x], V[t].power(x, v_shift));
    if (i + S < stop) load();
    if (!whole) {
#pragma unroll
      for (int g = 0; g < G; ++g)
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (!visible(at + 16 * t + 4 * q + j, pos[g], a.window, a.sinks)) s[g][t][j] = -INFINITY;
    }
    // weights, FINE as the sum of two bf16 numbers
    v8s p[G], rest[G];
#pragma unroll
    for (int g = 0; g < G; ++g) {
      float top = fmaxf(fmaxf(fmaxf(s[g][0][0], s[g][0][1]), fmaxf(s[g][0][2], s[g][0][3])),
                        fmaxf(fmaxf(s[g][1][0], s[g][1][1]), fmaxf(s[g][1][2], s[g][1][3])));
      top = max_quarters(top);
      if (__any(top * a.scale_log2 > m[g] * a.scale_log2 + kSlack)) {
        const float mn = fmaxf(m[g], top);
        const float alpha = mn == -INFINITY ? 1.f : __builtin_amdgcn_exp2f((m[g] - mn) * a.scale_log2);
        l[g] *= alpha;
#pragma unroll
        for (int x = 0; x < DT; ++x) o[g][x] *= alpha;
        m[g] = mn;
      }
      const float ref = m[g] == -INFINITY ? 0.f : m[g] * a.scale_log2;
      float e[8], sum = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        e[j] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[g][j >> 2][j & 3], a.scale_log2, -ref));
        sum += e[j];
      }
      l[g] += sum;
      u32x4 hi, lo;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (!FINE) {
          hi[j] = pack_bf16(e[2 * j], e[2 * j + 1]);
          continue;
        }
        const uint32_t x = __float_as_uint(e[2 * j]) & 0xFFFF0000u, y = __float_as_uint(e[2 * j + 1]) & 0xFFFF0000u;
        hi[j] = x >> 16 | y;
        lo[j] = pack_bf16(e[2 * j] - __uint_as_float(x), e[2 * j + 1] - __uint_as_float(y));
      }
      p[g] = __builtin_bit_cast(v8s, hi);
      if constexpr (FINE) rest[g] = __builtin_bit_cast(v8s, lo);
    }
    // O^T += V^T P^T: lane j of a quarter points at row j / 4 of four, elements
    // 4 (j % 4), and gets element j of the four rows
    const int j4 = lane & 15;
#pragma unroll
    for (int x = 0; x < DT; ++x) {
      v4s f[2];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const int row = 4 * q + (j4 >> 2), piece = 2 * x + ((j4 & 3) >> 1);
        f[t] = lds_read_tr(tile + (16 * t + row) * T::kRow + ((piece ^ T::swizzle(row)) << 4) + ((j4 & 1) << 3));
      }
      const v8s v = __builtin_shufflevector(f[0], f[1], 0, 1, 2, 3, 4, 5, 6, 7);
#pragma unroll
      for (int g = 0; g < G; ++g) {
        o[g][x] = mfma_16x16(v, p[g], o[g][x]);
        if constexpr (FINE) o[g][x] = mfma_16x16(v, rest[g], o[g][x]);
      }
    }
  }

  // join the streams, 16 rows at a time, over the tiles
  if (tid == 0) s_bad = 0;
#pragma unroll
  for (int g = 0; g < G; ++g) {
    const float sum = sum_quarters(l[g]);
    if (q == 0) {
      s_m[w][16 * g + n] = m[g];
      s_l[w][16 * g + n] = sum;
    }
  }
  const bool alone = runs == 1;
  const int64_t part = ((int64_t)unit * row_tiles + row_tile) * C::kRows;  // rows
  float* const sums = (float*)s_tiles;
#pragma unroll
  for (int g = 0; g < G; ++g) {
    __syncthreads();
    if (g == 0 && bad) s_bad = 1;
#pragma unroll
    for (int x = 0; x < DT; ++x) {
      float4 y = make_float4(o[g][x][0], o[g][x][1], o[g][x][2], o[g][x][3]);
      if (note[g] >> (x / 2) & 1) y = make_float4(NAN, NAN, NAN, NAN);
      *(float4*)(sums + (w * 16 + n) * D + (((4 * x + q) ^ (n & (D / 4 - 1))) << 2)) = y;
    }
    // a row's factors for its streams, the division by the sum in them where the row is complete
    float top = -INFINITY, den = 0.f;
    const int row_ = w0 + 16 * g + (tid & 15);
    const bool joins = tid < 16;
    if (joins) {
#pragma unroll
      for (int x = 0; x < S; ++x) top = fmaxf(top, s_m[x][16 * g + tid]);
      const float ref = top == -INFINITY ? 0.f : top;
#pragma unroll
      for (int x = 0; x < S; ++x) den += __builtin_amdgcn_exp2f((s_m[x][16 * g + tid] - ref) * a.scale_log2) * s_l[x][16 * g + tid];
      const float inv = !alone ? 1.f : den == 0.f ? 0.f : 1.f / den;
#pragma unroll
      for (int x = 0; x < S; ++x) s_f[x][tid] = __builtin_amdgcn_exp2f((s_m[x][16 * g + tid] - ref) * a.scale_log2) * inv;
    }
    __syncthreads();
    const bool spoilt = s_bad != 0;
    if (joins && row_ < rows) {
      if (spoilt) den = NAN;
      if (alone) {
        const int tok = row_ / a.group, hq = h * a.group + row_ - tok * a.group;
        if (a.lse)
          a.lse[(int64_t)(req.q0 + tok) * a.q_heads + hq] = den == 0.f ? -INFINITY : top * a.scale + logf(den);
      } else {
        *(float2*)(a.part_ml + (part + 16 * g + tid) * 2) = make_float2(top, den);
      }
    }
#pragma unroll 1
    for (int i = tid; i < 16 * (D / 4); i += C::kThreads) {
      const int piece = i % (D / 4), r = i / (D / 4), row = w0 + 16 * g + r;
      if (row >= rows) continue;
      float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int x = 0; x < S; ++x) {
        const float f = s_f[x][r];
        const float4 z = *(const float4*)(sums + (x * 16 + r) * D + ((piece ^ (r & (D / 4 - 1))) << 2));
        y.x += f * z.x;
        y.y += f * z.y;
        y.z += f * z.z;
        y.w += f * z.w;
      }
      if (alone) {
        if (spoilt) y = make_float4(NAN, NAN, NAN, NAN);
        const int tok = row / a.group, hq = h * a.group + row - tok * a.group;
        *(u32x2*)((bf16_t*)a.out + (req.q0 + tok) * a.o_tok + hq * a.o_head + 4 * piece) =
            u32x2{pack_bf16(y.x, y.y), pack_bf16(y.z, y.w)};
      } else {
        *(float4*)(a.part_o + (part + 16 * g + r) * D + 4 * piece) = y;
      }
    }
  }
}

// Joins the runs of a request and key head, 1024 / D rows to a workgroup.
template <int D, int ROWS>
__global__ __launch_bounds__(256) void join_few_kernel(AttendArgs a, FewArgs f, int row_tiles) {
  constexpr int PER = 1024 / D;
  const int b = blockIdx.z, h = blockIdx.y;
  const Request req = request_of(a.q_start, a.kv_len, b, a.tokens, a.max_new, a.max_kv);
  const int rows = req.n * a.group, row = blockIdx.x * PER + threadIdx.x / (D / 4), piece = threadIdx.x % (D / 4);
  if (row >= rows) return;
  int runs;
  int64_t first;
  if (a.requests > 64) {
    runs = min(quotient_up(few_tiles(a, req), f.per, 1.f / (float)f.per), f.most);
    first = (int64_t)b * f.most * a.kv_heads + h;
  } else {
    first = a.plan[b] + h;
    runs = (a.plan[b + 1] - a.plan[b]) / a.kv_heads;
  }
  if (runs == 1) return;
  float top = -INFINITY, den = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int g = 0; g < runs; ++g) {
    const int64_t at = (first + (int64_t)g * a.kv_heads) * row_tiles * ROWS + row;
    const float2 ml = *(const float2*)(a.part_ml + at * 2);
    const float4 y = *(const float4*)(a.part_o + at * D + 4 * piece);
    const float mn = fmaxf(top, ml.x), ref = mn == -INFINITY ? 0.f : mn;
    const float fo = __builtin_amdgcn_exp2f((top - ref) * a.scale_log2);
    const float fn = __builtin_amdgcn_exp2f((ml.x - ref) * a.scale_log2);
    den = den * fo + ml.y * fn;
    o.x = o.x * fo + y.x * fn;
    o.y = o.y * fo + y.y * fn;
    o.z = o.z * fo + y.z * fn;
    o.w = o.w * fo + y.w * fn;
    top = mn;
  }
  const float inv = den == 0.f ? 0.f : 1.f / den;
  const int tok = row / a.group, hq = h * a.group + row - tok * a.group;
  *(u32x2*)((bf16_t*)a.out + (req.q0 + tok) * a.o_tok + hq * a.o_head + 4 * piece) =
      u32x2{pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv)};
  if (piece == 0 && a.lse)
    a.lse[(int64_t)(req.q0 + tok) * a.q_heads + hq] = den == 0.f ? -INFINITY : top * a.scale + logf(den);
}

template <int D, int G, int S, bool FINE>
hipError_t allow_few() {
  return hipFuncSetAttribute((const void*)attend_few_kernel<D, G, S, FINE>, hipFuncAttributeMaxDynamicSharedMemorySize,
                             FewShape<D, G, S>::kLds);
}

constexpr int kMostY = 1 << 15;  // below the limit of a grid's second dimension

// rows of the workspace that parts may take: as attend_split_floats
constexpr int few_rows(int head_dim, int cus) { return 2 * cus * (head_dim == 256 ? 128 : 256); }

// the most keys that the rows of a request see
inline int64_t few_keys(const AttendArgs& a) {
  const int64_t seen = (int64_t)a.window + a.max_new + a.sinks + 65;
  return a.window && seen < a.max_kv ? seen : a.max_kv;
}

// Cutting takes a second launch and the parts, on the host (one token over 1800 keys 13.1 us a
// call whole and 14.2 in runs) and on the GPU, so requests have more tiles than kWorth and
// lose more than kLess of them: a request can have units / segments runs, which leave it
// about the share segments / units.  With 8 key heads, whole and cut, us on the GPU:
//   heads of 128  one token of 1 request over 1024 keys 11 and 13, 2048 15 and 13; of 12 (3/8
//                 left) over 2048 16 and 17, 4096 24 and 22; 8 tokens of 20 requests over 2048
//                 28 and 26, of 32 (half left) over 2048 28 and 31, 2560 34 and 34, 4096 49 and 46
//   64            one token of 1 over 1536 10 and 11, 2048 12 and 12, of 16 (half left) over
//                 2560 14 and 15, 4096 18 and 19, 6144 24 and 22
//   256           one token of 4 over 1024 19 and 15; 8 tokens of 16 (half left) over 1024 20
//                 and 20, 1536 26 and 23
template <int D>
constexpr int kWorth = D == 256 ? 32 : 64;
template <int D>
constexpr int kLess = D == 256 ? 22 : D == 128 ? 44 : 60;

// `units`: workgroups that the chip holds at once, divided among the row tiles
template <int D, int G, int S, bool FINE>
void launch_few(const AttendArgs& a, int units, int cus, hipStream_t st) {
  using C = FewShape<D, G, S>;
  constexpr int PER = 1024 / D;
  const int64_t rows = (int64_t)a.max_new * a.group;
  const int row_tiles = (int)((rows + C::kRows - 1) / C::kRows);
  const int64_t segments = (int64_t)a.requests * a.kv_heads;
  const int64_t tiles = (few_keys(a) + 31) / 32 + 2;
  FewArgs f{};
  f.least = S;
  units /= row_tiles;
  const int64_t room = few_rows(D, cus) / (C::kRows * row_tiles);
  if (units > room) units = (int)room;
  if (2 * segments <= units && tiles > kWorth<D> && tiles * (units - segments) > (int64_t)kLess<D> * units &&
      a.requests * tiles < (int64_t)1 << 30) {
    f.units = units;
    if (a.requests > 64) {
      f.most = (int)(units / segments);
      f.per = (int)((tiles + f.most - 1) / f.most);
      f.units = (int)(segments * f.most);
    } else if (f.units > segments * ((tiles + f.least - 1) / f.least)) {
      f.units = (int)(segments * ((tiles + f.least - 1) / f.least));
    }
  }
  // row tiles of a unit meet in one XCD's cache
  const int64_t grid = f.units ? f.units : segments;
  const int y = row_tiles < kMostY ? row_tiles : kMostY, z = (row_tiles + y - 1) / y;
  hipLaunchKernelGGL((attend_few_kernel<D, G, S, FINE>), dim3((unsigned)grid, y, z), dim3(C::kThreads), C::kLds, st, a, f);
  if (!f.units || hipPeekAtLastError() != hipSuccess) return;  // the join would follow the parts of an earlier call
  hipLaunchKernelGGL((join_few_kernel<D, C::kRows>), dim3((unsigned)((rows + PER - 1) / PER), a.kv_heads, a.requests),
                     dim3(256), 0, st, a, f, row_tiles);
}

}  // namespace
