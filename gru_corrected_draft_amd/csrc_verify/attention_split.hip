// bf16 attention of few rows over long caches: the work of all requests is one
// list of steps, dealt evenly to the workgroups, and split segments are joined
// by a second launch.
//
// Steps.  A segment is one (request, row tile, key head); it has one step for
// each W key tiles (one for each of the workgroup's W waves), and at least
// one, so that rows without keys are written too.  The steps of all segments
// in order are cut into equal shares, one for each workgroup, whatever the
// lengths of the requests: each workgroup sums up the lengths itself.  A share
// ends at most two segments inside; those leave their unnormalised output,
// maximum and sum in the workspace.
//
// Bound by the cache's bytes.  Each wave copies its own tiles into its own
// ring in LDS and never waits for another: no barrier in the walk.
#include "attention_bf16.h"

namespace {

template <int D>
struct Split {
  static constexpr int kWaves = D == 256 ? 2 : 4;
  static constexpr int kRing = D == 64 ? 4 : 2;
  static constexpr int kRingBytes = kRing * KeyTile<D>::kBytes;  // of a wave
  static constexpr int kLds = kWaves * kRingBytes;               // 128 KB for every D
  static constexpr int kThreads = kWaves * 64;
};

__device__ __forceinline__ int steps_of(int count, int waves) {
  return count > 0 ? (count + waves - 1) / waves : 1;
}

template <int ROWS>
__device__ __forceinline__ KeySpan row_tile_span(const AttendArgs& a, const Request& r, int rt) {
  const int rows = r.n * a.group, r0 = rt * ROWS;
  const int last = (r0 + ROWS < rows ? r0 + ROWS : rows) - 1;
  return key_span<32>(r, r0 / a.group, last / a.group, a.window, a.sinks);
}

// steps of request b
template <int ROWS, int W>
__device__ __forceinline__ int request_steps(const AttendArgs& a, int b) {
  const Request r = request_of(a.q_start, a.kv_len, b, a.tokens, a.max_new, a.max_kv);
  int n = 0;
  for (int rt = 0; rt * ROWS < r.n * a.group; ++rt) n += steps_of(row_tile_span<ROWS>(a, r, rt).count, W);
  return n * a.kv_heads;
}

template <int D, int NT>
__global__ __launch_bounds__(Split<D>::kThreads, D * NT < 128 ? 2 : 1) void attend_split_kernel(AttendArgs a) {
  using T = KeyTile<D>;
  constexpr int W = Split<D>::kWaves, ROWS = 32 * NT, RING = Split<D>::kRing, THREADS = Split<D>::kThreads;
  extern __shared__ __align__(1024) unsigned char ring[];
  __shared__ int s_pre[1025];
  __shared__ int s_sum[4];
  __shared__ float s_m[W][ROWS], s_l[W][ROWS];
  const int tid = threadIdx.x, lane = tid & 63, w = wave_index(), n = lane & 31, h2 = lane >> 5;

  // running sum of the requests' steps
  int carry = 0;
  for (int b0 = 0; b0 < a.requests; b0 += THREADS) {
    const int b = b0 + tid;
    int x = b < a.requests ? request_steps<ROWS, W>(a, b) : 0;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int y = __shfl_up(x, d, 64);
      if (lane >= d) x += y;
    }
    if (lane == 63) s_sum[w] = x;
    __syncthreads();
    for (int i = 0; i < w; ++i) x += s_sum[i];
    if (b < a.requests) s_pre[b + 1] = carry + x;
    for (int i = 0; i < W; ++i) carry += s_sum[i];
    __syncthreads();
  }
  if (tid == 0) s_pre[0] = 0;
  __syncthreads();
  const int total = __builtin_amdgcn_readfirstlane(carry);
  if (blockIdx.x == 0)
    for (int b = tid; b <= a.requests; b += THREADS) a.plan[b] = s_pre[b];
  const int share = max(a.min_share, (total + (int)gridDim.x - 1) / (int)gridDim.x);
  int at = blockIdx.x * share;
  const int end = min(at + share, total);
  if (at >= end) return;

  // request of the first step: the last one that begins at or before it
  int b = 0;
  {
    int hi = a.requests;  // s_pre[b] <= at < s_pre[hi]
    while (hi - b > 1) {
      const int mid = (b + hi) >> 1;
      if (s_pre[mid] <= at)
        b = mid;
      else
        hi = mid;
    }
  }
  b = __builtin_amdgcn_readfirstlane(b);

  lds_byte* const lds = (lds_byte*)ring;
  lds_byte* const mine = lds + w * Split<D>::kRingBytes;
  const uint32_t k0_off = T::k_first(lane);
  const uint32_t v0_off[2] = {T::v_first(lane, 0), T::v_first(lane, 1)};
  uint32_t src[T::kChunkLoads];
#pragma unroll
  for (int j = 0; j < T::kChunkLoads; ++j) src[j] = T::source(j, lane, 2 * a.row);

  while (at < end) {
    while (s_pre[b + 1] <= at) ++b;  // requests without rows have no steps
    const Request req = request_of(a.q_start, a.kv_len, b, a.tokens, a.max_new, a.max_kv);
    int off = at - __builtin_amdgcn_readfirstlane(s_pre[b]), rt = 0;
    KeySpan span = row_tile_span<ROWS>(a, req, 0);
    int seg = steps_of(span.count, W);
    while (off >= seg * a.kv_heads) {
      off -= seg * a.kv_heads;
      span = row_tile_span<ROWS>(a, req, ++rt);
      seg = steps_of(span.count, W);
    }
    const int h = off / seg, first = off - h * seg, stop = min(seg, first + end - at);

    const int rows = req.n * a.group, r0 = rt * ROWS, last = min(r0 + ROWS, rows) - 1;
    v8s Q[NT][D / 16];
    int pos[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int row = min(r0 + 32 * t + n, last), tok = row / a.group;
      pos[t] = req.kv - req.n + tok;
      const bf16_t* qp = (const bf16_t*)a.q + (req.q0 + tok) * a.q_tok +
                         (h * a.group + row - tok * a.group) * a.q_head + 8 * h2;
#pragma unroll
      for (int kc = 0; kc < D / 16; ++kc) Q[t][kc] = load_frag_bf16(qp + 16 * kc);
    }
    RowState<D> st[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) st[t].clear();
    bool bad = req.bad;

    const_i32* const table = (const_i32*)(a.table + b * a.table_stride);
    const int64_t head = h * a.head;
    const int page_mask = (1 << a.page_shift) - 1;
    const int tiles = min(stop * W, span.count);
    int next = first * W + w, ahead = 0, slot_in = 0, slot_out = 0;

    // copies the wave's next tile into its ring
    auto fetch = [&]() {
      const int key = tile_of(span, next) * 32;
      next += W;
      ++ahead;
      const lds_byte* dst = mine + slot_in * T::kBytes;
      slot_in = slot_in + 1 == RING ? 0 : slot_in + 1;
      int64_t base[2];
      int page[2];
      // a chunk of 16 keys lies in one page; one that no row sees may have
      // none, and takes its neighbour's
      const bool see0 = key < span.hi && (key + 15 >= span.lo || key < a.sinks);
      const bool see1 = key + 16 < span.hi && (key + 31 >= span.lo || key + 16 < a.sinks);
      page[0] = table[(see0 ? key : key + 16) >> a.page_shift];
      page[1] = table[(see1 ? key + 16 : key) >> a.page_shift];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        if (page[c] < 0 || page[c] >= a.num_pages) {
          bad = true;
          page[c] = 0;
        }
        base[c] = 2 * (page[c] * a.page + head + (int64_t)((key + 16 * c) & page_mask) * a.row);
      }
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const char* from = (const char*)(x ? a.v : a.k) + base[c];
#pragma unroll
          for (int j = 0; j < T::kChunkLoads; ++j)
            __builtin_amdgcn_global_load_lds(
                (const __attribute__((address_space(1))) void*)(from + src[j]),
                (__attribute__((address_space(3))) void*)(dst + x * T::kHalf + (c * T::kChunkLoads + j) * 1024), 16,
                0, 0);
        }
    };
    for (int i = first * W + w - (RING - 1) * W; i < tiles; i += W) {
      if (next < tiles) fetch();
      if (i < first * W) continue;  // fills the ring
      --ahead;
      if (ahead >= RING - 1)
        wait_copies<(RING - 1) * T::kLoads>();
      else if (RING > 2 && ahead == 2)
        wait_copies<2 * T::kLoads>();
      else if (RING > 2 && ahead == 1)
        wait_copies<T::kLoads>();
      else
        wait_copies<0>();
      const lds_byte* tile = mine + slot_out * T::kBytes;
      slot_out = slot_out + 1 == RING ? 0 : slot_out + 1;
      const int key = tile_of(span, i) * 32;
      v16f s[NT];
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int j = 0; j < 16; ++j) s[t][j] = 0.f;
#pragma unroll
      for (int kc = 0; kc < D / 16; ++kc) {
        const v8s k = lds_read16(tile + T::k_step(k0_off, kc));
#pragma unroll
        for (int t = 0; t < NT; ++t) s[t] = mfma_32x32(k, Q[t][kc], s[t]);
      }
      const bool edge = !all_visible(span, key, 32, a.window, a.sinks);
      v8s p[NT][2];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        if (edge) {
#pragma unroll
          for (int j = 0; j < 16; ++j)
            if (!visible(key + 16 * (j >> 3) + 8 * h2 + (j & 7), pos[t], a.window, a.sinks)) s[t][j] = -INFINITY;
        }
        softmax_step<D>(s[t], st[t], p[t], a.scale_log2);
      }
      if (edge && odd_values<D>(tile, lane)) {
#pragma unroll
        for (int t = 0; t < NT; ++t) careful_values<D>(tile, st[t], s[t], key, pos[t], a.window, a.sinks, lane);
      } else {
        weighted_values<D, NT>(tile, v0_off, st, p);
      }
    }

    // join the waves: each writes its rows to LDS over the rings
    __syncthreads();
    float* const so = (float*)ring;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const float l = sum_halves(st[t].l);
      const int row = 32 * t + n;
      if (h2 == 0) {
        s_m[w][row] = st[t].m;
        s_l[w][row] = bad ? NAN : l;
      }
#pragma unroll
      for (int blk = 0; blk < D / 32; ++blk)
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int piece = (8 * blk + 2 * x + h2) ^ (row & (D / 4 - 1));
          *(float4*)(so + ((w * ROWS + row) * D + piece * 4)) =
              make_float4(st[t].o[blk][4 * x], st[t].o[blk][4 * x + 1], st[t].o[blk][4 * x + 2], st[t].o[blk][4 * x + 3]);
        }
    }
    __syncthreads();
    const bool whole = first == 0 && stop == seg;
    const int64_t part = 2 * (int64_t)blockIdx.x + (first == 0);
    for (int i = tid; i < (last - r0 + 1) * (D / 4); i += THREADS) {
      const int row = i / (D / 4), piece = i - row * (D / 4);
      float top = -INFINITY;
#pragma unroll
      for (int x = 0; x < W; ++x) top = fmaxf(top, s_m[x][row]);
      const float ref = top == -INFINITY ? 0.f : top;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
      float den = 0.f;
#pragma unroll
      for (int x = 0; x < W; ++x) {
        const float f = __builtin_amdgcn_exp2f((s_m[x][row] - ref) * a.scale_log2);
        den += f * s_l[x][row];
        const float4 y = *(const float4*)(so + ((x * ROWS + row) * D + (piece ^ (row & (D / 4 - 1))) * 4));
        o.x += f * y.x;
        o.y += f * y.y;
        o.z += f * y.z;
        o.w += f * y.w;
      }
      if (whole) {
        const float inv = den == 0.f ? 0.f : 1.f / den;
        const int tok = (r0 + row) / a.group, hq = h * a.group + r0 + row - tok * a.group;
        *(u32x2*)((bf16_t*)a.out + (req.q0 + tok) * a.o_tok + hq * a.o_head + 4 * piece) =
            u32x2{pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv)};
        if (piece == 0 && a.lse)
          a.lse[(int64_t)(req.q0 + tok) * a.q_heads + hq] = den == 0.f ? -INFINITY : top * a.scale + logf(den);
      } else {
        *(float4*)(a.part_o + (part * ROWS + row) * D + 4 * piece) = o;
        if (piece == 0) {
          a.part_ml[(part * ROWS + row) * 2] = top;
          a.part_ml[(part * ROWS + row) * 2 + 1] = den;
        }
      }
    }
    __syncthreads();
    at += stop - first;
  }
}

// Joins the parts of split segments: 256 threads take 1024 / D rows of one
// (request, row tile, key head).
template <int D, int NT>
__global__ __launch_bounds__(256) void attend_join_kernel(AttendArgs a, int workers, int row_groups) {
  constexpr int W = Split<D>::kWaves, ROWS = 32 * NT, PER = 1024 / D;
  const int b = blockIdx.z, rt = blockIdx.x, h = blockIdx.y / row_groups, group = blockIdx.y - h * row_groups;
  const Request req = request_of(a.q_start, a.kv_len, b, a.tokens, a.max_new, a.max_kv);
  const int rows = req.n * a.group, r0 = rt * ROWS;
  const int row = group * PER + threadIdx.x / (D / 4), piece = threadIdx.x % (D / 4);
  if (r0 + row >= rows || row >= ROWS) return;
  const int total = a.plan[a.requests];
  const int share = max(a.min_share, (total + workers - 1) / workers);
  int from = a.plan[b];
  for (int x = 0; x < rt; ++x) from += steps_of(row_tile_span<ROWS>(a, req, x).count, W) * a.kv_heads;
  const int seg = steps_of(row_tile_span<ROWS>(a, req, rt).count, W);
  from += h * seg;
  const int g0 = from / share, g1 = (from + seg - 1) / share;
  if (g0 == g1) return;
  float top = -INFINITY, den = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int g = g0; g <= g1; ++g) {
    const int64_t part = 2 * (int64_t)g + (g == g0);
    const float2 ml = *(const float2*)(a.part_ml + (part * ROWS + row) * 2);
    const float4 y = *(const float4*)(a.part_o + (part * ROWS + row) * D + 4 * piece);
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
  const int tok = (r0 + row) / a.group, hq = h * a.group + r0 + row - tok * a.group;
  *(u32x2*)((bf16_t*)a.out + (req.q0 + tok) * a.o_tok + hq * a.o_head + 4 * piece) =
      u32x2{pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv)};
  if (piece == 0 && a.lse)
    a.lse[(int64_t)(req.q0 + tok) * a.q_heads + hq] = den == 0.f ? -INFINITY : top * a.scale + logf(den);
}

template <int D, int NT>
void launch(const AttendArgs& a, int cus, hipStream_t st) {
  constexpr int ROWS = 32 * NT, W = Split<D>::kWaves, PER = 1024 / D;
  const int64_t rows = (int64_t)a.max_new * a.group;
  const int64_t row_tiles = (rows + ROWS - 1) / ROWS;
  const int64_t seg_most = a.max_kv > 32 * W ? (a.max_kv + 32 * W - 1) / (32 * W) + 1 : 1;
  const int64_t most = (int64_t)a.requests * row_tiles * a.kv_heads * seg_most;
  const int64_t need = (most + a.min_share - 1) / a.min_share;
  const int workers = (int)(need < cus ? need : cus);
  static const hipError_t big = hipFuncSetAttribute((const void*)&attend_split_kernel<D, NT>,
                                                    hipFuncAttributeMaxDynamicSharedMemorySize, Split<D>::kLds);
  (void)big;
  hipLaunchKernelGGL((attend_split_kernel<D, NT>), dim3(workers), dim3(Split<D>::kThreads), Split<D>::kLds, st, a);
  if (workers == 1) return;  // nothing is split
  const int groups = (int)(((rows < ROWS ? rows : ROWS) + PER - 1) / PER);
  hipLaunchKernelGGL((attend_join_kernel<D, NT>), dim3((unsigned)row_tiles, a.kv_heads * groups, a.requests), dim3(256),
                     0, st, a, workers, groups);
}

template <int D>
void launch_d(const AttendArgs& a, int cus, hipStream_t st) {
  // two row tiles to a wave halve the reads of the keys; at D = 256 their
  // sums do not fit the registers
  if (D == 256 || (int64_t)a.max_new * a.group <= 32)
    launch<D, 1>(a, cus, st);
  else
    launch<D == 256 ? 128 : D, 2>(a, cus, st);
}

}  // namespace

// workspace: two parts of 64 rows, their outputs and (m, l), for each workgroup
size_t attend_split_floats(int head_dim, int cus) { return (size_t)2 * cus * 64 * (head_dim + 2); }

void launch_attend_split(int head_dim, const AttendArgs& a, int cus, hipStream_t st) {
  if (head_dim == 64)
    launch_d<64>(a, cus, st);
  else if (head_dim == 128)
    launch_d<128>(a, cus, st);
  else
    launch_d<256>(a, cus, st);
}
