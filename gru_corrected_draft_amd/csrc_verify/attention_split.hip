// bf16 attention kernels.
//
// A workgroup takes R * 32 rows of one request and key head (a row tile) and S
// streams of key tiles: wave w works for row group w / S on stream w % S, with
// its own running maximum and sum (softmax in one pass: sums against a maximum
// m are rescaled by e^(m - m') when it becomes m').  The streams of a row group
// are joined in LDS at the end.  One group of 32 rows to a wave keeps a wave's
// sums, queries and scores in 256 registers; with more rows the sums move to
// accumulation registers, and the moves cost more than the halved reads of LDS
// save.
//   R = 1: a wave copies its own tiles into its own ring and never waits for
//          another; no barrier in the walk.  For few rows, bound by the
//          cache's bytes: 64 requests with one token each over 4 to 8 thousand
//          keys take 285 us, 5.7 TB/s (a large copy reaches 5.2).
//   R > 1: the R waves on a stream share its tiles, each copies a part, and a
//          barrier separates the steps.  R = 2 and 4 for up to 64 and 128 rows,
//          so that a draft block of 16 positions with 4 or 8 heads to a key
//          head reads its keys once: 8 requests over 2 to 4 thousand keys take
//          36 us, 2.9 TB/s, of which 2.4 find the work, 4 fill the rings and 4.5
//          join; 16 requests with a window of 4096 70 us, 3.9 TB/s.
//   R = 8: for prompts; steps of 64 keys (234 us against 262 with 32 for 2
//          requests of up to 2048 tokens over up to 5120 keys), 970 TFLOP/s
//          (a large product 1390 to 1490).  Bound by issue: vector and matrix
//          instructions are busy 41 and 40 % of the time and those of
//          two waves of a SIMD overlap only in part (beside a wave of products
//          alone, one of softmax alone takes 1.4 times as long).  Products of
//          the next tile put between a tile's softmax (278 us against 262),
//          waves half a step apart (269 against 242) and two workgroups of 4
//          waves to a CU (243 against 234) were slower.
//
// Steps.  A segment is one (request, row tile, key head); it has one step for
// each S (R = 8: 2) key tiles, and at least one, so that rows without keys are
// written too.  With WHOLE a workgroup takes one segment.  Otherwise the steps of
// all segments in order are cut into equal shares, one for each workgroup,
// whatever the lengths of the requests: each workgroup sums up the lengths
// itself.  A share ends at most two segments inside; those leave their
// unnormalised output, maximum and sum in the workspace, and a second launch
// joins them (the last workgroup of a segment in its place, without a launch but
// alone with the loads: block of 8 requests 40 us against 35).  With no more
// segments than half the workgroups, of no more row tiles than a wave has lanes,
// each segment is cut into pieces of its own instead, one to a workgroup: a share
// that straddles two segments would pay for two starts and two ends (block of 8
// requests 42 us against 36, one prompt of 512 tokens over 4096 keys 73 against
// 64).
#include "attention_bf16.h"

namespace {

constexpr int kMinShare = 2;  // steps: fewer to a workgroup would be all start and end

template <int D, int R>
struct Shape {
  // R = 2: 4 streams with rings of 2 take as long as 2 with rings of 4 (36.1 and
  // 35.6 us, block of 8 requests)
  static constexpr int S = D == 256 ? (R == 1 ? 2 : 1) : (R == 1 ? 4 : R == 2 ? 2 : 8 / R);  // streams
  static constexpr int W = R * S;                                                // waves
  static constexpr int kThreads = 64 * W;
  static constexpr int kRows = 32 * R;
  // tiles of a stream in LDS: 128 KB in all at D = 128 and 256 up to R = 4
  static constexpr int kRing = D == 64 ? 4 : (R == 1 ? 2 : 4);
  static constexpr int kLds = S * kRing * KeyTile<D>::kBytes;
  static constexpr int kJoin = kLds / (W * D * 4) < 32 ? kLds / (W * D * 4) : 32;  // rows joined at a time
  static constexpr int N = R == 8 ? 2 : 1;  // tiles of a stream in a step
  static constexpr int kStep = S * N;
  static constexpr int kAhead = kRing / N - 1;              // steps on their way
  static constexpr int kLoads = N * KeyTile<D>::kLoads / R;  // copies of a step by one wave
};

__device__ __forceinline__ int steps_of(int count, int streams) {
  return count > 0 ? (count + streams - 1) / streams : 1;
}

template <int ROWS>
__device__ __forceinline__ KeySpan row_tile_span(const AttendArgs& a, const Request& r, int rt) {
  const int rows = r.n * a.group, r0 = rt * ROWS;
  const int last = (r0 + ROWS < rows ? r0 + ROWS : rows) - 1;
  return key_span<32>(r, r0 / a.group, last / a.group, a.window, a.sinks);
}

// steps of row tile rt of a request, none past its rows
template <int ROWS, int STEP>
__device__ __forceinline__ int tile_steps(const AttendArgs& a, const Request& r, int rt) {
  return rt * ROWS < r.n * a.group ? steps_of(row_tile_span<ROWS>(a, r, rt).count, STEP) : 0;
}

// steps of a request, by each lane for a request of its own
template <int ROWS, int STEP>
__device__ __forceinline__ int request_steps(const AttendArgs& a, const Request& r) {
  int n = 0;
  for (int rt = 0; rt * ROWS < r.n * a.group; ++rt) n += tile_steps<ROWS, STEP>(a, r, rt);
  return n * a.kv_heads;
}

__device__ __forceinline__ int scan_lanes(int x, int lane) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int y = __shfl_up(x, d, 64);
    if (lane >= d) x += y;
  }
  return x;
}

// Row tile of step `off` of a request's, which becomes the step among the row
// tile's, by a wave for one request: a lane to each row tile.  A prompt of 2048 tokens has 32 row
// tiles, and gone through one by one they were a third of its time.
template <int ROWS, int STEP>
__device__ __forceinline__ int find_row_tile(const AttendArgs& a, const Request& r, int& off, int lane) {
  const int row_tiles = (r.n * a.group + ROWS - 1) / ROWS;
#pragma unroll 1
  for (int rt = 0; rt < row_tiles; rt += 64) {
    const int upto = scan_lanes(tile_steps<ROWS, STEP>(a, r, rt + lane), lane) * a.kv_heads;
    const uint64_t past = __ballot(upto > off);
    const int x = past ? __builtin_ctzll(past) : 64;
    if (x) off -= __builtin_amdgcn_readlane(upto, x - 1);
    if (past) return rt + x;
  }
  return row_tiles;
}

// steps of a request's first rt row tiles, in the same way
template <int ROWS, int STEP>
__device__ __forceinline__ int steps_before(const AttendArgs& a, const Request& r, int rt, int lane) {
  int n = 0;
#pragma unroll 1
  for (int x = 0; x < rt; x += 64)
    n += __builtin_amdgcn_readlane(scan_lanes(x + lane < rt ? tile_steps<ROWS, STEP>(a, r, x + lane) : 0, lane), 63);
  return n * a.kv_heads;
}

__device__ __forceinline__ Request of_lane(const Request& r, int lane) {
  return Request{__builtin_amdgcn_readlane(r.q0, lane), __builtin_amdgcn_readlane(r.n, lane),
                 __builtin_amdgcn_readlane(r.kv, lane), (bool)__builtin_amdgcn_readlane((int)r.bad, lane)};
}

template <int D, int R, bool WHOLE>
__global__ __launch_bounds__((Shape<D, R>::kThreads), (D < 256 ? 2 : 1)) void attend_split_kernel(AttendArgs a) {
  using T = KeyTile<D>;
  using C = Shape<D, R>;
  constexpr int S = C::S, N = C::N, STEP = C::kStep, ROWS = C::kRows, RING = C::kRing, THREADS = C::kThreads, JOIN = C::kJoin;
  extern __shared__ __align__(1024) unsigned char ring[];
  __shared__ int s_sum[C::W];
  __shared__ float s_m[C::W][32], s_l[C::W][32], s_f[C::W][32];
  __shared__ int s_bad;
  __shared__ uint16_t s_notes[C::W][32 * (D / 8)];
  __shared__ int s_noting[C::W];
  const int tid = threadIdx.x, lane = tid & 63, w = wave_index(), n = lane & 31, h2 = lane >> 5;
  const int rg = w / S, stream = w - rg * S;

  int b = 0, begin = 0, at = 0, end = 1, upto = 0, mine_pieces = 0;
  Request mine{0, 0, 0, false};
  const bool few = a.requests <= 64;
  if constexpr (!WHOLE) {
    // Running sum of the requests' steps.  Up to 64 requests a wave holds it in
    // its lanes, each wave for itself, without a barrier; beyond that it goes
    // through LDS, over the rings.
    int total;
    if (few) {
      // (a lane to each request, or with pieces to each row tile of one)
      const int own = a.pieces ? lane / a.row_tiles : lane;
      if (own < a.requests) mine = request_of(a.q_start, a.kv_len, own, a.tokens, a.max_new, a.max_kv);
      if (a.pieces) {
        upto = own < a.requests ? tile_steps<ROWS, STEP>(a, mine, lane - own * a.row_tiles) * a.kv_heads : 0;
      } else if (a.row_tiles <= 2) {
        upto = lane < a.requests ? request_steps<ROWS, STEP>(a, mine) : 0;
      } else {
#pragma unroll 1
        for (int x = 0; x < a.requests; ++x) {
          const int n = steps_before<ROWS, STEP>(a, of_lane(mine, x), a.row_tiles, lane);
          if (lane == x) upto = n;
        }
      }
      if (a.pieces) {
        // The shortest piece at which there are workgroups for all, each lane
        // trying one between an even share and twice that, where there are.
        int all = upto;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) all += __shfl_xor(all, d, 64);
        const int even = max(kMinShare, (all + (int)gridDim.x - 1) / (int)gridDim.x);
        const int steps = upto / a.kv_heads, size = even + lane + (int)((int64_t)even * lane / 63);
        int need = 0;
#pragma unroll 1
        for (int i = 0; i < a.requests * a.row_tiles; ++i) need += (__builtin_amdgcn_readlane(steps, i) + size - 1) / size;
        const uint64_t fits = __ballot(need * a.kv_heads <= (int)gridDim.x);
        const int piece = __builtin_amdgcn_readlane(size, fits ? __builtin_ctzll(fits) : 63);
        mine_pieces = (steps + piece - 1) / piece;
        upto = mine_pieces * a.kv_heads;
      }
      upto = scan_lanes(upto, lane);
      total = __builtin_amdgcn_readlane(upto, 63);
    } else {
      int* const s_pre = (int*)ring;
      int carry = 0;
      for (int b0 = 0; b0 < a.requests; b0 += THREADS) {
        const int b = b0 + tid;
        int x = b < a.requests
                    ? request_steps<ROWS, STEP>(a, request_of(a.q_start, a.kv_len, b, a.tokens, a.max_new, a.max_kv))
                    : 0;
        x = scan_lanes(x, lane);
        if (lane == 63) s_sum[w] = x;
        __syncthreads();
        for (int i = 0; i < w; ++i) x += s_sum[i];
        if (b < a.requests) s_pre[b + 1] = carry + x;
        for (int i = 0; i < C::W; ++i) carry += s_sum[i];
        __syncthreads();
      }
      if (tid == 0) s_pre[0] = 0;
      __syncthreads();
      total = carry;
    }
    total = uniform(total);
    const int share = a.pieces ? 1 : max(kMinShare, (total + (int)gridDim.x - 1) / (int)gridDim.x);
    at = blockIdx.x * share;
    end = min(at + share, total);
    if (at >= end) return;
    if (blockIdx.x == 0) {  // for the join
      if (few) {
        if (w == 0 && lane == 0) a.plan[0] = 0;
        if (w == 0) a.plan[lane + 1] = upto;
      } else {
        for (int i = tid; i <= a.requests; i += THREADS) a.plan[i] = ((const int*)ring)[i];
      }
    }

    // request of the first step (the last one that begins at or before it) and
    // the step its own begin at
    if (!few) {
      const int* const s_pre = (const int*)ring;
      int hi = a.requests;  // s_pre[b] <= at < s_pre[hi]
      while (hi - b > 1) {
        const int mid = (b + hi) >> 1;
        if (s_pre[mid] <= at)
          b = mid;
        else
          hi = mid;
      }
      begin = s_pre[b];
      __syncthreads();  // the rings are free again
    }
    // the branches above hide from the compiler that these are the same in
    // every lane
    begin = uniform(begin);
    b = uniform(b);
    at = uniform(at);
    end = uniform(end);
  }

  lds_byte* const own = (lds_byte*)ring + stream * (RING * T::kBytes);
  lds_u16* const notes = (lds_u16*)s_notes[w];
  const uint32_t k0_off = T::k_first(lane);
  const uint32_t v0_off[2] = {T::v_first(lane, 0), T::v_first(lane, 1)};
  uint32_t src[T::kChunkLoads];
#pragma unroll
  for (int j = 0; j < T::kChunkLoads; ++j) src[j] = T::source(j, lane, 2 * a.row);

  while (at < end) {
    Request req;
    int rt = 0, tile = 0, h, first, stop, seg;  // tile: of all requests' row tiles, with pieces
    KeySpan span;
    if constexpr (WHOLE) {
      // key heads vary fastest, so that the row tiles of a head, which read the
      // same keys, meet in one XCD's cache when there are 8 of them; the last
      // row tiles see the most keys and go first
      b = blockIdx.z;
      h = blockIdx.x;
      rt = gridDim.y - 1 - blockIdx.y;
      req = request_of(a.q_start, a.kv_len, b, a.tokens, a.max_new, a.max_kv);
      if (rt * ROWS >= req.n * a.group) return;
      span = row_tile_span<ROWS>(a, req, rt);
      first = 0;
      stop = seg = uniform(steps_of(span.count, STEP));
    } else {
      if (few) {
        b = __builtin_ctzll(__ballot(upto > at));
        begin = b ? __builtin_amdgcn_readlane(upto, b - 1) : 0;
        req = of_lane(mine, b);
        tile = b;
        if (a.pieces) {
          b = uniform(tile / a.row_tiles);
          rt = tile - b * a.row_tiles;
        }
      } else {
        for (;;) {  // requests without rows have no steps
          req = request_of(a.q_start, a.kv_len, b, a.tokens, a.max_new, a.max_kv);
          const int steps = request_steps<ROWS, STEP>(a, req);
          if (uniform(at < begin + steps)) break;
          begin = uniform(begin + steps);
          b = uniform(b + 1);
        }
      }
      int off = at - begin;
      if (!a.pieces && a.row_tiles > 1) rt = find_row_tile<ROWS, STEP>(a, req, off, lane);
      span = row_tile_span<ROWS>(a, req, rt);
      seg = steps_of(span.count, STEP);
      if (a.pieces) {
        const int pieces = __builtin_amdgcn_readlane(mine_pieces, tile);
        h = uniform(off / pieces);
        const int x = off - h * pieces;
        first = uniform((int)((int64_t)seg * x / pieces));
        stop = uniform((int)((int64_t)seg * (x + 1) / pieces));
      } else {
        h = off / seg;
        first = off - h * seg;
        stop = min(seg, first + end - at);
      }
      rt = uniform(rt);
      seg = uniform(seg);
      h = uniform(h);
      first = uniform(first);
      stop = uniform(stop);
    }
    span = uniform(span);
    req = Request{uniform(req.q0), uniform(req.n), uniform(req.kv), (bool)uniform(req.bad)};
    bool bad = req.bad;

    const_i32* const table = (const_i32*)(a.table + b * a.table_stride);
    const uint64_t head = 2 * (uint64_t)h * (uint64_t)a.head, page_bytes = 2 * (uint64_t)a.page;
    const uint32_t row_bytes = 2 * (uint32_t)a.row;
    const TileRange range = uniform(tile_range<32>(span, a.window, a.sinks));
    const int page_mask = (1 << a.page_shift) - 1;
    const int tiles = min(stop * STEP, span.count);
    int next = first * STEP + stream * N, ahead = 0, slot_in = 0, slot_out = 0;

    // The page of the 16 keys from `key` on; keys that no row sees may have
    // none and take that of `other`, the tile's other half.  Read for a tile
    // ahead of its copies.
    auto page_of = [&](int key, int other) -> int {
      const bool seen = key < span.hi && (key + 15 >= span.lo || key < a.sinks);
      return table[(seen ? key : other) >> a.page_shift];
    };
    // R >= 4: the half of a tile's keys, and of a step's tiles the one, that this
    // wave copies
    const int own_half = R >= 4 ? rg % 2 : 0, own_tile = R == 8 ? rg / 4 : 0;
    int page0 = 0, page1 = 0, next_key = 0;
    auto look_up = [&]() {
      // a step's last tile may not be there: the one before it in its place,
      // whose values are cleared
      const int i = min(next + own_tile, span.count - 1);
      next_key = tile_of(span, i) * 32;
      const int k0 = next_key + 16 * own_half, k1 = next_key + 16 - 16 * own_half;
      if (i >= range.whole_lo && i < range.whole_hi) {
        page0 = table[k0 >> a.page_shift];
        if (R < 4) page1 = table[k1 >> a.page_shift];
      } else {
        page0 = page_of(k0, k1);
        if (R < 4) page1 = page_of(k1, k0);
      }
    };
    if (next < tiles) look_up();
    // where 16 keys lie, in bytes
    auto chunk = [&](int key, int page) -> int64_t {
      if ((uint32_t)page >= (uint32_t)a.num_pages) {
        bad = true;
        page = 0;
      }
      return (int64_t)((uint32_t)page * page_bytes + head) + (uint32_t)(key & page_mask) * row_bytes;
    };
    auto copy = [&](const void* cache, int64_t at16, const lds_byte* dst) {
      const char* from = (const char*)cache + at16;
#pragma unroll
      for (int j = 0; j < T::kChunkLoads; ++j) copy_to_lds(from, src[j], dst + j * 1024);
    };
    // this wave's part of the stream's next tile, into the ring
    auto fetch = [&]() {
      const int key = next_key, p0 = page0, p1 = page1;
      next += STEP;
      ++ahead;
      if (next < tiles) look_up();
      const lds_byte* dst = own + slot_in * (N * T::kBytes);
      slot_in = slot_in + 1 == RING / N ? 0 : slot_in + 1;
      if constexpr (R >= 4) {  // 16 rows of K or of V
        const int x = rg / 2 % 2;
        copy(x ? a.v : a.k, chunk(key + 16 * own_half, p0),
             dst + own_tile * T::kBytes + x * T::kHalf + own_half * (T::kHalf / 2));
      } else {
        const int64_t c0 = chunk(key, p0), c1 = chunk(key + 16, p1);
        if (R == 1 || rg == 0) {
          copy(a.k, c0, dst);
          copy(a.k, c1, dst + T::kHalf / 2);
        }
        if (R == 1 || rg == 1) {
          copy(a.v, c0, dst + T::kHalf);
          copy(a.v, c1, dst + T::kHalf + T::kHalf / 2);
        }
      }
    };
    // waits until the oldest of `ahead` steps in flight has landed
    auto land = [&]() {
      --ahead;
      if (ahead >= 3)
        wait_copies<(C::kAhead >= 3 ? 3 : 0) * C::kLoads>();
      else if (ahead == 2)
        wait_copies<(C::kAhead >= 2 ? 2 : 0) * C::kLoads>();
      else if (ahead == 1)
        wait_copies<(C::kAhead >= 2 || R == 1 ? 1 : 0) * C::kLoads>();
      else
        wait_copies<0>();
    };
    // the ring's first copies leave before the queries are read, so that the
    // wait for the queries does not hold them up
#pragma unroll 1
    for (int i = 0; i < C::kAhead; ++i)
      if (next < tiles) fetch();

    const int rows = req.n * a.group, r0 = rt * ROWS, last = min(r0 + ROWS, rows) - 1;
    const int w0 = r0 + rg * 32;  // this wave's first row
    v8s Q[D / 16];
    int pos;
    {
      const int row = min(w0 + n, last), tok = row / a.group;
      pos = req.kv - req.n + tok;
      const bf16_t* qp = (const bf16_t*)a.q + (req.q0 + tok) * a.q_tok +
                         (h * a.group + row - tok * a.group) * a.q_head + 8 * h2;
#pragma unroll
      for (int kc = 0; kc < D / 16; ++kc) Q[kc] = load_frag_bf16(qp + 16 * kc);
    }
    // the queries are waited for here, not in the walk, where the wait would
    // hold up the copies in flight
#pragma unroll
    for (int kc = 0; kc < D / 16; ++kc) asm volatile("" : "+v"(Q[kc]));
    // positions of this wave's rows
    KeySpan seen = span;
    if (R > 1) {
      seen.pmin = uniform(req.kv - req.n + min(w0, last) / a.group);
      seen.pmax = uniform(req.kv - req.n + min(w0 + 31, last) / a.group);
    }
    const TileRange mine_range = R > 1 ? uniform(tile_range<32>(seen, a.window, a.sinks)) : range;
    RowState<D> st;
    st.clear();
    bool noting = false;

    // notes and clears the odd values of a tile that some row does not see whole
    auto note = [&](const lds_byte* tile, int key) -> bool {
      if (!odd_values<D>(tile, lane)) return false;
      if (!noting) {
        noting = true;
#pragma unroll 1
        for (int x = lane; x < 32 * (D / 8); x += 64) notes[x] = 0;
      }
      note_odd_values<D>(tile, notes, key, pos, a.window, a.sinks, lane);
      return true;
    };

#pragma unroll 1
    for (int i = first * STEP + stream * N; i - stream * N < tiles; i += STEP) {
      lds_byte* const tile = own + slot_out * (N * T::kBytes);
      if constexpr (R == 1) {
        if (i >= tiles) break;
        if (next < tiles) {
          fetch();
          --ahead;
          wait_copies<C::kAhead * C::kLoads>();
        } else {
          land();
        }
        if ((i < range.whole_lo || i >= range.whole_hi) && note(tile, tile_of(span, i) * 32))
          clear_odd_values<D>(tile, 0, 1, lane);
      } else {
        // every wave's copies of this step have landed, and every wave is done
        // with the step before it, whose place the next copies take
        if (next < tiles) {
          --ahead;
          wait_copies<(C::kAhead - 1) * C::kLoads>();
          asm volatile("s_barrier" ::: "memory");
          fetch();
        } else {
          if (i < tiles) land();
          asm volatile("s_barrier" ::: "memory");
        }
        // some stream's tile is not seen whole by all rows: all waves come to
        // the barriers
        if (i - stream * N < range.whole_lo || i - stream * N + STEP > range.whole_hi) {
          bool odd[N] = {};
          if (i < tiles) {
#pragma unroll
            for (int x = 0; x < N; ++x) odd[x] = note(tile + x * T::kBytes, tile_of(span, i + x) * 32);
          }
          __syncthreads();
#pragma unroll
          for (int x = 0; x < N; ++x)
            if (odd[x]) clear_odd_values<D>(tile + x * T::kBytes, rg, R, lane);
          __syncthreads();
        }
        if (i >= tiles) continue;
      }
      slot_out = slot_out + 1 == RING / N ? 0 : slot_out + 1;
      if (R > 1 && (i >= mine_range.some_hi || (i + N <= mine_range.some_lo && i >= mine_range.sink_hi)))
        continue;  // none of this wave's rows sees it
      v16f s[N];
#pragma unroll
      for (int x = 0; x < N; ++x) s[x] = scores<D>(tile + x * T::kBytes, k0_off, Q);
      ValueFrags v = read_values<D>(tile, v0_off, 0);
      __builtin_amdgcn_sched_barrier(0);
      if (i < mine_range.whole_lo || i + N > mine_range.whole_hi) {
#pragma unroll
        for (int x = 0; x < N; ++x) {
          const int key = tile_of(span, i + x) * 32;
#pragma unroll
          for (int j = 0; j < 16; ++j)
            if (!visible(key + 16 * (j >> 3) + 8 * h2 + (j & 7), pos, a.window, a.sinks)) s[x][j] = -INFINITY;
        }
      }
      constexpr bool FINE = R == 1;
      v8s p[N][2], rest[N][2];
      softmax_step<D, N, FINE>(s, st, p, rest, a.scale_log2);
      constexpr int PAIRS = D / 64;
#pragma unroll
      for (int x = 0; x < N * PAIRS; ++x) {
        // the next fragments are read under these products
        ValueFrags after;
        if (x + 1 < N * PAIRS)
          after = read_values<D>(tile + (x + 1) / PAIRS * T::kBytes, v0_off, (x + 1) % PAIRS);
        __builtin_amdgcn_sched_barrier(0);
        add_values<D>(v, x % PAIRS, st, p[x / PAIRS]);
        if constexpr (FINE) add_values<D>(v, x % PAIRS, st, rest[x / PAIRS]);
        v = after;
      }
    }

    // join the streams of a row group: each wave writes JOIN rows at a time to
    // LDS, over the rings
    const bool whole = WHOLE || (first == 0 && stop == seg);
    const int64_t part = 2 * (int64_t)blockIdx.x + (first == 0);
    float* const so = (float*)ring;
    if (tid == 0) s_bad = 0;
    if (lane == 0) s_noting[w] = noting;
    {
      const float l = sum_halves(st.l);
      if (h2 == 0) {
        s_m[w][n] = st.m;
        s_l[w][n] = l;
      }
    }
    __syncthreads();
    if (bad) s_bad = 1;
#pragma unroll 1
    for (int j0 = 0; j0 < 32; j0 += JOIN) {
      if (j0) __syncthreads();
      if (n >= j0 && n < j0 + JOIN) {
#pragma unroll
        for (int blk = 0; blk < D / 32; ++blk)
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int piece = (8 * blk + 2 * x + h2) ^ (n & (D / 4 - 1));
            *(float4*)(so + ((w * JOIN + n - j0) * D + piece * 4)) = make_float4(
                st.o[blk][4 * x], st.o[blk][4 * x + 1], st.o[blk][4 * x + 2], st.o[blk][4 * x + 3]);
          }
      }
      // a row's factors for its streams, the division by the sum in them where
      // the row is complete
      float top = -INFINITY, den = 0.f;
      const int row_ = tid & 31, g_ = tid >> 5;
      const bool joins = j0 == 0 && tid < 32 * R;
      if (joins) {
#pragma unroll
        for (int x = 0; x < S; ++x) top = fmaxf(top, s_m[g_ * S + x][row_]);
        const float ref = top == -INFINITY ? 0.f : top;
        float f[S];
#pragma unroll
        for (int x = 0; x < S; ++x) {
          f[x] = __builtin_amdgcn_exp2f((s_m[g_ * S + x][row_] - ref) * a.scale_log2);
          den += f[x] * s_l[g_ * S + x][row_];
        }
        const float inv = !whole ? 1.f : den == 0.f ? 0.f : 1.f / den;
#pragma unroll
        for (int x = 0; x < S; ++x) s_f[g_ * S + x][row_] = f[x] * inv;
      }
      __syncthreads();
      const bool spoilt = s_bad != 0;
      if (joins && r0 + g_ * 32 + row_ <= last) {
        if (spoilt) den = NAN;
        if (whole) {
          const int r = r0 + g_ * 32 + row_, tok = r / a.group, hq = h * a.group + r - tok * a.group;
          if (a.lse)
            a.lse[(int64_t)(req.q0 + tok) * a.q_heads + hq] = den == 0.f ? -INFINITY : top * a.scale + logf(den);
        } else {
          *(float2*)(a.part_ml + (part * ROWS + g_ * 32 + row_) * 2) = make_float2(top, den);
        }
      }
      int odd = 0;
#pragma unroll
      for (int x = 0; x < C::W; ++x) odd |= s_noting[x];
#pragma unroll 4
      for (int i = tid; i < R * JOIN * (D / 4); i += THREADS) {
        const int piece = i % (D / 4), row = j0 + (i / (D / 4)) % JOIN, g = i / (D / 4) / JOIN;
        const int in_tile = g * 32 + row;  // row of the row tile
        if (r0 + in_tile > last) continue;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int x = 0; x < S; ++x) {
          const float f = s_f[g * S + x][row];
          const float4 y =
              *(const float4*)(so + (((g * S + x) * JOIN + row - j0) * D + (piece ^ (row & (D / 4 - 1))) * 4));
          o.x += f * y.x;
          o.y += f * y.y;
          o.z += f * y.z;
          o.w += f * y.w;
        }
        if (__builtin_expect(odd, 0)) {
#pragma unroll 1
          for (int x = 0; x < S; ++x)
            if (s_noting[g * S + x]) {
              const uint32_t note = s_notes[g * S + x][row * (D / 8) + piece / 2] >> (8 * (piece & 1));
              o.x = noted(o.x, note & 3);
              o.y = noted(o.y, note >> 2 & 3);
              o.z = noted(o.z, note >> 4 & 3);
              o.w = noted(o.w, note >> 6 & 3);
            }
        }
        if (whole) {
          if (spoilt) o = make_float4(NAN, NAN, NAN, NAN);
          const int r = r0 + in_tile, tok = r / a.group, hq = h * a.group + r - tok * a.group;
          *(u32x2*)((bf16_t*)a.out + (req.q0 + tok) * a.o_tok + hq * a.o_head + 4 * piece) =
              u32x2{pack_bf16(o.x, o.y), pack_bf16(o.z, o.w)};
        } else {
          *(float4*)(a.part_o + (part * ROWS + in_tile) * D + 4 * piece) = o;
        }
      }
    }
    __syncthreads();
    at = uniform(WHOLE || a.pieces ? end : at + stop - first);
  }
}

// Joins the parts of split segments: 256 threads take 1024 / D rows of one
// (request, row tile, key head).  4.5 us for 8 requests with 16 tokens, of which
// the launch and the way to memory and back are most.
template <int D, int R>
__global__ __launch_bounds__(256) void attend_join_kernel(AttendArgs a, int workers, int row_groups) {
  constexpr int STEP = Shape<D, R>::kStep, ROWS = Shape<D, R>::kRows, PER = 1024 / D;
  const int b = blockIdx.z, rt = blockIdx.x, h = blockIdx.y / row_groups, group = blockIdx.y - h * row_groups;
  const Request req = request_of(a.q_start, a.kv_len, b, a.tokens, a.max_new, a.max_kv);
  const int rows = req.n * a.group, r0 = rt * ROWS;
  const int row = group * PER + threadIdx.x / (D / 4), piece = threadIdx.x % (D / 4);
  if (r0 >= rows || group * PER >= ROWS) return;
  const int tile = a.pieces ? b * a.row_tiles + rt : b;
  const int from0 = a.plan[tile];
  int g0, g1;
  if (a.pieces) {
    const int pieces = (a.plan[tile + 1] - from0) / a.kv_heads;
    g0 = from0 + h * pieces;
    g1 = g0 + pieces - 1;
  } else {
    const int total = a.plan[a.requests];
    const int share = max(kMinShare, (total + workers - 1) / workers);
    int from = from0 + steps_before<ROWS, STEP>(a, req, rt, threadIdx.x & 63);
    const int seg = steps_of(row_tile_span<ROWS>(a, req, rt).count, STEP);
    from += h * seg;
    g0 = from / share;
    g1 = (from + seg - 1) / share;
  }
  if (g0 == g1 || r0 + row >= rows) return;
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
    o.x = scaled(o.x, fo) + scaled(y.x, fn);
    o.y = scaled(o.y, fo) + scaled(y.y, fn);
    o.z = scaled(o.z, fo) + scaled(y.z, fn);
    o.w = scaled(o.w, fo) + scaled(y.w, fn);
    top = mn;
  }
  const float inv = den == 0.f ? 0.f : 1.f / den;
  const int tok = (r0 + row) / a.group, hq = h * a.group + r0 + row - tok * a.group;
  *(u32x2*)((bf16_t*)a.out + (req.q0 + tok) * a.o_tok + hq * a.o_head + 4 * piece) =
      u32x2{pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv)};
  if (piece == 0 && a.lse)
    a.lse[(int64_t)(req.q0 + tok) * a.q_heads + hq] = den == 0.f ? -INFINITY : top * a.scale + logf(den);
}

template <int D, int R, bool WHOLE>
void launch_kernel(const AttendArgs& a, dim3 grid, hipStream_t st) {
  using C = Shape<D, R>;
  hipLaunchKernelGGL((attend_split_kernel<D, R, WHOLE>), grid, dim3(C::kThreads), C::kLds, st, a);
}

// more than the default 64 KB of LDS
template <int D, int R>
hipError_t allow_lds() {
  for (const void* k : {(const void*)&attend_split_kernel<D, R, false>, (const void*)&attend_split_kernel<D, R, true>}) {
    const hipError_t e = hipFuncSetAttribute(k, hipFuncAttributeMaxDynamicSharedMemorySize, Shape<D, R>::kLds);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}
template <int D>
hipError_t allow_lds_d() {
  hipError_t e = allow_lds<D, 1>();
  if (e == hipSuccess) e = allow_lds<D, 4>();
  if constexpr (D < 256) {
    if (e == hipSuccess) e = allow_lds<D, 2>();
    if (e == hipSuccess) e = allow_lds<D, 8>();
  }
  return e;
}

template <int D, int R>
void launch(AttendArgs a, int cus, hipStream_t st) {
  using C = Shape<D, R>;
  constexpr int ROWS = C::kRows, PER = 1024 / D;
  const int64_t rows = (int64_t)a.max_new * a.group;
  const int64_t row_tiles = (rows + ROWS - 1) / ROWS;
  const int64_t segments = a.requests * row_tiles * a.kv_heads;
  int64_t keys = a.max_kv;  // the most that a segment has
  if (a.window && (int64_t)a.window + ROWS / a.group + a.sinks + 65 < keys)
    keys = (int64_t)a.window + ROWS / a.group + a.sinks + 65;
  const int64_t seg_most = (keys + 32 * C::kStep - 1) / (32 * C::kStep) + 1;
  // One launch where there is little to split, or enough segments to fill the
  // chip several times over.  Prompts cost much to split (256 or 128 rows' sums
  // go through memory), about 10 steps: undivided, one prompt of 1000 tokens over
  // 1000 keys (8.5 steps more than an even share) takes 41 us against 46, but of
  // 512 over 1024 (12.8) 41 against 37, over 2048 (24.8) 68 against 46.
  // Also where the bounds allow more steps than 32 bits count (from 2^27 keys
  // with thousands of segments): lengths are not trusted, and a sum that wraps
  // would lead past the cache.
  const bool prompt = R == 8 || (D == 256 && R == 4);
  if (seg_most <= 4 || segments * seg_most >= (int64_t)1 << 31 || (prompt ? seg_most * (cus - segments) <= 10 * (int64_t)cus
                               : segments >= (R == 4 ? 2 : 8) * (int64_t)cus))
    return launch_kernel<D, R, true>(a, dim3(a.kv_heads, (unsigned)row_tiles, a.requests), st);
  const int64_t need = (segments * seg_most + kMinShare - 1) / kMinShare;
  const int workers = (int)(need < cus ? need : cus);
  a.row_tiles = (int)row_tiles;
  a.pieces = a.requests * row_tiles <= 64 && 2 * segments <= workers;
  launch_kernel<D, R, false>(a, dim3(workers), st);
  if (hipPeekAtLastError() != hipSuccess) return;  // the join would follow the plan of an earlier call
  const int groups = (int)(((rows < ROWS ? rows : ROWS) + PER - 1) / PER);
  hipLaunchKernelGGL((attend_join_kernel<D, R>), dim3((unsigned)row_tiles, a.kv_heads * groups, a.requests),
                     dim3(256), 0, st, a, workers, groups);
}

// The fewest rows to a workgroup that hold a request's, so that its keys are
// read once; beyond 128 rows the largest.  A wave costs the same whether its
// rows are there or not.
template <int D>
void launch_d(const AttendArgs& a, int cus, hipStream_t st) {
  const int64_t rows = (int64_t)a.max_new * a.group;
  if (rows <= 32) return launch<D, 1>(a, cus, st);
  if constexpr (D == 256) {
    launch<D, 4>(a, cus, st);
  } else {
    if (rows <= 64) return launch<D, 2>(a, cus, st);
    if (rows <= 128) return launch<D, 4>(a, cus, st);
    launch<D, 8>(a, cus, st);
  }
}

}  // namespace

// workspace: two parts of the most rows, their outputs and (m, l), for each
// workgroup
size_t attend_split_floats(int head_dim, int cus) {
  return (size_t)2 * cus * (head_dim == 256 ? 128 : 256) * (head_dim + 2);
}

hipError_t attend_split_prepare(int head_dim) {
  return head_dim == 64 ? allow_lds_d<64>() : head_dim == 128 ? allow_lds_d<128>() : allow_lds_d<256>();
}

void launch_attend_split(int head_dim, const AttendArgs& a, int cus, hipStream_t st) {
  if (head_dim == 64)
    launch_d<64>(a, cus, st);
  else if (head_dim == 128)
    launch_d<128>(a, cus, st);
  else
    launch_d<256>(a, cus, st);
}
