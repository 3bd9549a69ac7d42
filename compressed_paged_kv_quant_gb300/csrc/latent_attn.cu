// latent_attn.cu -- attention of new tokens over the paged latents, absorbed form, on the
// tcgen05 tensor cores.
//
//   out[row][h] = sum_t softmax_t(scale (q_c . c_t + q_r . r_t)) c_t,  c 512 dims, r 64 dims
//
// One latent serves every head, so a token's 1,152 (bf16) or 656 (MXFP8) bytes feed
// 2 * 1,088 * heads FLOP: with 16 rows (query, head) in a CTA the bound is HBM, with 64 it is the rate at
// which shared memory feeds the tensor cores, with 32 it is near both.
//
// Tile: 64 keys (a page) x N rows (16, 32 or 64; row = query * heads + head), transposed:
//   S^T [64 keys][N]   = K . Q^T   M = 64, K = 576: A = the page as it lies (K-major, swizzled)
//   O^T [512 dims][N] += V^T . P^T  M = 4 x 128, K = 64: A = the same bytes read dims-major
// so a page is fetched once, by bulk copies of contiguous 8 and 16 KB, and serves as K and V with no
// transposition.  Rows as the N dimension let few heads cost few tensor cycles, and the
// 512-dim output of 64 rows takes half of the tensor memory, which leaves room for two S tiles.
//
// Warps: 0-3 softmax and output (thread: 2 keys x N / 4 rows of S^T), 4 MMA issue, 5 bulk copies, 6-7 the
// queries; MXFP8 8-15, which turn codes into the bf16 tile (exact: mx_quad); with 64 rows the last four help
// with the softmax, half of the rows each.
//
// Softmax: a row's scores are taken relative to a reference that follows the row's maximum.  It moves only when
// a score passes it by more than 2^8 (and with a part's first keys), which one barrier with a vote
// detects; the maxima are reduced, and O is rescaled, only then.  l is summed in FP32 from the unrounded weights,
// P goes to the tensor cores in bf16 (the type of V): half a bf16 step a weight, as much as the output's own rounding
// (with it the error against 64 bits is 1.7e-3 to 2.1e-3 of the output's norm, 1.7e-3 of which a P in 32 bits has too).  P as
// two bf16 terms would double the products of P.V.
//
// Work: the (lane, page) list is cut into W equal ranges, one CTA a range and row tile, so ragged
// lanes balance; a lane within one range is finished there, else its parts are FP32 partials that
// latent_attn_combine merges.  A range holds two parts at most that are not a whole lane: the rest of a lane that began
// before it, and the first pages of one that goes on behind it.  The former takes slot w of 2 W, the latter W + w.
// The kernels are launched programmatically: a start overlaps the end of the kernel before it.
// Every wait is bounded; on a timeout the CTA flags KVQ_STATUS_TIMEOUT and ends.
//
// Measured, whole calls: 8 lanes x 40,960 tokens, bf16, 16 heads 70 us (5.4 TB/s, 80% of the copy bandwidth: HBM
// bound), 32 heads 75, 64 heads 84, 128 heads 112 (815 TFLOP/s).  With 64 rows a page takes 2,570 clocks: the tensor cores read 147 KB
// for the scores and 98 for P.V, the page's copy writes 74, all through shared memory at 128 B a clock.  MXFP8, 16
// heads 58 us (1.2 us a page; 236 KB through shared memory, and the conversion's latencies), 128 heads 131.  One lane
// of 257 tokens 12.4 us, latencies of five pages one after another.
#include "latent.cuh"
#include "tcgen05.cuh"

#include <algorithm>

namespace kvq {

constexpr int LA_SMS = 152;
constexpr int LA_MIN_TILES = 4;      // pages of a range, at least
constexpr int LA_LANE_TILES = 8;     // lanes of at most so many pages are one range each
constexpr int LA_MAX_T = LA_SMS / 2; // more row tiles than this a lane: one range a lane
constexpr int LA_PREFETCH = 3;       // tiles
constexpr float LA_SLACK = 8.0f;
constexpr float LA_LOW = -3e38f;     // the maximum of a part without keys: finite, so that -inf - it is -inf

template <int FMT, int N>
struct LaCfg {
  static constexpr bool MX = FMT == KVQ_LATENT_MXFP8;
  // Groups of four softmax warps, each with a part of the rows: two for 64 rows.  Long parts are bound by shared memory
  // and do not gain, but a part's start and end and masked tiles take half as long (16 lanes x 4 drafted tokens x
  // 128 heads: bf16 85 -> 81 us, MXFP8 97 -> 93; one lane of 500 tokens 20.3 -> 18.2; MXFP8 8 x 40,960 x 128
  // heads 129 -> 131, with fewer registers for the conversion).  W2: first warp of the second group.
  static constexpr int SG = N == 64 ? 2 : 1, W2 = MX ? 16 : 8;
  static constexpr int THREADS = (MX ? 512 : 256) + 128 * (SG - 1);
  // Slots of the rings, in as much shared memory as there is.  A barrier's phase is told by its parity, so
  // nobody may wait for a phase two ahead: at least 4 slots where a tile's 4 pairs go side by side.
  static constexpr int NROPE = 2;
  static constexpr int NPAIR = N == 64 ? 8 : N == 32 ? 10 : 11;
  // Pairs of the next scores before P.V.  All 4, with two P buffers, where there is room: scores and softmax
  // of neighbouring tiles then overlap entirely.  64 rows have room for 8 pairs and one P buffer: with 3 or 4
  // ahead the next scores would wait for a page whose slots only P.V frees (8 x 40,960 x 128 heads: 129 us with
  // 2, 140 with 3).
  static constexpr uint32_t AHEAD = N == 64 ? 2 : 4;
  static constexpr int NP = N == 64 ? 1 : 2;
  static constexpr int SM_Q = 0;
  static constexpr int SM_P = SM_Q + LNCHUNK * N * 128;
  static constexpr int SM_ROPE = SM_P + NP * N * 128;
  static constexpr int SM_PAIR = SM_ROPE + NROPE * LCHUNK;
  static constexpr int SM_RED = SM_PAIR + NPAIR * 2 * LCHUNK;   // float [4][N], then int64 [N] of the output rows
  static constexpr int SM_FAC = SM_RED + 16 * N;             // float [N]
  static constexpr int SM_LIM = SM_FAC + 4 * N;              // int [N]
  static constexpr int SM_BAR = SM_LIM + 4 * N;
  // What has landed is told by half tiles (rotary chunk and pairs 0, 1; pairs 2, 3), which costs the MMA warp two
  // waits a tile; what is free, by slots.  No more than 3 tiles are under way.
  static constexpr int B_FULL = 0, B_PAIR_EMPTY = 6, B_ROPE_EMPTY = B_PAIR_EMPTY + NPAIR, B_S_FULL = B_ROPE_EMPTY + NROPE,
                       B_P_FULL = B_S_FULL + 2, B_PV_DONE = B_P_FULL + NP, B_Q_FULL = B_PV_DONE + 2,
                       B_Q_EMPTY = B_Q_FULL + 1, B_END = B_Q_EMPTY + 1, NBAR = B_END + 1;
  static constexpr int SM_TMEM = SM_BAR + 8 * NBAR;
  static constexpr int SM_START = SM_TMEM + 8;               // the range's first lane, pages before it
  static constexpr int SM_STOP = SM_START + 8;               // softmax warps: tile at which they stop, + 1
  static constexpr int SM_PROG = SM_STOP + 4;               // tiles whose copies are issued
  static constexpr int SM_SCAN = SM_STOP + 8;                // int a warp
  static constexpr int SMEM = SM_SCAN + 96 + 1024;           // + slack to align the base to 1,024 B
  static constexpr uint32_t TMEM_COLS = N == 64 ? 512 : N == 32 ? 256 : 128;
  static_assert(SMEM <= 232448, "shared memory of a CTA");
};

// loads that stay where they are written
__device__ __forceinline__ uint4 ld_global16(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.v4.b32 {%0, %1, %2, %3}, [%4];\n" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t ld_global4(const void* p) {
  uint32_t v;
  asm volatile("ld.global.nc.b32 %0, [%1];\n" : "=r"(v) : "l"(p) : "memory");
  return v;
}

struct LaGrid {
  int T;        // row tiles a lane
  int W;        // ranges of the page list; 0: one range a lane
};

static int la_rows(int heads, int max_n_q) {   // N: rows of a tile
  const int64_t rows = (int64_t)heads * max_n_q;
  return rows <= 16 ? 16 : rows <= 32 ? 32 : 64;
}

static LaGrid la_grid(int heads, int max_n_q, int max_seq_len) {
  const int N = la_rows(heads, max_n_q);
  LaGrid g;
  g.T = (int)(((int64_t)heads * max_n_q + N - 1) / N);
  const bool ranges = g.T > 0 && g.T <= LA_MAX_T && max_seq_len > LA_LANE_TILES * P;
  g.W = ranges ? LA_SMS / g.T : 0;
  return g;
}

static size_t la_bytes(int64_t rows, int lanes) {   // rows of partials
  return (size_t)rows * (LAT + 2) * sizeof(float) + ((size_t)lanes + 1) * sizeof(int) + 256;
}

// Bytes that this very call touches, and a bound of them for it and every smaller one (W T is at most the SMs, for any T).
size_t latent_attn_needs(int heads, int lanes, int max_n_q, int max_seq_len) {
  const LaGrid g = la_grid(heads, max_n_q, max_seq_len);
  return g.W == 0 ? 256 : la_bytes((int64_t)2 * g.W * g.T * la_rows(heads, max_n_q), lanes);
}

size_t latent_attn_workspace(int heads, int lanes, int max_n_q, int max_seq_len) {
  const bool ranges = max_n_q > 0 && max_seq_len > LA_LANE_TILES * P;
  return ranges ? la_bytes((int64_t)2 * LA_SMS * la_rows(heads, max_n_q), lanes) : 256;
}

// After the partials: pages of a range, then for each lane the pages of the list before it.
__device__ __forceinline__ int* la_meta(const LatentAttnArgs& a, const LaGrid& g, int N) {
  return reinterpret_cast<int*>(a.ws + (int64_t)2 * g.W * g.T * N * (LAT + 2));
}

// pages of lane b in the list
__device__ __forceinline__ int la_lane_tiles(const LatentAttnArgs& a, int b, bool report) {
  int nq, row0, pos0;
  return latent_lane(a, b, nq, row0, pos0, report) ? (pos0 + nq + P - 1) / P : 0;
}

// The lane that holds page `target(total)` of the list, in res[0], and the pages of the list before it, in
// res[1], by all threads of the block (each sums a run of lanes); res[0] is a.c.lanes if the list is
// shorter.  Returns the page asked for.  scan: an int a warp.  The reporting block also leaves the pages
// before each lane at `before_lane`.
template <int THREADS, class F>
__device__ __forceinline__ int64_t la_find(const LatentAttnArgs& a, int* scan, int* res, bool report, int* before_lane,
                                           F target) {
  const int lanes = a.c.lanes, per = (lanes + THREADS - 1) / THREADS;
  const int i0 = min(lanes, (int)threadIdx.x * per), i1 = min(lanes, i0 + per);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int sum = 0;
  for (int b = i0; b < i1; b++) sum += la_lane_tiles(a, b, report);
  int inc = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xFFFFFFFFu, inc, o);
    if (lane >= o) inc += v;
  }
  if (lane == 31) scan[warp] = inc;
  if (threadIdx.x == 0) res[0] = lanes;
  __syncthreads();
  int before = 0, total = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; w++) {
    const int v = scan[w];
    if (w < warp) before += v;
    total += v;
  }
  const int64_t want = target(total);
  int at = before + inc - sum;
  if (report || (want >= at && want < at + sum)) {
    for (int b = i0; b < i1; b++) {
      const int n = per == 1 ? sum : la_lane_tiles(a, b, false);
      if (want >= at && want < at + n) {
        res[0] = b;
        res[1] = at;
      }
      if (report) before_lane[b] = at;
      at += n;
    }
  }
  __syncthreads();
  return want;
}

__device__ __forceinline__ int la_range(int total, int W) {   // pages of a range
  return max((int)(((unsigned)total + W - 1) / (unsigned)W), LA_MIN_TILES);
}

// The parts of a CTA's range, in order.
struct LaPart {
  int b, nq, row0, pos0;
  int t0, t1;      // pages [t0, t1) of the lane
  int rows;        // rows of the lane, all tiles
  int tiles;       // pages that this row tile attends
};
struct LaIter {
  int b, off, left;
  template <int N>
  __device__ __forceinline__ bool next(const LatentAttnArgs& a, int rt, LaPart& p) {
    while (left > 0 && b < a.c.lanes) {
      if (!latent_lane(a, b, p.nq, p.row0, p.pos0, false)) {
        b++;
        off = 0;
        continue;
      }
      const int n = (p.pos0 + p.nq + P - 1) / P;
      p.b = b++;
      p.t0 = off;
      off = 0;
      const int take = min(n - p.t0, left);
      left -= take;
      p.rows = p.nq * a.heads;
      const int r0 = rt * N;
      if (r0 >= p.rows) continue;
      const int qlast = min(p.nq - 1, (r0 + N - 1) / a.heads);
      p.tiles = (p.pos0 + qlast + P) / P;
      p.t1 = min(p.t0 + take, p.tiles);
      if (p.t0 < p.t1) return true;
    }
    return false;
  }
};

// Maxima of 2 K values with those of the lane `o` away: a lane keeps K of them, `first` the number of the first one
// (K = 0: of one value, kept by both).
template <int K, int M>
__device__ __forceinline__ void la_halve(float (&v)[M], int& first, int lane, int o) {
  if (K == 0) v[0] = fmaxf(v[0], __shfl_xor_sync(0xFFFFFFFFu, v[0], o));
  const bool up = (lane & o) != 0;
#pragma unroll
  for (int i = 0; i < K; i++) {
    const float give = up ? v[i] : v[i + K], keep = up ? v[i + K] : v[i];
    v[i] = fmaxf(keep, __shfl_xor_sync(0xFFFFFFFFu, give, o));
  }
  first += up ? K : 0;
}

template <int FMT, int N>
__global__ void __launch_bounds__(LaCfg<FMT, N>::THREADS, 1) latent_attn_tc(LatentAttnArgs a, LaGrid g) {
  using C = LaCfg<FMT, N>;
  constexpr bool MX = C::MX;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t sm = smem_u32(smem);
  // (the shuffle tells the compiler that the warp index is the same in all lanes: the roles'
  // branches are uniform)
  const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int rt = blockIdx.x % g.T, w = blockIdx.x / g.T;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::SM_TMEM + 4);
  int* start = reinterpret_cast<int*>(smem + C::SM_START);
  auto BAR = [&](int i) { return sm + C::SM_BAR + 8u * i; };

  if (threadIdx.x < C::NBAR) {   // a barrier a thread
    const int i = threadIdx.x;
    const int arrivals = i < 3                ? 3 + 2 * MX     // copies of a half tile, or the warps that convert it
                         : i < C::B_PAIR_EMPTY ? 2 + 2 * MX
                         : i >= C::B_P_FULL && i < C::B_PV_DONE ? 4 * C::SG
                         : i == C::B_Q_FULL   ? 2
                                              : 1;
    mbar_init(BAR(i), arrivals);
    if (i == 0) {
      *abort_flag = 0;
      *reinterpret_cast<int*>(smem + C::SM_STOP) = 0;
      *reinterpret_cast<int*>(smem + C::SM_PROG) = 0;
    }
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  }
  if (warp == 4) t5_alloc(sm + C::SM_TMEM, C::TMEM_COLS);
  t5_fence_before();
  latent_wait();
  LaIter it0;
  if (g.W > 0) {
    int R = 0, total = 0;
    int* meta = la_meta(a, g, N);
    const int64_t page = la_find<C::THREADS>(a, reinterpret_cast<int*>(smem + C::SM_SCAN), start, blockIdx.x == 0, meta + 1,
                                             [&](int tot) {
                                               total = tot;
                                               R = la_range(tot, g.W);
                                               return (int64_t)w * R;
                                             });
    if (blockIdx.x == 0 && threadIdx.x == 0) meta[0] = R;
    it0.b = start[0];
    it0.off = it0.b < a.c.lanes ? (int)(page - start[1]) : 0;
    it0.left = (int)min((int64_t)R, total - page);
  } else {
    __syncthreads();
    it0.b = w;
    it0.off = 0;
    it0.left = la_lane_tiles(a, w, rt == 0 && threadIdx.x == 0);
  }
  t5_fence_after();
  const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, *reinterpret_cast<volatile uint32_t*>(smem + C::SM_TMEM), 0);
  constexpr uint32_t TM_S = 4 * N;
  bool timed_out = false;
  LaIter it = it0;
  LaPart p;

  if (warp < 4 || (C::SG == 2 && warp >= C::W2)) {
    // ================================================================= softmax and output
    constexpr int SG = C::SG, J = N / 8 / SG; // 8-row blocks of S^T; this thread's rows c0 + 8j + {0, 1}
    float* red = reinterpret_cast<float*>(smem + C::SM_RED);
    float* fac = reinterpret_cast<float*>(smem + C::SM_FAC);
    int* lim = reinterpret_cast<int*>(smem + C::SM_LIM);
    int64_t* rowoff = reinterpret_cast<int64_t*>(smem + C::SM_RED);
    const int grp = SG == 2 && warp >= C::W2, quad = warp & 3, tid = threadIdx.x - (32 * C::W2 - 128) * grp;
    const int kA = 16 * quad + (lane >> 2), c0 = grp * (N / SG) + 2 * (lane & 3);
    const uint32_t tl = tmem + ((uint32_t)(32 * quad) << 16);
    auto sync4 = [] { asm volatile("barrier.cta.sync 1, %0;\n" ::"n"(128 * SG) : "memory"); };
    auto vote4 = [](bool x) {
      uint32_t any;
      asm volatile(
          "{\n .reg .pred p, q;\n setp.ne.u32 q, %1, 0;\n barrier.cta.red.or.pred p, 2, %2, q;\n selp.u32 %0, 1, 0, p;\n}\n"
          : "=r"(any)
          : "r"((uint32_t)x), "n"(128 * SG)
          : "memory");
      return any != 0;
    };
    // A warp whose wait ran out goes on to the next vote of the four warps, so that none is left
    // at a barrier: it leaves the tile's number before the vote, and all four stop behind it.
    volatile int* stop = reinterpret_cast<volatile int*>(smem + C::SM_STOP);
    bool bad = false;
    int j = 0;                               // tiles of the CTA so far
    while (!timed_out && it.template next<N>(a, rt, p)) {
      const int r0 = rt * N, first_pos = p.pos0 + r0 / a.heads;
      sync4();                               // the last part's readers are done
      for (int r = tid; r < N; r += 128 * SG) {
        const int gr = r0 + r, qi = gr / a.heads;
        const bool ok = gr < p.rows;
        lim[r] = ok ? p.pos0 + qi : -1;
      }
      sync4();
      float m[2 * J], l[2 * J];
#pragma unroll
      for (int i = 0; i < 2 * J; i++) {
        m[i] = 0.f;
        l[i] = 0.f;
      }
      const int zero_from = p.pos0 + min(p.nq - 1, (r0 + N - 1) / a.heads) + 1;   // keys attended by the tile's rows
      const int64_t pt = (int64_t)p.b * a.c.max_pages;
      int32_t phys = a.c.page_table[pt + p.t0];
      bool fresh = true;                     // no keys yet: the references follow the first maxima, up or down
      for (int t = p.t0; t < p.t1; t++, j++) {
        const bool oob = phys < 0 || phys >= a.c.pool_pages;
        if (t + 1 < p.t1) phys = a.c.page_table[pt + t + 1];
        const int buf = j & 1;
        if (!bad) bad = __any_sync(0xFFFFFFFFu, *abort_flag != 0) || !mbar_wait_warp(BAR(C::B_S_FULL + buf), (j >> 1) & 1);
        if (bad) {
          *abort_flag = 1;
          *stop = j + 1;
        }
        t5_fence_after();
        uint32_t sv[4 * J];
        t5_ld_frag(tl + TM_S + buf * N + grp * (N / SG), sv);
        t5_wait_ld();
        t5_ready(sv);
        // x = score (log2 domain) - its row's reference; masked keys are -inf
        float x[4 * J], over[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        const bool all = !oob && t * P + P - 1 <= first_pos && r0 + N <= p.rows;
#pragma unroll
        for (int i = 0; i < 2 * J; i++) {      // row c0 + 8 (i / 2) + i % 2: keys A and B
          const int e = 4 * (i >> 1) + (i & 1);
          x[e] = fmaf(__uint_as_float(sv[e]), a.scale_log2, -m[i]);
          x[e + 2] = fmaf(__uint_as_float(sv[e + 2]), a.scale_log2, -m[i]);
        }
        if (!all) {
          const int keyA = oob ? INT_MAX : t * P + kA, keyB = oob ? INT_MAX : t * P + kA + 8;
#pragma unroll
          for (int jj = 0; jj < J; jj++) {
            const int2 lm = *reinterpret_cast<const int2*>(lim + c0 + 8 * jj);
            x[4 * jj] = keyA <= lm.x ? x[4 * jj] : -INFINITY;
            x[4 * jj + 1] = keyA <= lm.y ? x[4 * jj + 1] : -INFINITY;
            x[4 * jj + 2] = keyB <= lm.x ? x[4 * jj + 2] : -INFINITY;
            x[4 * jj + 3] = keyB <= lm.y ? x[4 * jj + 3] : -INFINITY;
          }
        }
#pragma unroll
        for (int i = 0; i < 2 * J; i++) {
          const int e = 4 * (i >> 1) + (i & 1);
          over[i & 3] = max3(over[i & 3], x[e], x[e + 2]);
        }
        // does any score pass its row's reference by more than the slack?
        const bool any = vote4(fmaxf(fmaxf(over[0], over[1]), fmaxf(over[2], over[3])) > LA_SLACK);
        if (*stop != 0 && *stop <= j + 1) {
          timed_out = true;
          break;
        }
        if (any || fresh) {
          // The rows' maxima over the warp's keys: each step the lanes exchange half of their values, so that
          // a thread ends with the maxima of one row or two.  (Code that runs once a part costs the fetch of its
          // instructions: kept short.)
          float mx[2 * J];
#pragma unroll
          for (int i = 0; i < 2 * J; i++) mx[i] = fmaxf(x[4 * (i >> 1) + (i & 1)], x[4 * (i >> 1) + (i & 1) + 2]);
          int first = 0;
          la_halve<J>(mx, first, lane, 16);
          la_halve<J / 2>(mx, first, lane, 8);
          la_halve<J / 4>(mx, first, lane, 4);
#pragma unroll
          for (int i = 0; i < (J + 3) / 4; i++) red[quad * N + c0 + 8 * ((first + i) >> 1) + ((first + i) & 1)] = mx[i];
          sync4();
          if (tid < N) {                       // how far each reference moves, and what that scales the sums by
            const float d = fmaxf(fmaxf(red[tid], red[N + tid]), fmaxf(red[2 * N + tid], red[3 * N + tid]));
            const bool move = fresh ? d > -INFINITY : d > LA_SLACK;
            red[tid] = move ? d : 0.f;
            fac[tid] = move && !fresh ? ex2(-d) : 1.0f;   // (fresh: the sums are zeros)
          }
          sync4();
#pragma unroll
          for (int i = 0; i < 2 * J; i++) {
            const int r = c0 + 8 * (i >> 1) + (i & 1), e = 4 * (i >> 1) + (i & 1);
            const float d = red[r];
            m[i] += d;
            l[i] *= fac[r];
            x[e] -= d;
            x[e + 2] -= d;
          }
          if (!fresh) {     // O must be stable: P.V of the tile before complete (with one P buffer S came after it)
            if (C::NP == 2) {
              bad = !mbar_wait_warp(BAR(C::B_PV_DONE + ((j - 1) & 1)), ((j - 1) >> 1) & 1);
              t5_fence_after();
            }
#pragma unroll 1
            for (int cb = grp * (4 * N / SG); cb < (grp + 1) * (4 * N / SG); cb += 16) {
              uint32_t o[16];
              t5_ld16(tl + cb, o);
              t5_wait_ld();
              t5_ready(o);
#pragma unroll
              for (int i = 0; i < 16; i++) o[i] = __float_as_uint(__uint_as_float(o[i]) * fac[(cb & (N - 1)) + i]);
              t5_st16(tl + cb, o);
            }
            t5_wait_st();
          }
          fresh = fresh && oob;
        }
#pragma unroll
        for (int i = 0; i < 2 * J; i++) {
          const int e = 4 * (i >> 1) + (i & 1);
          x[e] = ex2(x[e]);
          x[e + 2] = ex2(x[e + 2]);
          l[i] += x[e] + x[e + 2];
        }
        // (the P buffer is free: the last MMAs of this S were issued behind the last P.V that read it)
        {
          const uint32_t pst = sm + C::SM_P + (j % C::NP) * (N * 128);
          const int blk = lane >> 3, half = blk & 1;   // lane's address: row lane % 8 of 8x8 block `blk`
          const uint32_t unit = 2 * quad + half;
#pragma unroll
          for (int jj = 0; jj < J; jj += 2) {
            const uint32_t row = grp * (N / SG) + 8 * (jj + (blk >> 1)) + (lane & 7);
            st_matrix4_t(pst + row * 128 + ((unit ^ (row & 7)) << 4), pack_bf2(x[4 * jj], x[4 * jj + 1]),
                         pack_bf2(x[4 * jj + 2], x[4 * jj + 3]), pack_bf2(x[4 * jj + 4], x[4 * jj + 5]),
                         pack_bf2(x[4 * jj + 6], x[4 * jj + 7]));
          }
        }
        // slots past the tile's last key may hold anything: their values must not meet P = 0
        // (MXFP8: the conversion wrote zeros there)
        if (!MX) {
          const int z = oob ? 0 : min(P, zero_from - t * P);
          if (z < P) {
            for (int i = tid; i < (P - z) * 64; i += 128 * SG) {
              const int slot = z + (i >> 6), u = i & 63;
              const uint32_t unit = (uint32_t)(4 * j + (u >> 4)) % C::NPAIR;
              st_shared16(sm + C::SM_PAIR + unit * 16384 + ((u >> 3) & 1) * 8192 + slot * 128 + (u & 7) * 16,
                          make_uint4(0u, 0u, 0u, 0u));
            }
          }
        }
        fence_async_smem();
        t5_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(BAR(C::B_P_FULL + j % C::NP));
      }
      if (timed_out) break;
      // ---- the part's output
      if (vote4(bad || !mbar_wait_warp(BAR(C::B_PV_DONE + ((j - 1) & 1)), ((j - 1) >> 1) & 1))) {
        timed_out = true;
        break;
      }
      t5_fence_after();
#pragma unroll
      for (int i = 0; i < 2 * J; i++) {
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) l[i] += __shfl_xor_sync(0xFFFFFFFFu, l[i], o);
        if (lane < 4) red[quad * N + 8 * (i >> 1) + c0 + (i & 1)] = l[i];
      }
      sync4();
      const bool whole = p.t0 == 0 && p.t1 == p.tiles;
      const int64_t slot = (int64_t)(w + (p.t0 == 0 ? g.W : 0)) * g.T + rt;
      if (whole) {
        if (tid < N) {
          const int r = tid;
          const float s = (red[r] + red[N + r]) + (red[2 * N + r] + red[3 * N + r]);
          fac[r] = s > 0.f ? 1.0f / s : 0.f;
        }
      } else if (quad == 0 && lane < 4) {
        float2* ml = reinterpret_cast<float2*>(a.ws + (int64_t)2 * g.W * g.T * N * LAT) + slot * N;
#pragma unroll
        for (int i = 0; i < 2 * J; i++) {
          const int r = 8 * (i >> 1) + c0 + (i & 1);
          const float s = (red[r] + red[N + r]) + (red[2 * N + r] + red[3 * N + r]);
          ml[r] = make_float2(s > 0.f ? m[i] : LA_LOW, s);
        }
      }
      sync4();
      if (whole && tid < N) {
        const int gr = r0 + tid, qi = gr / a.heads;
        rowoff[tid] =
            gr < p.rows ? (int64_t)(p.row0 + qi) * a.out.row + (int64_t)(gr - qi * a.heads) * a.out.head : INT64_MIN;
      }
      sync4();
#pragma unroll 2
      for (int cb = grp * (4 * N / SG); cb < (grp + 1) * (4 * N / SG); cb += 8) {
        uint32_t o[8];
        t5_ld8(tl + cb, o);
        const int rb = cb & (N - 1), d = (cb / N) * 128 + 32 * quad + lane;
        if (whole) {
          // (all of shared memory that the 8 rows' stores need is read before the first store)
          int64_t ro[4];
          float f[8];
#pragma unroll
          for (int i = 0; i < 8; i++) f[i] = fac[rb + i];
#pragma unroll
          for (int i = 0; i < 4; i++) ro[i] = rowoff[rb + 2 * i + (lane & 1)];
          t5_wait_ld();
          t5_ready(o);
          // neighbouring lanes hold neighbouring dims: they swap so that each stores a pair of dims of one
          // row, even lanes row i, odd lanes row i + 1
          uint32_t w2[4];
#pragma unroll
          for (int i = 0; i < 8; i += 2) {
            const float v0 = __uint_as_float(o[i]) * f[i], v1 = __uint_as_float(o[i + 1]) * f[i + 1];
            const float got = __shfl_xor_sync(0xFFFFFFFFu, (lane & 1) ? v0 : v1, 1);
            w2[i >> 1] = (lane & 1) ? pack_bf2(got, v1) : pack_bf2(v0, got);
          }
#pragma unroll
          for (int i = 0; i < 4; i++)
            if (ro[i] != INT64_MIN) *reinterpret_cast<uint32_t*>(a.out.p + ro[i] + (d & ~1)) = w2[i];
        } else {
          t5_wait_ld();
          t5_ready(o);
          // partials [row][dim]: a warp's store is 128 contiguous bytes of one row
          float* dst = a.ws + (slot * N + rb) * LAT + d;
#pragma unroll
          for (int i = 0; i < 8; i++) dst[i * LAT] = __uint_as_float(o[i]);
        }
      }
      t5_fence_before();   // O is read: the next part's first P.V comes after the P barrier
    }
  } else if (warp == 4) {
    // ================================================================= MMA issue
    // The whole warp runs the loop and one elected lane issues: in warp-uniform code, with
    // descriptors that are a base plus constants, an MMA costs its tensor cycles (M 64, N 64: 32;
    // M 128, N 64: 48, the rate of shared memory); from a one-lane branch each took ~150 to issue.
    // The order is fixed: the scores of tile j up to pair AHEAD, P.V of tile j - 1, the rest of the
    // scores.  The softmax of tile j - 1 hides behind the first pairs, and P.V frees its pages
    // before the scores wait for the next ones, so a ring of AHEAD + 4 pairs cannot lock up.
    constexpr uint32_t ID_S = t5_idesc(64, N, false, false), ID_PV = t5_idesc(128, N, true, false);
    constexpr uint32_t AHEAD = C::AHEAD, ALL = 0xFFFFFFFFu;
    static_assert((AHEAD == 2 || AHEAD == 4) && C::NPAIR >= 4 + AHEAD && C::NPAIR <= 12, "ring");
    const uint32_t one = t5_elect();
    const uint32_t d_pair = t5_desc(sm + C::SM_PAIR), d_pair_mn = t5_desc(sm + C::SM_PAIR, 8192),
                   d_rope = t5_desc(sm + C::SM_ROPE), d_q = t5_desc(sm + C::SM_Q), d_p = t5_desc(sm + C::SM_P);
    // (polled by the elected lane and voted on: no branch in which the warp diverges)
    auto wait = [&](uint32_t bar, uint32_t parity) {
      for (uint32_t n = 0; n < (1u << 22); n++) {
        if (mbar_try_warp(one, bar, parity)) return true;
        if ((n & 255u) == 255u && __any_sync(ALL, *abort_flag != 0)) return false;
      }
      return false;
    };
    uint32_t j = 0, part = 0;                    // score tiles begun, parts begun
    uint32_t s_slot = 0, v_slot = 0;             // next pair of the scores and of P.V
    uint32_t stage = 0, round = 0;               // j % 3, (j / 3) & 1
    uint32_t keep = 0;                           // 0: the tile whose P.V is next begins a part
    bool ok = true;
    auto pv = [&](uint32_t jp) {
      ok = wait(BAR(C::B_P_FULL + jp % C::NP), (jp / C::NP) & 1);
      if (!ok) return;
      t5_fence_after();
      const uint32_t pb = d_p + (jp % C::NP) * (N * (128 >> 4));
#pragma unroll
      for (uint32_t mb = 0; mb < 4; mb++) {
        const uint32_t v = d_pair_mn + v_slot * (16384 >> 4);
#pragma unroll
        for (int ks = 0; ks < 4; ks++)
          t5_mma_ss_if(one, tmem + mb * N, v + ks * (2048 >> 4), pb + ks * (32 >> 4), ID_PV, ks > 0 ? 1u : keep);
        t5_commit_if(one, BAR(C::B_PAIR_EMPTY) + 8 * v_slot);
        v_slot = v_slot + 1 == C::NPAIR ? 0 : v_slot + 1;
      }
      t5_commit_if(one, BAR(C::B_PV_DONE + (jp & 1)));
    };
    while (ok && __any_sync(ALL, it.template next<N>(a, rt, p))) {
      const uint32_t n = __shfl_sync(ALL, p.t1 - p.t0, 0);
      for (uint32_t i = 0; ok && __any_sync(ALL, i < n); i++, j++) {
        if (i == 0) {          // new queries: P.V of the last part first, it does not wait for them
          if (j > 0) pv(j - 1);
          ok = ok && wait(BAR(C::B_Q_FULL), part & 1);
        }
        const uint32_t d = tmem + TM_S + (j & 1) * N;
        ok = ok && wait(BAR(C::B_FULL) + 8 * stage, round);
        if (!ok) break;
        {
          const uint32_t k = d_rope + (j % C::NROPE) * (8192 >> 4), q = d_q + 8 * N * (128 >> 4);
#pragma unroll
          for (int ks = 0; ks < 4; ks++) t5_mma_ss_if(one, d, k + ks * 2, q + ks * 2, ID_S, ks > 0 ? 1u : 0u);
          t5_commit_if(one, BAR(C::B_ROPE_EMPTY + j % C::NROPE));
        }
#pragma unroll
        for (uint32_t us = 0; us < 4; us++) {
          if (us == 2) {
            if (AHEAD == 2 && i > 0) pv(j - 1);
            ok = ok && wait(BAR(C::B_FULL + 3) + 8 * stage, round);
            if (!ok) break;
          }
          const uint32_t k = d_pair + s_slot * (16384 >> 4), q = d_q + us * (2 * N * (128 >> 4));
#pragma unroll
          for (int ks = 0; ks < 8; ks++)
            t5_mma_ss_if(one, d, k + (ks >> 2) * (8192 >> 4) + (ks & 3) * 2, q + (ks >> 2) * (N * (128 >> 4)) + (ks & 3) * 2,
                         ID_S, 1u);
          s_slot = s_slot + 1 == C::NPAIR ? 0 : s_slot + 1;
        }
        if (!ok) break;
        t5_commit_if(one, BAR(C::B_S_FULL + (j & 1)));
        if (AHEAD == 4 && i > 0) pv(j - 1);
        keep = i == 0 ? 0u : 1u;   // (after P.V of the tile before used it)
        if (++stage == 3) {
          stage = 0;
          round ^= 1;
        }
      }
      if (ok) t5_commit_if(one, BAR(C::B_Q_EMPTY));   // the part's scores are issued: its queries may go
      part++;
    }
    if (ok && j > 0) pv(j - 1);
    if (!ok) {
      timed_out = true;
      *abort_flag = 1;
    }
    t5_commit_if(one, BAR(C::B_END));   // every MMA issued must be complete before the tensor memory goes, also where
    mbar_wait(BAR(C::B_END), 0);        // the softmax gave up on them
    __syncwarp();
  } else if (warp == 5) {
    // ================================================================= bulk copies
    // Lanes 0-3 bring the tile's pairs of chunks (MXFP8: the converting warps load the codes), lane 4 the
    // rotary chunk, each as soon as its own slot is free.
    uint32_t j = 0, issued = 0;              // tiles, and those this lane has copied its part of
    while (!timed_out && it.template next<N>(a, rt, p)) {
      const int64_t pt = (int64_t)p.b * a.c.max_pages;
      int32_t ids = 0;
      for (int t = p.t0; t < p.t1 && !timed_out; t++, j++) {
        const int k = (t - p.t0) & 31;
        if (k == 0) ids = t + lane < p.t1 ? a.c.page_table[pt + t + lane] : 0;
        int32_t phys = __shfl_sync(0xFFFFFFFFu, ids, k);
        if (phys < 0 || phys >= a.c.pool_pages) {   // masked by the softmax; any page will do
          if (lane == 0) flag(a.c.status, KVQ_STATUS_PAGE_OOB);
          phys = 0;
        }
        const uint8_t* blk = a.c.pool + (int64_t)phys * a.c.page_bytes + a.c.layer_off;
        // copy number, ring and its barriers of this lane
        const uint32_t u = lane < 4 ? 4 * j + lane : j, ring = lane < 4 ? C::NPAIR : C::NROPE, slot = u % ring, par = (u / ring) & 1;
        const uint32_t full = BAR(C::B_FULL + j % 3 + (lane == 2 || lane == 3 ? 3 : 0)),
                       empty = BAR((lane < 4 ? C::B_PAIR_EMPTY : C::B_ROPE_EMPTY) + slot);
        const uint32_t bytes = lane < 4 ? 16384 : 8192, dst = sm + (lane < 4 ? C::SM_PAIR : C::SM_ROPE) + slot * bytes;
        const uint8_t* src = blk + (lane < 4 ? lane * 16384 : MX ? LMX_CODES : 8 * LCHUNK);
        bool done = lane > 4 || (MX && lane < 4);
        for (uint32_t n = 0; n < (1u << 22); n++) {
          if (!done && mbar_test(empty, par ^ 1)) {
            mbar_expect(full, bytes);
            bulk_load(dst, src, bytes, full);
            done = true;
            issued = j + 1;
          }
          if (__all_sync(0xFFFFFFFFu, done)) break;
          if ((n & 255u) == 255u && __any_sync(0xFFFFFFFFu, *abort_flag != 0)) break;
        }
        timed_out = !__all_sync(0xFFFFFFFFu, done);
        if (lane == 0) *reinterpret_cast<volatile int*>(smem + C::SM_PROG) = j + 1;
      }
    }
    // Copies in flight must land before the CTA ends, also where another role gave up after the last one was issued: the
    // lane's last few.  (None of these phases can be two behind: the next one lacks this lane's arrival.)
    if (timed_out) *abort_flag = 1;
    for (uint32_t i = issued > 3 ? issued - 3 : 0; i < issued; i++)
      mbar_wait(BAR(C::B_FULL + i % 3 + (lane == 2 || lane == 3 ? 3 : 0)), (i / 3) & 1);
    __syncwarp();
  } else if (warp < 8) {
    // ================================================================= queries
    int part = 0, done = 0;
    while (!timed_out && it.template next<N>(a, rt, p)) {
      // (a part may be long: many bounded waits, until the CTA gives up)
      bool ok = false;
      for (int i = 0; i < 64 && !ok && __all_sync(0xFFFFFFFFu, *abort_flag == 0); i++)
        ok = mbar_wait_warp(BAR(C::B_Q_EMPTY), (part & 1) ^ 1);
      if (!ok) {
        timed_out = true;
        break;
      }
      // a row is 72 units of 16 B, copied by a warp; rows past the lane's are zeros.  Lane i holds the addresses
      // of the warp's row i: computed in turn for each row they would cost more instructions than the copies.
      const int mine = min(rt * N + (warp - 6) + 2 * min(lane, N / 2 - 1), p.rows - 1), qi = mine / a.heads, h = mine - qi * a.heads;
      const int64_t row = p.row0 + qi;
      const uint64_t ql = reinterpret_cast<uint64_t>(a.ql.p + row * a.ql.row + h * a.ql.head),
                     qr = reinterpret_cast<uint64_t>(a.qr.p + row * a.qr.row + h * a.qr.head);
      uint32_t dst = sm + C::SM_Q + (lane >> 3) * (N * 128) + (warp - 6) * 128;
#pragma unroll 4
      for (int i = 0; i < N / 2; i++, dst += 256) {
        const int r = (warp - 6) + 2 * i;
        const uint32_t bytes = rt * N + r < p.rows ? 16 : 0;
        const uint4* l = reinterpret_cast<const uint4*>(__shfl_sync(0xFFFFFFFFu, ql, i));
        const uint4* o = reinterpret_cast<const uint4*>(__shfl_sync(0xFFFFFFFFu, qr, i));
        const uint32_t at = dst + (((lane & 7) ^ (r & 7)) << 4);
        cp_async16(at, l + lane, bytes);
        cp_async16(at + 4 * (N * 128), l + lane + 32, bytes);
        if (lane < 8) cp_async16(at + 8 * (N * 128), o + lane, bytes);
      }
      cp_async_wait_all();
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(BAR(C::B_Q_FULL));
      part++;
      // While the part runs: where row tiles share its pages, these go to L2 a few tiles ahead of the copies
      // (the ring holds less than the memory's latency).
      if (!MX && LA_PREFETCH && g.T > 1) {
        const int32_t* table = a.c.page_table + (int64_t)p.b * a.c.max_pages;
        int32_t ids = 0;
        for (int t = p.t0; t < p.t1; t++, done++) {
          if (((t - p.t0) & 31) == 0) ids = t + lane < p.t1 ? table[t + lane] : -1;
          const int32_t phys = __shfl_sync(0xFFFFFFFFu, ids, (t - p.t0) & 31);
          int at = 0;
          for (int i = 0; i < (1 << 18); i++) {
            at = *reinterpret_cast<volatile int*>(smem + C::SM_PROG);
            if (__all_sync(0xFFFFFFFFu, at + LA_PREFETCH > done || *abort_flag)) break;
            __nanosleep(100);
          }
          if (phys >= 0 && phys < a.c.pool_pages && at < done && (t % g.T) == rt) {
            const uint8_t* blk = a.c.pool + (int64_t)phys * a.c.page_bytes + a.c.layer_off + (threadIdx.x - 192) * 128;
#pragma unroll
            for (int i = 0; i < LBF16_BLOCK / 8192; i++)
              asm volatile("prefetch.global.L2 [%0];\n" ::"l"(blk + i * 8192) : "memory");
          }
          __syncwarp();
        }
      }
    }
  } else {
    // ================================================================= MXFP8: codes -> bf16 tile
    // Two warps a pair of chunks (pair mb = 0 .. 3 of every tile), so that the four pairs' waits, loads and
    // stores overlap.  The codes go from memory to registers, which leaves the shared memory to the bf16 ring: a
    // run's registers take the next tile's codes as soon as they are converted (8 x 40,960 x 16 heads: 58 us, 67
    // with the loads behind the tile).  Two pages further on the codes are fetched to L2.
    const int mb = (warp - 8) >> 1, tid = threadIdx.x & 63, seg = tid & 3, slot0 = tid >> 2;
    const uint32_t my = mb * 8192 + slot0 * 64 + seg * 16;   // this thread's first run of 16 codes in a block
    uint4 q[8];
    uint32_t sc[4];
    uint32_t j = 0;
    while (!timed_out && it.template next<N>(a, rt, p)) {
      const int zero_from = p.pos0 + min(p.nq - 1, (rt * N + N - 1) / a.heads) + 1;
      const int32_t* table = a.c.page_table + (int64_t)p.b * a.c.max_pages;
      int32_t ids = 0;
      // page id of tile t (the lanes hold 32 of them), -1 if it is outside the pool
      auto page = [&](int t) {
        const int32_t phys = __shfl_sync(0xFFFFFFFFu, ids, (t - p.t0) & 31);
        return phys >= 0 && phys < a.c.pool_pages ? phys : -1;
      };
      auto block = [&](int32_t phys) { return a.c.pool + (int64_t)max(phys, 0) * a.c.page_bytes + a.c.layer_off; };
      auto codes = [&](const uint8_t* blk, int i) { return ld_global16(blk + my + (i >> 2) * 4096 + (i & 3) * 1024); };
      auto scales = [&](const uint8_t* blk, int k) { return ld_global4(blk + LMX_SCALES + (slot0 + 16 * k) * 16 + 4 * mb); };
      // the codes of the pair and two of the page's eight lines of scales, to L2: a lane a 128 B line
      auto prefetch = [&](int32_t at) {
        const uint8_t* blk = a.c.pool + (int64_t)at * a.c.page_bytes + a.c.layer_off;
        if ((tid & 7) == 0) {
#pragma unroll
          for (int i = 0; i < 8; i++)
            asm volatile("prefetch.global.L2 [%0];\n" ::"l"(blk + my + (i >> 2) * 4096 + (i & 3) * 1024) : "memory");
        } else if (tid < 3) {
          asm volatile("prefetch.global.L2 [%0];\n" ::"l"(blk + LMX_SCALES + (2 * mb + tid - 1) * 128) : "memory");
        }
      };
      ids = p.t0 + lane < p.t1 ? table[p.t0 + lane] : 0;
      int32_t phys = page(p.t0);
      for (int k = 1; k < 3; k++) {
        const int32_t soon = page(p.t0 + k);
        if (p.t0 + k < p.t1 && soon >= 0) prefetch(soon);
      }
      {
        const uint8_t* blk = block(phys);
#pragma unroll
        for (int i = 0; i < 8; i++) q[i] = codes(blk, i);
#pragma unroll
        for (int k = 0; k < 4; k++) sc[k] = scales(blk, k);
      }
      for (int t = p.t0; t < p.t1 && !timed_out; t++, j++) {
        const int z = phys < 0 ? 0 : min(P, zero_from - t * P);
        const uint32_t u = 4 * j + mb, ps = u % C::NPAIR, dst = sm + C::SM_PAIR + ps * 16384;
        if (__any_sync(0xFFFFFFFFu, *abort_flag != 0) || !mbar_wait_warp(BAR(C::B_PAIR_EMPTY + ps), ((u / C::NPAIR) & 1) ^ 1)) {
          timed_out = true;
          break;
        }
        const bool more = t + 1 < p.t1;
        if (more && ((t + 1 - p.t0) & 31) == 0) ids = t + 1 + lane < p.t1 ? table[t + 1 + lane] : 0;
        phys = page(t + 1);
        const uint8_t* next = block(phys);
#pragma unroll
        for (int i = 0; i < 8; i++) {
          const int slot = slot0 + 16 * (i & 3);
          const uint32_t f2 = mx_factor(__byte_perm(sc[i & 3], 0u, 0x4440u + 2 * (i >> 2) + (seg >> 1)));
          const uint2 d0 = mx_quad(q[i].x, f2), d1 = mx_quad(q[i].y, f2), d2 = mx_quad(q[i].z, f2), d3 = mx_quad(q[i].w, f2);
          st_shared16(dst + (i >> 2) * 8192 + chunk_unit(slot, 2 * seg), make_uint4(d0.x, d0.y, d1.x, d1.y));
          st_shared16(dst + (i >> 2) * 8192 + chunk_unit(slot, 2 * seg + 1), make_uint4(d2.x, d2.y, d3.x, d3.y));
          if (more) {
            q[i] = codes(next, i);
            if (i >= 4) sc[i & 3] = scales(next, i & 3);
          }
        }
        if (z < P) {       // zeros past the last key (this thread's own stores, overwritten)
#pragma unroll
          for (int i = 0; i < 8; i++) {
            const int slot = slot0 + 16 * (i & 3);
            if (slot >= z) {
              st_shared16(dst + (i >> 2) * 8192 + chunk_unit(slot, 2 * seg), make_uint4(0u, 0u, 0u, 0u));
              st_shared16(dst + (i >> 2) * 8192 + chunk_unit(slot, 2 * seg + 1), make_uint4(0u, 0u, 0u, 0u));
            }
          }
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(BAR(C::B_FULL + j % 3 + (mb >= 2 ? 3 : 0)));
        if (more) {
          const int32_t soon = page(t + 3);
          if (t + 3 < p.t1 && ((t + 1 - p.t0) & 31) < 30 && soon >= 0) prefetch(soon);
        }
      }
    }
  }
  if (timed_out) {
    *abort_flag = 1;
    if (lane == 0) flag(a.c.status, KVQ_STATUS_TIMEOUT);
  }
  t5_fence_before();
  __syncthreads();
  if (warp == 4) {
    t5_fence_after();
    t5_dealloc(tmem, C::TMEM_COLS);
  }
}

// Merges the parts of the lanes that cross a range border.  Block: a row of a row tile of a lane (or half of its
// dims), then further ones; warp: every eighth part, so that a lane of ten parts costs two round trips to
// L2 (the maxima and sums, then the rows).  With many rows, lanes of few parts take a warp a row, which leaves
// fewer blocks (32 lanes x 4,000 tokens x 64 heads: 59.8 -> 54.8 us for the whole call).  blockIdx.y is
// the lane, or, where there are more lanes than borders, a border, whose block takes the lane that the border
// is the first one inside of.
constexpr int LC_THREADS = 256;
constexpr int LC_ALONE = 16;         // lanes of at most so many parts: a warp a row, where there are many rows
template <int N, int Z>
__global__ void __launch_bounds__(LC_THREADS, Z == 1 ? 3 : 2) latent_attn_combine(LatentAttnArgs a, LaGrid g, int by_lane,
                                                                       int many_rows) {
  constexpr int D = LAT / 4 / Z, Q = D / 32;      // float4 of a block's share of a row, and of a lane's
  __shared__ float4 acc[LC_THREADS / 32][D];
  const int z = blockIdx.x % Z, x = blockIdx.x / Z, rt = x % g.T, r_first = x / g.T, r_step = gridDim.x / Z / g.T;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  latent_wait();
  const int* meta = la_meta(a, g, N);
  const int R = meta[0];
  int b = blockIdx.y;
  if (!by_lane) {   // the last lane that begins before the border
    const int64_t edge = (int64_t)(blockIdx.y + 1) * R;
    int lo = 0, hi = a.c.lanes;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (meta[1 + mid] < edge) lo = mid;
      else hi = mid;
    }
    b = lo;
  }
  const int at = meta[1 + b], r0 = rt * N;
  int nq, row0, pos0;
  if (!latent_lane(a, b, nq, row0, pos0, false)) return;
  const int rows = nq * a.heads, first = at / R;
  if (r0 >= rows || (!by_lane && first != (int)blockIdx.y)) return;   // (the lane's first border takes it)
  const int tiles = (pos0 + min(nq - 1, (r0 + N - 1) / a.heads) + P) / P;
  const int parts = (at + tiles - 1) / R - first + 1;
  if (parts < 2) return;                                              // finished by its only part
  auto slot = [&](int s) { return (int64_t)((s == 0 ? g.W : s) + first); };   // of the lane's part s
  const float2* ml = reinterpret_cast<const float2*>(a.ws + (int64_t)2 * g.W * g.T * N * LAT);
  static_assert(Z == 1 || Z == 2, "a lane's share of a row is 4 float4 or 2");
  constexpr int WARPS = LC_THREADS / 32, PER = (LA_SMS + 31) / 32;   // parts a lane of the warp weighs
  const int64_t step = (int64_t)g.T * N * LAT / 4;                   // from a part to the next, in float4
  const bool alone = Z == 1 && many_rows && parts <= LC_ALONE;
  const int s0 = alone ? 0 : warp, s_step = alone ? 1 : WARPS;
  for (int rb = alone ? r_first * WARPS : r_first; rb < N && r0 + rb < rows; rb += alone ? r_step * WARPS : r_step) {
    const int r = alone ? rb + warp : rb;
    if (r >= N || r0 + r >= rows) break;               // (alone: no barrier follows)
    const float4* src = reinterpret_cast<const float4*>(a.ws + ((int64_t)rt * N + r) * LAT) + z * D + lane;
    float2 e[PER];
    float mx = -INFINITY;
#pragma unroll
    for (int k = 0; k < PER; k++) {
      const int s = 32 * k + lane;
      e[k] = s < parts ? ml[(slot(s) * g.T + rt) * N + r] : make_float2(-INFINITY, 0.f);
      mx = fmaxf(mx, e[k].x);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, o));
    float den = 0.f;
#pragma unroll
    for (int k = 0; k < PER; k++) {
      e[k].x = e[k].x == -INFINITY ? 0.f : ex2(e[k].x - mx);         // the part's weight
      den = fmaf(e[k].y, e[k].x, den);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) den += __shfl_xor_sync(0xFFFFFFFFu, den, o);
    float4 sum[Q];
#pragma unroll
    for (int q = 0; q < Q; q++) sum[q] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (Z > 1) {                                       // ten of the warp's parts at once
      constexpr int B = 2 * PER;
#pragma unroll
      for (int half = 0; half < 2; half++) {
        if (half * B * WARPS >= parts) break;
        float4 o[B][Q];
#pragma unroll
        for (int i = 0; i < B; i++) {
          const int s = warp + WARPS * (half * B + i);
#pragma unroll
          for (int q = 0; q < Q; q++) o[i][q] = s < parts ? src[slot(s) * step + 32 * q] : make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll
        for (int i = 0; i < B; i++) {
          const float f = __shfl_sync(0xFFFFFFFFu, e[(half * B + i) >> 2].x, warp + WARPS * ((half * B + i) & 3));
#pragma unroll
          for (int q = 0; q < Q; q++) {
            sum[q].x = fmaf(o[i][q].x, f, sum[q].x);
            sum[q].y = fmaf(o[i][q].y, f, sum[q].y);
            sum[q].z = fmaf(o[i][q].z, f, sum[q].z);
            sum[q].w = fmaf(o[i][q].w, f, sum[q].w);
          }
        }
      }
    }
#pragma unroll
    for (int k = 0; Z == 1 && k < PER; k++) {
#pragma unroll 4
      for (int i = s0; i < 32 && 32 * k + i < parts; i += s_step) {
        const float f = __shfl_sync(0xFFFFFFFFu, e[k].x, i);
#pragma unroll
        for (int q = 0; q < Q; q++) {
          const float4 o = src[slot(32 * k + i) * step + 32 * q];
          sum[q].x = fmaf(o.x, f, sum[q].x);
          sum[q].y = fmaf(o.y, f, sum[q].y);
          sum[q].z = fmaf(o.z, f, sum[q].z);
          sum[q].w = fmaf(o.w, f, sum[q].w);
        }
      }
    }
    const float inv = den > 0.f ? 1.0f / den : 0.f;
    const int gr = r0 + r, qi = gr / a.heads;
    uint2* dst = reinterpret_cast<uint2*>(a.out.p + (int64_t)(row0 + qi) * a.out.row + (int64_t)(gr - qi * a.heads) * a.out.head) + z * D;
    if (alone) {
#pragma unroll
      for (int q = 0; q < Q; q++)
        dst[32 * q + lane] = make_uint2(pack_bf2(sum[q].x * inv, sum[q].y * inv), pack_bf2(sum[q].z * inv, sum[q].w * inv));
      continue;
    }
#pragma unroll
    for (int q = 0; q < Q; q++) acc[warp][32 * q + lane] = sum[q];
    __syncthreads();
    const int live = min(WARPS, parts);
    if (threadIdx.x < D) {
      float4 o = acc[0][threadIdx.x];
      for (int k = 1; k < live; k++) {
        const float4 x = acc[k][threadIdx.x];
        o.x += x.x;
        o.y += x.y;
        o.z += x.z;
        o.w += x.w;
      }
      dst[threadIdx.x] = make_uint2(pack_bf2(o.x * inv, o.y * inv), pack_bf2(o.z * inv, o.w * inv));
    }
    __syncthreads();
  }
}

template <int FMT, int N>
static int launch_la(const LatentAttnArgs& a, const LaGrid& g, cudaStream_t stream) {
  using C = LaCfg<FMT, N>;
  const int64_t blocks = (int64_t)g.T * (g.W > 0 ? g.W : a.c.lanes);
  if (blocks > INT32_MAX) return KVQ_ERR_UNSUPPORTED;
  if (cudaFuncSetAttribute(latent_attn_tc<FMT, N>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM) != cudaSuccess)
    return KVQ_ERR_CUDA;
  const int rc = latent_launch(latent_attn_tc<FMT, N>, dim3((unsigned)blocks), C::THREADS, C::SMEM, stream, a, g);
  if (rc || g.W < 2) return rc;
  const int by_lane = a.c.lanes < g.W, count = by_lane ? a.c.lanes : g.W - 1;
  // Few rows: half of a row's dims a block, so that more SMs read the parts of a long lane (131,072 + 8 x 4,096 tokens
  // of 16 heads: 45.4 -> 41.3 us), as long as all blocks run at once.  Many: groups of rows, about eight blocks an SM.
  const int64_t rows = (int64_t)g.T * count * N;
  const int groups = (int)std::min<int64_t>(N, std::max<int64_t>(1, 8 * LA_SMS / ((int64_t)g.T * count)));
  const bool few = rows <= LA_SMS;
  const int many = rows >= LA_SMS * 6;
  const dim3 grid((unsigned)(g.T * groups * (few ? 2 : 1)), (unsigned)count);
  return few ? latent_launch(latent_attn_combine<N, 2>, grid, LC_THREADS, 0, stream, a, g, by_lane, many)
             : latent_launch(latent_attn_combine<N, 1>, grid, LC_THREADS, 0, stream, a, g, by_lane, many);
}

int launch_latent_attn(int fmt, const LatentAttnArgs& a, cudaStream_t stream) {
  const LaGrid g = la_grid(a.heads, a.max_n_q, a.max_seq_len);
  const int N = la_rows(a.heads, a.max_n_q);
  if (fmt == KVQ_LATENT_BF16)
    return N == 16 ? launch_la<KVQ_LATENT_BF16, 16>(a, g, stream)
           : N == 32 ? launch_la<KVQ_LATENT_BF16, 32>(a, g, stream)
                     : launch_la<KVQ_LATENT_BF16, 64>(a, g, stream);
  return N == 16 ? launch_la<KVQ_LATENT_MXFP8, 16>(a, g, stream)
         : N == 32 ? launch_la<KVQ_LATENT_MXFP8, 32>(a, g, stream)
                   : launch_la<KVQ_LATENT_MXFP8, 64>(a, g, stream);
}

}  // namespace kvq
