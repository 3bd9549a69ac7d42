// latent_prefill.cu -- causal attention of the expanded form on the tcgen05 tensor cores.
//
//   out[row][h] = sum_t softmax_t(scale (q_n . k_n[t][h] + q_r . k_r[t])) v[t][h],  128 + 64 and 128 dims
//
// 640 FLOP a (query, key, head) against a few bytes: the bound is the tensor cores, and beside them
// the exponentials (128 a row and tile).  CTA: one head, 256 queries as two tiles A and B of 128 rows
// that share every key tile of 128 keys and take turns: while the softmax works on one tile's scores
// the tensor pipe runs the other tile's products, so neither waits for the other.
//   TMEM: S_A, S_B (128 columns each, P in bf16 over the first 64), O_A, O_B (128 each).
//   Shared memory: Q (3 chunks of [256 rows][64 dims]), a ring of 8 units [128 keys][64 dims]; a key
//   tile is 5 units: k_nope x 2, k_rope, v x 2, all 128-byte swizzled; K is the K-major B of S = Q K^T,
//   V the N-major B of O += P V, P the A operand from tensor memory.
// Warps: 0-3 softmax of A (a row a thread), 4-7 of B, 8 MMA issue, 9 copies (TMA boxes of 64 dims).
// A box may run past the keys that the lane's queries attend, into rows of another lane: the softmax masks the
// scores and, in the lane's last tile, writes zeros over those value rows before their products.
// The softmax's reference maximum moves only when a row's maximum passes it by more than 2^8; l is
// summed in FP32 from the unrounded weights, P is bf16 (the type of V): half a bf16 step a weight, as much as the
// output's own rounding (with it the error against 64 bits is 1.8e-3 to 2.3e-3 of the output's norm, 1.5e-3 to 1.7e-3 of which
// a P in 32 bits has too).  P as two bf16 terms would double the products of P.V.
// Few rows over long keys are split along the keys: FP32 partials, merged by latent_prefill_combine.
// Measured, inputs changing from call to call: 4,096 x 128 heads 515 us (1.33 PFLOP/s, 70% of the matrix-product rate),
// 1,024 x 32 heads after 15,000 tokens 229 us (1.42 PFLOP/s).  With the same inputs again and again 480 to 500 (the power
// limit decides) and 214.  While a CTA's tiles run
// the tensor pipe is full; the rest is a CTA's start (2.5 us until the first 224 KB have come), its first
// softmax and its end.
// Every wait is bounded; on a timeout the CTA flags KVQ_STATUS_TIMEOUT and ends.
#include "latent.cuh"
#include "tcgen05.cuh"

#include <cuda.h>

#include <algorithm>

namespace kvq {

constexpr int LP_KEYS = 128;                     // keys of a tile
constexpr int LP_ROWS = 256;                     // queries of a CTA
constexpr int LP_UNIT = LP_KEYS * 128;           // 16,384 B: [128 keys][64 dims]
constexpr int LP_RING = 8;
constexpr int LP_THREADS = 10 * 32;
constexpr int LP_SM_Q = 0;
constexpr int LP_SM_RING = 3 * LP_ROWS * 128;
constexpr int LP_SM_BAR = LP_SM_RING + LP_RING * LP_UNIT;
enum { LPB_FULL = 0, LPB_EMPTY = LP_RING, LPB_Q = 2 * LP_RING, LPB_S, LPB_P = LPB_S + 2, LPB_O = LPB_P + 2, LPB_END = LPB_O + 2, LPB_N };
constexpr int LP_SM_TMEM = LP_SM_BAR + 8 * LPB_N;
constexpr int LP_SMEM = LP_SM_TMEM + 16 + 1024;  // + slack to align the base to 1,024 B
static_assert(LP_SMEM <= 232448, "shared memory of a CTA");
constexpr float LP_SLACK = 8.0f, LP_LOW = -3e38f;
constexpr int LP_SPLIT_TILES = 8, LP_TAIL_TILES = 12, LP_CTA_TILES = 5;   // key tiles of a split, at least (see lp_split)
constexpr int LP_SMS = 152;

__device__ __forceinline__ uint64_t pack_f2(float a, float b) {
  uint64_t p;
  asm("mov.b64 %0, {%1, %2};\n" : "=l"(p) : "f"(a), "f"(b));
  return p;
}
__device__ __forceinline__ void unpack_f2(uint64_t p, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;\n" : "=f"(a), "=f"(b) : "l"(p));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;\n" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;\n" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// Tensor maps of the inputs, [row][head][dim] with boxes of 64 dims of one head of 128 or 256 rows; *_h is 0
// where the heads share the rows (head stride 0: a map of one head), else 1.
struct LpMaps {
  CUtensorMap qn, qr, kn, kr, v;
  int qn_h, qr_h, kn_h, v_h;
};

__device__ __forceinline__ void tma_rows(uint32_t dst, const CUtensorMap* map, int dim, int head, int row, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];\n" ::"r"(dst),
      "l"(map), "r"(dim), "r"(head), "r"(row), "r"(bar)
      : "memory");
}

struct LpSplit {
  int splits, tiles;   // splits of a row's keys; key tiles of one
};

// Order of the CTAs: groups of heads; within a group the longest rows (the last ones) of all its heads first, so
// that the last CTAs of a call are short ones.  A group's keys and values stay in L2 while its rows read them.
struct LpOrder {
  int rows, heads;     // row tiles of a lane, heads of a group
};
constexpr int64_t LP_GROUP_BYTES = 64 << 20;

static LpOrder lp_order(int heads, int max_n_q, int max_n_k) {
  const int64_t fit = std::max<int64_t>(1, LP_GROUP_BYTES / ((int64_t)std::max(max_n_k, 1) * (NOPE + VDIM) * 2));
  const int groups = (int)((heads + fit - 1) / fit);
  return LpOrder{(max_n_q - 1) / LP_ROWS + 1, (heads + groups - 1) / groups};
}

static LpSplit lp_split(int lanes, int heads, int max_n_q, int max_n_k) {
  const int64_t ctas = (int64_t)lanes * heads * ((max_n_q + LP_ROWS - 1) / LP_ROWS);
  const int tiles = (max_n_k + LP_KEYS - 1) / LP_KEYS;
  LpSplit s{1, std::max(1, tiles)};
  if (ctas <= 0 || ctas >= LP_SMS) return s;
  if (2 * ctas <= LP_SMS) {          // even splits, a CTA an SM
    if (tiles < 2 * LP_SPLIT_TILES) return s;
    const int64_t want = LP_SMS / ctas;
    s.tiles = (int)std::max<int64_t>(LP_SPLIT_TILES, (tiles + want - 1) / want);
    s.splits = (tiles + s.tiles - 1) / s.tiles;
    return s;
  }
  // One CTA on most SMs: the last x tiles of each go to the SMs that are left, `each` CTAs an SM one after
  // another, so that both end together; a CTA's start and end cost as much as LP_CTA_TILES tiles.  Only
  // behind a prefix that all rows attend, and only for enough tiles to pay for the merge (32 heads x 1,024
  // queries after 15,000 tokens: 220 -> 211 us, after 60,000 804 -> 729; 25 heads 218 -> 164).
  const int left = LP_SMS - (int)ctas, each = ((int)ctas + left - 1) / left;
  const int x = (tiles + LP_CTA_TILES - each * LP_CTA_TILES) / (each + 1);
  if (x >= LP_TAIL_TILES && (max_n_k - max_n_q) / LP_KEYS >= tiles - x) s = LpSplit{2, tiles - x};
  return s;
}

// Partials lie by (lane, query, head, split), so that their bytes follow from the arguments that decide the split.
__host__ __device__ static int64_t lp_partials(const LatentPrefillArgs& a) { return (int64_t)a.lanes * a.max_n_q * a.heads; }   // of a split
static size_t lp_bytes(int64_t partials) { return (size_t)partials * (VDIM + 2) * sizeof(float) + 256; }

// Bytes that this very call touches, and a bound of them for it and every smaller one.  No fewer than
// 2 LP_SPLIT_TILES key tiles are split (LP_TAIL_TILES are more than half of such), into LP_SPLIT_TILES each at least; and
// splits x CTAs are at most the SMs, or 2 for each of fewer CTAs than SMs, of LP_ROWS rows each.
size_t latent_prefill_needs(int lanes, int heads, int max_n_q, int max_n_k) {
  const LpSplit s = lp_split(lanes, heads, max_n_q, max_n_k);
  return s.splits == 1 ? 256 : lp_bytes((int64_t)lanes * max_n_q * heads * s.splits);
}

size_t latent_prefill_workspace(int lanes, int heads, int max_n_q, int max_n_k) {
  const int tiles = (max_n_k + LP_KEYS - 1) / LP_KEYS;
  static_assert(2 * LP_TAIL_TILES >= 2 * LP_SPLIT_TILES, "tails only of as many tiles");
  if (tiles < 2 * LP_SPLIT_TILES) return 256;
  const int64_t most = (int64_t)2 * LP_SMS * LP_ROWS, splits = std::min(LP_SMS, (tiles + LP_SPLIT_TILES - 1) / LP_SPLIT_TILES);
  return lp_bytes(std::min(most, std::min(most, (int64_t)heads * max_n_q) * std::min<int64_t>(most, lanes) * splits));
}

// grid: (row tiles x heads, lanes, splits)
__global__ void __launch_bounds__(LP_THREADS, 1) latent_prefill_tc(LatentPrefillArgs a, LpSplit sp, LpOrder od,
                                                                 const __grid_constant__ LpMaps maps) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t sm = smem_u32(smem);
  const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + LP_SM_TMEM + 4);
  auto BAR = [&](int i) { return sm + LP_SM_BAR + 8u * i; };
  if (warp == 9) {   // (the warp that copies: its first copies need no other warp)
    if (lane < LPB_N) mbar_init(BAR(lane), lane >= LPB_P && lane < LPB_O ? 4 : 1);
    if (lane == 0) *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    if (lane < 5) {
      const CUtensorMap* map = lane == 0 ? &maps.qn : lane == 1 ? &maps.qr : lane == 2 ? &maps.kn : lane == 3 ? &maps.kr : &maps.v;
      asm volatile("prefetch.tensormap [%0];\n" ::"l"(map) : "memory");
    }
    __syncwarp();
  }
  const int s = blockIdx.z, group = blockIdx.x / (od.heads * od.rows), left = blockIdx.x - group * od.heads * od.rows;
  const int in_group = min(od.heads, a.heads - group * od.heads), rt = left / in_group;
  const int b = blockIdx.y, h = group * od.heads + left - rt * in_group, q0 = LP_ROWS * (od.rows - 1 - rt);
  latent_wait();
  int nq, row0, pos0, nk, key0;
  if (!latent_prefill_lane(a, b, nq, row0, pos0, nk, key0, blockIdx.x == 0 && s == 0 && threadIdx.x == 0) || q0 >= nq) return;
  // key tiles [j0, end of A) and [j0, end of B)
  const int j0 = s * sp.tiles;
  const int endA = min(j0 + sp.tiles, (pos0 + min(nq, q0 + 128) - 1) / LP_KEYS + 1);
  const int endB = q0 + 128 < nq ? min(j0 + sp.tiles, (pos0 + min(nq, q0 + 256) - 1) / LP_KEYS + 1) : j0;
  const int nA = max(0, endA - j0), nB = max(0, endB - j0), n = max(nA, nB);   // (nA <= nB, or B has no rows)
  if (n == 0) return;

  bool timed_out = false;
  int u = 0;             // copies: units issued
  auto copy_unit = [&] {
    const int k = u / 5, c = u - 5 * k, slot = u % LP_RING, row = key0 + (j0 + k) * LP_KEYS;
    if (*abort_flag || !mbar_wait(BAR(LPB_EMPTY + slot), ((u / LP_RING) & 1) ^ 1)) {
      timed_out = true;
      return;
    }
    const uint32_t dst = sm + LP_SM_RING + slot * LP_UNIT, full = BAR(LPB_FULL + slot);
    mbar_expect(full, LP_UNIT);
    if (c < 2) tma_rows(dst, &maps.kn, 64 * c, h * maps.kn_h, row, full);
    else if (c == 2) tma_rows(dst, &maps.kr, 0, 0, row, full);
    else tma_rows(dst, &maps.v, 64 * (c - 3), h * maps.v_h, row, full);
    u++;
  };
  if (warp == 9 && lane == 0) {
    mbar_expect(BAR(LPB_Q), 3 * LP_ROWS * 128);
    for (int c = 0; c < 3; c++)
      tma_rows(sm + LP_SM_Q + c * LP_ROWS * 128, c < 2 ? &maps.qn : &maps.qr, c < 2 ? 64 * c : 0,
               c < 2 ? h * maps.qn_h : h * maps.qr_h, row0 + q0, BAR(LPB_Q));
    while (u < min(LP_RING, 5 * n) && !timed_out) copy_unit();   // (the ring is empty: no wait)
  }
  if (warp == 8) t5_alloc(sm + LP_SM_TMEM, 512);
  t5_fence_before();
  __syncthreads();
  t5_fence_after();
  const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, *reinterpret_cast<volatile uint32_t*>(smem + LP_SM_TMEM), 0);

  if (warp < 8) {
    // ================================================================= softmax and output
    const int x = warp >> 2;                                 // tile A or B
    const int qi = q0 + 128 * x + 32 * (warp & 3) + lane;    // this thread's row
    const bool live = qi < nq;
    const int pos = pos0 + qi, mine = x ? nB : nA;
    const uint32_t tl = tmem + ((uint32_t)(32 * (warp & 3)) << 16), ts = tl + 128 * x, to = tl + 256 + 128 * x;
    float m = LP_LOW, l = 0.f;
    for (int k = 0; k < mine; k++) {
      if (__any_sync(0xFFFFFFFFu, *abort_flag != 0) || !mbar_wait_warp(BAR(LPB_S + x), k & 1)) { timed_out = true; break; }
      t5_fence_after();
      const int kt = (j0 + k) * LP_KEYS;
      // keys of the tile that this row attends (rows past the last query: none)
      const int lim = live ? pos - kt : -1;
      const bool all = __all_sync(0xFFFFFFFFu, lim >= LP_KEYS - 1);
      // One pass with the reference so far: the scores come 32 columns at a time, the next ones while
      // these are worked on, and P stays in registers until it is known that no score passed the
      // reference by more than the slack.  Else (and for the first tile) the reference moves first.
      uint32_t p[4][16];
      uint64_t sum[4];
      float over = INFINITY;
      auto weights = [&](bool masked) {
        uint32_t r[2][32];
        float o4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        const uint64_t sc2 = pack_f2(a.scale_log2, a.scale_log2), nm2 = pack_f2(-m, -m);
#pragma unroll
        for (int i = 0; i < 4; i++) sum[i] = 0ull;
        t5_ld32(ts, r[0]);
        t5_wait_ld();
        t5_ready(r[0]);
#pragma unroll
        for (int c = 0; c < 4; c++) {
          if (c < 3) t5_ld32(ts + 32 * (c + 1), r[(c + 1) & 1]);
#pragma unroll
          for (int i = 0; i < 16; i++) {
            float d0, d1;
            unpack_f2(fma2(pack_f2(__uint_as_float(r[c & 1][2 * i]), __uint_as_float(r[c & 1][2 * i + 1])), sc2, nm2), d0, d1);
            if (masked) {
              d0 = 32 * c + 2 * i <= lim ? d0 : -INFINITY;
              d1 = 32 * c + 2 * i + 1 <= lim ? d1 : -INFINITY;
            }
            o4[i & 3] = max3(o4[i & 3], d0, d1);
            const float e0 = ex2(d0), e1 = ex2(d1);
            sum[i & 3] = add2(sum[i & 3], pack_f2(e0, e1));
            p[c][i] = pack_bf2(e0, e1);
          }
          if (c < 3) {
            t5_wait_ld();
            t5_ready(r[(c + 1) & 1]);
          }
        }
        over = fmaxf(fmaxf(o4[0], o4[1]), fmaxf(o4[2], o4[3]));
      };
      if (k > 0) {
        if (all) weights(false);
        else weights(true);
      }
      if (__any_sync(0xFFFFFFFFu, over > LP_SLACK)) {
        float mx = -INFINITY;
#pragma unroll 1
        for (int c = 0; c < 4; c++) {
          uint32_t r[32];
          t5_ld32(ts + 32 * c, r);
          t5_wait_ld();
          t5_ready(r);
#pragma unroll
          for (int i = 0; i < 32; i++) mx = fmaxf(mx, 32 * c + i <= lim ? __uint_as_float(r[i]) : -INFINITY);
        }
        mx = mx == -INFINITY ? mx : mx * a.scale_log2;
        const bool up = mx > m + LP_SLACK;
        const float alpha = up ? ex2(m - mx) : 1.0f;   // (from the first reference: 2^-huge = 0)
        if (up) m = mx;
        l *= alpha;
        if (k > 0) {                                   // (O is stable: these scores came after the P.V before)
#pragma unroll 1
          for (int c = 0; c < 4; c++) {
            uint32_t o[32];
            t5_ld32(to + 32 * c, o);
            t5_wait_ld();
            t5_ready(o);
#pragma unroll
            for (int i = 0; i < 32; i++) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
            t5_st32(to + 32 * c, o);
          }
        }
        if (all) weights(false);
        else weights(true);
      }
#pragma unroll
      for (int c = 0; c < 4; c++) t5_st16(ts + 16 * c, p[c]);
      {
        float q[8];
#pragma unroll
        for (int i = 0; i < 4; i++) unpack_f2(sum[i], q[2 * i], q[2 * i + 1]);
        l += ((q[0] + q[1]) + (q[2] + q[3])) + ((q[4] + q[5]) + (q[6] + q[7]));
      }
      if (kt + LP_KEYS > pos0 + nq) {   // value rows past the lane's last query may hold anything, and 0 times that
        bool landed = true;
        for (int c = 3; c < 5; c++) {
          const int u = 5 * k + c;
          landed = mbar_wait_warp(BAR(LPB_FULL + u % LP_RING), (u / LP_RING) & 1) && landed;
        }
        if (!landed) { timed_out = true; break; }
        const int z = pos0 + nq - kt;
        for (int i = threadIdx.x & 127; i < (LP_KEYS - z) * 16; i += 128) {
          const int slot = (5 * k + 3 + ((i >> 3) & 1)) % LP_RING;
          st_shared16(sm + LP_SM_RING + slot * LP_UNIT + (z + (i >> 4)) * 128 + (i & 7) * 16, make_uint4(0u, 0u, 0u, 0u));
        }
        fence_async_smem();
      }
      t5_wait_st();
      t5_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(BAR(LPB_P + x));
    }
    if (!timed_out && mine > 0) {
      if (!mbar_wait_warp(BAR(LPB_O + x), 0)) timed_out = true;
    }
    if (!timed_out && mine > 0) {
      t5_fence_after();
      // A thread holds a row; stored from there, every 16 B of a warp would go to another row.  The rows go through
      // the warp's own rows of Q in shared memory (its tile's scores are complete) and out 128 B at a time.
      const int w0 = q0 + 128 * x + 32 * (warp & 3);          // the warp's first row
      const float inv = l > 0.f ? 1.0f / l : 0.f;
      const bool whole = sp.splits == 1;
      const int64_t part = (((int64_t)b * a.max_n_q + qi) * a.heads + h) * sp.splits + s;
      auto out_rows = [&](int c, const uint32_t (&v)[32], uint8_t* base, int64_t row_bytes) {
        const uint32_t mine = sm + LP_SM_Q + (c & 1) * (LP_ROWS * 128) + (128 * x + 32 * (warp & 3)) * 128;
#pragma unroll
        for (int i = 0; i < 8; i++)
          st_shared16(mine + lane * 128 + ((i ^ (lane & 7)) << 4), make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]));
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 8; i++) {
          const int r = 4 * i + (lane >> 3), e = lane & 7;
          const uint4 t = ld_shared16(mine + r * 128 + ((e ^ (r & 7)) << 4));
          if (w0 + r < nq) *reinterpret_cast<uint4*>(base + r * row_bytes + 16 * e) = t;
        }
        __syncwarp();
      };
      if (whole) {
        uint8_t* base = reinterpret_cast<uint8_t*>(a.out.p + (int64_t)(row0 + w0) * a.out.row + h * a.out.head);
#pragma unroll 1
        for (int c = 0; c < 2; c++) {
          uint32_t o[2][32], v[32];
          t5_ld32(to + 64 * c, o[0]);
          t5_ld32(to + 64 * c + 32, o[1]);
          t5_wait_ld();
          t5_ready(o[0]);
          t5_ready(o[1]);
#pragma unroll
          for (int i = 0; i < 32; i++)
            v[i] = pack_bf2(__uint_as_float(o[i >> 4][2 * (i & 15)]) * inv, __uint_as_float(o[i >> 4][2 * (i & 15) + 1]) * inv);
          out_rows(c, v, base + 128 * c, a.out.row * 2);
        }
      } else {
        const int64_t per_row = (int64_t)a.heads * sp.splits;   // parts from a row to the next
        uint8_t* base = reinterpret_cast<uint8_t*>(a.ws + ((((int64_t)b * a.max_n_q + w0) * a.heads + h) * sp.splits + s) * VDIM);
#pragma unroll 1
        for (int c = 0; c < 4; c++) {
          uint32_t o[32];
          t5_ld32(to + 32 * c, o);
          t5_wait_ld();
          t5_ready(o);
          out_rows(c, o, base + 128 * c, per_row * VDIM * 4);
        }
        if (live)
          reinterpret_cast<float2*>(a.ws + lp_partials(a) * sp.splits * VDIM)[part] = make_float2(m, l);
      }
    }
  } else if (warp == 8) {
    // ================================================================= MMA issue (an elected lane of a uniform warp)
    constexpr uint32_t ID_S = t5_idesc(128, 128, false, false), ID_PV = t5_idesc(128, VDIM, false, true),
                       ID_PV64 = t5_idesc(128, 64, false, true), ALL = 0xFFFFFFFFu;
    const uint32_t one = t5_elect();
    const uint32_t d_q = t5_desc(sm + LP_SM_Q), d_ring = t5_desc(sm + LP_SM_RING), d_ring_n = t5_desc(sm + LP_SM_RING, LP_UNIT);
    auto wait = [&](uint32_t bar, uint32_t parity) {
      for (uint32_t i = 0; i < (1u << 22); i++) {
        if (mbar_try_warp(one, bar, parity)) return true;
        if ((i & 255u) == 255u && __any_sync(ALL, *abort_flag != 0)) return false;
      }
      return false;
    };
    // (votes make the conditions uniform to the compiler: a branch in which this warp diverged would mix up
    // the descriptors of its halves, which share the uniform registers)
    auto is = [&](bool c) { return __any_sync(ALL, c) != 0; };
    // S of row tile x against key tile k; the keys' units may go after the last of their two uses
    auto scores = [&](uint32_t x, uint32_t k, bool last) {
#pragma unroll
      for (uint32_t c = 0; c < 3; c++) {
        const uint32_t u = 5 * k + c, slot = u % LP_RING;
        if (!wait(BAR(LPB_FULL + slot), (u / LP_RING) & 1)) return false;
        const uint32_t q = d_q + (c * LP_ROWS + x * 128) * (128 >> 4), kd = d_ring + slot * (LP_UNIT >> 4);
#pragma unroll
        for (int ks = 0; ks < 4; ks++) t5_mma_ss_if(one, tmem + 128 * x, q + 2 * ks, kd + 2 * ks, ID_S, c > 0 || ks > 0 ? 1u : 0u);
      }
      t5_commit_if(one, BAR(LPB_S + x));
      if (last) {
#pragma unroll
        for (uint32_t c = 0; c < 3; c++) t5_commit_if(one, BAR(LPB_EMPTY + (5 * k + c) % LP_RING));
      }
      return true;
    };
    auto products = [&](uint32_t x, uint32_t k, bool last, bool end) {
      if (!wait(BAR(LPB_P + x), k & 1)) return false;
      t5_fence_after();
      const uint32_t u = 5 * k + 3, s0 = u % LP_RING, s1 = (u + 1) % LP_RING;
      if (!wait(BAR(LPB_FULL + s0), (u / LP_RING) & 1) || !wait(BAR(LPB_FULL + s1), ((u + 1) / LP_RING) & 1)) return false;
      const uint32_t o = tmem + 256 + 128 * x, p = tmem + 128 * x, v = d_ring_n + s0 * (LP_UNIT >> 4);
      if (is(s1 > s0)) {   // the value units lie side by side
#pragma unroll
        for (int ks = 0; ks < 8; ks++) t5_mma_ts_if(one, o, p + 8 * ks, v + ks * (2048 >> 4), ID_PV, k > 0 || ks > 0 ? 1u : 0u);
      } else {             // the second one is the ring's first: 64 dims at a time
#pragma unroll
        for (int ks = 0; ks < 8; ks++) t5_mma_ts_if(one, o, p + 8 * ks, v + ks * (2048 >> 4), ID_PV64, k > 0 || ks > 0 ? 1u : 0u);
#pragma unroll
        for (int ks = 0; ks < 8; ks++)
          t5_mma_ts_if(one, o + 64, p + 8 * ks, d_ring_n + ks * (2048 >> 4), ID_PV64, k > 0 || ks > 0 ? 1u : 0u);
      }
      if (last) {
#pragma unroll
        for (uint32_t c = 0; c < 2; c++) t5_commit_if(one, BAR(LPB_EMPTY + (5 * k + 3 + c) % LP_RING));
      }
      if (end) t5_commit_if(one, BAR(LPB_O + x));
      return true;
    };
    const uint32_t na = nA, nb = nB, nn = n;
    const bool a0 = is(na > 0), b0 = is(nb > 0);
    bool ok = wait(BAR(LPB_Q), 0);
    if (ok && a0) ok = scores(0, 0, !b0);
    if (ok && b0) ok = scores(1, 0, true);
    for (uint32_t k = 0; ok && is(k < nn); k++) {
      const bool pa = is(k < na), sa = is(k + 1 < na), pb = is(k < nb), sb = is(k + 1 < nb);
      if (pa) ok = products(0, k, !pb, !sa);
      if (ok && sa) ok = scores(0, k + 1, !sb);
      if (ok && pb) ok = products(1, k, true, !sb);
      if (ok && sb) ok = scores(1, k + 1, true);
    }
    if (!ok) {
      timed_out = true;
      *abort_flag = 1;
    }
    t5_commit_if(one, BAR(LPB_END));   // every MMA issued must be complete before the tensor memory goes, also where
    mbar_wait(BAR(LPB_END), 0);        // the softmax gave up on them
    __syncwarp();
  } else {
    // ================================================================= copies
    if (lane == 0) {
      while (u < 5 * n && !timed_out) copy_unit();
      // copies in flight must land before the CTA ends, also where another role gave up after the last one was issued
      if (timed_out) *abort_flag = 1;
      mbar_wait(BAR(LPB_Q), 0);
      for (int i = max(0, u - LP_RING); i < u; i++) mbar_wait(BAR(LPB_FULL + i % LP_RING), (i / LP_RING) & 1);
    }
    timed_out = __shfl_sync(0xFFFFFFFFu, timed_out, 0);
  }
  if (timed_out) {
    *abort_flag = 1;
    if (lane == 0) flag(a.status, KVQ_STATUS_TIMEOUT);
  }
  t5_fence_before();
  __syncthreads();
  if (warp == 8) {
    t5_fence_after();
    t5_dealloc(tmem, 512);
  }
}

// Merges the splits of a (row, head): a warp each, 4 dims a lane.  grid: (ceil(max_n_q * heads / 8), lanes)
__global__ void __launch_bounds__(256) latent_prefill_combine(LatentPrefillArgs a, LpSplit sp) {
  int nq, row0, pos0, nk, key0;
  latent_wait();
  const bool ok = latent_prefill_lane(a, blockIdx.y, nq, row0, pos0, nk, key0, false);
  const int64_t item = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int qi = (int)(item / a.heads), h = (int)(item % a.heads), lane = threadIdx.x & 31;
  if (!ok || qi >= nq) return;
  const int parts = (pos0 + qi) / LP_KEYS / sp.tiles + 1;
  const int64_t part = (((int64_t)blockIdx.y * a.max_n_q + qi) * a.heads + h) * sp.splits;
  const float2* ml = reinterpret_cast<const float2*>(a.ws + lp_partials(a) * sp.splits * VDIM) + part;
  const float4* o = reinterpret_cast<const float4*>(a.ws + part * VDIM) + lane;
  float mx = -INFINITY, den = 0.f;
  for (int s = 0; s < parts; s++) mx = fmaxf(mx, ml[s].x);
  float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int s = 0; s < parts; s++) {
    const float2 e = ml[s];
    const float4 v = o[s * (VDIM / 4)];
    const float f = ex2(e.x - mx);
    den = fmaf(e.y, f, den);
    sum.x = fmaf(v.x, f, sum.x);
    sum.y = fmaf(v.y, f, sum.y);
    sum.z = fmaf(v.z, f, sum.z);
    sum.w = fmaf(v.w, f, sum.w);
  }
  const float inv = den > 0.f ? 1.0f / den : 0.f;
  uint2* dst = reinterpret_cast<uint2*>(a.out.p + (int64_t)(row0 + qi) * a.out.row + h * a.out.head);
  dst[lane] = make_uint2(pack_bf2(sum.x * inv, sum.y * inv), pack_bf2(sum.z * inv, sum.w * inv));
}

// The same for two splits and many rows: a warp takes LP_PAIRS (row, head) one behind another, with all of their loads
// under way at once (32 heads x 1,024 rows after 15,000: whole call 214 -> 211 us).
constexpr int LP_PAIRS = 4;
__global__ void __launch_bounds__(256) latent_prefill_combine2(LatentPrefillArgs a, LpSplit sp) {
  int nq, row0, pos0, nk, key0;
  latent_wait();
  if (!latent_prefill_lane(a, blockIdx.y, nq, row0, pos0, nk, key0, false)) return;
  const int64_t first = ((int64_t)blockIdx.x * 8 + (threadIdx.x >> 5)) * LP_PAIRS, items = (int64_t)nq * a.heads;
  const int lane = threadIdx.x & 31;
  const float4* o = reinterpret_cast<const float4*>(a.ws) + lane;
  const float4* ml = reinterpret_cast<const float4*>(a.ws + lp_partials(a) * 2 * VDIM);   // (m, l) of both
  float4 e[LP_PAIRS], v[LP_PAIRS][2];
#pragma unroll
  for (int k = 0; k < LP_PAIRS; k++) {
    if (first + k >= items) break;
    const int64_t at = (int64_t)blockIdx.y * a.max_n_q * a.heads + first + k;
    const bool two = pos0 + (int)((first + k) / a.heads) >= LP_KEYS * sp.tiles;   // does the row reach the second split?
    e[k] = ml[at];
    v[k][0] = o[at * (2 * VDIM / 4)];
    v[k][1] = two ? o[at * (2 * VDIM / 4) + VDIM / 4] : make_float4(0.f, 0.f, 0.f, 0.f);
    if (!two) {
      e[k].z = -INFINITY;
      e[k].w = 0.f;
    }
  }
#pragma unroll
  for (int k = 0; k < LP_PAIRS; k++) {
    if (first + k >= items) break;
    const float mx = fmaxf(e[k].x, e[k].z), f0 = ex2(e[k].x - mx), f1 = ex2(e[k].z - mx);
    const float den = fmaf(e[k].w, f1, e[k].y * f0), inv = den > 0.f ? 1.0f / den : 0.f;
    const float4 x = v[k][0], y = v[k][1];
    const int qi = (int)((first + k) / a.heads), h = (int)((first + k) - (int64_t)qi * a.heads);
    uint2* dst = reinterpret_cast<uint2*>(a.out.p + (int64_t)(row0 + qi) * a.out.row + h * a.out.head);
    dst[lane] = make_uint2(pack_bf2(fmaf(y.x, f1, x.x * f0) * inv, fmaf(y.y, f1, x.y * f0) * inv),
                           pack_bf2(fmaf(y.z, f1, x.z * f0) * inv, fmaf(y.w, f1, x.w * f0) * inv));
  }
}

using EncodeTiled = decltype(&cuTensorMapEncodeTiled);

// the driver's encoder, through the runtime (the library does not link the driver); null without one
static EncodeTiled tensor_map_encoder() {
  static const EncodeTiled fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<EncodeTiled>(p);
  }();
  return fn;
}

static bool rows_map(CUtensorMap* map, int* by_head, const RowsView& r, int rows, int heads, int dims, int box_rows) {
  const EncodeTiled encode = tensor_map_encoder();
  *by_head = heads > 1 && r.head != 0;
  const cuuint64_t dim[3] = {(cuuint64_t)dims, (cuuint64_t)(*by_head ? heads : 1), (cuuint64_t)rows};
  const cuuint64_t stride[2] = {(cuuint64_t)(*by_head ? r.head : 64) * 2, (cuuint64_t)(rows > 1 ? r.row : 64) * 2};
  const cuuint32_t box[3] = {64, 1, (cuuint32_t)box_rows}, step[3] = {1, 1, 1};
  return encode && encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, r.p, dim, stride, box, step,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int launch_latent_prefill(const LatentPrefillArgs& a, cudaStream_t stream) {
  LpMaps maps;
  int kr_h;
  if (!rows_map(&maps.qn, &maps.qn_h, a.qn, a.n_q_rows, a.heads, NOPE, LP_ROWS) ||
      !rows_map(&maps.qr, &maps.qr_h, a.qr, a.n_q_rows, a.heads, LROPE, LP_ROWS) ||
      !rows_map(&maps.kn, &maps.kn_h, a.kn, a.n_k_rows, a.heads, NOPE, LP_KEYS) ||
      !rows_map(&maps.kr, &kr_h, a.kr, a.n_k_rows, 1, LROPE, LP_KEYS) ||
      !rows_map(&maps.v, &maps.v_h, a.v, a.n_k_rows, a.heads, VDIM, LP_KEYS))
    return KVQ_ERR_UNSUPPORTED;
  const LpSplit sp = lp_split(a.lanes, a.heads, a.max_n_q, a.max_n_k);
  if (cudaFuncSetAttribute(latent_prefill_tc, cudaFuncAttributeMaxDynamicSharedMemorySize, LP_SMEM) != cudaSuccess)
    return KVQ_ERR_CUDA;
  const LpOrder od = lp_order(a.heads, a.max_n_q, a.max_n_k);
  for (int b0 = 0; b0 < a.lanes; b0 += 65535) {   // gridDim.y limit
    LatentPrefillArgs c = a;
    c.lanes = std::min(a.lanes - b0, 65535);
    c.q_pos0 += b0;
    c.n_q += b0;
    c.q_offset += b0;
    c.n_k += b0;
    c.k_offset += b0;
    int rc = latent_launch(latent_prefill_tc, dim3((unsigned)(od.rows * a.heads), (unsigned)c.lanes, (unsigned)sp.splits),
                           LP_THREADS, LP_SMEM, stream, c, sp, od, maps);
    if (!rc && sp.splits == 2 && (int64_t)a.max_n_q * a.heads >= 2 * 64 * LP_SMS)   // (two waves of warps)
      rc = latent_launch(latent_prefill_combine2,
                         dim3((unsigned)(((int64_t)a.max_n_q * a.heads + 8 * LP_PAIRS - 1) / (8 * LP_PAIRS)), (unsigned)c.lanes),
                         256, 0, stream, c, sp);
    else if (!rc && sp.splits > 1)
      rc = latent_launch(latent_prefill_combine, dim3((unsigned)(((int64_t)a.max_n_q * a.heads + 7) / 8), (unsigned)c.lanes),
                         256, 0, stream, c, sp);
    if (rc) return rc;
  }
  return KVQ_OK;
}

}  // namespace kvq
