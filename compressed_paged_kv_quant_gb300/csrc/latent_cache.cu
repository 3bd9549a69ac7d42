// latent_cache.cu -- the latent cache: append (lay out / quantize) and read-back of tokens, and the
// host side (validation, sizes) of every latent-attention entry point.
//
// Append, per token: 512 latent dims and 64 rotary dims, bf16.  bf16 blocks store them as they
// are, swizzled; MXFP8 blocks store, for each 32 dims, e = the least integer with
// max|x| <= 448 * 2^e (in [-120, 7]) and E4M3(x * 2^-e).  With max|x| = 1.M * 2^(E - 127) in
// fp32, 448 = 1.75 * 2^8 gives e = E - 135, plus one if 1.M > 1.75: no logarithm, no rounding.
// The read is code * 2^e, exact in bf16.
//
// A warp takes one token; lane l holds dims 16l .. 16l + 15 (32 contiguous bytes), so a group's
// maximum is one shuffle away and a lane's codes are one 16 B store.  Both kernels are bound by
// HBM (1,152 + 1,152 or 656 B a token).  Measured: append of 65,536 tokens to MXFP8 20 us (5.9 TB/s), read of
// 307,000 tokens from MXFP8 86 us (6.2 TB/s, 91% of the copy bandwidth), a step of 32 tokens 2 us (launch).
#include "latent.cuh"

namespace kvq {

constexpr int LTOK_WARPS = 8;
constexpr int LTOK_FULL = 152 * 8;   // blocks that fill the SMs

// Page block and slot of position pos of lane b; null (after flagging) if it has none.
__device__ __forceinline__ uint8_t* latent_slot(const LatentView& c, int b, int64_t pos, int& slot, bool report) {
  const int64_t pi = pos / P;
  slot = (int)(pos % P);
  if (pi >= c.max_pages) {
    if (report) flag(c.status, KVQ_STATUS_LEN_GT_TABLE);
    return nullptr;
  }
  const int32_t phys = c.page_table[(int64_t)b * c.max_pages + pi];
  if (phys < 0 || phys >= c.pool_pages) {
    if (report) flag(c.status, KVQ_STATUS_PAGE_OOB);
    return nullptr;
  }
  return c.pool + (int64_t)phys * c.page_bytes + c.layer_off;
}

// Lane of this warp and its first token; false if the lane has none for it.  A warp takes TOK tokens,
// LTOK_WARPS apart.
template <int TOK>
__device__ __forceinline__ bool latent_tokens_of(const LatentTokenArgs& a, int per_lane, int& b, int& i, int& n,
                                                 int64_t& pos0, int64_t& row0) {
  latent_wait();
  b = blockIdx.x / per_lane;
  const int chunk = blockIdx.x - b * per_lane;
  i = chunk * (LTOK_WARPS * TOK) + (threadIdx.x >> 5);
  n = a.n_tok[b];
  const int off = a.tok_offset[b], start = a.start_pos[b];
  if (n < 0 || n > a.max_tok || (n > 0 && (off < 0 || (int64_t)off + n > a.n_rows || start < 0))) {
    if (chunk == 0 && threadIdx.x == 0) flag(a.c.status, KVQ_STATUS_BAD_LEN);
    return false;
  }
  pos0 = start;
  row0 = off;
  return i < n;
}

// Larger magnitudes of two pairs of bf16, as bits: without the sign they are in the order of the values, infinities
// and NaN last.
__device__ __forceinline__ uint32_t max_abs2(uint32_t a, uint32_t b) {
  uint32_t m;
  asm("max.u16x2 %0, %1, %2;\n" : "=r"(m) : "r"(a), "r"(b & 0x7FFF7FFFu));
  return m;
}

// One token's 16 latent dims of a lane (x0, x1) and, of lanes 0-7, 8 rotary dims (r) into its slot.
template <int FMT>
__device__ __forceinline__ void store_token(const LatentView& c, uint8_t* blk, int slot, uint4 x0, uint4 x1, uint4 r) {
  const int l = threadIdx.x & 31;
  const uint32_t w[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
  uint32_t most = 0, rope = 0;
#pragma unroll
  for (int k = 0; k < 8; k++) most = max_abs2(most, w[k]);
  rope = max_abs2(max_abs2(max_abs2(max_abs2(0, r.x), r.y), r.z), r.w);
  uint32_t amax = max(most & 0xFFFFu, most >> 16);
  // 0x4760: 57,344; 0x7F80: infinity
  const bool bad = (FMT == KVQ_LATENT_MXFP8 ? amax > 0x4760u : amax >= 0x7F80u) || max(rope & 0xFFFFu, rope >> 16) >= 0x7F80u;
  if (__any_sync(0xFFFFFFFFu, bad)) {
    if (l == 0) flag(c.status, KVQ_STATUS_BAD_INPUT);
    return;
  }
  if (!blk) return;
  if (FMT == KVQ_LATENT_BF16) {
    uint8_t* chunk = blk + (l >> 2) * LCHUNK;
    const int u = 2 * (l & 3);
    *reinterpret_cast<uint4*>(chunk + chunk_unit(slot, u)) = x0;
    *reinterpret_cast<uint4*>(chunk + chunk_unit(slot, u + 1)) = x1;
    if (l < 8) *reinterpret_cast<uint4*>(blk + (LNCHUNK - 1) * LCHUNK + chunk_unit(slot, l)) = r;
  } else {
    amax = max(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
    int e = (int)(amax >> 7) - 135 + ((amax & 0x7Fu) > 0x60u ? 1 : 0);
    e = min(7, max(-120, e));
    const float f = __uint_as_float((uint32_t)(127 - e) << 23);   // 2^-e
    uint32_t q[4];
#pragma unroll
    for (int k = 0; k < 4; k++) {
      const uint32_t u0 = w[2 * k], u1 = w[2 * k + 1];
      const uint32_t lo = (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(bf16_lo(u0) * f, bf16_hi(u0) * f),
                                                             __NV_SATFINITE, __NV_E4M3);
      const uint32_t hi = (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(bf16_lo(u1) * f, bf16_hi(u1) * f),
                                                             __NV_SATFINITE, __NV_E4M3);
      q[k] = lo | (hi << 16);
    }
    *reinterpret_cast<uint4*>(blk + (l >> 2) * 4096 + slot * 64 + (l & 3) * 16) = make_uint4(q[0], q[1], q[2], q[3]);
    if (l < 8) *reinterpret_cast<uint4*>(blk + LMX_CODES + chunk_unit(slot, l)) = r;
    // the 16 scale bytes (one in every even lane), four at a time
    uint32_t s = (uint32_t)(e + 127);
    s |= __shfl_down_sync(0xFFFFFFFFu, s, 2) << 8;
    s |= __shfl_down_sync(0xFFFFFFFFu, s, 4) << 16;
    if ((l & 7) == 0) *reinterpret_cast<uint32_t*>(blk + LMX_SCALES + slot * 16 + (l >> 1)) = s;
  }
}

template <int FMT>
__global__ void __launch_bounds__(32 * LTOK_WARPS) latent_append_kernel(LatentTokenArgs a, int per_lane) {
  int b, i, n, slot;
  int64_t pos0, row0;
  if (!latent_tokens_of<1>(a, per_lane, b, i, n, pos0, row0)) return;
  const int l = threadIdx.x & 31;
  const uint4* src = reinterpret_cast<const uint4*>(a.latent.p + (row0 + i) * a.latent.row) + 2 * l;
  const uint4 x0 = src[0], x1 = src[1];
  uint4 r = make_uint4(0u, 0u, 0u, 0u);
  if (l < 8) r = reinterpret_cast<const uint4*>(a.rope.p + (row0 + i) * a.rope.row)[l];
  uint8_t* blk = latent_slot(a.c, b, pos0 + i, slot, l == 0);
  store_token<FMT>(a.c, blk, slot, x0, x1, r);
}

template <int FMT, int TOK>
__global__ void __launch_bounds__(32 * LTOK_WARPS) latent_read_kernel(LatentTokenArgs a, int per_lane) {
  int b, i, n;
  int64_t pos0, row0;
  if (!latent_tokens_of<TOK>(a, per_lane, b, i, n, pos0, row0)) return;
  const int l = threadIdx.x & 31;
  uint4 x0[TOK], x1[TOK], r[TOK];       // MXFP8: the codes in x0, the scale byte in x1.x
  const uint8_t* blk[TOK];
  int slot[TOK];
#pragma unroll
  for (int k = 0; k < TOK; k++) {
    const int t = i + k * LTOK_WARPS;
    blk[k] = t < n ? latent_slot(a.c, b, pos0 + t, slot[k], l == 0) : nullptr;
  }
#pragma unroll
  for (int k = 0; k < TOK; k++) {
    if (!blk[k]) continue;
    if (FMT == KVQ_LATENT_BF16) {
      const uint8_t* chunk = blk[k] + (l >> 2) * LCHUNK;
      const int u = 2 * (l & 3);
      x0[k] = *reinterpret_cast<const uint4*>(chunk + chunk_unit(slot[k], u));
      x1[k] = *reinterpret_cast<const uint4*>(chunk + chunk_unit(slot[k], u + 1));
      if (l < 8) r[k] = *reinterpret_cast<const uint4*>(blk[k] + (LNCHUNK - 1) * LCHUNK + chunk_unit(slot[k], l));
    } else {
      x0[k] = *reinterpret_cast<const uint4*>(blk[k] + (l >> 2) * 4096 + slot[k] * 64 + (l & 3) * 16);
      x1[k].x = blk[k][LMX_SCALES + slot[k] * 16 + (l >> 1)];
      if (l < 8) r[k] = *reinterpret_cast<const uint4*>(blk[k] + LMX_CODES + chunk_unit(slot[k], l));
    }
  }
#pragma unroll
  for (int k = 0; k < TOK; k++) {
    if (!blk[k]) continue;
    if (FMT == KVQ_LATENT_MXFP8) {
      const uint4 q = x0[k];
      const uint32_t f2 = mx_factor(x1[k].x);
      const uint2 d0 = mx_quad(q.x, f2), d1 = mx_quad(q.y, f2), d2 = mx_quad(q.z, f2), d3 = mx_quad(q.w, f2);
      x0[k] = make_uint4(d0.x, d0.y, d1.x, d1.y);
      x1[k] = make_uint4(d2.x, d2.y, d3.x, d3.y);
    }
    const int64_t row = row0 + i + k * LTOK_WARPS;
    uint4* dst = reinterpret_cast<uint4*>(a.latent.p + row * a.latent.row) + 2 * l;
    dst[0] = x0[k];
    dst[1] = x1[k];
    if (l < 8) reinterpret_cast<uint4*>(a.rope.p + row * a.rope.row)[l] = r[k];
  }
}

// Blocks of a token kernel, per_lane a lane; more than a grid holds: -1.
static int64_t token_blocks(const LatentTokenArgs& a, int tok, int& per_lane) {
  per_lane = (a.max_tok - 1) / (LTOK_WARPS * tok) + 1;
  const int64_t n = (int64_t)per_lane * a.c.lanes;
  return n > INT32_MAX ? -1 : n;
}

template <int FMT>
static int launch_append(const LatentTokenArgs& a, cudaStream_t stream) {
  int per_lane;
  const int64_t n = token_blocks(a, 1, per_lane);
  if (n < 0) return KVQ_ERR_UNSUPPORTED;
  return latent_launch(latent_append_kernel<FMT>, dim3((unsigned)n), 32 * LTOK_WARPS, 0, stream, a, per_lane);
}

// Two tokens a warp once that fills the SMs (307,000 tokens: 95 us with one, 88 with two when that was chosen), else
// one (1,025 tokens: the same 3 us; half the warps would be idle).  The append is faster with one at every size
// (65,536 tokens: 24 us, 26 with two): its loads do not wait for the page table.
template <int FMT>
static int launch_read(const LatentTokenArgs& a, cudaStream_t stream) {
  int per_lane;
  int64_t n = token_blocks(a, 2, per_lane);
  if (n >= LTOK_FULL)
    return latent_launch(latent_read_kernel<FMT, 2>, dim3((unsigned)n), 32 * LTOK_WARPS, 0, stream, a, per_lane);
  if (n < 0 || (n = token_blocks(a, 1, per_lane)) < 0) return KVQ_ERR_UNSUPPORTED;
  return latent_launch(latent_read_kernel<FMT, 1>, dim3((unsigned)n), 32 * LTOK_WARPS, 0, stream, a, per_lane);
}

int launch_latent_append(int fmt, const LatentTokenArgs& a, cudaStream_t stream) {
  return fmt == KVQ_LATENT_BF16 ? launch_append<KVQ_LATENT_BF16>(a, stream) : launch_append<KVQ_LATENT_MXFP8>(a, stream);
}

int launch_latent_read(int fmt, const LatentTokenArgs& a, cudaStream_t stream) {
  return fmt == KVQ_LATENT_BF16 ? launch_read<KVQ_LATENT_BF16>(a, stream) : launch_read<KVQ_LATENT_MXFP8>(a, stream);
}

}  // namespace kvq

// ---------------------------------------------------------------------------- host side
using namespace kvq;

namespace {

constexpr float LOG2E = 1.4426950408889634f;

int check_latent_geom(const kvq_latent_geom* g) {
  if (!g) return KVQ_ERR_INVALID_ARG;
  if (g->format != KVQ_LATENT_BF16 && g->format != KVQ_LATENT_MXFP8) return KVQ_ERR_UNSUPPORTED;
  if (g->latent_dim != LAT || g->rope_dim != LROPE || g->page_tokens != P) return KVQ_ERR_UNSUPPORTED;
  if (g->num_layers <= 0 || g->num_q_heads <= 0) return KVQ_ERR_INVALID_ARG;
  if (g->num_layers > 4096 || g->num_q_heads > LMAX_HEADS) return KVQ_ERR_UNSUPPORTED;
  return KVQ_OK;
}

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

// bf16 rows: present, aligned, the strides that are used whole 16 B units
int check_rows(const kvq_rows* r, int rows, int heads) {
  if (!r || !r->ptr) return KVQ_ERR_INVALID_ARG;
  if (!aligned16(r->ptr) || (rows > 1 && r->row_stride % 8) || (heads > 1 && r->head_stride % 8)) return KVQ_ERR_ALIGNMENT;
  return KVQ_OK;
}

// Do two of the rows [row][head] of `dims` elements share an element?  Rows (r, h) and (r + i, h + k) are |i R - k H| apart
// (for strides of unlike sign it is the pair (r, h + k), (r + i, h)), so for each k the i nearest to k H / R decide.
bool rows_overlap(const kvq_rows* r, int rows, int heads, int dims) {
  using wide = __int128;
  const wide R = r->row_stride < 0 ? -(wide)r->row_stride : r->row_stride,
             H = r->head_stride < 0 ? -(wide)r->head_stride : r->head_stride;
  if (rows <= 1) return heads > 1 && H < dims;
  if (R < dims) return true;
  if (heads <= 1) return false;
  if (H < dims) return true;
  if (R >= (heads - 1) * H + dims || H >= (rows - 1) * R + dims) return false;   // one within the gaps of the other
  for (int k = 1; k < heads; k++) {
    const wide i = k * H / R < rows - 1 ? k * H / R : rows - 1, far = k * H - i * R;
    if (far < dims || (i + 1 < rows && R - far < dims)) return true;
  }
  return false;
}

// rows that are written: no two at one place
int check_out_rows(const kvq_rows* r, int rows, int heads, int dims) {
  const int rc = check_rows(r, rows, heads);
  if (rc) return rc;
  return rows_overlap(r, rows, heads, dims) ? KVQ_ERR_INVALID_ARG : KVQ_OK;
}

// rows that tensor maps describe: strides that go forward, below 2^40 bytes (0: heads that share the rows)
bool mappable(const kvq_rows* r, int rows, int heads) {
  const int64_t end = (int64_t)1 << 39;
  return (rows <= 1 || (r->row_stride > 0 && r->row_stride < end)) &&
         (heads <= 1 || (r->head_stride >= 0 && r->head_stride < end));
}

RowsView rows_view(const kvq_rows* r, int rows, int heads) {
  return RowsView{static_cast<__nv_bfloat16*>(r->ptr), rows > 1 ? r->row_stride : 0, heads > 1 ? r->head_stride : 0};
}

size_t latent_page_bytes(const kvq_latent_geom* g) { return (size_t)g->num_layers * latent_block(g->format); }

LatentView latent_view(const kvq_latent_geom* g, int layer, const void* pool, size_t pool_bytes,
                       const int32_t* page_table, int max_pages, int lanes, int32_t* status) {
  LatentView c;
  c.pool = static_cast<uint8_t*>(const_cast<void*>(pool));
  c.page_bytes = (int64_t)latent_page_bytes(g);
  c.pool_pages = (int64_t)(pool_bytes / (size_t)c.page_bytes);
  c.layer_off = (int64_t)layer * latent_block(g->format);
  c.page_table = page_table;
  c.max_pages = max_pages;
  c.lanes = lanes;
  c.status = status;
  return c;
}

int check_latent_cache(const kvq_latent_geom* g, int layer, int max_pages, int lanes) {
  const int rc = check_latent_geom(g);
  if (rc) return rc;
  if (layer < 0 || layer >= g->num_layers || lanes < 0 || max_pages < 0) return KVQ_ERR_INVALID_ARG;
  if ((int64_t)max_pages * P > (int64_t)INT32_MAX) return KVQ_ERR_INVALID_ARG;
  return KVQ_OK;
}

int latent_tokens(bool append, const kvq_latent_geom* g, int layer, const void* pool, size_t pool_bytes,
                  const int32_t* page_table, int max_pages, int lanes, const int32_t* start_pos, const int32_t* n_tok,
                  const int32_t* tok_offset, int max_tok, int n_rows, const kvq_rows* latent, const kvq_rows* rope,
                  int32_t* d_status, kvq_stream_t stream) {
  int rc = check_latent_cache(g, layer, max_pages, lanes);
  if (rc) return rc;
  if (max_tok < 0 || n_rows < 0) return KVQ_ERR_INVALID_ARG;
  if (lanes == 0 || max_tok == 0) return KVQ_OK;
  if (!pool || !page_table || !start_pos || !n_tok || !tok_offset || !d_status) return KVQ_ERR_INVALID_ARG;
  if (pool_bytes < latent_page_bytes(g)) return KVQ_ERR_INVALID_ARG;
  if (n_rows > 0) {
    rc = append ? check_rows(latent, n_rows, 1) : check_out_rows(latent, n_rows, 1, LAT);
    if (!rc) rc = append ? check_rows(rope, n_rows, 1) : check_out_rows(rope, n_rows, 1, LROPE);
    if (rc) return rc;
  }
  if (!latent || !rope) return KVQ_ERR_INVALID_ARG;
  if (!aligned16(pool)) return KVQ_ERR_ALIGNMENT;
  LatentTokenArgs a{};
  a.c = latent_view(g, layer, pool, pool_bytes, page_table, max_pages, lanes, d_status);
  a.start_pos = start_pos;
  a.n_tok = n_tok;
  a.tok_offset = tok_offset;
  a.max_tok = max_tok;
  a.n_rows = n_rows;
  a.latent = rows_view(latent, n_rows, 1);
  a.rope = rows_view(rope, n_rows, 1);
  return append ? launch_latent_append(g->format, a, (cudaStream_t)stream)
                : launch_latent_read(g->format, a, (cudaStream_t)stream);
}

}  // namespace

extern "C" {

size_t kvq_latent_page_bytes(const kvq_latent_geom* g) { return check_latent_geom(g) ? 0 : latent_page_bytes(g); }

size_t kvq_latent_token_bytes(const kvq_latent_geom* g) { return check_latent_geom(g) ? 0 : latent_page_bytes(g) / P; }

size_t kvq_latent_workspace_bytes(const kvq_latent_geom* g, int lanes, int max_n_q, int max_seq_len) {
  if (check_latent_geom(g) || lanes < 0 || max_n_q < 0 || max_seq_len < 0) return 0;
  if ((int64_t)g->num_q_heads * max_n_q > INT32_MAX) return 0;
  return latent_attn_workspace(g->num_q_heads, lanes, max_n_q, max_seq_len);
}

size_t kvq_latent_prefill_workspace_bytes(int lanes, int num_heads, int n_q_rows, int max_n_q, int max_n_k) {
  if (lanes < 0 || num_heads <= 0 || num_heads > LMAX_HEADS || n_q_rows < 0 || max_n_q < 0 || max_n_k < 0) return 0;
  if (max_n_q > LMAX_PREFILL || max_n_k > LMAX_PREFILL) return 0;
  return latent_prefill_workspace(lanes, num_heads, max_n_q, max_n_k);
}

int kvq_latent_append(const kvq_latent_geom* g, int layer, void* pool, size_t pool_bytes, const int32_t* page_table,
                      int max_pages, int lanes, const int32_t* start_pos, const int32_t* n_new,
                      const int32_t* tok_offset, int max_new, int n_rows, const kvq_rows* latent, const kvq_rows* rope,
                      int32_t* d_status, kvq_stream_t stream) {
  return latent_tokens(true, g, layer, pool, pool_bytes, page_table, max_pages, lanes, start_pos, n_new, tok_offset,
                       max_new, n_rows, latent, rope, d_status, stream);
}

int kvq_latent_read(const kvq_latent_geom* g, int layer, const void* pool, size_t pool_bytes,
                    const int32_t* page_table, int max_pages, int lanes, const int32_t* start_pos,
                    const int32_t* n_tok, const int32_t* tok_offset, int max_tok, int n_rows, const kvq_rows* latent,
                    const kvq_rows* rope, int32_t* d_status, kvq_stream_t stream) {
  return latent_tokens(false, g, layer, pool, pool_bytes, page_table, max_pages, lanes, start_pos, n_tok, tok_offset,
                       max_tok, n_rows, latent, rope, d_status, stream);
}

int kvq_paged_latent_attn(const kvq_latent_geom* g, int layer, const void* pool, size_t pool_bytes,
                          const int32_t* page_table, int max_pages, int lanes, const int32_t* q_pos0,
                          const int32_t* n_q, const int32_t* q_offset, int max_n_q, int n_q_rows,
                          const int32_t* seq_len, int max_seq_len, const kvq_rows* q_latent, const kvq_rows* q_rope,
                          float sm_scale, void* workspace, size_t ws_bytes, const kvq_rows* out, int32_t* d_status,
                          kvq_stream_t stream) {
  int rc = check_latent_cache(g, layer, max_pages, lanes);
  if (rc) return rc;
  if (max_n_q < 0 || n_q_rows < 0 || max_seq_len < 0) return KVQ_ERR_INVALID_ARG;
  if ((int64_t)max_seq_len > (int64_t)max_pages * P) return KVQ_ERR_INVALID_ARG;
  if (!(sm_scale >= 0.0f && sm_scale <= 1.0e38f)) return KVQ_ERR_INVALID_ARG;
  if ((int64_t)g->num_q_heads * max_n_q > INT32_MAX) return KVQ_ERR_UNSUPPORTED;
  if ((int64_t)lanes * (((int64_t)max_seq_len + P - 1) / P) > INT32_MAX) return KVQ_ERR_UNSUPPORTED;   // the page list
  if (lanes == 0 || max_n_q == 0 || n_q_rows == 0) return KVQ_OK;
  if (!pool || !page_table || !q_pos0 || !n_q || !q_offset || !seq_len || !workspace || !d_status)
    return KVQ_ERR_INVALID_ARG;
  if (pool_bytes < latent_page_bytes(g)) return KVQ_ERR_INVALID_ARG;
  if ((rc = check_rows(q_latent, n_q_rows, g->num_q_heads)) || (rc = check_rows(q_rope, n_q_rows, g->num_q_heads)) ||
      (rc = check_out_rows(out, n_q_rows, g->num_q_heads, LAT)))
    return rc;
  if (!aligned16(pool) || !aligned16(workspace)) return KVQ_ERR_ALIGNMENT;
  if (ws_bytes < latent_attn_needs(g->num_q_heads, lanes, max_n_q, max_seq_len)) return KVQ_ERR_WORKSPACE_TOO_SMALL;
  LatentAttnArgs a{};
  a.c = latent_view(g, layer, pool, pool_bytes, page_table, max_pages, lanes, d_status);
  a.q_pos0 = q_pos0;
  a.n_q = n_q;
  a.q_offset = q_offset;
  a.seq_len = seq_len;
  a.max_n_q = max_n_q;
  a.n_q_rows = n_q_rows;
  a.max_seq_len = max_seq_len;
  a.heads = g->num_q_heads;
  a.ql = rows_view(q_latent, n_q_rows, a.heads);
  a.qr = rows_view(q_rope, n_q_rows, a.heads);
  a.out = rows_view(out, n_q_rows, a.heads);
  a.scale_log2 = sm_scale * LOG2E;
  a.ws = static_cast<float*>(workspace);
  return launch_latent_attn(g->format, a, (cudaStream_t)stream);
}

int kvq_latent_prefill_attn(int num_heads, int lanes, const int32_t* q_pos0, const int32_t* n_q,
                            const int32_t* q_offset, int max_n_q, int n_q_rows, const int32_t* n_k,
                            const int32_t* k_offset, int max_n_k, int n_k_rows, const kvq_rows* q_nope,
                            const kvq_rows* q_rope, const kvq_rows* k_nope, const kvq_rows* k_rope, const kvq_rows* v,
                            float sm_scale, void* workspace, size_t ws_bytes, const kvq_rows* out, int32_t* d_status,
                            kvq_stream_t stream) {
  if (num_heads <= 0 || lanes < 0 || max_n_q < 0 || n_q_rows < 0 || max_n_k < 0 || n_k_rows < 0)
    return KVQ_ERR_INVALID_ARG;
  if (num_heads > LMAX_HEADS || max_n_q > LMAX_PREFILL || max_n_k > LMAX_PREFILL) return KVQ_ERR_UNSUPPORTED;
  if (!(sm_scale >= 0.0f && sm_scale <= 1.0e38f)) return KVQ_ERR_INVALID_ARG;
  if (lanes == 0 || max_n_q == 0 || n_q_rows == 0) return KVQ_OK;
  if (!q_pos0 || !n_q || !q_offset || !n_k || !k_offset || !workspace || !d_status) return KVQ_ERR_INVALID_ARG;
  int rc;
  if ((rc = check_rows(q_nope, n_q_rows, num_heads)) || (rc = check_rows(q_rope, n_q_rows, num_heads)) ||
      (rc = check_out_rows(out, n_q_rows, num_heads, VDIM)))
    return rc;
  if (n_k_rows == 0) return KVQ_ERR_INVALID_ARG;   // (a query attends its own position at least)
  if ((rc = check_rows(k_nope, n_k_rows, num_heads)) || (rc = check_rows(k_rope, n_k_rows, 1)) ||
      (rc = check_rows(v, n_k_rows, num_heads)))
    return rc;
  if (!mappable(q_nope, n_q_rows, num_heads) || !mappable(q_rope, n_q_rows, num_heads) ||
      !mappable(k_nope, n_k_rows, num_heads) || !mappable(k_rope, n_k_rows, 1) || !mappable(v, n_k_rows, num_heads))
    return KVQ_ERR_UNSUPPORTED;
  if (!aligned16(workspace)) return KVQ_ERR_ALIGNMENT;
  if (ws_bytes < latent_prefill_needs(lanes, num_heads, max_n_q, max_n_k)) return KVQ_ERR_WORKSPACE_TOO_SMALL;
  LatentPrefillArgs a{};
  a.q_pos0 = q_pos0;
  a.n_q = n_q;
  a.q_offset = q_offset;
  a.n_k = n_k;
  a.k_offset = k_offset;
  a.heads = num_heads;
  a.lanes = lanes;
  a.max_n_q = max_n_q;
  a.n_q_rows = n_q_rows;
  a.max_n_k = max_n_k;
  a.n_k_rows = n_k_rows;
  a.qn = rows_view(q_nope, n_q_rows, num_heads);
  a.qr = rows_view(q_rope, n_q_rows, num_heads);
  a.kn = rows_view(k_nope, n_k_rows, num_heads);
  a.kr = rows_view(k_rope, n_k_rows, 1);
  a.v = rows_view(v, n_k_rows, num_heads);
  a.out = rows_view(out, n_q_rows, num_heads);
  a.scale_log2 = sm_scale * LOG2E;
  a.ws = static_cast<float*>(workspace);
  a.status = d_status;
  return launch_latent_prefill(a, (cudaStream_t)stream);
}

}  // extern "C"
