// latent.cuh -- layout of the latent cache (include/kvq.h, "Latent attention") and the argument
// structs and launchers of its kernels.
#pragma once
#include "kvq_internal.cuh"

namespace kvq {

constexpr int LAT = 512;                       // latent dims (keys and values of the absorbed form)
constexpr int LROPE = 64;                      // rotary key dims
constexpr int LCHUNK = P * 128;                // 8,192 B: 64 slots of 64 bf16 dims, 128-byte swizzled
constexpr int LNCHUNK = (LAT + LROPE) / 64;    // 9 chunks a bf16 block, the last the rotary key
constexpr int LBF16_BLOCK = LNCHUNK * LCHUNK;  // 73,728 B
constexpr int LMX_CODES = P * LAT;             // 32,768 B: 8 chunks of [64 slots][64 B]
constexpr int LMX_SCALES = LMX_CODES + LCHUNK; // 40,960: the scale bytes, after the rotary chunk
constexpr int LMX_BLOCK = LMX_SCALES + P * 16; // 41,984 B
constexpr int LMAX_HEADS = 128;
constexpr int LMAX_PREFILL = INT32_MAX - 256;  // queries and keys of a lane, expanded form: sums with a tile fit 32 bits
constexpr int NOPE = 128, VDIM = 128;          // expanded form: dims a head of k (beside the rotary 64) and v

__host__ __device__ constexpr int latent_block(int fmt) { return fmt == KVQ_LATENT_MXFP8 ? LMX_BLOCK : LBF16_BLOCK; }

// byte of 16 B unit u (0 .. 7) of a slot within a swizzled chunk
__host__ __device__ __forceinline__ int chunk_unit(int slot, int u) { return slot * 128 + ((u ^ (slot & 7)) << 4); }

struct LatentView {
  uint8_t* pool;
  int64_t pool_pages, page_bytes;
  int64_t layer_off;          // byte of the layer's block within a page
  const int32_t* page_table;  // [lanes][max_pages]
  int max_pages, lanes;
  int32_t* status;
};

struct RowsView {   // bf16 rows, strides in elements
  __nv_bfloat16* p;
  int64_t row, head;
};

struct LatentTokenArgs {   // append and read
  LatentView c;
  const int32_t *start_pos, *n_tok, *tok_offset;
  int max_tok, n_rows;
  RowsView latent, rope;
};

struct LatentAttnArgs {
  LatentView c;
  const int32_t *q_pos0, *n_q, *q_offset, *seq_len;
  int max_n_q, n_q_rows, max_seq_len, heads;
  RowsView ql, qr, out;
  float scale_log2;
  float* ws;
};

struct LatentPrefillArgs {
  const int32_t *q_pos0, *n_q, *q_offset, *n_k, *k_offset;
  int heads, lanes, max_n_q, n_q_rows, max_n_k, n_k_rows;
  RowsView qn, qr, kn, kr, v, out;
  float scale_log2;
  float* ws;
  int32_t* status;
};

// Rows and positions of lane b of an absorbed attention call; false (after flagging, if asked to)
// for a lane that is skipped.
__device__ __forceinline__ bool latent_lane(const LatentAttnArgs& a, int b, int& nq, int& row0, int& pos0, bool report) {
  const int len = a.seq_len[b];
  nq = a.n_q[b];
  row0 = a.q_offset[b];
  pos0 = a.q_pos0[b];
  int err = 0;
  if (len < 0 || len > a.max_seq_len) err = KVQ_STATUS_BAD_LEN;
  else if (nq < 0 || nq > a.max_n_q) err = KVQ_STATUS_BAD_LEN;
  else if (nq > 0 && (row0 < 0 || (int64_t)row0 + nq > a.n_q_rows || pos0 < 0 || (int64_t)pos0 + nq > len))
    err = KVQ_STATUS_BAD_LEN;
  if (len > 0 && (int64_t)len > (int64_t)a.c.max_pages * P) err |= KVQ_STATUS_LEN_GT_TABLE;
  if (err) {
    if (report) flag(a.c.status, err);
    nq = 0;
    return false;
  }
  return nq > 0;
}

// The same for lane b of an expanded attention call.
__device__ __forceinline__ bool latent_prefill_lane(const LatentPrefillArgs& a, int b, int& nq, int& row0, int& pos0,
                                                    int& nk, int& key0, bool report) {
  nq = a.n_q[b];
  row0 = a.q_offset[b];
  pos0 = a.q_pos0[b];
  nk = a.n_k[b];
  key0 = a.k_offset[b];
  bool ok = nq >= 0 && nq <= a.max_n_q && nk >= 0 && nk <= a.max_n_k;
  if (ok && nq > 0)
    ok = row0 >= 0 && (int64_t)row0 + nq <= a.n_q_rows && key0 >= 0 && (int64_t)key0 + nk <= a.n_k_rows && pos0 >= 0 &&
         (int64_t)pos0 + nq <= nk;
  if (!ok) {
    if (report) flag(a.status, KVQ_STATUS_BAD_LEN);
    nq = 0;
    return false;
  }
  return nq > 0;
}

// four E4M3 codes (one word) times 2^e, as bf16 pairs (dims 0,1 and 2,3), exact.  A code's seven
// exponent and mantissa bits moved to bits 4 .. 10 of a half read as the bf16 number
// value * 2^-120 (subnormal codes as bf16 subnormals), so one bf16 multiply by 2^(120 + e) gives
// the value; f2 holds that factor twice, scale byte + 120 being its biased exponent.
__device__ __forceinline__ uint32_t mx_factor(uint32_t scale_byte) {
  const uint32_t f = (scale_byte + 120u) << 7;
  return f | (f << 16);
}
__device__ __forceinline__ uint32_t mx_pair(uint32_t placed, uint32_t f2) {   // codes in the high byte of each half
  const uint32_t v = (placed & 0x80008000u) | ((placed & 0x7F007F00u) >> 4);
  __nv_bfloat162 x = *reinterpret_cast<const __nv_bfloat162*>(&v), f = *reinterpret_cast<__nv_bfloat162*>(&f2);
  x = __hmul2(x, f);
  return *reinterpret_cast<uint32_t*>(&x);
}
__device__ __forceinline__ uint2 mx_quad(uint32_t codes, uint32_t f2) {
  return make_uint2(mx_pair(__byte_perm(codes, 0u, 0x1404u), f2), mx_pair(__byte_perm(codes, 0u, 0x3424u), f2));
}

// The latent kernels are launched programmatically: one may start while the kernel before it on the stream ends, and
// begins with latent_wait, before which it neither reads what that one could have written nor writes.  All its
// blocks wait, so that its own end covers everything before it.
__device__ __forceinline__ void latent_wait() {
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
}

template <class... P, class... A>
int latent_launch(void (*kernel)(P...), dim3 grid, int threads, int smem, cudaStream_t stream, const A&... args) {
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA;
}

int launch_latent_append(int fmt, const LatentTokenArgs& a, cudaStream_t stream);
int launch_latent_read(int fmt, const LatentTokenArgs& a, cudaStream_t stream);
int launch_latent_attn(int fmt, const LatentAttnArgs& a, cudaStream_t stream);
size_t latent_attn_needs(int heads, int lanes, int max_n_q, int max_seq_len);
size_t latent_attn_workspace(int heads, int lanes, int max_n_q, int max_seq_len);
int launch_latent_prefill(const LatentPrefillArgs& a, cudaStream_t stream);
size_t latent_prefill_needs(int lanes, int heads, int max_n_q, int max_n_k);
size_t latent_prefill_workspace(int lanes, int heads, int max_n_q, int max_n_k);

}  // namespace kvq
