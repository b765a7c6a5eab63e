// paged.cu -- writing into the paged FP4 cache: the fused rotate-and-quantise
// append, and the rotation of queries and outputs.
//
// "DeepSeek-V4.1-Flash: Pushing the Limits of KV Cache Compression", section
// 2.4.4: the main-KV latent is quantised after RoPE, its RoPE and non-RoPE
// channels in one format (E2M1 with one E4M3 scale per 16), the indexer key in
// OCP MXFP4.
#include "codec_blocks.cuh"
#include "paged_common.cuh"

namespace csa2 {

__device__ int g_paged_error = 0;

// x c - y s rounded once to fp32. Both products are split into their rounded
// value and its exact error (fma), and the difference of the rounded products
// into its value and error (Knuth's two-sum), so that the last addition is the
// only rounding that counts. The codes are decided on this value: with the
// usual two or three roundings, values next to a rounding border of 4 bits
// would depend on the order of operations.
__device__ __forceinline__ float diff_of_products(float x, float c, float y, float s) {
  const float p = __fmul_rn(x, c), q = __fmul_rn(y, s);
  const float pe = __fmaf_rn(x, c, -p), qe = __fmaf_rn(y, s, -q);
  const float h = __fsub_rn(p, q);
  const float z = __fsub_rn(h, p);
  const float e = __fsub_rn(__fsub_rn(p, __fsub_rn(h, z)), __fadd_rn(q, z));
  const float r = __fadd_rn(h, __fadd_rn(e, __fsub_rn(pe, qe)));
  return r != 0.0f ? r : h;  // (a zero keeps the sign that the difference has)
}

// (u, v) turned by the angle (cos, sin)
__device__ __forceinline__ void turn(float& u, float& v, float2 cs) {
  const float a = diff_of_products(u, cs.x, v, cs.y);
  v = diff_of_products(u, cs.y, v, -cs.x);
  u = a;
}

__device__ __forceinline__ uint32_t f32x2_to_bf16x2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// ---- append: one warp per new entry ---------------------------------------------
// Lane l holds latent channels 16l .. 16l+15 (one E4M3 block) and key channels
// 4l .. 4l+3 (eight lanes share an MXFP4 block).

// The rotation of one lane's kN consecutive channels of a row of kN * 32, the
// last `dim` of which are turned. Pairs in halves meet by a shuffle: the lane
// whose channels lie dim / 2 further on holds the partners. Every lane of the
// warp calls it.
template <int kN>
__device__ __forceinline__ void rotate_lane(float (&f)[kN], int lane, const float2* __restrict__ cs, int dim,
                                            bool interleaved) {
  const int c0 = lane * kN - (kN * 32 - dim);  // place of the lane's first channel in the turned part
  if (interleaved) {
    if (c0 >= 0) {
#pragma unroll
      for (int i = 0; i < kN / 2; ++i) turn(f[2 * i], f[2 * i + 1], cs[c0 / 2 + i]);
    }
    return;
  }
  const int half = dim / 2;
  const bool second = c0 >= half;
  const int partner = (lane + (second ? -half : half) / kN) & 31;
  float o[kN];
#pragma unroll
  for (int i = 0; i < kN; ++i) o[i] = __shfl_sync(0xffffffffu, f[i], partner);
  if (c0 < 0) return;
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    const float2 r = cs[(second ? c0 - half : c0) + i];
    f[i] = second ? diff_of_products(o[i], r.y, f[i], -r.x) : diff_of_products(f[i], r.x, o[i], r.y);
  }
}

struct AppendArgs {
  const uint16_t *kv, *ik;
  int32_t n_tokens, B, per_seq;
  const int32_t* cu;
  const float2* rope;  // null: rows are taken as they are
  int64_t n_rope;
  int32_t rope_dim;
  const int32_t* positions;
  bool interleaved;
  uint8_t *kv_data, *kv_scale, *ik_data, *ik_scale;
  PageTable pages;
  const int32_t* n_visible;
  int32_t* n_visible_out;  // null: none, or advanced in place by advance_paged_kernel
  int32_t token_blocks;    // blocks of the grid that take tokens; the rest take counts
};

// The sequence of token row i: the number of the boundaries cu[1] .. cu[B] that
// are <= i, found 32 at a time by the lanes of a warp. Ends for any contents.
__device__ __forceinline__ int32_t sequence_of(const int32_t* __restrict__ cu, int32_t B, int32_t i, int lane) {
  int32_t lo = 0, hi = B;
  while (lo < hi) {
    const int32_t step = (hi - lo + 31) / 32;
    const int64_t at = lo + (int64_t)(lane + 1) * step;
    const bool below = at <= hi && cu[at] <= i;
    const int32_t c = __popc(__ballot_sync(0xffffffffu, below));
    lo += c * step;
    if (lo + step - 1 < hi) hi = lo + step - 1;
  }
  return lo;
}

constexpr int kPagedWarps = 8;

__device__ __forceinline__ bool append_fits(int64_t nv, int32_t count, const PageTable& pages) {
  return nv >= 0 && nv + count <= pages.capacity();
}

__global__ void __launch_bounds__(kPagedWarps * 32) paged_append_kernel(AppendArgs a) {
  static_assert(kIdxDim == 32 * 4 && kHeadDim == 32 * 16, "a lane holds 16 latent and 4 key channels");
  pdl_begin();
  const int lane = threadIdx.x & 31;
  if ((int32_t)blockIdx.x >= a.token_blocks) {
    // counts: one thread per sequence
    const int32_t b = ((int32_t)blockIdx.x - a.token_blocks) * (int32_t)blockDim.x + (int32_t)threadIdx.x;
    if (b >= a.B) return;
    const TokenRun run = token_run(a.cu, b, a.n_tokens, a.per_seq);
    const int64_t nv = a.n_visible[b];
    const bool ok = run.count >= 0 && append_fits(nv, run.count, a.pages);
    if (!ok) record_error(&g_paged_error, CSA2_ERR_DEVICE);
    if (a.n_visible_out) a.n_visible_out[b] = (int32_t)(ok ? nv + run.count : nv);
    return;
  }
  const int32_t i = (int32_t)((int64_t)blockIdx.x * kPagedWarps + (threadIdx.x >> 5));
  if (i >= a.n_tokens) return;
  const uint4* src = reinterpret_cast<const uint4*>(a.kv + (int64_t)i * kHeadDim + lane * 16);
  const uint4 v0 = src[0], v1 = src[1];
  const uint2 kw = reinterpret_cast<const uint2*>(a.ik + (int64_t)i * kIdxDim)[lane];
  const int32_t b = a.cu ? sequence_of(a.cu, a.B, i, lane) : i / a.per_seq;
  if (b >= a.B) return;  // behind the last sequence
  const TokenRun run = token_run(a.cu, b, a.n_tokens, a.per_seq);
  const int32_t t = i - run.first;
  if (run.count < 0 || t < 0 || t >= run.count) return;
  const int64_t nv = a.n_visible[b];
  if (!append_fits(nv, run.count, a.pages)) return;  // reported with the counts
  const int64_t row = a.pages.row(b, nv + t);
  const int64_t pos = !a.rope ? 0 : a.positions ? (int64_t)a.positions[i] : nv + t;
  if (row < 0 || (a.rope && (pos < 0 || pos >= a.n_rope))) {
    if (lane == 0) record_error(&g_paged_error, CSA2_ERR_DEVICE);
    return;
  }
  const uint32_t w[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
  float f[16], g[4];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    f[2 * j] = bf16_bits_to_f32(w[j] & 0xFFFFu);
    f[2 * j + 1] = bf16_bits_to_f32(w[j] >> 16);
  }
  g[0] = bf16_bits_to_f32(kw.x & 0xFFFFu);
  g[1] = bf16_bits_to_f32(kw.x >> 16);
  g[2] = bf16_bits_to_f32(kw.y & 0xFFFFu);
  g[3] = bf16_bits_to_f32(kw.y >> 16);
  if (a.rope) {
    const float2* cs = a.rope + pos * (a.rope_dim / 2);
    rotate_lane<16>(f, lane, cs, a.rope_dim, a.interleaved);
    rotate_lane<4>(g, lane, cs, a.rope_dim, a.interleaved);
  }
  {
    uint2 d;
    uint8_t sc;
    encode_kv_fp4_values(f, d, sc);
    *reinterpret_cast<uint2*>(a.kv_data + row * kKvBytes + lane * 8) = d;
    a.kv_scale[row * kKvScales + lane] = sc;
  }
  {
    float amax = fmaxf(fmaxf(fabsf(g[0]), fabsf(g[1])), fmaxf(fabsf(g[2]), fabsf(g[3])));
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    float inv;
    // (the exponent field of the fp32 value is the one its upper half has as bf16)
    const int X = mxfp4_exponent(__float_as_uint(amax) >> 16, inv);
    *reinterpret_cast<uint16_t*>(a.ik_data + row * kIkBytes + lane * 2) =
        (uint16_t)(cvt_e2m1x2(g[0] * inv, g[1] * inv) | (cvt_e2m1x2(g[2] * inv, g[3] * inv) << 8));
    if ((lane & 7) == 0) a.ik_scale[row * kIkScales + lane / 8] = (uint8_t)(X + 127);
  }
}

// In-place advance of the counts, after the append grid has finished reading them.
__global__ void advance_paged_kernel(int32_t* __restrict__ n_visible, const int32_t* __restrict__ cu, int32_t B,
                                     int32_t n_tokens, int32_t per_seq, PageTable pages) {
  pdl_begin();
  const int32_t b = blockIdx.x * blockDim.x + threadIdx.x;
  if (b >= B) return;
  const TokenRun run = token_run(cu, b, n_tokens, per_seq);
  const int64_t nv = n_visible[b];
  if (run.count > 0 && append_fits(nv, run.count, pages)) n_visible[b] = (int32_t)(nv + run.count);
}

// ---- rotation of [tokens][heads][dim] rows --------------------------------------
// One thread per unit of a row: a 16-byte chunk of untouched or interleaved
// channels, or the two chunks that a half pairing joins. In place the untouched
// chunks are no units at all (units_copy = 0).
struct RopeArgs {
  const uint16_t* x;
  uint16_t* out;
  int64_t n_tokens;
  int32_t heads, dim;
  const float2* rope;
  int64_t n_rope;
  int32_t rope_dim;
  const int32_t* positions;
  int32_t units_copy, units;  // units of a row, the copied ones first
  bool interleaved, inverse;
};

__device__ __forceinline__ void unpack8(uint4 v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = bf16_bits_to_f32(w[i] & 0xFFFFu);
    f[2 * i + 1] = bf16_bits_to_f32(w[i] >> 16);
  }
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(f32x2_to_bf16x2(f[0], f[1]), f32x2_to_bf16x2(f[2], f[3]), f32x2_to_bf16x2(f[4], f[5]),
                    f32x2_to_bf16x2(f[6], f[7]));
}

__global__ void __launch_bounds__(256) rope_kernel(RopeArgs a) {
  pdl_begin();
  const int64_t per_token = (int64_t)a.heads * a.units;
  const int64_t u = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  const int64_t t = u / per_token;
  if (t >= a.n_tokens) return;
  const int64_t in_token = u - t * per_token;
  const int32_t head = (int32_t)(in_token / a.units), unit = (int32_t)(in_token - (int64_t)head * a.units);
  const int64_t pos = a.positions ? (int64_t)a.positions[t] : t;
  if (pos < 0 || pos >= a.n_rope) {
    if (in_token == 0) record_error(&g_paged_error, CSA2_ERR_DEVICE);
    return;
  }
  const int64_t base = (t * a.heads + head) * a.dim;
  if (unit < a.units_copy) {
    reinterpret_cast<uint4*>(a.out + base)[unit] = reinterpret_cast<const uint4*>(a.x + base)[unit];
    return;
  }
  const int32_t c = (unit - a.units_copy) * 8;  // place in the turned part
  const int64_t at = base + (a.dim - a.rope_dim) + c;
  const float2* cs = a.rope + pos * (a.rope_dim / 2);
  const float sign = a.inverse ? -1.0f : 1.0f;
  float f[8];
  unpack8(*reinterpret_cast<const uint4*>(a.x + at), f);
  if (a.interleaved) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 r = cs[c / 2 + i];
      turn(f[2 * i], f[2 * i + 1], make_float2(r.x, r.y * sign));
    }
    *reinterpret_cast<uint4*>(a.out + at) = pack8(f);
    return;
  }
  float g[8];
  const int64_t at2 = at + a.rope_dim / 2;
  unpack8(*reinterpret_cast<const uint4*>(a.x + at2), g);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 r = cs[c + i];
    turn(f[i], g[i], make_float2(r.x, r.y * sign));
  }
  *reinterpret_cast<uint4*>(a.out + at) = pack8(f);
  *reinterpret_cast<uint4*>(a.out + at2) = pack8(g);
}

// ---- selected entries to rows of the pool ----------------------------------------
__global__ void page_rows_kernel(const int32_t* __restrict__ idx, int32_t B, int32_t k,
                                 const int32_t* __restrict__ n_visible, PageTable pages, int32_t* __restrict__ rows) {
  pdl_begin();
  const int64_t j = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (j >= (int64_t)B * k) return;
  const int32_t b = (int32_t)(j / k);
  const int32_t e = idx[j];
  int64_t row = -1;
  if (e >= 0) {
    if (e < n_visible[b] && e < pages.capacity()) row = pages.row(b, e);
    if (row < 0) record_error(&g_paged_error, CSA2_ERR_DEVICE);
  }
  rows[j] = (int32_t)row;
}

}  // namespace csa2

using namespace csa2;

int csa2_read_and_clear_paged_error(cudaStream_t s) {
  int v = 0, z = 0;
  if (cudaMemcpyFromSymbolAsync(&v, g_paged_error, sizeof(int), 0, cudaMemcpyDeviceToHost, s) != cudaSuccess)
    return CSA2_ERR_CUDA;
  if (cudaMemcpyToSymbolAsync(g_paged_error, &z, sizeof(int), 0, cudaMemcpyHostToDevice, s) != cudaSuccess)
    return CSA2_ERR_CUDA;
  if (cudaStreamSynchronize(s) != cudaSuccess) return CSA2_ERR_CUDA;
  return v;
}

static int check_rope(const float* rope, int64_t n_rope, int32_t rope_dim) {
  if (n_rope < 0 || rope_dim < 0) return CSA2_ERR_INVALID_ARG;
  if (rope_dim % 32 || rope_dim > CSA2_MAX_ROPE_DIM) return CSA2_ERR_UNSUPPORTED_SHAPE;
  if (rope && !csa2_aligned(rope, 16)) return CSA2_ERR_ALIGNMENT;
  return CSA2_OK;
}

extern "C" int csa2_rope(const void* x_bf16, int64_t n_tokens, int32_t heads, int32_t dim, const float* rope,
                         int64_t n_rope, int32_t rope_dim, const int32_t* positions, int32_t interleaved,
                         int32_t inverse, void* out_bf16, csa2_stream_t stream) {
  if (!rope || n_tokens < 0 || heads < 0 || dim <= 0) return CSA2_ERR_INVALID_ARG;
  if (n_tokens > 0 && heads > 0 && (!x_bf16 || !out_bf16)) return CSA2_ERR_INVALID_ARG;
  if (int rc = check_rope(rope, n_rope, rope_dim)) return rc;
  if (rope_dim == 0 || dim % 8 || dim < rope_dim) return CSA2_ERR_UNSUPPORTED_SHAPE;
  if (!csa2_aligned(x_bf16, 16) || !csa2_aligned(out_bf16, 16) || !csa2_aligned(positions, 4))
    return CSA2_ERR_ALIGNMENT;
  if (n_tokens == 0 || heads == 0) return CSA2_OK;
  RopeArgs a{};
  a.x = (const uint16_t*)x_bf16;
  a.out = (uint16_t*)out_bf16;
  a.n_tokens = n_tokens;
  a.heads = heads;
  a.dim = dim;
  a.rope = (const float2*)rope;
  a.n_rope = n_rope;
  a.rope_dim = rope_dim;
  a.positions = positions;
  a.units_copy = x_bf16 == out_bf16 ? 0 : (dim - rope_dim) / 8;
  a.units = a.units_copy + (interleaved ? rope_dim / 8 : rope_dim / 16);
  a.interleaved = interleaved != 0;
  a.inverse = inverse != 0;
  // the units of a call within int64 and its grid within 2^31 - 1 blocks
  if (n_tokens > (0x7FFFFFFFLL * 256) / ((int64_t)heads * a.units)) return CSA2_ERR_UNSUPPORTED_SHAPE;
  const int64_t units = n_tokens * heads * a.units;
  CSA2_LAUNCH_PDL(rope_kernel, dim3((unsigned)((units + 255) / 256)), dim3(256), 0, (cudaStream_t)stream, a);
  return CSA2_OK;
}

extern "C" int csa2_paged_kv_append(const void* kv_bf16, const void* ik_bf16, int32_t n_tokens,
                                    const int32_t* cu_tokens, int32_t B, const float* rope, int64_t n_rope,
                                    int32_t rope_dim, const int32_t* positions, int32_t interleaved,
                                    uint8_t* kv_data, uint8_t* kv_scale, uint8_t* ik_data, uint8_t* ik_scale,
                                    int64_t n_pages, int32_t page_size, const int32_t* page_table, int32_t max_pages,
                                    const int32_t* n_visible, int32_t* n_visible_out, csa2_stream_t stream) {
  if (B != 0 && (!kv_data || !kv_scale || !ik_data || !ik_scale || !n_visible)) return CSA2_ERR_INVALID_ARG;
  if (n_tokens > 0 && (!kv_bf16 || !ik_bf16)) return CSA2_ERR_INVALID_ARG;
  AppendArgs a{};
  if (int rc = paged_check(page_table, n_pages, page_size, max_pages, B, a.pages)) return rc;
  if (int rc = paged_runs(cu_tokens, n_tokens, B, a.per_seq)) return rc;
  if (int rc = check_rope(rope, n_rope, rope_dim)) return rc;
  if (!csa2_aligned(kv_bf16, 16) || !csa2_aligned(ik_bf16, 16) || !csa2_aligned(kv_data, 16) ||
      !csa2_aligned(kv_scale, 16) || !csa2_aligned(ik_data, 16) || !csa2_aligned(ik_scale, 16) ||
      !csa2_aligned(positions, 4) || !csa2_aligned(n_visible, 4) || !csa2_aligned(n_visible_out, 4))
    return CSA2_ERR_ALIGNMENT;
  if (B == 0) return CSA2_OK;
  cudaStream_t s = (cudaStream_t)stream;
  const bool in_place = n_visible_out == n_visible;
  a.kv = (const uint16_t*)kv_bf16;
  a.ik = (const uint16_t*)ik_bf16;
  a.n_tokens = n_tokens;
  a.B = B;
  a.cu = cu_tokens;
  a.rope = rope_dim > 0 ? (const float2*)rope : nullptr;
  a.n_rope = n_rope;
  a.rope_dim = rope_dim;
  a.positions = positions;
  a.interleaved = interleaved != 0;
  a.kv_data = kv_data;
  a.kv_scale = kv_scale;
  a.ik_data = ik_data;
  a.ik_scale = ik_scale;
  a.n_visible = n_visible;
  a.n_visible_out = in_place ? nullptr : n_visible_out;
  a.token_blocks = (n_tokens + kPagedWarps - 1) / kPagedWarps;
  const unsigned count_blocks = (unsigned)((B + kPagedWarps * 32 - 1) / (kPagedWarps * 32));
  CSA2_LAUNCH_PDL(paged_append_kernel, dim3((unsigned)a.token_blocks + count_blocks), dim3(kPagedWarps * 32), 0, s, a);
  if (in_place)
    CSA2_LAUNCH_PDL(advance_paged_kernel, dim3((unsigned)((B + 255) / 256)), dim3(256), 0, s, n_visible_out,
                    cu_tokens, B, n_tokens, a.per_seq, a.pages);
  return CSA2_OK;
}

// Rows of the pool of the selected entries (csa2_paged_sparse_attn_decode).
int csa2_launch_page_rows(const int32_t* idx, int32_t B, int32_t k, const int32_t* n_visible, const PageTable& pages,
                          int32_t* rows, cudaStream_t s) {
  const int64_t n = (int64_t)B * k;
  if (n == 0) return CSA2_OK;
  CSA2_LAUNCH_PDL(page_rows_kernel, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, s, idx, B, k, n_visible, pages,
                  rows);
  return CSA2_OK;
}
