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
// would depend on the order of operations. An infinite channel or product has no
// error terms (they are NaN): the difference of the products is then the result.
__device__ __forceinline__ float diff_of_products(float x, float c, float y, float s) {
  const float p = __fmul_rn(x, c), q = __fmul_rn(y, s);
  const float pe = __fmaf_rn(x, c, -p), qe = __fmaf_rn(y, s, -q);
  const float h = __fsub_rn(p, q);
  const float z = __fsub_rn(h, p);
  const float e = __fsub_rn(__fsub_rn(p, __fsub_rn(h, z)), __fadd_rn(q, z));
  const float r = __fadd_rn(h, __fadd_rn(e, __fsub_rn(pe, qe)));
  return fabsf(r) > 0.0f ? r : h;  // (r NaN, or a zero, which keeps the sign that the difference has)
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

// ---- append --------------------------------------------------------------------
// One warp holds an entry: lane l latent channels 16l .. 16l+15 (one E4M3
// block) and key channels 4l .. 4l+3 (eight lanes share an MXFP4 block).

// The pairs of the turned parts go over the lanes evenly (a lane that owned 16
// turned channels would hold up the 28 that own none), both parts of a pair
// from the rows themselves, and the turned values to the owning lanes through
// shared memory: turned[0][c] is channel c of the latent's turned part,
// turned[1][c] of the key's.
__device__ __forceinline__ void turn_pairs(float (&turned)[2][CSA2_MAX_ROPE_DIM], const uint16_t* __restrict__ kv_row,
                                           const uint16_t* __restrict__ ik_row, const float2* __restrict__ cs, int dim,
                                           bool interleaved, int lane) {
  const uint16_t* part[2] = {kv_row + (kHeadDim - dim), ik_row + (kIdxDim - dim)};
  for (int p = lane; p < dim / 2; p += 32) {
    const float2 r = cs[p];
    const int u = interleaved ? 2 * p : p, v = interleaved ? 2 * p + 1 : p + dim / 2;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      float x = bf16_bits_to_f32(part[k][u]), y = bf16_bits_to_f32(part[k][v]);
      turn(x, y, r);
      turned[k][u] = x;
      turned[k][v] = y;
    }
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
// are <= i. Ends for any contents.
__device__ __forceinline__ int32_t sequence_of(const int32_t* __restrict__ cu, int32_t B, int32_t i) {
  int32_t lo = 0, hi = B;
  while (lo < hi) {
    const int32_t mid = lo + (hi - lo) / 2;
    if (cu[mid + 1] <= i)
      lo = mid + 1;
    else
      hi = mid;
  }
  return lo;
}

constexpr int kPagedWarps = 8;
constexpr int kTokensPerWarp = 4;
constexpr int32_t kManyTokens = 152 * kPagedWarps * kTokensPerWarp;

__device__ __forceinline__ bool append_fits(int64_t nv, int32_t count, const PageTable& pages) {
  return nv >= 0 && nv + count <= pages.capacity();
}

// Row of the pool (-1: not written) and position of token row i.
__device__ __forceinline__ void resolve_token(const AppendArgs& a, int32_t i, int64_t& row, int64_t& pos) {
  row = -1;
  pos = 0;
  const int32_t given = a.rope && a.positions ? a.positions[i] : 0;
  const int32_t b = a.cu ? sequence_of(a.cu, a.B, i) : i / a.per_seq;
  if (b >= a.B) return;  // behind the last sequence
  const TokenRun run = token_run(a.cu, b, a.n_tokens, a.per_seq);
  const int32_t t = i - run.first;
  if (run.count < 0 || t < 0 || t >= run.count) return;
  const int64_t nv = a.n_visible[b];
  if (!append_fits(nv, run.count, a.pages)) return;  // reported with the counts
  const int64_t r = a.pages.row(b, nv + t);
  if (a.rope) pos = a.positions ? (int64_t)given : nv + t;
  if (r < 0 || (a.rope && (pos < 0 || pos >= a.n_rope))) {
    record_error(&g_paged_error, CSA2_ERR_DEVICE);
    return;
  }
  row = r;
}

// kPerWarp consecutive tokens to a warp: their rows of the pool are looked up
// by as many lanes at once (the chain boundary -> count -> page -> angles is
// four dependent reads), while the rows of all of them are on their way.
// Bound: 1,636 bytes an entry would take 19 us for 76,831 entries in pages of 16;
// 39.5 us measured (3.2 TB/s), 29.0 without a rotation. 397 warp instructions an
// entry keep the schedulers 62 % busy, with 22 warps on an SM (79 registers a
// thread), and a warp's entries wait for their angles one after another (all four's
// at once took longer). A step of 32: 3.2 us.
template <int kPerWarp>
__global__ void __launch_bounds__(kPagedWarps * 32) paged_append_kernel(AppendArgs a) {
  static_assert(kIdxDim == 32 * 4 && kHeadDim == 32 * 16, "a lane holds 16 latent and 4 key channels");
  __shared__ __align__(16) float s_turned[kPagedWarps][2][CSA2_MAX_ROPE_DIM];
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
  const int64_t first = ((int64_t)blockIdx.x * kPagedWarps + (threadIdx.x >> 5)) * kPerWarp;
  // rows of no sequence are not read: their owner may still be writing them
  const int32_t row0 = a.cu ? max(a.cu[0], 0) : 0, row1 = a.cu ? min(a.cu[a.B], a.n_tokens) : a.n_tokens;
  if (first + kPerWarp <= row0 || first >= row1) return;
  uint4 v[kPerWarp][2];
  uint2 kw[kPerWarp];
#pragma unroll
  for (int j = 0; j < kPerWarp; ++j) {
    const int32_t i = min(max((int32_t)first + j, row0), row1 - 1);
    const uint4* src = reinterpret_cast<const uint4*>(a.kv + (int64_t)i * kHeadDim + lane * 16);
    v[j][0] = __ldcs(src);  // (read once)
    v[j][1] = __ldcs(src + 1);
    kw[j] = __ldcs(reinterpret_cast<const uint2*>(a.ik + (int64_t)i * kIdxDim) + lane);
  }
  int64_t my_row = -1, my_pos = 0;
  if (lane < kPerWarp && first + lane >= row0 && first + lane < row1)
    resolve_token(a, (int32_t)(first + lane), my_row, my_pos);
  float(&turned)[2][CSA2_MAX_ROPE_DIM] = s_turned[threadIdx.x >> 5];
#pragma unroll
  for (int j = 0; j < kPerWarp; ++j) {
    const int64_t row = __shfl_sync(0xffffffffu, my_row, j), pos = __shfl_sync(0xffffffffu, my_pos, j);
    if (row < 0) continue;
    if (a.rope) {
      __syncwarp();
      turn_pairs(turned, a.kv + (first + j) * kHeadDim, a.ik + (first + j) * kIdxDim, a.rope + pos * (a.rope_dim / 2),
                 a.rope_dim, a.interleaved, lane);
      __syncwarp();
    }
    const uint32_t w[8] = {v[j][0].x, v[j][0].y, v[j][0].z, v[j][0].w, v[j][1].x, v[j][1].y, v[j][1].z, v[j][1].w};
    float f[16];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      f[2 * i] = bf16_bits_to_f32(w[i] & 0xFFFFu);
      f[2 * i + 1] = bf16_bits_to_f32(w[i] >> 16);
    }
    float4 g = make_float4(bf16_bits_to_f32(kw[j].x & 0xFFFFu), bf16_bits_to_f32(kw[j].x >> 16),
                           bf16_bits_to_f32(kw[j].y & 0xFFFFu), bf16_bits_to_f32(kw[j].y >> 16));
    if (a.rope) {
      // (rope_dim is a multiple of 32, so a lane's channels are turned all or none)
      if (const int c = lane * 16 - (kHeadDim - a.rope_dim); c >= 0) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float4 t = *reinterpret_cast<const float4*>(&turned[0][c + 4 * i]);
          f[4 * i] = t.x, f[4 * i + 1] = t.y, f[4 * i + 2] = t.z, f[4 * i + 3] = t.w;
        }
      }
      if (const int c = lane * 4 - (kIdxDim - a.rope_dim); c >= 0) g = *reinterpret_cast<const float4*>(&turned[1][c]);
    }
    uint2 d;
    uint8_t sc;
    encode_kv_fp4_values(f, d, sc);
    *reinterpret_cast<uint2*>(a.kv_data + row * kKvBytes + lane * 8) = d;
    a.kv_scale[row * kKvScales + lane] = sc;
    // (a NaN counts as the largest, as in csa2_quant_mxfp4, which compares bit patterns)
    float amax = max_abs3_nan(g.x, g.y, max_abs3_nan(g.z, g.w, 0.0f));
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    float inv;
    // (the exponent field of the fp32 value is the one its upper half has as bf16)
    const int X = mxfp4_exponent(__float_as_uint(amax) >> 16, inv);
    *reinterpret_cast<uint16_t*>(a.ik_data + row * kIkBytes + lane * 2) =
        (uint16_t)(cvt_e2m1x2(g.x * inv, g.y * inv) | (cvt_e2m1x2(g.z * inv, g.w * inv) << 8));
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
// A warp takes kRopeRows consecutive rows. Their untouched 16-byte chunks are
// copied chunk by chunk over the lanes (in place there are none, copy = 0);
// their turned parts are units of one chunk (interleaved pairs) or of the two
// chunks that a half pairing joins, and the units of all the rows go over the
// lanes together: with 64 turned channels a row has 8 units, four rows a warp's
// worth, and no lane waits for another's rotation.
// Bound by HBM: 4,096 x 64 rows of 512 in 82 us, 6.5 TB/s of 4 bytes an element
// (two rows to a warp 94 us, eight 103; one thread to a 16-byte chunk, its row
// found by division, 157). The queries of a step of 32 take 2.6 us.
struct RopeArgs {
  const uint16_t* x;
  uint16_t* out;
  int64_t n_tokens;
  int32_t heads, dim;
  const float2* rope;
  int64_t n_rope;
  int32_t rope_dim;
  const int32_t* positions;
  int32_t copy, units;  // chunks of a row to copy, units of a row to turn
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

constexpr int kRopeRows = 4;

__global__ void __launch_bounds__(256) rope_kernel(RopeArgs a) {
  // (no pdl_launch_dependents(): the selected attention behind loads its queries, which
  // are written here, before it waits for this kernel)
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int64_t row0 = ((int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5)) * kRopeRows;
  const int64_t left = a.n_tokens * a.heads - row0;
  if (left <= 0) return;
  const int rows = left < kRopeRows ? (int)left : kRopeRows;
  const int64_t t0 = row0 / a.heads;
  const int32_t head0 = (int32_t)(row0 - t0 * a.heads);
  // lane r: the position of row r, -1 outside the table (that row is not written)
  int64_t pos = -1;
  if (lane < rows) {
    const int64_t t = t0 + (head0 + lane) / a.heads;
    pos = a.positions ? (int64_t)a.positions[t] : t;
    if (pos < 0 || pos >= a.n_rope) {
      pos = -1;
      record_error(&g_paged_error, CSA2_ERR_DEVICE);
    }
  }
  const uint32_t good = __ballot_sync(0xffffffffu, pos >= 0);
  const uint16_t* x = a.x + row0 * a.dim;
  uint16_t* out = a.out + row0 * a.dim;
  for (int c = lane; c < a.copy; c += 64) {
    uint4 v[kRopeRows][2];
#pragma unroll
    for (int r = 0; r < kRopeRows; ++r) {
      const uint4* src = reinterpret_cast<const uint4*>(x + (int64_t)r * a.dim);
      if (good >> r & 1) {
        v[r][0] = src[c];
        if (c + 32 < a.copy) v[r][1] = src[c + 32];
      }
    }
#pragma unroll
    for (int r = 0; r < kRopeRows; ++r) {
      uint4* dst = reinterpret_cast<uint4*>(out + (int64_t)r * a.dim);
      if (good >> r & 1) {
        dst[c] = v[r][0];
        if (c + 32 < a.copy) dst[c + 32] = v[r][1];
      }
    }
  }
  const float sign = a.inverse ? -1.0f : 1.0f;
  for (int u = 0; u < kRopeRows * a.units; u += 32) {
    const int r = min((u + lane) / a.units, kRopeRows - 1);
    const int c = (u + lane - r * a.units) * 8;  // place in the turned part
    const int64_t at_pos = __shfl_sync(0xffffffffu, pos, r);
    if (c >= a.units * 8 || at_pos < 0) continue;
    const int64_t at = (int64_t)r * a.dim + (a.dim - a.rope_dim) + c;
    const float2* cs = a.rope + at_pos * (a.rope_dim / 2);
    float f[8];
    unpack8(*reinterpret_cast<const uint4*>(x + at), f);
    if (a.interleaved) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float4 p = *reinterpret_cast<const float4*>(cs + c / 2 + 2 * i);  // two angles
        turn(f[4 * i], f[4 * i + 1], make_float2(p.x, p.y * sign));
        turn(f[4 * i + 2], f[4 * i + 3], make_float2(p.z, p.w * sign));
      }
      *reinterpret_cast<uint4*>(out + at) = pack8(f);
      continue;
    }
    float g[8];
    const int64_t at2 = at + a.rope_dim / 2;
    unpack8(*reinterpret_cast<const uint4*>(x + at2), g);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 p = *reinterpret_cast<const float4*>(cs + c + 2 * i);
      turn(f[2 * i], g[2 * i], make_float2(p.x, p.y * sign));
      turn(f[2 * i + 1], g[2 * i + 1], make_float2(p.z, p.w * sign));
    }
    *reinterpret_cast<uint4*>(out + at) = pack8(f);
    *reinterpret_cast<uint4*>(out + at2) = pack8(g);
  }
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
  a.copy = x_bf16 == out_bf16 ? 0 : (dim - rope_dim) / 8;
  a.units = interleaved ? rope_dim / 8 : rope_dim / 16;
  a.interleaved = interleaved != 0;
  a.inverse = inverse != 0;
  // the grid within 2^31 - 1 blocks of 8 warps
  if (n_tokens > 0x7FFFFFFFLL * 8 * kRopeRows / heads) return CSA2_ERR_UNSUPPORTED_SHAPE;
  const int64_t warps = (n_tokens * heads + kRopeRows - 1) / kRopeRows;
  CSA2_LAUNCH_PDL(rope_kernel, dim3((unsigned)((warps + 7) / 8)), dim3(256), 0, (cudaStream_t)stream, a);
  return CSA2_OK;
}

extern "C" int csa2_paged_kv_append(const void* kv_bf16, const void* ik_bf16, int32_t n_tokens,
                                    const int32_t* cu_tokens, int32_t B, const float* rope, int64_t n_rope,
                                    int32_t rope_dim, const int32_t* positions, int32_t interleaved,
                                    uint8_t* kv_data, uint8_t* kv_scale, uint8_t* ik_data, uint8_t* ik_scale,
                                    int64_t n_pages, int32_t page_size, const int32_t* page_table, int32_t max_pages,
                                    const int32_t* n_visible, int32_t* n_visible_out, csa2_stream_t stream) {
  if (B != 0 && (!paged_planes(n_pages, kv_data, kv_scale) || !paged_planes(n_pages, ik_data, ik_scale) || !n_visible))
    return CSA2_ERR_INVALID_ARG;
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
  // 76,801 tokens: 39.5 us with four tokens to a warp, 48 with one; but a warp's
  // tokens follow each other, so while SMs would stay idle it takes one
  const int per_warp = n_tokens >= kManyTokens ? kTokensPerWarp : 1;
  const int32_t per_block = kPagedWarps * per_warp;
  a.token_blocks = (int32_t)(((int64_t)n_tokens + per_block - 1) / per_block);
  const unsigned count_blocks = (unsigned)((B + kPagedWarps * 32 - 1) / (kPagedWarps * 32));
  const dim3 grid((unsigned)a.token_blocks + count_blocks);
  if (per_warp == 1)
    CSA2_LAUNCH_PDL(paged_append_kernel<1>, grid, dim3(kPagedWarps * 32), 0, s, a);
  else
    CSA2_LAUNCH_PDL(paged_append_kernel<kTokensPerWarp>, grid, dim3(kPagedWarps * 32), 0, s, a);
  if (in_place)
    CSA2_LAUNCH_PDL(advance_paged_kernel, dim3((unsigned)((B + 255) / 256)), dim3(256), 0, s, n_visible_out,
                    cu_tokens, B, n_tokens, a.per_seq, a.pages);
  return CSA2_OK;
}
