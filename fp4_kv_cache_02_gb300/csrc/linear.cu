// linear.cu -- products with 4-bit weights: out = scale * x W^T for bf16 rows x and
// a weight matrix in the library's packed formats (E2M1 with one E8M0 scale per 32
// inputs, as csa2_quant_mxfp4 writes it, or one E4M3 scale per 16, as
// csa2_pack_kv_fp4 does).
//
// "DeepSeek-V4.1-Flash: Pushing the Limits of KV Cache Compression": section 2.3
// (latents, indexer keys and both queries are projections), the notes' section 4.4
// (FP4 weights counted at a quarter of bf16).
//
// The weights go to the tensor cores as they lie in memory: block-scaled FP4
// products with both operands E2M1. A bf16 row enters as a sum of kTerms = 8 E2M1
// vectors. With s = 2^e the block's scale such that its largest |x| / s is in
// [3.5, 7), the first term is x / s rounded to E2M1; what is left is at most s and
// is rounded on the grid of s / 4, what is left then (at most s / 8) on that of
// s / 32, and so on by 8: the remainder after eight terms is at most 2^-21 s, 2^-22 of
// the block's largest, and zero for every channel within 2^-14 of it (its last bit is
// a multiple of the eighth scale). All remainders are exact in fp32 on the way. The terms
// of a token are eight columns of the second operand, so the products cost tensor
// time that a product bound by its weights' bytes has to spare, and no instruction
// of the CUDA cores per weight.
#include "tc_common.cuh"

namespace csa2 {

__device__ int g_linear_error = 0;

namespace linear {

constexpr int kTerms = 8;
constexpr int kChunk = 256;                 // inputs to a block of weights: 128 bytes of a row
constexpr int kRows = 128;                  // outputs to a block
constexpr int kDataBytes = kRows * kChunk / 2;
constexpr int kTileTokens = 32;             // tokens to a tile: 256 columns
constexpr int kMaxStages = 8;
constexpr int kThreads = 192;
constexpr int kProducerWarp = 4;
constexpr int kMmaWarp = 5;
constexpr int kTermThreads = 256;
constexpr int kMinExp = -100;               // of a block's scale: all the terms' scales are E8M0 then

// Groups of scales in a block of 256 inputs: a group is what one tcgen05.cp moves,
// four bytes (128 inputs at one scale per 32, 64 at one per 16) of 128 rows.
__host__ __device__ constexpr int groups(bool e4m3) { return e4m3 ? 4 : 2; }
__host__ __device__ constexpr int group_bytes() { return 512; }
__host__ __device__ constexpr int block_bytes(bool e4m3) { return kDataBytes + groups(e4m3) * group_bytes(); }
// Rows of the second operand (columns of the accumulator) for a tile of tokens.
__host__ __device__ constexpr int columns(int tokens) { return (tokens * kTerms + 15) / 16 * 16; }
__host__ __device__ constexpr int column_groups(int n) { return (n + 127) / 128; }
__host__ __device__ constexpr int terms_bytes(bool e4m3, int n) {
  return n * (kChunk / 2) + groups(e4m3) * column_groups(n) * group_bytes();
}
// Place of the four scale bytes of row r in a group of 128 rows, as tcgen05.cp reads them.
__host__ __device__ constexpr int scale_place(int r) { return (r % 32) * 16 + (r / 32) * 4; }

// ---- weights -------------------------------------------------------------------
// One block of 128 rows x 256 inputs: 16 KiB of codes at their places in a 128-byte
// swizzled operand tile, behind them the scales by groups; block (i, c) of row tile
// i and chunk c is number i * chunks + c. One bulk copy then brings a whole stage of
// the product's pipeline, whatever the matrix's sizes. Rows and inputs that do not
// exist are zeros with scale byte 0.
template <bool kE4M3>
__global__ void weights_kernel(const uint8_t* __restrict__ data, const uint8_t* __restrict__ scale, int32_t n_out,
                               int32_t n_in, int32_t chunks, uint8_t* __restrict__ out) {
  const int32_t c = blockIdx.x % chunks;
  const int64_t row0 = (int64_t)(blockIdx.x / chunks) * kRows;
  uint8_t* block = out + (int64_t)blockIdx.x * block_bytes(kE4M3);
  for (int i = threadIdx.x; i < kRows * 8; i += blockDim.x) {
    const int r = i / 8, at = i % 8;
    const int64_t row = row0 + r;
    const int32_t k = c * kChunk + at * 32;
    uint4 v = make_uint4(0, 0, 0, 0);
    if (row < n_out && k < n_in) v = *reinterpret_cast<const uint4*>(data + row * (n_in / 2) + k / 2);
    *reinterpret_cast<uint4*>(block + tc::sw128_offset(r, at)) = v;
  }
  constexpr int kPer = kE4M3 ? 16 : 32;  // inputs to a scale
  constexpr int kOfRow = kChunk / kPer;
  for (int i = threadIdx.x; i < kRows * kOfRow; i += blockDim.x) {
    const int r = i / kOfRow, at = i % kOfRow;
    const int64_t row = row0 + r;
    const int32_t k = c * kChunk + at * kPer;
    uint8_t v = 0;
    if (row < n_out && k < n_in) v = scale[row * (n_in / kPer) + k / kPer];
    block[kDataBytes + (at / 4) * group_bytes() + scale_place(r) + at % 4] = v;
  }
}

// ---- the rows' terms -------------------------------------------------------------

__device__ __forceinline__ uint32_t max_halves(uint32_t a, uint32_t b) { return __vmaxu2(a, b); }

// The exponent e of the scale of a block whose largest magnitude has these bf16 bits.
__device__ __forceinline__ int scale_exp(uint32_t bits) {
  const int e = (int)(bits >> 7) - 127 - 2 + ((bits & 0x60u) == 0x60u ? 1 : 0);
  return e < kMinExp ? kMinExp : e;
}

__device__ __forceinline__ float2 e2m1x2_to_f32x2(uint32_t byte) {
  uint32_t h;
  asm("{\n\t.reg .b8 t;\n\tcvt.u8.u32 t, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, t;\n\t}" : "=r"(h) : "r"(byte));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

struct TermArgs {
  const uint16_t* x;
  int32_t T, n_in, chunks, n, slices;
  uint8_t* terms;
  float* factor;
};

// One CTA takes 2,048 channels of a token, eight to a thread. With E4M3 scales the
// terms' scales are powers of two relative to the row's own (2^-9 .. 2^8 relative to
// 2^-8 of the row's largest block scale; a block below that takes the smallest), and
// term j counts 2^(1-3j) of term 0: both are put back behind the product, the first as
// the token's factor. With E8M0 scales they stand in the scale bytes themselves. A
// row with an infinity or a NaN has the factor NaN.
template <bool kE4M3>
__global__ void __launch_bounds__(kTermThreads) terms_kernel(TermArgs a) {
  pdl_begin();
  __shared__ uint32_t s_max[kTermThreads / 32];
  const int32_t t = blockIdx.x / a.slices, slice = blockIdx.x % a.slices;
  const uint16_t* row = a.x + (int64_t)t * a.n_in;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t k = ((int64_t)slice * kTermThreads + threadIdx.x) * 8;

  uint32_t top2 = 0;
  for (int64_t i = (int64_t)threadIdx.x * 8; i < a.n_in; i += kTermThreads * 8) {
    const uint4 v = *reinterpret_cast<const uint4*>(row + i);
    top2 = max_halves(top2, max_halves(max_halves(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu),
                                       max_halves(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu)));
  }
  uint32_t top = max(top2 & 0xFFFFu, top2 >> 16);
  top = __reduce_max_sync(0xffffffffu, top);
  if (lane == 0) s_max[warp] = top;
  __syncthreads();
  top = s_max[0];
#pragma unroll
  for (int i = 1; i < kTermThreads / 32; ++i) top = max(top, s_max[i]);
  const int row_exp = scale_exp(top) - 8;
  if (slice == 0 && threadIdx.x == 0)
    a.factor[t] = top >= 0x7F80u ? __uint_as_float(0x7FC00000u)
                  : kE4M3 ? __uint_as_float((uint32_t)(row_exp + 127) << 23) : 1.0f;

  const int32_t c = (int32_t)(k / kChunk);
  if (c >= a.chunks) return;  // (whole warps: a warp has one chunk)
  uint4 v = make_uint4(0, 0, 0, 0);
  if (k < a.n_in) v = *reinterpret_cast<const uint4*>(row + k);
  uint32_t m2 = max_halves(max_halves(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu),
                           max_halves(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu));
  uint32_t m = max(m2 & 0xFFFFu, m2 >> 16);
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
  if (!kE4M3) m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
  int e = scale_exp(m);
  if (kE4M3) e = max(e, row_exp - 9);
  // (a row that is not finite: any terms do)
  e = min(e, 126);
  const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
  float r[8];
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    r[2 * i] = bf16_bits_to_f32((uint16_t)(w[i] & 0xFFFFu)) * inv;
    r[2 * i + 1] = bf16_bits_to_f32((uint16_t)(w[i] >> 16)) * inv;
  }
  const int tl = t % kTileTokens;
  uint8_t* block = a.terms + ((int64_t)(t / kTileTokens) * a.chunks + c) * terms_bytes(kE4M3, a.n);
  uint8_t* scales = block + a.n * (kChunk / 2);
  const int at = lane;  // 8 channels = 4 bytes of the row's 128
  constexpr int kLanesPer = kE4M3 ? 2 : 4;
  const int s_at = lane / kLanesPer;  // scale of the row: group s_at / 4, byte s_at % 4
  uint32_t s_code;
  if (kE4M3) {
    const int rel = e - row_exp;  // -9 .. 8
    s_code = rel >= -6 ? (uint32_t)(rel + 7) << 3 : 1u << (rel + 9);
  }
#pragma unroll
  for (int j = 0; j < kTerms; ++j) {
    const uint32_t codes = cvt_e2m1x8(r);
    const float up = j == 0 ? 4.0f : 8.0f;  // the next grid
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 q = e2m1x2_to_f32x2((codes >> (8 * i)) & 0xFFu);
      r[2 * i] = (r[2 * i] - q.x) * up;
      r[2 * i + 1] = (r[2 * i + 1] - q.y) * up;
    }
    const int n = tl * kTerms + j;
    *reinterpret_cast<uint32_t*>(block + tc::sw128_offset(n, at / 4) + (at % 4) * 4) = codes;
    if (!kE4M3) s_code = (uint32_t)(e + 127 - (j == 0 ? 0 : 3 * j - 1));
    if (lane % kLanesPer == 0)
      scales[((s_at / 4) * column_groups(a.n) + n / 128) * group_bytes() + scale_place(n % 128) + s_at % 4] =
          (uint8_t)s_code;
  }
}

// ---- the product -----------------------------------------------------------------

struct Params {
  const uint8_t* weights;
  const uint8_t* terms;
  const float* factor;
  __nv_bfloat16* out_bf16;
  float* out_f32;
  float scale;
  int32_t T, n_out, chunks, token_tiles, n, stages, cluster;
  uint32_t tmem_cols;
};

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t peer(uint32_t addr, int rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ float ld_peer(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

constexpr int kHeadBytes = 256;  // barriers and words ahead of the ring's 1,024-byte boundary

// One CTA: 128 outputs x a tile of tokens x a range of chunks. A cluster's CTAs
// share the chunks of one tile; each sums its range, and their sums are added in
// rank order out of one another's shared memory.
//   warp 4     producer: one bulk copy of a block of weights and one of the terms
//              per stage; the first stages' weights before the terms are ready;
//   warp 5     scales to tensor memory, four products of K = 64 a stage;
//   warps 0-3  the tokens' eight columns summed, stored.
template <bool kE4M3, int kCtas>
__global__ void __launch_bounds__(kThreads, kCtas) linear_kernel(Params p) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = tc::smem_u32(smem_raw);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem_raw);
  uint64_t* empty = full + kMaxStages;
  uint64_t* acc_full = empty + kMaxStages;
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(acc_full + 1);
  volatile int* s_abort = reinterpret_cast<volatile int*>(s_tmem + 1);
  uint8_t* ring = smem_raw + (((raw + kHeadBytes + 1023u) & ~1023u) - raw);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)(blockIdx.x % (uint32_t)p.cluster);
  const int64_t tile = blockIdx.x / (uint32_t)p.cluster;
  const int32_t token_tile = (int32_t)(tile % p.token_tiles);
  const int64_t row_tile = tile / p.token_tiles;
  const int32_t c0 = (int32_t)((int64_t)p.chunks * rank / p.cluster);
  const int32_t n_chunks = (int32_t)((int64_t)p.chunks * (rank + 1) / p.cluster) - c0;
  const int blk_b = terms_bytes(kE4M3, p.n);
  const int stage_bytes = block_bytes(kE4M3) + blk_b;

  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      tc::mbar_init(&full[s], 1);
      tc::mbar_init(&empty[s], 1);
    }
    tc::mbar_init(acc_full, 1);
    *s_abort = 0;
    tc::fence_mbar_init();
  }
  if (warp == kMmaWarp) tc::tmem_alloc(s_tmem, p.tmem_cols);
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = *s_tmem;

  if (warp == kProducerWarp) {
    if (lane == 0) {
      const uint8_t* wsrc = p.weights + (row_tile * p.chunks + c0) * block_bytes(kE4M3);
      const uint8_t* tsrc = p.terms + ((int64_t)token_tile * p.chunks + c0) * blk_b;
      const int ahead = n_chunks < p.stages ? n_chunks : p.stages;
      for (int i = 0; i < ahead; ++i) {
        tc::mbar_arrive_expect_tx(&full[i], (uint32_t)stage_bytes);
        tc::bulk_load(ring + i * stage_bytes, wsrc + (int64_t)i * block_bytes(kE4M3), block_bytes(kE4M3), &full[i]);
      }
      pdl_wait();
      for (int i = 0; i < ahead; ++i)
        tc::bulk_load(ring + i * stage_bytes + block_bytes(kE4M3), tsrc + (int64_t)i * blk_b, (uint32_t)blk_b, &full[i]);
      int issued = ahead;
      for (; issued < n_chunks; ++issued) {
        const int s = issued % p.stages;
        if (!tc::mbar_wait_bounded(&empty[s], ((uint32_t)(issued / p.stages) & 1u) ^ 1u, s_abort, &g_linear_error)) break;
        tc::mbar_arrive_expect_tx(&full[s], (uint32_t)stage_bytes);
        tc::bulk_load(ring + s * stage_bytes, wsrc + (int64_t)issued * block_bytes(kE4M3), block_bytes(kE4M3), &full[s]);
        tc::bulk_load(ring + s * stage_bytes + block_bytes(kE4M3), tsrc + (int64_t)issued * blk_b, (uint32_t)blk_b,
                      &full[s]);
      }
      // copies land before the CTA's memory goes away
      for (int i = max(0, issued - p.stages); i < issued; ++i)
        tc::mbar_wait_issued(&full[i % p.stages], (uint32_t)(i / p.stages));
    }
    __syncwarp();
  } else if (warp == kMmaWarp) {
    const uint32_t one = tc::elect_one();
    const uint32_t ring_at = tc::smem_u32(ring);
    const int nh = column_groups(p.n);
    constexpr int kG = groups(kE4M3);
    const uint32_t sf_cols = (uint32_t)(kG * 4 * (1 + nh));  // scale columns of a stage
    const uint32_t idesc = kE4M3 ? tc::idesc_nvf4(128, p.n) : tc::idesc_mxf4(128, p.n, 0, 0);
    int done = 0;
    for (; done < n_chunks; ++done) {
      const int s = done % p.stages;
      const bool ok = tc::mbar_wait_bounded(&full[s], (uint32_t)(done / p.stages) & 1u, s_abort, &g_linear_error);
      if (!__all_sync(0xffffffffu, ok)) break;
      tc::tc_fence_after();
      const uint32_t a_at = ring_at + (uint32_t)(s * stage_bytes);
      const uint32_t b_at = a_at + block_bytes(kE4M3);
      // The stage's own scale columns: they are written again only when its barrier
      // says that the products that read them are done.
      const uint32_t sfa = tmem + (uint32_t)p.n + (uint32_t)s * sf_cols, sfb = sfa + kG * 4;
      for (int g = 0; g < kG; ++g)
        tc::tmem_cp_32x128_x4_one(one, sfa + 4 * g,
                                  tc::smem_desc(a_at + kDataBytes + g * group_bytes(), 0, 128, tc::kSwizzleNone));
      for (int g = 0; g < kG * nh; ++g)
        tc::tmem_cp_32x128_x4_one(one, sfb + 4 * g,
                                  tc::smem_desc(b_at + p.n * (kChunk / 2) + g * group_bytes(), 0, 128, tc::kSwizzleNone));
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        const int g = kE4M3 ? m : m / 2;
        const uint32_t id = kE4M3 ? 0u : (uint32_t)(m % 2) * 2;  // two products share a group's four bytes
        tc::mma_fp4_one<kE4M3>(one, tmem, tc::smem_desc(a_at + 32 * m, 0, 1024, tc::kSwizzle128B),
                               tc::smem_desc(b_at + 32 * m, 0, 1024, tc::kSwizzle128B), idesc | id << 4 | id << 29,
                               sfa + 4 * g, sfb + 4 * g * nh, (done | m) != 0);
      }
      tc::mma_commit_one(one, &empty[s]);
    }
    // whatever was issued ends before tensor memory is freed
    tc::mma_commit_one(one, acc_full);
    tc::mbar_wait_issued(acc_full, 0);
    __syncwarp();
  }

  // ---- epilogue ----
  const int32_t t0 = token_tile * kTileTokens;
  const int nt = p.T - t0 < kTileTokens ? p.T - t0 : kTileTokens;
  float* part = reinterpret_cast<float*>(ring);  // [nt][128], once the ring is done with
  if (warp < 4) {
    bool ok = tc::mbar_wait_bounded(acc_full, 0, s_abort, &g_linear_error);
    ok = __all_sync(0xffffffffu, ok) && !*s_abort;
    ok = __all_sync(0xffffffffu, ok);
    pdl_wait();  // the factors; and the outputs may have readers before this call
    if (ok) {
      tc::tc_fence_after();
      const int row = warp * 32 + lane;
      const int64_t out_row = row_tile * kRows + row;
      for (int t = 0; t < nt; t += 2) {
        uint32_t r[16];
        tc::tmem_ld_32x32b_x16(tmem + ((uint32_t)(warp * 32) << 16) + (uint32_t)(t * kTerms), r);
        tc::tmem_ld_wait();
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (t + h >= nt) break;
          float y = __uint_as_float(r[8 * h + 7]);
          if (kE4M3) {
#pragma unroll
            for (int j = 6; j >= 0; --j) y = fmaf(y, j == 0 ? 0.25f : 0.125f, __uint_as_float(r[8 * h + j]));
          } else {
#pragma unroll
            for (int j = 6; j >= 0; --j) y += __uint_as_float(r[8 * h + j]);
          }
          y *= p.factor[t0 + t + h];
          if (p.cluster > 1) {
            part[(t + h) * kRows + row] = y;
          } else if (out_row < p.n_out) {
            y *= p.scale;
            const int64_t at = (int64_t)(t0 + t + h) * p.n_out + out_row;
            if (p.out_bf16) p.out_bf16[at] = __float2bfloat16_rn(y);
            if (p.out_f32) p.out_f32[at] = y;
          }
        }
      }
      tc::tc_fence_before();
    }
  }
  __syncthreads();
  if (p.cluster > 1) {
    cluster_sync();
    bool ok = true;
    for (int c = 0; c < p.cluster; ++c) ok = ok && __float_as_int(ld_peer(peer(tc::smem_u32((const void*)s_abort), c))) == 0;
    const int per = nt * kRows / p.cluster;
    for (int i = threadIdx.x; ok && i < per; i += kThreads) {
      const int at = rank * per + i;
      const int t = at / kRows, row = at % kRows;
      const uint32_t here = tc::smem_u32(part + at);
      float y = 0.0f;
      for (int c = 0; c < p.cluster; ++c) y += ld_peer(peer(here, c));
      const int64_t out_row = row_tile * kRows + row;
      if (out_row < p.n_out) {
        y *= p.scale;
        const int64_t o = (int64_t)(t0 + t) * p.n_out + out_row;
        if (p.out_bf16) p.out_bf16[o] = __float2bfloat16_rn(y);
        if (p.out_f32) p.out_f32[o] = y;
      }
    }
    cluster_sync();  // the peers have read this CTA's sums
  }
  if (warp == kMmaWarp) tc::tmem_dealloc(tmem, p.tmem_cols);
}

}  // namespace linear
}  // namespace csa2

using namespace csa2;

int csa2_read_and_clear_linear_error(cudaStream_t s) {
  int v = 0, z = 0;
  if (cudaMemcpyFromSymbolAsync(&v, g_linear_error, sizeof(int), 0, cudaMemcpyDeviceToHost, s) != cudaSuccess)
    return CSA2_ERR_CUDA;
  if (cudaMemcpyToSymbolAsync(g_linear_error, &z, sizeof(int), 0, cudaMemcpyHostToDevice, s) != cudaSuccess)
    return CSA2_ERR_CUDA;
  if (cudaStreamSynchronize(s) != cudaSuccess) return CSA2_ERR_CUDA;
  return v;
}

static size_t al256(size_t x) { return (x + 255) / 256 * 256; }

// The sizes both the weights and the product are checked for.
static int check_sizes(int32_t n_out, int32_t n_in, int32_t format) {
  if (n_out < 0 || n_in < 0) return CSA2_ERR_INVALID_ARG;
  if (format != CSA2_FP4_E8M0 && format != CSA2_FP4_E4M3) return CSA2_ERR_INVALID_ARG;
  if (n_in == 0 || n_in % 32) return CSA2_ERR_UNSUPPORTED_SHAPE;
  return CSA2_OK;
}
static int64_t chunks_of(int32_t n_in) { return ((int64_t)n_in + linear::kChunk - 1) / linear::kChunk; }
static int64_t row_tiles_of(int32_t n_out) { return ((int64_t)n_out + linear::kRows - 1) / linear::kRows; }

extern "C" size_t csa2_fp4_weights_size(int32_t n_out, int32_t n_in, int32_t format) {
  if (check_sizes(n_out, n_in, format) != CSA2_OK) return 0;
  return (size_t)row_tiles_of(n_out) * (size_t)chunks_of(n_in) * linear::block_bytes(format == CSA2_FP4_E4M3);
}

extern "C" int csa2_fp4_weights(const uint8_t* data, const uint8_t* scale, int32_t n_out, int32_t n_in, int32_t format,
                                uint8_t* weights, csa2_stream_t stream) {
  int rc = check_sizes(n_out, n_in, format);
  if (rc) return rc;
  const int64_t blocks = row_tiles_of(n_out) * chunks_of(n_in);
  if (blocks > 0x7FFFFFFFLL) return CSA2_ERR_UNSUPPORTED_SHAPE;
  if (n_out == 0) return CSA2_OK;
  if (!data || !scale || !weights) return CSA2_ERR_INVALID_ARG;
  if (!csa2_aligned(data, 16) || !csa2_aligned(weights, 16)) return CSA2_ERR_ALIGNMENT;
  if (format == CSA2_FP4_E4M3)
    linear::weights_kernel<true><<<(unsigned)blocks, 256, 0, (cudaStream_t)stream>>>(data, scale, n_out, n_in,
                                                                                     (int32_t)chunks_of(n_in), weights);
  else
    linear::weights_kernel<false><<<(unsigned)blocks, 256, 0, (cudaStream_t)stream>>>(data, scale, n_out, n_in,
                                                                                      (int32_t)chunks_of(n_in), weights);
  CSA2_CHECK_LAUNCH();
  return CSA2_OK;
}

// Tokens of the (only or full) tiles: their columns are the workspace's and the product's.
static int tile_columns(int32_t n_tokens) {
  return linear::columns(n_tokens < linear::kTileTokens ? n_tokens : linear::kTileTokens);
}
static int64_t token_tiles_of(int32_t n_tokens) {
  return ((int64_t)n_tokens + linear::kTileTokens - 1) / linear::kTileTokens;
}

extern "C" size_t csa2_fp4_linear_workspace_size(int32_t n_tokens, int32_t n_in, int32_t format) {
  if (n_tokens <= 0 || check_sizes(1, n_in, format) != CSA2_OK) return 0;
  const size_t terms = (size_t)token_tiles_of(n_tokens) * (size_t)chunks_of(n_in) *
                       linear::terms_bytes(format == CSA2_FP4_E4M3, tile_columns(n_tokens));
  return al256((size_t)n_tokens * sizeof(float)) + al256(terms);
}

template <bool kE4M3>
static int launch_linear(const void* x, int32_t T, const uint8_t* weights, int32_t n_out, int32_t n_in, float scale,
                         void* out_bf16, float* out_f32, void* workspace, cudaStream_t stream) {
  using namespace linear;
  float* factor = (float*)workspace;
  uint8_t* terms = (uint8_t*)workspace + al256((size_t)T * sizeof(float));
  const int n = tile_columns(T);
  const int64_t chunks = chunks_of(n_in), token_tiles = token_tiles_of(T), tiles = row_tiles_of(n_out) * token_tiles;
  const int64_t slices = ((int64_t)n_in + kTermThreads * 8 - 1) / (kTermThreads * 8);
  TermArgs ta{(const uint16_t*)x, T, n_in, (int32_t)chunks, n, (int32_t)slices, terms, factor};
  CSA2_LAUNCH_PDL(terms_kernel<kE4M3>, dim3((unsigned)(T * slices)), dim3(kTermThreads), (size_t)0, stream, ta);

  const bool two = n <= 64;  // two CTAs to an SM
  const int stage = block_bytes(kE4M3) + terms_bytes(kE4M3, n);
  const int room = (two ? 113 : 226) * 1024 - kHeadBytes - 1024;
  const int sf_cols = groups(kE4M3) * 4 * (1 + column_groups(n));
  const int cols = two ? 256 : 512;
  int stages = room / stage;
  if (stages > (cols - n) / sf_cols) stages = (cols - n) / sf_cols;
  if (stages > kMaxStages) stages = kMaxStages;
  int cluster = 1;
  while (cluster < 8 && tiles * cluster * 2 <= 304 && cluster * 2 <= chunks) cluster *= 2;
  Params p{weights, terms, factor, (__nv_bfloat16*)out_bf16, out_f32, scale, T, n_out, (int32_t)chunks,
           (int32_t)token_tiles, n, stages, cluster, (uint32_t)cols};
  const int smem = kHeadBytes + 1024 + stages * stage;
  static Csa2PerDeviceOnce once1, once2;
  if (two) {
    if (csa2_smem_optin((const void*)linear_kernel<kE4M3, 2>, 113 * 1024, once2) != CSA2_OK) return CSA2_ERR_CUDA;
    if (csa2_launch_pdl_cluster(linear_kernel<kE4M3, 2>, dim3((unsigned)(tiles * cluster)), dim3(kThreads), (size_t)smem,
                                stream, (unsigned)cluster, p) == cudaSuccess)
      return CSA2_OK;
  } else {
    if (csa2_smem_optin((const void*)linear_kernel<kE4M3, 1>, 226 * 1024, once1) != CSA2_OK) return CSA2_ERR_CUDA;
    if (csa2_launch_pdl_cluster(linear_kernel<kE4M3, 1>, dim3((unsigned)(tiles * cluster)), dim3(kThreads), (size_t)smem,
                                stream, (unsigned)cluster, p) == cudaSuccess)
      return CSA2_OK;
  }
  (void)cudaGetLastError();
  return CSA2_ERR_CUDA;
}

extern "C" int csa2_fp4_linear(const void* x_bf16, int32_t n_tokens, const uint8_t* weights, int32_t n_out, int32_t n_in,
                               int32_t format, float scale, void* out_bf16, float* out_f32, void* workspace,
                               size_t workspace_bytes, csa2_stream_t stream) {
  if (n_tokens < 0) return CSA2_ERR_INVALID_ARG;
  int rc = check_sizes(n_out, n_in, format);
  if (rc) return rc;
  if (n_tokens == 0 || n_out == 0) return CSA2_OK;
  if (!x_bf16 || !weights || (!out_bf16 && !out_f32)) return CSA2_ERR_INVALID_ARG;
  if (!csa2_aligned(x_bf16, 16) || !csa2_aligned(weights, 16) || !csa2_aligned(out_bf16, 2) || !csa2_aligned(out_f32, 4))
    return CSA2_ERR_ALIGNMENT;
  // a grid of at most 2^31 - 1 blocks for each kernel
  if (row_tiles_of(n_out) * token_tiles_of(n_tokens) > 0x0FFFFFFFLL ||
      (int64_t)n_tokens * (((int64_t)n_in + 2047) / 2048) > 0x7FFFFFFFLL)
    return CSA2_ERR_UNSUPPORTED_SHAPE;
  const size_t need = csa2_fp4_linear_workspace_size(n_tokens, n_in, format);
  if (!workspace || workspace_bytes < need || !csa2_aligned(workspace, 256)) return CSA2_ERR_WORKSPACE;
  return format == CSA2_FP4_E4M3 ? launch_linear<true>(x_bf16, n_tokens, weights, n_out, n_in, scale, out_bf16, out_f32,
                                                       workspace, (cudaStream_t)stream)
                                 : launch_linear<false>(x_bf16, n_tokens, weights, n_out, n_in, scale, out_bf16, out_f32,
                                                        workspace, (cudaStream_t)stream);
}
