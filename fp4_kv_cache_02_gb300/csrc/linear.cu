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
// vectors, the digits of its channels in base 8. With 2^E the leading power of two of
// a block's largest channel, each channel is rounded to a multiple of 2^(E-21): off by
// at most 2^-22 of the largest, and by nothing within 2^-14 of it, where all eight
// bits of a bf16 lie on that grid. The multiple, below 2^22, has eight digits of
// -4 .. 3, and those times 1/2 are E2M1 values, whose code is the digit's sign and
// magnitude; the scales of the eight vectors are 2^(E+1), 2^(E-2) .. 2^(E-20). The terms
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
constexpr int kTermTokens = 64;             // tokens that enter as terms
constexpr int kFewTokens = 3;               // tokens whose terms the product's own warps make
constexpr int kMaxSplit = 8;                // CTAs that split the inputs of such a product
constexpr int kStreamCtas = 152;            // of a product of more tokens: one to an SM
constexpr int kMaxStages = 8;
constexpr int kSumWarps = 8;                // warps that make terms and sum columns
constexpr int kProducerWarp = kSumWarps;
constexpr int kMmaWarp = kSumWarps + 1;
constexpr int kThreads = 32 * (kSumWarps + 2);
constexpr int kTermThreads = 256;           // of terms_kernel, eight channels each
constexpr int kFactorThreads = 1024;        // of factors_kernel
constexpr int kLongSlices = 16;             // CTAs to a token's terms above which it goes ahead of them
constexpr int kMinExp = -100;               // of a block's largest: all the terms' scales are E8M0 then

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

// The exponent E of a block whose largest magnitude has these bf16 bits.
__device__ __forceinline__ int block_exp(uint32_t bits) {
  const int e = (int)(bits >> 7) - 127;
  return e < kMinExp ? kMinExp : e;
}

// The largest magnitude's bf16 bits of eight channels.
__device__ __forceinline__ uint32_t top_bits(uint4 v) {
  const uint32_t m2 = max_halves(max_halves(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu),
                                 max_halves(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu));
  return max(m2 & 0xFFFFu, m2 >> 16);
}

// The terms' scales are held relative to a power of two, 2^base, put back behind the
// product as the token's factor. With E8M0 scales base is 1: the first scale of a block
// with E = 127 is 2^128. With E4M3 scales it is such that the largest block's first one
// is 2^8, the largest power of two that E4M3 holds, and the terms' common ratios are left
// to sum_terms. A row that holds an infinity or a NaN has NaN for the scales of that block
// (E8M0: the factor is 2 for every token, and none has to be found out: looked up by all
// CTAs, eight words a token, it cost 2 us for 8 tokens by 4,096 x 32,768) or as its factor.
constexpr int kE8M0Base = 1;
__device__ __forceinline__ int base_exp(uint32_t top) { return block_exp(top) - 7; }
__device__ __forceinline__ float factor_of(uint32_t top) {
  return top >= 0x7F80u ? __uint_as_float(0x7FC00000u) : __uint_as_float((uint32_t)(base_exp(top) + 127) << 23);
}

// Base-8 digits (24 bits) one to a nibble; each nibble's highest bit is not defined.
__device__ __forceinline__ uint32_t spread_digits(uint32_t v) {
  v = (v & 0x00000FFFu) | ((v << 4) & ~0x00000FFFu);
  v = (v & 0x00FF00FFu) | ((v << 2) & ~0x00FF00FFu);
  return (v & 0x0F0F0F0Fu) | ((v << 1) & ~0x0F0F0F0Fu);
}
// Eight digits + 4 (0 .. 7, one to a nibble) to E2M1 codes of the digits times 1/2: the
// digit itself from 4 on, else the sign and 4 - digit.
__device__ __forceinline__ uint32_t digit_codes(uint32_t w) {
  w &= 0x77777777u;
  const uint32_t positive = ((w >> 2) & 0x11111111u) * 15u;
  return (positive & w & 0x33333333u) | (~positive & (0xCCCCCCCCu - w));
}

// One warp: the eight terms of a token's chunk of 256 channels, eight channels v to a
// lane, into rows 8 tl .. 8 tl + 7 of the second operand's block. (With a conversion to
// E2M1, one back and a remainder for each term the terms of 1,021 x 4,096 channels took
// 12 us; conversions are a quarter of the rate of other instructions.)
template <bool kE4M3>
__device__ __forceinline__ void put_terms(uint4 v, int base, int tl, uint8_t* data, uint8_t* scales, int nh, int lane) {
  uint32_t m = top_bits(v);
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
  if (!kE4M3) m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
  int e = block_exp(m);
  if (kE4M3) e = max(e, base + 7 - 17);  // (the smallest power of two that E4M3 holds is 2^-9)
  e = min(e, 127);                       // (of a row that is not finite any terms do)
  // x 2^(21-e), |x| < 2^(e+1), to the nearest integer: in the low bits of a sum with
  // 1.5 x 2^23; then eight digits + 4
  const float up = __uint_as_float((uint32_t)(127 + 21 - e) << 23);
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t z[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    z[2 * i] = __float_as_uint(fmaf(__uint_as_float(w[i] << 16), up, 12582912.0f));
    z[2 * i + 1] = __float_as_uint(fmaf(__uint_as_float(w[i] & 0xFFFF0000u), up, 12582912.0f));
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) z[i] = spread_digits((z[i] - 0x4B400000u + 044444444u) & 0xFFFFFFu);
  // channel i's digits 0 .. 7 -> digit d of the eight channels: halves, bytes, nibbles
  uint32_t h[8], b[8], d[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    h[i] = __byte_perm(z[i], z[i + 4], 0x5410);      // digits 0 .. 3
    h[i + 4] = __byte_perm(z[i], z[i + 4], 0x7632);  // digits 4 .. 7
  }
#pragma unroll
  for (int i = 0; i < 8; i += 4)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      b[i + j] = __byte_perm(h[i + j], h[i + j + 2], 0x6240);      // digits i, i + 1 of channels j, j + 2, ..
      b[i + j + 2] = __byte_perm(h[i + j], h[i + j + 2], 0x7351);  // digits i + 2, i + 3
    }
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    d[i] = (b[i] & 0x0F0F0F0Fu) | ((b[i + 1] << 4) & 0xF0F0F0F0u);
    d[i + 1] = ((b[i] >> 4) & 0x0F0F0F0Fu) | (b[i + 1] & 0xF0F0F0F0u);
  }
  constexpr int kLanesPer = kE4M3 ? 2 : 4;
  const int s_at = lane / kLanesPer;  // scale of the row: group s_at / 4, byte s_at % 4
  const int n0 = tl * kTerms;         // (eight rows lie in one group of 32)
  uint8_t* s_to = scales + ((s_at / 4) * nh + n0 / 128) * group_bytes() + scale_place(n0 % 128) + s_at % 4;
  const int rel = e + 1 - base;  // of the first term's scale; E4M3: -9 .. 8
  const uint32_t e4m3 = rel >= -6 ? (uint32_t)(rel + 7) << 3 : 1u << ((rel + 9) & 31);
  uint8_t* to = data + n0 * (kChunk / 2) + (lane % 4) * 4;
#pragma unroll
  for (int j = 0; j < kTerms; ++j) {
    *reinterpret_cast<uint32_t*>(to + tc::sw128_offset(j, lane / 4)) = digit_codes(d[7 - j]);
    if (lane % kLanesPer == 0) s_to[16 * j] = (uint8_t)(kE4M3 ? e4m3 : m >= 0x7F80u ? 0xFFu : (uint32_t)(rel + 127 - 3 * j));
  }
}

struct TermArgs {
  const uint16_t* x;
  int32_t T, n_in, chunks, n, slices;
  bool known;  // the factors are there
  uint8_t* terms;
  float* factor;
  int32_t* joined;
};

// E4M3: the factors of tokens of more than 32,768 inputs, a CTA to a token, ahead of their
// terms, every CTA of which would look at the whole row otherwise: work that grows with the
// square of the inputs (a product's time, 512 outputs: 64 tokens of 32,768 inputs 20.3 us so,
// 20.7 otherwise, but 8 of them 13.8 and 12.8; 2 and 64 of 65,536 18.2 and 29.3 so, 19.6 and
// 39.0 otherwise; 64 of 262,144 93 and 245).
__global__ void __launch_bounds__(kFactorThreads) factors_kernel(const uint16_t* x, int32_t n_in, float* factor) {
  pdl_begin();
  __shared__ uint32_t s_max[kFactorThreads / 32];
  const uint16_t* row = x + (int64_t)blockIdx.x * n_in;
  uint32_t top = 0;
#pragma unroll 8
  for (int64_t i = (int64_t)threadIdx.x * 8; i < n_in; i += kFactorThreads * 8)
    top = max(top, top_bits(*reinterpret_cast<const uint4*>(row + i)));
  top = __reduce_max_sync(0xffffffffu, top);
  if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = top;
  __syncthreads();
  if (threadIdx.x >= 32) return;
  top = __reduce_max_sync(0xffffffffu, s_max[threadIdx.x]);
  if (threadIdx.x == 0) factor[blockIdx.x] = factor_of(top);
}

// The terms of all tokens, ahead of the product: eight channels of a token to a thread.
// With E4M3 scales every CTA of a token looks at its whole row for its base, unless that is
// long. (With half as many CTAs of twice the threads 8 tokens by 4,096 x 4,096, E4M3, took
// 7.2 us, so 6.9; with twice as many of 128 6.8, but by 4,096 x 32,768 21.1 and 19.5.)
template <bool kE4M3>
__global__ void __launch_bounds__(kTermThreads) terms_kernel(TermArgs a) {
  pdl_begin();
  static_assert(kTermThreads >= kStreamCtas, "a count to a thread");
  if (blockIdx.x == 0 && threadIdx.x < kStreamCtas) a.joined[threadIdx.x] = 0;
  const int32_t t = blockIdx.x / a.slices, slice = blockIdx.x % a.slices;
  const uint16_t* row = a.x + (int64_t)t * a.n_in;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t k = ((int64_t)slice * kTermThreads + threadIdx.x) * 8;
  const uint4 v = k < a.n_in ? *reinterpret_cast<const uint4*>(row + k) : make_uint4(0, 0, 0, 0);
  int base = kE8M0Base;
  if (kE4M3 && a.known) {
    base = (int)(__float_as_uint(__ldcg(a.factor + t)) >> 23) - 127;
  } else if constexpr (kE4M3) {
    __shared__ uint32_t s_max[kTermThreads / 32];
    uint32_t top = top_bits(v);
    if (a.slices > 1)
#pragma unroll 4
      for (int64_t i = (int64_t)threadIdx.x * 8; i < a.n_in; i += kTermThreads * 8)
        top = max(top, top_bits(*reinterpret_cast<const uint4*>(row + i)));
    top = __reduce_max_sync(0xffffffffu, top);
    if (lane == 0) s_max[warp] = top;
    __syncthreads();
    top = s_max[0];
#pragma unroll
    for (int i = 1; i < kTermThreads / 32; ++i) top = max(top, s_max[i]);
    if (threadIdx.x == 0 && slice == 0) a.factor[t] = factor_of(top);
    base = base_exp(top);
  }
  const int32_t c = (int32_t)(k / kChunk);  // (a warp has one chunk)
  if (c >= a.chunks) return;
  uint8_t* block = a.terms + ((int64_t)(t / kTileTokens) * a.chunks + c) * terms_bytes(kE4M3, a.n);
  put_terms<kE4M3>(v, base, t % kTileTokens, block, block + a.n * (kChunk / 2), column_groups(a.n), lane);
}

// ---- the product -----------------------------------------------------------------

// Block (row tile, chunk) of the weights, (token tile, chunk) of the terms: number
// tile * chunks + chunk.
struct Params {
  const uint8_t* weights;
  const uint16_t* x;
  const uint8_t* terms;
  const float* factor;  // [tokens], with E4M3 scales
  int32_t* joined;  // stream_kernel: parts that are there of the tile that CTA g is the first to have a part of
  float* parts;     // stream_kernel: [CTA][2][tokens of a tile][128]
  __nv_bfloat16* out_bf16;
  float* out_f32;
  float scale;
  int32_t T, n_out, n_in, chunks, token_tiles, n, stages, split;
  int64_t units;          // tiles x chunks
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
__device__ __forceinline__ float4 ld_peer4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void sync_sum_warps() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

constexpr int kHeadBytes = 512;  // barriers and words ahead of the ring's 1,024-byte boundary

__device__ __forceinline__ uint8_t* ring_of(uint8_t* smem) {
  const uint32_t raw = tc::smem_u32(smem);
  return smem + (((raw + kHeadBytes + 1023u) & ~1023u) - raw);
}

// A stage's scales to its own columns of tensor memory (written again only when the
// stage's barrier says that the products that read them are done), and its four products.
// By a converged warp.
template <bool kE4M3>
__device__ __forceinline__ void stage_products(uint32_t one, uint32_t a_at, uint32_t b_at, int n, uint32_t acc, uint32_t sfa,
                                               uint32_t idesc, bool add) {
  constexpr int kG = groups(kE4M3);
  const int nh = column_groups(n);
  const uint32_t sfb = sfa + kG * 4;
  for (int g = 0; g < kG; ++g)
    tc::tmem_cp_32x128_x4_one(one, sfa + 4 * g,
                              tc::smem_desc(a_at + kDataBytes + g * group_bytes(), 0, 128, tc::kSwizzleNone));
  for (int g = 0; g < kG * nh; ++g)
    tc::tmem_cp_32x128_x4_one(one, sfb + 4 * g,
                              tc::smem_desc(b_at + n * (kChunk / 2) + g * group_bytes(), 0, 128, tc::kSwizzleNone));
#pragma unroll
  for (int m = 0; m < 4; ++m) {
    const int g = kE4M3 ? m : m / 2;
    const uint32_t id = kE4M3 ? 0u : (uint32_t)(m % 2) * 2;  // two products share a group's four bytes
    tc::mma_fp4_one<kE4M3>(one, acc, tc::smem_desc(a_at + 32 * m, 0, 1024, tc::kSwizzle128B),
                           tc::smem_desc(b_at + 32 * m, 0, 1024, tc::kSwizzle128B), idesc | id << 4 | id << 29, sfa + 4 * g,
                           sfb + 4 * g * nh, add || m);
  }
}
template <bool kE4M3>
__device__ __forceinline__ uint32_t idesc_of(int n) {
  return kE4M3 ? tc::idesc_nvf4(128, n) : tc::idesc_mxf4(128, n, 0, 0);
}
// Scale columns of a stage.
__host__ __device__ constexpr int scale_cols(bool e4m3, int n) { return groups(e4m3) * 4 * (1 + column_groups(n)); }

// Tokens of a sum warp: half of a tile's, in fours, at most 16.
__device__ __forceinline__ int tokens_of_warp(int n) { return (n / kTerms / 2 + 3) / 4 * 4; }

// A token's eight columns.
template <bool kE4M3>
__device__ __forceinline__ float sum_terms(const uint32_t* v) {
  float y = __uint_as_float(v[7]);
#pragma unroll
  for (int j = 6; j >= 0; --j)
    y = kE4M3 ? fmaf(y, 0.125f, __uint_as_float(v[j])) : y + __uint_as_float(v[j]);
  return y;
}

// Token t's factor out of its lane.
template <bool kE4M3>
__device__ __forceinline__ float factor_from(float lanes, int t) {
  return kE4M3 ? __shfl_sync(0xffffffffu, lanes, t & 31) : (float)(1 << kE8M0Base);
}

__device__ __forceinline__ void put_out(const Params& p, int64_t t, int64_t row, float y) {
  if (row >= p.n_out) return;
  y *= p.scale;
  if (p.out_bf16) p.out_bf16[t * p.n_out + row] = __float2bfloat16_rn(y);
  if (p.out_f32) p.out_f32[t * p.n_out + row] = y;
}

// Behind a cluster's barrier: this CTA's share of the tile's sums [nt][128], added in rank
// order out of the shared memory of the CTAs that have a part of it (a power of two).
__device__ __forceinline__ void add_parts(const Params& p, const float* sums, int part, int nt, int64_t t0, int64_t row_tile) {
  const int per = nt * kRows / p.split;
  for (int i = threadIdx.x * 4; i < per; i += blockDim.x * 4) {
    const int at = part * per + i;
    const uint32_t here = tc::smem_u32(sums + at);
    float4 v[kMaxSplit];
#pragma unroll
    for (int c = 0; c < kMaxSplit; ++c)
      if (c < p.split) v[c] = ld_peer4(peer(here, c));
    float4 y = v[0];
#pragma unroll
    for (int c = 1; c < kMaxSplit; ++c)
      if (c < p.split) y.x += v[c].x, y.y += v[c].y, y.z += v[c].z, y.w += v[c].w;
    const int64_t t = t0 + at / kRows, r = row_tile * kRows + at % kRows;
    put_out(p, t, r, y.x), put_out(p, t, r + 1, y.y), put_out(p, t, r + 2, y.z), put_out(p, t, r + 3, y.w);
  }
}

// ---- few tiles -------------------------------------------------------------------
// Products of too few tiles (128 outputs x up to 32 tokens) to fill the SMs, and those
// of few tokens. The CTAs of a cluster split a tile's chunks, and their sums are added in
// rank order out of one another's shared memory. kOwnTerms: up to three tokens, whose terms
// each CTA makes itself: ahead of the product they would cost a launch and a trip through
// L2 (4 us of 15 for a token by 32,768 x 4,096 weights).
//   warp 8     producer: a bulk copy of a block of weights per stage (and one of the
//              terms); behind terms ahead the first weights before those are waited for
//              (weights that nobody waited for would gain nothing: a token by 4,096 x 640
//              4.9 us either way, by 4,096 x 32,768 14.0);
//   warp 9     scales to tensor memory, products;
//   warps 0-7  kOwnTerms: the terms, a (chunk, token) to a warp; then the columns summed
//              (a quarter of the rows, half of the tokens each), stored.
template <bool kE4M3, bool kOwnTerms, int kCtas>
__global__ void __launch_bounds__(kThreads, kCtas) split_kernel(Params p) {
  extern __shared__ uint8_t smem_raw[];
  uint64_t* full = reinterpret_cast<uint64_t*>(smem_raw);
  uint64_t* empty = full + kMaxStages;
  uint64_t* ready = empty + kMaxStages;  // kOwnTerms: the stage's terms are there
  uint64_t* acc_full = ready + kMaxStages;
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(acc_full + 1);
  volatile int* s_abort = reinterpret_cast<volatile int*>(s_tmem + 1);
  uint32_t* s_top = s_tmem + 2;  // [warp][token]: the largest channel that the warp has seen
  uint8_t* ring = ring_of(smem_raw);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int part = (int)(blockIdx.x % (uint32_t)p.split);
  const int64_t tile = blockIdx.x / (uint32_t)p.split;
  const int32_t token_tile = (int32_t)(tile % p.token_tiles);
  const int64_t row_tile = tile / p.token_tiles;
  const int32_t t0 = token_tile * kTileTokens;
  const int nt = min(p.T - t0, kTileTokens);
  const int32_t c0 = (int32_t)((int64_t)p.chunks * part / p.split);
  const int32_t n_chunks = (int32_t)((int64_t)p.chunks * (part + 1) / p.split) - c0;
  const int blk_b = terms_bytes(kE4M3, p.n);
  const int stage_bytes = block_bytes(kE4M3) + blk_b;

  const uint8_t* from = p.weights + (row_tile * p.chunks + c0) * block_bytes(kE4M3);
  const auto load_weights = [&](int i, int s) {
    tc::mbar_arrive_expect_tx(&full[s], (uint32_t)(kOwnTerms ? block_bytes(kE4M3) : stage_bytes));
    tc::bulk_load(ring + s * stage_bytes, from + (int64_t)i * block_bytes(kE4M3), block_bytes(kE4M3), &full[s]);
  };
  const int ahead = n_chunks < p.stages ? n_chunks : p.stages;
  if (warp == kProducerWarp && lane == 0) {
    for (int s = 0; s < p.stages; ++s) {
      tc::mbar_init(&full[s], 1);
      tc::mbar_init(&ready[s], p.T);
      tc::mbar_init(&empty[s], 1);
    }
    tc::mbar_init(acc_full, 1);
    *s_abort = 0;
    tc::fence_mbar_init();
    tc::fence_proxy_async_smem();
    // The kernel before may have written the weights. With terms ahead that is their
    // kernel, which lets this one start once it has waited for all that was before it.
    if constexpr (kOwnTerms) pdl_wait();
    for (int i = 0; i < ahead; ++i) load_weights(i, i);
  }
  // kOwnTerms: x is looked at before the set-up is through. With E4M3 scales all of this
  // CTA's channels, for the scales' base.
  const auto channels = [&](int c, int t) {
    const int32_t k = (c0 + c) * kChunk + lane * 8;
    return k < p.n_in ? *reinterpret_cast<const uint4*>(p.x + (int64_t)t * p.n_in + k) : make_uint4(0, 0, 0, 0);
  };
  uint4 ahead_v = make_uint4(0, 0, 0, 0);
  if (kOwnTerms && warp < kSumWarps) {
    pdl_wait();  // x; and the outputs may have readers before this call
    if (kE4M3) {
      uint32_t top[kFewTokens] = {};
      for (int c = warp; c < n_chunks; c += kSumWarps)
#pragma unroll
        for (int t = 0; t < kFewTokens; ++t)
          if (t < p.T) top[t] = max(top[t], top_bits(channels(c, t)));
#pragma unroll
      for (int t = 0; t < kFewTokens; ++t) {
        const uint32_t m = __reduce_max_sync(0xffffffffu, top[t]);
        if (lane == 0) s_top[warp * kFewTokens + t] = m;
      }
    } else if (warp < n_chunks * p.T) {
      ahead_v = channels(warp / p.T, warp % p.T);
    }
  }
  if (warp == kMmaWarp) tc::tmem_alloc(s_tmem, p.tmem_cols);
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = *s_tmem;

  if (warp == kProducerWarp) {
    if (lane == 0) {
      const uint8_t* terms = kOwnTerms ? nullptr : p.terms + ((int64_t)token_tile * p.chunks + c0) * blk_b;
      const auto load_terms = [&](int i, int s) {
        if constexpr (!kOwnTerms)
          tc::bulk_load(ring + s * stage_bytes + block_bytes(kE4M3), terms + (int64_t)i * blk_b, (uint32_t)blk_b, &full[s]);
      };
      if constexpr (!kOwnTerms) pdl_wait();
      for (int i = 0; i < ahead; ++i) load_terms(i, i);
      int issued = ahead;
      for (; issued < n_chunks; ++issued) {
        const int s = issued % p.stages;
        if (!tc::mbar_wait_bounded(&empty[s], ((uint32_t)(issued / p.stages) & 1u) ^ 1u, s_abort, &g_linear_error)) break;
        load_weights(issued, s);
        load_terms(issued, s);
      }
      // copies land before the CTA's memory goes away
      for (int i = max(0, issued - p.stages); i < issued; ++i)
        tc::mbar_wait_issued(&full[i % p.stages], (uint32_t)(i / p.stages));
    }
    __syncwarp();
  } else if (warp == kMmaWarp) {
    const uint32_t one = tc::elect_one();
    const uint32_t ring_at = tc::smem_u32(ring), idesc = idesc_of<kE4M3>(p.n);
    for (int done = 0; done < n_chunks; ++done) {
      const int s = done % p.stages;
      const uint32_t phase = (uint32_t)(done / p.stages) & 1u;
      bool ok = tc::mbar_wait_bounded(&full[s], phase, s_abort, &g_linear_error);
      if (kOwnTerms) ok = ok && tc::mbar_wait_bounded(&ready[s], phase, s_abort, &g_linear_error);
      if (!__all_sync(0xffffffffu, ok)) break;
      tc::tc_fence_after();
      const uint32_t a_at = ring_at + (uint32_t)(s * stage_bytes);
      stage_products<kE4M3>(one, a_at, a_at + block_bytes(kE4M3), p.n, tmem,
                            tmem + (uint32_t)(p.n + s * scale_cols(kE4M3, p.n)), idesc, done != 0);
      tc::mma_commit_one(one, &empty[s]);
    }
    // whatever was issued ends before tensor memory is freed
    tc::mma_commit_one(one, acc_full);
    tc::mbar_wait_issued(acc_full, 0);
    __syncwarp();
  } else {
    if (!kOwnTerms) pdl_wait();  // the factors; and the outputs may have readers before this call
  }
  const auto top_of = [&](int t) {  // kOwnTerms, E4M3
    uint32_t m = s_top[t];
#pragma unroll
    for (int i = 1; i < kSumWarps; ++i) m = max(m, s_top[i * kFewTokens + t]);
    return m;
  };
  if (kOwnTerms && warp < kSumWarps) {
    // No more warps than there are (stage, token) places: a warp's last task is then at
    // most a round of the ring behind its next, so that the stage it waits for is in the
    // phase before the awaited one or later (a barrier tells two phases apart, not three).
    const int n_tasks = n_chunks * p.T, workers = min(kSumWarps, p.stages * p.T);
    for (int i = warp < workers ? warp : n_tasks; i < n_tasks; i += workers) {
      const int c = i / p.T, t = i % p.T, s = c % p.stages;
      const uint4 v = !kE4M3 && i == warp ? ahead_v : channels(c, t);
      const bool ok = tc::mbar_wait_bounded(&empty[s], ((uint32_t)(c / p.stages) & 1u) ^ 1u, s_abort, &g_linear_error);
      if (!__all_sync(0xffffffffu, ok)) break;
      uint8_t* data = ring + s * stage_bytes + block_bytes(kE4M3);
      put_terms<kE4M3>(v, kE4M3 ? base_exp(top_of(t)) : kE8M0Base, t, data, data + p.n * (kChunk / 2), 1, lane);
      tc::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&ready[s]);
    }
  }

  float* sums = reinterpret_cast<float*>(ring);  // [nt][128], once the ring is done with
  if (warp < kSumWarps) {
    // lane t holds token t's factor (asked for one by one they cost a trip to L2 each)
    float factor = 0.0f;
    if (kE4M3 && lane < nt) factor = kOwnTerms ? factor_of(top_of(lane)) : __ldcg(p.factor + t0 + lane);
    const bool ok = __all_sync(0xffffffffu, tc::mbar_wait_bounded(acc_full, 0, s_abort, &g_linear_error));
    if (ok) tc::tc_fence_after();
    const int row = (warp & 3) * 32 + lane;
    const int half = tokens_of_warp(p.n), first = (warp >> 2) * half;
    for (int t = first; t < min(first + half, nt); t += 4) {
      uint32_t v[32];
      if (ok) {
        // (columns past the accumulator hold scales: read, not used)
        tc::tmem_ld_32x32b_x32(tmem + ((uint32_t)((warp & 3) * 32) << 16) + (uint32_t)(t * kTerms), v);
        tc::tmem_ld_wait();
      }
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        const float y = sum_terms<kE4M3>(v + 8 * h) * factor_from<kE4M3>(factor, t + h);
        if (t + h >= min(first + half, nt) || !ok) continue;
        if (p.split > 1)
          sums[(t + h) * kRows + row] = y;
        else
          put_out(p, t0 + t + h, row_tile * kRows + row, y);
      }
    }
    if (ok) tc::tc_fence_before();
  }
  __syncthreads();
  // (before the peers are waited for: of two calls at once neither then waits for tensor
  // memory that the other one's waiting CTAs hold)
  if (warp == kMmaWarp) tc::tmem_dealloc(tmem, p.tmem_cols);
  if (p.split > 1) {
    cluster_sync();
    add_parts(p, sums, part, nt, t0, row_tile);
    cluster_sync();  // the peers have read this CTA's sums
  }
}

// ---- many tiles ------------------------------------------------------------------
// Tiles of 128 outputs x up to 32 tokens. All tiles' chunks form one list (a row tile's
// token tiles one after another, so that its weights are in L2 for them), cut into one
// equal run to an SM. A run begins and ends inside tiles. There are more tiles than runs, so
// that no run is shorter than a tile, and a tile has two parts at most: the CTA that is
// done with its own last adds the other's, out of the workspace (in either order the
// same). Nobody waits for another CTA.
//   warp 8     producer: bulk copies of a block of weights and one of terms per stage,
//              ahead across tiles;
//   warp 9     scales to tensor memory, products; two accumulators up to 16 tokens;
//   warps 0-7  the columns summed (a quarter of the rows, half of the tokens each), the
//              accumulator given back, then stored or joined.
__device__ __forceinline__ int load_acquire(const int* at) {
  int v;
  asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(at) : "memory");
  return v;
}
template <bool kE4M3>
__global__ void __launch_bounds__(kThreads, 1) stream_kernel(Params p) {
  extern __shared__ uint8_t smem_raw[];
  uint64_t* full = reinterpret_cast<uint64_t*>(smem_raw);
  uint64_t* empty = full + kMaxStages;
  uint64_t* acc_full = empty + kMaxStages;
  uint64_t* acc_empty = acc_full + 2;
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(acc_empty + 2);
  volatile int* s_abort = reinterpret_cast<volatile int*>(s_tmem + 1);
  volatile int* s_last = reinterpret_cast<volatile int*>(s_tmem + 2);
  volatile int* s_complete = reinterpret_cast<volatile int*>(s_tmem + 3);  // [2]: of the first and the last tile
  uint8_t* ring = ring_of(smem_raw);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t G = gridDim.x, g = blockIdx.x;
  const int64_t u0 = p.units * g / G, u1 = p.units * (g + 1) / G;
  const int64_t tile0 = u0 / p.chunks;
  const int32_t chunk0 = (int32_t)(u0 - tile0 * p.chunks);
  const int blk_b = terms_bytes(kE4M3, p.n);
  const int stage_bytes = block_bytes(kE4M3) + blk_b;
  const int accs = p.n <= 128 ? 2 : 1;

  struct Place {
    int64_t row_tile;
    int32_t token_tile, chunk;
  };
  const Place start{tile0 / p.token_tiles, (int32_t)(tile0 % p.token_tiles), chunk0};
  const auto advance = [&](Place& at) {
    if (++at.chunk < p.chunks) return;
    at.chunk = 0;
    if (++at.token_tile < p.token_tiles) return;
    at.token_tile = 0;
    ++at.row_tile;
  };
  const auto load_weights = [&](const Place& at, int s) {
    tc::mbar_arrive_expect_tx(&full[s], (uint32_t)stage_bytes);
    tc::bulk_load(ring + s * stage_bytes, p.weights + (at.row_tile * p.chunks + at.chunk) * block_bytes(kE4M3),
                  block_bytes(kE4M3), &full[s]);
  };
  const int64_t n_units = u1 - u0;
  const int ahead = n_units < p.stages ? (int)n_units : p.stages;
  if (warp == kProducerWarp && lane == 0) {
    for (int s = 0; s < p.stages; ++s) {
      tc::mbar_init(&full[s], 1);
      tc::mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      tc::mbar_init(&acc_full[a], 1);
      tc::mbar_init(&acc_empty[a], kSumWarps);
    }
    *s_abort = 0;
    tc::fence_mbar_init();
    tc::fence_proxy_async_smem();
    // (before the terms are waited for: their kernel has waited for whatever wrote weights)
    Place at = start;
    for (int i = 0; i < ahead; ++i, advance(at)) load_weights(at, i);
  }
  if (warp == kSumWarps + 1) tc::tmem_alloc(s_tmem, p.tmem_cols);
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = *s_tmem;

  if (warp == kSumWarps) {
    if (lane == 0) {
      const auto load_terms = [&](const Place& at, int s) {
        tc::bulk_load(ring + s * stage_bytes + block_bytes(kE4M3), p.terms + ((int64_t)at.token_tile * p.chunks + at.chunk) * blk_b,
                      (uint32_t)blk_b, &full[s]);
      };
      pdl_wait();
      Place at = start;
      for (int i = 0; i < ahead; ++i, advance(at)) load_terms(at, i);
      int64_t issued = ahead;
      int s = ahead % p.stages;
      uint32_t turn = (uint32_t)(ahead / p.stages);  // times that the ring has gone round
      for (; issued < n_units; ++issued, advance(at)) {
        if (!tc::mbar_wait_bounded(&empty[s], (turn & 1u) ^ 1u, s_abort, &g_linear_error)) break;
        load_weights(at, s);
        load_terms(at, s);
        if (++s == p.stages) s = 0, ++turn;
      }
      // copies land before the CTA's memory goes away
      for (int64_t i = issued > p.stages ? issued - p.stages : 0; i < issued; ++i)
        tc::mbar_wait_issued(&full[i % p.stages], (uint32_t)(i / p.stages));
    }
    __syncwarp();
  } else if (warp == kSumWarps + 1) {
    const uint32_t one = tc::elect_one();
    const uint32_t ring_at = tc::smem_u32(ring), idesc = idesc_of<kE4M3>(p.n);
    int32_t chunk = chunk0;
    int s = 0, a = 0;
    uint32_t turn = 0, acc_turn = 0;
    bool ok = true;
    for (int64_t u = u0; ok && u < u1;) {
      ok = __all_sync(0xffffffffu, tc::mbar_wait_bounded(&acc_empty[a], (acc_turn & 1u) ^ 1u, s_abort, &g_linear_error));
      bool add = false;
      const uint32_t acc = tmem + (uint32_t)(a * p.n);
      for (; ok && u < u1 && chunk < p.chunks; ++u, ++chunk) {
        ok = __all_sync(0xffffffffu, tc::mbar_wait_bounded(&full[s], turn & 1u, s_abort, &g_linear_error));
        if (!ok) break;
        tc::tc_fence_after();
        const uint32_t a_at = ring_at + (uint32_t)(s * stage_bytes);
        stage_products<kE4M3>(one, a_at, a_at + block_bytes(kE4M3), p.n, acc,
                              tmem + (uint32_t)(accs * p.n + s * scale_cols(kE4M3, p.n)), idesc, add);
        add = true;
        tc::mma_commit_one(one, &empty[s]);
        if (++s == p.stages) s = 0, ++turn;
      }
      chunk = 0;
      // (whatever was issued ends before tensor memory is freed, an aborted run's too)
      tc::mma_commit_one(one, &acc_full[a]);
      if (u >= u1 || !ok) tc::mbar_wait_issued(&acc_full[a], acc_turn);
      if (++a == accs) a = 0, ++acc_turn;
    }
    __syncwarp();
  } else {
    pdl_wait();  // the factors and the counts; and the outputs may have readers before this call
    const int row = (warp & 3) * 32 + lane;
    const int half = tokens_of_warp(p.n), first = (warp >> 2) * half;
    // where CTA c's part of its first tile, or of the tile that it begins, goes
    const auto part_of = [&](int64_t c, bool begun) { return p.parts + (c * 2 + begun) * (p.n / kTerms) * kRows; };
    int64_t tile = tile0;
    int32_t chunk = chunk0;
    int a = 0;
    uint32_t acc_turn = 0;
    for (int64_t u = u0; u < u1; ++tile) {
      const int64_t token_tile = tile % p.token_tiles;
      const int64_t t0 = token_tile * kTileTokens, out_row = tile / p.token_tiles * kRows;
      const int nt = (int)(p.T - t0 < kTileTokens ? p.T - t0 : kTileTokens);
      const bool begins = chunk == 0, ends = p.chunks - chunk <= u1 - u;
      u += ends ? p.chunks - chunk : u1 - u;
      chunk = 0;
      // lane t holds token t's factor
      float factor = 0.0f;
      if (kE4M3 && lane < nt) factor = __ldcg(p.factor + t0 + lane);
      // A tile in two parts, the other one the next CTA's or the last one's. Where that is
      // there already (the next CTA began with it: mostly it is), it is added to this one's,
      // which need not be written.
      const bool shared = !begins || !ends;
      int* joined = p.joined + (begins ? g : g - 1);
      const float* from = part_of(begins ? g + 1 : g - 1, !begins) + (int64_t)first * kRows + row;
      bool complete = false;
      float other[16];
      const auto load_other = [&]() {
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (i < half && first + i < nt) other[i] = __ldcg(from + i * kRows);
      };
      if (shared) {
        if (threadIdx.x == 0) s_complete[begins] = load_acquire(joined);
        sync_sum_warps();
        complete = s_complete[begins] != 0;
        if (complete) load_other();
      }
      // (after a wait that ran out the warps still meet at the same barriers: the waits of
      // an aborted run end at once. A tile whose products were cut short is stored as it is.)
      const bool ok = __all_sync(0xffffffffu, tc::mbar_wait_bounded(&acc_full[a], acc_turn & 1u, s_abort, &g_linear_error));
      float y[16];
      if (ok) {
        tc::tc_fence_after();
        const uint32_t acc = tmem + ((uint32_t)((warp & 3) * 32) << 16) + (uint32_t)(a * p.n + first * kTerms);
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
          if (i >= half || first + i >= nt) break;
          uint32_t v[32];
          // (columns past the accumulator hold scales or the other one: read, not used)
          tc::tmem_ld_32x32b_x32(acc + (uint32_t)(i * kTerms), v);
          tc::tmem_ld_wait();
#pragma unroll
          for (int h = 0; h < 4; ++h)
            y[i + h] = sum_terms<kE4M3>(v + 8 * h) * factor_from<kE4M3>(factor, first + i + h);
        }
        tc::tc_fence_before();
      }
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&acc_empty[a]);
      if (++a == accs) a = 0, ++acc_turn;

      const int mine = ok ? min(half, nt - first) : 0;  // (none or fewer at the last tokens)
      if (shared && !complete) {
        float* to = part_of(g, begins) + (int64_t)first * kRows + row;
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (i < mine) __stcg(to + i * kRows, y[i]);
        __threadfence();
        sync_sum_warps();
        if (threadIdx.x == 0) *s_last = ok && atomicAdd(joined, 1) == 1;
        sync_sum_warps();
        if (*s_last == 0) continue;
        __threadfence();
        load_other();
      }
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (i < mine) put_out(p, t0 + first + i, out_row + row, shared ? y[i] + other[i] : y[i]);
    }
  }
  __syncthreads();
  if (warp == kSumWarps + 1) tc::tmem_dealloc(tmem, p.tmem_cols);
}

// ---- many tokens -----------------------------------------------------------------
// More than 64 tokens: the weights' values are exact in bf16 (two bits, or with an E4M3
// scale six), so they are made on the way and multiplied by x as it is, 128 outputs x up
// to 256 tokens a CTA. A token's eight columns take 1/32 of an FP4 block's time of 880
// cycles (with E4M3 scales); a bf16 block takes 2,150 to 2,300 for 80 to 256 tokens alike (a
// product with A in tensor memory takes 134 cycles for its 16 inputs however few its columns;
// neither 30 % fewer instructions in the values' making nor half as many warps again changed
// that): 96 tokens by 4,096 x 4,096 take 11.9 us, 64 11.3, 10.1 as terms.
//   warp 16    producer of blocks of weights;
//   warp 17    products, A from tensor memory: in shared memory the weights' values would
//              be written and read beside x, more than its 128 bytes a cycle;
//   warp 18    producer of 64 channels of the tile's tokens at a time, by a tensor map
//              (zeros past the last token and channel);
//   warps 0-15 the values of 64 inputs of a row to a thread, four sets of four warps in
//              turn (with two sets their making held the products up: 33 us for 1,021
//              tokens by 4,096 x 4,096, 26 with four); then the accumulator, stored or (clusters that split the inputs)
//              added in rank order out of one another's shared memory.
constexpr int kWideTokens = 256;
constexpr int kSub = 64;             // inputs of a step: 128 bytes of a token, 32 columns of A
constexpr int kRawStages = 3;
constexpr int kMaxXStages = 16;      // as many as fit: a trip to L2 is about five steps of 256 tokens
constexpr int kSlots = 8;            // steps of A in tensor memory, behind 256 accumulator columns
constexpr int kSets = 4;             // of four warps
constexpr int kWideThreads = 32 * (4 * kSets + 3);

// Equal tiles of tokens, a multiple of 16 each.
constexpr int32_t wide_tiles(int64_t T) { return (int32_t)((T + kWideTokens - 1) / kWideTokens); }
constexpr int32_t wide_tokens(int64_t T) { return (int32_t)((T + wide_tiles(T) - 1) / wide_tiles(T) + 15) / 16 * 16; }
static_assert(wide_tiles(0x7FFFFFFF) == 1 << 23 && wide_tokens(0x7FFFFFFF) == kWideTokens, "sums past 32 bits");
static_assert(wide_tiles(65) == 1 && wide_tokens(65) == 80 && wide_tiles(257) == 2 && wide_tokens(257) == 144 &&
              wide_tiles(4097) == 17 && wide_tokens(4097) == kWideTokens, "equal tiles");

struct WideParams {
  Params p;
  int32_t tokens;  // of a tile, a multiple of 16
  int32_t x_bytes, x_stages;
};

// Eight E2M1 codes to bf16, times a scale and 1/4: the bytes of the magnitudes' quarters
// are looked up (0, 1/8 .. 3/2: high 00 3E 3E 3E 3F 3F 3F 3F, low 00 00 80 C0 00 40 80 C0),
// the signs put to the high ones, and both interleaved. So 6 x 2^127 has a place in bf16,
// and 1/2 x 2^-127 too. An E4M3 scale is held four times as large; with E8M0 ones the
// quarter is put back behind the product.
__device__ __forceinline__ void e2m1x8_to_bf16(uint32_t w, __nv_bfloat162 scale, uint32_t* out) {
  const uint32_t m = w & 0x77777777u;
  const uint32_t even = (w << 4) & 0x80808080u, odd = w & 0x80808080u;
  const uint32_t h0 = __byte_perm(0x3E3E3E00u, 0x3F3F3F3Fu, m) | __byte_perm(even, odd, 0x5140);
  const uint32_t h1 = __byte_perm(0x3E3E3E00u, 0x3F3F3F3Fu, m >> 16) | __byte_perm(even, odd, 0x7362);
  const uint32_t l0 = __byte_perm(0xC0800000u, 0xC0804000u, m), l1 = __byte_perm(0xC0800000u, 0xC0804000u, m >> 16);
  const uint32_t v[4] = {__byte_perm(l0, h0, 0x5140), __byte_perm(l0, h0, 0x7362), __byte_perm(l1, h1, 0x5140),
                         __byte_perm(l1, h1, 0x7362)};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 y = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&v[i]), scale);
    out[i] = *reinterpret_cast<const uint32_t*>(&y);
  }
}

template <bool kE4M3>
__global__ void __launch_bounds__(kWideThreads, 1) wide_kernel(const __grid_constant__ CUtensorMap x_map, WideParams wp) {
  const Params& p = wp.p;
  extern __shared__ uint8_t smem_raw[];
  uint64_t* full_w = reinterpret_cast<uint64_t*>(smem_raw);
  uint64_t* empty_w = full_w + kRawStages;
  uint64_t* full_x = empty_w + kRawStages;
  uint64_t* empty_x = full_x + kMaxXStages;
  uint64_t* full_a = empty_x + kMaxXStages;
  uint64_t* empty_a = full_a + kSlots;
  uint64_t* acc_full = empty_a + kSlots;
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(acc_full + 1);
  volatile int* s_abort = reinterpret_cast<volatile int*>(s_tmem + 1);
  uint8_t* s_x = ring_of(smem_raw);
  uint8_t* s_w = s_x + wp.x_stages * wp.x_bytes;
  const int n_x = wp.x_stages;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int part = (int)(blockIdx.x % (uint32_t)p.split);
  const int64_t tile = blockIdx.x / (uint32_t)p.split;
  const int32_t t0 = (int32_t)(tile % p.token_tiles) * wp.tokens;
  const int64_t row_tile = tile / p.token_tiles;
  const int nt = min(p.T - t0, wp.tokens);
  const int32_t c0 = (int32_t)((int64_t)p.chunks * part / p.split);
  const int32_t c1 = (int32_t)((int64_t)p.chunks * (part + 1) / p.split);
  const int steps = min((c1 - c0) * (kChunk / kSub), (p.n_in - c0 * kChunk + kSub - 1) / kSub);
  constexpr int kOfChunk = kChunk / kSub;

  const uint8_t* from = p.weights + (row_tile * p.chunks + c0) * block_bytes(kE4M3);
  const int n_raw = (steps + kOfChunk - 1) / kOfChunk;
  const auto load_raw = [&](int i, int s) {
    tc::mbar_arrive_expect_tx(&full_w[s], block_bytes(kE4M3));
    tc::bulk_load(s_w + s * block_bytes(kE4M3), from + (int64_t)i * block_bytes(kE4M3), block_bytes(kE4M3), &full_w[s]);
  };
  if (warp == 4 * kSets && lane == 0) {
    for (int s = 0; s < kRawStages; ++s) {
      tc::mbar_init(&full_w[s], 1);
      tc::mbar_init(&empty_w[s], kOfChunk * 4);  // each step's four warps
    }
    for (int s = 0; s < n_x; ++s) {
      tc::mbar_init(&full_x[s], 1);
      tc::mbar_init(&empty_x[s], 1);
    }
    for (int s = 0; s < kSlots; ++s) {
      tc::mbar_init(&full_a[s], 4);
      tc::mbar_init(&empty_a[s], 1);
    }
    tc::mbar_init(acc_full, 1);
    *s_abort = 0;
    tc::fence_mbar_init();
    tc::fence_proxy_async_smem();
    pdl_wait();  // (the kernel before may have written the weights)
    for (int i = 0; i < min(n_raw, kRawStages); ++i) load_raw(i, i);
  }
  if (warp == 4 * kSets + 1) tc::tmem_alloc(s_tmem, 512);
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = *s_tmem, a_cols = tmem + kWideTokens;

  if (warp == 4 * kSets) {
    if (lane == 0) {
      int i = min(n_raw, kRawStages);
      for (; i < n_raw; ++i) {
        const int s = i % kRawStages;
        if (!tc::mbar_wait_bounded(&empty_w[s], ((uint32_t)(i / kRawStages) & 1u) ^ 1u, s_abort, &g_linear_error)) break;
        load_raw(i, s);
      }
      // copies land before the CTA's memory goes away
      for (int l = max(0, i - kRawStages); l < i; ++l) tc::mbar_wait_issued(&full_w[l % kRawStages], (uint32_t)(l / kRawStages));
    }
    __syncwarp();
  } else if (warp == 4 * kSets + 2) {
    if (lane == 0) {
      pdl_wait();
      int j = 0, s = 0;
      uint32_t turn = 1;
      for (; j < steps; ++j) {
        if (!tc::mbar_wait_bounded(&empty_x[s], turn, s_abort, &g_linear_error)) break;
        tc::mbar_arrive_expect_tx(&full_x[s], (uint32_t)wp.x_bytes);
        tc::tma_load_2d(s_x + s * wp.x_bytes, &x_map, c0 * kChunk + j * kSub, t0, &full_x[s]);
        if (++s == n_x) s = 0, turn ^= 1u;
      }
      for (int l = max(0, j - n_x); l < j; ++l) tc::mbar_wait_issued(&full_x[l % n_x], (uint32_t)(l / n_x));
    }
    __syncwarp();
  } else if (warp == 4 * kSets + 1) {
    const uint32_t one = tc::elect_one();
    const uint32_t idesc = tc::idesc_bf16(128, wp.tokens, 0, 0), x_at = tc::smem_u32(s_x);
    // (places in the rings carried along: a division by the number of stages is longer
    // than a step's products)
    int s = 0;
    uint32_t turn = 0;
    for (int j = 0; j < steps; ++j) {
      const int a = j % kSlots;
      const bool ok = tc::mbar_wait_bounded(&full_x[s], turn, s_abort, &g_linear_error) &&
                      tc::mbar_wait_bounded(&full_a[a], (uint32_t)(j / kSlots) & 1u, s_abort, &g_linear_error);
      if (!__all_sync(0xffffffffu, ok)) break;
      tc::tc_fence_after();
      const uint32_t at = x_at + (uint32_t)(s * wp.x_bytes);
#pragma unroll
      for (int m = 0; m < kSub / 16; ++m)
        tc::mma_f16_ta_one(one, tmem, a_cols + (uint32_t)(a * (kSub / 2) + m * 8),
                           tc::smem_desc(at + 32 * m, 0, 1024, tc::kSwizzle128B), idesc, (j | m) != 0);
      tc::mma_commit_one(one, &empty_x[s]);
      tc::mma_commit_one(one, &empty_a[a]);
      if (++s == n_x) s = 0, turn ^= 1u;
    }
    // whatever was issued ends before tensor memory is freed
    tc::mma_commit_one(one, acc_full);
    tc::mbar_wait_issued(acc_full, 0);
    __syncwarp();
  } else {
    const int row = (warp & 3) * 32 + lane;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    for (int j = warp >> 2; j < steps; j += kSets) {
      const int raw = j / kOfChunk, q = j % kOfChunk, a = j % kSlots;
      const bool ok = tc::mbar_wait_bounded(&full_w[raw % kRawStages], (uint32_t)(raw / kRawStages) & 1u, s_abort, &g_linear_error) &&
                      tc::mbar_wait_bounded(&empty_a[a], ((uint32_t)(j / kSlots) & 1u) ^ 1u, s_abort, &g_linear_error);
      if (!__all_sync(0xffffffffu, ok)) break;
      const uint8_t* block = s_w + (raw % kRawStages) * block_bytes(kE4M3);
      const uint8_t* sf = block + kDataBytes + scale_place(row);
      __nv_bfloat162 scales[4];  // of each sixteen inputs
      if (kE4M3) {
        // an E4M3 byte at a bf16's exponent and first bits is its value times 2^-120
        const uint32_t four = *reinterpret_cast<const uint32_t*>(sf + q * group_bytes());
        const __nv_bfloat162 up = __float2bfloat162_rn(__uint_as_float((120u + 2u + 127u) << 23));
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t two = (four >> (16 * i) & 0x7Fu) << 4 | (four >> (16 * i + 8) & 0x7Fu) << 20;
          const __nv_bfloat162 f = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&two), up);
          scales[2 * i] = __low2bfloat162(f);
          scales[2 * i + 1] = __high2bfloat162(f);
        }
      } else {
        const uint32_t two = *reinterpret_cast<const uint16_t*>(sf + (q / 2) * group_bytes() + (q % 2) * 2);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t e = two >> (8 * i) & 0xFFu;  // (0: 2^-127, a subnormal; 255: NaN)
          const uint32_t bits = (e << 7 | (((e + 1) & 0xFFu) < 2 ? 0x40u : 0u)) * 0x10001u;
          scales[2 * i] = scales[2 * i + 1] = *reinterpret_cast<const __nv_bfloat162*>(&bits);
        }
      }
      uint32_t v[32];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint4 c = *reinterpret_cast<const uint4*>(block + tc::sw128_offset(row, 2 * q + h));
        const uint32_t w[4] = {c.x, c.y, c.z, c.w};
        const __nv_bfloat162* scale = scales + 2 * h;  // of the first and second sixteen
#pragma unroll
        for (int i = 0; i < 4; ++i) e2m1x8_to_bf16(w[i], scale[i / 2], v + 16 * h + 4 * i);
      }
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&empty_w[raw % kRawStages]);
      tc::tc_fence_after();
      tc::tmem_st_32x32b_x32(a_cols + lanes + (uint32_t)(a * (kSub / 2)), v);
      tc::tmem_st_wait();
      tc::tc_fence_before();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&full_a[a]);
    }
    pdl_wait();  // (the outputs may have readers before this call)
  }

  float* sums = reinterpret_cast<float*>(s_x);  // [nt][128], once the rings are done with
  if (warp < 4 * kSets) {
    const bool ok = __all_sync(0xffffffffu, tc::mbar_wait_bounded(acc_full, 0, s_abort, &g_linear_error));
    const int row = (warp & 3) * 32 + lane;
    if (ok) {
      tc::tc_fence_after();
      for (int t = (warp >> 2) * 16; t < nt; t += 16 * kSets) {
        uint32_t v[16];
        tc::tmem_ld_32x32b_x16(tmem + ((uint32_t)((warp & 3) * 32) << 16) + (uint32_t)t, v);
        tc::tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          if (t + i >= nt) break;
          const float y = __uint_as_float(v[i]) * (kE4M3 ? 1.0f : 4.0f);
          if (p.split > 1)
            sums[(t + i) * kRows + row] = y;
          else
            put_out(p, t0 + t + i, row_tile * kRows + row, y);
        }
      }
      tc::tc_fence_before();
    }
  }
  __syncthreads();
  if (warp == 4 * kSets + 1) tc::tmem_dealloc(tmem, 512);  // (first, as above)
  if (p.split > 1) {
    cluster_sync();
    add_parts(p, sums, part, nt, t0, row_tile);
    cluster_sync();  // the peers have read this CTA's sums
  }
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
  if (n_in == 0 || n_in % 32 || n_in > 1 << 30) return CSA2_ERR_UNSUPPORTED_SHAPE;
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

// CTAs to a token's terms.
static int64_t slices_of(int32_t n_in) { return ((int64_t)n_in + linear::kTermThreads * 8 - 1) / (linear::kTermThreads * 8); }

// Workspace of a product of more than kFewTokens: the tokens' factors, the counts and
// parts of the tiles that CTAs share, the terms.
struct LinearSpace {
  size_t joined, parts, terms, bytes;
};
static LinearSpace space_of(int32_t T, int32_t n_in, bool e4m3) {
  const int n = tile_columns(T);
  LinearSpace s;
  s.joined = e4m3 ? al256((size_t)T * sizeof(float)) : 0;
  s.parts = s.joined + al256(linear::kStreamCtas * sizeof(int32_t));
  s.terms = s.parts + (size_t)linear::kStreamCtas * 2 * (n / linear::kTerms) * linear::kRows * sizeof(float);
  s.bytes = s.terms + (size_t)token_tiles_of(T) * (size_t)chunks_of(n_in) * linear::terms_bytes(e4m3, n);
  return s;
}

// Whether the weights' values are made (a tensor map's box of 64 channels wants as many).
static bool is_wide(int32_t T, int32_t n_in) { return T > linear::kTermTokens && n_in >= linear::kSub; }

extern "C" size_t csa2_fp4_linear_workspace_size(int32_t n_tokens, int32_t n_in, int32_t format) {
  if (n_tokens <= 0 || check_sizes(1, n_in, format) != CSA2_OK) return 0;
  // (a product of bf16 values keeps nothing there; the size never falls with more tokens,
  // so that one workspace does for all calls of up to as many)
  return space_of(is_wide(n_tokens, n_in) ? linear::kTermTokens : n_tokens, n_in, format == CSA2_FP4_E4M3).bytes;
}

// CTAs in clusters of that many that are on the SMs at once, one to an SM: a cluster lies
// within a group of SMs, and clusters of eight leave 32 of the 152 SMs over (as the runtime's
// occupancy query says; past that a product takes a second wave: 8 tokens by 2,048 x 2,048
// in 16 clusters of eight took 8.4 us).
static int64_t cluster_room(int n) { return n == 8 ? 120 : n == 4 ? 144 : linear::kStreamCtas; }

// Stages that fit beside `acc` accumulator columns.
static int stages_for(bool e4m3, int n, int acc, int cols, int smem) {
  const int by_smem = (smem - linear::kHeadBytes - 1024) / (linear::block_bytes(e4m3) + linear::terms_bytes(e4m3, n));
  const int by_cols = (cols - acc) / linear::scale_cols(e4m3, n);
  const int most = by_smem < by_cols ? by_smem : by_cols;
  return most < linear::kMaxStages ? most : linear::kMaxStages;
}

// CTAs to a tile: for all SMs; two to an SM where each has four chunks and more to itself
// (a token by 4,096 x 32,768: 14.8 us with 256 CTAs, 16.0 with 128; by 4,096 x 4,096: 6.2
// and 5.7).
static int split_of(int64_t tiles, int32_t chunks, int ctas) {
  int split = 1;
  while (split < linear::kMaxSplit && split * 2 <= chunks &&
         (tiles * split * 2 <= cluster_room(split * 2) ||
          (tiles * split * 2 <= ctas * cluster_room(split * 2) && chunks >= 8 * split)))
    split *= 2;
  return split;
}

template <bool kE4M3, bool kOwnTerms, int kCtas>
static int launch_split(linear::Params p, cudaStream_t stream) {
  using namespace linear;
  static Csa2PerDeviceOnce once;
  constexpr int kSmem = 226 / kCtas * 1024, kCols = 512 / kCtas;
  if (csa2_smem_optin((const void*)split_kernel<kE4M3, kOwnTerms, kCtas>, kSmem, once) != CSA2_OK) return CSA2_ERR_CUDA;
  const int64_t tiles = row_tiles_of(p.n_out) * p.token_tiles;
  p.tmem_cols = kCols;
  p.stages = stages_for(kE4M3, p.n, p.n, kCols, kSmem);
  p.split = split_of(tiles, p.chunks, kCtas);
  if (csa2_launch_pdl_cluster(split_kernel<kE4M3, kOwnTerms, kCtas>, dim3((unsigned)(tiles * p.split)), dim3(kThreads),
                              (size_t)kSmem, stream, (unsigned)p.split, p) != cudaSuccess) {
    (void)cudaGetLastError();
    return CSA2_ERR_CUDA;
  }
  return CSA2_OK;
}

template <bool kE4M3>
static int launch_stream(linear::Params p, cudaStream_t stream) {
  using namespace linear;
  static Csa2PerDeviceOnce once;
  constexpr int kSmem = 226 * 1024;
  if (csa2_smem_optin((const void*)stream_kernel<kE4M3>, kSmem, once) != CSA2_OK) return CSA2_ERR_CUDA;
  const int64_t tiles = row_tiles_of(p.n_out) * p.token_tiles;
  p.tmem_cols = 512;
  p.stages = stages_for(kE4M3, p.n, p.n <= 128 ? 2 * p.n : p.n, 512, kSmem);
  p.units = tiles * p.chunks;
  CSA2_LAUNCH_PDL(stream_kernel<kE4M3>, dim3(kStreamCtas), dim3(kThreads), (size_t)kSmem, stream, p);
  return CSA2_OK;
}

template <bool kE4M3>
static int launch_wide(linear::Params p, cudaStream_t stream) {
  using namespace linear;
  static Csa2PerDeviceOnce once;
  constexpr int kSmem = 227 * 1024, kRoom = kSmem - kHeadBytes - 1024 - kRawStages * block_bytes(kE4M3);
  if (csa2_smem_optin((const void*)wide_kernel<kE4M3>, kSmem, once) != CSA2_OK) return CSA2_ERR_CUDA;
  auto encode = csa2_tensor_map_encoder();
  if (!encode) return CSA2_ERR_CUDA;
  p.token_tiles = wide_tiles(p.T);
  WideParams wp{p, wide_tokens(p.T)};
  wp.x_bytes = wp.tokens * kSub * 2;
  wp.x_stages = kRoom / wp.x_bytes < kMaxXStages ? kRoom / wp.x_bytes : kMaxXStages;
  CUtensorMap map;
  cuuint64_t dims[2] = {(cuuint64_t)p.n_in, (cuuint64_t)p.T};
  cuuint64_t strides[1] = {(cuuint64_t)p.n_in * 2};
  cuuint32_t box[2] = {(cuuint32_t)kSub, (cuuint32_t)wp.tokens};
  cuuint32_t estr[2] = {1, 1};
  if (encode(&map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, (void*)p.x, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return CSA2_ERR_CUDA;
  const int64_t tiles = row_tiles_of(p.n_out) * p.token_tiles;
  int split = 1;
  while (split < kMaxSplit && split * 2 <= p.chunks && tiles * split * 2 <= cluster_room(split * 2)) split *= 2;
  wp.p.split = split;
  if (csa2_launch_pdl_cluster(wide_kernel<kE4M3>, dim3((unsigned)(tiles * split)), dim3(kWideThreads), (size_t)kSmem, stream,
                              (unsigned)split, map, wp) != cudaSuccess) {
    (void)cudaGetLastError();
    return CSA2_ERR_CUDA;
  }
  return CSA2_OK;
}

template <bool kE4M3>
static int launch_linear(linear::Params p, uint8_t* workspace, cudaStream_t stream) {
  using namespace linear;
  // Up to three tokens, and row tiles for one wave: in one launch (E8M0, a token by 32,768
  // x 4,096: 13.8 us, 14.5 with the terms ahead; three 13.9 and 14.5; four 15.3 and 14.5; a
  // token by 131,072 x 4,096: 47.2 and 46.6). With E4M3 scales, whose base is a second look
  // at x, one or two (two by 16,384 x 4,096: 10.5 and 11.2; by 16,384 x 16,384 29.9 and 28.0).
  if (p.T <= (kE4M3 ? (p.n_in <= 4096 ? 2 : 1) : kFewTokens) && row_tiles_of(p.n_out) <= 2 * kStreamCtas)
    return launch_split<kE4M3, true, 2>(p, stream);
  if (is_wide(p.T, p.n_in)) return launch_wide<kE4M3>(p, stream);
  const LinearSpace space = space_of(p.T, p.n_in, kE4M3);
  p.factor = (const float*)workspace;
  p.joined = (int32_t*)(workspace + space.joined);
  p.parts = (float*)(workspace + space.parts);
  p.terms = workspace + space.terms;
  const int64_t slices = slices_of(p.n_in);
  const bool known = kE4M3 && slices > kLongSlices;
  if (known)
    CSA2_LAUNCH_PDL(factors_kernel, dim3((unsigned)p.T), dim3(kFactorThreads), (size_t)0, stream, p.x, p.n_in, (float*)workspace);
  TermArgs ta{p.x, p.T, p.n_in, p.chunks, p.n, (int32_t)slices, known, workspace + space.terms, (float*)workspace, p.joined};
  CSA2_LAUNCH_PDL(terms_kernel<kE4M3>, dim3((unsigned)(p.T * slices)), dim3(kTermThreads), (size_t)0, stream, ta);
  // Tiles for one wave (of up to 16 tokens two CTAs to an SM): clusters, or CTAs by
  // themselves. More: in equal runs, whose joins take 3 us (E8M0, 5 tokens by 16,384 x 4,096,
  // 128 tiles: 10.5 us, 13.6 in runs; by 32,768 x 4,096: 14.4 and 17.1; 32 tokens, 256 tiles:
  // 26.8 and 21.3 (E4M3); 16 tokens by 128,259 x 4,096: 51.7 and 48.0).
  // Two CTAs to an SM, each with half of the stages, where a tile gets more of them so (5
  // tokens by 4,864 x 16,384: 12.2 us, 15.6 with one; but 8 by 4,096 x 32,768, four to a tile
  // either way, 18.8 and 17.6).
  const int64_t tiles = row_tiles_of(p.n_out) * p.token_tiles;
  if (tiles > (p.n <= 128 ? 2 : 1) * kStreamCtas) return launch_stream<kE4M3>(p, stream);
  return p.n <= 128 && (tiles > kStreamCtas || split_of(tiles, p.chunks, 2) > split_of(tiles, p.chunks, 1))
             ? launch_split<kE4M3, false, 2>(p, stream)
             : launch_split<kE4M3, false, 1>(p, stream);
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
      (int64_t)n_tokens * slices_of(n_in) > 0x7FFFFFFFLL)
    return CSA2_ERR_UNSUPPORTED_SHAPE;
  const size_t need = csa2_fp4_linear_workspace_size(n_tokens, n_in, format);
  if (!workspace || workspace_bytes < need || !csa2_aligned(workspace, 256)) return CSA2_ERR_WORKSPACE;
  linear::Params p{};
  p.weights = weights;
  p.x = (const uint16_t*)x_bf16;
  p.out_bf16 = (__nv_bfloat16*)out_bf16;
  p.out_f32 = out_f32;
  p.scale = scale;
  p.T = n_tokens;
  p.n_out = n_out;
  p.n_in = n_in;
  p.chunks = (int32_t)chunks_of(n_in);
  p.token_tiles = (int32_t)token_tiles_of(n_tokens);
  p.n = tile_columns(n_tokens);
  return format == CSA2_FP4_E4M3 ? launch_linear<true>(p, (uint8_t*)workspace, (cudaStream_t)stream)
                                 : launch_linear<false>(p, (uint8_t*)workspace, (cudaStream_t)stream);
}
