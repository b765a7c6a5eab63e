// paged_attn.cu -- dense attention of ragged query tokens over the paged FP4
// latents: every token attends to all the entries that it sees.
//
// "DeepSeek-V4.1-Flash: Pushing the Limits of KV Cache Compression", section
// 2.3 (attention over the shared latents) and 2.4.4 (E2M1 + E4M3/16 latents
// dequantised before attention); mer.dev notes section 1 (64 heads of dim 512,
// one 512-channel latent as key and value).
//
// A token's entries are cut into tiles of 128. For a tile with rows R [128][512]
// and the token's 64 queries Q:
//   S^T = R Q^T            (M = 128 rows, N = 64 heads, K = 512)
//   P   = 2^(S' - ref)     S' = S scaled into the log2 domain, ref per head
//   O^T += R^T P^T         (4 x M = 128 channels, N = 64, K = 128)
// and l += sum of P; at the end O / l and ref + log2 l. ref is a head's running
// maximum moved only when a tile passes it by more than 2^kSlack: O^T then
// seldom needs rescaling, and whether it does is one comparison per thread.
//
// What bounds it: an entry costs 288 bytes and, per token, 131,072 FLOP, so the
// tensor cores (fp16) bind before HBM already at one token per sequence. With
// 64 heads on N, an SM's shared memory does: per tile it takes 128 KiB of
// writes (the dequantised rows) and 384 KiB of operand reads.
//
// Work split: the tiles of all tokens in batch order form one list, cut into
// one equal run per SM. A run may begin and end inside a token; the parts of
// such a token go to the workspace and a second kernel joins them in order.
// Few long sequences and many short ones load the SMs alike, and the workspace
// (two parts per SM) does not grow with the batch.
#include "attn_common.cuh"
#include "paged_common.cuh"

namespace csa2 {

__device__ int g_paged_attn_error = 0;

namespace pattn {

using attn_tc::e2m1x8_to_f16;
using attn_tc::e4m3x2_to_f16x2;
using attn_tc::f32x2_to_f16x2;
using attn_tc::fast_exp2;
using attn_tc::idesc_f16;
using attn_tc::mul_f16x2;
using attn_tc::named_barrier;
using attn_tc::warp_transpose_reduce16;

constexpr int kThreads = 512;             // 16 warps: 4 lane quadrants x 4 (a 17th would cap registers at 96)
constexpr int kWarps = kThreads / 32;
constexpr int kRows = 128;
constexpr int kBlkR = kRows * 128;        // one 64-channel block of R: [128 rows][128 B]
constexpr int kBlkQ = kHeads * 128;       // one 64-channel block of Q: [64 heads][128 B]
constexpr int kBlkP = kHeads * 128;       // 64 rows of P: [64 heads][128 B]
constexpr int kOffR = 0;                  // 8 blocks, 128 KiB
constexpr int kOffQ = kOffR + 8 * kBlkR;  // 8 blocks, 64 KiB
constexpr int kOffP = kOffQ + 8 * kBlkQ;  // 2 blocks, 16 KiB
constexpr int kOffMisc = kOffP + 2 * kBlkP;
constexpr int kSmemBytes = kOffMisc + 128 + 1024;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColS = 0;             // S^T: 64 columns (heads), lanes = rows
constexpr uint32_t kColO = 64;            // O^T: 4 blocks x 64 columns, lanes = channels

// P = 2^(S' - ref): at most 2^kTop when ref is the maximum itself, at most
// 2^(kTop + kSlack) = 2^15 before ref moves, below fp16's 65,504. The offset
// kTop keeps weights down to 2^-25 of the maximum at fp16's full precision
// (2^-14 is its smallest normal), and to 2^-35 above zero.
constexpr float kTop = 11.0f, kSlack = 4.0f;
constexpr float kNoRef = -1e30f;          // a head that has seen nothing yet

constexpr int kPartFloats = kHeads * kHeadDim;

// A part of a token that more than one CTA works on, for the joining kernel.
struct PartList {
  int32_t token;       // -1: this CTA begins no such token
  int32_t first_slot;  // slot of the first part
  int32_t cta0, cta1;  // the CTAs with parts: cta0 .. cta1 (those with tiles)
  int64_t tiles;       // tiles of the whole call
};

struct Args {
  const uint16_t* q;
  int32_t n_tokens, B, per_seq;
  const int32_t* cu;
  const uint8_t* kv_data;
  const uint8_t* kv_scale;
  PageTable pages;
  const int32_t* n_visible;
  int32_t causal;
  float scale_log2;  // sm_scale * log2(e)
  uint16_t* out;
  float* out_f32;
  float* lse;
  float* part_o;     // [2 * CTAs][64][512]
  float2* part_ml;   // [2 * CTAs][64] (ref, l)
  PartList* lists;   // [CTAs]
};

// ---- the list of tiles --------------------------------------------------------
__device__ __forceinline__ int64_t tiles_of(int64_t visible) {  // a token without entries has one empty tile
  return visible <= kRows ? 1 : (visible + kRows - 1) / kRows;
}
// sum of ceil(v / 128) for v = 1 .. x
__device__ __forceinline__ int64_t tiles_upto(int64_t x) {
  const int64_t n = x / kRows, r = x % kRows;
  return kRows * (n * (n + 1) / 2) + (n + 1) * r;
}
struct Seq {
  int32_t first, count;  // token rows
  int64_t visible;       // entries of its last token (of every one if not causal)
};
__device__ __forceinline__ Seq load_seq(const Args& a, int32_t b, bool report) {
  const TokenRun run = token_run(a.cu, b, a.n_tokens, a.per_seq);
  Seq s{run.first, run.count, a.n_visible[b]};
  const bool bad = s.count < 0 || (s.count > 0 && (s.visible < 0 || s.visible > a.pages.capacity()));
  if (bad) {
    if (report) record_error(&g_paged_attn_error, CSA2_ERR_DEVICE);
    s.count = 0;
  }
  return s;
}
__device__ __forceinline__ int64_t visible_of(const Args& a, const Seq& s, int32_t t) {
  return a.causal ? s.visible - s.count + 1 + t : s.visible;
}
// tiles of the sequence's first n tokens
__device__ __forceinline__ int64_t tiles_before(const Args& a, const Seq& s, int64_t n) {
  if (!a.causal) return n * tiles_of(s.visible);
  const int64_t v0 = s.visible - s.count + 1;  // entries of token 0
  const int64_t blind = v0 > 0 ? 0 : 1 - v0 < n ? 1 - v0 : n;  // tokens that see nothing
  const int64_t hi = v0 + n - 1;               // entries of the last of the n
  return blind + (hi > 0 ? tiles_upto(hi) - tiles_upto(v0 > 1 ? v0 - 1 : 0) : 0);
}

// bar.red.or over the 128 threads of a head group
__device__ __forceinline__ bool group_any(int id, bool p) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.or.pred q, %2, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)p), "r"(id)
      : "memory");
  return r != 0;
}

__global__ void __launch_bounds__(kThreads, 1) paged_attn_kernel(Args a) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_u32 = tc::smem_u32(smem_raw);
  uint8_t* sm = smem_raw + (((raw_u32 + 1023u) & ~1023u) - raw_u32);
  uint8_t* sR = sm + kOffR;
  uint8_t* sQ = sm + kOffQ;
  uint8_t* sP = sm + kOffP;
  uint64_t* bar_r = reinterpret_cast<uint64_t*>(sm + kOffMisc);  // R (and Q) of a tile written: 16 warps
  uint64_t* bar_s = bar_r + 1;                                   // S^T complete
  uint64_t* bar_p = bar_r + 2;                                   // P written, O^T rescaled: 16 warps
  uint64_t* bar_pv = bar_r + 3;                                  // [4] a channel block of O^T complete
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(sm + kOffMisc + 64);
  volatile int* s_abort = reinterpret_cast<volatile int*>(sm + kOffMisc + 68);
  __shared__ __align__(16) float s_mul[kHeads];     // sm_scale log2(e) 2^-k of the head's fp16 queries
  __shared__ __align__(16) float s_ref[kHeads];     // reference of P, log2 domain, less kTop
  __shared__ __align__(16) float s_red[4][kHeads];  // per-quadrant maxima, then sums
  __shared__ float s_inv[kHeads];
  __shared__ int64_t s_scan[kWarps];
  __shared__ int64_t s_at;       // first tile of the run, within its sequence
  __shared__ int32_t s_seq;      // the sequence of the run's first tile

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = (int)gridDim.x, cta = (int)blockIdx.x;

  if (tid == 0) {
    tc::mbar_init(bar_r, 16);
    tc::mbar_init(bar_s, 1);
    tc::mbar_init(bar_p, 16);
    for (int i = 0; i < 4; ++i) tc::mbar_init(bar_pv + i, 1);
    *s_abort = 0;
    s_seq = -1;
    tc::fence_mbar_init();
  }
  if (warp == 0) tc::tmem_alloc(s_tmem, kTmemCols);
  pdl_begin();

  // ---- this CTA's run [f0, f1) of the list: a scan over the sequences' tiles ----
  int64_t total = 0;
  for (int32_t b0 = 0; b0 < a.B; b0 += kThreads) {
    const int32_t b = b0 + tid;
    int64_t n = 0;
    if (b < a.B) {
      const Seq s = load_seq(a, b, cta == 0);
      n = tiles_before(a, s, s.count);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
    if (lane == 0) s_scan[warp] = n;
    __syncthreads();
    for (int w = 0; w < kWarps; ++w) total += s_scan[w];
    __syncthreads();
  }
  const int64_t f0 = total * cta / G, f1 = total * (cta + 1) / G;
  if (tid == 0) a.lists[cta].token = -1;
  if (f0 < f1) {
    // the sequence that holds tile f0 (a second scan: the first did not know f0)
    int64_t base = 0;
    for (int32_t b0 = 0; b0 < a.B && base <= f0; b0 += kThreads) {
      const int32_t b = b0 + tid;
      int64_t n = 0;
      if (b < a.B) {
        const Seq s = load_seq(a, b, false);
        n = tiles_before(a, s, s.count);
      }
      int64_t incl = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
      }
      if (lane == 31) s_scan[warp] = incl;
      __syncthreads();
      int64_t lo = base + incl - n;
      for (int w = 0; w < kWarps; ++w) {
        if (w < warp) lo += s_scan[w];
        base += s_scan[w];
      }
      if (f0 >= lo && f0 < lo + n) {
        s_seq = b;
        s_at = f0 - lo;
      }
      __syncthreads();
    }
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = *s_tmem;
  const int64_t n_run = f1 - f0;  // tiles of this CTA

  if (n_run > 0) {
    // ---- workers: warp w, lane quadrant q = w % 4 (rows 32q ..), group g = w / 4
    // (channels 128g .. of R and O^T; heads 16g .. of S and P) ----
    const int quad = warp & 3, grp = warp >> 2, h0 = grp * 16;
    // ---- the products, issued by warp 0 once every warp's rows (or P) are there ----
    const auto issue_s = [&](uint32_t par) {
      if (!__all_sync(0xffffffffu, tc::mbar_wait_bounded(bar_r, par, s_abort, &g_paged_attn_error))) return;
      tc::tc_fence_after();
      if (lane == 0) {
        constexpr uint32_t idesc = idesc_f16(128, 64, 0, 0);
        const uint64_t ad = tc::smem_desc(tc::smem_u32(sR), 0, 1024, tc::kSwizzle128B);
        const uint64_t bd = tc::smem_desc(tc::smem_u32(sQ), 0, 1024, tc::kSwizzle128B);
#pragma unroll
        for (int j = 0; j < 32; ++j) {  // block j / 4 of 64 channels, K step j % 4
          const uint64_t ko = (uint64_t)((j & 3) * 2);
          tc::mma_bf16(tmem + kColS, ad + (uint64_t)((j >> 2) * (kBlkR >> 4)) + ko,
                       bd + (uint64_t)((j >> 2) * (kBlkQ >> 4)) + ko, idesc, j ? 1u : 0u);
        }
        tc::mma_commit(bar_s);
      }
      __syncwarp();
    };
    const auto issue_pv = [&](uint32_t par, bool anew) {
      if (!__all_sync(0xffffffffu, tc::mbar_wait_bounded(bar_p, par, s_abort, &g_paged_attn_error))) return;
      tc::tc_fence_after();
      if (lane == 0) {
        constexpr uint32_t idesc = idesc_f16(128, 64, 1, 0);  // A = R^T is MN-major
        const uint64_t ad = tc::smem_desc(tc::smem_u32(sR), kBlkR, 1024, tc::kSwizzle128B);
        const uint64_t bd = tc::smem_desc(tc::smem_u32(sP), 0, 1024, tc::kSwizzle128B);
#pragma unroll
        for (int j = 0; j < 32; ++j) {  // channel block j / 8, K step j % 8 (16 rows)
          const int mb = j >> 3, kk = j & 7;
          tc::mma_bf16(tmem + kColO + 64u * (uint32_t)mb, ad + (uint64_t)((2 * mb * kBlkR + kk * 16 * 128) >> 4),
                       bd + (uint64_t)(((kk >> 2) * kBlkP + (kk & 3) * 32) >> 4), idesc, kk || !anew ? 1u : 0u);
          if (kk == 7) tc::mma_commit(bar_pv + mb);
        }
      }
      __syncwarp();
    };
    // the place in the list: tile `tile` of token `tok` of sequence `b`
    int32_t b = s_seq;
    Seq seq = load_seq(a, b, false);
    int32_t tok;
    int64_t tile;
    {
      int64_t at = s_at;
      int32_t lo = 0, hi = seq.count;  // tiles_before(lo) <= at < tiles_before(hi)
      while (hi - lo > 1) {
        const int32_t mid = lo + (hi - lo) / 2;
        if (tiles_before(a, seq, mid) <= at) lo = mid;
        else hi = mid;
      }
      tok = lo;
      tile = at - tiles_before(a, seq, lo);
    }
    int64_t visible = visible_of(a, seq, tok);
    int64_t tiles = tiles_of(visible);

    // loads of a tile: lane l of a group of 8 rows takes row l / 4, channels
    // 128 grp + 32 (l % 4) .. +31 (16 bytes of codes, 2 of scales): 64 whole
    // bytes of a row per 4 lanes
    uint4 raw[4];
    uint32_t scl[4];
    uint32_t gone = 0;  // bit i: rows 8i .. 8i+7 of the warp's 32 lie in a page outside the pool
    auto load_rows = [&](int32_t lb, int64_t ltile, int64_t lvisible) {
int64_t row[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t e = ltile * kRows + quad * 32 + i * 8 + (lane >> 2);
        row[i] = e < lvisible ? a.pages.row(lb, e) : -2;
      }
      gone = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (row[i] == -1) {
          gone |= 1u << i;
          record_error(&g_paged_attn_error, CSA2_ERR_DEVICE);
        }
        raw[i] = make_uint4(0u, 0u, 0u, 0u);
        scl[i] = 0u;
        if (row[i] >= 0) {
          raw[i] = __ldg(reinterpret_cast<const uint4*>(a.kv_data + row[i] * kKvBytes + grp * 64) + (lane & 3));
          scl[i] = __ldg(reinterpret_cast<const uint16_t*>(a.kv_scale + row[i] * kKvScales + grp * 8) + (lane & 3));
        }
      }
      gone = __reduce_or_sync(0xffffffffu, gone);
    };
    // the loaded rows as fp16 (exact) into R; rows not seen are zero. The eight
    // lanes of a store phase (two rows) take their words in different orders, so
    // that they cover the eight bank groups: lanes of odd 64-channel blocks swap
    // words 0/1 and 2/3, those of odd rows the halves.
    auto write_rows = [&]() {
      const bool sw1 = (lane >> 1) & 1, sw2 = (lane >> 2) & 1;
      const uint32_t kx = (sw1 ? 1u : 0u) ^ (sw2 ? 2u : 0u);
      uint8_t* blk = sR + (2 * grp + ((lane >> 1) & 1)) * kBlkR;
      const uint32_t c0 = (uint32_t)(lane & 1) * 4u;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t r = (uint32_t)(quad * 32 + i * 8 + (lane >> 2));
        uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
        uint32_t u[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) u[k] = sw1 ? w[k ^ 1] : w[k];
#pragma unroll
        for (int k = 0; k < 4; ++k) w[k] = sw2 ? u[k ^ 2] : u[k];
        const uint32_t s2 = e4m3x2_to_f16x2(scl[i]);
        const uint32_t lo = __byte_perm(s2, 0u, 0x1010u), hi = __byte_perm(s2, 0u, 0x3232u);
        const uint32_t sa = sw2 ? hi : lo, sb = sw2 ? lo : hi;
#pragma unroll
        for (int k = 0; k < 4; ++k) {  // w[k]: word k ^ kx of the 16 bytes
          uint32_t o0, o1, o2, o3;
          e2m1x8_to_f16(w[k], o0, o1, o2, o3);
          const uint32_t m = k < 2 ? sa : sb;
          *reinterpret_cast<uint4*>(blk + tc::sw128_offset(r, c0 + ((uint32_t)k ^ kx))) =
              make_uint4(mul_f16x2(o0, m), mul_f16x2(o1, m), mul_f16x2(o2, m), mul_f16x2(o3, m));
        }
      }
    };
    // the token's queries as fp16 with a power-of-two scale per head (exact but
    // for values below 2^-28 of the head's largest): thread (h, j) takes 16
    // bytes of each 64-channel block
    auto write_q = [&](int64_t token) {
      const int h = tid >> 3, j = tid & 7;
      const uint4* src = reinterpret_cast<const uint4*>(a.q + (token * kHeads + h) * kHeadDim) + j;
      uint4 v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = src[k * 8];
      uint32_t amax = 0;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) amax = max(amax, max(w[i] & 0x7FFFu, (w[i] >> 16) & 0x7FFFu));
      }
      amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 4));
      int k2 = 0;
      if (amax != 0u) k2 = min(max(14 - ((int)(amax >> 7) - 127), -100), 100);
      const float up = __int_as_float((127 + k2) << 23);
      const uint32_t col = (uint32_t)((j ^ (h & 7)) << 4);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          o[i] = f32x2_to_f16x2(__uint_as_float(w[i] << 16) * up, __uint_as_float(w[i] & 0xFFFF0000u) * up);
        *reinterpret_cast<uint4*>(sQ + k * kBlkQ + h * 128 + col) = make_uint4(o[0], o[1], o[2], o[3]);
      }
      if (j == 0) {
        s_mul[h] = a.scale_log2 * __int_as_float((127 - k2) << 23);
        s_ref[h] = kNoRef;
      }
    };

    float l_acc[16];  // this row lane's share of l for the group's heads
    int slot = 2 * cta;     // where a part of the present token goes
    bool whole = tile == 0; // the CTA has the token from its first tile on
    int64_t rows_seen = 0;  // the present tile's entries
    uint32_t gone_now = 0;
    load_rows(b, tile, visible);
    write_q(seq.first + tok);
#pragma unroll
    for (int j = 0; j < 16; ++j) l_acc[j] = 0.0f;
    write_rows();
    bool first = true;
    rows_seen = visible - tile * kRows;
    gone_now = gone;
    tc::fence_proxy_async_smem();
    __syncthreads();  // s_mul, s_ref
    if (lane == 0) tc::mbar_arrive(bar_r);

    // A wait that runs out (2 s) raises s_abort, on which every later wait gives
    // up at once and nothing more is issued. The loop then runs to its end all
    // the same, so that no warp is missing at a barrier; the outputs are
    // worthless and TIMEOUT is recorded.
    const auto wait = [&](uint64_t* bar, uint32_t par) {
      const bool ok = tc::mbar_wait_bounded(bar, par, s_abort, &g_paged_attn_error);
      return __all_sync(0xffffffffu, ok);
    };
    if (warp == 0) issue_s(0);
    for (int64_t i = 0; i < n_run; ++i) {
      const uint32_t par = (uint32_t)i & 1u;
      const bool last_of_run = i + 1 == n_run;
      const bool last_of_token = tile + 1 == tiles;
      // the next tile of the list
      int32_t nb = b, ntok = tok;
      int64_t ntile = tile + 1, nvisible = visible, ntiles = tiles;
      Seq nseq = seq;
      if (!last_of_run) {
        if (last_of_token) {
          ntile = 0;
          ++ntok;
          while (ntok >= nseq.count) {  // ends: the list has a tile behind this one
            ++nb;
            nseq = load_seq(a, nb, false);
            ntok = 0;
          }
          nvisible = visible_of(a, nseq, ntok);
          ntiles = tiles_of(nvisible);
        }
        load_rows(nb, ntile, nvisible);
      }

      wait(bar_s, par);
      tc::tc_fence_after();
      // ---- P of the tile: this thread's row, the group's 16 heads ----
      {
        const int row = quad * 32 + lane;
        const bool rv = row < rows_seen && !((gone_now >> (lane >> 3)) & 1u);
        uint32_t sr[16];
        tc::tmem_ld_32x32b_x16(tmem + ((uint32_t)(quad * 32) << 16) + kColS + (uint32_t)h0, sr);
        tc::tmem_ld_wait();
        float p[16];
        float top = -INFINITY;
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          p[j] = rv ? __uint_as_float(sr[j]) * s_mul[h0 + j] : -INFINITY;
          top = fmaxf(top, p[j] - s_ref[h0 + j]);
        }
        if (group_any(1 + grp, top > kTop + kSlack)) {
          // a head's scores passed its reference: new references, O^T and l to match
          float v[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) v[j] = p[j];
          const float m = warp_transpose_reduce16<true>(v, lane);
          if (lane < 16) s_red[quad][h0 + lane] = m;
          named_barrier(1 + grp, 128);
          float alpha[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const float mt = fmaxf(fmaxf(s_red[0][h0 + j], s_red[1][h0 + j]), fmaxf(s_red[2][h0 + j], s_red[3][h0 + j]));
            const float old = s_ref[h0 + j];
            alpha[j] = mt > old + (kTop + kSlack) ? fast_exp2(old - (mt - kTop)) : 1.0f;
          }
          named_barrier(1 + grp, 128);  // everyone has read the old references
          if (quad == 0 && lane < 16) {
            const float mt = fmaxf(fmaxf(s_red[0][h0 + lane], s_red[1][h0 + lane]),
                                   fmaxf(s_red[2][h0 + lane], s_red[3][h0 + lane]));
            if (mt > s_ref[h0 + lane] + (kTop + kSlack)) s_ref[h0 + lane] = mt - kTop;
          }
          if (!first) {
#pragma unroll 1
            for (int mb = 0; mb < 4; ++mb) {
              const uint32_t at = tmem + ((uint32_t)(quad * 32) << 16) + kColO + 64u * (uint32_t)mb + (uint32_t)h0;
              uint32_t ov[16];
              tc::tmem_ld_32x32b_x16(at, ov);
              tc::tmem_ld_wait();
#pragma unroll
              for (int j = 0; j < 16; ++j) ov[j] = __float_as_uint(__uint_as_float(ov[j]) * alpha[j]);
              tc::tmem_st_32x32b_x16(at, ov);
            }
            tc::tmem_st_wait();
          }
#pragma unroll
          for (int j = 0; j < 16; ++j) l_acc[j] *= alpha[j];
          named_barrier(1 + grp, 128);  // the new references
        }
        uint8_t* blkp = sP + (row >> 6) * kBlkP;
        const uint32_t chunk = (uint32_t)(row & 63) >> 3, within = ((uint32_t)row & 7u) * 2u;
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const float e = fast_exp2(p[j] - s_ref[h0 + j]);
          l_acc[j] += e;  // summed in fp32 before P is rounded to fp16
          *reinterpret_cast<__half*>(blkp + tc::sw128_offset((uint32_t)(h0 + j), chunk) + within) = __float2half_rn(e);
        }
      }
      tc::fence_proxy_async_smem();
      tc::tc_fence_before();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(bar_p);
      if (warp == 0) issue_pv(par, first);
      first = false;

      if (!last_of_run && !last_of_token) {
        // ---- the next tile's rows, as the products over this tile's channels end ----
        wait(bar_pv + grp, par);
        write_rows();
        tc::fence_proxy_async_smem();
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(bar_r);
        if (warp == 0) issue_s(par ^ 1u);
      } else {
        // ---- the token's (or the run's) end: l over the rows, O^T out ----
        const float lsum = warp_transpose_reduce16<false>(l_acc, lane);
        if (lane < 16) s_red[quad][h0 + lane] = lsum;
        for (int mb = 0; mb < 4; ++mb) wait(bar_pv + mb, par);
        tc::tc_fence_after();
        __syncthreads();
        const bool complete = whole && last_of_token;
        const int64_t token = seq.first + tok;
        if (tid < kHeads) {
          const float l = s_red[0][tid] + s_red[1][tid] + s_red[2][tid] + s_red[3][tid];
          s_inv[tid] = !complete ? 1.0f : l > 0.0f ? 1.0f / l : 0.0f;
          if (!complete) a.part_ml[(int64_t)slot * kHeads + tid] = make_float2(s_ref[tid], l);
          else if (a.lse)
            a.lse[token * kHeads + tid] = l > 0.0f ? (s_ref[tid] + log2f(l)) * 0.6931471805599453f : -INFINITY;
        }
        __syncthreads();
        const int c = 128 * grp + 32 * quad + lane;
        const uint32_t o_base = tmem + ((uint32_t)(quad * 32) << 16) + kColO + 64u * (uint32_t)grp;
        float* po = a.part_o + (int64_t)slot * kPartFloats + c;
        float* of = a.out_f32 ? a.out_f32 + token * kPartFloats + c : nullptr;
        uint16_t* ob = a.out + token * kPartFloats + c;
#pragma unroll 1
        for (int hh = 0; hh < kHeads; hh += 16) {
          uint32_t ov[16];
          tc::tmem_ld_32x32b_x16(o_base + (uint32_t)hh, ov);
          tc::tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const float v = __uint_as_float(ov[j]) * s_inv[hh + j];
            if (!complete) {
              po[(hh + j) * kHeadDim] = v;
            } else {
              if (of) of[(hh + j) * kHeadDim] = v;
              ob[(hh + j) * kHeadDim] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
            }
          }
        }
        if (tid == 0 && whole && !last_of_token) {
          // the token's first part: its other parts lie with the next CTAs
          const int64_t last = f1 - 1 + (tiles - 1 - tile);  // the token's last tile in the list
          PartList pl;
          pl.token = (int32_t)token;
          pl.first_slot = slot;
          pl.cta0 = cta;
          pl.cta1 = (int32_t)(((last + 1) * G + total - 1) / total - 1);
          pl.tiles = total;
          a.lists[cta] = pl;
        }
        if (!last_of_run) {
          tc::tc_fence_before();
          write_rows();
          // S^T of this token is complete: Q may be replaced
          write_q(nseq.first + ntok);
#pragma unroll
          for (int j = 0; j < 16; ++j) l_acc[j] = 0.0f;
          first = true;
          whole = true;
          slot = 2 * cta + 1;
          tc::fence_proxy_async_smem();
          __syncthreads();  // s_mul, s_ref, s_red
          if (lane == 0) tc::mbar_arrive(bar_r);
          if (warp == 0) issue_s(par ^ 1u);
        }
      }
      b = nb;
      tok = ntok;
      tile = ntile;
      visible = nvisible;
      tiles = ntiles;
      seq = nseq;
      rows_seen = visible - tile * kRows;
      gone_now = gone;
    }
    if (*s_abort && warp == 0) {
      // a wait ran out: products in flight end before tensor memory is freed (one
      // more commit behind them, on a barrier of its own)
      uint64_t* bar_end = reinterpret_cast<uint64_t*>(sm + kOffMisc + 80);
      if (lane == 0) {
        tc::mbar_init(bar_end, 1);
        tc::fence_mbar_init();
        tc::mma_commit(bar_end);
        int never = 0;
        tc::mbar_wait_bounded(bar_end, 0, &never, &g_paged_attn_error, 100000000ull);
      }
      __syncwarp();
    }
  }
  tc::tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc::tc_fence_after();
    tc::tmem_dealloc(tmem, kTmemCols);
  }
}

// ---- the tokens whose tiles lie with several CTAs ---------------------------------
// One block per (token, head) at a time: out = sum_j 2^(ref_j - M) O_j / sum_j
// 2^(ref_j - M) l_j over the parts in list order, in a fixed tree (four groups
// of threads take every fourth part).
constexpr int kJoinThreads = 512;

__global__ void __launch_bounds__(kJoinThreads) paged_attn_join_kernel(Args a, int32_t G) {
  __shared__ int32_t s_list[1024];
  __shared__ int32_t s_n;
  __shared__ float s_w[1024];
  __shared__ int32_t s_slot[1024];
  __shared__ int32_t s_parts;
  __shared__ float s_inv;
  __shared__ __align__(16) float4 s_sum[3][128];
  pdl_begin();
  const int tid = threadIdx.x, lane = tid & 31;
  // the tokens to join, in order (G <= 1024: one place per thread, twice)
  if (tid < 32) {
    int n = 0;
    for (int c0 = 0; c0 < G; c0 += 32) {
      const bool has = c0 + lane < G && a.lists[c0 + lane].token >= 0;
      const uint32_t m = __ballot_sync(0xffffffffu, has);
      if (has) s_list[n + __popc(m & ((1u << lane) - 1u))] = c0 + lane;
      n += __popc(m);
    }
    if (lane == 0) s_n = n;
  }
  __syncthreads();
  const int items = s_n * kHeads;
  for (int it = blockIdx.x; it < items; it += gridDim.x) {
    const PartList pl = a.lists[s_list[it / kHeads]];
    const int h = it % kHeads;
    __syncthreads();  // the last item's shared values are done with
    if (tid < 32) {
      // the parts: the first one, then the CTAs up to cta1 that have tiles
      int n = 0;
      float M = kNoRef;
      for (int c0 = pl.cta0; c0 <= pl.cta1; c0 += 32) {
        const int c = c0 + lane;
        const bool has = c <= pl.cta1 && (c == pl.cta0 || pl.tiles * c / G < pl.tiles * (c + 1) / G);
        const uint32_t m = __ballot_sync(0xffffffffu, has);
        if (has) {
          const int at = n + __popc(m & ((1u << lane) - 1u));
          const int slot = c == pl.cta0 ? pl.first_slot : 2 * c;
          s_slot[at] = slot;
          const float2 ml = a.part_ml[(int64_t)slot * kHeads + h];
          if (ml.y > 0.0f) M = fmaxf(M, ml.x);
        }
        n += __popc(m);
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
      __syncwarp();
      float L = 0.0f;
      for (int j = lane; j < n; j += 32) {
        const float2 ml = a.part_ml[(int64_t)s_slot[j] * kHeads + h];
        const float w = ml.y > 0.0f ? fast_exp2(ml.x - M) : 0.0f;
        s_w[j] = w;
        L += w * ml.y;
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
      if (lane == 0) {
        s_parts = n;
        s_inv = L > 0.0f ? 1.0f / L : 0.0f;
        if (a.lse)
          a.lse[(int64_t)pl.token * kHeads + h] = L > 0.0f ? (M + log2f(L)) * 0.6931471805599453f : -INFINITY;
      }
    }
    __syncthreads();
    const int g = tid >> 7, c4 = tid & 127, n = s_parts;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int j = g; j < n; j += 4) {
      const float4 v =
          reinterpret_cast<const float4*>(a.part_o + (int64_t)s_slot[j] * kPartFloats + (int64_t)h * kHeadDim)[c4];
      const float w = s_w[j];
      // a part that saw nothing has weight 0 and zeros
      acc.x = fmaf(v.x, w, acc.x);
      acc.y = fmaf(v.y, w, acc.y);
      acc.z = fmaf(v.z, w, acc.z);
      acc.w = fmaf(v.w, w, acc.w);
    }
    if (g) s_sum[g - 1][c4] = acc;
    __syncthreads();
    if (g == 0) {
      const float inv = s_inv;
#pragma unroll
      for (int k = 0; k < 3; ++k) {
        const float4 v = s_sum[k][c4];
        acc.x += v.x;
        acc.y += v.y;
        acc.z += v.z;
        acc.w += v.w;
      }
      acc.x *= inv;
      acc.y *= inv;
      acc.z *= inv;
      acc.w *= inv;
      const int64_t o = ((int64_t)pl.token * kHeads + h) * kHeadDim + c4 * 4;
      if (a.out_f32) *reinterpret_cast<float4*>(a.out_f32 + o) = acc;
      const __nv_bfloat162 b0 = __floats2bfloat162_rn(acc.x, acc.y);
      const __nv_bfloat162 b1 = __floats2bfloat162_rn(acc.z, acc.w);
      *reinterpret_cast<uint2*>(a.out + o) =
          make_uint2(*reinterpret_cast<const uint32_t*>(&b0), *reinterpret_cast<const uint32_t*>(&b1));
    }
  }
}

}  // namespace pattn
}  // namespace csa2

using namespace csa2;

int csa2_read_and_clear_paged_attn_error(cudaStream_t s) {
  int v = 0, z = 0;
  if (cudaMemcpyFromSymbolAsync(&v, g_paged_attn_error, sizeof(int), 0, cudaMemcpyDeviceToHost, s) != cudaSuccess)
    return CSA2_ERR_CUDA;
  if (cudaMemcpyToSymbolAsync(g_paged_attn_error, &z, sizeof(int), 0, cudaMemcpyHostToDevice, s) != cudaSuccess)
    return CSA2_ERR_CUDA;
  if (cudaStreamSynchronize(s) != cudaSuccess) return CSA2_ERR_CUDA;
  return v;
}

static constexpr int kMaxCtas = 1024;  // the joining kernel's tables

static int paged_attn_ctas() {
  static int sms[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) {
    (void)cudaGetLastError();
    return 152;
  }
  if (!sms[dev]) {
    int v = 0;
    cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev);
    sms[dev] = v > 0 ? (v < kMaxCtas ? v : kMaxCtas) : 152;
  }
  return sms[dev];
}

static size_t al256(size_t x) { return (x + 255) / 256 * 256; }
static size_t part_o_bytes(int G) { return (size_t)2 * G * pattn::kPartFloats * 4; }
static size_t part_ml_bytes(int G) { return al256((size_t)2 * G * kHeads * sizeof(float2)); }

extern "C" size_t csa2_paged_attn_workspace_size(int32_t n_tokens, int32_t B) {
  if (n_tokens <= 0 || B <= 0) return 0;
  const int G = paged_attn_ctas();
  return part_o_bytes(G) + part_ml_bytes(G) + al256((size_t)G * sizeof(pattn::PartList));
}

extern "C" int csa2_paged_attn(const void* q_bf16, int32_t n_tokens, const int32_t* cu_q, int32_t B,
                               const uint8_t* kv_data, const uint8_t* kv_scale, int64_t n_pages, int32_t page_size,
                               const int32_t* page_table, int32_t max_pages, const int32_t* n_visible, int32_t causal,
                               float sm_scale, void* out_bf16, float* out_f32, float* lse, void* workspace,
                               size_t workspace_bytes, csa2_stream_t stream) {
  if (n_tokens > 0 && B != 0 && (!q_bf16 || !kv_data || !kv_scale || !n_visible || !out_bf16))
    return CSA2_ERR_INVALID_ARG;
  pattn::Args a{};
  if (int rc = paged_check(page_table, n_pages, page_size, max_pages, B, a.pages)) return rc;
  if (int rc = paged_runs(cu_q, n_tokens, B, a.per_seq)) return rc;
  if (!csa2_aligned(q_bf16, 16) || !csa2_aligned(kv_data, 16) || !csa2_aligned(kv_scale, 16) ||
      !csa2_aligned(out_bf16, 16) || !csa2_aligned(out_f32, 16) || !csa2_aligned(lse, 4) ||
      !csa2_aligned(n_visible, 4))
    return CSA2_ERR_ALIGNMENT;
  if (n_tokens == 0 || B == 0) return CSA2_OK;
  const int G = paged_attn_ctas();
  if (!workspace || !csa2_aligned(workspace, 256) ||
      workspace_bytes < csa2_paged_attn_workspace_size(n_tokens, B))
    return CSA2_ERR_WORKSPACE;
  a.q = (const uint16_t*)q_bf16;
  a.n_tokens = n_tokens;
  a.B = B;
  a.cu = cu_q;
  a.kv_data = kv_data;
  a.kv_scale = kv_scale;
  a.n_visible = n_visible;
  a.causal = causal != 0;
  a.scale_log2 = sm_scale * 1.4426950408889634f;
  a.out = (uint16_t*)out_bf16;
  a.out_f32 = out_f32;
  a.lse = lse;
  uint8_t* ws = (uint8_t*)workspace;
  a.part_o = (float*)ws;
  a.part_ml = (float2*)(ws + part_o_bytes(G));
  a.lists = (pattn::PartList*)(ws + part_o_bytes(G) + part_ml_bytes(G));
  static Csa2PerDeviceOnce optin;
  if (csa2_smem_optin((const void*)pattn::paged_attn_kernel, pattn::kSmemBytes, optin) != CSA2_OK) return CSA2_ERR_CUDA;
  cudaStream_t s = (cudaStream_t)stream;
  CSA2_LAUNCH_PDL(pattn::paged_attn_kernel, dim3((unsigned)G), dim3(pattn::kThreads), (size_t)pattn::kSmemBytes, s, a);
  CSA2_LAUNCH_PDL(pattn::paged_attn_join_kernel, dim3((unsigned)(2 * G)), dim3(pattn::kJoinThreads), (size_t)0, s, a,
                  (int32_t)G);
  return CSA2_OK;
}
