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
// 64 heads on N they take 2,560 cycles a tile: S^T with the rows from tensor
// memory 1,024 (32 a product, 48 from shared memory), O^T 1,536 (48: A and B
// both from shared memory). Beside them a tile costs 2,880 wavefronts of shared
// memory (the rows as fp16 written once, the codes read twice, P, the waits) and
// 3,060 issue slots per scheduler, most of them conversions: 65,536 codes, twice.
// Measured 4,600 to 4,900 cycles a tile: 32 sequences of 65,536 entries 288 us
// (954 TFLOP/s, 49 % of the measured bf16 rate; 2.1 TB/s), 2,048 tokens of a
// prompt behind 6,144 entries 1.93 ms (1,000 TFLOP/s), 24 sequences of 1 to 4
// tokens over up to 16,385 entries 108 us, one token over 317 entries 17 us (2.5
// the set-up, 2 the queries, 5 the tile's chain, 2 the output, 4 the joining
// kernel). A token costs 9,000 cycles beside its tiles, while the pipeline runs
// empty and full again (its queries converted 1,500, the first references 2,400,
// the output 3,600): four prompts of 512 tokens from their start, 2.5 tiles a
// token, take 183 us, twice what their tiles would.
//
// Tried and not kept (us for the 32 sequences at the time): all 16 warps in one
// role after another 470, with S^T from tensor memory 429; one warp for both
// products 549 (an issue blocks while the queue is full); rows by cp.async into
// private staging 418 (347 by tensor copies); eight warps that dequantise for S
// and O in turn 317 against 302 apart; every group by all eight of a set 303
// against 291 (twice the waits, 250 cycles each under load); one loop for both
// sets 330 against 295; a third place for O's groups and half the codes staged
// 316 against 291; the queries converted by the warps that feed S^T 332 against
// 291 (their loop then keeps less in registers).
//
// Work split: the tiles of all tokens in batch order form one list of units, cut
// into one equal run per SM. A token's first tile counts kTokenUnits units more
// than the others, about what a token costs beside its tiles (four prompts of 512
// tokens: 248 us with none, 187 with one, 179 with two, 184 with three). A run
// may begin and end inside a token; the parts of such a token go to the workspace
// and a second kernel joins them in order.
// Few long sequences and many short ones load the SMs alike, and the workspace
// (two parts per SM) does not grow with the batch.
#include <cudaTypedefs.h>

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

// Roles: warps 0 .. 7 take the softmax and the outputs, 8 .. 15 dequantise for
// S^T and 16 .. 23 for O^T, 24 and 25 issue the products for S^T and for O^T, 26
// walks the list and looks pages up, 27 copies the rows into shared memory. A
// warp's tensor-memory lanes are the quadrant warp % 4; the two warps of a
// quadrant in a role share its rows by heads (softmax) or by every second group
// of channels (dequantisation).
constexpr int kSoftWarps = 8, kFeedS = 8, kFeedO = 16, kSWarp = 24, kOWarp = 25, kWalkWarp = 26, kCopyWarp = 27;
constexpr int kThreads = 896;
constexpr int kWarps = kThreads / 32;
// Registers: 896 threads start with 72 each (64,512 in all, and all of them shared out).
constexpr int kRegsSoft = 112, kRegsFeed = 56, kRegsIssue = 56;
static_assert(256 * kRegsSoft + 512 * kRegsFeed + 128 * kRegsIssue <= kThreads * 72, "register split");
constexpr int kRows = 128;
constexpr int kPlacesA = 3, kPlaces = 2;  // rings of 128-channel groups of R, in tensor and in shared memory
constexpr int kBlkR = kRows * 128;        // 64 channels of R: [128 rows][128 B]
constexpr int kBlkQ = kHeads * 128;       // 64 channels of Q: [64 heads][128 B]
constexpr int kBlkP = kRows * kHeads * 2; // P: [128 rows][64 heads]
constexpr int kOffR = 0;                                // 2 groups of 2 blocks, 64 KiB
constexpr int kOffQ = kOffR + kPlaces * 2 * kBlkR;      // 8 blocks, 64 KiB
constexpr int kOffP = kOffQ + 8 * kBlkQ;                // 16 KiB
constexpr int kRawGroup = kRows * 64;                   // a group's codes, [128 rows][64 B] with the 64-byte swizzle
constexpr int kOffRaw = kOffP + kBlkP;              // two tiles' codes, group by group, 64 KiB
constexpr int kOffRawSc = kOffRaw + 8 * kRawGroup;      // and three tiles' scales, [128 rows][32 B], 12 KiB
constexpr int kOffMisc = kOffRawSc + 3 * kRows * kKvScales;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColS = 0;             // S^T: 64 columns (heads), lanes = rows
constexpr uint32_t kColO = 64;            // O^T: 4 blocks x 64 columns, lanes = channels
// R as the A operand of S^T: lanes = rows, 64 columns per 128 channels, a ring of
// three places
constexpr uint32_t kColA = 320;

// P = 2^(S' - ref): at most 2^kTop when ref is the maximum itself, at most
// 2^(kTop + kSlack) = 2^15 before ref moves, below fp16's 65,504. The offset
// kTop keeps weights down to 2^-25 of the maximum at fp16's full precision
// (2^-14 is its smallest normal), and to 2^-35 above zero.
constexpr float kTop = 11.0f, kSlack = 4.0f;

constexpr int kPartFloats = kHeads * kHeadDim;

// Tries of a wait (200 ns each or more) before it gives up.
#ifdef CSA2_WAIT_LIMIT
constexpr uint32_t kWaitTries = CSA2_WAIT_LIMIT / 32;  // (a look takes about 32 clocks)
#else
constexpr uint32_t kWaitTries = 1u << 22;
#endif

// A part of a token that more than one CTA works on, for the joining kernel.
struct PartList {
  int32_t token;       // -1: this CTA begins no such token
  int32_t first_slot;  // slot of the first part
  int32_t cta0, cta1;  // its first and last tile's CTAs
  int64_t units;       // of the whole call
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
// Unit u of a token with n tiles, u = 0 .. n + kTokenUnits - 1: tile i is at unit
// i + kTokenUnits, the ones before belong to its first tile's cost. A CTA has the
// tiles whose units are in its run.
constexpr int kTokenUnits = 2;
__device__ __forceinline__ int32_t tiles_of(int32_t visible) {  // a token without entries has one empty tile
  return visible <= kRows ? 1 : (int32_t)(((uint32_t)visible + kRows - 1) / kRows);
}
// sum of ceil(v / 128) for v = 1 .. x
__device__ __forceinline__ int64_t tiles_upto(int64_t x) {
  const int64_t n = x / kRows, r = x % kRows;
  return kRows * (n * (n + 1) / 2) + (n + 1) * r;
}
struct Seq {
  int32_t first, count;  // token rows
  int32_t visible;       // entries of its last token (of every one if not causal)
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
__device__ __forceinline__ int32_t visible_of(const Args& a, const Seq& s, int32_t t) {
  return a.causal ? s.visible - s.count + 1 + t : s.visible;
}
// tiles of the sequence's first n tokens
__device__ __forceinline__ int64_t tiles_before(const Args& a, const Seq& s, int32_t n) {
  if (!a.causal) return (int64_t)n * tiles_of(s.visible);
  const int64_t v0 = (int64_t)s.visible - s.count + 1;              // entries of token 0
  const int64_t blind = v0 > 0 ? 0 : 1 - v0 < n ? 1 - v0 : n;       // tokens that see nothing
  const int64_t hi = v0 + n - 1;                                    // entries of the last of the n
  return blind + (hi > 0 ? tiles_upto(hi) - tiles_upto(v0 > 1 ? v0 - 1 : 0) : 0);
}

// The place of unit `at` of a sequence: its token, and how many of that token's
// tiles lie before the unit.
struct Place {
  int32_t tok, tile;
};
__device__ __forceinline__ Place place_of(const Args& a, const Seq& s, int64_t at) {
  int32_t lo = 0, hi = s.count;  // units before lo <= at < units before hi
  while (hi - lo > 1) {
    const int32_t mid = lo + (hi - lo) / 2;
    if (tiles_before(a, s, mid) + (int64_t)kTokenUnits * mid <= at) lo = mid;
    else hi = mid;
  }
  const int64_t off = at - tiles_before(a, s, lo) - (int64_t)kTokenUnits * lo - kTokenUnits;
  return {lo, off > 0 ? (int32_t)off : 0};
}

// A walk along the list.
struct Walk {
  int32_t b, tok;
  Seq seq;
  int32_t tile, visible, tiles;  // the place in the token, its entries and tiles
  __device__ __forceinline__ void start(const Args& a, int32_t b_, int32_t tok_, int32_t tile_) {
    b = b_;
    seq = load_seq(a, b, false);
    tok = tok_;
    tile = tile_;
    visible = visible_of(a, seq, tok);
    tiles = tiles_of(visible);
  }
  // only called while the list has a tile behind this one
  __device__ __forceinline__ void step(const Args& a) {
    if (++tile < tiles) return;
    tile = 0;
    ++tok;
    while (tok >= seq.count) {
      ++b;
      seq = load_seq(a, b, false);
      tok = 0;
    }
    visible = visible_of(a, seq, tok);
    tiles = tiles_of(visible);
  }
};
// What the roles need to know of a tile, in a ring of kRing tiles.
constexpr int kRing = 8;
struct Info {
  int32_t page[8];  // the table's entries for its rows, 16 at a time
  int32_t rows;     // entries of the token from the tile's first row on
  int32_t at;       // its first entry
  int32_t token;    // row of q
  int32_t left;     // tiles of the token behind this one
  int32_t some;     // the tile has a row whose page is there
};

// Shared memory behind the operands.
struct __align__(16) Shared {
  Info info[kRing];
  float mul[kHeads];      // sm_scale log2(e) 2^-k of the head's fp16 queries
  float ref[kHeads];      // reference of P, log2 domain, less kTop
  float red[4][kHeads];   // per-quadrant maxima, then sums
  float up[kHeads];       // how far a reference moves; at a token's end what O^T is multiplied with
  float shrink[kHeads];   // what O^T and l shrink by when a reference moves
  int64_t scan[kWarps];   // tiles of the warps' sequences
  int32_t scan_tok[kWarps];  // and tokens
  int64_t tile0, tile1;   // tiles of the list before the run and at its end
  int64_t units, end_unit;  // of the list; behind the run
  Place first;            // the run's first tile, within its sequence
  int32_t seq;            // that sequence
  uint32_t tmem;
  volatile int abort;
  // barriers. Those of a tile complete once per tile, so that tile j waits for
  // phase j; those of a place once per use.
  uint64_t full[kPlacesA];    // a group is in its place in tensor memory: 4 warps
  uint64_t empty[kPlacesA];   // S^T over it is done
  uint64_t raw[8];            // a group's codes have arrived (group 0's: and the tile's scales)
  uint64_t raw_read[8];       // and been read: 8 warps (group 0's: waited for by all 16, for the scales)
  uint64_t r_full[kPlaces];   // a group is in its place in shared memory: 4 warps
  uint64_t r_empty[kPlaces];  // its channels of O^T are done
  uint64_t q_raw;             // a token's queries have arrived as they are
  uint64_t q;                 // and are fp16: 8 warps
  uint64_t s;                 // S^T complete
  uint64_t s_read;            // S^T read: 8 warps
  uint64_t p;                 // P written, O^T rescaled (or read out): 8 warps
  uint64_t o;                 // O^T complete
  uint64_t info_full[kRing];
  uint64_t info_used[kRing];  // 27 warps
  uint64_t soft;              // the softmax's warps meet at a token's end: 8 warps
  uint64_t end[2];
};
// (no static shared memory: dynamic shared memory then starts 1,024-byte aligned)
constexpr int kSmemBytes = kOffMisc + (int)sizeof(Shared);
static_assert(kSmemBytes <= 232448, "shared memory of one block");

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

// A token's queries on their way to q_smem, issued by the elected thread without
// a branch (the issuing loop has to stay uniform).
__device__ __forceinline__ void load_q_one(uint32_t elected, uint32_t q_smem, const CUtensorMap* map, int32_t token,
                                           uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %0, 0;\n\t"
      "@p mbarrier.arrive.expect_tx.shared::cta.b64 _, [%1], %2;\n\t}" ::"r"(elected),
      "r"(tc::smem_u32(bar)), "r"(8 * kBlkQ)
      : "memory");
#pragma unroll
  for (int b = 0; b < 8; ++b)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %0, 0;\n\t"
        "@p cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%1], "
        "[%2, {%3, %4, %5}], [%6];\n\t}" ::"r"(elected),
        "r"(q_smem + b * kBlkQ), "l"(reinterpret_cast<uint64_t>(map)), "r"(64 * b), "r"(0), "r"(token),
        "r"(tc::smem_u32(bar))
        : "memory");
}

__global__ void __launch_bounds__(kThreads, 1)
    paged_attn_kernel(const __grid_constant__ CUtensorMap rows_map, const __grid_constant__ CUtensorMap q_map,
                      Args a) {
  extern __shared__ __align__(1024) uint8_t sm[];
  uint8_t* sR = sm + kOffR;
  uint8_t* sQ = sm + kOffQ;
  uint8_t* sP = sm + kOffP;
  Shared& sh = *reinterpret_cast<Shared*>(sm + kOffMisc);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = (int)gridDim.x, cta = (int)blockIdx.x;

  if (tid == 0) {
    for (int i = 0; i < kPlacesA; ++i) {
      tc::mbar_init(sh.full + i, 4);
      tc::mbar_init(sh.empty + i, 1);
    }
    for (int i = 0; i < kPlaces; ++i) {
      tc::mbar_init(sh.r_full + i, 4);
      tc::mbar_init(sh.r_empty + i, 1);
    }
    for (int i = 0; i < 8; ++i) {
      tc::mbar_init(sh.raw + i, 1);
      tc::mbar_init(sh.raw_read + i, i % 4 ? 8 : 16);
    }
    tc::mbar_init(&sh.q_raw, 1);
    tc::mbar_init(&sh.q, kSoftWarps);
    tc::mbar_init(&sh.s, 1);
    tc::mbar_init(&sh.s_read, kSoftWarps);
    tc::mbar_init(&sh.p, kSoftWarps);
    tc::mbar_init(&sh.o, 1);
    tc::mbar_init(&sh.soft, kSoftWarps);
    for (int i = 0; i < 2; ++i) tc::mbar_init(sh.end + i, 1);
    for (int i = 0; i < kRing; ++i) {
      tc::mbar_init(sh.info_full + i, 1);
      tc::mbar_init(sh.info_used + i, 27);
    }
    sh.abort = 0;
    sh.seq = -1;
    tc::fence_mbar_init();
  }
  if (warp == 0) tc::tmem_alloc(&sh.tmem, kTmemCols);
  pdl_begin();

  // ---- this CTA's run [f0, f1) of the list's units: a scan over the sequences'
  // tiles and tokens, kThreads at a time. The total is known behind the last ones
  // only, so where there are more sequences than threads they are gone through
  // once more ----
  int64_t tiles = 0, n = 0, lo = 0;    // lo: tiles before this thread's sequence, n: its own
  int32_t tokens_all = 0, lo_tok = 0;  // and tokens
  Seq own{};
  const auto scan = [&](int32_t b, bool report) {
    own = b < a.B ? load_seq(a, b, report) : Seq{0, 0, 0};
    n = tiles_before(a, own, own.count);
    int64_t incl = n;
    int32_t incl_tok = own.count;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
      const int32_t w = __shfl_up_sync(0xffffffffu, incl_tok, o);
      if (lane >= o) incl += v, incl_tok += w;
    }
    if (lane == 31) sh.scan[warp] = incl, sh.scan_tok[warp] = incl_tok;
    __syncthreads();
    const int64_t of_warp = lane < kWarps ? sh.scan[lane] : 0;
    const int32_t of_warp_tok = lane < kWarps ? sh.scan_tok[lane] : 0;
    int64_t before = of_warp;
    int32_t before_tok = of_warp_tok;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t v = __shfl_up_sync(0xffffffffu, before, o);
      const int32_t w = __shfl_up_sync(0xffffffffu, before_tok, o);
      if (lane >= o) before += v, before_tok += w;
    }
    lo = tiles + incl - n + __shfl_sync(0xffffffffu, before - of_warp, warp);
    lo_tok = tokens_all + incl_tok - own.count + __shfl_sync(0xffffffffu, before_tok - of_warp_tok, warp);
    tiles += __shfl_sync(0xffffffffu, before, kWarps - 1);
    tokens_all += __shfl_sync(0xffffffffu, before_tok, kWarps - 1);
    __syncthreads();
  };
  for (int32_t b0 = 0; b0 < a.B; b0 += kThreads) scan(b0 + tid, cta == 0);
  const int64_t all = tiles + (int64_t)kTokenUnits * tokens_all, f0 = all * cta / G, f1 = all * (cta + 1) / G;
  if (tid == 0) {
    a.lists[cta].token = -1;
    sh.tile0 = sh.tile1 = tiles;  // (a run that ends with the list)
    sh.units = all;
    sh.end_unit = f1;
  }
  __syncthreads();
  const auto place = [&](int32_t b) {
    const int64_t u = lo + (int64_t)kTokenUnits * lo_tok, end = u + n + (int64_t)kTokenUnits * own.count;
    if (f0 >= u && f0 < end) {
      const Place at = place_of(a, own, f0 - u);
      sh.seq = b;
      sh.first = at;
      sh.tile0 = lo + tiles_before(a, own, at.tok) + at.tile;
    }
    if (f1 >= u && f1 < end) {
      const Place at = place_of(a, own, f1 - u);
      sh.tile1 = lo + tiles_before(a, own, at.tok) + at.tile;
    }
  };
  if (a.B <= kThreads) {
    place(tid);
  } else if (f0 < f1) {
    tiles = 0;
    tokens_all = 0;
    for (int32_t b0 = 0; b0 < a.B && tiles + (int64_t)kTokenUnits * tokens_all <= f1; b0 += kThreads) {
      scan(b0 + tid, false);
      place(b0 + tid);
    }
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = sh.tmem;
  // tiles of this CTA (the host has checked the range); reduced over equal values,
  // so that the compiler knows it as the warp's: the loops below cost 3 % more else
  const int32_t n_run = (int32_t)__reduce_max_sync(0xffffffffu, (uint32_t)(sh.tile1 - sh.tile0));

  // A wait that runs out (kWaitTries, a tenth of a second at least) raises
  // sh.abort, on which every later wait gives up at once and nothing more is
  // issued. The loops then run to their ends all the same, so that no warp is
  // missing at a barrier.sync, but write no more outputs, and TIMEOUT is recorded. An
  // Info that was not waited for names no token, and warps may read it differently:
  // where its word decides, the softmax's warps meet at an mbarrier (meet()), not at
  // a barrier.sync. What was issued is waited for by the warp that issued it, behind
  // its loop and whatever became of the run.
  // (Counted, not timed, and kept short: the code of all roles together has to
  // stay in the instruction cache.)
  const auto wait = [&](uint64_t* bar, uint32_t par) {
    if (!tc::mbar_look(bar, par & 1u, 0)) {
      uint32_t n = 0;
      while (!tc::mbar_look(bar, par & 1u, 200u)) {
        if (sh.abort || ++n >= kWaitTries) {
          sh.abort = 1;
          break;
        }
      }
    }
    __syncwarp();
  };
  const auto arrive = [&](uint64_t* bar) {  // once per warp, after all its lanes' work
    __syncwarp();
    if (lane == 0) tc::mbar_arrive(bar);
  };
  // tile j's Info; info_done() when a warp is done with it
  const auto info_of = [&](int32_t j) -> const Info& {
    wait(sh.info_full + j % kRing, (uint32_t)(j / kRing));
    return sh.info[j % kRing];
  };
  const auto info_done = [&](int32_t j) { arrive(sh.info_used + j % kRing); };
  const int quad = warp & 3, half = (warp >> 2) & 1;
  const int my_row = quad * 32 + lane;  // of a tile
  const uint32_t lanes = (uint32_t)(quad * 32) << 16;

  if (warp >= kSWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsIssue));
    // The two issuing warps. An issue blocks while the tensor pipe's queue is
    // full, and S^T of a tile and O^T of the one before depend on different
    // things: one warp for both would wait for each in turn. The votes say what is
    // so: every branch around the products is the whole warp's. Only then does the
    // compiler keep their operands in uniform registers; else each product costs
    // moves there, 80 to 100 cycles against the 32 or 48 of the tensor pipe.
    const auto all = [](bool c) { return __any_sync(0xffffffffu, c) != 0; };
    const uint32_t elected = tc::elect_one();
    uint32_t tokens = 0;  // of the run, begun by the warp that issues S^T
    if (warp == kSWarp) {
      constexpr uint32_t idesc = idesc_f16(128, 64, 0, 0);
      const uint32_t q_lo = tc::smem_u32(sQ);
      uint32_t place = 0, use = 0;  // the ring's next place, and how often it went round
#pragma unroll 1
      for (int32_t j = 0; all(j < n_run); ++j) {
        const Info& info = info_of(j);
        if (all(j > 0)) wait(&sh.s_read, (uint32_t)(j - 1));
        if (all(sh.abort != 0)) break;
        if (all(info.at == 0 || j == 0)) {
          // a new token: its queries take the place of the last one's (S^T of whose
          // last tile has been read, so it is complete) while that token's last
          // softmax runs
          load_q_one(elected, q_lo, &q_map, info.token, &sh.q_raw);
          wait(&sh.q, tokens++);
          if (all(sh.abort != 0)) break;
        }
#pragma unroll 1
        for (int g = 0; g < 4; ++g) {  // channels 128 g ..
          wait(sh.full + place, use);
          tc::tc_fence_after();
          const uint32_t at = tmem + kColA + 64u * place;
          const uint64_t bd = tc::smem_desc(q_lo + (uint32_t)(2 * g * kBlkQ), 0, 1024, tc::kSwizzle128B);
#pragma unroll
          for (int k = 0; k < 8; ++k)  // block 2g + k / 4 of 64 channels, K step k % 4
            tc::mma_f16_ta_one(elected, tmem + kColS, at + 8u * (uint32_t)k,
                               bd + (uint64_t)((k >> 2) * (kBlkQ >> 4) + (k & 3) * 2), idesc,
                               k ? 1u : (uint32_t)(g != 0));
          tc::mma_commit_one(elected, sh.empty + place);
          place = place + 1 == kPlacesA ? 0 : place + 1;
          use += place == 0 ? 1u : 0u;
        }
        tc::mma_commit_one(elected, &sh.s);
        info_done(j);
      }
    } else if (warp == kOWarp) {
      constexpr uint32_t idesc = idesc_f16(128, 64, 1, 1);  // A = R^T and B = P^T are MN-major
      const uint32_t r_lo = tc::smem_u32(sR), p_lo = tc::smem_u32(sP);
      uint32_t place = 0, use = 0;
#pragma unroll 1
      for (int32_t j = 0; all(j < n_run); ++j) {
        const uint32_t more = j > 0 && info_of(j).at != 0 ? 1u : 0u;  // 0: O^T starts anew
        wait(&sh.p, (uint32_t)j);
        if (all(sh.abort != 0)) break;
#pragma unroll 1
        for (int mb = 0; mb < 4; ++mb) {  // 128 channels
          wait(sh.r_full + place, use);
          tc::tc_fence_after();
          const uint64_t ad = tc::smem_desc(r_lo + place * (uint32_t)(2 * kBlkR), kBlkR, 1024, tc::kSwizzle128B);
          const uint64_t bd = tc::smem_desc(p_lo, 0, 1024, tc::kSwizzle128B);
#pragma unroll
          for (int k = 0; k < 8; ++k)  // 16 rows
            tc::mma_f16_one(elected, tmem + kColO + 64u * (uint32_t)mb, ad + (uint64_t)((k * 16 * 128) >> 4),
                            bd + (uint64_t)((k * 16 * 128) >> 4), idesc, k ? 1u : more);
          tc::mma_commit_one(elected, sh.r_empty + place);
          place = place + 1 == kPlaces ? 0 : place + 1;
          use += place == 0 ? 1u : 0u;
        }
        tc::mma_commit_one(elected, &sh.o);
        info_done(j);
      }
    } else if (warp == kWalkWarp && n_run > 0) {
      Walk w;
      w.start(a, sh.seq, sh.first.tok, sh.first.tile);
#pragma unroll 1
      for (int32_t j = 0; j < n_run; ++j) {
        const int32_t e = w.tile * kRows + 16 * lane;
        int32_t page = -1;
        if (lane < 8 && e < w.visible) {
          page = a.pages.table[(int64_t)w.b * a.pages.max_pages + (e >> a.pages.shift)];
          if (page < 0 || page >= a.pages.n_pages) {
            page = -1;
            record_error(&g_paged_attn_error, CSA2_ERR_DEVICE);
          }
        }
        const int some = __any_sync(0xffffffffu, page >= 0);
        if (j >= kRing) wait(sh.info_used + j % kRing, (uint32_t)(j / kRing) - 1u);
        Info& to = sh.info[j % kRing];
        if (lane < 8) to.page[lane] = page;
        if (lane == 0) {
          to.rows = w.visible - w.tile * kRows;
          to.at = w.tile * kRows;
          to.token = w.seq.first + w.tok;
          to.left = w.tiles - 1 - w.tile;
          to.some = some;
        }
        // (a later token's queries into L2, up to kRing tiles before they are needed)
        if (lane == 0 && j > 0 && w.tile == 0)
          asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(a.q + (int64_t)to.token * kPartFloats),
                       "r"(kPartFloats * 2)
                       : "memory");
        arrive(sh.info_full + j % kRing);
        if (j + 1 < n_run) w.step(a);
      }
    } else if (warp == kCopyWarp) {
      // a run of rows is a whole small page, or the tile's piece of a page; a
      // group's 64 bytes of its rows are one tensor copy, its scales a bulk copy.
      // What a missing run leaves behind is never used (its scales count as 0).
      const int run_shift = a.pages.shift < 7 ? a.pages.shift : 7;
      const int run = 1 << run_shift;
      const auto aborted = [&] { return __any_sync(0xffffffffu, sh.abort != 0); };
      uint32_t armed = 0;  // groups whose barrier expects a copy: nothing expects one that is not issued
#pragma unroll 1
      for (int32_t j = 0; j < n_run && !aborted(); ++j) {
        const Info& info = info_of(j);
        // lane i: run i
        const int r0 = lane << run_shift;
        const int32_t page = r0 < kRows && r0 < info.rows ? info.page[r0 >> 4] : -1;
        const uint32_t there = __popc(__ballot_sync(0xffffffffu, page >= 0));
        const int64_t row = ((int64_t)page << a.pages.shift) + ((info.at + r0) & (a.pages.page_size() - 1));
#pragma unroll 1
        for (int g = 0; g < 4; ++g) {
          const int at = 4 * (j & 1) + g;
          if (j > 1) wait(sh.raw_read + at, (uint32_t)(j >> 1) - 1u);
          if (aborted()) break;
          if (lane == 0) tc::mbar_arrive_expect_tx(sh.raw + at, there * (uint32_t)run * (g ? 64 : 64 + kKvScales));
          __syncwarp();
          if (page >= 0) {
            tc::tma_load_2d(sm + kOffRaw + at * kRawGroup + r0 * 64, &rows_map, g * 64, (int32_t)row, sh.raw + at);
            // (tile j - 3 is done with its scales: its groups were waited for before tile j - 1's were copied)
            if (g == 0)
              tc::bulk_load(sm + kOffRawSc + (j % 3 * kRows + r0) * kKvScales, a.kv_scale + row * kKvScales,
                            (uint32_t)(run * kKvScales), sh.raw + at);
          }
          __syncwarp();
          ++armed;
        }
        info_done(j);
      }
      // (the warps that read the last copies wait for them too, but not when a wait ran out)
      for (uint32_t i = armed > 8 ? armed - 8 : 0; i < armed; ++i) tc::mbar_wait_issued(sh.raw + i % 8, i / 8);
    }
    if ((warp == kSWarp || warp == kOWarp) && n_run > 0) {
      // products in flight end before tensor memory is freed
      tc::mma_commit_one(elected, sh.end + (warp - kSWarp));
      tc::mbar_wait_issued(sh.end + (warp - kSWarp), 0);
      if (tokens > 0) tc::mbar_wait_issued(&sh.q_raw, tokens - 1u);
      __syncwarp();
    }
  } else if (warp >= kFeedS) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsFeed));
    // ---- dequantise: a thread takes the channels of groups half and half + 2
    // (128 each: 64 bytes of codes, 8 of scales) of its row from where the copies
    // put them, eight warps into tensor memory for S^T and eight into shared
    // memory for O^T. (Plain loads from the pool into registers made a warp wait
    // for them at the next use of their scoreboard, 3,400 cycles a tile.) The
    // codes are given back as soon as they are in registers: the next tile's
    // copies do not wait for this tile's products ----
    struct Raw {
      uint32_t w[16];
      uint2 sc;
    };
    auto take = [&](Raw& r, int32_t t, int g, bool seen) {
      const uint8_t* src = sm + kOffRaw + (4 * (t & 1) + g) * kRawGroup;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint4 v = *reinterpret_cast<const uint4*>(src + tc::sw64_offset((uint32_t)my_row, (uint32_t)k));
        r.w[4 * k] = v.x;
        r.w[4 * k + 1] = v.y;
        r.w[4 * k + 2] = v.z;
        r.w[4 * k + 3] = v.w;
      }
      // (codes are finite whatever they are: times 0 they are zeros)
      r.sc = *reinterpret_cast<const uint2*>(sm + kOffRawSc + (t % 3 * kRows + my_row) * kKvScales + g * 8);
      if (!seen) r.sc = make_uint2(0u, 0u);
    };
    // channels 32 q .. +31 of a group as fp16 (exact; zeros for zero codes and scales)
    auto convert = [&](const Raw& r, int q, uint32_t (&o)[16]) {
      const uint32_t s2 = e4m3x2_to_f16x2(((q < 2 ? r.sc.x : r.sc.y) >> ((q & 1) * 16)) & 0xFFFFu);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t s = __byte_perm(s2, 0u, k < 2 ? 0x1010u : 0x3232u);
        uint32_t o0, o1, o2, o3;
        e2m1x8_to_f16(r.w[4 * q + k], o0, o1, o2, o3);
        o[4 * k] = mul_f16x2(o0, s);
        o[4 * k + 1] = mul_f16x2(o1, s);
        o[4 * k + 2] = mul_f16x2(o2, s);
        o[4 * k + 3] = mul_f16x2(o3, s);
      }
    };
    if (warp < kFeedO) {
#pragma unroll 1
      for (int32_t t = 0; t < n_run; ++t) {
        const Info& info = info_of(t);
        const bool seen = my_row < info.rows && info.page[my_row >> 4] >= 0;
        wait(sh.raw + 4 * (t & 1), (uint32_t)(t >> 1));
        if (half) arrive(sh.raw_read + 4 * (t & 1));  // (its own groups' codes come apart)
#pragma unroll 1
        for (int g = half; g < 4; g += 2) {
          Raw r;
          if (g) wait(sh.raw + 4 * (t & 1) + g, (uint32_t)(t >> 1));
          take(r, t, g, seen);
          arrive(sh.raw_read + 4 * (t & 1) + g);
          const uint32_t n = 4u * (uint32_t)t + (uint32_t)g, use = n / kPlacesA, place = n - use * kPlacesA;
          if (use > 0) wait(sh.empty + place, use - 1u);
          tc::tc_fence_after();
          const uint32_t at = tmem + lanes + kColA + 64u * place;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint32_t o[16];
            convert(r, q, o);
            tc::tmem_st_32x32b_x16(at + 16u * (uint32_t)q, o);
          }
          tc::tmem_st_wait();
          tc::tc_fence_before();
          arrive(sh.full + place);
        }
        info_done(t);
      }
    } else {
      // (a warp's groups all go to place half: the eight lanes of a store phase are
      // eight rows, eight bank groups)
#pragma unroll 1
      for (int32_t t = 0; t < n_run; ++t) {
        const Info& info = info_of(t);
        const bool seen = my_row < info.rows && info.page[my_row >> 4] >= 0;
        wait(sh.raw + 4 * (t & 1), (uint32_t)(t >> 1));
        if (half) arrive(sh.raw_read + 4 * (t & 1));  // (its own groups' codes come apart)
#pragma unroll 1
        for (int g = half; g < 4; g += 2) {
          Raw r;
          if (g) wait(sh.raw + 4 * (t & 1) + g, (uint32_t)(t >> 1));
          take(r, t, g, seen);
          arrive(sh.raw_read + 4 * (t & 1) + g);
          const uint32_t use = 2u * (uint32_t)t + (uint32_t)(g >> 1);
          if (use > 0) wait(sh.r_empty + half, use - 1u);
          uint8_t* blk = sR + half * (2 * kBlkR);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint32_t o[16];
            convert(r, q, o);
#pragma unroll
            for (int k = 0; k < 4; ++k)
              *reinterpret_cast<uint4*>(blk + (q >> 1) * kBlkR +
                                        tc::sw128_offset((uint32_t)my_row, (uint32_t)((q & 1) * 4 + k))) =
                  make_uint4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
          }
          tc::fence_proxy_async_smem();
          arrive(sh.r_full + half);
        }
        info_done(t);
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoft));
    if (n_run > 0) {
      // ---- softmax: a thread takes heads 32 half .. +31 of its row ----
      const int h0 = half * 32;
      // the token's queries, once they have arrived, as fp16 with a power-of-two
      // scale per head (exact but for values below 2^-28 of the head's largest), in
      // place: eight threads to a head, thread c with the 16-byte column c of each
      // 64-channel block (eight bank groups a row); 32 heads, then the other 32
      auto convert_q = [&](uint32_t token) {
        wait(&sh.q_raw, token);
#pragma unroll 1
        for (int h = tid >> 3; h < kHeads; h += 32) {
          uint8_t* at = sQ + tc::sw128_offset((uint32_t)h, (uint32_t)tid & 7u);
          uint32_t m2 = 0;  // the largest of the even and of the odd channels
          uint4 v[8];
#pragma unroll
          for (int b = 0; b < 8; ++b) v[b] = *reinterpret_cast<const uint4*>(at + b * kBlkQ);
#pragma unroll
          for (int b = 0; b < 8; ++b) {
            m2 = __vmaxu2(__vmaxu2(m2, v[b].x & 0x7FFF7FFFu), v[b].y & 0x7FFF7FFFu);
            m2 = __vmaxu2(__vmaxu2(m2, v[b].z & 0x7FFF7FFFu), v[b].w & 0x7FFF7FFFu);
          }
#pragma unroll
          for (int o = 1; o < 8; o <<= 1) m2 = __vmaxu2(m2, __shfl_xor_sync(0xffffffffu, m2, o));
          const uint32_t amax = max(m2 & 0xFFFFu, m2 >> 16);
          int k2 = 0;
          if (amax != 0u) k2 = min(14 - ((int)(amax >> 7) - 127), 126);  // (-113 at least: both powers are normal)
          const float up = __int_as_float((127 + k2) << 23);
#pragma unroll
          for (int b = 0; b < 8; ++b) {
            const uint32_t w[4] = {v[b].x, v[b].y, v[b].z, v[b].w};
            uint32_t o[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              o[e] = f32x2_to_f16x2(__uint_as_float(w[e] << 16) * up, __uint_as_float(w[e] & 0xFFFF0000u) * up);
            *reinterpret_cast<uint4*>(at + b * kBlkQ) = make_uint4(o[0], o[1], o[2], o[3]);
          }
          if ((tid & 7) == 0) sh.mul[h] = a.scale_log2 * __int_as_float((127 - k2) << 23);
        }
        tc::fence_proxy_async_smem();
        arrive(&sh.q);
      };

      float l_acc[32];  // this row lane's share of l
#pragma unroll
      for (int i = 0; i < 32; ++i) l_acc[i] = 0.0f;
      if (tid < kHeads) sh.ref[tid] = 0.0f;
      uint32_t tokens = 0;  // of the run, with queries converted
      // three times at a token's end, twice at the run's: phases 3 (tokens - 1) .. (not
      // wait(): the shorter loop is 0.5 % of a prompt chunk)
      const auto meet = [&](uint32_t phase) {
        arrive(&sh.soft);
        for (uint32_t n = 0; !tc::mbar_try_wait(&sh.soft, phase & 1u) && !sh.abort;)
          if (++n >= kWaitTries) sh.abort = 1;
        __syncwarp();
      };
      convert_q(tokens++);
      named_barrier(8, kSoftWarps * 32);  // mul, ref
      int slot = 2 * cta;               // where a part of the present token goes
      bool whole = info_of(0).at == 0;  // the CTA has the token from its first tile on
      bool first = true;                // the CTA's first tile of the token
      bool open = true;                 // the references are not set yet
#pragma unroll 1
      for (int32_t j = 0; j < n_run; ++j) {
        const uint32_t par = (uint32_t)j & 1u;
        const Info& info = info_of(j);
        const bool rv = my_row < info.rows && info.page[my_row >> 4] >= 0;

        wait(&sh.s, par);
        tc::tc_fence_after();
        uint32_t pr[32];
        tc::tmem_ld_32x32b_x32(tmem + lanes + kColS + (uint32_t)h0, pr);
        tc::tmem_ld_wait();
        tc::tc_fence_before();
        arrive(&sh.s_read);
        // S' - ref
        float top = -INFINITY;
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
          const float4 m4 = *reinterpret_cast<const float4*>(sh.mul + h0 + i);
          const float4 r4 = *reinterpret_cast<const float4*>(sh.ref + h0 + i);
          const float t0 = fmaf(__uint_as_float(pr[i]), m4.x, -r4.x);
          const float t1 = fmaf(__uint_as_float(pr[i + 1]), m4.y, -r4.y);
          const float t2 = fmaf(__uint_as_float(pr[i + 2]), m4.z, -r4.z);
          const float t3 = fmaf(__uint_as_float(pr[i + 3]), m4.w, -r4.w);
          top = fmaxf(fmaxf(fmaxf(top, t0), fmaxf(t1, t2)), t3);
          pr[i] = __float_as_uint(t0);
          pr[i + 1] = __float_as_uint(t1);
          pr[i + 2] = __float_as_uint(t2);
          pr[i + 3] = __float_as_uint(t3);
        }
        if (!rv) {
#pragma unroll
          for (int i = 0; i < 32; ++i) pr[i] = 0xFF800000u;  // -inf
        }
        if (group_any(1 + half, open || (rv && top > kTop + kSlack))) {
          // a head's scores passed its reference (or it has none yet): new
          // references, O^T and l to match
#pragma unroll
          for (int u = 0; u < 32; u += 16) {
            float v[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(pr[u + i]);
            const float m = warp_transpose_reduce16<true>(v, lane);
            if (lane < 16) sh.red[quad][h0 + u + lane] = m;
          }
          named_barrier(1 + half, 128);
          if (quad == 0) {
            const int h = h0 + lane;
            const float mt = fmaxf(fmaxf(sh.red[0][h], sh.red[1][h]), fmaxf(sh.red[2][h], sh.red[3][h]));
            const bool move = open ? mt > -INFINITY : mt > kTop + kSlack;
            const float up = move ? mt - kTop : 0.0f;
            sh.ref[h] += up;
            sh.up[h] = up;
            sh.shrink[h] = open ? 1.0f : fast_exp2(-up);  // (before the first reference O^T and l are 0)
          }
          // (a tile with a row sets every head's reference, of a head whose scores are all
          // -inf or NaN as well: the next tile's maxima may not be taken for the first)
          open = open && !info.some;
          named_barrier(1 + half, 128);
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            pr[i] = __float_as_uint(__uint_as_float(pr[i]) - sh.up[h0 + i]);
            l_acc[i] *= sh.shrink[h0 + i];
          }
          if (!first) {
            wait(&sh.o, (uint32_t)(j - 1));
            tc::tc_fence_after();
#pragma unroll 1
            for (int x = 0; x < 8; ++x) {  // channel block x / 2, heads h0 + 16 (x % 2) ..
              const int u = (x & 1) * 16;
              const uint32_t at = tmem + lanes + kColO + 64u * (uint32_t)(x >> 1) + (uint32_t)(h0 + u);
              uint32_t ov[16];
              tc::tmem_ld_32x32b_x16(at, ov);
              tc::tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 16; ++i) ov[i] = __float_as_uint(__uint_as_float(ov[i]) * sh.shrink[h0 + u + i]);
              tc::tmem_st_32x32b_x16(at, ov);
            }
            tc::tmem_st_wait();
            tc::tc_fence_before();
          }
        }
        // P = 2^(S' - ref), summed in fp32 and rounded to fp16
        uint32_t ph[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float e0 = fast_exp2(__uint_as_float(pr[2 * i])), e1 = fast_exp2(__uint_as_float(pr[2 * i + 1]));
          l_acc[2 * i] += e0;
          l_acc[2 * i + 1] += e1;
          ph[i] = f32x2_to_f16x2(e0, e1);
        }
        if (j > 0) wait(&sh.o, (uint32_t)(j - 1));  // the last product has read P
        {
          // row my_row of P: 64 heads, this thread's 32 of them
#pragma unroll
          for (int i = 0; i < 4; ++i)
            *reinterpret_cast<uint4*>(sP + tc::sw128_offset((uint32_t)my_row, (uint32_t)(4 * half + i))) =
                make_uint4(ph[4 * i], ph[4 * i + 1], ph[4 * i + 2], ph[4 * i + 3]);
        }
        tc::fence_proxy_async_smem();
        arrive(&sh.p);
        first = false;

        const bool last_of_token = info.left == 0;
        if (last_of_token || j + 1 == n_run) {
          // ---- the token's (or the run's) end: l over the rows, O^T out ----
#pragma unroll
          for (int u = 0; u < 32; u += 16) {
            float v[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              v[i] = l_acc[u + i];
              l_acc[u + i] = 0.0f;
            }
            const float lsum = warp_transpose_reduce16<false>(v, lane);
            if (lane < 16) sh.red[quad][h0 + u + lane] = lsum;
          }
          meet(tokens - 1);
          const bool complete = whole && last_of_token;
          const int64_t token = info.token;
          if (tid < kHeads && !sh.abort) {
            const float l = sh.red[0][tid] + sh.red[1][tid] + sh.red[2][tid] + sh.red[3][tid];
            sh.up[tid] = !complete ? 1.0f : l > 0.0f ? 1.0f / l : 0.0f;
            if (!complete) a.part_ml[(int64_t)slot * kHeads + tid] = make_float2(sh.ref[tid], l);
            else if (a.lse)
              a.lse[token * kHeads + tid] = l > 0.0f ? (sh.ref[tid] + log2f(l)) * 0.6931471805599453f : -INFINITY;
            sh.ref[tid] = 0.0f;
          }
          meet(tokens);
          // the next token's queries have come meanwhile; its O^T only after them
          if (j + 1 < n_run) convert_q(tokens++);
          wait(&sh.o, (uint32_t)j);  // O^T of this tile is complete
          tc::tc_fence_after();
          const bool lost = sh.abort != 0;
#pragma unroll 2
          for (int x = 0; x < 8 && !lost; ++x) {  // channel block 2 half + x / 4, heads 16 (x % 4) ..
            const int mb = 2 * half + (x >> 2), hh = (x & 3) * 16;
            const int c = 128 * mb + my_row;
            uint32_t ov[16];
            tc::tmem_ld_32x32b_x16(tmem + lanes + kColO + 64u * (uint32_t)mb + (uint32_t)hh, ov);
            tc::tmem_ld_wait();
            if (!complete) {
              float* po = a.part_o + (int64_t)slot * kPartFloats + hh * kHeadDim + c;
#pragma unroll
              for (int i = 0; i < 16; ++i) po[i * kHeadDim] = __uint_as_float(ov[i]);
            } else {
              const int64_t o = token * kPartFloats + hh * kHeadDim + c;
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                const float v = __uint_as_float(ov[i]) * sh.up[hh + i];
                if (a.out_f32) a.out_f32[o + i * kHeadDim] = v;
                a.out[o + i * kHeadDim] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
              }
            }
          }
          // every block of O^T is read before the next token's products replace it
          tc::tc_fence_before();
          if (tid == 0 && whole && !last_of_token && !lost) {
            // the token's first part: its other parts lie with the next CTAs
            const int64_t all = sh.units, last = sh.end_unit - 1 + info.left;  // the unit of the token's last tile
            PartList pl;
            pl.token = (int32_t)token;
            pl.first_slot = slot;
            pl.cta0 = (int32_t)blockIdx.x;
            pl.cta1 = (int32_t)(((last + 1) * (int32_t)gridDim.x + all - 1) / all - 1);
            pl.units = all;
            a.lists[blockIdx.x] = pl;
          }
          first = true;
          open = true;
          whole = true;
          slot = 2 * cta + 1;
          if (j + 1 < n_run) meet(tokens);  // mul, ref, up, red
        }
        info_done(j);
      }
    }
  }
  tc::tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc::tc_fence_after();
    tc::tmem_dealloc(tmem, kTmemCols);
    if (lane == 0 && sh.abort) record_error(&g_paged_attn_error, CSA2_ERR_TIMEOUT);
  }
}

// ---- the tokens whose tiles lie with several CTAs ---------------------------------
// One block per (token, head) at a time: out = sum_j 2^(ref_j - M) O_j / sum_j
// 2^(ref_j - M) l_j over the parts in list order, even and odd parts summed
// apart. Warp w takes channels 128 (w % 4) .. and the parts of parity w / 4, and
// works out the weights for itself, so that a block only meets for its two sums:
// a split token has two parts more often than many, and there may be one per SM
// (64 heads of each), so the chain of dependent reads of an item is what counts.
// (Blocks of 512 threads, two per SM, with the weights in shared memory took 70
// us after 2,048 tokens of one prompt; all of these calls are 4 to 12 % faster.)
constexpr int kJoinThreads = 256;
constexpr int kJoinBlocks = 8;  // per SM

__global__ void __launch_bounds__(kJoinThreads) paged_attn_join_kernel(Args a, int32_t G) {
  __shared__ int32_t s_list[1024];
  __shared__ int32_t s_n;
  __shared__ __align__(16) float4 s_sum[128];
  pdl_begin();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // the tokens to join, in order (G <= 1024)
  if (warp == 0) {
    int n = 0;
#pragma unroll 5
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
  const int parity = warp >> 2, c4 = (warp & 3) * 32 + lane;
  for (int it = blockIdx.x; it < items; it += gridDim.x) {
    const PartList pl = a.lists[s_list[it / kHeads]];
    const int h = it % kHeads;
    // Part j lies with the j-th CTA that has tiles: with fewer units than CTAs
    // the one that holds unit first + j, else simply the next.
    const bool sparse = pl.units < G;
    const int64_t first = sparse ? pl.units * pl.cta0 / G : 0;
    const int n = sparse ? (int)(pl.units * pl.cta1 / G - first) + 1 : pl.cta1 - pl.cta0 + 1;
    float M = -INFINITY, L = 0.0f;  // L: this lane's share
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int j0 = 0; j0 < n; j0 += 32) {
      const int j = j0 + lane;
      int slot = 0;
      float2 ml = make_float2(-INFINITY, 0.0f);
      if (j < n) {
        const int c = sparse ? (int)(((first + j + 1) * G + pl.units - 1) / pl.units) - 1 : pl.cta0 + j;
        slot = j == 0 ? pl.first_slot : 2 * c;
        ml = a.part_ml[(int64_t)slot * kHeads + h];
      }
      // (a part that saw nothing has l = 0, weight 0 and zeros)
      float top = ml.y > 0.0f ? fmaxf(M, ml.x) : M;
#pragma unroll
      for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      const float shrink = M > -INFINITY ? fast_exp2(M - top) : 0.0f;
      const float w = ml.y > 0.0f ? fast_exp2(ml.x - top) : 0.0f;
      M = top;
      L = L * shrink + w * ml.y;
      acc.x *= shrink;
      acc.y *= shrink;
      acc.z *= shrink;
      acc.w *= shrink;
      const int here = min(32, n - j0);
#pragma unroll 8
      for (int i = parity; i < here; i += 2) {
        const int64_t at = __shfl_sync(0xffffffffu, slot, i);
        const float wi = __shfl_sync(0xffffffffu, w, i);
        const float4 v = reinterpret_cast<const float4*>(a.part_o + at * kPartFloats + (int64_t)h * kHeadDim)[c4];
        acc.x = fmaf(v.x, wi, acc.x);
        acc.y = fmaf(v.y, wi, acc.y);
        acc.z = fmaf(v.z, wi, acc.z);
        acc.w = fmaf(v.w, wi, acc.w);
      }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
    if (parity) s_sum[c4] = acc;
    __syncthreads();
    if (!parity) {
      const float inv = L > 0.0f ? 1.0f / L : 0.0f;
      const float4 v = s_sum[c4];
      acc.x = (acc.x + v.x) * inv;
      acc.y = (acc.y + v.y) * inv;
      acc.z = (acc.z + v.z) * inv;
      acc.w = (acc.w + v.w) * inv;
      const int64_t o = ((int64_t)pl.token * kHeads + h) * kHeadDim + c4 * 4;
      if (a.out_f32) *reinterpret_cast<float4*>(a.out_f32 + o) = acc;
      const __nv_bfloat162 b0 = __floats2bfloat162_rn(acc.x, acc.y);
      const __nv_bfloat162 b1 = __floats2bfloat162_rn(acc.z, acc.w);
      *reinterpret_cast<uint2*>(a.out + o) =
          make_uint2(*reinterpret_cast<const uint32_t*>(&b0), *reinterpret_cast<const uint32_t*>(&b1));
      if (a.lse && c4 == 0)
        a.lse[(int64_t)pl.token * kHeads + h] = L > 0.0f ? (M + log2f(L)) * 0.6931471805599453f : -INFINITY;
    }
    __syncthreads();  // the sums are done with
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

static PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  if (!fn) {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
  }
  return fn;
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
  if (n_tokens > 0 && B != 0 && (!q_bf16 || !paged_planes(n_pages, kv_data, kv_scale) || !n_visible || !out_bf16))
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
  // a CTA counts its tiles' four groups in 32 bits (and has no more tiles than units)
  if ((int64_t)n_tokens * ((a.pages.capacity() + pattn::kRows) / pattn::kRows + pattn::kTokenUnits) / G >= 0x3FFFFFFELL)
    return CSA2_ERR_UNSUPPORTED_SHAPE;
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
  auto encode = tensor_map_encoder();
  if (!encode) return CSA2_ERR_CUDA;
  // the pool's codes, in boxes of one group's 64 bytes of a run of rows (an empty
  // pool has nothing to copy: the map then only has to be valid, over any memory)
  const int64_t pool = n_pages << a.pages.shift;
  CUtensorMap rows_map;
  cuuint64_t dims[2] = {(cuuint64_t)kKvBytes, (cuuint64_t)(pool > 0 ? pool : 1)};
  cuuint64_t strides[1] = {(cuuint64_t)kKvBytes};
  cuuint32_t box[2] = {64, (cuuint32_t)(page_size < pattn::kRows ? page_size : pattn::kRows)};
  cuuint32_t estr[2] = {1, 1};
  void* plane = (void*)(pool > 0 ? (const void*)kv_data : q_bf16);
  if (encode(&rows_map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, plane, dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return CSA2_ERR_CUDA;
  // the queries, in boxes of a token's 64 heads by 64 channels
  CUtensorMap q_map;
  cuuint64_t q_dims[3] = {(cuuint64_t)kHeadDim, (cuuint64_t)kHeads, (cuuint64_t)n_tokens};
  cuuint64_t q_strides[2] = {(cuuint64_t)kHeadDim * 2, (cuuint64_t)kHeadDim * kHeads * 2};
  cuuint32_t q_box[3] = {64, (cuuint32_t)kHeads, 1};
  cuuint32_t q_estr[3] = {1, 1, 1};
  if (encode(&q_map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, (void*)q_bf16, q_dims, q_strides, q_box, q_estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return CSA2_ERR_CUDA;
  static Csa2PerDeviceOnce optin;
  if (csa2_smem_optin((const void*)pattn::paged_attn_kernel, pattn::kSmemBytes, optin) != CSA2_OK) return CSA2_ERR_CUDA;
  cudaStream_t s = (cudaStream_t)stream;
  CSA2_LAUNCH_PDL(pattn::paged_attn_kernel, dim3((unsigned)G), dim3(pattn::kThreads), (size_t)pattn::kSmemBytes, s,
                  rows_map, q_map, a);
  CSA2_LAUNCH_PDL(pattn::paged_attn_join_kernel, dim3((unsigned)(pattn::kJoinBlocks * G)), dim3(pattn::kJoinThreads),
                  (size_t)0, s, a, (int32_t)G);
  return CSA2_OK;
}
