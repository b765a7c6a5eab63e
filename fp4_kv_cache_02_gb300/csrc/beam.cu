// beam.cu -- beam search around the paged cache: the selection over beams and
// vocabulary, and the states that follow it (page tables, partly filled pages,
// rows of any other state such as the sliding windows of "DeepSeek-V4.1-Flash:
// Pushing the Limits of KV Cache Compression", section 2.3).
//
// Candidate (w, v) of a sequence scores  score[w] + x[w][v] - lse(x[w]),  lse the
// log of the sum of exp over the vocabulary; the k largest are wanted, ties to the
// lowest w * V + v.
#include "paged_common.cuh"

namespace csa2 {

__device__ int g_beam_error = 0;

namespace beam {

constexpr int kThreads = 256;
constexpr int kMaxK = CSA2_MAX_BEAM_K;
constexpr int kMaxLists = 512;              // lists of a sequence that the joining kernel takes: one a thread
constexpr int kVectors = 4;                 // 16-byte loads of a thread in a tile
constexpr int kKeep = 512;                  // candidates held before they are cut down to about k
constexpr float kLog2e = 1.4426950408889634f;

// Values by size, equal ones by place, the lower first: larger is better, all
// different, 0 for none.
__device__ __forceinline__ uint64_t make_key(float x, uint32_t place) {
  return (uint64_t)score_key(x) << 32 | (uint32_t)~place;
}
__device__ __forceinline__ float key_value(uint64_t key) {
  const uint32_t b = (uint32_t)(key >> 32);
  return __uint_as_float((b & 0x80000000u) ? b & 0x7FFFFFFFu : ~b);
}
__device__ __forceinline__ uint32_t key_place(uint64_t key) { return ~(uint32_t)key; }

// The k-th largest of the block's keys, one a thread (0: none); 1 when there are
// fewer than k. Each thread counts the keys above its own.
__device__ __forceinline__ uint64_t kth_of_block(uint64_t key, int k, uint64_t* s_keys, uint64_t* s_kth) {
  __syncthreads();
  s_keys[threadIdx.x] = key;
  if (threadIdx.x == 0) *s_kth = 1;
  __syncthreads();
  int above = 0;
#pragma unroll 8
  for (int i = 0; i < kThreads; i += 2) {
    const ulonglong2 two = *reinterpret_cast<const ulonglong2*>(s_keys + i);
    above += (two.x > key) + (two.y > key);
  }
  if (key != 0 && above == k - 1) *s_kth = key;
  __syncthreads();
  return *s_kth;
}

template <typename T>
struct Vec;
template <>
struct Vec<float> {
  static constexpr int n = 4;
  static __device__ __forceinline__ void load(const float* p, float* x) {
    const float4 v = __ldcs(reinterpret_cast<const float4*>(p));
    x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
  }
  static __device__ __forceinline__ float one(const float* p) { return *p; }
};
template <>
struct Vec<uint16_t> {
  static constexpr int n = 8;
  static __device__ __forceinline__ void load(const uint16_t* p, float* x) {
    const uint4 v = __ldcs(reinterpret_cast<const uint4*>(p));
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
  static __device__ __forceinline__ float one(const uint16_t* p) { return bf16_bits_to_f32(*p); }
};

struct Part {     // of a row's softmax: sum of 2^(x log2e - ref)
  float ref, sum;
};

template <typename T>
struct RowArgs {
  const T* logits;
  int64_t ld;
  int32_t V, k, parts;
  Part* part;       // [rows][parts]
  uint64_t* lists;  // [rows][parts][k], falling, 0 behind the last
};

// One CTA reads a part of a row once: the softmax's running reference and sum, and
// the part's k largest. A tile of the part is in registers at a time. The k-th
// largest of the threads' own largest values bounds the k-th largest from below;
// what reaches the bound goes to a list in shared memory, which is cut down by the
// same rule when it is long. With random logits some 1.1 k values of the first tile
// and fewer of each later one reach it. A list that would overflow (rising logits) is
// taken back to the tile's start and the bound is raised by the tile's own values:
// then at most k threads' values pass.
template <typename T>
__global__ void __launch_bounds__(kThreads) rows_kernel(RowArgs<T> a) {
  constexpr int kN = Vec<T>::n, kX = kVectors * kN;
  constexpr int kRoom = kX == 32 ? 3072 : 2048;
  // what a cut leaves (k threads' entries), a tile's values over its own bound (k
  // threads' values) and the row's ends fit together
  static_assert(kMaxK * (kRoom / kThreads) + kMaxK * kX + 2 * kN <= kRoom && kRoom % kThreads == 0, "list too short");
  static_assert(kKeep + kMaxK * kX + 2 * kN <= kRoom, "list too short");
  __shared__ uint64_t s_list[kRoom];
  __shared__ __align__(16) uint64_t s_keys[kThreads];
  __shared__ uint64_t s_kth;
  __shared__ int s_n;
  __shared__ Part s_part[kThreads / 32];
  pdl_begin();
  const int32_t row = blockIdx.x / a.parts, part = blockIdx.x % a.parts;
  const T* x0 = a.logits + (int64_t)row * a.ld;
  // the row from its first 16-byte boundary on, in vectors; what lies before and
  // behind them goes to one thread of the first and last part
  const int32_t lead = min(a.V, (int32_t)(((16 - (reinterpret_cast<uintptr_t>(x0) & 15)) & 15) / sizeof(T)));
  const int32_t vectors = (a.V - lead) / kN;
  const int32_t per = (vectors + a.parts - 1) / a.parts;
  const int32_t v_begin = min(vectors, part * per), v_end = min(vectors, v_begin + per);
  const int k = a.k;

  float ref = -INFINITY, sum = 0.0f;
  uint64_t bound = 1;
  float bound_value = -INFINITY;
  int n = 0;  // entries of the list, as every thread knows it
  if (threadIdx.x == 0) s_n = 0;
  __syncthreads();

  const auto cut = [&]() {  // the list down to what reaches its own bound
    uint64_t mine[kRoom / kThreads];
    uint64_t best = 0;
#pragma unroll
    for (int i = 0; i < kRoom / kThreads; ++i) {
      const int at = i * kThreads + threadIdx.x;
      mine[i] = at < n ? s_list[at] : 0;
      best = max(best, mine[i]);
    }
    bound = max(bound, kth_of_block(best, k, s_keys, &s_kth));
    if (threadIdx.x == 0) s_n = 0;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kRoom / kThreads; ++i)
      if (mine[i] >= bound) s_list[atomicAdd(&s_n, 1)] = mine[i];
    __syncthreads();
    n = s_n;
    bound_value = bound > 1 ? key_value(bound) : -INFINITY;
  };

  // Tiles of the vectors; the first also holds the row's ends, as a last vector of
  // thread 0 (before) and 1 (behind).
  bool first = true;
  for (int32_t v0 = v_begin; first || v0 < v_end; v0 += kThreads * kVectors) {
    float x[kX];
#pragma unroll
    for (int j = 0; j < kVectors; ++j) {
      const int32_t v = v0 + j * kThreads + (int32_t)threadIdx.x;
      if (v < v_end) {
        Vec<T>::load(x0 + lead + (int64_t)v * kN, x + j * kN);
      } else {
#pragma unroll
        for (int i = 0; i < kN; ++i) x[j * kN + i] = -INFINITY;
      }
    }
    const auto place_of = [&](int i) {
      return (uint32_t)(lead + (v0 + (i / kN) * kThreads + (int32_t)threadIdx.x) * kN + i % kN);
    };
    float top = x[0];
#pragma unroll
    for (int i = 1; i < kX; ++i) top = fmaxf(top, x[i]);
    if (top > ref) {
      if (ref > -INFINITY) sum *= exp2f((ref - top) * kLog2e);
      ref = top;
    }
    // (x - ref first: exact where it counts, and 0 for a row of the type's lowest
    // value, whose product with log2 e is infinite; with ref +inf the sum is NaN)
    const float from = ref > -INFINITY ? ref : 0.0f;
    float add[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < kX; ++i) {
      float e;
      asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"((x[i] - from) * kLog2e));
      add[i % 4] += e;
    }
    sum += (add[0] + add[1]) + (add[2] + add[3]);

    const auto push = [&]() {
      if (!(top >= bound_value)) return;
#pragma unroll
      for (int i = 0; i < kX; ++i) {
        if (x[i] >= bound_value && x[i] > -INFINITY) {
          const uint64_t key = make_key(x[i], place_of(i));
          if (key >= bound) {
            const int at = atomicAdd(&s_n, 1);
            if (at < kRoom) s_list[at] = key;
          }
        }
      }
    };
    if (!first) push();
    __syncthreads();
    const int reached = s_n;
    if (first || reached > kRoom) {
      uint64_t best = 0;
#pragma unroll
      for (int i = kX - 1; i >= 0; --i)
        if (x[i] > -INFINITY) best = max(best, make_key(x[i], place_of(i)));
      bound = max(bound, kth_of_block(best, k, s_keys, &s_kth));
      bound_value = bound > 1 ? key_value(bound) : -INFINITY;
      if (threadIdx.x == 0) s_n = n;
      __syncthreads();
      push();
      __syncthreads();
    }
    n = s_n;
    if (n > kKeep) cut();
    __syncthreads();  // everyone knows the count before the next tile adds to it
    first = false;
  }

  // the row's ends: fewer than 2 kN values, one to a thread
  {
    const int32_t behind = lead + vectors * kN;
    int32_t at = -1;
    if (part == 0 && (int32_t)threadIdx.x < lead) at = (int32_t)threadIdx.x;
    if (part == a.parts - 1 && threadIdx.x >= 32 && behind + (int32_t)threadIdx.x - 32 < a.V)
      at = behind + (int32_t)threadIdx.x - 32;
    const float v = at >= 0 ? Vec<T>::one(x0 + at) : -INFINITY;
    if (at >= 0 && !(v == -INFINITY)) {
      if (v > ref) {
        if (ref > -INFINITY) sum *= exp2f((ref - v) * kLog2e);
        ref = v;
      }
      sum += exp2f((v - (ref > -INFINITY ? ref : 0.0f)) * kLog2e);
      const uint64_t key = make_key(v, (uint32_t)at);
      if (key >= bound) s_list[atomicAdd(&s_n, 1)] = key;
    }
    __syncthreads();
    n = s_n;
  }
  if (n > kThreads) cut();

  // the k largest, each to its rank
  uint64_t* list = a.lists + (int64_t)blockIdx.x * k;
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const uint64_t key = s_list[i];
    int above = 0;
    for (int j = 0; j < n; ++j) above += s_list[j] > key;
    if (above < k) list[above] = key;
  }
  for (int i = n + threadIdx.x; i < k; i += kThreads) list[i] = 0;

  // the threads' sums
  float top = ref;
#pragma unroll
  for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  sum = ref == -INFINITY ? sum : sum * exp2f((ref - top) * kLog2e);
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if ((threadIdx.x & 31) == 0) s_part[threadIdx.x >> 5] = {top, sum};
  __syncthreads();
  if (threadIdx.x == 0) {
    float all = s_part[0].ref;
    for (int i = 1; i < kThreads / 32; ++i) all = fmaxf(all, s_part[i].ref);
    float s = 0.0f;
    for (int i = 0; i < kThreads / 32; ++i)
      s += s_part[i].ref == -INFINITY ? s_part[i].sum : s_part[i].sum * exp2f((s_part[i].ref - all) * kLog2e);
    a.part[blockIdx.x] = {all, s};
  }
}

// ---- joining ---------------------------------------------------------------------

struct JoinArgs {
  int32_t W, V, k, parts;
  const Part* part;
  const uint64_t* lists;
  const float* scores;
  float* out_scores;
  int32_t *out_parents, *out_tokens;
  float* lse;
};

struct Best {
  uint64_t score;  // order-preserving bits of the double
  uint64_t place;  // ~(w * V + v)
};
__device__ __forceinline__ bool above(const Best& a, const Best& b) {
  return a.score > b.score || (a.score == b.score && a.place > b.place);
}
__device__ __forceinline__ uint64_t order(double v) {
  const uint64_t b = (uint64_t)__double_as_longlong(v);
  return b >> 63 ? ~b : b | 0x8000000000000000ull;
}
__device__ __forceinline__ double order_value(uint64_t b) {
  return __longlong_as_double((long long)(b >> 63 ? b & 0x7FFFFFFFFFFFFFFFull : ~b));
}

// One CTA to a sequence, a thread to a list. The rows' sums give lse; scores are
// held in 64 bits, so that their order is that of the formula to about 2^-23 (what the
// sums carry): in 32 bits x - lse would be rounded to 2^-20 for logits about 16. The
// k-th largest head of the lists bounds the k-th largest from below; what reaches it
// (at most k lists' entries) is ranked.
__global__ void __launch_bounds__(kMaxLists) join_kernel(JoinArgs a) {
  pdl_wait();
  extern __shared__ Best s_best[];  // [k * k] behind the heads
  __shared__ Best s_head[kMaxLists];
  __shared__ double s_lse[CSA2_MAX_BEAMS];  // NaN: the row takes no part
  __shared__ Best s_kth;
  __shared__ int s_n;
  const int b = blockIdx.x, tid = threadIdx.x;
  const int lists = a.W * a.parts;
  const int64_t row0 = (int64_t)b * a.W;
  if (tid == 0) {
    s_kth = {0, 0};
    s_n = 0;
  }
  for (int w = tid; w < a.W; w += blockDim.x) {
    const Part* p = a.part + (row0 + w) * a.parts;
    float ref = -INFINITY;
    for (int c = 0; c < a.parts; ++c) ref = fmaxf(ref, p[c].ref);
    float sum = 0.0f;
    for (int c = 0; c < a.parts; ++c)
      sum += p[c].ref == -INFINITY ? p[c].sum : p[c].sum * exp2f((p[c].ref - ref) * kLog2e);
    double lse = -INFINITY;
    if (!(sum <= 3.0e38f) || !(ref < INFINITY)) {
      record_error(&g_beam_error, CSA2_ERR_DEVICE);  // a NaN or +inf among the logits
      lse = NAN;
    } else if (sum > 0.0f) {
      lse = (double)ref + log((double)sum);
    }
    if (a.lse) a.lse[row0 + w] = (float)lse;
    const float s = a.scores ? a.scores[row0 + w] : 0.0f;
    s_lse[w] = fabsf(s) < INFINITY && sum > 0.0f ? lse : (double)NAN;
  }
  __syncthreads();
  const uint64_t* list = a.lists + (row0 * a.parts + tid) * a.k;
  const int w = tid < lists ? tid / a.parts : 0;
  const double lse = s_lse[w], score = a.scores ? (double)a.scores[row0 + w] : 0.0;
  const auto best_of = [&](uint64_t key) -> Best {
    if (key == 0 || isnan(lse)) return {0, 0};
    // (in this order: the lowest value of fp32 less itself leaves the score)
    return {order(score + ((double)key_value(key) - lse)), ~((uint64_t)w * (uint64_t)a.V + key_place(key))};
  };
  Best head{0, 0};
  if (tid < lists) head = best_of(list[0]);
  s_head[tid] = head;
  __syncthreads();
  if (head.place) {
    int n = 0;
    for (int i = 0; i < lists; ++i) n += above(s_head[i], head);
    if (n == a.k - 1) s_kth = head;
  }
  __syncthreads();
  const Best kth = s_kth;
  if (head.place && !above(kth, head)) {
    for (int i = 0; i < a.k; ++i) {
      const Best c = i == 0 ? head : best_of(list[i]);
      if (!c.place || above(kth, c)) break;
      s_best[atomicAdd(&s_n, 1)] = c;
    }
  }
  __syncthreads();
  const int n = s_n;
  for (int i = tid; i < n; i += blockDim.x) {
    const Best c = s_best[i];
    int r = 0;
    for (int j = 0; j < n; ++j) r += above(s_best[j], c);
    if (r < a.k) {
      const uint64_t at = ~c.place;
      const int64_t o = (int64_t)b * a.k + r;
      a.out_scores[o] = (float)order_value(c.score);
      a.out_parents[o] = (int32_t)(row0 + (int64_t)(at / (uint64_t)a.V));
      a.out_tokens[o] = (int32_t)(at % (uint64_t)a.V);
    }
  }
  for (int i = n + tid; i < a.k; i += blockDim.x) {
    const int64_t o = (int64_t)b * a.k + i;
    a.out_scores[o] = -INFINITY;
    a.out_parents[o] = -1;
    a.out_tokens[o] = -1;
  }
}

// ---- states ----------------------------------------------------------------------

struct ReorderArgs {
  const int32_t *parents, *fresh;
  int32_t R, rows_in, layers;
  uint8_t* planes[4];
  PageTable pages;
  const int32_t* n_visible;
  int32_t *table_out, *n_out;
};

constexpr int kReorderThreads = 256;

// Bytes of an entry in each plane.
__device__ __constant__ const int kPlaneBytes[4] = {kKvBytes, kKvScales, kIkBytes, kIkScales};

// Block (r, 0) writes row r's places of the table and its count, block (r, 1 + i)
// copies what row r needs of layer i: the entries of its last, partly filled page,
// if a lower row has the same parent. Every block finds that out for itself from
// the parents; nothing that is read is written.
__global__ void __launch_bounds__(kReorderThreads) reorder_kernel(ReorderArgs a) {
  const int32_t r = blockIdx.x;
  const int32_t p = a.parents[r];
  if (p < 0 || p >= a.rows_in) {
    if (blockIdx.y == 0 && threadIdx.x == 0) {
      if (p == -1)
        a.n_out[r] = 0;
      else
        record_error(&g_beam_error, CSA2_ERR_DEVICE);
    }
    return;
  }
  const int32_t n = a.n_visible[p];
  if (n < 0 || n > a.pages.capacity()) {
    if (blockIdx.y == 0 && threadIdx.x == 0) record_error(&g_beam_error, CSA2_ERR_DEVICE);
    return;
  }
  const int32_t page = a.pages.page_size();
  const int32_t full = n >> a.pages.shift, fill = n & (page - 1);
  const int32_t* from = a.pages.table + (int64_t)p * a.pages.max_pages;
  int again = 0;
  if (fill)
    for (int32_t i = threadIdx.x; i < r; i += kReorderThreads) again |= a.parents[i] == p;
  again = __syncthreads_or(again);
  if (blockIdx.y == 0) {
    int32_t* to = a.table_out + (int64_t)r * a.pages.max_pages;
    for (int32_t i = threadIdx.x; i < full; i += kReorderThreads) to[i] = from[i];
    if (threadIdx.x == 0) {
      a.n_out[r] = n;
      if (fill) {
        int32_t last = from[full];
        if (again) {
          const int32_t own = a.fresh[r];
          const bool ok = own >= 0 && own < a.pages.n_pages && last >= 0 && last < a.pages.n_pages;
          if (!ok) record_error(&g_beam_error, CSA2_ERR_DEVICE);
          last = ok ? own : -1;
        }
        to[full] = last;
      }
    }
    return;
  }
  if (!again) return;
  const int32_t src = from[full], dst = a.fresh[r];
  if (src < 0 || src >= a.pages.n_pages || dst < 0 || dst >= a.pages.n_pages) return;  // reported above
  const int64_t layer = (int64_t)(blockIdx.y - 1) * a.pages.n_pages;
  for (int i = 0; i < 4; ++i) {
    if (!a.planes[i]) continue;
    const int64_t width = (int64_t)kPlaneBytes[i] << a.pages.shift;
    const uint8_t* s = a.planes[i] + (layer + src) * width;
    uint8_t* d = a.planes[i] + (layer + dst) * width;
    const int bytes = fill * kPlaneBytes[i];
    for (int at = threadIdx.x * 16; at + 16 <= bytes; at += kReorderThreads * 16)
      *reinterpret_cast<uint4*>(d + at) = *reinterpret_cast<const uint4*>(s + at);
    const int tail = bytes & ~15;
    const int at = tail + (int)threadIdx.x * 4;
    if (at < bytes) *reinterpret_cast<uint32_t*>(d + at) = *reinterpret_cast<const uint32_t*>(s + at);
  }
}

constexpr int kRowSlice = kReorderThreads * 16 * 4;  // bytes of a row to a block

__global__ void __launch_bounds__(kReorderThreads)
    rows_copy_kernel(const uint8_t* __restrict__ src, int64_t rows_in, int64_t row_bytes, int64_t slices,
                     const int32_t* __restrict__ parents, uint8_t* __restrict__ dst) {
  const int64_t r = blockIdx.x / slices, slice = blockIdx.x % slices;
  const int32_t p = parents[r];
  if (p < 0 || p >= rows_in) {
    if (p != -1 && slice == 0 && threadIdx.x == 0) record_error(&g_beam_error, CSA2_ERR_DEVICE);
    return;
  }
  const uint8_t* s = src + (int64_t)p * row_bytes;
  uint8_t* d = dst + r * row_bytes;
  uint4 v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t at = slice * kRowSlice + (i * kReorderThreads + (int64_t)threadIdx.x) * 16;
    if (at < row_bytes) v[i] = __ldcs(reinterpret_cast<const uint4*>(s + at));
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t at = slice * kRowSlice + (i * kReorderThreads + (int64_t)threadIdx.x) * 16;
    if (at < row_bytes) __stcs(reinterpret_cast<uint4*>(d + at), v[i]);
  }
}

}  // namespace beam
}  // namespace csa2

using namespace csa2;

int csa2_read_and_clear_beam_error(cudaStream_t s) {
  int v = 0, z = 0;
  if (cudaMemcpyFromSymbolAsync(&v, g_beam_error, sizeof(int), 0, cudaMemcpyDeviceToHost, s) != cudaSuccess)
    return CSA2_ERR_CUDA;
  if (cudaMemcpyToSymbolAsync(g_beam_error, &z, sizeof(int), 0, cudaMemcpyHostToDevice, s) != cudaSuccess)
    return CSA2_ERR_CUDA;
  if (cudaStreamSynchronize(s) != cudaSuccess) return CSA2_ERR_CUDA;
  return v;
}

static size_t al256(size_t x) { return (x + 255) / 256 * 256; }

static int check_beam(int32_t B, int32_t W, int32_t V, int32_t k) {
  if (B < 0 || W < 0 || V < 0 || k < 0) return CSA2_ERR_INVALID_ARG;
  if (W > CSA2_MAX_BEAMS || k > CSA2_MAX_BEAM_K || k == 0 || (int64_t)B * W > 0x7FFFFFLL) return CSA2_ERR_UNSUPPORTED_SHAPE;
  return CSA2_OK;
}

// Parts of a row: about 4 CTAs an SM in all (152 SMs: the size of a workspace does
// not depend on the device), parts of 2,048 values at least.
static int beam_parts(int32_t B, int32_t W, int32_t V) {
  const int64_t rows = (int64_t)B * W;
  int64_t parts = (608 + rows - 1) / rows;
  const int64_t most = V / 2048;
  if (parts > most) parts = most;
  if (parts > beam::kMaxLists / W) parts = beam::kMaxLists / W;
  return parts < 1 ? 1 : (int)parts;
}

extern "C" size_t csa2_beam_select_workspace_size(int32_t B, int32_t W, int32_t V, int32_t k) {
  if (check_beam(B, W, V, k) != CSA2_OK || B == 0 || W == 0) return 0;
  const size_t lists = (size_t)B * W * beam_parts(B, W, V);
  return al256(lists * sizeof(beam::Part)) + al256(lists * k * sizeof(uint64_t));
}

template <typename T>
static int launch_rows(const void* logits, int64_t ld, int32_t V, int32_t k, int64_t rows, int parts, beam::Part* part,
                       uint64_t* lists, cudaStream_t stream) {
  beam::RowArgs<T> a{(const T*)logits, ld, V, k, parts, part, lists};
  CSA2_LAUNCH_PDL(beam::rows_kernel<T>, dim3((unsigned)(rows * parts)), dim3(beam::kThreads), (size_t)0, stream, a);
  return CSA2_OK;
}

extern "C" int csa2_beam_select(const void* logits, int32_t logits_f32, int32_t B, int32_t W, int32_t V, int64_t ld,
                                const float* scores, int32_t k, float* out_scores, int32_t* out_parents,
                                int32_t* out_tokens, float* lse, void* workspace, size_t workspace_bytes,
                                csa2_stream_t stream) {
  int rc = check_beam(B, W, V, k);
  if (rc) return rc;
  if (ld < V || (logits_f32 != 0 && logits_f32 != 1)) return CSA2_ERR_INVALID_ARG;
  if (B == 0) return CSA2_OK;
  if (W == 0 || V == 0) return CSA2_ERR_INVALID_ARG;
  if (!logits || !out_scores || !out_parents || !out_tokens) return CSA2_ERR_INVALID_ARG;
  if (!csa2_aligned(logits, logits_f32 ? 4 : 2) || !csa2_aligned(scores, 4) || !csa2_aligned(out_scores, 4) ||
      !csa2_aligned(out_parents, 4) || !csa2_aligned(out_tokens, 4) || !csa2_aligned(lse, 4))
    return CSA2_ERR_ALIGNMENT;
  if (!workspace || workspace_bytes < csa2_beam_select_workspace_size(B, W, V, k) || !csa2_aligned(workspace, 256))
    return CSA2_ERR_WORKSPACE;
  const int parts = beam_parts(B, W, V);
  const int64_t rows = (int64_t)B * W;
  beam::Part* part = (beam::Part*)workspace;
  uint64_t* lists = (uint64_t*)((char*)workspace + al256((size_t)rows * parts * sizeof(beam::Part)));
  cudaStream_t s = (cudaStream_t)stream;
  rc = logits_f32 ? launch_rows<float>(logits, ld, V, k, rows, parts, part, lists, s)
                  : launch_rows<uint16_t>(logits, ld, V, k, rows, parts, part, lists, s);
  if (rc) return rc;
  static Csa2PerDeviceOnce once;
  if (csa2_smem_optin((const void*)beam::join_kernel, beam::kMaxK * beam::kMaxK * (int)sizeof(beam::Best), once) != CSA2_OK)
    return CSA2_ERR_CUDA;
  beam::JoinArgs j{W, V, k, parts, part, lists, scores, out_scores, out_parents, out_tokens, lse};
  CSA2_LAUNCH_PDL(beam::join_kernel, dim3((unsigned)B), dim3(beam::kMaxLists), (size_t)k * k * sizeof(beam::Best), s, j);
  return CSA2_OK;
}

extern "C" int csa2_paged_reorder(const int32_t* parents, const int32_t* fresh_pages, int32_t R, uint8_t* kv_data,
                                  uint8_t* kv_scale, uint8_t* ik_data, uint8_t* ik_scale, int32_t layers, int64_t n_pages,
                                  int32_t page_size, const int32_t* page_table, int32_t rows_in, int32_t max_pages,
                                  const int32_t* n_visible, int32_t* page_table_out, int32_t* n_visible_out,
                                  csa2_stream_t stream) {
  PageTable pages;
  int rc = paged_check(page_table, n_pages, page_size, max_pages, rows_in, pages);
  if (rc) return rc;
  if (R < 0 || layers < 0) return CSA2_ERR_INVALID_ARG;
  if (layers > 65534) return CSA2_ERR_UNSUPPORTED_SHAPE;
  if (!csa2_aligned(parents, 4) || !csa2_aligned(fresh_pages, 4) || !csa2_aligned(n_visible, 4) ||
      !csa2_aligned(page_table_out, 4) || !csa2_aligned(n_visible_out, 4) || !csa2_aligned(kv_data, 16) ||
      !csa2_aligned(kv_scale, 16) || !csa2_aligned(ik_data, 16) || !csa2_aligned(ik_scale, 16))
    return CSA2_ERR_ALIGNMENT;
  if (R == 0) return CSA2_OK;
  if (!parents || !fresh_pages || !n_visible_out || (rows_in != 0 && !n_visible) || (max_pages != 0 && !page_table_out))
    return CSA2_ERR_INVALID_ARG;
  // codes and scales come together
  if (n_pages != 0 && (!kv_data != !kv_scale || !ik_data != !ik_scale)) return CSA2_ERR_INVALID_ARG;
  // rows read places that others write: not in place
  if (page_table_out == page_table || n_visible_out == n_visible) return CSA2_ERR_INVALID_ARG;
  beam::ReorderArgs a{parents, fresh_pages, R, rows_in, layers, {kv_data, kv_scale, ik_data, ik_scale}, pages, n_visible,
                      page_table_out, n_visible_out};
  beam::reorder_kernel<<<dim3((unsigned)R, (unsigned)(1 + layers)), beam::kReorderThreads, 0, (cudaStream_t)stream>>>(a);
  CSA2_CHECK_LAUNCH();
  return CSA2_OK;
}

extern "C" int csa2_reorder_rows(const void* src, int64_t rows_in, int64_t row_bytes, const int32_t* parents, int32_t R,
                                 void* dst, csa2_stream_t stream) {
  if (rows_in < 0 || row_bytes < 0 || R < 0) return CSA2_ERR_INVALID_ARG;
  if (row_bytes % 16) return CSA2_ERR_UNSUPPORTED_SHAPE;
  if (!csa2_aligned(src, 16) || !csa2_aligned(dst, 16) || !csa2_aligned(parents, 4)) return CSA2_ERR_ALIGNMENT;
  if (R == 0 || row_bytes == 0) return CSA2_OK;
  if ((!src && rows_in != 0) || !parents || !dst || src == dst) return CSA2_ERR_INVALID_ARG;
  const int64_t slices = (row_bytes + beam::kRowSlice - 1) / beam::kRowSlice;
  if (slices > 0x7FFFFFFFLL / R) return CSA2_ERR_UNSUPPORTED_SHAPE;
  beam::rows_copy_kernel<<<(unsigned)(R * slices), beam::kReorderThreads, 0, (cudaStream_t)stream>>>(
      (const uint8_t*)src, rows_in, row_bytes, slices, parents, (uint8_t*)dst);
  CSA2_CHECK_LAUNCH();
  return CSA2_OK;
}
