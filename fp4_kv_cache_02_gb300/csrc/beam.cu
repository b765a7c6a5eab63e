// beam.cu -- beam search around the paged cache: the selection over beams and
// vocabulary, and the states that follow it (page tables, partly filled pages,
// rows of any other state such as the sliding windows of "DeepSeek-V4.1-Flash:
// Pushing the Limits of KV Cache Compression", section 2.3).
//
// Candidate (w, v) of a sequence scores  score[w] + x[w][v] - lse(x[w]),  lse the
// log of the sum of exp over the vocabulary; the k largest are wanted, ties to the
// lowest w * V + v.
#include <float.h>

#include "paged_common.cuh"

namespace csa2 {

__device__ int g_beam_error = 0;

namespace beam {

constexpr int kThreads = 256;
constexpr int kMaxK = CSA2_MAX_BEAM_K;
constexpr int kX = 16;                      // values of a thread in a tile
constexpr int kRoom = 2560;                 // candidates that fit
constexpr int kJoinThreads = 512;
constexpr float kLog2e = 1.4426950408889634f;

// Values by size, equal ones (zeros of either sign too) by place, the lower first:
// larger is better, all different, 0 for none.
__device__ __forceinline__ uint64_t make_key(float x, uint32_t place) {
  return (uint64_t)score_key(__fadd_rn(x, 0.0f)) << 32 | (uint32_t)~place;
}
__device__ __forceinline__ float key_value(uint64_t key) {
  const uint32_t b = (uint32_t)(key >> 32);
  return __uint_as_float((b & 0x80000000u) ? b & 0x7FFFFFFFu : ~b);
}
__device__ __forceinline__ uint32_t key_place(uint64_t key) { return ~(uint32_t)key; }

// A bound from below on the k-th largest of the block's values: the k-th largest of
// 64 (k <= 16) or 128 of them, each the largest of four or two threads' (0: none); 1
// when there are fewer than k. Each counts the keys above its own: all 256 threads'
// would take four times the instructions of 128 for a bound that 8 % fewer values reach.
__device__ __forceinline__ int threads_to_rep(int k) { return k <= 16 ? 4 : 2; }
__device__ __forceinline__ uint64_t bound_of_block(uint64_t key, int k, uint64_t* s_keys, uint64_t* s_bound) {
  const int per = threads_to_rep(k), reps = kThreads / per;
  key = max(key, __shfl_xor_sync(0xffffffffu, key, 1));
  if (per == 4) key = max(key, __shfl_xor_sync(0xffffffffu, key, 2));
  __syncthreads();
  if (threadIdx.x % per == 0) s_keys[threadIdx.x / per] = key;
  if (threadIdx.x == 0) *s_bound = 1;
  __syncthreads();
  if ((int)threadIdx.x < reps) {
    key = s_keys[threadIdx.x];
    int above = 0;
#pragma unroll 8
    for (int i = 0; i < reps; i += 2) {
      const ulonglong2 two = *reinterpret_cast<const ulonglong2*>(s_keys + i);
      above += (two.x > key) + (two.y > key);
    }
    if (key != 0 && above == k - 1) *s_bound = key;
  }
  __syncthreads();
  return *s_bound;
}

// The same from each warp's own values in turn: the smallest of the warps' ceil(k / 8)-th
// largest ones, as score_key (0: there is none). Weaker, but a fifth of the time: enough
// for the first tile, whose list is cut soon. It does not tell equal values apart.
__device__ __forceinline__ uint32_t bound_of_warps(float top, int k, uint32_t* s_warps) {
  uint32_t key = top > -INFINITY ? score_key(top) : 0u, best = 0;
  const int rounds = (k + kThreads / 32 - 1) / (kThreads / 32);
  for (int i = 0; i < rounds; ++i) {
    best = __reduce_max_sync(0xffffffffu, key);
    const uint32_t who = __ballot_sync(0xffffffffu, key == best);
    if ((threadIdx.x & 31) == __ffs(who) - 1) key = 0;
  }
  if ((threadIdx.x & 31) == 0) s_warps[threadIdx.x >> 5] = best;
  __syncthreads();
  best = s_warps[0];
#pragma unroll
  for (int i = 1; i < kThreads / 32; ++i) best = min(best, s_warps[i]);
  return best;
}

// Two fp32 operations at once (the values come in pairs of registers).
__device__ __forceinline__ void add2(float a, float b, float x, float y, float& s, float& t) {
  asm("{\n\t.reg .b64 u, v;\n\tmov.b64 u, {%2, %3};\n\tmov.b64 v, {%4, %5};\n\tadd.rn.f32x2 u, u, v;\n\tmov.b64 {%0, %1}, u;\n\t}"
      : "=f"(s), "=f"(t) : "f"(a), "f"(b), "f"(x), "f"(y));
}
__device__ __forceinline__ void mul2(float a, float b, float x, float& s, float& t) {
  asm("{\n\t.reg .b64 u, v;\n\tmov.b64 u, {%2, %3};\n\tmov.b64 v, {%4, %4};\n\tmul.rn.f32x2 u, u, v;\n\tmov.b64 {%0, %1}, u;\n\t}"
      : "=f"(s), "=f"(t) : "f"(a), "f"(b), "f"(x));
}
__device__ __forceinline__ float ex2(float x) {
  float e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x));
  return e;
}

__device__ __forceinline__ float warp_max(float x) {  // (NaN only where all are)
  float m;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(x));
  return m;
}

template <typename T>
struct Vec;  // 16 bytes of logits
template <>
struct Vec<float> {
  static constexpr int n = 4;
  static constexpr uint32_t none = 0xFF800000u;  // -inf
  static __device__ __forceinline__ void unpack(const uint4& v, float* x) {
    x[0] = __uint_as_float(v.x); x[1] = __uint_as_float(v.y); x[2] = __uint_as_float(v.z); x[3] = __uint_as_float(v.w);
  }
  static __device__ __forceinline__ float one(const float* p) { return *p; }
};
template <>
struct Vec<uint16_t> {
  static constexpr int n = 8;
  static constexpr uint32_t none = 0xFF80FF80u;
  static __device__ __forceinline__ void unpack(const uint4& v, float* x) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
  static __device__ __forceinline__ float one(const uint16_t* p) { return bf16_bits_to_f32(*p); }
};

struct Part {  // of a row's softmax: its largest value, the sum of exp(x - ref)
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
// the part's k largest. A tile of 4,096 values is in registers while the next is loaded. What
// reaches the bound goes to a list in shared memory; the bound is taken from the first tile,
// and from the list whenever that is long, which cuts it down to about 1.2 k. A list
// that would overflow (rising logits) is taken back to the tile's start and the bound
// is raised by the tile's own values: then only few threads' values pass.
template <typename T>
__global__ void __launch_bounds__(kThreads, 4) rows_kernel(RowArgs<T> a) {
  constexpr int kN = Vec<T>::n, kVectors = kX / kN;
  // what is kept, a tile's values over its own bound (4 k threads' for k <= 16, 2 k
  // threads' above) and the row's ends fit together
  static_assert(kThreads + 2 * kMaxK * kX + 2 * kN <= kRoom && 4 * 16 <= 2 * kMaxK && kRoom % kThreads == 0, "list too short");
  __shared__ __align__(16) uint64_t s_list[kRoom];
  __shared__ __align__(16) uint64_t s_keys[kThreads / 2];
  __shared__ uint64_t s_kth;
  __shared__ int s_added[3], s_left;
  __shared__ uint32_t s_warps[kThreads / 32];
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
  const int keep = k <= 32 ? kThreads / 2 : kThreads;  // a longer list is cut

  float ref = -INFINITY, sum = 0.0f;
  uint64_t bound = 1;
  float bound_value = -FLT_MAX;  // (-inf is no candidate)
  int n = 0;  // entries of the list, as every thread knows it
  if (threadIdx.x < 3) s_added[threadIdx.x] = 0;
  __syncthreads();

  // The list down to what reaches its own bound: the entries of 4 k or 2 k threads, so
  // from n to n / 2 + keep / 2 at most.
  const auto cut = [&]() {
    uint64_t mine[kRoom / kThreads];
    uint64_t best = 0;
#pragma unroll
    for (int i = 0; i < kRoom / kThreads; ++i) {
      const int at = i * kThreads + threadIdx.x;
      mine[i] = at < n ? s_list[at] : 0;
      best = max(best, mine[i]);
    }
    bound = max(bound, bound_of_block(best, k, s_keys, &s_kth));
    if (threadIdx.x == 0) s_left = 0;
    __syncthreads();
    int stay = 0;
#pragma unroll
    for (int i = 0; i < kRoom / kThreads; ++i) stay += mine[i] >= bound;
    if (stay) {
      int at = atomicAdd(&s_left, stay);
#pragma unroll
      for (int i = 0; i < kRoom / kThreads; ++i)
        if (mine[i] >= bound) s_list[at++] = mine[i];
    }
    __syncthreads();
    n = s_left;
    bound_value = bound > 1 ? key_value(bound) : -FLT_MAX;
  };

  uint4 raw[kVectors];
  const auto fetch = [&](int32_t v0) {
#pragma unroll
    for (int j = 0; j < kVectors; ++j) {
      const int32_t v = v0 + j * kThreads + (int32_t)threadIdx.x;
      raw[j] = v < v_end ? __ldcs(reinterpret_cast<const uint4*>(x0 + lead) + v)
                         : make_uint4(Vec<T>::none, Vec<T>::none, Vec<T>::none, Vec<T>::none);
    }
  };
  fetch(v_begin);
  bool first = true;
  int turn = 0;  // the tile's counter of three
  for (int32_t v0 = v_begin; v0 < v_end; v0 += kThreads * kVectors) {
    float x[kX];
#pragma unroll
    for (int j = 0; j < kVectors; ++j) Vec<T>::unpack(raw[j], x + j * kN);
    fetch(v0 + kThreads * kVectors);
    const auto place_of = [&](int i) {
      return (uint32_t)(lead + (v0 + (i / kN) * kThreads + (int32_t)threadIdx.x) * kN + i % kN);
    };
    float top = x[0];
#pragma unroll
    for (int i = 1; i < kX; ++i) top = fmaxf(top, x[i]);
    // (one reference for a warp: each lane's own rises in most tiles)
    const float warp_top = warp_max(top);
    if (warp_top > ref) {
      if (ref > -INFINITY) sum *= exp2f((ref - warp_top) * kLog2e);
      ref = warp_top;
    }
    // (x - ref first: exact where it counts, and 0 for a row of the type's lowest
    // value, whose product with log2 e is infinite; with ref +inf the sum is NaN)
    const float from = ref > -INFINITY ? -ref : 0.0f;
    float add[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < kX; i += 2) {
      float u, v;
      add2(x[i], x[i + 1], from, from, u, v);
      mul2(u, v, kLog2e, u, v);
      add2(add[i % 4], add[i % 4 + 1], ex2(u), ex2(v), add[i % 4], add[i % 4 + 1]);
    }
    sum += (add[0] + add[1]) + (add[2] + add[3]);

    // (mostly it is one value of a thread, its largest: to look for it costs a third of
    // trying each in turn)
    const auto put = [&](uint64_t key) {
      if (key < bound) return;
      const int at = n + atomicAdd(&s_added[turn], 1);
      if (at < kRoom) s_list[at] = key;
    };
    const auto push = [&]() {
      if (!(top >= bound_value)) return;
      uint32_t pass = 0;
#pragma unroll
      for (int i = 0; i < kX; ++i)
        if (x[i] >= bound_value) pass |= 1u << i;
      if ((pass & (pass - 1)) == 0) {
        put(make_key(top, place_of(__ffs(pass) - 1)));
        return;
      }
#pragma unroll
      for (int i = 0; i < kX; ++i)
        if (pass >> i & 1u) put(make_key(x[i], place_of(i)));
    };
    if (first) {
      const uint32_t least = bound_of_warps(top, k, s_warps);
      if (least) {
        bound = (uint64_t)least << 32;
        bound_value = key_value(bound);
      }
    }
    push();
    __syncthreads();
    int added = s_added[turn];
    // the tile's before this one: everyone has read it, and it is added to again behind
    // the next barrier. So a tile has one barrier, and the list is not read before it.
    if (threadIdx.x == 0) s_added[turn == 0 ? 2 : turn - 1] = 0;
    if (n + added > kRoom) {
      int at = 0;
#pragma unroll
      for (int i = kX - 1; i > 0; --i)
        if (x[i] == top) at = i;
      if (x[0] == top) at = 0;
      const uint64_t best = top > -INFINITY ? make_key(top, place_of(at)) : 0;
      bound = max(bound, bound_of_block(best, k, s_keys, &s_kth));
      bound_value = bound > 1 ? key_value(bound) : -FLT_MAX;
      if (threadIdx.x == 0) s_added[turn] = 0;
      __syncthreads();
      push();
      __syncthreads();
      added = s_added[turn];
    }
    n += added;
    while (n > keep) cut();
    first = false;
    turn = turn == 2 ? 0 : turn + 1;
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
      if (key >= bound) s_list[n + atomicAdd(&s_added[turn], 1)] = key;
    }
    __syncthreads();
    n += s_added[turn];
  }
  while (n > keep) cut();
  if (threadIdx.x == 0) s_list[n] = 0;  // (read in pairs; n <= keep)
  __syncthreads();

  // the k largest, each to its rank
  uint64_t* list = a.lists + (int64_t)blockIdx.x * k;
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const uint64_t key = s_list[i];
    int above = 0;
#pragma unroll 4
    for (int j = 0; j < n; j += 2) {
      const ulonglong2 two = *reinterpret_cast<const ulonglong2*>(s_list + j);
      above += (two.x > key) + (two.y > key);
    }
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
  int32_t W, k, parts, merged, k_shift, row_shift;
  const Part* part;
  const uint64_t* lists;
  const float* scores;
  float* out_scores;
  int32_t *out_parents, *out_tokens;
  float* lse;
};

// Joins `lists` lists (each of 2^shift falling keys, one after another) in fours or pairs
// until `left` are left; of equal keys those of the lower list come first. A key's rank is
// its place in its own list and, by bisection, those in the others: one thread a key, the
// bisections side by side. x holds the lists and y half as many, xp and yp (kPlaces) what
// goes with the keys; returns where the last ones are.
template <int kWays, bool kPlaces>
__device__ __forceinline__ void join_round(const uint64_t* x, uint64_t* y, const uint64_t* xp, uint64_t* yp, int lists, int shift) {
  const int size = 1 << shift;
  for (int i = threadIdx.x; i < lists << shift; i += kJoinThreads) {
    const uint64_t e = x[i];
    const int l = i >> shift, l0 = l & ~(kWays - 1);
    int pos[kWays - 1] = {};
    const uint64_t* other[kWays - 1];
    uint64_t least[kWays - 1];  // keys from here on come before e
#pragma unroll
    for (int o = 0; o < kWays - 1; ++o) {
      const int m = l0 + ((l + 1 + o) & (kWays - 1));
      other[o] = x + (m << shift);
      least[o] = e + (m > l ? 1 : 0);
    }
    for (int s = size / 2; s; s /= 2) {
#pragma unroll
      for (int o = 0; o < kWays - 1; ++o)
        if (other[o][pos[o] + s - 1] >= least[o]) pos[o] += s;
    }
    int rank = i & (size - 1);
#pragma unroll
    for (int o = 0; o < kWays - 1; ++o) rank += pos[o] + (other[o][pos[o]] >= least[o] ? 1 : 0);
    if (rank < size) {
      const int at = ((l / kWays) << shift) + rank;
      y[at] = e;
      if (kPlaces) yp[at] = xp[i];
    }
  }
  __syncthreads();
}

// Ahead of that, where there are many lists: `merged` lists of a row, one after another in
// memory, into one by a warp, a list's 2^shift keys in kE registers of as many lanes. The
// larger ones of the keys so far and the next list's from its end are the best of both, rising
// and falling, and put in order by shift exchanges with the lanes 2^i apart. (A bisection
// reads shared memory at 32 places at once: with four times the lists, 4,096 keys, the
// kernel took 17 us longer, so merged 1.)
template <int kE>
__device__ __forceinline__ void merge_parts(const uint64_t* from, uint64_t* to, int lists, int merged, int k, int shift) {
  const int size = 1 << shift, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int place = lane & (size - 1);  // and place + 32
  const int at_once = kE == 1 ? 32 >> shift : 1;
  for (int g0 = warp * at_once; g0 < lists / merged; g0 += kJoinThreads / 32 * at_once) {
    const int g = g0 + (kE == 1 ? lane >> shift : 0);
    const bool here = g < lists / merged;
    const uint64_t* list = from + (int64_t)g * merged * k;
    const auto load = [&](int j, int at) { return here && j < merged && at < k ? list[(int64_t)j * k + at] : 0; };
    // two at a time, the even lists and the odd ones: an exchange waits 25 cycles for its lanes
    uint64_t best[2][kE];
    const auto order = [&](int n) {
      if (kE == 2)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const uint64_t a = best[c][0], b = best[c][kE - 1];
          best[c][0] = max(a, b);
          best[c][kE - 1] = min(a, b);
        }
      for (int o = kE == 2 ? 16 : size / 2; o; o /= 2)
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int e = 0; e < kE; ++e) {
            if (c >= n) continue;
            const uint64_t other = __shfl_xor_sync(0xffffffffu, best[c][e], o);
            best[c][e] = (lane & o) == 0 ? max(best[c][e], other) : min(best[c][e], other);
          }
    };
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int e = 0; e < kE; ++e) best[c][e] = load(c, c == 0 || merged > 2 ? place + 32 * e : size - 1 - place - 32 * e);
    for (int j0 = 2; j0 < merged; j0 += 4) {
      uint64_t next[4][kE];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int e = 0; e < kE; ++e) next[i][e] = load(j0 + i, size - 1 - place - 32 * e);
#pragma unroll
      for (int i = 0; i < 4; i += 2) {
        if (j0 + i >= merged) break;
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int e = 0; e < kE; ++e) best[c][e] = max(best[c][e], next[i + c][e]);
        order(2);
      }
    }
    if (merged > 1) {
#pragma unroll
      for (int e = 0; e < kE; ++e) {
        uint64_t other = best[1][kE - 1 - e];
        if (merged > 2) other = __shfl_xor_sync(0xffffffffu, other, kE == 2 ? 31 : size - 1);
        else other = best[1][e];
        best[0][e] = max(best[0][e], other);
      }
      order(1);
    }
#pragma unroll
    for (int e = 0; e < kE; ++e)
      if (here) to[(g << shift) + place + 32 * e] = best[0][e];
  }
}

struct Lists {
  const uint64_t *keys, *places;
};
template <bool kPlaces>
__device__ __forceinline__ Lists join_lists(uint64_t* x, uint64_t* y, uint64_t* xp, uint64_t* yp, int lists, int left, int shift) {
  while (lists > left) {
    const bool four = lists >= 4 * left;
    if (four)
      join_round<4, kPlaces>(x, y, xp, yp, lists, shift);
    else
      join_round<2, kPlaces>(x, y, xp, yp, lists, shift);
    lists /= four ? 4 : 2;
    uint64_t* t = x;
    x = y;
    y = t;
    t = xp;
    xp = yp;
    yp = t;
  }
  return {x, xp};
}

// score + (x - lse) as the sum of two fp32 values, the first its rounding: 48 bits, by
// exact sums of two (Knuth), where a 64-bit operation takes the time of 64 of these. Key:
// larger for a larger sum. (x - lse first: the lowest value of fp32 less itself leaves the
// score.)
__device__ __forceinline__ float two_sum(float a, float b, float& e) {
  const float s = __fadd_rn(a, b), z = __fsub_rn(s, a);
  e = __fadd_rn(__fsub_rn(a, __fsub_rn(s, z)), __fsub_rn(b, z));
  return s;
}
__device__ __forceinline__ uint64_t sum_key(float score, float x, float lse, float lse_rest) {
  float e, f, g;
  const float d = two_sum(x, -lse, e);
  const float t = two_sum(d, score, f);
  float sum = two_sum(t, __fadd_rn(__fsub_rn(e, lse_rest), f), g);
  if (!(fabsf(sum) <= FLT_MAX)) sum = -FLT_MAX, g = 0.0f;  // (a score below fp32's range)
  return (uint64_t)score_key(__fadd_rn(sum, 0.0f)) << 32 | score_key(__fadd_rn(g, 0.0f));
}

// Powers of two: a list's entries, a sequence's rows.
__host__ __device__ constexpr int power_shift(int n) {
  int s = 0;
  while ((1 << s) < n) ++s;
  return s;
}
// Lists that merge_parts() makes one: so many that a warp's lanes have one each, or a row's.
__host__ __device__ constexpr int merged_parts(int W, int parts, int k) {
  const int k2 = 1 << power_shift(k), at_once = kJoinThreads / 32 * (k2 < 32 ? 32 / k2 : 1);
  int merged = 1;
  while (merged < parts && W * (parts / merged) > at_once) merged *= 2;
  return merged;
}
__host__ __device__ constexpr int join_bytes(int W, int lists, int k) {
  const int k2 = 1 << power_shift(k), rows2 = 1 << power_shift(W);
  return (3 * lists * k2 + 2 * 3 * rows2 * k2) / 2 * (int)sizeof(uint64_t) + 64;
}
// (the lists merged are a row's or at most as many as the warps take at once)
constexpr int kMaxJoinBytes = 3 * 3 * CSA2_MAX_BEAMS * kMaxK / 2 * (int)sizeof(uint64_t) + 64;
static_assert(kJoinThreads / 32 * kMaxK <= CSA2_MAX_BEAMS * kMaxK && kMaxJoinBytes <= 226 * 1024, "lists too long");

// One CTA to a sequence: each row's lists are joined by value, the rows' lists by score,
// held to 48 bits so that their order is that of the formula to what the sums carry (in
// 32 bits x - lse would be rounded to 2^-20 for logits about 16). The time does not depend
// on the values.
__global__ void __launch_bounds__(kJoinThreads) join_kernel(JoinArgs a) {
  pdl_wait();
  extern __shared__ uint64_t s_lists[];  // the rows' keys and half as many, their places, the parts' keys
  __shared__ float s_lse[2][CSA2_MAX_BEAMS];  // two summands; NaN: the row takes no part
  __shared__ float s_score[CSA2_MAX_BEAMS];
  const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 31;
  const int k = a.k;
  const int64_t row0 = (int64_t)b * a.W;
  const int shift = a.k_shift, mask = (1 << shift) - 1;
  const int rows2 = 1 << a.row_shift;
  const int size = rows2 << shift, half = size / 2 + 1;
  uint64_t* x = s_lists;
  uint64_t* y = x + size;
  uint64_t* xp = y + half;
  uint64_t* yp = xp + size;
  uint64_t* keys = yp + half;
  const int lists = a.W * (a.parts / a.merged);
  const uint64_t* from = a.lists + row0 * a.parts * k;
  if (shift <= 5)
    merge_parts<1>(from, keys, a.W * a.parts, a.merged, k, shift);
  else
    merge_parts<2>(from, keys, a.W * a.parts, a.merged, k, shift);
  for (int w = tid >> 5; w < a.W; w += kJoinThreads / 32) {  // a warp to a row
    const Part* p = a.part + (row0 + w) * a.parts;
    float ref = -INFINITY;
    for (int c = lane; c < a.parts; c += 32) ref = fmaxf(ref, p[c].ref);
#pragma unroll
    for (int o = 16; o; o >>= 1) ref = fmaxf(ref, __shfl_xor_sync(0xffffffffu, ref, o));
    float sum = 0.0f;
    for (int c = lane; c < a.parts; c += 32) {
      const Part v = p[c];
      sum += v.ref == -INFINITY ? v.sum : v.sum * exp2f((v.ref - ref) * kLog2e);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) {
      float lse = -INFINITY, rest = 0.0f;
      if (!(sum <= 3.0e38f) || !(ref < INFINITY)) {
        record_error(&g_beam_error, CSA2_ERR_DEVICE);  // a NaN or +inf among the logits
        lse = __uint_as_float(0x7FC00000u);
      } else if (sum > 0.0f) {
        // the sum's exponent apart (ln 2 in two parts, the first of 15 bits: its products
        // are exact): the logarithm of a value in [1, 2) is off by 2^-24
        const uint32_t bits = __float_as_uint(sum);
        const float e = (float)((int)(bits >> 23) - 127), m = logf(__uint_as_float((bits & 0x7FFFFFu) | 0x3F800000u));
        float r0, r1;
        lse = two_sum(ref, e * 0.693145751953125f, r0);
        lse = two_sum(lse, m, r1);
        rest = fmaf(e, 1.42860682e-6f, r0 + r1);
        lse = two_sum(lse, rest, r0);
        rest = r0;
      }
      if (a.lse) a.lse[row0 + w] = lse;
      const float s = a.scores ? a.scores[row0 + w] : 0.0f;
      s_lse[0][w] = fabsf(s) < INFINITY && sum > 0.0f ? lse : __uint_as_float(0x7FC00000u);
      s_lse[1][w] = rest;
      s_score[w] = s;
    }
  }
  __syncthreads();
  // (the number of parts is a power of two: a row's lists are joined with one another)
  const uint64_t* rows = join_lists<false>(keys, keys + (lists << shift), nullptr, nullptr, lists, a.W, shift).keys;
  // (threads past the end take part in the shuffles)
  for (int i0 = 0; i0 < size; i0 += kJoinThreads) {
    const int i = i0 + tid, w = i >> shift;
    uint64_t mine = 0;
    if (i < size) {
      const uint64_t key = w < a.W ? rows[i] : 0;
      if (key != 0 && !isnan(s_lse[0][w])) mine = sum_key(s_score[w], key_value(key), s_lse[0][w], s_lse[1][w]);
      xp[i] = (uint64_t)w << 32 | key_place(key);
    }
    // A row's keys fall, as its logits do: logits closer than the last of the 48 bits may
    // come out in either order. (32 at a time; a list of 64 below.)
    const int place = lane & mask;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint64_t before = __shfl_up_sync(0xffffffffu, mine, o);
      if (place >= o) mine = min(mine, before);
    }
    if (i < size) x[i] = mine;
  }
  __syncthreads();
  if (mask >= 32) {
    for (int i = tid; i < size; i += kJoinThreads)
      if (i & 32) x[i] = min(x[i], x[(i & ~63) + 31]);
    __syncthreads();
  }
  const Lists best = join_lists<true>(x, y, xp, yp, rows2, 1, shift);
  for (int i = tid; i < k; i += kJoinThreads) {
    const uint64_t key = best.keys[i], at = best.places[i];
    const int64_t o = (int64_t)b * k + i;
    a.out_scores[o] = key ? key_value(key) : -INFINITY;
    a.out_parents[o] = key ? (int32_t)(row0 + (int64_t)(at >> 32)) : -1;
    a.out_tokens[o] = key ? (int32_t)at : -1;
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
  pdl_begin();
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
    const int64_t bytes = (int64_t)fill * kPlaneBytes[i];  // (a page of 2^23 entries holds 2^31 bytes of codes)
    for (int64_t at = threadIdx.x * 16; at + 16 <= bytes; at += kReorderThreads * 16)
      *reinterpret_cast<uint4*>(d + at) = *reinterpret_cast<const uint4*>(s + at);
    const int64_t tail = bytes & ~(int64_t)15;
    const int64_t at = tail + threadIdx.x * 4;
    if (at < bytes) *reinterpret_cast<uint32_t*>(d + at) = *reinterpret_cast<const uint32_t*>(s + at);
  }
}

constexpr int kRowSlice = kReorderThreads * 16 * 4;  // bytes of a row to a block

__global__ void __launch_bounds__(kReorderThreads)
    rows_copy_kernel(const uint8_t* __restrict__ src, int64_t rows_in, int64_t row_bytes, int64_t slices,
                     const int32_t* __restrict__ parents, uint8_t* __restrict__ dst) {
  // (no pdl_launch_dependents(): the selected attention behind reads its windows, which
  // this may have written, before its own wait)
  pdl_wait();
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

// Parts of a row, a power of two, of 2,048 values at least: at most 608 CTAs in all (four to
// each of 152 SMs: the size of a workspace does not depend on the device), 304 for k > 16,
// whose lists take longer (128 rows of 128,259 fp32, k 16: 22.4 us with 608, 23.8 with 304;
// 32 rows, k 32: 19.9 and 17.6), unless there are more rows.
static int beam_parts(int32_t B, int32_t W, int32_t V, int32_t k) {
  const int64_t rows = (int64_t)B * W;
  int64_t parts = 1;
  while (2 * parts * rows <= (k <= 16 ? 608 : 304) && 2 * parts * 2048 <= V) parts *= 2;
  return (int)parts;
}

extern "C" size_t csa2_beam_select_workspace_size(int32_t B, int32_t W, int32_t V, int32_t k) {
  if (check_beam(B, W, V, k) != CSA2_OK || B == 0 || W == 0) return 0;
  const size_t lists = (size_t)B * W * beam_parts(B, W, V, k);
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
  const int parts = beam_parts(B, W, V, k);
  const int64_t rows = (int64_t)B * W;
  beam::Part* part = (beam::Part*)workspace;
  uint64_t* lists = (uint64_t*)((char*)workspace + al256((size_t)rows * parts * sizeof(beam::Part)));
  cudaStream_t s = (cudaStream_t)stream;
  rc = logits_f32 ? launch_rows<float>(logits, ld, V, k, rows, parts, part, lists, s)
                  : launch_rows<uint16_t>(logits, ld, V, k, rows, parts, part, lists, s);
  if (rc) return rc;
  static Csa2PerDeviceOnce once;
  if (csa2_smem_optin((const void*)beam::join_kernel, beam::kMaxJoinBytes, once) != CSA2_OK) return CSA2_ERR_CUDA;
  const int merged = beam::merged_parts(W, parts, k);
  beam::JoinArgs j{W, k, parts, merged, beam::power_shift(k), beam::power_shift(W), part, lists, scores, out_scores, out_parents, out_tokens, lse};
  CSA2_LAUNCH_PDL(beam::join_kernel, dim3((unsigned)B), dim3(beam::kJoinThreads),
                  (size_t)beam::join_bytes(W, W * (parts / merged), k), s, j);
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
  CSA2_LAUNCH_PDL(beam::reorder_kernel, dim3((unsigned)R, (unsigned)(1 + layers)), dim3(beam::kReorderThreads), (size_t)0,
                  (cudaStream_t)stream, a);
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
  CSA2_LAUNCH_PDL(beam::rows_copy_kernel, dim3((unsigned)(R * slices)), dim3(beam::kReorderThreads), (size_t)0,
                  (cudaStream_t)stream, (const uint8_t*)src, rows_in, row_bytes, slices, parents, (uint8_t*)dst);
  return CSA2_OK;
}
