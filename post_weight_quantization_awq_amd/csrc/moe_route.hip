// Routing of tokens to experts: each token's k largest logits, their shares, and
// the (token, expert) pairs in expert order, as the grouped product takes them.
//
// Logits become unsigned keys that order as the values do.  Up to 256 experts, of
// which a token takes up to 8, a few lanes sort a token's logits (route_lanes_kernel);
// else a wave takes a token and k rounds of a wave maximum pick the experts
// (route_select_kernel).  A token has an expert at most once, so 64 tokens are a
// 64-bit mask for each expert in LDS: a pair's rank among its expert's is the number
// of set bits below its token's, the same in whatever order the bits were set.  Up to
// 64 tokens (a decoding step) one block does it all; more take two launches, the
// second of which adds the counts that the first left for each block.
//
// Bound by latency, not by the logits' bytes: 24 tokens of 128 experts, 8 each, take
// 3.9 us, of which a call that does next to nothing takes 3.2 (a wave for each token:
// 6.8); 16001 tokens take 12 to 14 us in two launches of 5 to 7 (10 MB: 2 us at a copy's
// rate).  The first has 251 blocks of four waves, one for each SIMD, so that nothing hides
// the chain of a token's comparisons; of the second 2 are the sums of 251 blocks' counts.
// 200000 tokens of 8 experts, 2 each, take 19 + 18 us, seven chunks a block.  A wave for
// each token, k rounds of a maximum: 24 tokens, 8 of 512 experts 11.6 us; 16001 tokens, 8 of
// 512 41 us, 16 of 256 38, 32 of 1024 146 (fp32; 66 MB, 14 us at a copy's rate).
#include "awq_launch.h"
#include "mx_device.h"

namespace awq {

constexpr int kRouteThreads = 1024, kRouteWaves = kRouteThreads / kWave, kRouteChunk = 64;
constexpr int kRouteTokens = kRouteChunk / kRouteWaves;  // a wave's tokens of a chunk

// Ascending with the value; NaN the largest, -0 as +0.  0: an expert that is not to be taken (-inf)
__device__ __forceinline__ uint32_t route_key(float f) {
  const uint32_t u = __builtin_bit_cast(uint32_t, f + 0.0f);
  if ((u & 0x7FFFFFFFu) > 0x7F800000u) return 0xFFFFFFFFu;
  if (u == 0xFF800000u) return 0;
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float route_value(uint32_t key) {  // of a key that is not 0
  return __builtin_bit_cast(float, key & 0x80000000u ? key & 0x7FFFFFFFu : ~key);
}

__device__ __forceinline__ float route_logit(const void* p, int dt, int64_t i) {
  if (dt == 2) return ((const float*)p)[i];
  const uint16_t v = ((const uint16_t*)p)[i];
  return dt == 0 ? h2f(v) : bf2f(v);
}

__device__ __forceinline__ uint32_t wave_top(uint32_t x) {
  x = max(x, dpp_u<0xB1>(x));
  x = max(x, dpp_u<0x4E>(x));
  x = max(x, dpp_u<0x141>(x));
  x = max(x, dpp_u<0x140>(x));
  const uint32_t a = __builtin_amdgcn_readlane(x, 0), b = __builtin_amdgcn_readlane(x, 16);
  const uint32_t c = __builtin_amdgcn_readlane(x, 32), d = __builtin_amdgcn_readlane(x, 48);
  return max(max(a, b), max(c, d));
}

struct RouteArgs {
  const void* logits;
  int dtype;  // 0 fp16, 1 bf16, 2 fp32
  int64_t ld;
  int64_t rows;
  int n_experts, top;
  bool renorm;
  float scale;
  int32_t* experts;
  float* weights;
  int32_t* rows_out;
  int32_t* places;
  int32_t* offsets;
  uint16_t* counts;  // [blocks][ld_counts]
  int ld_counts;     // n_experts, in eights
  int per, blocks;   // tokens a block (a multiple of 64)
};

// A token's experts in descending order, lane j its j-th one (-1: none left) and share
template <int EL>
__device__ __forceinline__ void route_token(const RouteArgs& a, uint32_t (&v)[EL], int lane, int* id, float* share) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < EL; ++i) top = max(top, v[i]);
  const uint32_t first = wave_top(top);
  const float most = route_value(first);
  float sum = 0.0f;
  if (!a.renorm) {  // the shares are of all experts
#pragma unroll
    for (int i = 0; i < EL; ++i)
      if (v[i] != 0) sum += expf(route_value(v[i]) - most);
    sum = wave_sum(sum);
  }
  int mine = -1;
  uint32_t key = 0;
  for (int j = 0; j < a.top; ++j) {
    const uint32_t t = j == 0 ? first : wave_top(top);
    if (t == 0) break;
    int e = 0;
#pragma unroll
    for (int i = EL - 1; i >= 0; --i) {
      const uint64_t who = __ballot(v[i] == t);
      if (who != 0) e = i * kWave + __builtin_ctzll(who);
    }
    top = 0;
#pragma unroll
    for (int i = 0; i < EL; ++i) {
      if (i * kWave + lane == e) v[i] = 0;
      top = max(top, v[i]);
    }
    if (lane == j) mine = e, key = t;
  }
  const float p = mine >= 0 ? expf(route_value(key) - most) : 0.0f;
  if (a.renorm) sum = wave_sum(p);
  *id = mine;
  *share = mine >= 0 ? p / sum * a.scale : 0.0f;
}

// The exclusive sum of `v` over the block's threads, and the total
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t* part, uint32_t* total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  uint32_t x = v;
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) {
    const uint32_t y = __shfl_up(x, d, kWave);
    if (lane >= d) x += y;
  }
  if (lane == 63) part[wave] = x;
  __syncthreads();
  uint32_t before = 0, all = 0;
#pragma unroll
  for (int i = 0; i < kRouteWaves; ++i) {
    before += i < wave ? part[i] : 0;
    all += part[i];
  }
  *total = all;
  return before + x - v;
}

// Rows behind the last pair name no token
__device__ __forceinline__ void route_rest(const RouteArgs& a, int64_t total, int64_t first, int64_t step) {
  for (int64_t i = total + first; i < a.rows * a.top; i += step) a.rows_out[i] = -1;
}

// ONE: the only block, which also places the pairs
template <int EL, bool ONE>
__global__ __launch_bounds__(kRouteThreads) void route_select_kernel(const RouteArgs a) {
  __shared__ unsigned long long mask[EL * kWave];
  __shared__ uint32_t base[ONE ? EL * kWave : 1], part[kRouteWaves];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t t0 = (int64_t)blockIdx.x * a.per;
  uint32_t count = 0;  // of expert `tid`
  int id[kRouteTokens];
  for (int c = 0; c < a.per && t0 + c < a.rows; c += kRouteChunk) {
    for (int e = tid; e < EL * kWave; e += kRouteThreads) mask[e] = 0;
    uint32_t v[kRouteTokens][EL];
#pragma unroll
    for (int i = 0; i < kRouteTokens; ++i) {
      const int64_t t = t0 + c + wave + kRouteWaves * i;
#pragma unroll
      for (int q = 0; q < EL; ++q) {
        const int e = q * kWave + lane;
        v[i][q] = t < a.rows && e < a.n_experts ? route_key(route_logit(a.logits, a.dtype, t * a.ld + e)) : 0;
      }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kRouteTokens; ++i) {
      const int64_t t = t0 + c + wave + kRouteWaves * i;
      id[i] = -1;
      if (t < a.rows) {
        float share;
        route_token<EL>(a, v[i], lane, &id[i], &share);
        if (lane < a.top) {
          a.experts[t * a.top + lane] = id[i];
          a.weights[t * a.top + lane] = share;
        }
        if (id[i] >= 0) atomicOr(&mask[id[i]], 1ull << (wave + kRouteWaves * i));
      }
    }
    __syncthreads();
    if (tid < a.n_experts) count += __popcll(mask[tid]);
    if constexpr (!ONE) __syncthreads();  // the masks are cleared for the next chunk
  }
  if constexpr (!ONE) {
    if (tid < a.ld_counts) a.counts[(int64_t)blockIdx.x * a.ld_counts + tid] = (uint16_t)count;
  } else {
    uint32_t total;
    const uint32_t first = block_scan(count, part, &total);
    if (tid < a.n_experts) a.offsets[tid] = (int)first, base[tid] = first;
    if (tid == 0) a.offsets[a.n_experts] = (int)total;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kRouteTokens; ++i) {
      const int tt = wave + kRouteWaves * i;
      if (tt < a.rows && lane < a.top) {
        int place = -1;
        if (id[i] >= 0) {
          place = (int)(base[id[i]] + __popcll(mask[id[i]] & ((1ull << tt) - 1)));
          a.rows_out[place] = tt;
        }
        a.places[tt * a.top + lane] = place;
      }
    }
    route_rest(a, total, tid, kRouteThreads);
  }
}

// L lanes take a token, each a part of its logits.  A lane sorts K of them at a time and merges them into its best K, in
// order; merges across the lanes join those.  A logit and its expert are one word that orders as
// they do, so that a comparison is a maximum and a minimum: for 16-bit logits 32 bits, the 19 of the key that such a
// value can set over the experts from the last to the first; for 32-bit ones a positive double, 32 bits of key over 30.
// Four lanes do that for 128 experts and 8 places with 300 comparisons each, all their logits in flight at once; a wave
// for each token takes 300 operations of 64 lanes (16001 tokens: 14 us, 22 with waves).  Up to 64 tokens 16 lanes take
// one, for latency (24 tokens: 3.9 us).
constexpr int kLaneExperts = 256;
constexpr uint32_t kNoKey = 0x007FFFFFu;  // -inf's: no larger one, no expert
template <int DT>
struct RouteWord {
  using type = uint32_t;
  static __device__ __forceinline__ type pack(uint32_t key, uint32_t e) { return (key & 0xFFFFE000u) | (0x1FFFu - e); }
  static __device__ __forceinline__ float value(type w) {
    return __builtin_bit_cast(float, __builtin_bit_cast(uint32_t, route_value(w)) & 0xFFFFE000u);
  }
  static __device__ __forceinline__ int expert(type w) { return (int)(0x1FFFu - (w & 0x1FFFu)); }
  static __device__ __forceinline__ bool some(type w) { return w > kNoKey; }
  static __device__ __forceinline__ void order(type& a, type& b) {  // a the larger
    const type m = max(a, b);
    b = min(a, b);
    a = m;
  }
  static __device__ __forceinline__ type larger(type a, type b) { return max(a, b); }
  template <int CTRL>
  static __device__ __forceinline__ type moved(type w) { return dpp_u<CTRL>(w); }
};
template <>
struct RouteWord<2> {
  using type = double;
  static __device__ __forceinline__ uint64_t bits(type w) { return __builtin_bit_cast(uint64_t, w); }
  static __device__ __forceinline__ type pack(uint32_t key, uint32_t e) {
    return __builtin_bit_cast(double, (uint64_t)key << 30 | (0x3FFFFFFFu - e));
  }
  static __device__ __forceinline__ uint32_t key(type w) { return (uint32_t)(bits(w) >> 30); }
  static __device__ __forceinline__ int expert(type w) { return (int)(0x3FFFFFFFu - ((uint32_t)bits(w) & 0x3FFFFFFFu)); }
  static __device__ __forceinline__ float value(type w) { return route_value(key(w)); }
  static __device__ __forceinline__ bool some(type w) { return key(w) > kNoKey; }
  // No word is a NaN; __builtin_fmax would make sure of it first, with an instruction for each operand
  static __device__ __forceinline__ type larger(type a, type b) {
    type m;
    asm("v_max_f64 %0, %1, %2" : "=v"(m) : "v"(a), "v"(b));
    return m;
  }
  static __device__ __forceinline__ void order(type& a, type& b) {
    const type m = larger(a, b);
    asm("v_min_f64 %0, %1, %2" : "=v"(b) : "v"(a), "v"(b));
    a = m;
  }
  template <int CTRL>
  static __device__ __forceinline__ type moved(type w) {
    asm("s_nop 1" : "+v"(w));  // the two states from an instruction's result, here an asm's, to its use by another lane
    return __builtin_bit_cast(double, (uint64_t)dpp_u<CTRL>((uint32_t)(bits(w) >> 32)) << 32 | dpp_u<CTRL>((uint32_t)bits(w)));
  }
};
// K words into descending order: odd-even merge sort
template <class W, int K>
__device__ __forceinline__ void sort_words(typename W::type* x) {
#pragma unroll
  for (int p = 1; p < K; p *= 2)
#pragma unroll
    for (int k = p; k >= 1; k /= 2)
#pragma unroll
      for (int j = k % p; j + k < K; j += 2 * k)
#pragma unroll
        for (int i = 0; i < k; ++i)
          if (i + j + k < K && (i + j) / (2 * p) == (i + j + k) / (2 * p)) W::order(x[i + j], x[i + j + k]);
}
// v: the K largest of v and o, both in descending order
template <class W, int K>
__device__ __forceinline__ void merge_words(typename W::type* v, const typename W::type* o) {
#pragma unroll
  for (int i = 0; i < K; ++i) v[i] = W::larger(v[i], o[K - 1 - i]);  // falls, then rises, or the other way round
#pragma unroll
  for (int d = K / 2; d >= 1; d /= 2)
#pragma unroll
    for (int i = 0; i < K; ++i)
      if ((i & d) == 0) W::order(v[i], v[i + d]);
}
template <class W, int K, int CTRL>
__device__ __forceinline__ void merge_lanes(typename W::type* v) {
  typename W::type o[K];
#pragma unroll
  for (int i = 0; i < K; ++i) o[i] = W::template moved<CTRL>(v[i]);
  merge_words<W, K>(v, o);
}

// The lane's 8 logits of 32 from e on; -inf for those that are not there
template <int DT>
__device__ __forceinline__ void load_logits8(const RouteArgs& a, int64_t at, int e, float (&f)[8]) {
  if (e + 8 <= a.n_experts) {
    if constexpr (DT == 2) {
      *(float4*)&f[0] = ld_any<float4>((const float*)a.logits + at + e);
      *(float4*)&f[4] = ld_any<float4>((const float*)a.logits + at + e + 4);
    } else {
      unpack8<DT>(ld_any<uint4>((const uint16_t*)a.logits + at + e), f);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = e + i < a.n_experts ? route_logit(a.logits, DT, at + e + i) : -INFINITY;
  }
}
// Ascending with the value; NaN the largest, -0 as +0
__device__ __forceinline__ uint32_t plain_key(float f) {
  const uint32_t u = __builtin_bit_cast(uint32_t, f + 0.0f), k = u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
  return f != f ? 0xFFFFFFFFu : k;
}

// L lanes a token.  ONE: the only block, which also places the pairs
template <int K, int DT, int L, bool ONE>
__global__ __launch_bounds__(L * kRouteChunk) void route_lanes_kernel(const RouteArgs a) {
  using W = RouteWord<DT>;
  static_assert(!ONE || L * kRouteChunk == kRouteThreads, "the scan is of 16 waves");
  __shared__ unsigned long long mask[kLaneExperts];
  __shared__ uint32_t base[ONE ? kLaneExperts : 1], part[kRouteWaves];
  constexpr int kGroups = 16 / L;  // of 8 logits a lane, for 128 experts
  constexpr int PL = (K + L - 1) / L;  // the lane's places: q, q + L
  const int tid = threadIdx.x, q = tid % L, tt = tid / L;
  const int64_t t0 = (int64_t)blockIdx.x * a.per;
  uint32_t count = 0;  // of expert `tid`
  int id[PL];
  for (int c = 0; c < a.per && t0 + c < a.rows; c += kRouteChunk) {
    if (tid < kLaneExperts) mask[tid] = 0;
    const int64_t t = t0 + c + tt;
    const bool live = t < a.rows;
    float share[PL];
#pragma unroll
    for (int i = 0; i < PL; ++i) id[i] = -1, share[i] = 0.0f;
    if (t0 + c + __builtin_amdgcn_readfirstlane(tt) < a.rows) {  // a token for some lanes of the wave
      const int64_t at = (live ? t : a.rows - 1) * a.ld;
      typename W::type v[K] = {};
      float sum = 0.0f;
      for (int e = 8 * q; e < a.n_experts; e += 128) {
        float f[kGroups][8];
#pragma unroll
        for (int g = 0; g < kGroups; ++g) load_logits8<DT>(a, at, e + 8 * L * g, f[g]);
#pragma unroll
        for (int g = 0; g < kGroups; ++g) {
          typename W::type x[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] = W::pack(plain_key(f[g][i]), (uint32_t)(e + 8 * L * g + i));
#pragma unroll
          for (int i = 0; i < 8; i += K) {
            sort_words<W, K>(x + i);
            merge_words<W, K>(v, x + i);
          }
        }
      }
      merge_lanes<W, K, 0xB1>(v);
      merge_lanes<W, K, 0x4E>(v);
      if constexpr (L == 16) {
        merge_lanes<W, K, 0x141>(v);
        merge_lanes<W, K, 0x140>(v);
      }
      const float most = W::value(v[0]);
      if (!a.renorm && W::some(v[0])) {
        for (int e = 8 * q; e < a.n_experts; e += 8 * L) {
          float f[8];
          load_logits8<DT>(a, at, e, f);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (f[i] != -INFINITY) sum += expf(f[i] - most);
        }
      }
#pragma unroll
      for (int i = 0; i < PL; ++i) {
        typename W::type d = 0;
#pragma unroll
        for (int s = 0; s < L; ++s)
          if (L * i + s < K) d = q == s ? v[L * i + s] : d;
        if (live && W::some(d) && L * i + q < a.top) id[i] = W::expert(d);
        share[i] = id[i] >= 0 ? expf(W::value(d) - most) : 0.0f;
        if (a.renorm) sum += share[i];
      }
      sum += dpp_m<0xB1>(sum);
      sum += dpp_m<0x4E>(sum);
      if constexpr (L == 16) {
        sum += dpp_m<0x141>(sum);
        sum += dpp_m<0x140>(sum);
      }
#pragma unroll
      for (int i = 0; i < PL; ++i) share[i] = id[i] >= 0 ? share[i] / sum * a.scale : 0.0f;
    }
    __syncthreads();  // the masks are clear
#pragma unroll
    for (int i = 0; i < PL; ++i)
      if (live && L * i + q < a.top) {
        a.experts[t * a.top + L * i + q] = id[i];
        a.weights[t * a.top + L * i + q] = share[i];
        if (id[i] >= 0) atomicOr(&mask[id[i]], 1ull << tt);
      }
    __syncthreads();
    if (tid < kLaneExperts) count += __popcll(mask[tid]);
    if constexpr (!ONE) __syncthreads();  // the masks are cleared for the next chunk
  }
  if constexpr (!ONE) {
    if (tid < a.ld_counts) a.counts[(int64_t)blockIdx.x * a.ld_counts + tid] = (uint16_t)count;
  } else {
    uint32_t total;
    const uint32_t first = block_scan(count, part, &total);
    if (tid < a.n_experts) a.offsets[tid] = (int)first, base[tid] = first;
    if (tid == 0) a.offsets[a.n_experts] = (int)total;
    __syncthreads();
    if (tt < a.rows && q < a.top) {
      int place = -1;
      if (id[0] >= 0) {
        place = (int)(base[id[0]] + __popcll(mask[id[0]] & ((1ull << tt) - 1)));
        a.rows_out[place] = tt;
      }
      a.places[tt * a.top + q] = place;
    }
    route_rest(a, total, tid, kRouteThreads);
  }
}

// Places of a block's pairs: the experts' totals and what lies in the blocks before, from the counts of all blocks,
// 8 experts a thread.
__global__ __launch_bounds__(kRouteThreads) void route_place_kernel(const RouteArgs a) {
  __shared__ unsigned long long mask[1024];
  __shared__ uint32_t base[1024], total[1024], part[kRouteWaves];
  const int tid = threadIdx.x;
  const int64_t t0 = (int64_t)blockIdx.x * a.per;
  const int slots = kRouteChunk * a.top;
  int id[2];  // of the chunk's pairs tid and tid + 1024: at most 64 x 32
  auto pairs_of = [&](int c) { return a.rows - t0 - c < kRouteChunk ? (int)(a.rows - t0 - c) * a.top : slots; };
  auto load_ids = [&](int c) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int s = tid + kRouteThreads * i;
      id[i] = s < pairs_of(c) ? a.experts[(t0 + c) * a.top + s] : -1;
    }
  };
  load_ids(0);  // ahead of the counts' sums
  base[tid] = total[tid] = 0;
  mask[tid] = 0;
  __syncthreads();
  // lanes of a row of counts: a power of two, so that the rows of a wave are summed across its lanes first
  const int cols = a.ld_counts / 8;
  int lanes = 1;
  while (lanes < cols) lanes *= 2;
  const int step = kRouteThreads / lanes, col = tid & (lanes - 1), seg = tid / lanes;
  uint32_t all[8] = {}, before[8] = {};
  if (col < cols) {
    for (int b0 = seg; b0 < a.blocks; b0 += 4 * step) {
      uint4 u[4];  // in flight at once
#pragma unroll
      for (int k = 0; k < 4; ++k)
        u[k] = b0 + k * step < a.blocks ? *(const uint4*)(a.counts + (int64_t)(b0 + k * step) * a.ld_counts + 8 * col)
                                        : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t w[4] = {u[k].x, u[k].y, u[k].z, u[k].w};
        const bool under = b0 + k * step < (int)blockIdx.x;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t n = i % 2 ? w[i / 2] >> 16 : w[i / 2] & 0xFFFFu;
          all[i] += n;
          before[i] += under ? n : 0;
        }
      }
    }
  }
  for (int d = kWave / 2; d >= lanes; d /= 2)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      all[i] += __shfl_xor(all[i], d, kWave);
      before[i] += __shfl_xor(before[i], d, kWave);
    }
  if ((tid & (kWave - 1)) < lanes && col < cols)
#pragma unroll
    for (int i = 0; i < 8; ++i) {  // expert 8 col + i at col + i lanes: one bank each
      if (all[i]) atomicAdd(&total[col + i * lanes], all[i]);
      if (before[i]) atomicAdd(&base[col + i * lanes], before[i]);
    }
  __syncthreads();
  const int at = (tid / 8 & (lanes - 1)) + tid % 8 * lanes;  // of expert `tid`
  const uint32_t mine = tid < a.ld_counts ? total[at] : 0, lower = tid < a.ld_counts ? base[at] : 0;
  uint32_t sum;
  const uint32_t first = block_scan(mine, part, &sum);  // all have read base
  base[tid] = lower + first;
  if (blockIdx.x == 0) {
    if (tid < a.n_experts) a.offsets[tid] = (int)first;
    if (tid == 0) a.offsets[a.n_experts] = (int)sum;
  }
  for (int c = 0; c < a.per && t0 + c < a.rows; c += kRouteChunk) {
    if (c > 0) load_ids(c);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int s = tid + kRouteThreads * i;
      if (id[i] >= 0) atomicOr(&mask[id[i]], 1ull << (s / a.top));
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int s = tid + kRouteThreads * i;
      if (s < pairs_of(c)) {
        int place = -1;
        if (id[i] >= 0) {
          place = (int)(base[id[i]] + __popcll(mask[id[i]] & ((1ull << (s / a.top)) - 1)));
          a.rows_out[place] = (int)(t0 + c) + s / a.top;
        }
        a.places[(t0 + c) * a.top + s] = place;
      }
    }
    __syncthreads();
    base[tid] += __popcll(mask[tid]);
    mask[tid] = 0;
    __syncthreads();
  }
  route_rest(a, sum, (int64_t)blockIdx.x * kRouteThreads + tid, (int64_t)a.blocks * kRouteThreads);
}

constexpr int64_t kRouteBlocks = 512;
static int route_per(int64_t rows) {  // at least a chunk, also without rows
  if (rows <= kRouteChunk) return kRouteChunk;
  return (int)((rows + kRouteBlocks * kRouteChunk - 1) / (kRouteBlocks * kRouteChunk)) * kRouteChunk;
}
static int64_t route_blocks(int64_t rows) {
  return rows <= kRouteChunk ? 1 : (rows + route_per(rows) - 1) / route_per(rows);
}

size_t moe_route_workspace(int64_t rows, int n_experts) {
  return rows <= kRouteChunk ? 0 : (size_t)route_blocks(rows) * ((n_experts + 7) / 8 * 8) * sizeof(uint16_t);
}

template <int K, int DT>
static void route_lanes_launch(const RouteArgs& a, hipStream_t stream) {
  if (a.blocks == 1) route_lanes_kernel<K, DT, 16, true><<<1, 16 * kRouteChunk, 0, stream>>>(a);
  else route_lanes_kernel<K, DT, 4, false><<<(unsigned)a.blocks, 4 * kRouteChunk, 0, stream>>>(a);
}
template <int K>
static void route_lanes_launch(const RouteArgs& a, hipStream_t stream) {
  if (a.dtype == 0) route_lanes_launch<K, 0>(a, stream);
  else if (a.dtype == 1) route_lanes_launch<K, 1>(a, stream);
  else route_lanes_launch<K, 2>(a, stream);
}

template <int EL>
static void route_select_launch(const RouteArgs& a, hipStream_t stream) {
  if (a.blocks == 1) route_select_kernel<EL, true><<<1, kRouteThreads, 0, stream>>>(a);
  else route_select_kernel<EL, false><<<(unsigned)a.blocks, kRouteThreads, 0, stream>>>(a);
}

hipError_t launch_moe_route(const void* logits, int dtype, int64_t rows, int n_experts, int64_t ld, int top,
                            bool renorm, float scale, int32_t* experts, float* weights, int32_t* rows_out,
                            int32_t* places, int32_t* offsets, void* ws, hipStream_t stream) {
  const RouteArgs a = {logits, dtype, ld, rows, n_experts, top, renorm, scale, experts, weights, rows_out, places,
                       offsets, (uint16_t*)ws, (n_experts + 7) / 8 * 8, route_per(rows), (int)route_blocks(rows)};
  if (n_experts <= kLaneExperts && top <= 8) {
    if (top > 4) route_lanes_launch<8>(a, stream);
    else if (top > 2) route_lanes_launch<4>(a, stream);
    else route_lanes_launch<2>(a, stream);
  } else if (n_experts <= 64) {
    route_select_launch<1>(a, stream);
  } else if (n_experts <= 128) {
    route_select_launch<2>(a, stream);
  } else if (n_experts <= 256) {
    route_select_launch<4>(a, stream);
  } else if (n_experts <= 512) {
    route_select_launch<8>(a, stream);
  } else {
    route_select_launch<16>(a, stream);
  }
  if (a.blocks > 1) route_place_kernel<<<(unsigned)a.blocks, kRouteThreads, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace awq
