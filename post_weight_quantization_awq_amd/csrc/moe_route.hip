// Routing of tokens to experts: each token's k largest logits, their shares, and
// the (token, expert) pairs in expert order, as the grouped product takes them.
//
// A wave takes a token: its lanes hold the logits as unsigned keys that order as
// the values do, and k rounds of a wave maximum pick the experts.  A token has an
// expert at most once, so 64 tokens are a 64-bit mask for each expert in LDS: a
// pair's rank among its expert's is the number of set bits below its token's, the
// same in whatever order the bits were set.  Up to 64 tokens (a decoding step) one
// block does it all; more take two launches, the second of which adds the counts
// that the first left for each block.
//
// Bound by latency, not by the logits' bytes.
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

// More tokens: 4 lanes take a token, each a fourth of its logits, and keep the best K of them in order by insertion
// (a maximum and a minimum for each place); two merges across the lanes join them.  A logit and its expert are one
// positive double that orders as they do: 32 bits of key, then the experts from the last to the first.  62 operations
// a token of 128 experts and 8 places, where a wave for each token takes 300.
constexpr int kLaneThreads = 4 * kRouteChunk, kLaneExperts = 256;
__device__ __forceinline__ double route_pack(uint32_t key, uint32_t e) {
  return __builtin_bit_cast(double, (uint64_t)key << 30 | (0x3FFFFFFFu - e));
}
__device__ __forceinline__ uint32_t packed_key(double d) { return (uint32_t)(__builtin_bit_cast(uint64_t, d) >> 30); }
__device__ __forceinline__ int packed_expert(double d) {
  return (int)(0x3FFFFFFFu - ((uint32_t)__builtin_bit_cast(uint64_t, d) & 0x3FFFFFFFu));
}
template <int CTRL>
__device__ __forceinline__ double dpp_d(double d) {
  const uint64_t u = __builtin_bit_cast(uint64_t, d);
  return __builtin_bit_cast(double, (uint64_t)dpp_u<CTRL>((uint32_t)(u >> 32)) << 32 | dpp_u<CTRL>((uint32_t)u));
}
__device__ __forceinline__ void order(double& a, double& b) {  // a the larger
  const double m = __builtin_fmax(a, b);
  b = __builtin_fmin(a, b);
  a = m;
}
// The best K of the lane's and another lane's lists, in order
template <int K, int CTRL>
__device__ __forceinline__ void merge_lists(double (&v)[K]) {
  double o[K];
#pragma unroll
  for (int i = 0; i < K; ++i) o[i] = dpp_d<CTRL>(v[K - 1 - i]);
#pragma unroll
  for (int i = 0; i < K; ++i) v[i] = __builtin_fmax(v[i], o[i]);  // falls, then rises, or the other way round
#pragma unroll
  for (int d = K / 2; d >= 1; d /= 2)
#pragma unroll
    for (int i = 0; i < K; ++i)
      if ((i & d) == 0) order(v[i], v[i + d]);
}

// The lane's 4 logits of 16 from e on; -inf for those that are not there
template <int DT>
__device__ __forceinline__ void load_logits4(const RouteArgs& a, int64_t at, int e, float (&f)[4]) {
  if (e + 4 <= a.n_experts) {
    if constexpr (DT == 2) {
      *(float4*)f = ld_any<float4>((const float*)a.logits + at + e);
    } else {
      const uint2 u = ld_any<uint2>((const uint16_t*)a.logits + at + e);
      f[0] = x2f<DT>(u.x & 0xFFFFu), f[1] = x2f<DT>(u.x >> 16), f[2] = x2f<DT>(u.y & 0xFFFFu), f[3] = x2f<DT>(u.y >> 16);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = e + i < a.n_experts ? route_logit(a.logits, DT, at + e + i) : -INFINITY;
  }
}

template <int K, int DT>
__global__ __launch_bounds__(kLaneThreads) void route_lanes_kernel(const RouteArgs a) {
  __shared__ unsigned long long mask[kLaneExperts];
  const int tid = threadIdx.x, q = tid % 4, tt = tid / 4;
  const int64_t t0 = (int64_t)blockIdx.x * a.per;
  uint32_t count = 0;  // of expert `tid`
  for (int c = 0; c < a.per && t0 + c < a.rows; c += kRouteChunk) {
    mask[tid] = 0;
    __syncthreads();
    const int64_t t = t0 + c + tt;
    const bool live = t < a.rows;
    const int64_t at = (live ? t : a.rows - 1) * a.ld;
    double v[K];
#pragma unroll
    for (int i = 0; i < K; ++i) v[i] = 0.0;
#pragma unroll 2
    for (int e = 4 * q; e < a.n_experts; e += 16) {
      float f[4];
      load_logits4<DT>(a, at, e, f);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t key = route_key(f[i]);
        double x = key != 0 ? route_pack(key, (uint32_t)(e + i)) : 0.0;
#pragma unroll
        for (int s = 0; s < K; ++s) order(v[s], x);
      }
    }
    merge_lists<K, 0xB1>(v);
    merge_lists<K, 0x4E>(v);
    const float most = route_value(packed_key(v[0]));
    float sum = 0.0f;
    if (!a.renorm && v[0] != 0.0) {
#pragma unroll 2
      for (int e = 4 * q; e < a.n_experts; e += 16) {
        float f[4];
        load_logits4<DT>(a, at, e, f);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (route_key(f[i]) != 0) sum += expf(f[i] - most);
      }
    }
    // the lane's places: q, q + 4
    constexpr int PL = (K + 3) / 4;
    int id[PL];
    float p[PL];
#pragma unroll
    for (int i = 0; i < PL; ++i) {
      double d = 0.0;
#pragma unroll
      for (int s = 0; s < 4; ++s)
        if (4 * i + s < K) d = q == s ? v[4 * i + s] : d;
      const bool some = d != 0.0 && 4 * i + q < a.top;
      id[i] = some ? packed_expert(d) : -1;
      p[i] = some ? expf(route_value(packed_key(d)) - most) : 0.0f;
      if (a.renorm) sum += p[i];
    }
    sum += dpp_m<0xB1>(sum);
    sum += dpp_m<0x4E>(sum);
#pragma unroll
    for (int i = 0; i < PL; ++i)
      if (live && 4 * i + q < a.top) {
        a.experts[t * a.top + 4 * i + q] = id[i];
        a.weights[t * a.top + 4 * i + q] = id[i] >= 0 ? p[i] / sum * a.scale : 0.0f;
        if (id[i] >= 0) atomicOr(&mask[id[i]], 1ull << tt);
      }
    __syncthreads();
    count += __popcll(mask[tid]);
    __syncthreads();  // the masks are cleared for the next chunk
  }
  if (tid < a.ld_counts) a.counts[(int64_t)blockIdx.x * a.ld_counts + tid] = (uint16_t)count;
}

// Places of a block's pairs: the experts' totals and what lies in the blocks before, from the counts of all blocks,
// 8 experts a thread.
__global__ __launch_bounds__(kRouteThreads) void route_place_kernel(const RouteArgs a) {
  __shared__ unsigned long long mask[1024];
  __shared__ uint32_t base[1024], total[1024], part[kRouteWaves];
  const int tid = threadIdx.x;
  base[tid] = total[tid] = 0;
  mask[tid] = 0;
  __syncthreads();
  const int lanes = a.ld_counts / 8, step = kRouteThreads / lanes;
  const int col = tid % lanes, seg = tid / lanes;
  if (seg < step) {
    uint32_t all[8] = {}, before[8] = {};
    for (int b = seg; b < a.blocks; b += step) {
      const uint4 u = *(const uint4*)(a.counts + (int64_t)b * a.ld_counts + 8 * col);
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t n = i % 2 ? w[i / 2] >> 16 : w[i / 2] & 0xFFFFu;
        all[i] += n;
        before[i] += b < (int)blockIdx.x ? n : 0;
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (all[i]) atomicAdd(&total[8 * col + i], all[i]);
      if (before[i]) atomicAdd(&base[8 * col + i], before[i]);
    }
  }
  __syncthreads();
  uint32_t sum;
  const uint32_t first = block_scan(total[tid], part, &sum);
  base[tid] += first;
  if (blockIdx.x == 0) {
    if (tid < a.n_experts) a.offsets[tid] = (int)first;
    if (tid == 0) a.offsets[a.n_experts] = (int)sum;
  }
  const int64_t t0 = (int64_t)blockIdx.x * a.per;
  const int slots = kRouteChunk * a.top;
  for (int c = 0; c < a.per && t0 + c < a.rows; c += kRouteChunk) {
    const int64_t left = a.rows - t0 - c;
    const int n = left < kRouteChunk ? (int)left * a.top : slots;
    const int64_t at = (t0 + c) * a.top;
    int id[2] = {-1, -1};  // of the chunk's pairs tid and tid + 1024: at most 64 x 32
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int s = tid + kRouteThreads * i;
      if (s < n) id[i] = a.experts[at + s];
      if (id[i] >= 0) atomicOr(&mask[id[i]], 1ull << (s / a.top));
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int s = tid + kRouteThreads * i;
      if (s < n) {
        int place = -1;
        if (id[i] >= 0) {
          place = (int)(base[id[i]] + __popcll(mask[id[i]] & ((1ull << (s / a.top)) - 1)));
          a.rows_out[place] = (int)(t0 + c) + s / a.top;
        }
        a.places[at + s] = place;
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

template <int K>
static void route_lanes_launch(const RouteArgs& a, hipStream_t stream) {
  if (a.dtype == 0) route_lanes_kernel<K, 0><<<(unsigned)a.blocks, kLaneThreads, 0, stream>>>(a);
  else if (a.dtype == 1) route_lanes_kernel<K, 1><<<(unsigned)a.blocks, kLaneThreads, 0, stream>>>(a);
  else route_lanes_kernel<K, 2><<<(unsigned)a.blocks, kLaneThreads, 0, stream>>>(a);
}

template <int EL>
static void route_launch(const RouteArgs& a, hipStream_t stream) {
  if (a.blocks == 1) {
    route_select_kernel<EL, true><<<1, kRouteThreads, 0, stream>>>(a);
    return;
  }
  if (a.n_experts > kLaneExperts || a.top > 8) route_select_kernel<EL, false><<<(unsigned)a.blocks, kRouteThreads, 0, stream>>>(a);
  else if (a.top > 4) route_lanes_launch<8>(a, stream);
  else if (a.top > 2) route_lanes_launch<4>(a, stream);
  else route_lanes_launch<2>(a, stream);
  route_place_kernel<<<(unsigned)a.blocks, kRouteThreads, 0, stream>>>(a);
}

hipError_t launch_moe_route(const void* logits, int dtype, int64_t rows, int n_experts, int64_t ld, int top,
                            bool renorm, float scale, int32_t* experts, float* weights, int32_t* rows_out,
                            int32_t* places, int32_t* offsets, void* ws, hipStream_t stream) {
  const RouteArgs a = {logits, dtype, ld, rows, n_experts, top, renorm, scale, experts, weights, rows_out, places,
                       offsets, (uint16_t*)ws, (n_experts + 7) / 8 * 8, route_per(rows), (int)route_blocks(rows)};
  if (n_experts <= 64) route_launch<1>(a, stream);
  else if (n_experts <= 128) route_launch<2>(a, stream);
  else if (n_experts <= 256) route_launch<4>(a, stream);
  else if (n_experts <= 512) route_launch<8>(a, stream);
  else route_launch<16>(a, stream);
  return hipGetLastError();
}

}  // namespace awq
