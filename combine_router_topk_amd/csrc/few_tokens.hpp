// Routing of at most 64 tokens inside the layer of a few tokens: each token's
// top-k and gate weights, and what the chosen experts are made of.
#pragma once

#include "device.hpp"

namespace moe {

namespace {

constexpr int kMaxTokens = 64;
constexpr int kMaxPairs = kMaxTokens * kMaxK;
constexpr int kRowsPerTile = 16;
constexpr int kFewPairs = 224;  // (token, slot) pairs that every block of the first launch finds by itself
constexpr int kRouteThreads = 1024;

struct RouteArgs {
  const float* logits;
  int T, E, k;
  int32_t* idx;
  float* w;
  int4* item;      // tables in the workspace, of more than kFewPairs pairs
  int32_t* order;
  int32_t* head;   // the items, and the next tile that nobody has taken
};

// The k best experts of one token, by one wave: slot j's expert and logit key
// end in lane j. Lane l holds experts l V .. l V + V - 1, so among equal keys
// the lowest expert sits in the lowest lane, at that lane's lowest slot.
template <int V>
__device__ __forceinline__ void topk_wave(const float* __restrict__ row, int E, int k, int lane, int& my_e,
                                          uint32_t& my_key, uint32_t& top_key) {
  uint32_t key[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = lane * V + v;
    key[v] = e < E ? logit_key(row[e]) : 0u;
  }
  my_e = 0;
  my_key = top_key = 0u;
  for (int j = 0; j < k; ++j) {
    uint32_t lm = key[0];
#pragma unroll
    for (int v = 1; v < V; ++v) lm = umax(lm, key[v]);
    const uint32_t best = wave_max_u32(lm);
    const int l = __builtin_ctzll(ballot(lm == best));
    int fv = V - 1;
#pragma unroll
    for (int v = V - 2; v >= 0; --v) fv = key[v] == best ? v : fv;
    const int fvs = __builtin_amdgcn_readlane(fv, l);
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (v == fvs) key[v] = lane == l ? 0u : key[v];
    if (lane == j) {
      my_e = l * V + fvs;
      my_key = best;
    }
    if (j == 0) top_key = best;
  }
}

// One token's top-k by one wave, its experts to idx[]; to memory with the gate
// weights, a softmax over the chosen logits in fp64, if `write`.
template <int V>
__device__ __forceinline__ void route_token(const RouteArgs& g, int t, int lane, int* idx, bool write) {
  int e;
  uint32_t key, top;
  topk_wave<V>(g.logits + static_cast<size_t>(t) * g.E, g.E, g.k, lane, e, key, top);
  if (lane < g.k) idx[t * g.k + lane] = e;
  if (write) {
    double ex = 0.0;
    if (lane < g.k) ex = exp(static_cast<double>(key_logit(key)) - static_cast<double>(key_logit(top)));
    const double sum = group_sum16_f64<kWave>(ex);
    if (lane < g.k) {
      g.idx[t * g.k + lane] = e;
      g.w[t * g.k + lane] = static_cast<float>(ex / sum);
    }
  }
}

// What the chosen experts are made of: pairs (token, slot) by expert, then by
// token, and items of at most 16 of one expert's: (expert, first place, pairs).
// An expert's tokens are a mask of 64 bits, so a pair's place is a count of bits.
struct Tables {
  int4* item;      // [pairs]
  int* order;      // [pairs]
  int* idx;        // [pairs]
  int* offset;     // [E]
  uint32_t* mask;  // [2 E]
  static size_t bytes(int pairs, int E) { return pairs * (sizeof(int4) + 2 * sizeof(int)) + 3 * E * sizeof(int); }
  __device__ __forceinline__ Tables(void* lds, int pairs, int E) {
    item = static_cast<int4*>(lds);
    order = reinterpret_cast<int*>(item + pairs);
    idx = order + pairs;
    offset = idx + pairs;
    mask = reinterpret_cast<uint32_t*>(offset + E);
  }
};

template <int NT>
__device__ __forceinline__ void build_tables(const RouteArgs& g, const Tables& sh, int* items) {
  const int tid = threadIdx.x, lane = tid & 63, pairs = g.T * g.k;
  for (int e = tid; e < 2 * g.E; e += NT) sh.mask[e] = 0;
  __syncthreads();  // the experts of every token, too
  for (int p = tid; p < pairs; p += NT) {
    const int t = p / g.k;
    atomicOr(&sh.mask[2 * sh.idx[p] + (t >> 5)], 1u << (t & 31));
  }
  __syncthreads();
  if (tid < kWave) {
    int off = 0, it = 0;
    for (int e0 = 0; e0 < g.E; e0 += kWave) {
      const int e = e0 + lane;
      const int c = e < g.E ? __builtin_popcount(sh.mask[2 * e]) + __builtin_popcount(sh.mask[2 * e + 1]) : 0;
      const int n = (c + kRowsPerTile - 1) / kRowsPerTile;
      const int o = off + wave_incl_scan(c, lane) - c;
      const int i0 = it + wave_incl_scan(n, lane) - n;
      if (e < g.E) sh.offset[e] = o;
      for (int i = 0; i < n; ++i)
        sh.item[i0 + i] = make_int4(e, o + i * kRowsPerTile, min(kRowsPerTile, c - i * kRowsPerTile), 0);
      off = __builtin_amdgcn_readlane(o + c, kWave - 1);
      it = __builtin_amdgcn_readlane(i0 + n, kWave - 1);
    }
    if (lane == 0) *items = it;
  }
  __syncthreads();
  for (int p = tid; p < pairs; p += NT) {
    const int e = sh.idx[p], t = p / g.k;
    const uint32_t lo = sh.mask[2 * e], hi = sh.mask[2 * e + 1], below = (1u << (t & 31)) - 1;
    const int rank = t < 32 ? __builtin_popcount(lo & below) : __builtin_popcount(lo) + __builtin_popcount(hi & below);
    sh.order[sh.offset[e] + rank] = p;
  }
  __syncthreads();
}

// More than kFewPairs pairs are found by one block, in a launch of its own.
template <int V>
__global__ __launch_bounds__(kRouteThreads) void layer_route_kernel(RouteArgs g) {
  __shared__ int items;
  extern __shared__ __align__(16) char tables[];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int pairs = g.T * g.k;
  const Tables sh(tables, pairs, g.E);
  for (int t = wave; t < g.T; t += kRouteThreads / kWave) route_token<V>(g, t, lane, sh.idx, true);
  build_tables<kRouteThreads>(g, sh, &items);
  for (int i = tid; i < items; i += kRouteThreads) g.item[i] = sh.item[i];
  for (int p = tid; p < pairs; p += kRouteThreads) g.order[p] = sh.order[p];
  if (tid == 0) {
    g.head[0] = items;
    g.head[1] = 0;
  }
}

}  // namespace

}  // namespace moe
