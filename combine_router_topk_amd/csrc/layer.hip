// A whole mixture-of-experts layer for at most 64 tokens, in two launches, with
// many pairs of token and expert three (the first then by itself), with large
// weights one more that adds up the down product's shares:
// top-k and gate weights, gate and up products with SwiGLU, then the down
// product with the weighted combine.
//
//   h[t, j] = round16(silu(Wg x[t]) * (Wu x[t])),  (Wg; Wu) = expert idx[t, j]'s
//   out[t]  = round(sum over j of w[t, j] (Wd h[t, j])), summed in fp32
//
// The time is that of reading the chosen experts' weights once: nothing is
// dispatched, rows are read where they are, and the weights go from memory
// to registers in the matrix instruction's layout (16 weight rows as its
// first operand, up to 16 tokens as its second). Activations stay in 16
// bits, as a few rows are not worth rounding to 8; e4m3 weights become 16-bit
// numbers in registers, exactly, and a block's scale is applied to the fp32
// sum of its 128 products. One token of 256 experts, top-8, 4096 x 2048 in
// e4m3: 29.5 us + 14.8 us for 201 MB (4.5 TB/s; starting and ending two launches
// is the rest); 8 tokens of top-2 of 64 in bf16: 91 us + 49 us for 755 MB, 5.4
// TB/s; 32 tokens of top-8 of 256, 7168 x 2048: 772 us + 474 us for 6.8 GB, 5.5
// TB/s, and 15 us for the launches that route and add up.
#include "device.hpp"
#include "launch.hpp"
#include "quant.hpp"

namespace moe {

namespace {

constexpr int kMaxTokens = 64;
constexpr int kMaxPairs = kMaxTokens * kMaxK;
constexpr int kUpThreads = 256, kUpWaves = kUpThreads / kWave;
// At most; five a CU with one step in flight each (one token of 256 experts, top-8,
// 4096 x 2048, e4m3: four blocks of two steps 52.0 us, this 49.5).
constexpr int kUpBlocks = 1280;
constexpr int kRowsPerTile = 16;
constexpr int kFewPairs = 224;  // (token, slot) pairs that every block of the first launch finds by itself
constexpr int kRouteThreads = 1024;

struct LayerArgs {
  const float* logits;
  const void* x;
  const void* w_up;
  const float* s_up;
  const void* w_down;
  const float* s_down;
  int T, E, k, H, I;
  int32_t* idx;
  float* w;
  void* h;
  void* out;
  bool out_f32;
  int4* item;      // tables in the workspace, of more than kFewPairs pairs
  int32_t* order;
  int32_t* head;   // the items, and the next tile that nobody has taken
  float* part;     // [shares][T][H]: sums of the down product's shares
};

// One step of K for a tile of 16 weight rows and 16 tokens: 128 bytes of each
// weight row (128 codes, or 64 values in 16 bits). Lane (r, g) = (lane % 16,
// lane / 16) holds chunk g and chunk 4 + g of row r's eight 16-byte chunks, and
// the same columns of its token; both operands place their columns alike, so
// their order inside the instruction does not matter.
template <int ACT, bool F8>
struct Step {
  static constexpr int kCols = F8 ? 128 : 64;  // columns of K
  static constexpr int kPer = F8 ? 16 : 8;     // columns of a chunk
  static constexpr int kB = F8 ? 2 : 1;        // 16-byte chunks of a token for one of weights
  struct Rows { uint4 v[2]; };
  struct Cols { uint4 v[2 * kB]; };

  // columns lane chunk j starts at
  static __device__ __forceinline__ int col(int kb, int j, int grp) { return kb * kCols + (j * 4 + grp) * kPer; }

  // `row` is the lane's weight row; columns from K on are zeros
  static __device__ __forceinline__ void load_rows(Rows& r, const unsigned char* row, int kb, int grp, int K) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int c = col(kb, j, grp);
      r.v[j] = make_uint4(0, 0, 0, 0);
      if (c < K) r.v[j] = *reinterpret_cast<const uint4*>(row + static_cast<size_t>(c) * (F8 ? 1 : 2));
    }
  }
  // K = 0 for a lane without a token: it loads nothing (with the loads of some
  // other token's row in its place 50 tokens of 16 experts, top-4, 2048 x 1024 took
  // 67 us, not 61)
  static __device__ __forceinline__ void load_cols(Cols& b, const uint16_t* tok, int kb, int grp, int K) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int c = col(kb, j, grp);
#pragma unroll
      for (int i = 0; i < kB; ++i) {
        b.v[j * kB + i] = make_uint4(0, 0, 0, 0);
        if (c < K) b.v[j * kB + i] = *reinterpret_cast<const uint4*>(tok + c + i * 8);
      }
    }
  }
  static __device__ __forceinline__ v4f product(const Rows& r, const Cols& b) {
    v4f p = {0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      if constexpr (F8) {
        const uint2 a0 = widen4<ACT>(r.v[j].x), a1 = widen4<ACT>(r.v[j].y);
        const uint2 a2 = widen4<ACT>(r.v[j].z), a3 = widen4<ACT>(r.v[j].w);
        p = mfma16<ACT>(make_uint4(a0.x, a0.y, a1.x, a1.y), b.v[j * 2], p);
        p = mfma16<ACT>(make_uint4(a2.x, a2.y, a3.x, a3.y), b.v[j * 2 + 1], p);
      } else {
        p = mfma16<ACT>(r.v[j], b.v[j], p);
      }
    }
    return p;
  }
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

// ---- routing -----------------------------------------------------------------

// One token's top-k by one wave, its experts to idx[]; to memory with the gate
// weights, a softmax over the chosen logits in fp64, if `write`.
template <int V>
__device__ __forceinline__ void route_token(const LayerArgs& g, int t, int lane, int* idx, bool write) {
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
__device__ __forceinline__ void build_tables(const LayerArgs& g, const Tables& sh, int* items) {
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
__global__ __launch_bounds__(kRouteThreads) void layer_route_kernel(LayerArgs g) {
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

// ---- launch 1: top-k, gate and up products, SwiGLU ---------------------------

// V > 0: every block routes the tokens itself, 0.08 us a pair, and takes tiles
// in turn. V = 0: the tables are there, which takes a launch of 10 us, and a block
// that is done takes the next tile that nobody has, as blocks' shares of the
// memory's bandwidth differ by half. Which is faster depends on how long the
// launch is beside that; kFewPairs lies between. The whole layer in us, V > 0 and
// V = 0 (rounds of both in turn):
//   pairs                                       32   64   96  128  160  192  224  256
//   top-8 of 256, 4096 x 2048, e4m3    V > 0   149  272  379  490  580  660  726  796
//                                      V = 0   162  279  385  477  573  650  718  782
//   top-4 of 64, 2048 x 1024, 16 bits  V > 0    86  122  150  173  195  205  219  231
//                                      V = 0    97  132  157  179  201  209  223  232
//   top-16 of 128, 2048 x 1024, e4m3   V > 0         89       144       172  184
//                                      V = 0        106       163       188  202
// and with 1024 pairs (64 tokens, top-16 of 128) 576 and 511.
template <int ACT, bool F8, int V>
__global__ __launch_bounds__(kUpThreads, 6) void layer_up_kernel(LayerArgs g) {
  __shared__ float4 part[2][kUpWaves][2][kWave];
  __shared__ int items, next_tile[2];
  extern __shared__ __align__(16) char tables[];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int pairs = g.T * g.k;
  const Tables sh(tables, pairs, V > 0 ? g.E : 0);
  if constexpr (V > 0) {
    for (int t = wave; t < g.T; t += kUpWaves) route_token<V>(g, t, lane, sh.idx, blockIdx.x == 0);
    build_tables<kUpThreads>(g, sh, &items);
  } else {
    if (tid == 0) items = g.head[0];
    for (int i = tid; i < pairs; i += kUpThreads) {  // those past the items are not used
      sh.item[i] = g.item[i];
      sh.order[i] = g.order[i];
    }
    __syncthreads();
  }

  using S = Step<ACT, F8>;
  const int r = lane & 15, grp = lane >> 4;
  const int n_tiles = g.I / kRowsPerTile;
  const int steps = (g.H + S::kCols - 1) / S::kCols;
  const int nbK = scale_blocks(g.H), nbN = scale_blocks(2 * g.I);
  const size_t row_bytes = static_cast<size_t>(g.H) * (F8 ? 1 : 2);
  const int work = items * n_tiles;
  const int blocks = gridDim.x;
  int turn = 0;
  for (int i = blockIdx.x; i < work; turn ^= 1) {
    int next = i + blocks;
    if constexpr (V == 0) {
      if (tid == 0) next = blocks + atomicAdd(&g.head[1], 1);
    }
    const int4 it = sh.item[i / n_tiles];
    const int n0 = (i % n_tiles) * kRowsPerTile;
    const int e = __builtin_amdgcn_readfirstlane(it.x), off = it.y, have = it.z;
    const unsigned char* gate_row = static_cast<const unsigned char*>(g.w_up) +
                                    (static_cast<size_t>(e) * 2 * g.I + n0 + r) * row_bytes;
    const unsigned char* up_row = gate_row + g.I * row_bytes;
    const int my_pair = sh.order[off + min(r, have - 1)];
    const uint16_t* tok = static_cast<const uint16_t*>(g.x) + static_cast<size_t>(my_pair / g.k) * g.H;
    const float* s_gate = g.s_up + (static_cast<size_t>(e) * nbN + n0 / kScaleBlock) * nbK;
    const float* s_upr = g.s_up + (static_cast<size_t>(e) * nbN + (g.I + n0) / kScaleBlock) * nbK;

    v4f gate = {0, 0, 0, 0}, up = {0, 0, 0, 0};
    constexpr int D = F8 ? 1 : 2;  // steps in flight
    for (int kb0 = wave; kb0 < steps; kb0 += kUpWaves * D) {
      typename S::Rows a[D], b[D];
      typename S::Cols c[D];
      float sg[D], su[D];
#pragma unroll
      for (int d = 0; d < D; ++d) {
        const int kb = kb0 + d * kUpWaves;
        S::load_rows(a[d], gate_row, kb, grp, g.H);
        S::load_rows(b[d], up_row, kb, grp, g.H);
        S::load_cols(c[d], tok, kb, grp, r < have ? g.H : 0);
        if constexpr (F8) {
          sg[d] = kb < steps ? s_gate[kb] : 0.0f;
          su[d] = kb < steps ? s_upr[kb] : 0.0f;
        }
      }
#pragma unroll
      for (int d = 0; d < D; ++d) {
        const v4f pg = S::product(a[d], c[d]), pu = S::product(b[d], c[d]);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          if constexpr (F8) {
            gate[q] = fmaf(pg[q], sg[d], gate[q]);
            up[q] = fmaf(pu[q], su[d], up[q]);
          } else {
            gate[q] += pg[q];
            up[q] += pu[q];
          }
        }
      }
    }
    part[turn][wave][0][lane] = make_float4(gate[0], gate[1], gate[2], gate[3]);
    part[turn][wave][1][lane] = make_float4(up[0], up[1], up[2], up[3]);
    if (V == 0 && tid == 0) next_tile[turn] = next;
    __syncthreads();
    i = V == 0 ? __builtin_amdgcn_readfirstlane(next_tile[turn]) : next;
    // thread tid sums value tid % 4 of lane tid / 4
    const int c = (tid >> 2) & 15, n = (tid >> 6) * 4 + (tid & 3);
    float zg = 0.0f, zu = 0.0f;
#pragma unroll
    for (int wv = 0; wv < kUpWaves; ++wv) {
      zg += reinterpret_cast<const float*>(part[turn][wv][0])[tid];
      zu += reinterpret_cast<const float*>(part[turn][wv][1])[tid];
    }
    if (c < have) {
      const float h = silu(zg) * zu;
      static_cast<uint16_t*>(g.h)[static_cast<size_t>(sh.order[off + c]) * g.I + n0 + n] =
          static_cast<uint16_t>(pack2<ACT>(h, 0.0f));
    }
  }
}

// ---- launch 2: down product and weighted combine ------------------------------

template <int TT, int NT>
struct DownShared {
  int idx[kMaxPairs];
  float w[kMaxPairs];
  int flag[kMaxE];
  int active[kMaxPairs];
  int n_active;
  float4 part[NT / kWave][TT][kWave];
};

// Each block owns 16 columns of the output for every token (TT groups of 16
// tokens: column c of a group's instruction is token c), its waves contiguous
// parts of the (expert, step of K) sequence. With several shares blockIdx.y is the
// share of the sequence, and layer_sum_kernel adds them up.
template <int ACT, bool F8, int TT, int NT>
__global__ __launch_bounds__(NT, 4) void layer_down_kernel(LayerArgs g) {
  constexpr int kThreads = NT, kWaves = NT / kWave;
  __shared__ DownShared<TT, NT> sh;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int pairs = g.T * g.k;
  for (int e = tid; e < g.E; e += kThreads) sh.flag[e] = 0;
  __syncthreads();
  for (int p = tid; p < pairs; p += kThreads) {
    const int e = min(max(g.idx[p], 0), g.E - 1);
    sh.idx[p] = e;
    sh.w[p] = g.w[p];
    sh.flag[e] = 1;
  }
  __syncthreads();
  if (wave == 0) {
    int n = 0;
    for (int e0 = 0; e0 < g.E; e0 += kWave) {
      const int e = e0 + lane;
      const bool on = e < g.E && sh.flag[e] != 0;
      const uint64_t m = ballot(on);
      if (on) sh.active[n + __builtin_popcountll(m & lanemask_lt(lane))] = e;
      n += __builtin_popcountll(m);
    }
    if (lane == 0) sh.n_active = n;
  }
  __syncthreads();

  using S = Step<ACT, F8>;
  const int r = lane & 15, grp = lane >> 4;
  const int n0 = blockIdx.x * kRowsPerTile;
  const int steps = (g.I + S::kCols - 1) / S::kCols;
  const int nbK = scale_blocks(g.I), nbN = scale_blocks(g.H);
  const size_t row_bytes = static_cast<size_t>(g.I) * (F8 ? 1 : 2);
  const int shares = gridDim.y, share = blockIdx.y;
  const int all = sh.n_active * steps;
  const int total = all / shares + (share < all % shares ? 1 : 0);
  int q = all / shares * share + min(share, all % shares) + total / kWaves * wave + min(wave, total % kWaves);
  const int q_end = q + total / kWaves + (wave < total % kWaves ? 1 : 0);

  v4f acc[TT];
#pragma unroll
  for (int u = 0; u < TT; ++u) acc[u] = v4f{0, 0, 0, 0};
  while (q < q_end) {
    const int ei = q / steps, k0 = q % steps, k1 = min(steps, k0 + q_end - q);
    q += k1 - k0;
    const int e = __builtin_amdgcn_readfirstlane(sh.active[ei]);
    const unsigned char* row = static_cast<const unsigned char*>(g.w_down) +
                               (static_cast<size_t>(e) * g.H + n0 + r) * row_bytes;
    const float* s_row = g.s_down + (static_cast<size_t>(e) * nbN + n0 / kScaleBlock) * nbK;
    const uint16_t* tok[TT];
    float wt[TT];
    bool on[TT], any[TT];
#pragma unroll
    for (int u = 0; u < TT; ++u) {
      const int t = u * kRowsPerTile + r;
      int pair = -1;
      if (t < g.T)
        for (int j = 0; j < g.k; ++j)
          if (sh.idx[t * g.k + j] == e) pair = t * g.k + j;
      on[u] = pair >= 0;
      any[u] = ballot(on[u]) != 0;
      wt[u] = on[u] ? sh.w[pair] : 0.0f;
      tok[u] = static_cast<const uint16_t*>(g.h) + static_cast<size_t>(on[u] ? pair : 0) * g.I;
    }
    constexpr int D = 2;  // steps in flight
    for (int kb0 = k0; kb0 < k1; kb0 += D) {
      typename S::Rows a[D];
      float s[D];
#pragma unroll
      for (int d = 0; d < D; ++d) {
        const int kb = kb0 + d;
        S::load_rows(a[d], row, kb, grp, kb < k1 ? g.I : 0);
        if constexpr (F8) s[d] = s_row[min(kb, nbK - 1)];
        else s[d] = 1.0f;
      }
#pragma unroll
      for (int u = 0; u < TT; ++u) {
        if (!any[u]) continue;
        typename S::Cols c[D];
#pragma unroll
        for (int d = 0; d < D; ++d) S::load_cols(c[d], tok[u], kb0 + d, grp, on[u] && kb0 + d < k1 ? g.I : 0);
#pragma unroll
        for (int d = 0; d < D; ++d) {
          const v4f p = S::product(a[d], c[d]);
          const float f = s[d] * wt[u];
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[u][i] = on[u] && kb0 + d < k1 ? fmaf(p[i], f, acc[u][i]) : acc[u][i];
        }
      }
    }
  }
#pragma unroll
  for (int u = 0; u < TT; ++u)
    sh.part[wave][u][lane] = make_float4(acc[u][0], acc[u][1], acc[u][2], acc[u][3]);
  __syncthreads();
  for (int o = tid; o < TT * 256; o += kThreads) {
    const int u = o >> 8, v = o & 255;
    const int t = u * kRowsPerTile + ((v >> 2) & 15), n = n0 + (v >> 6) * 4 + (v & 3);
    float z = 0.0f;
#pragma unroll
    for (int wv = 0; wv < kWaves; ++wv) z += reinterpret_cast<const float*>(sh.part[wv][u])[v];
    if (t < g.T) {
      const size_t at = static_cast<size_t>(t) * g.H + n;
      if (shares > 1) g.part[static_cast<size_t>(share) * g.T * g.H + at] = z;
      else if (g.out_f32) static_cast<float*>(g.out)[at] = z;
      else static_cast<uint16_t*>(g.out)[at] = static_cast<uint16_t>(pack2<ACT>(z, 0.0f));
    }
  }
}

template <int ACT>
__global__ __launch_bounds__(256) void layer_sum_kernel(LayerArgs g, int shares) {
  const int n = g.T * g.H / 4, i = blockIdx.x * 256 + threadIdx.x;
  if (i >= n) return;
  const float4* part = reinterpret_cast<const float4*>(g.part);
  float4 z = part[i];
  for (int y = 1; y < shares; ++y) {
    const float4 v = part[static_cast<size_t>(y) * n + i];
    z = make_float4(z.x + v.x, z.y + v.y, z.z + v.z, z.w + v.w);
  }
  if (g.out_f32) static_cast<float4*>(g.out)[i] = z;
  else static_cast<uint2*>(g.out)[i] = make_uint2(pack2<ACT>(z.x, z.y), pack2<ACT>(z.z, z.w));
}

// Shares of the down product: with a block a tile and, say, 448 tiles, a CU has
// one block or two, and blocks end at different times. Four blocks a tile come
// one after the other where there is room, which pays for the launch that adds
// them up. The whole layer in us without and with shares, top-8 of 256 experts,
// I = 2048, e4m3 (16 tokens; 8 tokens, 2^29 weights and more at each width):
//   columns   4096       4112       5120       6144       7168       8192
//   tiles     256        257        320        384        448        512
//   16        478 489    632 528    716 613    782 712    852 813    917 912
//   8         267 273    354 296    401 344    439 391    476 454    509 509
// Whole rounds of 256 tiles gain nothing. The bound on the weights is wider than it
// has to be: 2 tokens (2^27 weights) gain at 4112 to 6144 columns, too (108 and
// 95 us at 4112), and 4 us of 146 at 7168.
constexpr int kShares = 4;
bool in_shares(int T, int E, int k, int H, int I) {
  const int tiles = H / kRowsPerTile;
  const long long experts = T * k < E ? T * k : E;
  return tiles > 256 && tiles % 256 != 0 && experts * H * I >= 1ll << 29;
}

template <int ACT, bool F8>
hipError_t launch(const LayerArgs& g, hipStream_t s) {
  const int items = (g.T * g.k < g.E * ((g.T + 15) / 16) ? g.T * g.k : g.E * ((g.T + 15) / 16)) * (g.I / kRowsPerTile);
  const int blocks = items < kUpBlocks ? items : kUpBlocks;
  const size_t lds = Tables::bytes(g.T * g.k, g.E);
  if (g.T * g.k <= kFewPairs) {
    if (g.E <= 64) layer_up_kernel<ACT, F8, 1><<<blocks, kUpThreads, lds, s>>>(g);
    else if (g.E <= 256) layer_up_kernel<ACT, F8, 4><<<blocks, kUpThreads, lds, s>>>(g);
    else layer_up_kernel<ACT, F8, 16><<<blocks, kUpThreads, lds, s>>>(g);
  } else {
    if (g.E <= 64) layer_route_kernel<1><<<1, kRouteThreads, lds, s>>>(g);
    else if (g.E <= 256) layer_route_kernel<4><<<1, kRouteThreads, lds, s>>>(g);
    else layer_route_kernel<16><<<1, kRouteThreads, lds, s>>>(g);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
    layer_up_kernel<ACT, F8, 0><<<blocks, kUpThreads, Tables::bytes(g.T * g.k, 0), s>>>(g);
  }
  const hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  const int tiles = g.H / kRowsPerTile;
  // With fewer blocks than CUs a block has 16 waves (24 tokens of 64 experts,
  // top-4, 2048 x 1024 in 16 bits: 162 us with 8, 151 us), else 8 (one token of
  // 4096 x 2048 in e4m3: 50.9 us with 16, 49.4 us).
  const int shares = in_shares(g.T, g.E, g.k, g.H, g.I) ? kShares : 1;
  auto down = [&](auto TT) {
    if (tiles < 256) layer_down_kernel<ACT, F8, TT, 1024><<<tiles, 1024, 0, s>>>(g);
    else layer_down_kernel<ACT, F8, TT, 512><<<dim3(tiles, shares), 512, 0, s>>>(g);
  };
  if (g.T <= 16) down(std::integral_constant<int, 1>{});
  else if (g.T <= 32) down(std::integral_constant<int, 2>{});
  else down(std::integral_constant<int, 4>{});
  if (shares == 1) return hipGetLastError();
  const hipError_t down_err = hipGetLastError();
  if (down_err != hipSuccess) return down_err;
  layer_sum_kernel<ACT><<<(g.T * g.H / 4 + 255) / 256, 256, 0, s>>>(g, shares);
  return hipGetLastError();
}

}  // namespace

// The inner rows, the tables, the shares' sums.
static size_t whole(size_t bytes) { return (bytes + 255) / 256 * 256; }
static size_t inner_bytes(int T, int k, int I) { return whole(static_cast<size_t>(T) * k * I * 2); }
static size_t table_bytes(int T, int k) {
  return whole(static_cast<size_t>(T) * k * (sizeof(int4) + sizeof(int32_t)) + 2 * sizeof(int32_t));
}

size_t layer_ws_bytes(int T, int E, int k, int H, int I) {
  const size_t sums = in_shares(T, E, k, H, I) ? whole(static_cast<size_t>(kShares) * T * H * sizeof(float)) : 0;
  return inner_bytes(T, k, I) + table_bytes(T, k) + sums;
}

hipError_t launch_layer_few_tokens(const float* logits, const void* x, const void* w_up, const float* s_up,
                                   const void* w_down, const float* s_down, int T, int E, int k, int H, int I,
                                   int32_t* idx, float* w, void* out, void* ws, int act, bool out_f32,
                                   hipStream_t s) {
  char* tables = static_cast<char*>(ws) + inner_bytes(T, k, I);
  int4* item = reinterpret_cast<int4*>(tables);
  int32_t* order = reinterpret_cast<int32_t*>(item + T * k);
  float* part = reinterpret_cast<float*>(tables + table_bytes(T, k));
  LayerArgs g{logits, x, w_up, s_up, w_down, s_down, T, E, k, H, I, idx, w, ws, out, out_f32, item, order, order + T * k, part};
  if (act == 1) return s_up ? launch<1, true>(g, s) : launch<1, false>(g, s);
  return s_up ? launch<2, true>(g, s) : launch<2, false>(g, s);
}

}  // namespace moe
