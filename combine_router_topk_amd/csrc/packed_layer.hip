// A whole mixture-of-experts layer for at most 64 tokens with weights in 4 bits
// (packed.hpp), in the launches of the layer in layer.hip:
//
//   h[t, j] = round16(silu(Wg x[t]) * (Wu x[t])),  (Wg; Wu) = expert idx[t, j]'s
//   out[t]  = round(sum over j of w[t, j] (Wd h[t, j])), summed in fp32
//
// The tokens are the matrix instruction's first operand here and the weight rows
// its second, so that a lane's results belong to one weight row and take one
// scale.
//
// The weights' bytes bound it: 32 tokens of 256 experts, 7168 x 2048, read 4.0 GB and
// take 746 to 777 us, 5.2 to 5.4 TB/s where a large copy reaches 4.85. A few tokens are bound by two
// dependent launches instead: one token of 256 experts, 4096 x 2048, top-8, 102 MB,
// takes 30 us, 17 for the first and 10 to 12 for the second. (The down product needs
// all of h; a grid that waits inside one launch would need every block to be there at
// once.)
#include "device.hpp"
#include "few_tokens.hpp"
#include "launch.hpp"
#include "packed.hpp"
#include "quant.hpp"

namespace moe {

namespace {

constexpr int kUpThreads = 256, kUpWaves = kUpThreads / kWave;
constexpr int kUpBlocks = 1280;
// Pairs of tiles from which on a block takes two at a time, which share the loads of the
// tokens' rows: 32 tokens of 256 experts, 7168 x 2048, 795 us one at a time and 747 so.
// Below, each block of the grid has no more than four turns, and half of them as long
// leave more of the CUs idle at the end.
constexpr int kManyTiles = 4 * kUpBlocks;

struct PackedArgs : RouteArgs {
  const void* x;
  const unsigned char* w_up;
  const unsigned char* w_down;
  int H, I, scale_act;
  void* h;
  void* out;
  bool out_f32;
  float* part;  // [shares][T][H]: sums of the down product's shares
};

__device__ __forceinline__ void route_any(const RouteArgs& g, int t, int lane, int* idx, bool write) {
  if (g.E <= 64) route_token<1>(g, t, lane, idx, write);
  else if (g.E <= 256) route_token<4>(g, t, lane, idx, write);
  else route_token<16>(g, t, lane, idx, write);
}

__global__ __launch_bounds__(kRouteThreads) void packed_route_kernel(RouteArgs g) {
  __shared__ int items;
  extern __shared__ __align__(16) char tables[];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int pairs = g.T * g.k;
  const Tables sh(tables, pairs, g.E);
  for (int t = wave; t < g.T; t += kRouteThreads / kWave) route_any(g, t, lane, sh.idx, true);
  build_tables<kRouteThreads>(g, sh, &items);
  for (int i = tid; i < items; i += kRouteThreads) g.item[i] = sh.item[i];
  for (int p = tid; p < pairs; p += kRouteThreads) g.order[p] = sh.order[p];
  if (tid == 0) {
    g.head[0] = items;
    g.head[1] = 0;
  }
}

// ---- gate and up products, SwiGLU ----------------------------------------------

// ROUTES: every block routes the tokens itself and takes tiles in turn; else the
// tables are there, and a block that is done takes the next tile that nobody has. A
// block has PAIRS tiles of the gate's weight rows and the up's beside them at a time.
template <int ACT, int CODES, int PER, bool ROUTES, int PAIRS>
__global__ __launch_bounds__(kUpThreads, PAIRS == 1 ? 5 : 4) void packed_up_kernel(PackedArgs g) {
  __shared__ float4 part[2][kUpWaves][2 * PAIRS][kWave];
  __shared__ int items, next_tile[2];
  extern __shared__ __align__(16) char tables[];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int pairs = g.T * g.k;
  const Tables sh(tables, pairs, ROUTES ? g.E : 0);
  if constexpr (ROUTES) {
    for (int t = wave; t < g.T; t += kUpWaves) route_any(g, t, lane, sh.idx, blockIdx.x == 0);
    build_tables<kUpThreads>(g, sh, &items);
    if (blockIdx.x == 0) {  // for the down product
      for (int i = tid; i < pairs; i += kUpThreads) {
        if (i < items) g.item[i] = sh.item[i];
        g.order[i] = sh.order[i];
      }
      if (tid == 0) g.head[0] = items;
    }
  } else {
    if (tid == 0) items = g.head[0];
    for (int i = tid; i < pairs; i += kUpThreads) {  // those past the items are not used
      sh.item[i] = g.item[i];
      sh.order[i] = g.order[i];
    }
    __syncthreads();
  }

  constexpr int TB = packed_tile_bytes(PER);
  const int r = lane & 15, grp = lane >> 4;
  const int gate_tiles = g.I / kPackedRows, n_tiles = (gate_tiles + PAIRS - 1) / PAIRS, steps = packed_col_tiles(g.H);
  const int work = items * n_tiles, blocks = gridDim.x;
  const size_t strip = static_cast<size_t>(steps) * TB;  // a row of tiles
  int turn = 0;
  for (int i = blockIdx.x; i < work; turn ^= 1) {
    int next = i + blocks;
    if constexpr (!ROUTES) {
      if (tid == 0) next = blocks + atomicAdd(&g.head[1], 1);
    }
    const int4 it = sh.item[i / n_tiles];
    const int tile = i % n_tiles * PAIRS;
    const int e = __builtin_amdgcn_readfirstlane(it.x), off = it.y, have = it.z;
    const unsigned char* gate_row = g.w_up + (static_cast<size_t>(e) * 2 * gate_tiles + tile) * strip;
    const unsigned char* up_row = gate_row + gate_tiles * strip;
    const size_t beside = tile + 1 < gate_tiles ? strip : 0;  // of two pairs the second's
    const int my_pair = sh.order[off + min(r, have - 1)];
    const uint16_t* tok = static_cast<const uint16_t*>(g.x) + static_cast<size_t>(my_pair / g.k) * g.H;
    const int cols = r < have ? g.H : 0;

    v4f sum[2 * PAIRS];  // gate and up of each pair
#pragma unroll
    for (int n = 0; n < 2 * PAIRS; ++n) sum[n] = v4f{0, 0, 0, 0};
    for (int kb = wave; kb < steps; kb += kUpWaves) {
      PackedTile<PER> a[2 * PAIRS];
      PackedRows c;
      const size_t at = static_cast<size_t>(kb) * TB;
#pragma unroll
      for (int n = 0; n < PAIRS; ++n) {
        a[2 * n].load(gate_row + n * beside + at, lane);
        a[2 * n + 1].load(up_row + n * beside + at, lane);
      }
      c.load(tok, kb, grp, cols);
      v4f start[PER];
      packed_start<ACT, CODES, PER>(c, start);
#pragma unroll
      for (int n = 0; n < 2 * PAIRS; ++n) {
        float s[PER];
        a[n].scales(g.scale_act, s);
        packed_product<ACT, CODES, PER>(c, a[n], s, start, sum[n]);
      }
    }
#pragma unroll
    for (int n = 0; n < 2 * PAIRS; ++n)
      part[turn][wave][n][lane] = make_float4(sum[n][0], sum[n][1], sum[n][2], sum[n][3]);
    if (!ROUTES && tid == 0) next_tile[turn] = next;
    __syncthreads();
    i = ROUTES ? next : __builtin_amdgcn_readfirstlane(next_tile[turn]);
    // thread tid sums value tid % 4 of lane tid / 4: token 4 (tid / 64) + tid % 4 of
    // the item, weight row (tid / 4) % 16 of the tile
    const int c = (tid >> 6) * 4 + (tid & 3);
#pragma unroll
    for (int p = 0; p < PAIRS; ++p) {
      const int n = (tile + p) * kPackedRows + ((tid >> 2) & 15);
      float zg = 0.0f, zu = 0.0f;
#pragma unroll
      for (int wv = 0; wv < kUpWaves; ++wv) {
        zg += reinterpret_cast<const float*>(part[turn][wv][2 * p])[tid];
        zu += reinterpret_cast<const float*>(part[turn][wv][2 * p + 1])[tid];
      }
      if (c < have && n < g.I) {
        const float h = silu(zg) * zu;
        static_cast<uint16_t*>(g.h)[static_cast<size_t>(sh.order[off + c]) * g.I + n] =
            static_cast<uint16_t>(pack2<ACT>(h, 0.0f));
      }
    }
  }
}

// ---- down product and weighted combine -------------------------------------------
//
// Each block owns 16 columns of the output for every token, its waves contiguous parts
// of the (item, step of K) sequence. An item's at most 16 tokens fill the instruction
// from its first row on, whichever they are; their sums go, times their gate weights, to
// the wave's own sums of all tokens in LDS. (With fixed places of tokens an expert's
// two tokens often took two instructions' rows: 32 tokens of 256 experts, 7168 x 2048,
// 433 us for this kernel.) With several shares blockIdx.y is the share of the sequence,
// and packed_sum_kernel adds them up.

struct DownTables {
  int4* item;    // [pairs]
  int* order;    // [pairs]
  float* w;      // [pairs]
  float* sum;    // [waves][T][columns of the block]
  static size_t bytes(int pairs, int T, int waves, int columns) {
    return pairs * (sizeof(int4) + sizeof(int) + sizeof(float)) + sizeof(float) * waves * T * columns;
  }
  __device__ __forceinline__ DownTables(void* lds, int pairs) {
    item = static_cast<int4*>(lds);
    order = reinterpret_cast<int*>(item + pairs);
    w = reinterpret_cast<float*>(order + pairs);
    sum = w + pairs;
  }
};

template <int ACT, int CODES, int PER, int NT, int TILES>
__global__ __launch_bounds__(NT, 4) void packed_down_kernel(PackedArgs g) {
  constexpr int kWaves = NT / kWave, kColumns = TILES * kPackedRows;
  extern __shared__ __align__(16) char tables[];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int pairs = g.T * g.k, sums = g.T * kColumns;
  const DownTables sh(tables, pairs);
  for (int p = tid; p < pairs; p += NT) {  // those past the items are not used
    sh.item[p] = g.item[p];
    sh.order[p] = g.order[p];
    sh.w[p] = g.w[p];
  }
  for (int i = tid; i < kWaves * sums; i += NT) sh.sum[i] = 0.0f;
  const int items = g.head[0];
  __syncthreads();

  constexpr int TB = packed_tile_bytes(PER);
  const int r = lane & 15, grp = lane >> 4;
  const int tile = blockIdx.x * TILES, tiles = packed_row_tiles(g.H), steps = packed_col_tiles(g.I);
  const size_t strip = static_cast<size_t>(steps) * TB;
  const size_t next = tile + 1 < tiles ? strip : 0;  // of a block's two tiles
  const int shares = gridDim.y, share = blockIdx.y;
  const int all = items * steps;
  const int total = all / shares + (share < all % shares ? 1 : 0);
  int q = all / shares * share + min(share, all % shares) + total / kWaves * wave + min(wave, total % kWaves);
  const int q_end = q + total / kWaves + (wave < total % kWaves ? 1 : 0);
  float* const mine = sh.sum + wave * sums + r;
  while (q < q_end) {
    const int i = q / steps, k0 = q % steps, k1 = min(steps, k0 + q_end - q);
    q += k1 - k0;
    const int4 it = sh.item[i];
    const int e = __builtin_amdgcn_readfirstlane(it.x), off = it.y, have = it.z;
    const unsigned char* row = g.w_down + (static_cast<size_t>(e) * tiles + tile) * strip;
    const uint16_t* tok = static_cast<const uint16_t*>(g.h) + static_cast<size_t>(sh.order[off + min(r, have - 1)]) * g.I;
    const int cols = r < have ? g.I : 0;
    v4f sum[TILES];
#pragma unroll
    for (int n = 0; n < TILES; ++n) sum[n] = v4f{0, 0, 0, 0};
    constexpr int D = 2 / TILES;  // steps in flight
    for (int kb0 = k0; kb0 < k1; kb0 += D) {
      PackedTile<PER> a[D][TILES];
      PackedRows c[D];
#pragma unroll
      for (int d = 0; d < D; ++d) {
        if (kb0 + d < k1) {
#pragma unroll
          for (int n = 0; n < TILES; ++n) a[d][n].load(row + n * next + static_cast<size_t>(kb0 + d) * TB, lane);
          c[d].load(tok, kb0 + d, grp, cols);
        }
      }
#pragma unroll
      for (int d = 0; d < D; ++d) {
        if (kb0 + d < k1) {
          v4f start[PER];
          packed_start<ACT, CODES, PER>(c[d], start);
#pragma unroll
          for (int n = 0; n < TILES; ++n) {
            float s[PER];
            a[d][n].scales(g.scale_act, s);
            packed_product<ACT, CODES, PER>(c[d], a[d][n], s, start, sum[n]);
          }
        }
      }
    }
    // an expert's tokens are different ones
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int m = 4 * grp + j;
      if (m < have) {
        const int pair = sh.order[off + m];
        float* to = mine + pair / g.k * kColumns;
#pragma unroll
        for (int n = 0; n < TILES; ++n) to[n * 16] = fmaf(sum[n][j], sh.w[pair], to[n * 16]);
      }
    }
  }
  __syncthreads();
  for (int o = tid; o < sums; o += NT) {
    float z = 0.0f;
#pragma unroll
    for (int wv = 0; wv < kWaves; ++wv) z += sh.sum[wv * sums + o];
    const int col = tile * kPackedRows + o % kColumns;
    if (TILES > 1 && col >= g.H) continue;
    const size_t at = static_cast<size_t>(o / kColumns) * g.H + col;
    if (shares > 1) g.part[static_cast<size_t>(share) * g.T * g.H + at] = z;
    else if (g.out_f32) static_cast<float*>(g.out)[at] = z;
    else static_cast<uint16_t*>(g.out)[at] = static_cast<uint16_t>(pack2<ACT>(z, 0.0f));
  }
}

template <int ACT>
__global__ __launch_bounds__(256) void packed_sum_kernel(PackedArgs g, int shares) {
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

// With many weights one block on a column tile at a time leaves CUs without work at the
// end (448 tiles of 7168 columns: one CU in four has one, the others two), and waves'
// parts are long. The sequence is split then, and blocks, with two tiles each, become
// many. Whole layer, us without and with 8 shares (integers, groups of 128; 4 shares
// 3 % slower in the first, 5 and 12 the same), the same inputs again and again: where
// they have under 256 MB, the weights come from the last-level cache (the last case takes
// 44 us with three sets in turn, the one before 48; no width under 1024 was measured):
//   tokens, experts, top-k, H, I    weights of the down product
//   32, 256, 8, 7168, 2048          2^31.8    734, 633
//   32, 256, 8, 4096, 2048          2^31.0    411, 376
//   16, 128, 8, 7168, 2048          2^30.8    420, 369
//   32, 64, 8, 7168, 2048           2^29.8    331, 289
//   32, 64, 8, 4112, 2048           2^29.0    256, 188
//   8, 64, 8, 4096, 2048            2^29.0    125, 118
//   16, 160, 6, 2064, 1424          2^28.1    120, 102
//   8, 64, 2, 7168, 2048            2^27.8     81,  78
//   32, 64, 8, 2048, 1408           2^27.5    106,  82
//   32, 32, 4, 5120, 1024           2^27.3     67,  58
//   64, 64, 4, 1024, 2048           2^27.0    124,  83
//   8, 64, 2, 4096, 2048            2^27.0     40,  42
//   1, 64, 8, 7168, 2048            2^26.8     39,  40
//   5, 64, 6, 2064, 1424            2^26.4     39,  39
constexpr int kShares = 8;
int shares_of(int T, int E, int k, int H, int I) {
  const long long experts = T * k < E ? T * k : E;
  return experts * H * I >= (T * k >= 64 ? 1ll << 27 : 3ll << 26) ? kShares : 1;
}

size_t whole(size_t bytes) { return (bytes + 255) / 256 * 256; }
size_t inner_bytes(int T, int k, int I) { return whole(static_cast<size_t>(T) * k * I * 2); }
size_t table_bytes(int T, int k) {
  return whole(static_cast<size_t>(T) * k * (sizeof(int4) + sizeof(int32_t)) + 2 * sizeof(int32_t));
}

template <int ACT, int CODES, int PER>
hipError_t launch(const PackedArgs& g, hipStream_t s) {
  const int per_token = g.E * ((g.T + 15) / 16);
  const long long items = g.T * g.k < per_token ? g.T * g.k : per_token;
  const size_t lds = Tables::bytes(g.T * g.k, g.E);
  auto up = [&](auto R, auto P) {
    constexpr bool ROUTES = R;
    constexpr int PAIRS = P;
    const long long work = items * ((g.I / kPackedRows + PAIRS - 1) / PAIRS);
    const int blocks = work < kUpBlocks ? static_cast<int>(work) : kUpBlocks;
    packed_up_kernel<ACT, CODES, PER, ROUTES, PAIRS>
        <<<blocks, kUpThreads, ROUTES ? lds : Tables::bytes(g.T * g.k, 0), s>>>(g);
  };
  auto pairs = [&](auto R) {
    if (items * (g.I / kPackedRows) >= kManyTiles) up(R, std::integral_constant<int, 2>{});
    else up(R, std::integral_constant<int, 1>{});
  };
  if (g.T * g.k <= kFewPairs) {
    pairs(std::true_type{});
  } else {
    packed_route_kernel<<<1, kRouteThreads, lds, s>>>(g);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
    pairs(std::false_type{});
  }
  hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  const int shares = shares_of(g.T, g.E, g.k, g.H, g.I);
  auto down = [&](auto N, auto M) {
    constexpr int NT = N, TILES = M;
    const dim3 grid((packed_row_tiles(g.H) + TILES - 1) / TILES, shares);
    packed_down_kernel<ACT, CODES, PER, NT, TILES>
        <<<grid, NT, DownTables::bytes(g.T * g.k, g.T, NT / kWave, TILES * kPackedRows), s>>>(g);
  };
  // Up to 256 tiles a CU has one block, which then has 16 waves to keep loads in flight:
  // one token of 256 experts, 4096 x 2048, 30.2 us for 31.8 with 8. With more tiles
  // two blocks of 8 waves are better: one token's top-8 in 7168 x 2048 (64 experts) 48.3
  // us for 50.2 with 16, in 7168 x 1024 (256 experts) 31.8 for 33.5, inputs in turn.
  using One = std::integral_constant<int, 1>;
  if (shares > 1) down(std::integral_constant<int, 512>{}, std::integral_constant<int, 2>{});
  else if (packed_row_tiles(g.H) <= 256) down(std::integral_constant<int, 1024>{}, One{});
  else down(std::integral_constant<int, 512>{}, One{});
  err = hipGetLastError();
  if (err != hipSuccess || shares == 1) return err;
  packed_sum_kernel<ACT><<<(g.T * g.H / 4 + 255) / 256, 256, 0, s>>>(g, shares);
  return hipGetLastError();
}

}  // namespace

// The inner rows, the tables, the shares' sums.
size_t layer_packed_ws_bytes(int T, int E, int k, int H, int I) {
  const int shares = shares_of(T, E, k, H, I);
  const size_t sums = shares > 1 ? whole(static_cast<size_t>(shares) * T * H * sizeof(float)) : 0;
  return inner_bytes(T, k, I) + table_bytes(T, k) + sums;
}

hipError_t launch_layer_few_tokens_packed(const PackedFormat& f, const float* logits, const void* x, const void* w_up,
                                          const void* w_down, int T, int E, int k, int H, int I, int32_t* idx, float* w,
                                          void* out, void* ws, int act, bool out_f32, hipStream_t s) {
  char* tables = static_cast<char*>(ws) + inner_bytes(T, k, I);
  int4* item = reinterpret_cast<int4*>(tables);
  int32_t* order = reinterpret_cast<int32_t*>(item + T * k);
  float* part = reinterpret_cast<float*>(tables + table_bytes(T, k));
  const PackedArgs g{{logits, T, E, k, idx, w, item, order, order + T * k},
                     x,
                     static_cast<const unsigned char*>(w_up),
                     static_cast<const unsigned char*>(w_down),
                     H,
                     I,
                     f.scale_act,
                     ws,
                     out,
                     out_f32,
                     part};
  return with_packed(f, act, [&](auto A, auto C, auto P) { return launch<A(), C(), P()>(g, s); });
}

}  // namespace moe
