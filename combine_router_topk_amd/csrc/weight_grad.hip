// Gradient of the experts' weights over the routed rows:
//
//   dW[e, n, k] = sum over rows r of e's segment of dy[r, n] a[r', k],  r' = r or src[r] / k
//
// The sum runs along the rows, which both operands have outermost, so the matrix
// instructions' operands (8 rows of one column a lane) are columns of what lies in
// memory. Rows go to LDS as they are, and the LDS reads transpose: four lanes read
// 16 neighbouring values of one row, and each lane of 16 gets four rows of one
// column.
//
// A block sums 128 x 256 weights over one expert's rows, 32 at a time, its four waves
// 64 x 128 each, so that a step's 24 reads of 64 lanes x 8 bytes feed 32 products of a
// wave; two blocks run on a CU. (256 x 256 with one block on a CU, through registers:
// 2129 us for the second case below; steps of 64 rows the same.) With long segments the
// loop bounds it: 16384 rows an expert reach 1015 TFLOP/s (a library product of 8192^3
// with the first operand transposed 1096). With 512 rows an expert, 64 experts of 4096 x
// 4096 in bf16, it takes 1437 to 1455 us, 756 to 765 TFLOP/s: without its 2.1 GB of
// stores 1099, so the two blocks of a CU hide little of them. 16384 tokens of a skewed
// top-6, 64 experts of 2048 x 1024 into fp32 with what is there added, take 595 to 620
// us, 508 without the addition and 470 into bf16: the results' reads and stores behind
// the products are what is left over the 346 of its bytes at a large copy's rate. 1021
// tokens of top-2, 8 experts of 2872 x 1424 into fp32, 50 us again and again and 55 to 57
// with inputs that change, for 30.
#include <limits.h>

#include "device.hpp"
#include "launch.hpp"
#include "quant.hpp"

namespace moe {

namespace {

constexpr int kThreads = 256;  // 4 waves: 2 along N, 2 along K
constexpr int kTileN = 128, kTileK = 256;  // weights of a block
constexpr int kStep = 32;      // rows of a step
constexpr int kXcds = 8, kPanel = 8;
constexpr int kFragsK = 8, kFragsN = 4;    // of a wave: 128 x 64
constexpr int kChunksN = kTileN / 8, kChunksK = kTileK / 8;  // 16-byte chunks of a row
// 1024-byte loads of a wave in a step: 4 rows of dy each, 2 of a
constexpr int kWaves = kThreads / kWave;
constexpr int kDyLoads = kStep / 4 / kWaves, kALoads = kStep / 2 / kWaves;
constexpr int kStages = 3;
constexpr int kWindow = 1024;  // rows whose sources are in LDS

struct GradArgs {
  const uint16_t* a;
  const uint16_t* dy;
  const int32_t* src;
  const int32_t* counts;
  const int32_t* offsets;
  int rows, E, K, N, n_tiles, k_tiles;
  uint32_t inverse;  // 2^32 / k, rounded up: i / k is the product's high half (i < 2^24, k <= 16); 0 for k = 1
  bool out_f32, add;
  void* dw;
  // With a plan (see below), else null:
  int most;     // parts more than experts
  int* found;   // units, and experts that are cut
  int4* unit;   // expert, first step, end, place of its sums or -1
  int4* cut;    // expert, first place, places
  float* part;  // [place][N][K]: sums of a part of an expert's rows
};

// A step: 32 rows of dy's 128 columns and of a's 256, 16-byte chunk c of row r at place
// c ^ 2 (r % 8): a transposing read takes 16 lanes at a time, 32 bytes of each of four
// rows, and these meet different banks (with c ^ r % 16 two rows in each four met the
// same).
__device__ __forceinline__ int swizzle(int row) { return (row & 7) << 1; }
struct Shared {
  uint4 stage[kStages][kStep * (kChunksN + kChunksK)];  // dy, then a
  int source[kWindow];
};
constexpr uint32_t kStageBytes = kStep * (kChunksN + kChunksK) * 16, kABytes = kStep * kChunksN * 16;

// What is loaded in place of rows past the segment's end and columns past the matrix's.
__device__ const uint4 zeros = {0, 0, 0, 0};

// Each lane's 16 bytes go to LDS at byte lds + 16 * lane without passing through
// registers. Written as assembly because the compiler, which cannot tell the stages
// apart, waits for every such load of its own before the next LDS read; here the loop
// counts them. `lds` is the same in all lanes; M0 may be read one wait state after it
// was written.
__device__ __forceinline__ void load_lds(const void* from, uint32_t lds) {
  asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(from), "{m0}"(lds) : "memory");
}
// Waits until at most N of this wave's loads are in flight, then for the other waves.
template <int N>
__device__ __forceinline__ void wait_loads() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

typedef short v4s __attribute__((ext_vector_type(4)));
__device__ __forceinline__ uint2 read_transposed(uint32_t at) {
  const auto p = reinterpret_cast<__attribute__((address_space(3))) v4s*>(at);
  return __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(p));
}
__device__ __forceinline__ uint32_t lds_address(const void* p) {
  return static_cast<uint32_t>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) const void*)p));
}

// Among lanes l, l + 16, l + 32, l + 48 (g = 0 .. 3) with values (a, g) and (b, g): lane
// g gets what lanes 2 (g % 2) and 2 (g % 2) + 1 had of a (g < 2) or b.
__device__ __forceinline__ void exchange(uint32_t& a, uint32_t& b) {
  const auto s = __builtin_amdgcn_permlane32_swap(a, b, false, false);
  const auto t = __builtin_amdgcn_permlane16_swap(s[0], s[1], false, false);
  a = t[0], b = t[1];
}

// Tile `in` of an expert. Neighbouring blocks go to the eight dies in turn, so each die
// takes a run of tiles, in panels of eight along N: they share rows in its cache. (Panels
// of 4 and of 16: 1453 and 1431 us for the 1442 of 64 experts of 4096 x 4096, 593 and 600
// for 600 of the skewed batch.)
__device__ __forceinline__ void tile_of(const GradArgs& g, int in, int& tn, int& tk) {
  const int tiles = g.n_tiles * g.k_tiles;
  if (tiles % kXcds == 0) in = in % kXcds * (tiles / kXcds) + in / kXcds;
  const int panel = in / (kPanel * g.k_tiles), left = in - panel * kPanel * g.k_tiles;
  const int wide = min(kPanel, g.n_tiles - panel * kPanel);
  tn = panel * kPanel + left % wide;
  tk = left / wide;
}

template <int ACT>
__global__ __launch_bounds__(kThreads, 2) void weight_grad_kernel(GradArgs g) {
  extern __shared__ __align__(16) char lds[];
  Shared& sh = *reinterpret_cast<Shared*>(lds);
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int tiles = g.n_tiles * g.k_tiles;
  const int u = blockIdx.x / tiles, in = blockIdx.x % tiles;
  if (g.unit != nullptr && u >= g.found[0]) return;
  const int4 unit = g.unit != nullptr ? g.unit[u] : make_int4(u, 0, INT_MAX, -1);
  const int e = unit.x, slot = unit.w;
  int tn, tk;
  tile_of(g, in, tn, tk);

  const int at = min(max(g.offsets[e], 0), g.rows), have = min(max(g.counts[e], 0), g.rows - at);
  const int s0 = unit.y, s1 = min(unit.z, (have + kStep - 1) / kStep);
  if (g.add && slot < 0 && s0 >= s1) return;

  // What this lane loads: chunk of dy's rows 4 q + lane / 16 and of a's 2 q + lane / 32, q
  // the wave's first load of a step and each fourth from there.
  const uint16_t* dy[kDyLoads];
  int dy_row[kDyLoads];
#pragma unroll
  for (int i = 0; i < kDyLoads; ++i) {
    dy_row[i] = 4 * (wave + kWaves * i) + (lane >> 4);
    const int col = tn * kTileN + ((lane & 15) ^ swizzle(dy_row[i])) * 8;
    dy[i] = g.dy + (static_cast<size_t>(at) + s0 * kStep + dy_row[i]) * g.N + col;
    if (col >= g.N) dy_row[i] = 1 << 30;
  }
  const unsigned char* a0[kALoads];
  uint32_t a_stride[kALoads];
#pragma unroll
  for (int i = 0; i < kALoads; ++i) {
    const int col = tk * kTileK + ((lane & 31) ^ swizzle(2 * (wave + kWaves * i) + (lane >> 5))) * 8;
    a0[i] = reinterpret_cast<const unsigned char*>(col < g.K ? static_cast<const void*>(g.a + col) : &zeros);
    a_stride[i] = col < g.K ? static_cast<uint32_t>(g.K) * 2 : 0;
  }
  // the sources of rows from step s on, -1 past the end
  auto fill = [&](int s) {
    for (int i = tid; i < kWindow; i += kThreads) {
      const int r = s * kStep + i;
      int from = -1;
      if (r < have) {
        from = at + r;
        if (g.src != nullptr) {
          const int i = min(max(g.src[from], 0), g.rows - 1);
          from = g.inverse == 0 ? i : static_cast<int>(__umulhi(static_cast<uint32_t>(i), g.inverse));
        }
      }
      sh.source[i] = from;
    }
    __syncthreads();
  };
  const uint32_t lds0 = lds_address(&sh.stage[0][0]) + wave * 1024;
  auto load_dy = [&](int i, int s, uint32_t stage) {
    const uint64_t zero = reinterpret_cast<uint64_t>(&zeros), from = reinterpret_cast<uint64_t>(dy[i]);
    load_lds(reinterpret_cast<const void*>(s * kStep + dy_row[i] < have ? from : zero), lds0 + stage + i * (kWaves * 1024));
    dy[i] += static_cast<size_t>(kStep) * g.N;
  };
  int source[kALoads];  // of the rows of the next step that is loaded
  auto read_sources = [&](int s) {
    const int window = (s - s0) * kStep % kWindow;
#pragma unroll
    for (int i = 0; i < kALoads; ++i) source[i] = sh.source[window + 2 * (wave + kWaves * i) + (lane >> 5)];
  };
  auto load_a = [&](int i, uint32_t stage) {
    const uint64_t zero = reinterpret_cast<uint64_t>(&zeros);
    const uint64_t from = reinterpret_cast<uint64_t>(a0[i]) +
                          static_cast<uint64_t>(static_cast<uint32_t>(source[i])) * a_stride[i];
    load_lds(reinterpret_cast<const void*>(source[i] >= 0 ? from : zero), lds0 + stage + kABytes + i * (kWaves * 1024));
  };

  // where this lane reads: row 4 (lane / 16) + (lane / 4) % 4 and 16 rows further, piece
  // lane % 4 of a fragment's 16 columns
  const int wn = wave & 1, wk = wave >> 1, grp = lane >> 4;
  const int lrow = lane >> 2, piece = lane & 3;
  uint32_t at_k[kFragsK], at_n[kFragsN];
#pragma unroll
  for (int f = 0; f < kFragsK; ++f)
    at_k[f] = lds_address(&sh.stage[0][0]) + kABytes + lrow * (kChunksK * 16) + ((wk * 16 + 2 * f + (piece >> 1)) ^ swizzle(lrow)) * 16 + (piece & 1) * 8;
#pragma unroll
  for (int f = 0; f < kFragsN; ++f)
    at_n[f] = lds_address(&sh.stage[0][0]) + lrow * (kChunksN * 16) + ((wn * 8 + 2 * f + (piece >> 1)) ^ swizzle(lrow)) * 16 + (piece & 1) * 8;

  v4f acc[kFragsK][kFragsN];
#pragma unroll
  for (int i = 0; i < kFragsK; ++i)
#pragma unroll
    for (int j = 0; j < kFragsN; ++j) acc[i][j] = v4f{0, 0, 0, 0};

  // Two steps' loads are in flight while a third is multiplied, issued between the
  // products, their rows' sources read from LDS a step before.
  uint32_t now = 0, ahead = 2 * kStageBytes;
  if (s0 < s1) {
    fill(s0);
    for (int s = s0; s < min(s0 + 2, s1); ++s) {
      read_sources(s);
#pragma unroll
      for (int i = 0; i < kDyLoads; ++i) load_dy(i, s, (s - s0) * kStageBytes);
#pragma unroll
      for (int i = 0; i < kALoads; ++i) load_a(i, (s - s0) * kStageBytes);
    }
    read_sources(s0 + 2);
  }
  for (int s = s0; s < s1; ++s) {
    if (s + 1 < s1) wait_loads<kDyLoads + kALoads>();
    else wait_loads<0>();
    if ((s + 3 - s0) % (kWindow / kStep) == 0 && s + 3 < s1) fill(s + 3);
    const bool more = s + 2 < s1;
    uint4 n[kFragsN], k[2];
    auto read = [&](uint32_t from, uint32_t half) {
      const uint2 lo = read_transposed(from + now), hi = read_transposed(from + now + half);
      return make_uint4(lo.x, lo.y, hi.x, hi.y);
    };
#pragma unroll
    for (int f = 0; f < kFragsN; ++f) n[f] = read(at_n[f], 16 * kChunksN * 16);
    k[0] = read(at_k[0], 16 * kChunksK * 16);
#pragma unroll
    for (int i = 0; i < kFragsK; ++i) {
      // the next fragment is read under this one's products
      if (i + 1 < kFragsK) k[(i + 1) & 1] = read(at_k[i + 1], 16 * kChunksK * 16);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int j = 0; j < kFragsN; ++j) acc[i][j] = mfma16<ACT>(k[i & 1], n[j], acc[i][j]);
      __builtin_amdgcn_sched_barrier(0);
      if (more) {
        if (i < kDyLoads) load_dy(i, s + 2, ahead);
        else if (i < kDyLoads + kALoads) load_a(i - kDyLoads, ahead);
        else if (i == kDyLoads + kALoads) read_sources(s + 3);
      }
    }
    now = now == 2 * kStageBytes ? 0 : now + kStageBytes;
    ahead = ahead == 2 * kStageBytes ? 0 : ahead + kStageBytes;
  }

  // A lane's four results of a fragment are four neighbouring k of one n: 16 bytes in
  // fp32, 64 of a row by four lanes. In 16 bits these four exchange the results of two
  // fragments, so that each has 8 neighbours: stores of 32 bytes of a row instead took
  // 1650 us for 64 experts of 4096 x 4096, this 1455. (Whole lines by way of LDS, 1440
  // there and 560 for 457 where fp32 sums are added up in 2048 x 2048; stores past the
  // caches, 62 for 22 us in 110 MB of odd rows.)
  const size_t matrix = static_cast<size_t>(e) * g.N * g.K;
#pragma unroll
  for (int j = 0; j < kFragsN; ++j) {
    const int n = tn * kTileN + wn * 64 + j * 16 + (lane & 15);
    const size_t line = static_cast<size_t>(n) * g.K;
    if (slot >= 0 || g.out_f32) {
#pragma unroll
      for (int i = 0; i < kFragsK; ++i) {
        const int k = tk * kTileK + wk * 128 + i * 16 + grp * 4;
        if (n >= g.N || k >= g.K) continue;
        v4f v = acc[i][j];
        v4f* to = reinterpret_cast<v4f*>(slot >= 0 ? g.part + static_cast<size_t>(slot) * g.N * g.K + line + k
                                                   : static_cast<float*>(g.dw) + matrix + line + k);
        if (slot < 0 && g.add) v += *to;
        *to = v;
      }
    } else {
#pragma unroll
      for (int i = 0; i < kFragsK; i += 2) {
        const v4f a = acc[i][j], b = acc[i + 1][j];
        uint2 p = make_uint2(pack2<ACT>(a[0], a[1]), pack2<ACT>(a[2], a[3]));
        uint2 q = make_uint2(pack2<ACT>(b[0], b[1]), pack2<ACT>(b[2], b[3]));
        exchange(p.x, q.x);
        exchange(p.y, q.y);
        const int k = tk * kTileK + wk * 128 + i * 16 + grp * 8;
        if (n < g.N && k < g.K)
          *reinterpret_cast<uint4*>(static_cast<uint16_t*>(g.dw) + matrix + line + k) = make_uint4(p.x, p.y, q.x, q.y);
      }
    }
  }
}

// ---- the plan ------------------------------------------------------------------------
//
// Where routing is skewed one expert's rows can be more than a block's share of all the
// work, and where an expert has few tiles there are too few blocks. Then experts with
// more than C steps of rows are cut into parts of at most that many, the longest parts
// are first in the grid, and a kernel adds up the parts' sums in their order. C is
// what a block takes if the steps of all tiles are dealt out to kSlots blocks: all
// steps / most, most = kSlots / tiles. So parts are at most `most` more than experts,
// whatever the counts are, and the parts of cut experts at most 2 most: their sums take
// about 2 kSlots tiles of 128 x 256 at most, 134 MB. (C half of that, the skewed top-6
// batch: 664 us for 640; a quarter: 727.)

constexpr int kSlots = 512;      // blocks that run at once
constexpr int kLeastSteps = 8;   // C is no less
constexpr int kPlanThreads = 1024;

__global__ __launch_bounds__(kPlanThreads) void weight_grad_plan_kernel(GradArgs g) {
  __shared__ int sums[kPlanThreads / kWave];
  __shared__ int2 key[kMaxE];  // steps of a part, parts
  const int e = threadIdx.x, lane = e & 63, wave = e >> 6;
  int steps = 0;
  if (e < g.E) {
    const int at = min(max(g.offsets[e], 0), g.rows);
    steps = (min(max(g.counts[e], 0), g.rows - at) + kStep - 1) / kStep;
  }
  const int upto = wave_incl_scan(steps, lane);
  if (lane == kWave - 1) sums[wave] = upto;
  __syncthreads();
  long long all = 0;  // segments that overlap, which moe_layout does not write, add up to more than the rows
  for (int w = 0; w < kPlanThreads / kWave; ++w) all += sums[w];
  const int c = max(kLeastSteps, static_cast<int>((all + g.most - 1) / g.most));
  const int parts = steps > c ? (steps + c - 1) / c : 1;
  if (e < g.E) key[e] = make_int2((steps + parts - 1) / parts, parts);
  __syncthreads();
  if (e >= g.E) return;
  int units = 0, places = 0, cuts = 0;  // of the experts before this one
  bool last = true;
  const int mine = key[e].x;
#pragma unroll 8
  for (int j = 0; j < g.E; ++j) {
    const int2 k = key[j];
    const bool before = k.x > mine || (k.x == mine && j < e);
    const int n = before ? k.y : 0, cut = n > 1 ? n : 0;
    units += n;
    places += cut;
    cuts += n > 1 ? 1 : 0;
    last = last && (before || j == e);
  }
  for (int i = 0; i < parts; ++i)
    g.unit[units + i] = make_int4(e, static_cast<int>(static_cast<long long>(steps) * i / parts),
                                  static_cast<int>(static_cast<long long>(steps) * (i + 1) / parts),
                                  parts > 1 ? places + i : -1);
  if (parts > 1) g.cut[cuts] = make_int4(e, places, parts, 0);
  if (last) {  // it knows the sums
    g.found[0] = units + parts;
    g.found[1] = cuts + (parts > 1);
  }
}

template <int ACT>
__global__ __launch_bounds__(256) void weight_grad_sum_kernel(GradArgs g) {
  if (static_cast<int>(blockIdx.y) >= g.found[1]) return;
  const int4 cut = g.cut[blockIdx.y];
  const size_t fours = static_cast<size_t>(g.N) * g.K / 4, i = static_cast<size_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= fours) return;
  const float4* part = reinterpret_cast<const float4*>(g.part) + cut.y * fours + i;
  float4 v = part[0];
  for (int s = 1; s < cut.z; ++s) {
    const float4 p = part[s * fours];
    v = make_float4(v.x + p.x, v.y + p.y, v.z + p.z, v.w + p.w);
  }
  if (g.out_f32) {
    float4* to = static_cast<float4*>(g.dw) + cut.x * fours + i;
    if (g.add) {
      const float4 o = *to;
      v = make_float4(o.x + v.x, o.y + v.y, o.z + v.z, o.w + v.w);
    }
    *to = v;
  } else {
    static_cast<uint2*>(g.dw)[cut.x * fours + i] = make_uint2(pack2<ACT>(v.x, v.y), pack2<ACT>(v.z, v.w));
  }
}

// Of N and K from 1 up to the end of 32 bits.
int n_tiles_of(int N) { return (N - 1) / kTileN + 1; }
int k_tiles_of(int K) { return (K - 1) / kTileK + 1; }

// The plan's sizes; `units` 0 for no plan. A token chooses an expert once, so no tile has
// more than T rows; with k tiles >= kSlots that is no more than a block's share of the
// work, and below a thousand tokens the plan's two launches take longer than it saves.
struct Plan {
  int most = 0, units = 0, places = 0, cuts = 0;
  size_t unit_bytes = 0, cut_bytes = 0, bytes = 0;
  Plan(int T, int E, int k, int K, int N) {
    const long long tiles = static_cast<long long>(n_tiles_of(N)) * k_tiles_of(K);
    if (k * tiles >= kSlots || T < 1024) return;
    const long long steps = static_cast<long long>(T) * k / kStep + E;
    const long long by_share = kSlots / tiles, by_least = steps / kLeastSteps;
    most = static_cast<int>(by_share < by_least ? by_share : by_least);  // at least 1
    units = E + most;
    places = 2 * most;
    cuts = E < most ? E : most;
    unit_bytes = (units * sizeof(int4) + 255) / 256 * 256;
    cut_bytes = (cuts * sizeof(int4) + 255) / 256 * 256;
    bytes = 256 + unit_bytes + cut_bytes + static_cast<size_t>(places) * N * K * sizeof(float);
  }
};

}  // namespace

bool weight_grad_fits(int E, int K, int N) {
  return static_cast<long long>(E) * n_tiles_of(N) * k_tiles_of(K) < 1ll << 23;
}

size_t weight_grad_ws_bytes(int T, int E, int k, int K, int N) { return Plan(T, E, k, K, N).bytes; }

hipError_t launch_weight_grad(const void* a, const int32_t* src, const void* dy, const int32_t* counts,
                              const int32_t* offsets, int T, int E, int k, int K, int N, bool add, void* dw, void* ws,
                              int act, bool out_f32, hipStream_t s) {
  const Plan plan(T, E, k, K, N);
  GradArgs g{};
  g.a = static_cast<const uint16_t*>(a);
  g.dy = static_cast<const uint16_t*>(dy);
  g.src = src;
  g.counts = counts;
  g.offsets = offsets;
  g.rows = T * k;
  g.E = E;
  g.K = K;
  g.N = N;
  g.n_tiles = n_tiles_of(N);
  g.k_tiles = k_tiles_of(K);
  g.inverse = k == 1 ? 0 : static_cast<uint32_t>(((1ull << 32) + k - 1) / k);
  g.out_f32 = out_f32;
  g.add = add;
  g.dw = dw;
  if (plan.units > 0) {
    char* p = static_cast<char*>(ws);
    g.most = plan.most;
    g.found = reinterpret_cast<int*>(p);
    g.unit = reinterpret_cast<int4*>(p + 256);
    g.cut = reinterpret_cast<int4*>(p + 256 + plan.unit_bytes);
    g.part = reinterpret_cast<float*>(p + 256 + plan.unit_bytes + plan.cut_bytes);
    weight_grad_plan_kernel<<<1, kPlanThreads, 0, s>>>(g);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
  }
  const unsigned grid = static_cast<unsigned>(plan.units > 0 ? plan.units : E) * g.n_tiles * g.k_tiles;
  if (act == 1) weight_grad_kernel<1><<<grid, kThreads, sizeof(Shared), s>>>(g);
  else weight_grad_kernel<2><<<grid, kThreads, sizeof(Shared), s>>>(g);
  const hipError_t err = hipGetLastError();
  if (err != hipSuccess || plan.units == 0) return err;
  const dim3 sums(static_cast<unsigned>((static_cast<size_t>(N) * K / 4 + 255) / 256), plan.cuts);
  if (act == 1) weight_grad_sum_kernel<1><<<sums, 256, 0, s>>>(g);
  else weight_grad_sum_kernel<2><<<sums, 256, 0, s>>>(g);
  return hipGetLastError();
}

}  // namespace moe
