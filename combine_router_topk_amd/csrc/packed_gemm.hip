// Products of the routed rows in 16 bits with experts' weights in 4 bits
// (packed.hpp):
//
//   z[r, n] = sum over groups g of s[e, n, g] (sum over k in g of a[r', k] code(e, n, k))
//
// for every row r of expert e's segment, r' = r or the token of the row (src[r] /
// k). The epilogue writes z in the activation format or fp32, or takes the two halves
// of the weights' rows as gate and up and writes silu(gate) up in 16 bits.
#include <stddef.h>

#include "device.hpp"
#include "launch.hpp"
#include "packed.hpp"
#include "quant.hpp"

namespace moe {

namespace {

struct PackedGemmArgs {
  const uint16_t* a;
  const int32_t* src;
  const unsigned char* w;
  const int32_t* counts;
  const int32_t* offsets;
  int rows, a_rows, k, E, K, N;  // N: weight rows of an expert
  int half;                      // SwiGLU: N / 2
  int n_tiles;                   // of a kernel's tiles along N
  int scale_act;
  bool out_f32;
  void* y;
};

// The row of `a` that send row `row` takes.
__device__ __forceinline__ size_t source_row(const PackedGemmArgs& g, int row) {
  if (g.src == nullptr) return row;
  const int i = g.src[row];
  return i < 0 ? 0 : min(i / g.k, g.a_rows - 1);
}

// An expert's segment, cut to the rows there are.
__device__ __forceinline__ int2 segment_of(const PackedGemmArgs& g, int e) {
  const int at = min(max(g.offsets[e], 0), g.rows);
  return make_int2(at, min(max(g.counts[e], 0), g.rows - at));
}

// First tile of each expert, with `per` rows a tile: first[E] is their number. Segments
// that do not overlap, as moe_layout writes them, have rows / per + E times n_tiles of
// them at most, which fits 32 bits; where counts say more, the tiles end there. (Without
// n_tiles, all experts with all rows are 2^30 at most.)
struct Segments {
  int first[kMaxE + 1];
};
template <int NT>
__device__ __forceinline__ void find_segments(const PackedGemmArgs& g, int per, Segments& sh, int* sums) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  auto first_tile = [&](int m_tiles) {
    const long long n = static_cast<long long>(m_tiles) * g.n_tiles;
    const int most = (g.rows / per + g.E) * g.n_tiles;
    return n < most ? static_cast<int>(n) : most;
  };
  int base = 0;
  for (int e0 = 0; e0 < g.E; e0 += NT) {
    const int e = e0 + tid;
    int tiles = 0;
    if (e < g.E) tiles = (segment_of(g, e).y + per - 1) / per;
    const int upto = wave_incl_scan(tiles, lane);
    if (lane == kWave - 1) sums[wave] = upto;
    __syncthreads();
    int before = base;
    for (int w = 0; w < NT / kWave; ++w) {
      if (w < wave) before += sums[w];
      base += sums[w];
    }
    if (e < g.E) sh.first[e] = first_tile(before + upto - tiles);
    __syncthreads();
  }
  if (tid == 0) sh.first[g.E] = first_tile(base);
  __syncthreads();
}
// The expert of tile i: the last one whose first tile is not behind it (experts
// without tiles share their first tile with the next one).
__device__ __forceinline__ int expert_of(const Segments& sh, int E, int i) {
  int lo = 0, hi = E;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (sh.first[mid] <= i) lo = mid;
    else hi = mid;
  }
  return lo;
}

template <int ACT>
__device__ __forceinline__ void store_one(const PackedGemmArgs& g, size_t at, float z) {
  if (g.out_f32) static_cast<float*>(g.y)[at] = z;
  else static_cast<uint16_t*>(g.y)[at] = static_cast<uint16_t>(pack2<ACT>(z, 0.0f));
}

// ---- few rows an expert ------------------------------------------------------------

constexpr int kThinThreads = 256, kThinWaves = kThinThreads / kWave;
constexpr int kThinBlocks = 1280;

// A block owns 16 rows of a segment and TILES tiles of 16 weight rows (with SwiGLU half
// of them the gate's and half the up's beside them), its waves every fourth step of K.
// Four tiles share the rows' loads, which take as many instructions as four tiles do:
// gate and up of 8 rows for each of 256 experts, 4096 x 2048, 532 us with two.
template <int ACT, int CODES, int PER, bool SWIGLU, int TILES>
__global__ __launch_bounds__(kThinThreads, TILES == 2 ? 5 : 4) void packed_thin_kernel(PackedGemmArgs g) {
  __shared__ Segments sh;
  __shared__ int sums[kThinWaves];
  __shared__ float4 part[2][kThinWaves][TILES][kWave];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  find_segments<kThinThreads>(g, 16, sh, sums);

  constexpr int TB = packed_tile_bytes(PER), kApart = SWIGLU ? TILES / 2 : TILES;  // tiles of y
  const int r = lane & 15, grp = lane >> 4;
  const int steps = packed_col_tiles(g.K), row_tiles = packed_row_tiles(g.N);
  const int half_tiles = g.half / kPackedRows, y_tiles = SWIGLU ? half_tiles : row_tiles;
  const size_t strip = static_cast<size_t>(steps) * TB;  // a row of tiles
  const int work = sh.first[g.E];
  int turn = 0;
  for (int i = blockIdx.x; i < work; i += gridDim.x, turn ^= 1) {
    const int e = __builtin_amdgcn_readfirstlane(expert_of(sh, g.E, i));
    const int2 seg = segment_of(g, e);
    const int in = i - sh.first[e], m_tiles = (seg.y + 15) / 16;
    const int tile = in / m_tiles * kApart, m0 = (in % m_tiles) * 16;  // rows of the same weights follow each other
    const int row0 = seg.x + m0, have = min(16, seg.y - m0);
    const unsigned char* w[TILES];  // tiles past the end are the last one again
#pragma unroll
    for (int n = 0; n < TILES; ++n) {
      const int t = min(tile + n % kApart, y_tiles - 1) + (SWIGLU && n >= kApart ? half_tiles : 0);
      w[n] = g.w + (static_cast<size_t>(e) * row_tiles + t) * strip;
    }
    const uint16_t* row = g.a + source_row(g, row0 + min(r, have - 1)) * g.K;
    const int cols = r < have ? g.K : 0;

    v4f z[TILES];
#pragma unroll
    for (int n = 0; n < TILES; ++n) z[n] = v4f{0, 0, 0, 0};
    for (int kb = wave; kb < steps; kb += kThinWaves) {
      PackedTile<PER> a[TILES];
      PackedRows x;
#pragma unroll
      for (int n = 0; n < TILES; ++n) a[n].load(w[n] + static_cast<size_t>(kb) * TB, lane);
      x.load(row, kb, grp, cols);
      v4f start[PER];
      packed_start<ACT, CODES, PER>(x, start);
#pragma unroll
      for (int n = 0; n < TILES; ++n) {
        float s[PER];
        a[n].scales(g.scale_act, s);
        packed_product<ACT, CODES, PER>(x, a[n], s, start, z[n]);
      }
    }
#pragma unroll
    for (int n = 0; n < TILES; ++n) part[turn][wave][n][lane] = make_float4(z[n][0], z[n][1], z[n][2], z[n][3]);
    __syncthreads();
    // thread tid sums value tid % 4 of lane tid / 4: row 4 (tid / 64) + tid % 4 of the
    // segment's 16, weight row (tid / 4) % 16 of the tiles
    const int c = (tid >> 6) * 4 + (tid & 3), nn = (tid >> 2) & 15;
    auto sum = [&](int n) {
      float s = 0.0f;
#pragma unroll
      for (int wv = 0; wv < kThinWaves; ++wv) s += reinterpret_cast<const float*>(part[turn][wv][n])[tid];
      return s;
    };
#pragma unroll
    for (int n = 0; n < kApart; ++n) {
      const int col = (tile + n) * kPackedRows + nn;
      if constexpr (SWIGLU) {
        const float h = silu(sum(n)) * sum(n + kApart);
        if (c < have && col < g.half)
          static_cast<uint16_t*>(g.y)[static_cast<size_t>(row0 + c) * g.half + col] =
              static_cast<uint16_t>(pack2<ACT>(h, 0.0f));
      } else {
        const float y = sum(n);
        if (c < have && col < g.N) store_one<ACT>(g, static_cast<size_t>(row0 + c) * g.N + col, y);
      }
    }
  }
}

// ---- many rows an expert -----------------------------------------------------------
//
// A block multiplies 128 rows by 256 weight rows, its 8 waves 64 by 64 each (2 along the
// rows, 4 along the weights). Rows, codes and scales of a step of 128 columns go to LDS
// without passing registers, three steps in a ring. A wave takes 64 rows of a group's
// columns into registers, then one tile of weights after the other: its codes become
// 16-bit numbers between the products, and the group's sums are multiplied by their
// scales under the next tile's products.
//
// The vector unit bounds it beside the matrix cores: 8 codes take 4 to 7 of its
// instructions, each group's sums of a fragment four more, and a fragment's product
// occupies the matrix cores for 16 cycles at best. With e2m1 in groups of 32 the vector
// unit issues in 61 % (K = 1024) to 69 % (gate and up, K = 2048) of the cycles and the
// matrix cores are busy in 31 to 33 %: together nearly all of them, so the two waves of a
// SIMD, which pass the same barrier in each step, hardly run them at once. Measured with 8192 tokens of a top-6
// over 64 experts, N = 2048, TFLOP/s: K = 4096, e2m1 955 in groups of 128 and 766 in
// groups of 32, integers 811 and 672; K = 1024 (8 steps a tile, where a tile's first
// loads and its results take a sixth) 812, 670, 701 and 595. (Operands through
// registers into LDS, scales under the products of the same tile: 413 us for the 309 of
// e2m1 in groups of 32, K = 1024. The next tile's first loads under the results' stores:
// 1 % at K = 1024, none at 4096, and spilled registers.)

constexpr int kFatThreads = 512, kFatWaves = kFatThreads / kWave;
constexpr int kFatRows = 128;              // of a tile: 2 waves of 64
constexpr int kFatTiles = 4;               // of weights, a wave
constexpr int kFatFrags = 4;               // of 16 rows, a wave
constexpr int kFatBlocks = 256;
constexpr int kFatStages = 3;
constexpr int kFatLoads = 7;               // of a wave in a step: 4 of rows, 2 of codes, 1 of scales

// Rows of a step: 256 bytes each, 16-byte chunk c of row r at place c ^ (r % 16), so that
// 16 lanes that read one chunk of 16 rows meet all banks. Two tiles' scales follow each
// other, from each 256 bytes on.
struct FatStage {
  uint4 rows[kFatRows * 16];
  uint4 codes[4 * kFatTiles * 64];
  unsigned char scales[kFatWaves * 256];
};
struct FatShared {
  FatStage stage[kFatStages];
  Segments seg;
  int sums[kFatWaves];
};
constexpr uint32_t kFatStageBytes = sizeof(FatStage);
static_assert(sizeof(FatShared) <= 160 * 1024, "LDS");

// What is loaded in place of columns past the rows' end.
__device__ const uint4 zeros = {0, 0, 0, 0};

// Each lane's 16 (or 4) bytes go to LDS at byte lds + 16 (or 4) * lane without passing
// through registers. Written as assembly because the compiler, which cannot tell the
// stages apart, waits for every such load of its own before the next LDS read; here the
// loop counts them. `lds` is the same in all lanes; M0 may be read one wait state after
// it was written.
__device__ __forceinline__ void load_lds16(const void* from, uint32_t lds) {
  asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(from), "{m0}"(lds) : "memory");
}
__device__ __forceinline__ void load_lds4(const void* from, uint32_t lds) {
  asm volatile("s_nop 0\n\tglobal_load_lds_dword %0, off" ::"v"(from), "{m0}"(lds) : "memory");
}
// Waits until at most N of this wave's loads are in flight, then for the other waves.
template <int N>
__device__ __forceinline__ void wait_loads() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint32_t lds_address(const void* p) {
  return static_cast<uint32_t>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) const void*)p));
}

template <int ACT, int CODES, int PER, bool SWIGLU>
__global__ __launch_bounds__(kFatThreads, 2) void packed_fat_kernel(PackedGemmArgs g) {
  extern __shared__ __align__(16) char lds[];
  FatShared& sh = *reinterpret_cast<FatShared*>(lds);
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  find_segments<kFatThreads>(g, kFatRows, sh.seg, sh.sums);

  constexpr int TB = packed_tile_bytes(PER), kIn = 4 / PER;  // steps of 32 columns in a group
  const int wn = wave & 3, wm = wave >> 2;
  const int r = lane & 15, grp = lane >> 4;
  const int steps = packed_col_tiles(g.K), row_tiles = packed_row_tiles(g.N);
  const size_t strip = static_cast<size_t>(steps) * TB;
  const int work = sh.seg.first[g.E];
  // weight tile l (of 16) of block column nb; those past the end are the last one again
  auto tile_of = [&](int nb, int l) {
    if constexpr (SWIGLU) {
      const int last = g.half / kPackedRows - 1, n = l & 3;
      return min(nb * 8 + (l >> 2) * 2 + (n & 1), last) + (n >> 1) * (last + 1);
    } else {
      return min(nb * 16 + l, row_tiles - 1);
    }
  };
  for (int i = blockIdx.x; i < work; i += gridDim.x) {
    const int e = __builtin_amdgcn_readfirstlane(expert_of(sh.seg, g.E, i));
    const int2 seg = segment_of(g, e);
    const int in = i - sh.seg.first[e], m_tiles = (seg.y + kFatRows - 1) / kFatRows;
    const int nb = in / m_tiles, m0 = (in % m_tiles) * kFatRows;
    const int row0 = seg.x + m0, have = min(kFatRows, seg.y - m0);
    const bool idle = have <= wm * 64;

    // what this lane loads in each step
    const int chunk = (lane & 15) ^ ((4 * wave + (lane >> 4)) & 15);
    const uint16_t* row[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int m = 4 * (wave + kFatWaves * q) + (lane >> 4);
      row[q] = g.a + source_row(g, row0 + min(m, have - 1)) * g.K + chunk * 8;
    }
    const unsigned char* w = g.w + static_cast<size_t>(e) * row_tiles * strip;
    const unsigned char* code[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) code[q] = w + tile_of(nb, 2 * wave + q) * strip + lane * 16;
    constexpr int kScaleLanes = 8 * PER;  // of a tile
    const unsigned char* scale = w + tile_of(nb, 2 * wave + (lane / kScaleLanes & 1)) * strip + kPackedCodes +
                                 lane % kScaleLanes * 4;
    const uint32_t lds0 = lds_address(&sh.stage[0]);
    auto load = [&](int q, int kb, uint32_t at) {  // the q-th of a step's loads
      if (q < 4) {
        const uint64_t from = reinterpret_cast<uint64_t>(row[q] + kb * kPackedCols), zero = reinterpret_cast<uint64_t>(&zeros);
        load_lds16(reinterpret_cast<const void*>(kb * kPackedCols + chunk * 8 < g.K ? from : zero),
                   lds0 + at + (wave + kFatWaves * q) * 1024);
      } else if (q < 6) {
        load_lds16(code[q - 4] + static_cast<size_t>(kb) * TB,
                   lds0 + at + static_cast<uint32_t>(offsetof(FatStage, codes)) + (2 * wave + q - 4) * 1024);
      } else {
        load_lds4(scale + static_cast<size_t>(kb) * TB,
                  lds0 + at + static_cast<uint32_t>(offsetof(FatStage, scales)) + wave * 256);
      }
    };

    v4f acc[kFatTiles][kFatFrags];
#pragma unroll
    for (int n = 0; n < kFatTiles; ++n)
#pragma unroll
      for (int f = 0; f < kFatFrags; ++f) acc[n][f] = v4f{0, 0, 0, 0};
    __syncthreads();  // the stages are free
    for (int kb = 0; kb < min(2, steps); ++kb)
#pragma unroll
      for (int q = 0; q < kFatLoads; ++q) load(q, kb, kb * kFatStageBytes);
    uint32_t now = 0, ahead = 2 * kFatStageBytes;
    for (int kb = 0; kb < steps; ++kb) {
      if (kb + 1 < steps) wait_loads<kFatLoads>();
      else wait_loads<0>();
      if (kb + 2 < steps)
#pragma unroll
        for (int q = 0; q < kFatLoads; ++q) load(q, kb + 2, ahead);
      if (!idle) {
        const FatStage& st = *reinterpret_cast<const FatStage*>(lds + now);
        uint4 codes[kFatTiles];
        uint32_t raw[kFatTiles][PER == 4 ? 2 : 1];
#pragma unroll
        for (int n = 0; n < kFatTiles; ++n) {
          const int l = wn * kFatTiles + n;
          codes[n] = st.codes[l * 64 + lane];
          const unsigned char* s = st.scales + (l >> 1) * 256 + (l & 1) * (32 * PER) + r * (2 * PER);
          if constexpr (PER == 1) raw[n][0] = *reinterpret_cast<const uint16_t*>(s);
          else raw[n][0] = *reinterpret_cast<const uint32_t*>(s);
          if constexpr (PER == 4) raw[n][1] = *reinterpret_cast<const uint32_t*>(s + 4);
        }
        v4f z[2][kFatFrags];
        float sc[2];
#pragma unroll
        for (int p = 0; p < PER; ++p) {
          uint4 x[kIn][kFatFrags];
#pragma unroll
          for (int j = 0; j < kIn; ++j)
#pragma unroll
            for (int f = 0; f < kFatFrags; ++f)
              x[j][f] = st.rows[(wm * 64 + f * 16 + r) * 16 + ((4 * (p * kIn + j) + grp) ^ r)];
          v4f start[kFatFrags];
#pragma unroll
          for (int f = 0; f < kFatFrags; ++f) {
            start[f] = v4f{0, 0, 0, 0};
            if constexpr (CODES == kPackedInt) {
              constexpr uint32_t kMinus8 = ACT == 1 ? 0xc800c800u : 0xc100c100u;
#pragma unroll
              for (int j = 0; j < kIn; ++j)
                start[f] = mfma16<ACT>(x[j][f], make_uint4(kMinus8, kMinus8, kMinus8, kMinus8), start[f]);
            }
          }
#pragma unroll
          for (int n = 0; n < kFatTiles; ++n) {
            const int step = p * kFatTiles + n, b = step & 1;
            __builtin_amdgcn_sched_barrier(0);
            sc[b] = packed_scale(g.scale_act, raw[n][p >> 1], p & 1);
#pragma unroll
            for (int j = 0; j < kIn; ++j) {
              const int c = p * kIn + j;
              const uint4 v = packed_values<ACT, CODES>(c == 0 ? codes[n].x : c == 1 ? codes[n].y : c == 2 ? codes[n].z
                                                                                                          : codes[n].w);
#pragma unroll
              for (int f = 0; f < kFatFrags; ++f) z[b][f] = mfma16<ACT>(x[j][f], v, j == 0 ? start[f] : z[b][f]);
            }
            if (step > 0) {
              const int before = (step - 1) % kFatTiles;
#pragma unroll
              for (int f = 0; f < kFatFrags; ++f)
#pragma unroll
                for (int q = 0; q < 4; ++q) acc[before][f][q] = fmaf(z[b ^ 1][f][q], sc[b ^ 1], acc[before][f][q]);
            }
            // one product, then what the vector unit does meanwhile
#pragma unroll
            for (int m = 0; m < kIn * kFatFrags; ++m) {
              __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
              __builtin_amdgcn_sched_group_barrier(0x002, 2 + 4 / kIn, 0);
            }
          }
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int f = 0; f < kFatFrags; ++f)
#pragma unroll
          for (int q = 0; q < 4; ++q)
            acc[kFatTiles - 1][f][q] = fmaf(z[1][f][q], sc[1], acc[kFatTiles - 1][f][q]);
      }
      now = now == 2 * kFatStageBytes ? 0 : now + kFatStageBytes;
      ahead = ahead == 2 * kFatStageBytes ? 0 : ahead + kFatStageBytes;
    }

    // A lane's results lie in 16 rows, one column of a tile each: they go through the
    // wave's part of the stages, and whole pieces of a row are stored.
    __syncthreads();
    if (!idle) {
      constexpr int kColumns = SWIGLU ? 32 : 64;
      constexpr uint32_t kPart = kFatStages * kFatStageBytes / kFatWaves / 256 * 256;
      unsigned char* const mine = reinterpret_cast<unsigned char*>(lds) + wave * kPart;
      auto pass = [&](auto F32) {
        constexpr bool f32 = F32;
        constexpr int kLine = kColumns * (f32 ? 4 : 2), kPitch = kLine + 16, kLanes = kLine / 16;
        static_assert(64 * kPitch <= kPart, "");
#pragma unroll
        for (int n = 0; n < kColumns / 16; ++n)
#pragma unroll
          for (int f = 0; f < kFatFrags; ++f)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              float v = acc[n][f][q];
              if constexpr (SWIGLU) v = silu(v) * acc[n + 2][f][q];
              unsigned char* to = mine + (f * 16 + 4 * grp + q) * kPitch + (n * 16 + r) * (f32 ? 4 : 2);
              if constexpr (f32) *reinterpret_cast<float*>(to) = v;
              else *reinterpret_cast<uint16_t*>(to) = static_cast<uint16_t>(pack2<ACT>(v, 0.0f));
            }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // the wave's lanes exchange them
        const int width = SWIGLU ? g.half : g.N;
        const int col = (nb * 4 + wn) * kColumns + lane % kLanes * (f32 ? 4 : 8);
#pragma unroll 2
        for (int m = 0; m < 64; m += kWave / kLanes) {
          const int at = m + lane / kLanes, mm = wm * 64 + at;
          const uint4 v = *reinterpret_cast<const uint4*>(mine + at * kPitch + lane % kLanes * 16);
          if (mm < have && col < width) {
            const size_t to = static_cast<size_t>(row0 + mm) * width + col;
            if constexpr (f32) *reinterpret_cast<uint4*>(static_cast<float*>(g.y) + to) = v;
            else *reinterpret_cast<uint4*>(static_cast<uint16_t*>(g.y) + to) = v;
          }
        }
      };
      if constexpr (SWIGLU) pass(std::false_type{});
      else if (g.out_f32) pass(std::true_type{});
      else pass(std::false_type{});
    }
  }
}

// Which kernel: the thin one takes every 16 rows (half of an expert's last ones are not
// there on average) through the expert's weights, at 8.5e12 weights a second. A tile of
// the fat one takes 1.55 us a step with up to 64 rows and 2.2 with more, on each of 256
// CUs. Measured, us of both (int4, groups of 128; rows an expert on average), the same
// inputs again and again: all but the second case's weights stay in the last-level cache:
//   experts, K, N             8         16        24        32        64        128
//   64, 2048, 2048        34,  55   55,  53   76,  52   82,  52  157,  77  300, 157
//   256, 2048, 4096      255, 389  352, 393  433, 399  531, 409  950, 546 1857, 917
//   32, 1024, 7168        27,  57   41,  55   56,  55   66,  55  123,  72  218, 122
//   8, 4096, 2048         12,  44   16,  45   21,  45   25,  46   41,  69   75,  71
//   4, 1024, 1024         11,  14   11,  15   11,  15   12,  15   11,  21   11,  21
bool few_rows(int rows, int E, int K, int n) {
  const double experts = rows < E ? rows : E, average = rows / experts;
  const double thin = (rows / 16.0 + experts / 2) * n * K / 8.5e6;
  const double tiles = ceil(experts * (average <= 128 ? 1 : average / 128 + 0.5) * ((n + 255) / 256) / 256);
  const double fat = 5 + tiles * packed_col_tiles(K) * (average <= 48 ? 1.55 : 2.2);
  return thin <= fat;
}

template <int ACT, int CODES, int PER, bool SWIGLU>
hipError_t launch(PackedGemmArgs& g, hipStream_t s) {
  if (few_rows(g.rows, g.E, g.K, g.N)) {
    const int y_tiles = packed_row_tiles(SWIGLU ? g.half : g.N);
    auto thin = [&](auto N) {
      constexpr int TILES = N, kApart = SWIGLU ? TILES / 2 : TILES;
      g.n_tiles = (y_tiles + kApart - 1) / kApart;
      packed_thin_kernel<ACT, CODES, PER, SWIGLU, TILES><<<kThinBlocks, kThinThreads, 0, s>>>(g);
    };
    // experts with rows, at most
    const long long experts = g.rows < g.E ? g.rows : g.E;
    if (experts * y_tiles >= (SWIGLU ? 4 : 8) * kThinBlocks) thin(std::integral_constant<int, 4>{});
    else thin(std::integral_constant<int, 2>{});
  } else {
    g.n_tiles = SWIGLU ? (g.half + 127) / 128 : (g.N + 255) / 256;
    packed_fat_kernel<ACT, CODES, PER, SWIGLU><<<kFatBlocks, kFatThreads, sizeof(FatShared), s>>>(g);
  }
  return hipGetLastError();
}

}  // namespace

// Tiles are counted in 32 bits; the thin kernel has the most of them.
bool packed_gemm_fits(int T, int E, int k, int n) {
  const long long tiles = (static_cast<long long>(T) * k / 16 + E) * ((n + 31) / 32);
  return n <= 1 << 24 && tiles < 1ll << 30;
}

hipError_t launch_packed_gemm(const PackedFormat& f, const void* a, const int32_t* src, const void* w,
                              const int32_t* counts, const int32_t* offsets, int T, int E, int k, int K, int n,
                              bool swiglu, void* y, int act, bool out_f32, hipStream_t s) {
  PackedGemmArgs g{static_cast<const uint16_t*>(a), src, static_cast<const unsigned char*>(w), counts, offsets, T * k,
                   src != nullptr ? T : T * k, k, E, K, n, n / 2, 0, f.scale_act, out_f32, y};
  return with_packed(f, act, [&](auto A, auto C, auto P) {
    return swiglu ? launch<A(), C(), P(), true>(g, s) : launch<A(), C(), P(), false>(g, s);
  });
}

}  // namespace moe
