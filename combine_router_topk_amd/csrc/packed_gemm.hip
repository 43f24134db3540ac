// Products of the routed rows in 16 bits with experts' weights in 4 bits
// (packed.hpp):
//
//   z[r, n] = sum over groups g of s[e, n, g] (sum over k in g of a[r', k] code(e, n, k))
//
// for every row r of expert e's segment, r' = r or the token of the row (src[r] /
// k). The epilogue writes z in the activation format or fp32, or takes the two halves
// of the weights' rows as gate and up and writes silu(gate) up in 16 bits.
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

// First tile of each expert, with `per` rows a tile: first[E] is their number.
// A segment is cut to the rows there are.
struct Segments {
  int first[kMaxE + 1];
  int seg[kMaxE];
  int have[kMaxE];
};
template <int NT>
__device__ __forceinline__ void find_segments(const PackedGemmArgs& g, int per, Segments& sh, int* sums) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  int base = 0;
  for (int e0 = 0; e0 < g.E; e0 += NT) {
    const int e = e0 + tid;
    int tiles = 0;
    if (e < g.E) {
      const int at = min(max(g.offsets[e], 0), g.rows), have = min(max(g.counts[e], 0), g.rows - at);
      sh.seg[e] = at;
      sh.have[e] = have;
      tiles = (have + per - 1) / per * g.n_tiles;
    }
    const int upto = wave_incl_scan(tiles, lane);
    if (lane == kWave - 1) sums[wave] = upto;
    __syncthreads();
    int before = base;
    for (int w = 0; w < NT / kWave; ++w) {
      if (w < wave) before += sums[w];
      base += sums[w];
    }
    if (e < g.E) sh.first[e] = before + upto - tiles;
    __syncthreads();
  }
  if (tid == 0) sh.first[g.E] = base;
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

// A block owns 16 rows of a segment and two tiles of 16 weight rows (with SwiGLU the
// gate's and the up's beside it), its waves every fourth step of K.
template <int ACT, int CODES, int PER, bool SWIGLU>
__global__ __launch_bounds__(kThinThreads, 5) void packed_thin_kernel(PackedGemmArgs g) {
  __shared__ Segments sh;
  __shared__ int sums[kThinWaves];
  __shared__ float4 part[2][kThinWaves][2][kWave];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  find_segments<kThinThreads>(g, 16, sh, sums);

  constexpr int TB = packed_tile_bytes(PER);
  const int r = lane & 15, grp = lane >> 4;
  const int steps = packed_col_tiles(g.K), row_tiles = packed_row_tiles(g.N);
  const size_t strip = static_cast<size_t>(steps) * TB;  // a row of tiles
  const int work = sh.first[g.E];
  int turn = 0;
  for (int i = blockIdx.x; i < work; i += gridDim.x, turn ^= 1) {
    const int e = __builtin_amdgcn_readfirstlane(expert_of(sh, g.E, i));
    const int in = i - sh.first[e], m_tiles = (sh.have[e] + 15) / 16;
    const int n = in / m_tiles, m0 = (in % m_tiles) * 16;  // rows of the same weights follow each other
    const int row0 = sh.seg[e] + m0, have = min(16, sh.have[e] - m0);
    const int ta = SWIGLU ? n : 2 * n, tb = SWIGLU ? n + g.half / kPackedRows : min(2 * n + 1, row_tiles - 1);
    const unsigned char* wa = g.w + (static_cast<size_t>(e) * row_tiles + ta) * strip;
    const unsigned char* wb = g.w + (static_cast<size_t>(e) * row_tiles + tb) * strip;
    const uint16_t* row = g.a + source_row(g, row0 + min(r, have - 1)) * g.K;
    const int cols = r < have ? g.K : 0;

    v4f za = {0, 0, 0, 0}, zb = {0, 0, 0, 0};
    for (int kb = wave; kb < steps; kb += kThinWaves) {
      PackedTile<PER> a, b;
      PackedRows x;
      a.load(wa + static_cast<size_t>(kb) * TB, lane);
      b.load(wb + static_cast<size_t>(kb) * TB, lane);
      x.load(row, kb, grp, cols);
      float sa[PER], sb[PER];
      a.scales(g.scale_act, sa);
      b.scales(g.scale_act, sb);
      v4f start[PER];
      packed_start<ACT, CODES, PER>(x, start);
      packed_product<ACT, CODES, PER>(x, a, sa, start, za);
      packed_product<ACT, CODES, PER>(x, b, sb, start, zb);
    }
    part[turn][wave][0][lane] = make_float4(za[0], za[1], za[2], za[3]);
    part[turn][wave][1][lane] = make_float4(zb[0], zb[1], zb[2], zb[3]);
    __syncthreads();
    // thread tid sums value tid % 4 of lane tid / 4: row 4 (tid / 64) + tid % 4 of the
    // segment's 16, weight row (tid / 4) % 16 of the tiles
    const int c = (tid >> 6) * 4 + (tid & 3), nn = (tid >> 2) & 15;
    float sa = 0.0f, sb = 0.0f;
#pragma unroll
    for (int wv = 0; wv < kThinWaves; ++wv) {
      sa += reinterpret_cast<const float*>(part[turn][wv][0])[tid];
      sb += reinterpret_cast<const float*>(part[turn][wv][1])[tid];
    }
    if (c < have) {
      if constexpr (SWIGLU) {
        static_cast<uint16_t*>(g.y)[static_cast<size_t>(row0 + c) * g.half + ta * kPackedRows + nn] =
            static_cast<uint16_t>(pack2<ACT>(silu(sa) * sb, 0.0f));
      } else {
        const size_t at = static_cast<size_t>(row0 + c) * g.N;
        const int na = ta * kPackedRows + nn, nb = (2 * n + 1) * kPackedRows + nn;
        if (na < g.N) store_one<ACT>(g, at + na, sa);
        if (nb < g.N) store_one<ACT>(g, at + nb, sb);
      }
    }
  }
}

// ---- many rows an expert -----------------------------------------------------------

constexpr int kFatThreads = 512;
constexpr int kFatRows = 128;              // of a tile: 2 waves of 64
constexpr int kFatTiles = 4;               // of weights, a wave: 4 waves of 64 weight rows
constexpr int kFatFrags = 4;               // of 16 rows, a wave
constexpr int kFatBlocks = 256;

// Rows of a step in LDS: 256 bytes each, 16-byte chunk c of row r at place c ^ (r %
// 16), so that 16 lanes that read one chunk of 16 rows meet all banks.
struct FatShared {
  uint4 rows[2][kFatRows * 16];
  Segments seg;
  int sums[kFatThreads / kWave];
};

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
  for (int i = blockIdx.x; i < work; i += gridDim.x) {
    const int e = __builtin_amdgcn_readfirstlane(expert_of(sh.seg, g.E, i));
    const int in = i - sh.seg.first[e], m_tiles = (sh.seg.have[e] + kFatRows - 1) / kFatRows;
    const int nb = in / m_tiles, m0 = (in % m_tiles) * kFatRows;
    const int row0 = sh.seg.seg[e] + m0, have = min(kFatRows, sh.seg.have[e] - m0);
    // the wave's tiles of weights; those past the end are the last one again
    int tile[kFatTiles];
    const unsigned char* w[kFatTiles];
#pragma unroll
    for (int n = 0; n < kFatTiles; ++n) {
      if constexpr (SWIGLU) {
        const int t = nb * 8 + wn * 2 + (n & 1), last = g.half / kPackedRows - 1;
        tile[n] = t;
        w[n] = g.w + (static_cast<size_t>(e) * row_tiles + min(t, last) + (n >> 1) * (last + 1)) * strip;
      } else {
        tile[n] = nb * 16 + wn * 4 + n;
        w[n] = g.w + (static_cast<size_t>(e) * row_tiles + min(tile[n], row_tiles - 1)) * strip;
      }
    }
    const bool idle = have <= wm * 64;
    // the thread's four chunks of the rows
    const uint16_t* from[4];
    const int chunk = tid & 15;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int m = (tid >> 4) + 32 * j;
      from[j] = g.a + source_row(g, row0 + min(m, have - 1)) * g.K + chunk * 8;
    }
    uint4 rows[4];
    PackedTile<PER> t[kFatTiles];
    auto load_rows = [&](int kb) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        rows[j] = make_uint4(0, 0, 0, 0);
        if (kb * kPackedCols + chunk * 8 < g.K) rows[j] = *reinterpret_cast<const uint4*>(from[j] + kb * kPackedCols);
      }
    };
    auto load_tiles = [&](int kb) {
#pragma unroll
      for (int n = 0; n < kFatTiles; ++n) t[n].load(w[n] + static_cast<size_t>(kb) * TB, lane);
    };

    v4f acc[kFatTiles][kFatFrags];
#pragma unroll
    for (int n = 0; n < kFatTiles; ++n)
#pragma unroll
      for (int f = 0; f < kFatFrags; ++f) acc[n][f] = v4f{0, 0, 0, 0};
    __syncthreads();  // the last tile's rows have been read
    load_rows(0);
    load_tiles(0);
    for (int kb = 0; kb < steps; ++kb) {
      uint4* stage = sh.rows[kb & 1];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int m = (tid >> 4) + 32 * j;
        stage[m * 16 + (chunk ^ (m & 15))] = rows[j];
      }
      __syncthreads();
      PackedTile<PER> now[kFatTiles];
#pragma unroll
      for (int n = 0; n < kFatTiles; ++n) now[n] = t[n];
      if (kb + 1 < steps) {
        load_rows(kb + 1);
        load_tiles(kb + 1);
      }
      if (idle) continue;
      float s[kFatTiles][PER];
#pragma unroll
      for (int n = 0; n < kFatTiles; ++n) now[n].scales(g.scale_act, s[n]);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        // one 32 columns' operands at a time: more in flight would not fit the registers
        __builtin_amdgcn_sched_barrier(0);
        uint4 x[kFatFrags];
#pragma unroll
        for (int f = 0; f < kFatFrags; ++f) x[f] = stage[(wm * 64 + f * 16 + r) * 16 + ((4 * j + grp) ^ r)];
        constexpr uint32_t kMinus8 = ACT == 1 ? 0xc800c800u : 0xc100c100u;
        v4f start[kFatFrags];
#pragma unroll
        for (int f = 0; f < kFatFrags; ++f) {
          start[f] = v4f{0, 0, 0, 0};
          if constexpr (CODES == kPackedInt)
            start[f] = mfma16<ACT>(x[f], make_uint4(kMinus8, kMinus8, kMinus8, kMinus8), start[f]);
        }
#pragma unroll
        for (int n = 0; n < kFatTiles; ++n) {
          const uint32_t d = j == 0 ? now[n].codes.x : j == 1 ? now[n].codes.y : j == 2 ? now[n].codes.z : now[n].codes.w;
          const uint4 v = packed_values<ACT, CODES>(d);
#pragma unroll
          for (int f = 0; f < kFatFrags; ++f) {
            const v4f z = mfma16<ACT>(x[f], v, start[f]);
#pragma unroll
            for (int q = 0; q < 4; ++q) acc[n][f][q] = fmaf(z[q], s[n][j / kIn], acc[n][f][q]);
          }
        }
      }
    }
#pragma unroll
    for (int f = 0; f < kFatFrags; ++f) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int m = wm * 64 + f * 16 + 4 * grp + q;
        if (m >= have) continue;
        const size_t row = row0 + m;
        if constexpr (SWIGLU) {
#pragma unroll
          for (int n = 0; n < 2; ++n)
            if (tile[n] < g.half / kPackedRows)
              static_cast<uint16_t*>(g.y)[row * g.half + tile[n] * kPackedRows + r] =
                  static_cast<uint16_t>(pack2<ACT>(silu(acc[n][f][q]) * acc[n + 2][f][q], 0.0f));
        } else {
#pragma unroll
          for (int n = 0; n < kFatTiles; ++n)
            if (tile[n] * kPackedRows + r < g.N) store_one<ACT>(g, row * g.N + tile[n] * kPackedRows + r, acc[n][f][q]);
        }
      }
    }
  }
}

template <int ACT, int CODES, int PER, bool SWIGLU>
hipError_t launch(PackedGemmArgs& g, hipStream_t s) {
  if (g.rows <= 32ll * g.E) {
    g.n_tiles = SWIGLU ? g.half / kPackedRows : (packed_row_tiles(g.N) + 1) / 2;
    packed_thin_kernel<ACT, CODES, PER, SWIGLU><<<kThinBlocks, kThinThreads, 0, s>>>(g);
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
