// Gradient of the experts' weights over the routed rows:
//
//   dW[e, n, k] = sum over rows r of e's segment of dy[r, n] a[r', k],  r' = r or src[r] / k
//
// The sum runs along the rows, which both operands have outermost, so the matrix
// instructions' operands (8 rows of one column a lane) are columns of what lies in
// memory. Rows go to LDS as they are, and the LDS reads transpose: four lanes read
// 16 neighbouring values of one row, and each lane of 16 gets four rows of one
// column.
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
  int rows, a_rows, E, K, N, n_tiles, k_tiles, splits;
  uint32_t inverse;  // 2^32 / k, rounded up: i / k is the product's high half (i < 2^24, k <= 16); 0 for k = 1
  bool out_f32, add;
  void* dw;
  float* part;  // [splits][E][N][K] with more than one
};

// A step: 32 rows of dy's 128 columns and of a's 256, 16-byte chunk c of row r at place
// c ^ (r % 16): the 16 rows that one transposing read takes meet all banks.
struct Shared {
  uint4 stage[kStages][kStep * (kChunksN + kChunksK)];  // dy, then a
  int source[kWindow];
};
constexpr uint32_t kStageBytes = kStep * (kChunksN + kChunksK) * 16, kABytes = kStep * kChunksN * 16;

constexpr int kWaveBytes = kStages * kStageBytes / kWaves;  // for a wave's results

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

// Tile `in` of an expert. Neighbouring blocks go to the eight dies in turn, so each die
// takes a run of tiles, in panels of four along N: they share rows in its cache.
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
  const int e = blockIdx.x / tiles, in = blockIdx.x % tiles;
  int tn, tk;
  tile_of(g, in, tn, tk);

  // this block's share of the expert's rows, whole steps but for the last one
  const int at = min(max(g.offsets[e], 0), g.rows), have = min(max(g.counts[e], 0), g.rows - at);
  const int all_steps = (have + kStep - 1) / kStep, split = blockIdx.y;
  const int s0 = static_cast<int>(static_cast<long long>(all_steps) * split / g.splits);
  const int s1 = static_cast<int>(static_cast<long long>(all_steps) * (split + 1) / g.splits);
  if (g.add && g.splits == 1 && s0 == s1) return;

  // What this lane loads: chunk of dy's rows 4 q + lane / 16 and of a's 2 q + lane / 32, q
  // the wave's first load of a step and each fourth from there.
  const uint16_t* dy[kDyLoads];
  int dy_row[kDyLoads];
#pragma unroll
  for (int i = 0; i < kDyLoads; ++i) {
    dy_row[i] = 4 * (wave + kWaves * i) + (lane >> 4);
    const int col = tn * kTileN + ((lane & 15) ^ (dy_row[i] & 15)) * 8;
    dy[i] = g.dy + (static_cast<size_t>(at) + s0 * kStep + dy_row[i]) * g.N + col;
    if (col >= g.N) dy_row[i] = 1 << 30;
  }
  int a_col[kALoads];
#pragma unroll
  for (int i = 0; i < kALoads; ++i) {
    const int col = tk * kTileK + ((lane & 31) ^ ((2 * (wave + kWaves * i) + (lane >> 5)) & 15)) * 8;
    a_col[i] = col < g.K ? col : -1;
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
  auto load = [&](int s, uint32_t stage) {
#pragma unroll
    for (int i = 0; i < kDyLoads; ++i) {
      const void* from = s * kStep + dy_row[i] < have ? static_cast<const void*>(dy[i]) : &zeros;
      load_lds(from, lds0 + stage + i * (kWaves * 1024));
      dy[i] += static_cast<size_t>(kStep) * g.N;
    }
    const int window = (s - s0) * kStep % kWindow;
#pragma unroll
    for (int i = 0; i < kALoads; ++i) {
      const int from = sh.source[window + 2 * (wave + kWaves * i) + (lane >> 5)];
      const void* p = from >= 0 && a_col[i] >= 0
                          ? static_cast<const void*>(g.a + static_cast<size_t>(from) * g.K + a_col[i]) : &zeros;
      load_lds(p, lds0 + stage + kABytes + i * (kWaves * 1024));
    }
  };

  // where this lane reads: row 4 (lane / 16) + (lane / 4) % 4 and 16 rows further, piece
  // lane % 4 of a fragment's 16 columns
  const int wn = wave & 1, wk = wave >> 1, grp = lane >> 4;
  const int lrow = lane >> 2, piece = lane & 3;
  uint32_t at_k[kFragsK], at_n[kFragsN];
#pragma unroll
  for (int f = 0; f < kFragsK; ++f)
    at_k[f] = lds_address(&sh.stage[0][0]) + kABytes + lrow * (kChunksK * 16) + ((wk * 16 + 2 * f + (piece >> 1)) ^ lrow) * 16 + (piece & 1) * 8;
#pragma unroll
  for (int f = 0; f < kFragsN; ++f)
    at_n[f] = lds_address(&sh.stage[0][0]) + lrow * (kChunksN * 16) + ((wn * 8 + 2 * f + (piece >> 1)) ^ lrow) * 16 + (piece & 1) * 8;

  v4f acc[kFragsK][kFragsN];
#pragma unroll
  for (int i = 0; i < kFragsK; ++i)
#pragma unroll
    for (int j = 0; j < kFragsN; ++j) acc[i][j] = v4f{0, 0, 0, 0};

  // Two steps' loads are in flight while a third is multiplied.
  uint32_t now = 0, ahead = 2 * kStageBytes;
  if (s0 < s1) {
    fill(s0);
    load(s0, 0);
    if (s0 + 1 < s1) load(s0 + 1, kStageBytes);
  }
  for (int s = s0; s < s1; ++s) {
    if (s + 1 < s1) wait_loads<kDyLoads + kALoads>();
    else wait_loads<0>();
    if (s + 2 < s1) {
      if ((s + 2 - s0) % (kWindow / kStep) == 0) fill(s + 2);
      load(s + 2, ahead);
    }
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
    }
    now = now == 2 * kStageBytes ? 0 : now + kStageBytes;
    ahead = ahead == 2 * kStageBytes ? 0 : ahead + kStageBytes;
  }

  // A lane's four results of a fragment are four neighbouring k of one n, so that stores
  // straight from there would take 16 rows' lines for 32 or 64 bytes each. The wave's
  // results go through its part of the stages instead, and whole lines of a row are
  // stored: without that 64 experts of 4096 x 4096 take 1650 us.
  __syncthreads();  // all waves have read the last step
  unsigned char* const mine = reinterpret_cast<unsigned char*>(lds) + wave * kWaveBytes;
  const bool whole = g.splits > 1 || g.out_f32;  // fp32
  const size_t matrix = static_cast<size_t>(e) * g.N * g.K;
  const int k0 = tk * kTileK + wk * 128;
  auto pass = [&](auto F32) {
    constexpr bool f32 = F32;
    constexpr int kFrags = f32 ? 2 : 4;  // along N at a time
    constexpr int kLine = 128 * (f32 ? 4 : 2), kPitch = kLine + 16;
    constexpr int kLanes = kLine / 16;  // of a row
    static_assert(16 * kFrags * kPitch <= kWaveBytes, "");
#pragma unroll
    for (int j0 = 0; j0 < kFragsN; j0 += kFrags) {
#pragma unroll
      for (int j = 0; j < kFrags; ++j) {
#pragma unroll
        for (int i = 0; i < kFragsK; ++i) {
          const v4f v = acc[i][j0 + j];
          unsigned char* to = mine + (16 * j + (lane & 15)) * kPitch + (16 * i + 4 * grp) * (f32 ? 4 : 2);
          if constexpr (f32) *reinterpret_cast<float4*>(to) = make_float4(v[0], v[1], v[2], v[3]);
          else *reinterpret_cast<uint2*>(to) = make_uint2(pack2<ACT>(v[0], v[1]), pack2<ACT>(v[2], v[3]));
        }
      }
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // the wave's lanes exchange them
#pragma unroll
      for (int r = 0; r < 16 * kFrags; r += kWave / kLanes) {
        const int row = r + lane / kLanes, n = tn * kTileN + wn * 64 + 16 * j0 + row;
        const int k = k0 + lane % kLanes * (f32 ? 4 : 8);
        const uint4 v = *reinterpret_cast<const uint4*>(mine + row * kPitch + lane % kLanes * 16);
        if (n >= g.N || k >= g.K) continue;
        const size_t at = matrix + static_cast<size_t>(n) * g.K + k;
        if constexpr (!f32) {
          *reinterpret_cast<uint4*>(static_cast<uint16_t*>(g.dw) + at) = v;
        } else if (g.splits > 1) {
          *reinterpret_cast<uint4*>(g.part + static_cast<size_t>(split) * g.E * g.N * g.K + at) = v;
        } else {
          float4 f = __builtin_bit_cast(float4, v);
          float4* to = reinterpret_cast<float4*>(static_cast<float*>(g.dw) + at);
          if (g.add) {
            const float4 o = *to;
            f = make_float4(o.x + f.x, o.y + f.y, o.z + f.z, o.w + f.w);
          }
          *to = f;
        }
      }
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    }
  };
  if (whole) pass(std::true_type{});
  else pass(std::false_type{});
}

// The splits' sums, in their order.
template <int ACT>
__global__ __launch_bounds__(256) void weight_grad_sum_kernel(GradArgs g, long long fours) {
  const long long i = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= fours) return;
  const float4* part = reinterpret_cast<const float4*>(g.part);
  float4 v = part[i];
  for (int s = 1; s < g.splits; ++s) {
    const float4 p = part[s * fours + i];
    v = make_float4(v.x + p.x, v.y + p.y, v.z + p.z, v.w + p.w);
  }
  if (g.out_f32) {
    float4* to = static_cast<float4*>(g.dw) + i;
    if (g.add) {
      const float4 o = *to;
      v = make_float4(o.x + v.x, o.y + v.y, o.z + v.z, o.w + v.w);
    }
    *to = v;
  } else {
    static_cast<uint2*>(g.dw)[i] = make_uint2(pack2<ACT>(v.x, v.y), pack2<ACT>(v.z, v.w));
  }
}

long long tiles_of(int E, int K, int N) {
  return static_cast<long long>(E) * ((N + kTileN - 1) / kTileN) * ((K + kTileK - 1) / kTileK);
}
int splits_of(int T, int E, int k, int K, int N) {
  const long long blocks = tiles_of(E, K, N), steps = static_cast<long long>(T) * k / E / kStep;
  if (blocks >= 256 || steps < 8) return 1;
  const long long want = 512 / blocks, most = steps / 4;
  const long long s = want < most ? want : most;
  return static_cast<int>(s < 1 ? 1 : s > 16 ? 16 : s);
}

}  // namespace

bool weight_grad_fits(int E, int K, int N) { return tiles_of(E, K, N) < 1ll << 23; }

size_t weight_grad_ws_bytes(int T, int E, int k, int K, int N) {
  const int splits = splits_of(T, E, k, K, N);
  return splits > 1 ? static_cast<size_t>(splits) * E * N * K * sizeof(float) : 0;
}

hipError_t launch_weight_grad(const void* a, const int32_t* src, const void* dy, const int32_t* counts,
                              const int32_t* offsets, int T, int E, int k, int K, int N, bool add, void* dw, void* ws,
                              int act, bool out_f32, hipStream_t s) {
  const int splits = splits_of(T, E, k, K, N);
  const GradArgs g{static_cast<const uint16_t*>(a), static_cast<const uint16_t*>(dy), src, counts, offsets, T * k,
                   src != nullptr ? T : T * k, E, K, N, (N + kTileN - 1) / kTileN, (K + kTileK - 1) / kTileK, splits,
                   k == 1 ? 0 : static_cast<uint32_t>(((1ull << 32) + k - 1) / k), out_f32, add, dw, static_cast<float*>(ws)};
  const dim3 grid(static_cast<unsigned>(tiles_of(E, K, N)), splits);
  if (act == 1) weight_grad_kernel<1><<<grid, kThreads, sizeof(Shared), s>>>(g);
  else weight_grad_kernel<2><<<grid, kThreads, sizeof(Shared), s>>>(g);
  const hipError_t err = hipGetLastError();
  if (err != hipSuccess || splits == 1) return err;
  const long long fours = static_cast<long long>(E) * N * K / 4;
  const unsigned blocks = static_cast<unsigned>((fours + 255) / 256);
  if (act == 1) weight_grad_sum_kernel<1><<<blocks, 256, 0, s>>>(g, fours);
  else weight_grad_sum_kernel<2><<<blocks, 256, 0, s>>>(g, fours);
  return hipGetLastError();
}

}  // namespace moe
