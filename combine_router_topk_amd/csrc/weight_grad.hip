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

constexpr int kThreads = 512;  // 8 waves: 4 along N, 2 along K
constexpr int kTile = 256;     // weights of a block: 256 x 256
constexpr int kStep = 32;      // rows of a step
constexpr int kFragsK = 8, kFragsN = 4;  // of a wave: 128 x 64

struct GradArgs {
  const uint16_t* a;
  const uint16_t* dy;
  const int32_t* src;
  const int32_t* counts;
  const int32_t* offsets;
  int rows, a_rows, k, E, K, N, n_tiles, k_tiles, splits;
  bool out_f32, add;
  void* dw;
  float* part;  // [splits][E][N][K] with more than one
};

// A step of one operand: 32 rows of 512 bytes, 16-byte chunk c of row r at place c ^
// (r % 16): the 16 rows that one transposing read takes meet all banks.
struct Stage {
  uint4 v[kStep * 32];
};
struct Shared {
  Stage dy[2], a[2];
};

typedef short v4s __attribute__((ext_vector_type(4)));
__device__ __forceinline__ uint2 read_transposed(uint32_t at) {
  const auto p = reinterpret_cast<__attribute__((address_space(3))) v4s*>(at);
  return __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(p));
}
__device__ __forceinline__ uint32_t lds_address(const void* p) {
  return static_cast<uint32_t>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) const void*)p));
}

template <int ACT>
__global__ __launch_bounds__(kThreads, 2) void weight_grad_kernel(GradArgs g) {
  extern __shared__ __align__(16) char lds[];
  Shared& sh = *reinterpret_cast<Shared*>(lds);
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int tiles = g.n_tiles * g.k_tiles;
  const int e = blockIdx.x / tiles, in = blockIdx.x % tiles;
  const int tn = in % g.n_tiles, tk = in / g.n_tiles;

  // this block's share of the expert's rows, whole steps but for the last one
  const int at = min(max(g.offsets[e], 0), g.rows), have = min(max(g.counts[e], 0), g.rows - at);
  const int all_steps = (have + kStep - 1) / kStep, split = blockIdx.y;
  const int s0 = static_cast<int>(static_cast<long long>(all_steps) * split / g.splits);
  const int s1 = static_cast<int>(static_cast<long long>(all_steps) * (split + 1) / g.splits);
  if (g.add && g.splits == 1 && s0 == s1) return;

  const int chunk = tid & 31, row = tid >> 5;  // and row + 16
  const bool dy_on = tn * kTile + chunk * 8 < g.N, a_on = tk * kTile + chunk * 8 < g.K;
  const uint16_t* dy0 = g.dy + static_cast<size_t>(at) * g.N + tn * kTile + chunk * 8;
  const uint16_t* a0 = g.a + tk * kTile + chunk * 8;
  uint4 next_dy[2], next_a[2];
  int pair[2];
  auto load_pairs = [&](int s) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = s * kStep + row + 16 * i;
      pair[i] = g.src != nullptr && r < have ? g.src[at + r] : 0;
    }
  };
  auto load = [&](int s) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = s * kStep + row + 16 * i;
      next_dy[i] = next_a[i] = make_uint4(0, 0, 0, 0);
      if (r < have) {
        const size_t from = g.src == nullptr ? at + r : pair[i] < 0 ? 0 : min(pair[i] / g.k, g.a_rows - 1);
        if (dy_on) next_dy[i] = *reinterpret_cast<const uint4*>(dy0 + static_cast<size_t>(r) * g.N);
        if (a_on) next_a[i] = *reinterpret_cast<const uint4*>(a0 + from * g.K);
      }
    }
  };

  // where this lane reads: row 4 (lane / 16) + (lane / 4) % 4 and 16 rows further, piece
  // lane % 4 of a fragment's 16 columns
  const int wn = wave & 3, wk = wave >> 2, grp = lane >> 4;
  const int lrow = lane >> 2, piece = lane & 3;
  uint32_t at_k[kFragsK], at_n[kFragsN];
#pragma unroll
  for (int f = 0; f < kFragsK; ++f)
    at_k[f] = lds_address(&sh.a[0]) + lrow * 512 + ((wk * 16 + 2 * f + (piece >> 1)) ^ lrow) * 16 + (piece & 1) * 8;
#pragma unroll
  for (int f = 0; f < kFragsN; ++f)
    at_n[f] = lds_address(&sh.dy[0]) + lrow * 512 + ((wn * 8 + 2 * f + (piece >> 1)) ^ lrow) * 16 + (piece & 1) * 8;

  v4f acc[kFragsK][kFragsN];
#pragma unroll
  for (int i = 0; i < kFragsK; ++i)
#pragma unroll
    for (int j = 0; j < kFragsN; ++j) acc[i][j] = v4f{0, 0, 0, 0};

  if (s0 < s1) {
    load_pairs(s0);
    load(s0);
    load_pairs(s0 + 1);
  }
  for (int s = s0; s < s1; ++s) {
    const int stage = (s - s0) & 1;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = row + 16 * i, place = r * 32 + (chunk ^ row);
      sh.dy[stage].v[place] = next_dy[i];
      sh.a[stage].v[place] = next_a[i];
    }
    __syncthreads();
    if (s + 1 < s1) {
      load(s + 1);
      load_pairs(s + 2);
    }
    const uint32_t off = stage * sizeof(Stage);
    uint4 n[kFragsN];
#pragma unroll
    for (int f = 0; f < kFragsN; ++f) {
      const uint2 lo = read_transposed(at_n[f] + off), hi = read_transposed(at_n[f] + off + 16 * 512);
      n[f] = make_uint4(lo.x, lo.y, hi.x, hi.y);
    }
#pragma unroll
    for (int i = 0; i < kFragsK; ++i) {
      const uint2 lo = read_transposed(at_k[i] + off), hi = read_transposed(at_k[i] + off + 16 * 512);
      const uint4 k = make_uint4(lo.x, lo.y, hi.x, hi.y);
#pragma unroll
      for (int j = 0; j < kFragsN; ++j) acc[i][j] = mfma16<ACT>(k, n[j], acc[i][j]);
    }
  }

  // a lane's four results of a fragment are four neighbouring k of one n
#pragma unroll
  for (int j = 0; j < kFragsN; ++j) {
    const int n = tn * kTile + wn * 64 + j * 16 + (lane & 15);
    if (n >= g.N) continue;
    const size_t line = (static_cast<size_t>(e) * g.N + n) * g.K;
#pragma unroll
    for (int i = 0; i < kFragsK; ++i) {
      const int k = tk * kTile + wk * 128 + i * 16 + grp * 4;
      if (k >= g.K) continue;
      float4 v = make_float4(acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]);
      if (g.splits > 1) {
        *reinterpret_cast<float4*>(g.part + static_cast<size_t>(split) * g.E * g.N * g.K + line + k) = v;
      } else if (g.out_f32) {
        float4* to = reinterpret_cast<float4*>(static_cast<float*>(g.dw) + line + k);
        if (g.add) {
          const float4 o = *to;
          v = make_float4(o.x + v.x, o.y + v.y, o.z + v.z, o.w + v.w);
        }
        *to = v;
      } else {
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(g.dw) + line + k) =
            make_uint2(pack2<ACT>(v.x, v.y), pack2<ACT>(v.z, v.w));
      }
    }
  }
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
  return static_cast<long long>(E) * ((N + kTile - 1) / kTile) * ((K + kTile - 1) / kTile);
}
int splits_of(int T, int E, int k, int K, int N) {
  const long long blocks = tiles_of(E, K, N), steps = static_cast<long long>(T) * k / E / kStep;
  if (blocks >= 256 || steps < 8) return 1;
  const long long want = 512 / blocks, most = steps / 4;
  const long long s = want < most ? want : most;
  return static_cast<int>(s < 1 ? 1 : s > 16 ? 16 : s);
}

}  // namespace

bool weight_grad_fits(int E, int K, int N) { return tiles_of(E, K, N) < 1ll << 22; }

size_t weight_grad_ws_bytes(int T, int E, int k, int K, int N) {
  const int splits = splits_of(T, E, k, K, N);
  return splits > 1 ? static_cast<size_t>(splits) * E * N * K * sizeof(float) : 0;
}

hipError_t launch_weight_grad(const void* a, const int32_t* src, const void* dy, const int32_t* counts,
                              const int32_t* offsets, int T, int E, int k, int K, int N, bool add, void* dw, void* ws,
                              int act, bool out_f32, hipStream_t s) {
  const int splits = splits_of(T, E, k, K, N);
  const GradArgs g{static_cast<const uint16_t*>(a), static_cast<const uint16_t*>(dy), src, counts, offsets, T * k,
                   src != nullptr ? T : T * k, k, E, K, N, (N + kTile - 1) / kTile, (K + kTile - 1) / kTile, splits,
                   out_f32, add, dw, static_cast<float*>(ws)};
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
