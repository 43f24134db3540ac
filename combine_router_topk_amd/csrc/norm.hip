// Root-mean-square norm of the rows in front of the router, with the
// residual's addition and 8-bit output, and its gradient.
//
// Forward, per row: h = round16(x + r), rstd = 1 / sqrt(mean(h^2) + eps),
// v = h rstd g; y = round16(v), and 8-bit rows of v (see quant.hpp). The
// residual stream that is stored is the rounded one, so the norm and its
// gradient use that.
// Backward, with n = h rstd and t = dy g: dx = rstd (t - n mean(t n)) + dh,
// dgamma = sum over rows of dy n.
//
// Both are bound by HBM: the forward reads 4 and writes 5 bytes an element
// (with residual, y and q), the backward reads 6 and writes 2. A row is held
// in registers by one block, each lane owning 16-byte chunks (8 elements), so
// every input is read once; a scale block of 128 elements is 16 lanes, one
// DPP row, and its maximum never leaves the registers. At 16384 rows of 4096 in
// bf16 the forward with all outputs takes 116 us (5.2 TB/s), 8-bit rows alone
// 33.8 us, the backward without dh 75.4 us and 5 for dgamma's last sum. What a
// small batch waits for is its instructions and its rounds: with loads of 4 bytes
// under four branches each, which the compiler makes of `c < n ? p[c] : zero`,
// 8-bit rows of 4099 x 2872 took 15.8 us and not 10.5.
#include "device.hpp"
#include "launch.hpp"
#include "quant.hpp"

namespace moe {

namespace {

// Blocks of a forward launch: what the chip holds of NT threads at this
// kernel's registers (24 waves a CU; its narrow forms would fit 32), fewer if that
// evens out the rows a block takes: with a few rows left for another round, that
// round costs as much as a full one. (4099 rows of 2872 are three rounds of 1367
// blocks, 16 waves a CU.)
constexpr int norm_blocks(int T, int NT) {
  const int most = 256 * (24 * kWave / NT);
  const int rounds = (T + most - 1) / most;
  return (T + rounds - 1) / rounds;
}

// Sum over the block in a fixed order: a butterfly in each row of 16 lanes, the
// wave's rows, then the waves' sums in order. Uses one slot of `part` per wave;
// the caller puts a barrier between two uses of the same slots.
template <int NT>
__device__ __forceinline__ float block_sum(float v, float* part) {
  auto from = [](float x, auto ctrl) {
    return __uint_as_float(dpp<decltype(ctrl)::value>(__float_as_uint(x)));
  };
  v += from(v, std::integral_constant<int, kDppXor1>{});
  v += from(v, std::integral_constant<int, kDppXor2>{});
  v += from(v, std::integral_constant<int, kDppHalfMirror>{});
  v += from(v, std::integral_constant<int, kDppMirror>{});
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < kWave; i += 16) s += __uint_as_float(readlane(__float_as_uint(v), i));
  if constexpr (NT == kWave) return s;
  if ((threadIdx.x & (kWave - 1)) == 0) part[threadIdx.x / kWave] = s;
  __syncthreads();
  s = 0.0f;
#pragma unroll
  for (int i = 0; i < NT / kWave; ++i) s += part[i];
  return s;
}

// What a lane owns of a row: chunks i, i + NT, ... for lane i of the block. A
// lane past the row takes the row's last chunk (loads without branches; its
// scale block has a lane with the same values) and is left out of sums.
template <int NT, int U>
struct Chunks {
  int at[U];
  bool in[U];
  __device__ __forceinline__ explicit Chunks(int cpr) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = static_cast<int>(threadIdx.x) + u * NT;
      in[u] = c < cpr;
      at[u] = min(c, cpr - 1);
    }
  }
  __device__ __forceinline__ void load(const uint4* row, uint4 (&v)[U]) const {
#pragma unroll
    for (int u = 0; u < U; ++u) v[u] = row[at[u]];
  }
};

// The larger of two magnitudes; NaN if either is.
__device__ __forceinline__ float larger(float a, float b) { return __builtin_elementwise_maximum(a, fabsf(b)); }

// Rows blockIdx.x, blockIdx.x + gridDim.x, ... The next row is loaded before
// this one's sum goes round the block: with a block for each row a CU holds
// 64 KiB in flight and then waits (16384 rows of 4096, y alone, with the loads of
// then: 63.7 us, and 46.8 with the next row's ahead; 40.9 with today's). h_out
// and y may be x or res themselves: a lane reads its chunks of a row before it
// writes them. A lane past the row may read another's after it was written, but
// its values go nowhere.
template <int ACT, int NT, int U>
__global__ __launch_bounds__(NT) void rms_norm_kernel(
    const uint4* x, const uint4* res, const uint4* __restrict__ gamma, float eps, int T, int H,
    uint4* h_out, uint4* y, uint2* __restrict__ q, float* __restrict__ q_scale,
    float* __restrict__ rstd_out) {
  __shared__ float part[3][NT / kWave];
  const int cpr = H / 8, nb = scale_blocks(H);
  const Chunks<NT, U> own(cpr);
  uint4 xv[U], rv[U], gv[U];
  auto load = [&](int r) {
    const size_t base = static_cast<size_t>(r) * cpr;
    own.load(x + base, xv);
    if (res != nullptr) own.load(res + base, rv);
  };
  load(blockIdx.x);
  own.load(gamma, gv);
  int turn = 0;
  for (int r = blockIdx.x; r < T; r += gridDim.x, turn ^= 1) {
    const size_t row = r;
    float f[U][8];
    float ss = 0.0f;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      unpack8<ACT>(xv[u], f[u]);
      if (res != nullptr) {
        float a[8];
        unpack8<ACT>(rv[u], a);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[u][i] = keep_f32(f[u][i] + a[i]);
        const uint4 hv = round8<ACT>(f[u]);
        if (own.in[u]) h_out[row * cpr + own.at[u]] = hv;
        unpack8<ACT>(hv, f[u]);
      }
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) sum = fmaf(f[u][i], f[u][i], sum);
      ss += own.in[u] ? sum : 0.0f;
    }
    if (r + static_cast<int>(gridDim.x) < T) load(r + gridDim.x);
    ss = block_sum<NT>(ss, part[turn]);
    float rstd = 1.0f / sqrtf(ss / static_cast<float>(H) + eps);
    if (!(ss < 0x1p126f) || (ss < 0x1p-90f && eps < 0x1p-90f)) {
      // Squares that fp32 does not hold, as bf16 values may have: once more, of
      // the values brought near 1. Rare, and the same for the whole block.
      const float scale = ss < 1.0f ? 0x1p60f : 0x1p-80f;
      float again = 0.0f;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) sum = fmaf(f[u][i] * scale, f[u][i] * scale, sum);
        again += own.in[u] ? sum : 0.0f;
      }
      again = block_sum<NT>(again, part[2]);
      rstd = scale / sqrtf(again / static_cast<float>(H) + eps * scale * scale);
    }
    if (rstd_out != nullptr && threadIdx.x == 0) rstd_out[row] = rstd;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = own.at[u];
      float g[8];
      unpack8<ACT>(gv[u], g);
      float most = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        f[u][i] = keep_f32(f[u][i] * rstd * g[i]);
        most = larger(most, f[u][i]);
      }
      if (y != nullptr && own.in[u]) y[row * cpr + c] = round8<ACT>(f[u]);
      if (q != nullptr) {
        // among bits NaN is the largest magnitude
        const uint32_t bits = own.in[u] ? __float_as_uint(most) & 0x7fffffffu : 0u;
        const float s = block_scale(group_max<16>(bits));
        if (own.in[u]) {
          q[row * cpr + c] = quant8(f[u], inverse(s));
          if ((c & 15) == 0) q_scale[row * nb + c / 16] = s;
        }
      }
    }
  }
}

// Rows blockIdx.x, blockIdx.x + gridDim.x, ...; the block's sums of dy n per
// column stay in registers and end as one row of `part_dg`. dx may be dy or
// dh: a lane writes a chunk after its only read. (The
// next row's loads ahead of this row's sum brought nothing: 126.7 us against
// 125.5 at 16384 rows of 4096, 38.0 against 34.4 at rows of 1024.)
template <int ACT, int NT, int U>
__global__ __launch_bounds__(NT) void rms_norm_backward_kernel(
    const uint4* dy, const uint4* dh, const uint4* __restrict__ h,
    const uint4* __restrict__ gamma, const float* __restrict__ rstd, int T, int H,
    uint4* dx, float* __restrict__ part_dg) {
  __shared__ float part[2][NT / kWave];
  const int cpr = H / 8;
  const Chunks<NT, U> own(cpr);
  uint4 gv[U];
  float g[U][8], dg[U][8];
  own.load(gamma, gv);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    unpack8<ACT>(gv[u], g[u]);
#pragma unroll
    for (int i = 0; i < 8; ++i) dg[u][i] = 0.0f;
  }
  int turn = 0;
  for (int r = blockIdx.x; r < T; r += gridDim.x, turn ^= 1) {
    const size_t base = static_cast<size_t>(r) * cpr;
    uint4 dyv[U], hv[U], dhv[U];
    own.load(dy + base, dyv);
    own.load(h + base, hv);
    if (dh != nullptr) own.load(dh + base, dhv);
    const float rs = rstd[r];
    float t[U][8], n[U][8];
    float dot = 0.0f;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      unpack8<ACT>(dyv[u], t[u]);
      unpack8<ACT>(hv[u], n[u]);
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        n[u][i] *= rs;
        dg[u][i] += t[u][i] * n[u][i];
        t[u][i] *= g[u][i];
        sum += t[u][i] * n[u][i];
      }
      dot += own.in[u] ? sum : 0.0f;
    }
    dot = block_sum<NT>(dot, part[turn]) / static_cast<float>(H);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float d[8];
      if (dh != nullptr) {
        unpack8<ACT>(dhv[u], d);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) d[i] = 0.0f;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) d[i] = keep_f32(rs * (t[u][i] - n[u][i] * dot) + d[i]);
      if (own.in[u]) dx[base + own.at[u]] = round8<ACT>(d);
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (own.in[u]) {
      float4* o = reinterpret_cast<float4*>(part_dg + static_cast<size_t>(blockIdx.x) * H + own.at[u] * 8);
      o[0] = make_float4(dg[u][0], dg[u][1], dg[u][2], dg[u][3]);
      o[1] = make_float4(dg[u][4], dg[u][5], dg[u][6], dg[u][7]);
    }
  }
}

// dgamma[c] = sum over the blocks' rows, in a fixed order: 32 segments of
// rows, met in LDS. One block per 32 columns.
__global__ __launch_bounds__(1024) void dgamma_sum_kernel(const float* __restrict__ part_dg, int rows,
                                                          int H, float* __restrict__ dgamma) {
  __shared__ float part[32][32];
  const int col = threadIdx.x & 31, seg = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + col;
  const int per = (rows + 31) / 32;
  const int lo = seg * per, hi = min(rows, lo + per);
  float s = 0.0f;
  if (c < H) {
#pragma unroll 8
    for (int r = lo; r < hi; ++r) s += part_dg[static_cast<size_t>(r) * H + c];
  }
  part[seg][col] = s;
  __syncthreads();
  if (seg == 0 && c < H) {
    float t = 0.0f;
#pragma unroll
    for (int i = 0; i < 32; ++i) t += part[i][col];
    dgamma[c] = t;
  }
}

// Calls launch(NT, U) as compile-time values for a row of `chunks` chunks.
template <typename F>
void by_row(int chunks, F&& launch) {
  using std::integral_constant;
#define MOE_NORM_CASE(NT, U) \
  if (chunks <= NT * U) return launch(integral_constant<int, NT>{}, integral_constant<int, U>{})
  MOE_NORM_CASE(64, 1);
  MOE_NORM_CASE(128, 1);
  MOE_NORM_CASE(256, 1);
  MOE_NORM_CASE(192, 2);  // 8-bit rows of 4099 x 2872: 11.2 us with 256 x 2, 10.5 us
  MOE_NORM_CASE(256, 2);
  MOE_NORM_CASE(512, 2);
  MOE_NORM_CASE(1024, 2);
#undef MOE_NORM_CASE
}

template <typename F>
void by_act(int act, F&& launch) {
  if (act == 1) launch(std::integral_constant<int, 1>{});
  else launch(std::integral_constant<int, 2>{});
}

}  // namespace

hipError_t launch_rms_norm(const void* x, const void* residual, const void* gamma, float eps, void* h,
                           void* y, void* q, float* q_scale, float* rstd, int T, int H, int act,
                           hipStream_t s) {
  by_act(act, [&](auto A) {
    by_row(H / 8, [&](auto NT, auto U) {
      rms_norm_kernel<A, NT, U><<<norm_blocks(T, NT), int(NT), 0, s>>>(
          static_cast<const uint4*>(x), static_cast<const uint4*>(residual),
          static_cast<const uint4*>(gamma), eps, T, H, static_cast<uint4*>(h), static_cast<uint4*>(y),
          static_cast<uint2*>(q), q_scale, rstd);
    });
  });
  return hipGetLastError();
}

int rms_norm_backward_blocks(int T) { return T < 1024 ? T : 1024; }

hipError_t launch_rms_norm_backward(const void* dy, const void* dh, const void* h, const void* gamma,
                                    const float* rstd, void* dx, float* dgamma, float* ws, int T, int H,
                                    int act, hipStream_t s) {
  const int blocks = rms_norm_backward_blocks(T);
  if (blocks > 0) {
    by_act(act, [&](auto A) {
      by_row(H / 8, [&](auto NT, auto U) {
        rms_norm_backward_kernel<A, NT, U><<<blocks, int(NT), 0, s>>>(
            static_cast<const uint4*>(dy), static_cast<const uint4*>(dh), static_cast<const uint4*>(h),
            static_cast<const uint4*>(gamma), rstd, T, H, static_cast<uint4*>(dx), ws);
      });
    });
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
  }
  dgamma_sum_kernel<<<(H + 31) / 32, 1024, 0, s>>>(ws, blocks, H, dgamma);
  return hipGetLastError();
}

}  // namespace moe
