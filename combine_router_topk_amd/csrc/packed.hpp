// Weights in 4 bits with a 16-bit scale for each group of 32, 64 or 128
// columns, in tiles of 16 rows by 128 columns. A tile is 1024 bytes of codes, lane
// (r, g) = (lane % 16, lane / 16) of a wave its 16 bytes at 16 (16 g + r), and 16
// rows of 128 / group scales: a wave reads a tile as one run of memory. Dword j of
// a lane's chunk holds columns 32 j + 8 g .. + 7 of row r, so the four lanes of a
// row hold 32 neighbouring columns in dword j and one matrix instruction stays
// inside a group of any size.
//
// Codes become 16-bit numbers in registers, exactly:
//   integers -8 .. 7 (as 0 .. 15): nibble 2 b is column b, nibble 2 b + 1 column 4 +
//     b. Masked and, for the odd ones, shifted, they are bytes 0 .. 15, which are
//     the e4m3 numbers code 2^-9; the conversion multiplies by 2^9. The 8 comes off
//     in the sum: the products start from -8 times the sum of the row's values, one
//     matrix instruction with a constant operand, which all of a wave's tiles
//     share. 7 instructions for 8 codes.
//   e2m1 (0, .5, 1, 1.5, 2, 3, 4, 6 and their negatives): nibble i is column i, one
//     conversion for two. 4 instructions for 8 codes.
// A group's products are summed by the matrix cores in fp32, and the sum is
// multiplied by the scale in fp32.
#pragma once

#include "device.hpp"
#include "launch.hpp"
#include "quant.hpp"

namespace moe {

constexpr int kPackedInt = MOE_PACKED_INT, kPackedE2m1 = MOE_PACKED_E2M1;
constexpr int kPackedRows = 16, kPackedCols = 128, kPackedCodes = 1024;
__host__ __device__ constexpr int packed_tile_bytes(int per) { return kPackedCodes + 32 * per; }
__host__ __device__ constexpr int packed_row_tiles(int rows) { return (rows + kPackedRows - 1) / kPackedRows; }
__host__ __device__ constexpr int packed_col_tiles(int cols) { return (cols + kPackedCols - 1) / kPackedCols; }

// 8 columns' codes as 8 values in 16 bits; integer codes without the 8 taken off.
template <int ACT, int CODES>
__device__ __forceinline__ uint4 packed_values(uint32_t d) {
  if constexpr (CODES == kPackedInt) {
    const int lo = static_cast<int>(d & 0x0f0f0f0fu), hi = static_cast<int>((d >> 4) & 0x0f0f0f0fu);
    if constexpr (ACT == 1)
      return make_uint4(__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 512.0f, false)),
                        __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 512.0f, true)),
                        __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 512.0f, false)),
                        __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 512.0f, true)));
    else
      return make_uint4(__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 512.0f, false)),
                        __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 512.0f, true)),
                        __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 512.0f, false)),
                        __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 512.0f, true)));
  } else {
    if constexpr (ACT == 1)
      return make_uint4(__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(d, 1.0f, 0)),
                        __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(d, 1.0f, 1)),
                        __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(d, 1.0f, 2)),
                        __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(d, 1.0f, 3)));
    else
      return make_uint4(__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, 1.0f, 0)),
                        __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, 1.0f, 1)),
                        __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, 1.0f, 2)),
                        __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, 1.0f, 3)));
  }
}

// One of two scales as fp32. Both formats' conversions and a selection: a branch on
// the format for each scale costs more than they do.
__device__ __forceinline__ float packed_scale(int act, uint32_t two, int high) {
  const uint32_t b = high ? two >> 16 : two & 0xffffu;
  const float h = f16_to_f32(b), f = bf16_to_f32(b);
  return act == 1 ? h : f;
}

// A lane's part of a tile: its 32 codes and its row's scales as they lie there.
template <int PER>
struct PackedTile {
  uint4 codes;
  uint32_t scale[PER == 4 ? 2 : 1];

  __device__ __forceinline__ void load(const unsigned char* tile, int lane) {
    codes = *reinterpret_cast<const uint4*>(tile + lane * 16);
    const unsigned char* s = tile + kPackedCodes + (lane & 15) * (2 * PER);
    if constexpr (PER == 1) {
      scale[0] = *reinterpret_cast<const uint16_t*>(s);
    } else if constexpr (PER == 2) {
      scale[0] = *reinterpret_cast<const uint32_t*>(s);
    } else {
      const uint2 v = *reinterpret_cast<const uint2*>(s);
      scale[0] = v.x, scale[1] = v.y;
    }
  }
  __device__ __forceinline__ void scales(int act, float (&f)[PER]) const {
#pragma unroll
    for (int p = 0; p < PER; ++p) f[p] = packed_scale(act, scale[p >> 1], p & 1);
  }
};

// The rows of the other operand, 16 of them, at a tile's columns: lane (r, g)
// holds columns 32 j + 8 g .. + 7 of row r in v[j]. Nothing is read from `cols` on.
struct PackedRows {
  uint4 v[4];
  __device__ __forceinline__ void load(const uint16_t* row, int kb, int grp, int cols) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int c = kb * kPackedCols + 32 * j + 8 * grp;
      v[j] = make_uint4(0, 0, 0, 0);
      if (c < cols) v[j] = *reinterpret_cast<const uint4*>(row + c);
    }
  }
};

// What a group's products start from: -8 times the sum of the row's values.
template <int ACT, int CODES, int PER>
__device__ __forceinline__ void packed_start(const PackedRows& x, v4f (&start)[PER]) {
  constexpr uint32_t kMinus8 = ACT == 1 ? 0xc800c800u : 0xc100c100u;
#pragma unroll
  for (int p = 0; p < PER; ++p) {
    start[p] = v4f{0, 0, 0, 0};
    if constexpr (CODES == kPackedInt)
#pragma unroll
      for (int j = 0; j < 4 / PER; ++j)
        start[p] = mfma16<ACT>(x.v[p * (4 / PER) + j], make_uint4(kMinus8, kMinus8, kMinus8, kMinus8), start[p]);
  }
}

// acc += rows x tile: lane (r, g) gets rows 4 g .. 4 g + 3 against the tile's row r.
template <int ACT, int CODES, int PER>
__device__ __forceinline__ void packed_product(const PackedRows& x, const PackedTile<PER>& t, const float (&s)[PER],
                                               const v4f (&start)[PER], v4f& acc) {
  const uint32_t d[4] = {t.codes.x, t.codes.y, t.codes.z, t.codes.w};
#pragma unroll
  for (int p = 0; p < PER; ++p) {
    v4f z = start[p];
#pragma unroll
    for (int j = 0; j < 4 / PER; ++j) {
      const int i = p * (4 / PER) + j;
      z = mfma16<ACT>(x.v[i], packed_values<ACT, CODES>(d[i]), z);
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) acc[q] = fmaf(z[q], s[p], acc[q]);
  }
}

// Calls f with the constants of a format and an activation type.
template <typename F>
inline auto with_packed(const PackedFormat& fmt, int act, F&& f) {
  auto per = [&](auto A, auto C) {
    if (fmt.per == 1) return f(A, C, std::integral_constant<int, 1>{});
    if (fmt.per == 2) return f(A, C, std::integral_constant<int, 2>{});
    return f(A, C, std::integral_constant<int, 4>{});
  };
  auto codes = [&](auto A) {
    if (fmt.codes == kPackedInt) return per(A, std::integral_constant<int, kPackedInt>{});
    return per(A, std::integral_constant<int, kPackedE2m1>{});
  };
  if (act == 1) return codes(std::integral_constant<int, 1>{});
  return codes(std::integral_constant<int, 2>{});
}

}  // namespace moe
