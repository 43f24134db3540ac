// Products of the routed rows with their experts' weights, both operands in
// block-scaled 8-bit floating point (see quant.hpp):
//
//   z[r, n] = sum over blocks b of sa[r', b] sb[e, n / 128, b] *
//             (sum over k in block b of a[r', k] w[e, n, k])
//
// for every row r of expert e's segment, r' = r or the token of the row
// (src[r] / k: the dispatch's gather happens in the product's loads). One
// matrix instruction multiplies 16 x 128 codes by 128 x 16 (the format's
// scale block is the instruction's depth), so its result is exactly the inner
// sum; a multiply-add with the two scales' product accumulates it in fp32.
// The epilogue writes z in the activation format or fp32, or takes the two
// halves of the weights' rows as gate and up and writes silu(gate) up as
// 8-bit rows.
//
// The weights are the instruction's first operand, the rows its second: a
// lane then holds one row's results, so the row's scale is one value a lane,
// and four neighbouring columns an instruction.
#include "device.hpp"
#include "launch.hpp"
#include "quant.hpp"

namespace moe {

namespace {

typedef int v8i __attribute__((ext_vector_type(8)));

constexpr int kTileN = 256;        // weight rows of a tile
constexpr int kUnit = 64;          // rows of the second operand per step of MF
constexpr int kMaxUnits = 4;       // a tile has 64 to 256 rows
constexpr int kGemmThreads = 512;  // 8 waves: 2 along the weights, 4 along the rows
constexpr int kGemmBlocks = 256;   // one block a CU
constexpr int kXcds = 8;
constexpr int kDepth = 128;        // codes (bytes) of a row per step

struct GemmArgs {
  const uint8_t* a;
  const float* a_scale;
  const int32_t* src;
  const uint8_t* w;
  const float* w_scale;
  const int32_t* counts;
  const int32_t* offsets;
  int rows, a_rows, k, E, K, N;  // N: weight rows of an expert
  int half;                      // SwiGLU: N / 2
  int n_tiles;
  bool scales16;                 // rows of scales are whole, aligned 16-byte groups
  void* y;
  uint8_t* q;
  float* q_scale;
};

// LDS: two stages, each a step of K: 256 weight rows and up to 256 rows of 128
// codes; two places for scales, which come for four steps at once (a step's
// scales of 64 rows lie in 64 lines of memory, and fetched one by one in each
// step they were a third of all that the loads moved); the source rows of
// this tile and of the next.
constexpr int kRows = kMaxUnits * kUnit;
constexpr int kWBytes = kTileN * kDepth;
constexpr int kStageBytes = kWBytes + kRows * kDepth;
constexpr int kGroup = 4;  // steps whose scales are loaded together
constexpr int kScalePlace = (kMaxUnits + 1) * kUnit * kGroup;  // floats: the units' rows, the weights

struct Shared {
  unsigned char stage[2][kStageBytes];
  float scale[2][kScalePlace];
  uint32_t amax[2][kRows];
  uint32_t row[2][kRows];
  int count[kMaxE];
  int first_tile[kMaxE];
};
static_assert(sizeof(Shared) <= 160 * 1024, "one block's LDS");

// Each lane's 16 (or 4) bytes from base + offset go to LDS at byte lds + 16
// (or 4) * lane without passing through registers. Written as assembly because the
// compiler, which cannot tell the stages of the ring apart, waits for every
// such load of its own before the next LDS read; here the loop counts them
// (wait_loads). They have no output register.
// `base` and `lds` are the same in all lanes.
__device__ __forceinline__ uint64_t uniform(const void* p) {
  const uint64_t u = reinterpret_cast<uint64_t>(p);
  const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(u));
  const uint32_t hi = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(u >> 32));
  return lo | static_cast<uint64_t>(hi) << 32;
}
__device__ __forceinline__ void load_lds16(const void* base, uint32_t offset, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(
                   __builtin_amdgcn_readfirstlane(lds)), "v"(offset), "s"(uniform(base))
               : "memory");
}
__device__ __forceinline__ void load_lds4(const void* base, uint32_t offset, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, %2" ::"s"(
                   __builtin_amdgcn_readfirstlane(lds)), "v"(offset), "s"(uniform(base))
               : "memory");
}

__device__ __forceinline__ uint32_t lds_address(const void* p) {
  return static_cast<uint32_t>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) const void*)p));
}

// Waits until at most N of this wave's loads are in flight and all its LDS
// reads have returned, then for the other waves.
template <int N>
__device__ __forceinline__ void wait_loads() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

// Waits until all this wave's LDS reads have returned, then for the others'.
__device__ __forceinline__ void wait_reads() {
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// Weight row of LDS row rho (0..255) of a tile. The order inside a wave's 128
// rows gives each lane 16 neighbouring columns of the result: fragment f of a
// group of four holds rows (a / 4) 16 + 4 f + a % 4 of the group's 64.
template <bool SWIGLU>
__device__ __forceinline__ int weight_row(const GemmArgs& g, int n_tile, int rho) {
  const int wn = rho >> 7, quad = (rho >> 6) & 1, f = (rho >> 4) & 3, a = rho & 15;
  const int nn = (a >> 2) * 16 + f * 4 + (a & 3);
  if constexpr (SWIGLU) {
    const int col = min(n_tile * 128 + wn * 64 + nn, g.half - 1);
    return quad * g.half + col;
  } else {
    return min(n_tile * kTileN + wn * 128 + quad * 64 + nn, g.N - 1);
  }
}

// The 32 codes of a fragment's lane as fp16.
struct Wide { uint4 v[4]; };
__device__ __forceinline__ Wide widen(const v8i& c) {
  Wide o;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint2 lo = widen4<1>(static_cast<uint32_t>(c[2 * j])), hi = widen4<1>(static_cast<uint32_t>(c[2 * j + 1]));
    o.v[j] = make_uint4(lo.x, lo.y, hi.x, hi.y);
  }
  return o;
}

// A tile: `left` rows (64 units at most) from row m0 of the segment that starts
// at row `seg`, against the weights n_tile of expert e.
struct Tile {
  int e, seg, m0, left, n_tile, units;
};

// What a lane loads in each step: chunk `chunk` of the step's 128 bytes of
// these rows, as byte offsets (the host checked that 32 bits hold them) from
// the expert's weights and from the first row or token; and its scales. Row r
// of a stage keeps chunk c at place c ^ (r / 2 % 8), so that the 16 lanes that
// read one chunk of 16 rows together meet all LDS banks.
struct Loads {
  uint32_t w[4], a[kMaxUnits], s;
  const uint8_t* w0;
  const uint8_t* a0;
  const float* s0;
};

__device__ __forceinline__ uint32_t chunk_of(int tid) { return (tid & 7) ^ ((tid >> 4) & 7); }

// The rows of a tile counted from its first row, or from the first token,
// those behind the last valid row its copies.
__device__ __forceinline__ void fill_rows(const GemmArgs& g, const Tile& t, uint32_t* row) {
  const int tid = threadIdx.x;
  if (tid < kRows) {
    const int m = min(tid, t.left - 1);
    int r = m;
    if (g.src != nullptr) {
      const int i = g.src[t.seg + t.m0 + m];
      r = i < 0 ? 0 : min(i / g.k, g.a_rows - 1);
    }
    row[tid] = r;
  }
}

template <bool SWIGLU>
__device__ __forceinline__ Loads loads_of(const GemmArgs& g, const Tile& t, const uint32_t* row) {
  // taken anew for each tile: what follows from it is cheap, and held over the
  // tile loop it would take registers that the accumulators need
  int tid = threadIdx.x;
  asm volatile("" : "+v"(tid));
  const int lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int nbK = scale_blocks(g.K), nbN = scale_blocks(g.N);
  const uint32_t c = chunk_of(tid) * 16;
  Loads l;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    l.w[i] = static_cast<uint32_t>(weight_row<SWIGLU>(g, t.n_tile, i * 64 + (tid >> 3))) * g.K + c;
    asm volatile("" : "+v"(l.w[i]));  // a plain register: 64-bit multiplications would keep a pair
  }
#pragma unroll
  for (int i = 0; i < kMaxUnits; ++i) {
    l.a[i] = row[i * 64 + (tid >> 3)] * g.K + c;
    asm volatile("" : "+v"(l.a[i]));
  }
  const int row0 = g.src == nullptr ? t.seg + t.m0 : 0;
  l.w0 = g.w + static_cast<size_t>(t.e) * g.N * g.K;
  l.a0 = g.a + static_cast<size_t>(row0) * g.K;
  // The first waves load their unit's scales, the others the weights' (all the
  // same 16, so that every wave counts the same loads).
  if (wave < t.units) {
    l.s0 = g.a_scale + static_cast<size_t>(row0) * nbK;
    l.s = row[wave * 64 + lane] * nbK * 4;
  } else {
    const int col = lane & 15;
    l.s0 = g.w_scale + static_cast<size_t>(t.e) * nbN * nbK;
    l.s = weight_row<SWIGLU>(g, t.n_tile, (col >> 2) * 64 + (col & 3) * 4) / kScaleBlock * nbK * 4;
  }
  asm volatile("" : "+v"(l.s));
  return l;
}

// The loads of a step come in two parts: the rows' codes and the first half of
// each wave's weight rows, which the step is done with in its middle, and the
// second half. Each is loaded again as soon as nobody reads it any more. Of
// part's loads, all (-1) or one.
template <int ITEM = -1>
__device__ __forceinline__ void load_part(const GemmArgs& g, Shared& sh, const Loads& l, int units, int kb,
                                          bool first) {
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), nbK = scale_blocks(g.K);
  const uint32_t st = lds_address(sh.stage[0]) + (kb & 1) * kStageBytes + wave * 1024;
  const uint8_t* wk = l.w0 + kb * kDepth;
  const uint8_t* ak = l.a0 + kb * kDepth;
  // Chunks past the end of K: their lanes take the row's last one instead, and
  // the weights' are overwritten with zeros in LDS.
  uint32_t back = 0;
  if (kb == nbK - 1) {
    const uint32_t c = chunk_of(threadIdx.x), end = g.K / 16 - (nbK - 1) * 8;
    back = (c - min(c, end - 1)) * 16;
  }
  auto at_chunk = [&](uint32_t o) { return o - back; };
  if (first) {
    if (ITEM <= 0 && kb % kGroup == 0) {
      // With rows of whole 16-byte groups one load takes the scales of four
      // steps and lane l's lie at 4 l; else four loads take one step each and
      // step j's lie at 64 j.
      const int group = kb / kGroup;
      const uint32_t at = lds_address(sh.scale[0]) + (min(wave, units) * (kUnit * kGroup) + (group & 1) * kScalePlace) * 4;
      if (g.scales16) {
        load_lds16(l.s0 + group * kGroup, l.s, at);
      } else {
#pragma unroll
        for (int j = 0; j < kGroup; ++j) load_lds4(l.s0 + min(group * kGroup + j, nbK - 1), l.s, at + j * 256);
      }
    }
    if constexpr (ITEM < 0) {
      load_lds16(wk, at_chunk(l.w[0]), st);
      load_lds16(wk, at_chunk(l.w[2]), st + 2 * 8192);
#pragma unroll
      for (int i = 0; i < kMaxUnits; ++i)
        if (i < units) load_lds16(ak, at_chunk(l.a[i]), st + kWBytes + i * 8192);
    } else if constexpr (ITEM < 2) {
      load_lds16(wk, at_chunk(l.w[2 * ITEM]), st + 2 * ITEM * 8192);
    } else {
      load_lds16(ak, at_chunk(l.a[ITEM - 2]), st + kWBytes + (ITEM - 2) * 8192);
    }
  } else {
    if constexpr (ITEM != 1) load_lds16(wk, at_chunk(l.w[1]), st + 8192);
    if constexpr (ITEM != 0) load_lds16(wk, at_chunk(l.w[3]), st + 3 * 8192);
  }
}

// The loads that run before a tile's first step: all of step 0, the first part
// of step 1.
__device__ __forceinline__ void load_ahead(const GemmArgs& g, Shared& sh, const Loads& l, int units) {
  load_part(g, sh, l, units, 0, true);
  load_part(g, sh, l, units, 0, false);
  if (g.K > kDepth) load_part(g, sh, l, units, 1, true);
}

// The products of one tile whose first loads are under way; `then()` runs
// between the last step and the tile's output.
template <int MF, bool SWIGLU, int ACT, bool F32, typename F>
__device__ __forceinline__ void run_tile(const GemmArgs& g, Shared& sh, const Tile& t, const Loads& l, F&& then) {
  int tid = threadIdx.x;
  asm volatile("" : "+v"(tid));  // as in loads_of
  const int lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wn = wave & 1, wm = wave >> 1;
  const int col = lane & 15, grp = lane >> 4;
  const int nbK = scale_blocks(g.K);
  const int end_chunks = g.K / 16 - (nbK - 1) * 8;  // of the last step
  constexpr int kFirst = 2 + MF;  // loads of each wave in a first part, without scales
  constexpr int kGap = MF == 1 ? 1 : 2;  // instructions from one load to the next
  constexpr bool kPrecise = SWIGLU || F32;
  const int s_row = g.scales16 ? kGroup : 1, s_step = g.scales16 ? 1 : kUnit;

  v4f acc[8][MF];
#pragma unroll
  for (int n = 0; n < 8; ++n)
#pragma unroll
    for (int f = 0; f < MF; ++f) acc[n][f] = v4f{0, 0, 0, 0};
  using Frag = std::conditional_t<kPrecise, Wide, v8i>;
  Frag b[MF];
  v8i w[2];
  float s[2][MF];

  auto read_frag = [&](const unsigned char* rows, int r) {
    const uint4* p = reinterpret_cast<const uint4*>(rows) + r * 8;
    const uint4 lo = p[(2 * grp) ^ ((r >> 1) & 7)];
    const uint4 hi = p[(2 * grp + 1) ^ ((r >> 1) & 7)];
    return v8i{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
  };
  auto read_w = [&](int kb, int n) { return read_frag(sh.stage[kb & 1], wn * 128 + n * 16 + col); };
  auto read_b = [&](int kb, int f) {
    const v8i c = read_frag(sh.stage[kb & 1] + kWBytes, (f * 4 + wm) * 16 + col);
    if constexpr (kPrecise) b[f] = widen(c);
    else b[f] = c;
  };
  auto read_scales = [&](int kb) {
    const float* at = sh.scale[(kb / kGroup) & 1] + (kb % kGroup) * s_step;
    const float sw0 = at[MF * kUnit * kGroup + (wn * 8 + grp) * s_row];
    const float sw1 = at[MF * kUnit * kGroup + (wn * 8 + 4 + grp) * s_row];
#pragma unroll
    for (int f = 0; f < MF; ++f) {
      const float sa = at[f * kUnit * kGroup + (wm * 16 + col) * s_row];
      s[0][f] = sa * sw0;
      s[1][f] = sa * sw1;
    }
  };
  auto add = [&](const v4f& p, int i) {
    const int n = i / MF, f = i % MF;
#pragma unroll
    for (int q = 0; q < 4; ++q) acc[n][f][q] = fmaf(p[q], s[n >> 2][f], acc[n][f][q]);
    asm volatile("" : "+v"(acc[n][f]));  // here, not after the branches of the loads
  };
  // Step kb's codes are in LDS, and nobody reads the step before it any more.
  // Only a first part of the step after it may be in flight (scales among its
  // loads make the wait longer than it has to be); at a tile's start also the
  // stores of the tile before, so all is waited for.
  auto begin = [&](int kb) {
    if (kb > 0 && kb + 1 < nbK) wait_loads<kFirst>();
    else wait_loads<0>();
    if (kb == nbK - 1 && end_chunks < 8) {  // zeros for the weights past the end of K
      if (static_cast<int>(chunk_of(tid)) >= end_chunks)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          reinterpret_cast<uint4*>(sh.stage[kb & 1])[i * 512 + tid] = make_uint4(0, 0, 0, 0);
      wait_reads();
    }
  };
  // The first part of step kb is read: load it anew.
  // The loads are spread over the matrix instructions: issued at once, the
  // 48 that all waves issue hold up the waves for as long as they take.
  auto middle = [&](int) { wait_reads(); };
  auto first_load = [&](int kb, auto item) {
    if (kb + 2 < nbK) load_part<decltype(item)::value>(g, sh, l, MF, kb + 2, true);
  };
  auto second_load = [&](int kb, auto item) {
    if (kb + 1 < nbK) load_part<decltype(item)::value>(g, sh, l, MF, kb + 1, false);
  };
  using std::integral_constant;

  begin(0);
  second_load(0, integral_constant<int, -1>{});
  w[0] = read_w(0, 0);
#pragma unroll
  for (int f = 0; f < MF; ++f) read_b(0, f);
  read_scales(0);
  // What is loaded after matrix instruction i of a step: the first part from
  // the middle on, the second part of the next step but one at its end.
  auto spread = [&](int kb, int i) {
    const int j = i - 4 * MF;
    if (j == 0) first_load(kb, integral_constant<int, 0>{});
    if (j == 1 * kGap) first_load(kb, integral_constant<int, 1>{});
    if (j == 2 * kGap) first_load(kb, integral_constant<int, 2>{});
    if constexpr (MF > 1) if (j == 3 * kGap) first_load(kb, integral_constant<int, 3>{});
    if constexpr (MF > 2) if (j == 4 * kGap) first_load(kb, integral_constant<int, 4>{});
    if constexpr (MF > 3) if (j == 5 * kGap) first_load(kb, integral_constant<int, 5>{});
    if (i == 7 * MF) second_load(kb + 1, integral_constant<int, 0>{});
    if (i == 8 * MF - 1) second_load(kb + 1, integral_constant<int, 1>{});
  };
#pragma clang loop unroll(disable)
  for (int kb = 0; kb < nbK; ++kb) {
    // A matrix instruction's multiply-adds follow two instructions later. The
    // next step begins before this one's last weight fragment is used, so its
    // first reads run under those instructions.
    const bool more = kb + 1 < nbK;
    if constexpr (kPrecise) {
#pragma unroll
      for (int n = 0; n < 8; ++n) {
        if (n == 4) middle(kb);
        const Wide wide = widen(w[n & 1]);
        if (n < 7) {
          w[(n + 1) & 1] = read_w(kb, n + 1);
        } else if (more) {
          begin(kb + 1);
          w[0] = read_w(kb + 1, 0);
        }
        v4f p[MF];
#pragma unroll
        for (int f = 0; f < MF; ++f) p[f] = v4f{0, 0, 0, 0};
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int f = 0; f < MF; ++f) p[f] = mfma16<1>(wide.v[j], b[f].v[j], p[f]);
#pragma unroll
        for (int f = 0; f < MF; ++f) {
          add(p[f], n * MF + f);
          spread(kb, n * MF + f);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      if (more)
#pragma unroll
        for (int f = 0; f < MF; ++f) read_b(kb + 1, f);
    } else {
      v4f p[3];
#pragma unroll
      for (int n = 0; n < 8; ++n) {
        if (n == 4) middle(kb);
        if (n < 7) {
          w[(n + 1) & 1] = read_w(kb, n + 1);
        } else if (more) {
          begin(kb + 1);
          w[0] = read_w(kb + 1, 0);
        }
#pragma unroll
        for (int f = 0; f < MF; ++f) {
          const int i = n * MF + f;
          const v4f z = {0, 0, 0, 0};
          p[i % 3] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w[n & 1], b[f], z, 0, 0, 0, 0, 0, 0);
          if (i >= 2) add(p[(i - 2) % 3], i - 2);
          if (n == 7 && more) read_b(kb + 1, f);
          spread(kb, i);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
      add(p[(8 * MF - 2) % 3], 8 * MF - 2);
      add(p[(8 * MF - 1) % 3], 8 * MF - 1);
    }
    if (more) read_scales(kb + 1);
  }
  wait_reads();  // nobody reads the stages any more
  then();

  const int seg = t.seg, m0 = t.m0, left = t.left, n_tile = t.n_tile;
  if constexpr (SWIGLU) {
    const int c0 = n_tile * 128 + wn * 64 + grp * 16;
#pragma unroll
    for (int f = 0; f < MF; ++f) {
      uint32_t top = 0;
#pragma unroll
      for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float gate = acc[n][f][i], up = acc[n + 4][f][i];
          const float h = gate / (1.0f + expf(-gate)) * up;
          acc[n][f][i] = h;
          top = umax(top, __float_as_uint(h) & 0x7fffffffu);
        }
      if (c0 >= g.half) top = 0;
      top = umax(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), 16, kWave)));
      top = umax(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), 32, kWave)));
      if (grp == 0) sh.amax[wn][(f * 4 + wm) * 16 + col] = top;
    }
    wait_reads();
    const int nbH = scale_blocks(g.half);
#pragma unroll
    for (int f = 0; f < MF; ++f) {
      const int m = (f * 4 + wm) * 16 + col;
      const float s = block_scale(umax(sh.amax[0][m], sh.amax[1][m]));
      if (m >= left) continue;
      const size_t r = static_cast<size_t>(seg) + m0 + m;
      if (c0 < g.half) {
        const float inv = 1.0f / s;
        uint32_t o[4];
#pragma unroll
        for (int n = 0; n < 4; ++n)
          o[n] = quant4(acc[n][f][0], acc[n][f][1], acc[n][f][2], acc[n][f][3], inv);
        *reinterpret_cast<uint4*>(g.q + r * g.half + c0) = make_uint4(o[0], o[1], o[2], o[3]);
      }
      if (wn == 0 && grp == 0) g.q_scale[r * nbH + n_tile] = s;
    }
  } else {
#pragma unroll
    for (int f = 0; f < MF; ++f) {
      const int m = (f * 4 + wm) * 16 + col;
      if (m >= left) continue;
      const size_t r = static_cast<size_t>(seg) + m0 + m;
#pragma unroll
      for (int c8 = 0; c8 < 4; ++c8) {
        const int n = n_tile * kTileN + wn * 128 + (c8 >> 1) * 64 + grp * 16 + (c8 & 1) * 8;
        if (n >= g.N) continue;
        const v4f lo = acc[c8 * 2][f], hi = acc[c8 * 2 + 1][f];
        if constexpr (F32) {
          float4* o = reinterpret_cast<float4*>(static_cast<float*>(g.y) + r * g.N + n);
          o[0] = make_float4(lo[0], lo[1], lo[2], lo[3]);
          o[1] = make_float4(hi[0], hi[1], hi[2], hi[3]);
        } else {
          *reinterpret_cast<uint4*>(static_cast<uint16_t*>(g.y) + r * g.N + n) =
              make_uint4(pack2<ACT>(lo[0], lo[1]), pack2<ACT>(lo[2], lo[3]), pack2<ACT>(hi[0], hi[1]),
                         pack2<ACT>(hi[2], hi[3]));
        }
      }
    }
  }
}

// A segment of R rows is cut into ceil(R / 256) tiles of whole 64-row units,
// as even as they go, so a segment just past a multiple of 256 rows costs one
// unit more and not one tile more.
template <int UNITS>
__device__ __forceinline__ int tiles_of(int rows) { return (rows + UNITS * kUnit - 1) / (UNITS * kUnit); }

template <bool SWIGLU, int ACT, bool F32>
__global__ __launch_bounds__(kGemmThreads, 2) void expert_gemm_kernel(GemmArgs g) {
  constexpr int kUnits = SWIGLU || F32 ? 3 : 4;
  extern __shared__ __align__(16) char smem[];
  Shared& sh = *reinterpret_cast<Shared*>(smem);
  const int tid = threadIdx.x, lane = tid & 63;

  // every expert's rows and first tile. Counts are cut so that they never add
  // up to more than the rows there are, whatever the table holds.
  if (tid < kWave) {
    const int per = (g.E + kWave - 1) / kWave, e0 = lane * per;
    int sum = 0;
    for (int e = e0; e < min(g.E, e0 + per); ++e) sum += min(max(0, g.counts[e]), g.rows - sum);
    // partial sums stay below 2^30: 64 lanes of at most 2^24 rows
    int before = wave_incl_scan(sum, lane) - sum;
    int tiles = 0;
    for (int e = e0; e < min(g.E, e0 + per); ++e) {
      const int c = max(0, min(max(0, g.counts[e]), g.rows - before));
      before += c;
      sh.count[e] = c;
      tiles += tiles_of<kUnits>(c);
    }
    int first = wave_incl_scan(tiles, lane) - tiles;
    for (int e = e0; e < min(g.E, e0 + per); ++e) {
      sh.first_tile[e] = first;
      first += tiles_of<kUnits>(sh.count[e]);
    }
  }
  __syncthreads();

  // Each XCD takes one run of tiles, and its blocks neighbouring ones: an
  // expert's weights and rows then pass through one L2.
  const int total = __builtin_amdgcn_readfirstlane(sh.first_tile[g.E - 1] + tiles_of<kUnits>(sh.count[g.E - 1])) *
                    g.n_tiles;  // the host checked that it fits
  const int per_xcd = (total + kXcds - 1) / kXcds;
  const int first = static_cast<int>(blockIdx.x % kXcds) * per_xcd;
  const int last = min(total, first + per_xcd);
  auto find = [&](int t) {
    const int mt = t / g.n_tiles;
    int lo = 0, hi = g.E;  // the last expert whose first tile is at most mt
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (__builtin_amdgcn_readfirstlane(sh.first_tile[mid]) <= mt) lo = mid;
      else hi = mid;
    }
    Tile x;
    x.e = lo;
    const int rows = __builtin_amdgcn_readfirstlane(sh.count[x.e]), tiles = tiles_of<kUnits>(rows);
    const int in = t - __builtin_amdgcn_readfirstlane(sh.first_tile[x.e]) * g.n_tiles;
    const int m_tile = in % tiles;
    x.n_tile = in / tiles;
    const int units = (rows + kUnit - 1) / kUnit, base = units / tiles, more = units % tiles;
    const int u0 = m_tile * base + min(m_tile, more);
    x.units = base + (m_tile < more ? 1 : 0);
    x.m0 = u0 * kUnit;
    // a segment that would end past the rows is moved back inside
    x.seg = __builtin_amdgcn_readfirstlane(max(0, min(g.offsets[x.e], g.rows - rows)));
    x.left = min(rows, (u0 + x.units) * kUnit) - x.m0;
    return x;
  };
  int t = first + static_cast<int>(blockIdx.x / kXcds);
  if (t >= last) return;
  Tile cur = find(t);
  fill_rows(g, cur, sh.row[0]);
  __syncthreads();
  Loads l = loads_of<SWIGLU>(g, cur, sh.row[0]);
  load_ahead(g, sh, l, cur.units);
  for (int turn = 1;; turn ^= 1) {
    // the next tile's rows are looked up while this one runs, and its first
    // loads run under this one's output
    t += kGemmBlocks / kXcds;
    const bool more = t < last;
    Tile next = cur;
    if (more) {
      next = find(t);
      fill_rows(g, next, sh.row[turn]);
    }
    Loads nl = l;
    auto then = [&] {
      if (more) {
        nl = loads_of<SWIGLU>(g, next, sh.row[turn]);
        load_ahead(g, sh, nl, next.units);
      }
    };
    switch (cur.units) {
      case 1: run_tile<1, SWIGLU, ACT, F32>(g, sh, cur, l, then); break;
      case 2: run_tile<2, SWIGLU, ACT, F32>(g, sh, cur, l, then); break;
      case 3: run_tile<3, SWIGLU, ACT, F32>(g, sh, cur, l, then); break;
      default: run_tile<kUnits, SWIGLU, ACT, F32>(g, sh, cur, l, then); break;
    }
    if (!more) break;
    cur = next;
    l = nl;
  }
}

}  // namespace

bool expert_gemm_fits(int T, int E, int k, int K, int n, bool gather) {
  const long long rows = static_cast<long long>(T) * k, most = 1ll << 32;
  const long long tiles = rows / (3 * kUnit) + 1 + (rows < E ? rows : E);
  // with SwiGLU a tile holds 128 columns of each half: one more at most
  const long long across = (static_cast<long long>(n) + kTileN - 1) / kTileN + 1;
  return (gather ? static_cast<long long>(T) : 256) * K < most && static_cast<long long>(n) * K < most &&
         tiles * across < (1ll << 30);
}

static bool whole_groups(const float* a_scale, const float* w_scale, int K) {
  const uintptr_t both = reinterpret_cast<uintptr_t>(a_scale) | reinterpret_cast<uintptr_t>(w_scale);
  return scale_blocks(K) % kGroup == 0 && both % 16 == 0;
}

hipError_t launch_expert_gemm(const void* a, const float* a_scale, const int32_t* src, const void* w,
                              const float* w_scale, const int32_t* counts, const int32_t* offsets,
                              int T, int E, int k, int K, int N, void* y, int act, bool out_f32,
                              hipStream_t s) {
  GemmArgs g{};
  g.a = static_cast<const uint8_t*>(a);
  g.a_scale = a_scale;
  g.src = src;
  g.w = static_cast<const uint8_t*>(w);
  g.w_scale = w_scale;
  g.counts = counts;
  g.offsets = offsets;
  g.rows = T * k;
  g.a_rows = src ? T : T * k;
  g.k = k;
  g.E = E;
  g.K = K;
  g.N = N;
  g.scales16 = whole_groups(a_scale, w_scale, K);
  g.n_tiles = (N + kTileN - 1) / kTileN;
  g.y = y;
  if (out_f32) expert_gemm_kernel<false, 1, true><<<kGemmBlocks, kGemmThreads, sizeof(Shared), s>>>(g);
  else if (act == 1) expert_gemm_kernel<false, 1, false><<<kGemmBlocks, kGemmThreads, sizeof(Shared), s>>>(g);
  else expert_gemm_kernel<false, 2, false><<<kGemmBlocks, kGemmThreads, sizeof(Shared), s>>>(g);
  return hipGetLastError();
}

hipError_t launch_expert_gemm_swiglu(const void* a, const float* a_scale, const int32_t* src, const void* w,
                                     const float* w_scale, const int32_t* counts, const int32_t* offsets,
                                     int T, int E, int k, int K, int I, void* q, float* q_scale,
                                     hipStream_t s) {
  GemmArgs g{};
  g.a = static_cast<const uint8_t*>(a);
  g.a_scale = a_scale;
  g.src = src;
  g.w = static_cast<const uint8_t*>(w);
  g.w_scale = w_scale;
  g.counts = counts;
  g.offsets = offsets;
  g.rows = T * k;
  g.a_rows = src ? T : T * k;
  g.k = k;
  g.E = E;
  g.K = K;
  g.N = 2 * I;
  g.half = I;
  g.scales16 = whole_groups(a_scale, w_scale, K);
  g.n_tiles = (I + 127) / 128;
  g.q = static_cast<uint8_t*>(q);
  g.q_scale = q_scale;
  expert_gemm_kernel<true, 1, false><<<kGemmBlocks, kGemmThreads, sizeof(Shared), s>>>(g);
  return hipGetLastError();
}

}  // namespace moe
