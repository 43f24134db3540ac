// Products of the routed rows with their experts' weights, both operands in
// block-scaled 8-bit floating point (see quant.hpp):
//
//   z[r, n] = sum over blocks b of sa[r', b] sb[e, n / 128, b] *
//             (sum over k in block b of a[r', k] w[e, n, k])
//
// for every row r of expert e's segment, r' = r or the token of the row
// (src[r] / k: the dispatch's gather happens in the product's loads). One
// matrix instruction multiplies 16 x 128 codes by 128 x 16 (the format's
// scale block is the instruction's depth), so its result is the inner sum; a
// multiply-add with the two scales' product accumulates it in fp32.
// That instruction cuts products off at 2^-13 of a power of two that the
// largest of eight neighbours reaches: a group of eight loses at most 7 2^-13 of
// its largest product, 8.5e-4. Normal codes lose 1.2e-5 of a sum; one large
// product beside seven small ones of one sign in every group lost 8.0e-4, which
// is 0.20 of half a step of a bf16 result and 1.64 of an fp16 one. So it is used
// for bf16 results alone, and not for those of a caller who asks for exact sums.
// These, fp16 and fp32 results, and the SwiGLU's, whose fp32 scales show it, come from the codes widened to fp16 instead, exact products
// summed in fp32, at half the rate (EXACT below).
// The epilogue writes z in the activation format or fp32, or takes the two
// halves of the weights' rows as gate and up and writes silu(gate) up as
// 8-bit rows.
//
// What bounds it: with few rows an expert the weights' bytes (gate and up of 256
// experts, 4096 x 2048, 8 rows each: 768 us, 5.6 TB/s). With hundreds of rows
// several things. A block per CU holds 256 weight rows by up to 256 rows, which
// takes half of its registers: a step of 128 codes takes 64 KiB from L2, 192 KiB
// of LDS reads (8 waves of 128 x 64) and 256 matrix instructions with 1024
// multiply-adds. 32768 rows of one expert, K = N = 4096: matrix cores are busy
// 55 % of the cycles, and power takes a part of the clock (475 us at 1.99 GHz with
// random codes, 424 us at 2.32 GHz with codes of zero). The same rows in 64
// segments: 590 us in a row, 1.87 PFLOP/s (a library product of 8192^3 in 8 bits
// reaches 2.66). With K = 1024 there are 8 steps a tile, power makes no
// difference (272 and 269 us, skewed top-6 of 16384 tokens), and 9 of a tile's 25
// us pass without matrix instructions, in its look-up, its first loads and its
// stores. In fp16 the widening adds 5.5 conversions to each 3 matrix
// instructions, and the whole runs at 1.08 PFLOP/s (a bf16 library product: 1.30):
// 22 us against 33 for 2042 rows in 8 segments of 1424 x 2872, 592 against 984 for
// the 64 segments, 280 against 430 for the skewed ones.
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

// LDS: stages, each a step of K (256 weight rows and the rows' codes), two of a
// tile of 3 or 4 units and three of a smaller one; two places for scales, which
// come for four steps at once (a step's scales of 64 rows lie in 64 lines of
// memory, and fetched one by one in each step they were a third of all that the
// loads moved); the source rows of the next tile.
constexpr int kWBytes = kTileN * kDepth;
constexpr int kABytes = kUnit * kDepth;  // of one unit
constexpr int kGroup = 4;                // steps whose scales are loaded together
__host__ __device__ constexpr int stage_bytes(int units) { return kWBytes + units * kABytes; }

template <int UNITS, bool AMAX>
struct Shared {
  static constexpr int kUnits = UNITS;
  static constexpr int kRows = UNITS * kUnit;
  static constexpr int kStages = 2 * stage_bytes(UNITS) > 3 * stage_bytes(2) ? 2 * stage_bytes(UNITS) : 3 * stage_bytes(2);
  static constexpr int kScalePlace = (UNITS + 1) * kUnit * kGroup;  // floats: the units' rows, the weights
  unsigned char stages[kStages];
  float scale[2][kScalePlace];
  uint32_t amax[AMAX ? 2 * kRows : 1];
  uint32_t row[kRows];
  int first_tile[kMaxE];
};

// Each lane's 16 (or 4) bytes from base + offset go to LDS at byte lds + 16
// (or 4) * lane without passing through registers. Written as assembly because the
// compiler, which cannot tell the stages of the ring apart, waits for every
// such load of its own before the next LDS read; here the loop counts them
// (wait_loads). They have no output register.
// `base` and `lds` are the same in all lanes. The scalar registers that hold the
// base may just have been written by readfirstlane, and a memory instruction may
// read them only 5 wait states later, which the compiler does not insert in here.
// (A scalar move of the base in between, which may read it at once, in place of
// the wait takes the same time: 605 us for 32768 rows in 64 segments of 4096 x 4096.)
__device__ __forceinline__ uint64_t uniform(const void* p) {
  const uint64_t u = reinterpret_cast<uint64_t>(p);
  const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(u));
  const uint32_t hi = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(u >> 32));
  return lo | static_cast<uint64_t>(hi) << 32;
}
// The LDS address goes in as M0 itself, so that the compiler writes it and knows
// what it holds.
template <int PLUS = 0>  // added to lds
__device__ __forceinline__ void load_lds16(const void* base, uint32_t offset, uint32_t lds) {
  asm volatile("s_nop 4\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(offset), "s"(uniform(base)),
               "{m0}"(__builtin_amdgcn_readfirstlane(lds) + PLUS)
               : "memory");
}
__device__ __forceinline__ void load_lds4(const void* base, uint32_t offset, uint32_t lds) {
  asm volatile("s_nop 4\n\tglobal_load_lds_dword %0, %1" ::"v"(offset), "s"(uniform(base)),
               "{m0}"(__builtin_amdgcn_readfirstlane(lds))
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
// rows makes what a lane stores whole and its neighbours' follow: rows a of a
// fragment go in fours to the four groups of lanes, and with SwiGLU the four
// fragments of each half give a lane 16 neighbouring columns (16 bytes of
// codes), else each two fragments 8 (16 bytes in 16 bits).
template <bool SWIGLU>
__device__ __forceinline__ int weight_row(const GemmArgs& g, int n_tile, int rho) {
  const int wn = rho >> 7, quad = (rho >> 6) & 1, f = (rho >> 4) & 3, a = rho & 15;
  if constexpr (SWIGLU) {
    const int col = min(n_tile * 128 + wn * 64 + (a >> 2) * 16 + f * 4 + (a & 3), g.half - 1);
    return quad * g.half + col;
  } else {
    const int nn = (f >> 1) * 32 + (a >> 2) * 8 + (f & 1) * 4 + (a & 3);
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

// Of the matrix instructions of a step, in their order: weight fragment and row
// fragment; and which of three places a weight fragment is held in.
template <int MF>
constexpr int order_n(int i) { return i < 6 * MF ? i / MF : 6 + (i & 1); }
template <int MF>
constexpr int order_f(int i) { return i < 6 * MF ? i % MF : (i - 6 * MF) / 2; }
constexpr int place(int n) { return n == 1 || n == 4 || n == 6 ? 1 : n == 2 || n == 7 ? 2 : 0; }

// A tile: `left` rows (64 units at most) from row m0 of the segment that starts
// at row `seg`, against the weights n_tile of expert e.
struct Tile {
  int e, seg, m0, left, n_tile, units;
};

// What a lane loads in each step: chunk `chunk` of the step's 128 bytes of
// these rows, as byte offsets (the host checked that 32 bits hold them) from
// the expert's weights and from the first row or token; and its scales.
struct Loads {
  uint32_t w[4], a[kMaxUnits], s;
  const uint8_t* w0;
  const uint8_t* a0;
  const float* s0;
};

// Row r of a stage keeps 16-byte chunk c at place c ^ swizzle(r): a 128-bit LDS
// read takes 16 lanes at a time, four by four from two neighbouring groups of
// 16 lanes (which read chunks c and c ^ 2 here), and with this the 16 meet all
// 64 banks.
__device__ __forceinline__ int swizzle(int r) {
  const int i = r >> 1;
  return ((i & 1) << 1) | ((i >> 2) & 1) | ((((i >> 1) ^ (i >> 2)) & 1) << 2);
}
__device__ __forceinline__ uint32_t chunk_of(int tid) { return (tid & 7) ^ swizzle(tid >> 3); }

// The thread's number, from its wave's in a scalar register. Computed anew
// wherever it is asked for: held over the tile loop, it and what follows from it
// would take registers that the accumulators need.
__device__ __forceinline__ int thread_of(int wave) {
  uint32_t zero = 0;
  asm volatile("" : "+s"(zero));
  return wave * kWave + static_cast<int>(__builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, zero)));
}

// The rows of a tile counted from its first row, or from the first token,
// those behind the last valid row its copies.
__device__ __forceinline__ void fill_rows(const GemmArgs& g, int wave, const Tile& t, uint32_t* row, int rows) {
  const int tid = thread_of(wave);
  if (tid < rows) {
    const int m = min(tid, t.left - 1);
    int r = m;
    if (g.src != nullptr) {
      const int i = g.src[t.seg + t.m0 + m];
      r = i < 0 ? 0 : min(i / g.k, g.a_rows - 1);
    }
    row[tid] = r;
  }
}

template <int UNITS, bool SWIGLU>
__device__ __forceinline__ Loads loads_of(const GemmArgs& g, int wave, const Tile& t, const uint32_t* row) {
  const int tid = thread_of(wave), lane = tid & 63;
  const int nbK = scale_blocks(g.K), nbN = scale_blocks(g.N);
  const uint32_t c = chunk_of(tid) * 16;
  Loads l;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    l.w[i] = static_cast<uint32_t>(weight_row<SWIGLU>(g, t.n_tile, i * 64 + (tid >> 3))) * g.K + c;
    asm volatile("" : "+v"(l.w[i]));  // a plain register: 64-bit multiplications would keep a pair
  }
#pragma unroll
  for (int i = 0; i < UNITS; ++i) {
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

// Chunks past the end of K: in the last step their lanes take the row's last
// one instead, and the weights' are overwritten with zeros in LDS. How far back
// that is:
__device__ __forceinline__ uint32_t past_end(const GemmArgs& g, int wave) {
  const uint32_t c = chunk_of(thread_of(wave)), end = g.K / 16 - (scale_blocks(g.K) - 1) * 8;
  return (c - min(c, end - 1)) * 16;
}

template <int UNITS>
__device__ __forceinline__ void step_back(Loads& l, uint32_t by) {
#pragma unroll
  for (int i = 0; i < 4; ++i) l.w[i] -= by;
#pragma unroll
  for (int i = 0; i < UNITS; ++i) l.a[i] -= by;
}

// The scales of steps 4 group .. 4 group + 3. With rows of whole 16-byte groups
// one load takes them and lane l's lie at 4 l; else four loads take one step
// each and step j's lie at 64 j.
template <typename S>
__device__ __forceinline__ void load_scales(const GemmArgs& g, int wave, S& sh, const Loads& l, int units,
                                            int group) {
  const uint32_t at = lds_address(sh.scale[0]) +
                      (min(wave, units) * (kUnit * kGroup) + (group & 1) * S::kScalePlace) * 4;
  if (g.scales16) {
    load_lds16(l.s0 + group * kGroup, l.s, at);
  } else {
#pragma unroll
    for (int j = 0; j < kGroup; ++j)
      load_lds4(l.s0 + min(group * kGroup + j, scale_blocks(g.K) - 1), l.s, at + j * 256);
  }
}

// The loads that run before a tile's first step: all of steps 0 and 1.
template <typename S>
__device__ __forceinline__ void load_ahead(const GemmArgs& g, int wave, S& sh, Loads& l, int units) {
  const int nbK = scale_blocks(g.K);
  load_scales(g, wave, sh, l, units, 0);
  for (int kb = 0; kb < min(nbK, 2); ++kb) {
    const uint32_t st = lds_address(sh.stages) + kb * stage_bytes(units) + wave * 1024;
    if (kb == nbK - 1) step_back<S::kUnits>(l, past_end(g, wave));
#pragma unroll
    for (int i = 0; i < 4; ++i) load_lds16(l.w0 + kb * kDepth, l.w[i], st + i * 8192);
#pragma unroll
    for (int i = 0; i < S::kUnits; ++i)
      if (i < units) load_lds16(l.a0 + kb * kDepth, l.a[i], st + kWBytes + i * 8192);
  }
}

// The products of one tile whose first loads are under way; `then()` runs
// between the last step and the tile's output.
//
// With two stages, the rows' codes and the first half of each wave's weight rows
// are read by a step's middle, the second half by its end; each is then loaded
// anew for the next step but one. With three, the step before's stage is loaded
// for the step after next, and there is no barrier in the middle: such tiles
// have little to do in a step and wait for memory (2042 rows in 8 segments at
// K = 1424: 1.2 us a step of two units with two stages).
//
// THIN: a tile of at most 16 rows, as in decode. All waves take the same rows,
// and each two fragments of the weights (with SwiGLU one of the gate's and the
// up's beside it) where three of four would have none of the rows: gate and up of
// 8 rows for each of 256 experts 786 -> 757 us in one run (757 to 790 on other
// cards), of 8 rows in all 42.5 -> 25.1 us.
template <int MF, bool SWIGLU, int ACT, bool F32, bool EXACT, bool THIN, typename S, typename F>
__device__ __forceinline__ void run_tile(const GemmArgs& g, int wave, S& sh, const Tile& t, Loads& l,
                                         F&& then) {
  const int tid = thread_of(wave), lane = tid & 63;
  const int wn = wave & 1, wm = wave >> 1;
  const int col = lane & 15, grp = lane >> 4;
  const int nbK = scale_blocks(g.K);
  const int end_chunks = g.K / 16 - (nbK - 1) * 8;  // of the last step
  constexpr bool kThree = MF <= 2;  // stages
  // loads of each wave that may be in flight when a step begins, without scales
  constexpr int kInFlight = kThree ? 4 + MF : 2 + MF;
  constexpr int kStage = stage_bytes(MF), UNITS = S::kUnits;
  constexpr int kFrags = THIN ? 2 : 8;  // of the weights, a wave
  static_assert(!THIN || MF == 1, "one unit");

  v4f acc[kFrags][MF];
#pragma unroll
  for (int n = 0; n < kFrags; ++n)
#pragma unroll
    for (int f = 0; f < MF; ++f) acc[n][f] = v4f{0, 0, 0, 0};
  using Frag = std::conditional_t<EXACT, Wide, v8i>;
  Frag b[MF];
  float s[2][MF];

  // this lane's two chunks in the stage of the current step, of weight and of
  // row fragments
  const unsigned char* const stage0 = sh.stages;
  // a wave's first fragment, and how far the next one is
  const int w_row = wn * 128 + col + (THIN ? wm * (SWIGLU ? 16 : 32) : 0);
  constexpr int kNext = THIN && SWIGLU ? 64 * 128 : 16 * 128;
  const int a_row = col + (THIN ? 0 : wm * 16);
  const int w_lo = w_row * 128 + ((2 * grp) ^ swizzle(col)) * 16;
  const int w_hi = w_row * 128 + ((2 * grp + 1) ^ swizzle(col)) * 16;
  const int w_to_a = kWBytes + (a_row - w_row) * 128;
  int now = 0;  // the current step's stage, in bytes
  int wl = w_lo, wh = w_hi, al = wl + w_to_a, ah = wh + w_to_a;
  auto read2 = [&](int lo, int hi) {
    const uint4 x = *reinterpret_cast<const uint4*>(stage0 + lo), y = *reinterpret_cast<const uint4*>(stage0 + hi);
    return v8i{(int)x.x, (int)x.y, (int)x.z, (int)x.w, (int)y.x, (int)y.y, (int)y.z, (int)y.w};
  };
  auto read_w = [&](int n) { return read2(wl + n * kNext, wh + n * kNext); };
  // Rows past the segment's end are zeros where all 16 of a fragment are: they
  // cost the least power, and no reads (gate and up of 8 rows for each of 256
  // experts: 866 -> 797 us).
  const bool last_empty = !THIN && ((MF - 1) * 4 + wm) * 16 >= t.left;
  auto read_b = [&](int f, Frag& to) {
    if (f == MF - 1 && last_empty) return;
    const v8i c = read2(al + f * 8192, ah + f * 8192);
    if constexpr (EXACT) to = widen(c);
    else to = c;
  };
  constexpr int kLast = (kThree ? 2 : 1) * kStage;
  auto next_stage = [&] {
    now = now == kLast ? 0 : now + kStage;
    wl = w_lo + now;
    wh = w_hi + now;
    al = wl + w_to_a;
    ah = wh + w_to_a;
  };
  const int s_row = g.scales16 ? kGroup : 1, s_step = g.scales16 ? 1 : kUnit;
  const int sa_at = a_row * s_row, sw_at = MF * kUnit * kGroup + (wn * 8 + grp) * s_row;
  // One multiply-add a value takes the scales' product, which has to be finite
  // (the header says so): one after the other would take two.
  auto read_scales = [&](int kb) {
    const float* at = sh.scale[0] + ((kb / kGroup) & 1) * S::kScalePlace + (kb % kGroup) * s_step;
    const float sw0 = at[sw_at], sw1 = at[sw_at + 4 * s_row];
#pragma unroll
    for (int f = 0; f < MF; ++f) {
      const float sa = at[f * kUnit * kGroup + sa_at];
      s[0][f] = sa * sw0;
      s[1][f] = sa * sw1;
    }
  };
  auto add1 = [&](const v4f& p, int i, int q) {
    const int n = i / MF, f = i % MF;
    acc[n][f][q] = fmaf(p[q], s[n >> 2][f], acc[n][f][q]);
  };
  auto add = [&](const v4f& p, int i) {
#pragma unroll
    for (int q = 0; q < 4; ++q) add1(p, i, q);
    asm volatile("" : "+v"(acc[i / MF][i % MF]));  // here, not after the branches of the loads
  };

  // where the loads of step kb + 2 come from and the stage they go to
  const uint8_t* wk = l.w0 + 2 * kDepth;
  const uint8_t* ak = l.a0 + 2 * kDepth;
  const uint32_t lds0 = lds_address(sh.stages) + wave * 1024;
  uint32_t st = lds0 + (kThree ? 2 * kStage : 0);
  auto prepare = [&](int kb) {
    if (kb + 3 == nbK) step_back<UNITS>(l, past_end(g, wave));
    if ((kb + 2) % kGroup == 0) load_scales(g, wave, sh, l, MF, (kb + 2) / kGroup);
  };
  auto weight_load = [&](auto item) {
    constexpr int I = decltype(item)::value;
    load_lds16<I * 8192>(wk, l.w[I], st);
  };
  auto row_load = [&](auto item) {
    constexpr int I = decltype(item)::value;
    if constexpr (I < MF) load_lds16<kWBytes + I * 8192>(ak, l.a[I], st);
  };
  auto loaded = [&] {
    wk += kDepth;
    ak += kDepth;
    st = st == lds0 + kLast ? lds0 : st + kStage;
  };
  using std::integral_constant;
  using C0 = integral_constant<int, 0>;
  using C1 = integral_constant<int, 1>;
  using C2 = integral_constant<int, 2>;
  using C3 = integral_constant<int, 3>;
  // The loads are spread over a step's matrix instructions: issued at once they
  // would hold up every wave. With two stages the first part comes once everyone
  // has read the step's, before the next step begins, and the second after
  // that; with three all come before it. The waits count on this order.
  auto spread = [&](int kb, int i) {
    if constexpr (kThree) {
      if (i == 0) prepare(kb), weight_load(C0{});
      if (i == 1 * MF) weight_load(C1{});
      if (i == 2 * MF) weight_load(C2{});
      if (i == 3 * MF) weight_load(C3{});
      if (i == 4 * MF) row_load(C0{});
      if (i == 5 * MF) row_load(C1{});
      if (i == 6 * MF - 1) loaded();
    } else {
      constexpr int kStart = 3 * MF;
      static_assert(kStart + 2 * (MF + 1) < 6 * MF, "the first part is on its way before the next step begins");
      const int j = i - kStart;
      if (j == 0) prepare(kb), weight_load(C0{});
      if (j == 2) weight_load(C2{});
      if (j == 4) row_load(C0{});
      if (j == 6) row_load(C1{});
      if (j == 8) row_load(C2{});
      if (j == 10) row_load(C3{});
      if (i == 7 * MF) weight_load(C1{});
      if (i == 8 * MF - 1) weight_load(C3{}), loaded();
    }
  };
  auto zero_tail = [&](int kb) {  // zeros for the weights past the end of K
    if (kb == nbK - 1 && end_chunks < 8) {
      const int me = thread_of(wave);
      if (static_cast<int>(chunk_of(me)) >= end_chunks) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          reinterpret_cast<uint4*>(sh.stages + now)[i * 512 + me] = make_uint4(0, 0, 0, 0);
      }
      wait_reads();
    }
  };

  // One step. LOAD: there is a step kb + 2 to load; MORE: there is a step kb + 1.
  // That one begins before this one's last two weight fragments are used, so its
  // first reads run under those instructions: its codes are in LDS and nobody reads
  // this step any more; only the step after it, or its first part, may be in
  // flight (scales among its loads make the wait longer than it has to be).
  v8i w[3];
  Wide wide[2];
  auto step = [&](int kb, auto load, auto has_next) {
    constexpr bool LOAD = decltype(load)::value, MORE = decltype(has_next)::value;
    auto next = [&] {
      if constexpr (MORE) {
        wait_loads<LOAD ? kInFlight : 0>();
        next_stage();
        if constexpr (!LOAD) zero_tail(kb + 1);
      }
    };
    if constexpr (THIN) {
      if constexpr (LOAD) {
        prepare(kb);
        weight_load(C0{}), weight_load(C1{}), weight_load(C2{}), weight_load(C3{}), row_load(C0{});
        loaded();
      }
      v4f p[2] = {v4f{0, 0, 0, 0}, v4f{0, 0, 0, 0}};
      if constexpr (EXACT) {
#pragma unroll
        for (int n = 0; n < 2; ++n) wide[n] = widen(w[n]);
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int n = 0; n < 2; ++n) p[n] = mfma16<1>(wide[n].v[j], b[0].v[j], p[n]);
      } else {
#pragma unroll
        for (int n = 0; n < 2; ++n)
          p[n] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w[n], b[0], p[n], 0, 0, 0, 0, 0, 0);
      }
      next();
      if constexpr (MORE) {
        w[0] = read_w(0);
        w[1] = read_w(1);
        read_b(0, b[0]);
      }
#pragma unroll
      for (int n = 0; n < 2; ++n) {
#pragma unroll
        for (int q = 0; q < 4; ++q) acc[n][0][q] = fmaf(p[n][q], s[SWIGLU ? n : 0][0], acc[n][0][q]);
        asm volatile("" : "+v"(acc[n][0]));  // fp32, not rounded to 16 bits in the same instruction
      }
    } else if constexpr (EXACT) {
      // Under the matrix instructions of fragment n run the multiply-adds of
      // n - 1 and the widening of n + 1, whose codes were read under n - 1.
      v4f p[2][MF];
#pragma unroll
      for (int n = 0; n < 8; ++n) {
        if (!kThree && n == 3) wait_reads();  // the step's first part is read
        if (n == 6) next();
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int f = 0; f < MF; ++f) {
            const int q = j * MF + f;
            const v4f z = {0, 0, 0, 0};
            p[n & 1][f] = mfma16<1>(wide[n & 1].v[j], b[f].v[j], j == 0 ? z : p[n & 1][f]);
            if (n > 0) {
              add1(p[(n - 1) & 1][q / 4], (n - 1) * MF + q / 4, q % 4);
              if (q % 4 == 3) asm volatile("" : "+v"(acc[n - 1][q / 4]));
            }
            if (f == 0 && (n < 7 || MORE)) {
              const v8i& c = w[(n + 1) & 1];
              const uint2 lo = widen4<1>(static_cast<uint32_t>(c[2 * j]));
              const uint2 hi = widen4<1>(static_cast<uint32_t>(c[2 * j + 1]));
              wide[(n + 1) & 1].v[j] = make_uint4(lo.x, lo.y, hi.x, hi.y);
            }
            if (j == 0 && f == 0) {
              if (n < 6) w[n & 1] = read_w(n + 2);
              else if constexpr (MORE) w[n & 1] = read_w(n - 6);
            }
            if constexpr (LOAD) {
              const int i = n * MF + f;
              if (j == 3) spread(kb, i);
            }
            __builtin_amdgcn_sched_barrier(0);
          }
      }
      if constexpr (MORE)
#pragma unroll
        for (int f = 0; f < MF; ++f) read_b(f, b[f]);
#pragma unroll
      for (int f = 0; f < MF; ++f) add(p[1][f], 7 * MF + f);
    } else {
      // A matrix instruction's multiply-adds follow two instructions later. The
      // last two fragments go through the rows' fragments together, so that the
      // next step's take their places over twice as many instructions (16384
      // rows, top-2 of 64 experts, K = N = 4096: 612 -> 598 us).
      v4f p[3];
#pragma unroll
      for (int i = 0; i < 8 * MF; ++i) {
        const int n = order_n<MF>(i), f = order_f<MF>(i);
        if (i == 3 * MF && !kThree) wait_reads();  // the step's first part is read
        if (i == 6 * MF) next();
        if (i % MF == 0 && n < 5) w[place(n + 1)] = read_w(n + 1);
        if (i == 5 * MF) w[place(6)] = read_w(6), w[place(7)] = read_w(7);
        if constexpr (MORE) if (i == 6 * MF) w[0] = read_w(0);
        const v4f z = {0, 0, 0, 0};
        p[i % 3] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w[place(n)], b[f], z, 0, 0, 0, 0, 0, 0);
        if (i >= 2) add(p[(i - 2) % 3], order_n<MF>(i - 2) * MF + order_f<MF>(i - 2));
        if constexpr (MORE) if (n == 7) read_b(f, b[f]);
        if constexpr (LOAD) spread(kb, i);
        __builtin_amdgcn_sched_barrier(0);
      }
      add(p[(8 * MF - 2) % 3], 7 * MF - 1);
      add(p[(8 * MF - 1) % 3], 8 * MF - 1);
    }
    if constexpr (MORE) read_scales(kb + 1);
  };

  // all of the tile's first loads, and the stores of the tile before
  wait_loads<0>();
  zero_tail(0);
#pragma unroll
  for (int f = 0; f < MF; ++f) {
    b[f] = Frag{};
    read_b(f, b[f]);
  }
  w[0] = read_w(0);
  if constexpr (THIN) {
    w[1] = read_w(1);
  } else if constexpr (EXACT) {
    wide[0] = widen(w[0]);
    w[1] = read_w(1);
  }
  read_scales(0);
  using std::bool_constant;
  int kb = 0;
#pragma clang loop unroll(disable)
  for (; kb + 2 < nbK; ++kb) step(kb, bool_constant<true>{}, bool_constant<true>{});
  if (kb + 1 < nbK) {
    step(kb, bool_constant<false>{}, bool_constant<true>{});
    ++kb;
  }
  step(kb, bool_constant<false>{}, bool_constant<false>{});
  wait_reads();  // nobody reads the stages any more
  then();

  const int seg = t.seg, m0 = t.m0, left = t.left, n_tile = t.n_tile;
  if constexpr (THIN && SWIGLU) {
    uint32_t* amax = sh.amax;
    const int c0 = n_tile * 128 + wn * 64 + grp * 16 + wm * 4;
    float h[4];
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      h[i] = silu(acc[0][0][i]) * acc[1][0][i];
      top = umax(top, __float_as_uint(h[i]) & 0x7fffffffu);
    }
    if (c0 >= g.half) top = 0;
    top = umax(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), 16, kWave)));
    top = umax(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), 32, kWave)));
    if (grp == 0) amax[wave * 16 + col] = top;
    wait_reads();
    if (col >= left) return;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = umax(top, amax[i * 16 + col]);
    const float s = block_scale(top);
    const size_t r = static_cast<size_t>(seg) + m0 + col;
    if (c0 < g.half)
      *reinterpret_cast<uint32_t*>(g.q + r * g.half + c0) = quant4(h[0], h[1], h[2], h[3], inverse(s));
    if (wave == 0 && grp == 0) g.q_scale[r * scale_blocks(g.half) + n_tile] = s;
  } else if constexpr (SWIGLU) {
    uint32_t* amax = sh.amax;
    const int c0 = n_tile * 128 + wn * 64 + grp * 16;
#pragma unroll
    for (int f = 0; f < MF; ++f) {
      uint32_t top = 0;
#pragma unroll
      for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float gate = acc[n][f][i], up = acc[n + 4][f][i];
          const float h = silu(gate) * up;
          acc[n][f][i] = h;
          top = umax(top, __float_as_uint(h) & 0x7fffffffu);
        }
      if (c0 >= g.half) top = 0;
      top = umax(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), 16, kWave)));
      top = umax(top, static_cast<uint32_t>(__shfl_xor(static_cast<int>(top), 32, kWave)));
      if (grp == 0) amax[wn * S::kRows + (f * 4 + wm) * 16 + col] = top;
    }
    wait_reads();
    const int nbH = scale_blocks(g.half);
#pragma unroll
    for (int f = 0; f < MF; ++f) {
      const int m = (f * 4 + wm) * 16 + col;
      const float s = block_scale(umax(amax[m], amax[S::kRows + m]));
      if (m >= left) continue;
      const size_t r = static_cast<size_t>(seg) + m0 + m;
      if (c0 < g.half) {
        const float inv = inverse(s);
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
      const int m = f * 64 + a_row;
      if (m >= left) continue;
      const size_t r = static_cast<size_t>(seg) + m0 + m;
#pragma unroll
      for (int c8 = 0; c8 < kFrags / 2; ++c8) {
        const int n = n_tile * kTileN + wn * 128 + (THIN ? wm : c8) * 32 + grp * 8;
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

// A segment of R rows is cut into tiles of whole 64-row units, `cap` at most
// and as even as they go, so a segment just past a whole number of tiles costs
// one unit more and not one tile more.
__device__ __forceinline__ int tiles_of(int rows, int cap) {
  return ((rows + kUnit - 1) / kUnit + cap - 1) / cap;
}

template <bool SWIGLU, int ACT, bool F32, bool EXACT>
__global__ __launch_bounds__(kGemmThreads, 2) void expert_gemm_kernel(GemmArgs g) {
  constexpr int kUnits = EXACT ? 3 : kMaxUnits;
  extern __shared__ __align__(16) char smem[];
  using S = Shared<kUnits, SWIGLU>;
  static_assert(sizeof(S) <= 160 * 1024, "one block's LDS");
  S& sh = *reinterpret_cast<S*>(smem);
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);

  // Every expert's first tile. Counts are cut so that they never add up to more
  // than the rows there are, whatever the table holds.
  for (int e = tid; e < g.E; e += kGemmThreads) sh.first_tile[e] = max(0, g.counts[e]);
  __syncthreads();
  if (tid < kWave) {
    const int per = (g.E + kWave - 1) / kWave, e0 = lane * per, e1 = min(g.E, e0 + per);
    int sum = 0;
    for (int e = e0; e < e1; ++e) sum += min(sh.first_tile[e], g.rows - sum);
    // partial sums stay below 2^30: 64 lanes of at most 2^24 rows
    const int before = wave_incl_scan(sum, lane) - sum;
    // Units a tile: as many as give the shortest run of rounds. A round of
    // tiles of u units takes about 2 u + 3 (a step of 4, 2 and 1 units takes
    // 1.5, 0.85 and 0.6 us), and there are 256 tiles in it.
    int cap = 1, best = 0x7fffffff;
    for (int u = kUnits; u >= 1; --u) {
      int tiles = 0, left = g.rows - before;
      for (int e = e0; e < e1; ++e) {
        const int c = max(0, min(sh.first_tile[e], left));
        left -= c;
        tiles += tiles_of(c, u);
      }
      tiles = wave_sum(tiles);
      const long long rounds = (static_cast<long long>(tiles) * g.n_tiles + kGemmBlocks - 1) / kGemmBlocks;
      const int cost = static_cast<int>(min(rounds * (2 * u + 3), 0x7ffffffell));
      if (cost < best) best = cost, cap = u;
    }
    int tiles = 0, left = g.rows - before;
    for (int e = e0; e < e1; ++e) {
      const int c = max(0, min(sh.first_tile[e], left));
      left -= c;
      sh.first_tile[e] = tiles;
      tiles += tiles_of(c, cap);
    }
    const int first = wave_incl_scan(tiles, lane) - tiles;
    for (int e = e0; e < e1; ++e) sh.first_tile[e] += first;
    if (lane == kWave - 1) {
      sh.row[0] = first + tiles;
      sh.row[1] = cap;
    }
  }
  __syncthreads();

  // Each XCD takes one run of tiles, and its blocks neighbouring ones: an
  // expert's weights and rows then pass through one L2.
  const int total = __builtin_amdgcn_readfirstlane(sh.row[0]) * g.n_tiles;  // the host checked that it fits
  const int cap = __builtin_amdgcn_readfirstlane(sh.row[1]);
  const int per_xcd = (total + kXcds - 1) / kXcds;
  const int first = static_cast<int>(blockIdx.x % kXcds) * per_xcd;
  const int last = min(total, first + per_xcd);
  auto find = [&](int t) {
    const int mt = t / g.n_tiles;
    int lo = 0, hi = g.E;  // the last expert whose first tile is at most mt: one with rows
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (__builtin_amdgcn_readfirstlane(sh.first_tile[mid]) <= mt) lo = mid;
      else hi = mid;
    }
    Tile x;
    x.e = lo;
    const int rows = __builtin_amdgcn_readfirstlane(min(max(1, g.counts[x.e]), g.rows));
    const int tiles = tiles_of(rows, cap);
    const int in = t - __builtin_amdgcn_readfirstlane(sh.first_tile[x.e]) * g.n_tiles;
    const int m_tile = in % tiles;
    x.n_tile = min(in / tiles, g.n_tiles - 1);
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
  __syncthreads();  // everyone has read the table's totals
  fill_rows(g, wave, cur, sh.row, S::kRows);
  __syncthreads();
  Loads l = loads_of<kUnits, SWIGLU>(g, wave, cur, sh.row);
  load_ahead(g, wave, sh, l, cur.units);
  for (;;) {
    // the next tile's rows are looked up while this one runs, and its first
    // loads run under this one's output
    t += kGemmBlocks / kXcds;
    const bool more = t < last;
    Tile next = cur;
    if (more) {
      next = find(t);
      wait_reads();  // everyone has read this tile's rows
      fill_rows(g, wave, next, sh.row, S::kRows);
    }
    Loads nl = l;
    auto then = [&] {
      if (more) {
        nl = loads_of<kUnits, SWIGLU>(g, wave, next, sh.row);
        load_ahead(g, wave, sh, nl, next.units);
      }
    };
    switch (cur.units) {
      case 1:
        if (cur.left <= 16) run_tile<1, SWIGLU, ACT, F32, EXACT, true>(g, wave, sh, cur, l, then);
        else run_tile<1, SWIGLU, ACT, F32, EXACT, false>(g, wave, sh, cur, l, then);
        break;
      case 2: run_tile<2, SWIGLU, ACT, F32, EXACT, false>(g, wave, sh, cur, l, then); break;
      case 3: run_tile<3, SWIGLU, ACT, F32, EXACT, false>(g, wave, sh, cur, l, then); break;
      default: run_tile<kUnits, SWIGLU, ACT, F32, EXACT, false>(g, wave, sh, cur, l, then); break;
    }
    if (!more) break;
    cur = next;
    l = nl;
  }
}

}  // namespace

bool expert_gemm_fits(int T, int E, int k, int K, int n, bool gather) {
  const long long rows = static_cast<long long>(T) * k, most = 1ll << 32;
  const long long tiles = rows / kUnit + 1 + (rows < E ? rows : E);
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
                              bool exact, hipStream_t s) {
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
  constexpr size_t kLds = sizeof(Shared<kMaxUnits, false>), kLds3 = sizeof(Shared<3, false>);
  if (out_f32) expert_gemm_kernel<false, 1, true, true><<<kGemmBlocks, kGemmThreads, kLds3, s>>>(g);
  else if (act == 1) expert_gemm_kernel<false, 1, false, true><<<kGemmBlocks, kGemmThreads, kLds3, s>>>(g);
  else if (exact) expert_gemm_kernel<false, 2, false, true><<<kGemmBlocks, kGemmThreads, kLds3, s>>>(g);
  else expert_gemm_kernel<false, 2, false, false><<<kGemmBlocks, kGemmThreads, kLds, s>>>(g);
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
  expert_gemm_kernel<true, 1, false, true><<<kGemmBlocks, kGemmThreads, sizeof(Shared<3, true>), s>>>(g);
  return hipGetLastError();
}

}  // namespace moe
