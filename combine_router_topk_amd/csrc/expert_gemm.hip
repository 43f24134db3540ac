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

// LDS: a ring of stages, one step of K each. A stage of a tile of MF units
// holds 256 weight rows and 64 MF rows of 128 codes. The ring is as deep as
// fits. Scales come for four steps at once, into one of two places: a step's
// scales of 64 rows lie in 64 lines of memory, and fetched one by one in each
// step they were a third of all that the loads moved.
constexpr int kWBytes = kTileN * kDepth;
constexpr int kABytes = kUnit * kDepth;  // of one unit
constexpr int stage_bytes(int mf) { return kWBytes + mf * kABytes; }
constexpr int kGroup = 4;  // steps whose scales are loaded together
constexpr int ring_depth(int mf) { return mf <= 2 ? 3 : 2; }
constexpr int scale_place(int mf) { return (mf + 1) * kUnit * kGroup * 4; }  // the units' rows, the weights
constexpr int ring_bytes(int mf) { return stage_bytes(mf) * ring_depth(mf) + 2 * scale_place(mf); }
constexpr int kRingBytes = ring_bytes(2);
static_assert(ring_bytes(1) <= kRingBytes && ring_bytes(3) <= kRingBytes && ring_bytes(4) <= kRingBytes,
              "every ring fits");

struct Shared {
  unsigned char ring[kRingBytes];  // stages, then the two places for scales
  uint32_t amax[2][kMaxUnits * kUnit];
  int count[kMaxE];
  int first_tile[kMaxE];
};
static_assert(sizeof(Shared) <= 160 * 1024, "one block's LDS");

// Each lane's 16 (or 4) bytes from base + offset go to LDS at byte lds + 16
// (or 4) * lane without passing through registers. Written as assembly because the
// compiler, which cannot tell the stages of the ring apart, waits for every
// such load of its own before the next LDS read; here the loop counts them
// (wait_loads). They have no output register.
__device__ __forceinline__ void load_lds16(const void* base, uint32_t offset, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(lds), "v"(offset), "s"(base)
               : "memory");
}
__device__ __forceinline__ void load_lds4(const void* base, uint32_t offset, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, %2" ::"s"(lds), "v"(offset), "s"(base)
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

// One tile: 64 MF rows from m0 on of the segment that starts at row `seg`
// (`left` of them valid) against the weights n_tile of expert e.
template <int MF, bool SWIGLU, int ACT, bool F32>
__device__ __forceinline__ void tile(const GemmArgs& g, Shared& sh, int e, int seg, int m0, int left,
                                     int n_tile) {
  // taken anew for each tile: what follows from it is cheap, and held over the
  // tile loop it would take registers that the accumulators need
  int tid = threadIdx.x;
  asm volatile("" : "+v"(tid));
  const int lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wn = wave & 1, wm = wave >> 1;
  const int col = lane & 15, grp = lane >> 4;
  const int nbK = scale_blocks(g.K), nbN = scale_blocks(g.N);

  // What this lane loads in each step: chunk my_chunk of the step's 128 bytes
  // of these rows, as byte offsets (the host checked that 32 bits hold them)
  // from the expert's weights and from the first row or token. Row r of a
  // stage keeps chunk c at place c ^ (r / 2 % 8), so that the 16 lanes that
  // read one chunk of 16 rows together meet all LDS banks.
  const uint32_t my_chunk = (tid & 7) ^ ((tid >> 4) & 7);
  uint32_t wo[4], ao[MF];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    wo[i] = static_cast<uint32_t>(weight_row<SWIGLU>(g, n_tile, i * 64 + (tid >> 3))) * g.K + my_chunk * 16;
  const int row0 = g.src == nullptr ? seg + m0 : 0;
  auto row_of = [&](int m) {  // counted from row0
    m = min(m, left - 1);
    if (g.src == nullptr) return m;
    const int i = g.src[seg + m0 + m];
    return i < 0 ? 0 : min(i / g.k, g.a_rows - 1);
  };
#pragma unroll
  for (int i = 0; i < MF; ++i) ao[i] = static_cast<uint32_t>(row_of(i * 64 + (tid >> 3))) * g.K + my_chunk * 16;
  const uint8_t* const w0 = g.w + static_cast<size_t>(e) * g.N * g.K;
  const uint8_t* const a0 = g.a + static_cast<size_t>(row0) * g.K;
  // Chunks past the end of K: their lanes take the row's last one instead, and
  // the weights' are overwritten with zeros in LDS.
  const int end_chunks = g.K / 16 - (nbK - 1) * 8;  // of the last step
  const uint32_t past = my_chunk * 16 - min(my_chunk, static_cast<uint32_t>(end_chunks - 1)) * 16;
  // The first MF waves load their unit's scales, the others the weights' (all
  // the same 16, so that every wave counts the same loads).
  const float* s0;
  uint32_t so;
  if (wave < MF) {
    s0 = g.a_scale + static_cast<size_t>(row0) * nbK;
    so = static_cast<uint32_t>(row_of(wave * 64 + lane)) * nbK * 4;
  } else {
    s0 = g.w_scale + static_cast<size_t>(e) * nbN * nbK;
    so = weight_row<SWIGLU>(g, n_tile, (col >> 2) * 64 + (col & 3) * 4) / kScaleBlock * nbK * 4;
  }

  // as plain registers: computed by 64-bit multiplications they would stay pairs
#pragma unroll
  for (int i = 0; i < 4; ++i) asm volatile("" : "+v"(wo[i]));
#pragma unroll
  for (int i = 0; i < MF; ++i) asm volatile("" : "+v"(ao[i]));
  asm volatile("" : "+v"(so));

  constexpr int kSteps = ring_depth(MF);
  constexpr int kFirst = 2 + MF, kSecond = 2;  // loads of each wave and part, without scales
  constexpr int kScales = stage_bytes(MF) * kSteps;
  const uint32_t ring = lds_address(sh.ring);
  // With rows of whole 16-byte groups one load takes the scales of four steps
  // and lane l's lie at 4 l; else four loads take one step each and step j's
  // lie at 64 j.
  auto load_scales = [&](int group) {
    const uint32_t at = ring + kScales + min(wave, MF) * (kUnit * kGroup * 4) + (group & 1) * scale_place(MF);
    if (g.scales16) {
      load_lds16(s0 + group * kGroup, so, at);
    } else {
#pragma unroll
      for (int j = 0; j < kGroup; ++j) load_lds4(s0 + min(group * kGroup + j, nbK - 1), so, at + j * 256);
    }
  };
  // The loads come in two parts: the rows' codes and the first half of each
  // wave's weight rows, which a step is done with in its middle, and the second
  // half. Each is loaded again as soon as nobody reads it any more.
  auto load_part = [&](int kb, bool first) {
    const uint32_t st = ring + (kb % kSteps) * stage_bytes(MF) + wave * 1024;
    const uint8_t* wk = w0 + kb * kDepth;
    const uint8_t* ak = a0 + kb * kDepth;
    const uint32_t back = kb == nbK - 1 ? past : 0;
    if (first) {
      if (kb % kGroup == 0) load_scales(kb / kGroup);
#pragma unroll
      for (int i = 0; i < MF; ++i) load_lds16(ak, ao[i] - back, st + kWBytes + i * 8192);
      load_lds16(wk, wo[0] - back, st);
      load_lds16(wk, wo[2] - back, st + 2 * 8192);
    } else {
      load_lds16(wk, wo[1] - back, st + 8192);
      load_lds16(wk, wo[3] - back, st + 3 * 8192);
    }
  };
  const int s_row = g.scales16 ? kGroup : 1, s_step = g.scales16 ? 1 : kUnit;

  v4f acc[8][MF];
#pragma unroll
  for (int n = 0; n < 8; ++n)
#pragma unroll
    for (int f = 0; f < MF; ++f) acc[n][f] = v4f{0, 0, 0, 0};

  constexpr bool kPrecise = SWIGLU || F32;
  auto read_frag = [&](const unsigned char* rows, int r) {
    const uint4* p = reinterpret_cast<const uint4*>(rows) + r * 8;
    const uint4 lo = p[(2 * grp) ^ ((r >> 1) & 7)];
    const uint4 hi = p[(2 * grp + 1) ^ ((r >> 1) & 7)];
    return v8i{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
  };

#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    if (i < nbK) load_part(i, true);
    if (i < kSteps - 1 && i < nbK) load_part(i, false);
  }
  // the first part of the step is read: load it anew
  auto middle = [&](int kb) {
    wait_reads();
    if (kb + kSteps < nbK) load_part(kb + kSteps, true);
  };
#pragma clang loop unroll(disable)
  for (int kb = 0; kb < nbK; ++kb) {
    // Step kb's codes are in LDS, and nobody reads the step before it any
    // more. Loads issued since then may be in flight; scales among them only
    // make the wait longer than it has to be.
    if (kb + kSteps - 1 < nbK) {
      wait_loads<(kSteps - 1) * kFirst + (kSteps - 2) * kSecond>();
      load_part(kb + kSteps - 1, false);
    } else {
      wait_loads<0>();
    }
    unsigned char* st = sh.ring + (kb % kSteps) * stage_bytes(MF);
    if (kb == nbK - 1 && end_chunks < 8) {  // zeros for the weights past the end of K
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (static_cast<int>(my_chunk) >= end_chunks)
          reinterpret_cast<uint4*>(st)[i * 512 + tid] = make_uint4(0, 0, 0, 0);
      wait_reads();
    }
    const float* scales = reinterpret_cast<const float*>(sh.ring + kScales + ((kb / kGroup) & 1) * scale_place(MF)) +
                          (kb % kGroup) * s_step;
    float s[2][MF];
    const float sw0 = scales[MF * kUnit * kGroup + (wn * 8 + grp) * s_row];
    const float sw1 = scales[MF * kUnit * kGroup + (wn * 8 + 4 + grp) * s_row];
#pragma unroll
    for (int f = 0; f < MF; ++f) {
      const float sa = scales[f * kUnit * kGroup + (wm * 16 + col) * s_row];
      s[0][f] = sa * sw0;
      s[1][f] = sa * sw1;
    }
    auto add = [&](const v4f& p, int t) {
      const int n = t / MF, f = t % MF;
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[n][f][i] = fmaf(p[i], s[n >> 2][f], acc[n][f][i]);
      asm volatile("" : "+v"(acc[n][f]));  // here, not after the branches of the loads
    };
    v8i w[2];
    w[0] = read_frag(st, wn * 128 + col);
    if constexpr (kPrecise) {
      Wide b[MF];
#pragma unroll
      for (int f = 0; f < MF; ++f) b[f] = widen(read_frag(st + kWBytes, (f * 4 + wm) * 16 + col));
#pragma unroll
      for (int n = 0; n < 8; ++n) {
        if (n == 4) middle(kb);
        if (n < 7) w[(n + 1) & 1] = read_frag(st, wn * 128 + (n + 1) * 16 + col);
        const Wide wide = widen(w[n & 1]);
        v4f p[MF];
#pragma unroll
        for (int f = 0; f < MF; ++f) p[f] = v4f{0, 0, 0, 0};
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int f = 0; f < MF; ++f) p[f] = mfma16<1>(wide.v[j], b[f].v[j], p[f]);
#pragma unroll
        for (int f = 0; f < MF; ++f) add(p[f], n * MF + f);
        __builtin_amdgcn_sched_barrier(0);
      }
    } else {
      v8i b[MF];
#pragma unroll
      for (int f = 0; f < MF; ++f) b[f] = read_frag(st + kWBytes, (f * 4 + wm) * 16 + col);
      // a matrix instruction's multiply-adds follow two instructions later
      v4f p[3];
#pragma unroll
      for (int n = 0; n < 8; ++n) {
        if (n == 4) middle(kb);
        if (n < 7) w[(n + 1) & 1] = read_frag(st, wn * 128 + (n + 1) * 16 + col);
#pragma unroll
        for (int f = 0; f < MF; ++f) {
          const int t = n * MF + f;
          const v4f z = {0, 0, 0, 0};
          p[t % 3] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w[n & 1], b[f], z, 0, 0, 0, 0, 0, 0);
          if (t >= 2) add(p[(t - 2) % 3], t - 2);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
      add(p[(8 * MF - 2) % 3], 8 * MF - 2);
      add(p[(8 * MF - 1) % 3], 8 * MF - 1);
    }
  }

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
    __syncthreads();
    const int nbH = scale_blocks(g.half);
#pragma unroll
    for (int f = 0; f < MF; ++f) {
      const int m = (f * 4 + wm) * 16 + col;
      const float s = block_scale(umax(sh.amax[0][m], sh.amax[1][m]));
      if (m >= left) continue;
      const size_t r = static_cast<size_t>(seg) + m0 + m;
      if (c0 < g.half) {
        uint32_t o[4];
#pragma unroll
        for (int n = 0; n < 4; ++n)
          o[n] = quant4(acc[n][f][0], acc[n][f][1], acc[n][f][2], acc[n][f][3], s);
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
  __syncthreads();  // the next tile's loads overwrite the stages
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
  const int total = __builtin_amdgcn_readfirstlane(sh.first_tile[g.E - 1] + tiles_of<kUnits>(sh.count[g.E - 1])) * g.n_tiles;  // the host checked that it fits
  const int per_xcd = (total + kXcds - 1) / kXcds;
  const int first = static_cast<int>(blockIdx.x % kXcds) * per_xcd;
  const int last = min(total, first + per_xcd);
  for (int t = first + static_cast<int>(blockIdx.x / kXcds); t < last; t += kGemmBlocks / kXcds) {
    const int mt = t / g.n_tiles;
    int lo = 0, hi = g.E;  // the last expert whose first tile is at most mt
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (sh.first_tile[mid] <= mt) lo = mid;
      else hi = mid;
    }
    const int e = __builtin_amdgcn_readfirstlane(lo);
    const int rows = __builtin_amdgcn_readfirstlane(sh.count[e]), tiles = tiles_of<kUnits>(rows);
    const int in = t - __builtin_amdgcn_readfirstlane(sh.first_tile[e]) * g.n_tiles;
    const int m_tile = in % tiles, n_tile = in / tiles;
    const int units = (rows + kUnit - 1) / kUnit, base = units / tiles, more = units % tiles;
    const int u0 = m_tile * base + min(m_tile, more);
    const int u1 = u0 + base + (m_tile < more ? 1 : 0);
    const int m0 = u0 * kUnit;
    // a segment that would end past the rows is moved back inside
    const int seg = __builtin_amdgcn_readfirstlane(max(0, min(g.offsets[e], g.rows - rows)));
    const int left = min(rows, u1 * kUnit) - m0;
    switch (u1 - u0) {
      case 1: tile<1, SWIGLU, ACT, F32>(g, sh, e, seg, m0, left, n_tile); break;
      case 2: tile<2, SWIGLU, ACT, F32>(g, sh, e, seg, m0, left, n_tile); break;
      case 3: tile<3, SWIGLU, ACT, F32>(g, sh, e, seg, m0, left, n_tile); break;
      default: tile<kUnits, SWIGLU, ACT, F32>(g, sh, e, seg, m0, left, n_tile); break;
    }
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
