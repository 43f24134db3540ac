// One AdamW step over a list of tensors, states in fp32 or in 8 bits:
//
//   m = b1 m + (1 - b1) g          v = b2 v + (1 - b2) g^2
//   w = w - lr decay w - lr (m / c1) / (sqrt(v / c2) + eps),   ci = 1 - bi^step
//
// A block takes 2048 elements of one tensor, a thread 8 neighbours at a time
// (whole 16-byte loads of every array). The tensors come as kernel arguments,
// up to 56 a launch, with each one's first block: the lanes of a wave compare
// those with their block's number at once. Nothing is read that a later call
// could find changed, so gradients may live somewhere else in each step.
//
// The bytes bound it: 284 million weights in 16 bits with fp32 masters, 28 bytes
// each, take 1485 us (5.36 TB/s; a large copy reaches 4.85), with 8-bit states, 16.1
// bytes each, 885 us (5.2 TB/s). 150 tensors of 14.6 million in all, 235 MB in
// three launches: 65 us.
//
// 8-bit states are e4m3 codes with one fp32 scale for each 128 elements (16
// lanes, whose largest magnitude is a few lane exchanges away). v is held as its
// root, which halves the exponents it spans: a code reaches down to 2^-9 / 448 of
// the block's largest root, 1.9e-11 of its largest v. Below that it takes the
// smallest code and not zero, so that no step divides by eps alone for want of
// bits. The step itself uses m and v in fp32 as just computed; the states' rounding
// shows in the next one. Codes carry over, so a value that another order of
// rounding puts on the other side of a border shows as a whole step of its code
// from then on; therefore products are rounded before they are added and quotients
// are divisions: the states are what the formulas give operation by operation.
#include "device.hpp"
#include "launch.hpp"
#include "quant.hpp"

namespace moe {

namespace {

constexpr int kThreads = 256;
constexpr int kPer = 8;                                // elements of a thread at a time
// elements of a block. (Four times as many: 6 tensors of 284 million elements 1530
// us for 1505 in fp32 and 871 for 889 with 8-bit states, 150 of 14.6 million 75 for
// 65.)
constexpr int kChunk = kThreads * kPer;
constexpr int kMaxTensors = 56;                        // of a launch: the arguments stay below 4 KiB
constexpr uint32_t kMaxBlocks = (1u << 24) - 1;        // of a launch: below 2^32 work-items

struct AdamWTensor {
  void* w;
  float* master;
  const void* g;
  void* m;
  void* v;
  float* m_scale;
  float* v_scale;
  int64_t n;
  float decay;
  uint32_t first;  // its first block of the launch
};
struct Args {
  AdamWTensor t[kMaxTensors];
  int n;
  float lr, beta1, beta2, rest1, rest2, eps, step, ln1, ln2;  // resti = 1 - betai
  const float* control;
};
static_assert(sizeof(Args) <= 4096, "kernel arguments");

template <bool F32, int ACT>
__device__ __forceinline__ void load8(const void* base, int64_t at, float (&f)[kPer]) {
  if constexpr (F32) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + at);
    const float4 a = p[0], b = p[1];
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w;
    f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
  } else {
    unpack8<ACT>(*reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + at), f);
  }
}
// the first `have` of 8, zeros behind them
template <bool F32, int ACT>
__device__ __forceinline__ void load_some(const void* base, int64_t at, int have, float (&f)[kPer]) {
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    f[i] = 0.0f;
    if (i < have) {
      if constexpr (F32) f[i] = static_cast<const float*>(base)[at + i];
      else f[i] = act_to_f32<ACT>(static_cast<const uint16_t*>(base)[at + i]);
    }
  }
}
// Nothing of what is written is read again in the step: 1 to 3 % less than with
// ordinary stores. (Loads that do not keep it either cost 4 % in fp32.)
typedef uint32_t v4u __attribute__((ext_vector_type(4)));
template <bool F32, int ACT>
__device__ __forceinline__ void store8(void* base, int64_t at, const float (&f)[kPer]) {
  if constexpr (F32) {
    v4f* p = reinterpret_cast<v4f*>(static_cast<float*>(base) + at);
    __builtin_nontemporal_store(v4f{f[0], f[1], f[2], f[3]}, p);
    __builtin_nontemporal_store(v4f{f[4], f[5], f[6], f[7]}, p + 1);
  } else {
    const uint4 v = round8<ACT>(f);
    __builtin_nontemporal_store(v4u{v.x, v.y, v.z, v.w}, reinterpret_cast<v4u*>(static_cast<uint16_t*>(base) + at));
  }
}
template <bool F32, int ACT>
__device__ __forceinline__ void store_some(void* base, int64_t at, int have, const float (&f)[kPer]) {
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    if (i < have) {
      if constexpr (F32) static_cast<float*>(base)[at + i] = f[i];
      else static_cast<uint16_t*>(base)[at + i] = static_cast<uint16_t>(f32_to_act<ACT>(f[i]));
    }
  }
}

__device__ __forceinline__ uint2 load_codes(const void* base, int64_t at, int have) {
  const uint8_t* p = static_cast<const uint8_t*>(base) + at;
  if (have == kPer) return *reinterpret_cast<const uint2*>(p);
  uint32_t w[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < kPer; ++i)
    if (i < have) w[i >> 2] |= static_cast<uint32_t>(p[i]) << ((i & 3) * 8);
  return make_uint2(w[0], w[1]);
}
__device__ __forceinline__ void store_codes(void* base, int64_t at, int have, uint2 c) {
  uint8_t* p = static_cast<uint8_t*>(base) + at;
  if (have == kPer) {
    *reinterpret_cast<uint2*>(p) = c;
    return;
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i)
    if (i < have) p[i] = static_cast<uint8_t>((i < 4 ? c.x : c.y) >> ((i & 3) * 8));
}
__device__ __forceinline__ void values_of(uint2 c, float s, float (&f)[kPer]) {
  const int lo = static_cast<int>(c.x), hi = static_cast<int>(c.y);
  f[0] = __builtin_amdgcn_cvt_f32_fp8(lo, 0) * s, f[1] = __builtin_amdgcn_cvt_f32_fp8(lo, 1) * s;
  f[2] = __builtin_amdgcn_cvt_f32_fp8(lo, 2) * s, f[3] = __builtin_amdgcn_cvt_f32_fp8(lo, 3) * s;
  f[4] = __builtin_amdgcn_cvt_f32_fp8(hi, 0) * s, f[5] = __builtin_amdgcn_cvt_f32_fp8(hi, 1) * s;
  f[6] = __builtin_amdgcn_cvt_f32_fp8(hi, 2) * s, f[7] = __builtin_amdgcn_cvt_f32_fp8(hi, 3) * s;
}
// The scale of the 128 values that 16 lanes hold: amax times the rounded 1 / 448,
// one operation (block_scale's correction makes it the rounded quotient), so that
// amax / scale may be 448 and a rounding, which is the code of 448 too.
__device__ __forceinline__ float scale_of(const float (&f)[kPer]) {
  uint32_t amax = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) amax = umax(amax, __float_as_uint(f[i]) & 0x7fffffffu);
  amax = group_max<16>(amax);
  return amax >= 0x7f800000u ? __uint_as_float(0x7fc00000u) : fmaxf(__uint_as_float(amax), 0x1p-100f) * (1.0f / kE4m3Max);
}
__device__ __forceinline__ uint2 codes_of(const float (&f)[kPer], float s) {
  // f / s is at most 448 and its rounding
  return make_uint2(quant4(f[0] / s, f[1] / s, f[2] / s, f[3] / s, 1.0f),
                    quant4(f[4] / s, f[5] / s, f[6] / s, f[7] / s, 1.0f));
}
// codes of 0 where the value is above it become the smallest code
__device__ __forceinline__ uint32_t not_zero(uint32_t c, float a, float b, float d, float e) {
  if ((c & 0x000000ffu) == 0 && a > 0.0f) c |= 0x00000001u;
  if ((c & 0x0000ff00u) == 0 && b > 0.0f) c |= 0x00000100u;
  if ((c & 0x00ff0000u) == 0 && d > 0.0f) c |= 0x00010000u;
  if ((c & 0xff000000u) == 0 && e > 0.0f) c |= 0x01000000u;
  return c;
}

template <bool W32, bool G32, int ACT, bool S8>
__global__ __launch_bounds__(kThreads) void adamw_kernel(Args a) {
  const int tid = threadIdx.x, lane = tid & 63;
  const uint32_t first = lane < a.n ? a.t[lane].first : ~0u;
  const int which = __builtin_popcountll(ballot(first <= blockIdx.x)) - 1;
  const AdamWTensor t = a.t[which];
  const int64_t chunk = static_cast<int64_t>(blockIdx.x - readlane(first, which)) * kChunk;

  float lr = a.lr, step = a.step, scale = 1.0f;
  if (a.control != nullptr) {
    lr = a.control[0], step = a.control[1], scale = a.control[2];
    if (!(fabsf(scale) < __builtin_inff())) return;  // the caller found no step to make
  }
  const float c1 = -expm1f(step * a.ln1), c2 = -expm1f(step * a.ln2);
  const float lr1 = lr / c1, root2 = 1.0f / sqrtf(c2), shrink = lr * t.decay;

  const int64_t at = chunk + tid * kPer;
  const int64_t left = t.n - at;
  const int have = left >= kPer ? kPer : left > 0 ? static_cast<int>(left) : 0;
  if constexpr (S8) {
    if (ballot(have > 0) == 0) return;
  } else {
    if (have == 0) return;
  }
  float w[kPer], g[kPer], m[kPer], v[kPer];
  if (have == kPer) {
    if (t.master != nullptr) load8<true, ACT>(t.master, at, w);
    else load8<W32, ACT>(t.w, at, w);
    load8<G32, ACT>(t.g, at, g);
    if constexpr (!S8) {
      load8<true, ACT>(t.m, at, m);
      load8<true, ACT>(t.v, at, v);
    }
  } else {
    if (t.master != nullptr) load_some<true, ACT>(t.master, at, have, w);
    else load_some<W32, ACT>(t.w, at, have, w);
    load_some<G32, ACT>(t.g, at, have, g);
    if constexpr (!S8) {
      load_some<true, ACT>(t.m, at, have, m);
      load_some<true, ACT>(t.v, at, have, v);
    }
  }
  const int64_t block = at / kScaleBlock;
  if constexpr (S8) {
    const uint2 mc = load_codes(t.m, at, have), vc = load_codes(t.v, at, have);
    values_of(mc, have > 0 ? t.m_scale[block] : 0.0f, m);
    values_of(vc, have > 0 ? t.v_scale[block] : 0.0f, v);
#pragma unroll
    for (int i = 0; i < kPer; ++i) v[i] *= v[i];
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
#pragma clang fp contract(off)
    const float gs = g[i] * scale;
    m[i] = a.beta1 * m[i] + a.rest1 * gs;
    v[i] = a.beta2 * v[i] + a.rest2 * gs * gs;
    const float root = sqrtf(v[i]);
    w[i] = w[i] - fmaf(shrink, w[i], lr1 * m[i] / fmaf(root, root2, a.eps));
    if constexpr (S8) v[i] = root;
  }
  if constexpr (S8) {
    // places past the tensor's end are zeros and do not count
    if (have < kPer) {
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (i >= have) m[i] = v[i] = 0.0f;
    }
    const float ms = scale_of(m), vs = scale_of(v);
    uint2 vc = codes_of(v, vs);
    vc = make_uint2(not_zero(vc.x, v[0], v[1], v[2], v[3]), not_zero(vc.y, v[4], v[5], v[6], v[7]));
    store_codes(t.m, at, have, codes_of(m, ms));
    store_codes(t.v, at, have, vc);
    if ((lane & 15) == 0 && have > 0) {
      t.m_scale[block] = ms;
      t.v_scale[block] = vs;
    }
  }
  if (have == kPer) {
    if (t.master != nullptr) store8<true, ACT>(t.master, at, w);
    store8<W32, ACT>(t.w, at, w);
    if constexpr (!S8) {
      store8<true, ACT>(t.m, at, m);
      store8<true, ACT>(t.v, at, v);
    }
  } else {
    if (t.master != nullptr) store_some<true, ACT>(t.master, at, have, w);
    store_some<W32, ACT>(t.w, at, have, w);
    if constexpr (!S8) {
      store_some<true, ACT>(t.m, at, have, m);
      store_some<true, ACT>(t.v, at, have, v);
    }
  }
}

template <bool S8, typename F>
void with_types(bool w32, bool g32, int act, F&& f) {
  using T = std::true_type;
  using N = std::false_type;
  using A = std::integral_constant<int, 1>;
  using B = std::integral_constant<int, 2>;
  std::integral_constant<bool, S8> s8;
  if (w32 && g32) f(T{}, T{}, A{}, s8);
  else if (w32) act == 1 ? f(T{}, N{}, A{}, s8) : f(T{}, N{}, B{}, s8);
  else if (g32) act == 1 ? f(N{}, T{}, A{}, s8) : f(N{}, T{}, B{}, s8);
  else act == 1 ? f(N{}, N{}, A{}, s8) : f(N{}, N{}, B{}, s8);
}

}  // namespace

int64_t adamw_most_elements() { return static_cast<int64_t>(kMaxBlocks) * kChunk; }

hipError_t launch_adamw(const AdamWStep& h, const moe_adamw_tensor* tensors, int n, bool w32, bool g32, int act, bool s8,
                        hipStream_t s) {
  Args a;
  auto f = [](double v) { return static_cast<float>(v); };
  a.lr = f(h.lr), a.beta1 = f(h.beta1), a.beta2 = f(h.beta2), a.rest1 = f(1.0 - h.beta1), a.rest2 = f(1.0 - h.beta2);
  a.eps = f(h.eps), a.step = f(h.step), a.ln1 = f(log(h.beta1)), a.ln2 = f(log(h.beta2));
  a.control = h.control;
  for (int i = 0; i < n;) {
    uint32_t blocks = 0;
    a.n = 0;
    for (; i < n && a.n < kMaxTensors; ++i) {
      const uint32_t more = static_cast<uint32_t>((tensors[i].n + kChunk - 1) / kChunk);
      if (more == 0) continue;
      if (blocks + more > kMaxBlocks) break;
      const moe_adamw_tensor& t = tensors[i];
      a.t[a.n++] = {t.w, t.master, t.g, t.m, t.v, t.m_scale, t.v_scale, t.n, t.weight_decay, blocks};
      blocks += more;
    }
    if (blocks == 0) continue;
    auto go = [&](auto W, auto G, auto A, auto S) {
      adamw_kernel<decltype(W)::value, decltype(G)::value, decltype(A)::value, decltype(S)::value>
          <<<blocks, kThreads, 0, s>>>(a);
    };
    if (s8) with_types<true>(w32, g32, act, go);
    else with_types<false>(w32, g32, act, go);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
  }
  return hipSuccess;
}

}  // namespace moe
