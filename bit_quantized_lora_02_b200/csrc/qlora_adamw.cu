// qlora_adamw.cu -- one AdamW step (Loshchilov and Hutter, "Decoupled Weight
// Decay Regularization", ICLR 2019) over many tensors at once: the adapters' A
// and B of every projection.
//
//     g  = grad_scale grad, held to +-2^60
//     m' = beta1 m + (1 - beta1) g,   v' = beta2 v + (1 - beta2) g^2
//     p' = p (1 - lr wd) - lr / (1 - beta1^t) m' / (sqrt(v') / sqrt(1 - beta2^t) + eps)
//
// The moments are kept in 32 bits or in 8.  In 8 bits they are block-wise
// quantised (Dettmers, Lewis, Shleifer and Zettlemoyer, "8-bit Optimizers via
// Block-wise Quantization", ICLR 2022: blocks of a tensor are scaled by their
// largest value, so that an outlier spoils one block only), 256 values to a
// block, with codes that fit the two moments:
//   m: E4M3 of 448 m / s_m, s_m = max |m| (nearest, ties to even).  Momentum has
//      both signs and any size; a relative error of 2^-4 is far below the tenth
//      that every step replaces.  A block whose s_m is below 2^-100 stores zeros.
//   v: round(255 u / s_u) of the fourth root u = v^(1/4), s_u = max u, and at
//      least 1 where v > 0.  v's range within a block is the square of the
//      gradients'; linear steps in its fourth root resolve 1.6% of v at the
//      block's largest value and still reach down to 2^-32 of it, and a positive v
//      never becomes 0, which would turn the step into m / eps.
// g is held to 2^60 because its square has to fit fp32: an infinite v' would stay
// so, and with 8-bit states its block's with it, and freeze the parameters.  The
// step does not depend on the gradients' scale, so beside moments of less than 2^60
// it is that of the gradient as it came.  One that is not finite becomes NaN.
// p' is computed from m' and v' before they are coded.  Every operation on the
// way to a stored moment is one fp32 operation rounded on its own (no fused
// multiply-add), so the states are bit-reproducible from this definition.
//
// Bound: HBM.  bf16 parameters with fp32 gradients and 8-bit states move 12 bytes
// per value, fp32 masters with bf16 copies and 32-bit states 30.  A warp holds one
// block of 256 values, 8 to a lane, with the loads of the next ones in flight
// (cp.async: registers cannot hold them as well); the block's maxima are one redux
// each.  128M bf16 parameters with fp32 gradients and 8-bit states: 247 us, the
// measured rate of a plain copy (101%); 51 instructions per value fill half of the
// issue slots.  448 adapter tensors (40M values) with fp32 masters, bf16 copies and
// 32-bit states: 183 us (101%).
// Tensors, their pointers and the chunk where each starts travel as kernel
// parameters (up to 28 KB): nothing has to be copied to the device before the
// launch, and a captured graph keeps them.
#include <cmath>
#include <type_traits>

#include "qlora_device.cuh"
#include "qlora_internal.h"
#include "qlora_vec.cuh"

namespace qlora {

namespace {

constexpr int kBlock = 256;
constexpr int kWarps = 4;               // warps of a CTA, one block each at a time
// Blocks that a warp's loads run ahead.  128M values: with 8-bit states, whose
// arithmetic takes long, 247 us at three; with 32-bit ones one is enough (564 us
// with fp32 parameters; two and three were 15% slower at some combinations of
// types, where their rings fill an SM's shared memory).
template <bool EIGHT>
constexpr int kAheadBlocks = EIGHT ? 3 : 1;
constexpr float kMagic = 12582912.0f;   // 1.5 * 2^23

struct Scalars {
  float b1, c1, b2, c2;      // beta, 1 - beta
  float decay, size, rbc2;   // 1 - lr wd, lr / (1 - beta1^t), 1 / sqrt(1 - beta2^t)
  float eps;
};

template <int CAP>
struct Batch {
  AdamTensor t[CAP];
  int32_t first[CAP];   // first chunk of each tensor
  int32_t count, iters;
  Scalars s;
  const float* scale;   // gradient scale on the device (has_scale), else any readable float
  const float* clock;   // decay, size, rbc2 on the device (has_clock)
  int32_t has_scale, has_clock;
};

// Advance the clock by one step and leave the step's scalars behind it: powers
// in 64 bits, since 1 - beta^t of the first steps cancels.
__global__ void k_adamw_clock(double* clock, double beta1, double beta2, double wd) {
  griddep_launch_dependents();
  griddep_wait();
  const double lr = clock[0], t = clock[1] + 1.0;
  clock[1] = t;
  float* out = reinterpret_cast<float*>(clock + 2);
  out[0] = static_cast<float>(1.0 - lr * wd);
  out[1] = static_cast<float>(lr / (1.0 - pow(beta1, t)));
  out[2] = static_cast<float>(1.0 / sqrt(1.0 - pow(beta2, t)));
}

// Four neighbouring elements of 4, 2 or 1 bytes: one load or store per lane, a
// warp's together contiguous.  `have` of the four exist (the array has n); at the
// array's end every load's address is clamped into it.
template <typename E>
struct Four;
template <>
struct Four<float> {
  using Raw = uint4;
};
template <>
struct Four<__nv_bfloat16> {
  using Raw = uint2;
};
template <>
struct Four<uint8_t> {
  using Raw = uint32_t;
};
template <typename E>
__device__ __forceinline__ uint32_t bits_of(E x) {
  if constexpr (sizeof(E) == 4)
    return __float_as_uint(x);
  else if constexpr (sizeof(E) == 2)
    return __bfloat16_as_ushort(x);
  else
    return x;
}
template <typename E>
__device__ __forceinline__ typename Four<E>::Raw load4(const void* base, int64_t i, int64_t n, int have) {
  const E* p = reinterpret_cast<const E*>(base);
  if (have == 4) return *reinterpret_cast<const typename Four<E>::Raw*>(p + i);
  uint32_t x[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t b = bits_of(p[min(i + k, n - 1)]);
    x[k] = k < have ? b : 0u;
  }
  if constexpr (sizeof(E) == 4)
    return make_uint4(x[0], x[1], x[2], x[3]);
  else if constexpr (sizeof(E) == 2)
    return make_uint2(x[0] | x[1] << 16, x[2] | x[3] << 16);
  else
    return x[0] | x[1] << 8 | x[2] << 16 | x[3] << 24;
}
template <typename E>
__device__ __forceinline__ void store4(void* base, int64_t i, int have, const typename Four<E>::Raw& v) {
  E* p = reinterpret_cast<E*>(base) + i;
  if (have == 4) {
    *reinterpret_cast<typename Four<E>::Raw*>(p) = v;
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (k >= have) continue;
      if constexpr (sizeof(E) == 4)
        p[k] = __uint_as_float(k == 0 ? v.x : k == 1 ? v.y : k == 2 ? v.z : v.w);
      else if constexpr (sizeof(E) == 2)
        p[k] = __ushort_as_bfloat16(static_cast<unsigned short>((k < 2 ? v.x : v.y) >> (16 * (k & 1))));
      else
        p[k] = static_cast<uint8_t>(v >> (8 * k));
    }
  }
}
__device__ __forceinline__ void pairs(const uint4& v, f2 (&f)[2]) {
  f[0] = f2_make(__uint_as_float(v.x), __uint_as_float(v.y));
  f[1] = f2_make(__uint_as_float(v.z), __uint_as_float(v.w));
}
__device__ __forceinline__ void pairs(const uint2& v, f2 (&f)[2]) {
  f[0] = f2_make(bf16_lo(v.x), bf16_hi(v.x));
  f[1] = f2_make(bf16_lo(v.y), bf16_hi(v.y));
}
__device__ __forceinline__ uint4 raw_f32(const f2 (&f)[2]) { return pack2(f, 0.0f); }
__device__ __forceinline__ uint2 raw_bf16(const f2 (&f)[2]) { return make_uint2(pack2_bf16(f[0]), pack2_bf16(f[1])); }

// m and v of four codes each (dm, dv: the block's scales over 448 and 255)
__device__ __forceinline__ void decode(uint32_t mc, uint32_t vc, f2 dm, f2 dv, f2 (&m)[2], f2 (&v)[2]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t half2;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(half2) : "h"(static_cast<uint16_t>(mc >> (16 * h))));
    float lo, hi;
    asm("{\n\t.reg .f16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
        : "=f"(lo), "=f"(hi)
        : "r"(half2));
    m[h] = f2_mul(f2_make(lo, hi), dm);
    // a byte b as 2^23 + b, so that one exact subtraction gives the float
    const float a = __uint_as_float(prmt(vc, 0x4B000000u, h ? 0x7442u : 0x7440u));
    const float b = __uint_as_float(prmt(vc, 0x4B000000u, h ? 0x7443u : 0x7441u));
    f2 t = f2_mul(f2_add(f2_make(a, b), f2_dup(-8388608.0f)), dv);
    t = f2_mul(t, t);
    v[h] = f2_mul(t, t);
  }
}
__device__ __forceinline__ float unit_m(float s) { return __fmul_rn(s, 1.0f / 448.0f); }
__device__ __forceinline__ float unit_v(float s) { return __fmul_rn(s, 1.0f / 255.0f); }

__device__ __forceinline__ float sqrt_approx(float x) {
  float r;
  asm("sqrt.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float sqrt_approx_ftz(float x) {
  float r;
  asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float rcp_approx(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// g held to +-2^60, NaN where it is not finite (then g * 0 is).  It costs 8-bit
// states 1 to 2% (128M values: fp32 gradients 245 -> 247 us, bf16 ones 240 -> 245),
// 32-bit ones nothing.  One test for a lane's eight values took as long; a second
// pass over a block whose largest v' tells of such a gradient took 1 to 4%.
__device__ __forceinline__ f2 hold(f2 g) {
  float lo, hi;
  f2_get(g, lo, hi);
  asm("min.xorsign.abs.f32 %0, %0, %1;" : "+f"(lo) : "f"(0x1p60f));
  asm("min.xorsign.abs.f32 %0, %0, %1;" : "+f"(hi) : "f"(0x1p60f));
  return f2_fma(g, 0, f2_make(lo, hi));
}
// largest of a and two magnitudes, NaN if one is
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(fabsf(b)), "f"(fabsf(c)));
  return r;
}

enum { kParamBf16 = 0, kParamF32 = 1, kParamMaster = 2 };   // master: fp32 and a bf16 copy

// One block of 256 values, 8 to a lane: elements 4 lane + k and 128 + 4 lane + k.
template <int PARAM, typename G, bool EIGHT>
struct Block {
  using P = typename std::conditional<PARAM == kParamBf16, __nv_bfloat16, float>::type;
  using S = typename std::conditional<EIGHT, uint8_t, float>::type;
  typename Four<G>::Raw g[2];
  typename Four<P>::Raw p[2];
  typename Four<S>::Raw m[2], v[2];
  uint2 copy[2];
  float ms, vs;

  // the moments, the parameter and, in 8 bits, the codes after the step
  __device__ __forceinline__ void step(const Scalars& s, f2 gs) {
    const f2 b1 = f2_dup(s.b1), c1 = f2_dup(s.c1), b2 = f2_dup(s.b2), c2 = f2_dup(s.c2);
    const f2 decay = f2_dup(s.decay), size = f2_dup(-s.size), rbc2 = f2_dup(s.rbc2), eps = f2_dup(s.eps);
    f2 mn[4], vn[4], root[4];
    float mtop = 0.0f, vtop = 0.0f;
    f2 dm = 0, dv = 0;
    if constexpr (EIGHT) {
      dm = f2_dup(unit_m(ms));
      dv = f2_dup(unit_v(vs));
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      f2 gr[2], pa[2], mo[2], vo[2];
      pairs(g[j], gr);
      pairs(p[j], pa);
      if constexpr (EIGHT) {
        decode(m[j], v[j], dm, dv, mo, vo);
      } else {
        pairs(m[j], mo);
        pairs(v[j], vo);
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int q = 2 * j + h;
        gr[h] = hold(f2_mul(gr[h], gs));
        // packed products, but scalar sums: the compiler fuses a packed product
        // into the packed sum behind it, which would round once instead of twice
        float a0, a1, q0, q1, x0, x1;
        f2_get(f2_mul(mo[h], b1), a0, a1);
        f2_get(f2_mul(gr[h], c1), q0, q1);
        x0 = __fadd_rn(a0, q0);
        x1 = __fadd_rn(a1, q1);
        if constexpr (EIGHT) mtop = max3_nan(mtop, x0, x1);
        mn[q] = f2_make(x0, x1);
        f2_get(f2_mul(vo[h], b2), a0, a1);
        f2_get(f2_mul(f2_mul(gr[h], gr[h]), c2), q0, q1);
        x0 = __fadd_rn(a0, q0);
        x1 = __fadd_rn(a1, q1);
        if constexpr (EIGHT) vtop = max3_nan(vtop, x0, x1);
        vn[q] = f2_make(x0, x1);
        root[q] = f2_make(sqrt_approx(x0), sqrt_approx(x1));
        // p (1 - lr wd) + m' (-lr / (1 - beta1^t)) / (sqrt(v') / sqrt(1 - beta2^t) + eps)
        f2_get(f2_fma(root[q], rbc2, eps), a0, a1);
        pa[h] = f2_fma(pa[h], decay, f2_mul(f2_mul(mn[q], size), f2_make(rcp_approx(a0), rcp_approx(a1))));
      }
      if constexpr (PARAM == kParamBf16) {
        p[j] = raw_bf16(pa);
      } else {
        p[j] = raw_f32(pa);
        if constexpr (PARAM == kParamMaster) copy[j] = raw_bf16(pa);
      }
      if constexpr (!EIGHT) {
        m[j] = raw_f32({mn[2 * j], mn[2 * j + 1]});
        v[j] = raw_f32({vn[2 * j], vn[2 * j + 1]});
      }
    }
    if constexpr (EIGHT) {
      // magnitudes order as integers, NaN above infinity
      ms = __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(mtop) & 0x7FFFFFFFu));
      const float vmax = __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(vtop) & 0x7FFFFFFFu));
      // rounded square roots keep the order, so the largest root is the root of the largest
      vs = __fsqrt_rn(__fsqrt_rn(vmax));
      if (ms < 0x1p-100f) ms = 0.0f;
      const float im = ms > 0.0f ? __fdiv_rn(448.0f, ms) : 0.0f;
      const float iv = vs > 0.0f ? __fdiv_rn(255.0f, vs) : 0.0f;
      const f2 im2 = f2_dup(im), iv2 = f2_dup(iv), unmagic = f2_dup(-kMagic), minus = f2_dup(-1.0f);
      // y = u 255 / s_u from approximate roots first: they are off by at most 2^-23
      // of their value each, and the definition's y by roundings of its own, 6.5 *
      // 2^-24 in all or 1e-4 of y <= 255.  Where y is not within 2^-13 of a half
      // between two codes, both give the same code.
      f2 t[4];
      float worst = 0.0f;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float x0, x1;
        f2_get(root[q], x0, x1);
        const f2 y = f2_mul(f2_make(sqrt_approx_ftz(x0), sqrt_approx_ftz(x1)), iv2);
        f2_get(y, x0, x1);
        // adding 1.5 * 2^23 rounds to an integer (ties to even) in the low byte
        t[q] = f2_make(__fadd_rn(x0, kMagic), __fadd_rn(x1, kMagic));
        f2_get(f2_fma(f2_add(t[q], unmagic), minus, y), x0, x1);
        worst = fmaxf(fmaxf(fabsf(x0), fabsf(x1)), worst);
      }
      if (worst > 0.5f - 0x1p-13f) {   // one block in fifteen: the roots as the definition has them
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          float x0, x1;
          f2_get(vn[q], x0, x1);
          x0 = __fmul_rn(__fsqrt_rn(__fsqrt_rn(x0)), iv);
          x1 = __fmul_rn(__fsqrt_rn(__fsqrt_rn(x1)), iv);
          t[q] = f2_make(__fadd_rn(x0, kMagic), __fadd_rn(x1, kMagic));
        }
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        uint16_t e[2];
        float c[4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float x0, x1;
          f2_get(f2_mul(mn[2 * j + h], im2), x0, x1);
          asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(e[h]) : "f"(x1), "f"(x0));
          f2_get(t[2 * j + h], c[2 * h], c[2 * h + 1]);
          f2_get(vn[2 * j + h], x0, x1);
          if (x0 > 0.0f) c[2 * h] = fmaxf(c[2 * h], kMagic + 1.0f);
          if (x1 > 0.0f) c[2 * h + 1] = fmaxf(c[2 * h + 1], kMagic + 1.0f);
        }
        m[j] = static_cast<uint32_t>(e[0]) | (static_cast<uint32_t>(e[1]) << 16);
        v[j] = prmt(prmt(__float_as_uint(c[0]), __float_as_uint(c[1]), 0x0040u),
                    prmt(__float_as_uint(c[2]), __float_as_uint(c[3]), 0x0040u), 0x5410u);
      }
    }
  }
};

// The lane's place in the arrays of a tensor, and steps of kWarps blocks.
template <int PARAM, typename G, bool EIGHT>
struct Place {
  using B = Block<PARAM, G, EIGHT>;
  const uint8_t* g;
  uint8_t *p, *m, *v, *copy;
  template <typename E>
  static __device__ __forceinline__ uint8_t* at(const void* base, int64_t i) {
    return const_cast<uint8_t*>(reinterpret_cast<const uint8_t*>(base)) + i * static_cast<int64_t>(sizeof(E));
  }
  __device__ __forceinline__ Place(const AdamTensor& T, int64_t block, int lane) {
    const int64_t i = block * kBlock + 4 * lane;
    g = at<G>(T.g, i);
    p = at<typename B::P>(T.p, i);
    m = at<typename B::S>(T.m, i);
    v = at<typename B::S>(T.v, i);
    copy = PARAM == kParamMaster ? at<uint16_t>(T.copy, i) : p;
  }
  __device__ __forceinline__ void advance() {
    constexpr int E = kWarps * kBlock;
    g += E * sizeof(G);
    p += E * sizeof(typename B::P);
    m += E * sizeof(typename B::S);
    v += E * sizeof(typename B::S);
    if constexpr (PARAM == kParamMaster) copy += E * 2;
  }
  template <typename E>
  static __device__ __forceinline__ void put(uint8_t* q, int j, const typename Four<E>::Raw& x) {
    *reinterpret_cast<typename Four<E>::Raw*>(q + j * 128 * sizeof(E)) = x;
  }
  // A block's loads run ahead through a ring in shared memory (cp.async); a lane
  // reads back only what it copied itself.  Every array has two slots of four
  // elements per thread and stage.
  static constexpr uint32_t kT = 32 * kWarps;
  static constexpr uint32_t kG = 0, kP = kG + 8 * kT * sizeof(G), kM = kP + 8 * kT * sizeof(typename B::P),
                            kV = kM + 8 * kT * sizeof(typename B::S), kStage = kV + 8 * kT * sizeof(typename B::S);
  template <typename E>
  static __device__ __forceinline__ void copy_in(uint32_t ring, const uint8_t* q) {
#pragma unroll
    for (int j = 0; j < 2; ++j)
      cp_async<4 * sizeof(E)>(ring + (j * kT + threadIdx.x) * 4 * sizeof(E), q + j * 128 * sizeof(E));
  }
  __device__ __forceinline__ void issue(uint32_t stage) const {
    copy_in<G>(stage + kG, g);
    copy_in<typename B::P>(stage + kP, p);
    copy_in<typename B::S>(stage + kM, m);
    copy_in<typename B::S>(stage + kV, v);
  }
  template <typename E>
  static __device__ __forceinline__ typename Four<E>::Raw take(uint32_t ring, int j) {
    return lds<typename Four<E>::Raw>(ring + (j * kT + threadIdx.x) * 4 * sizeof(E));
  }
  static __device__ __forceinline__ void load(B& b, uint32_t stage) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      b.g[j] = take<G>(stage + kG, j);
      b.p[j] = take<typename B::P>(stage + kP, j);
      b.m[j] = take<typename B::S>(stage + kM, j);
      b.v[j] = take<typename B::S>(stage + kV, j);
    }
  }
  __device__ __forceinline__ void store(const B& b) const {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      put<typename B::P>(p, j, b.p[j]);
      if constexpr (PARAM == kParamMaster) put<__nv_bfloat16>(copy, j, b.copy[j]);
      put<typename B::S>(m, j, b.m[j]);
      put<typename B::S>(v, j, b.v[j]);
    }
  }
};

template <int PARAM, typename G, bool EIGHT, int CAP>
__global__ void __launch_bounds__(32 * kWarps, 5) k_adamw(const __grid_constant__ Batch<CAP> b) {
  using B = Block<PARAM, G, EIGHT>;
  constexpr int kAhead = kAheadBlocks<EIGHT>;
  griddep_launch_dependents();
  // the tensor whose chunks hold this CTA's
  int lo = 0, hi = b.count - 1;
  const int chunk = static_cast<int>(blockIdx.x);
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (b.first[mid] <= chunk)
      lo = mid;
    else
      hi = mid - 1;
  }
  const AdamTensor& T = b.t[lo];
  const int64_t n = T.n;
  const int lane = threadIdx.x & 31;
  const int64_t block = static_cast<int64_t>(chunk - b.first[lo]) * kWarps * b.iters + (threadIdx.x >> 5);
  // this warp's blocks: `whole` of 256 values, kWarps apart, and maybe the tensor's
  // shorter last one
  const int64_t full = n / kBlock;
  const int whole = static_cast<int>(min(max((full - block + kWarps - 1) / kWarps, int64_t(0)), static_cast<int64_t>(b.iters)));
  griddep_wait();
  Scalars s = b.s;
  if (b.has_clock) {
    s.decay = b.clock[0];
    s.size = b.clock[1];
    s.rbc2 = b.clock[2];
  }
  const f2 gs = f2_dup(b.has_scale ? *b.scale : 1.0f);
  if (whole > 0) {
    using At = Place<PARAM, G, EIGHT>;
    extern __shared__ __align__(16) uint8_t ring_mem[];
    const uint32_t ring = smem_u32(ring_mem);
    At ahead(T, block, lane), at = ahead;
    for (int k = 0; k < kAhead; ++k) {
      if (k < whole) {
        ahead.issue(ring + k * At::kStage);
        ahead.advance();
      }
      cp_async_commit();
    }
    // lane k holds the scales of the warp's block k, old ones and then new ones
    float ms = 0.0f, vs = 0.0f;
    const int64_t mine = block + kWarps * min(lane, whole - 1);
    if constexpr (EIGHT) {
      ms = T.ms[mine];
      vs = T.vs[mine];
    }
    uint32_t stage = 0;
#pragma unroll 1
    for (int k = 0; k < whole; ++k) {
      B now;
      cp_async_wait(kAhead - 1);
      At::load(now, ring + stage);
      if constexpr (EIGHT) {
        now.ms = __shfl_sync(0xFFFFFFFFu, ms, k);
        now.vs = __shfl_sync(0xFFFFFFFFu, vs, k);
      }
      now.step(s, gs);
      at.store(now);
      at.advance();
      if constexpr (EIGHT) {
        ms = lane == k ? now.ms : ms;
        vs = lane == k ? now.vs : vs;
      }
      if (k + kAhead < whole) {
        ahead.issue(ring + stage);
        ahead.advance();
      }
      cp_async_commit();
      stage = stage == (kAhead - 1) * At::kStage ? 0 : stage + At::kStage;
    }
    if (EIGHT && lane < whole) {
      T.ms[mine] = ms;
      T.vs[mine] = vs;
    }
  }
  const int64_t last = block + kWarps * whole;
  if (whole < b.iters && last == full && full * kBlock < n) {
    B now;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int64_t i = last * kBlock + 128 * j + 4 * lane;
      const int have = static_cast<int>(min(max(n - i, int64_t(0)), int64_t(4)));
      now.g[j] = load4<G>(T.g, i, n, have);
      now.p[j] = load4<typename B::P>(T.p, i, n, have);
      now.m[j] = load4<typename B::S>(T.m, i, n, have);
      now.v[j] = load4<typename B::S>(T.v, i, n, have);
    }
    if constexpr (EIGHT) {
      now.ms = T.ms[last];
      now.vs = T.vs[last];
    }
    now.step(s, gs);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int64_t i = last * kBlock + 128 * j + 4 * lane;
      const int have = static_cast<int>(min(max(n - i, int64_t(0)), int64_t(4)));
      store4<typename B::P>(T.p, i, have, now.p[j]);
      if constexpr (PARAM == kParamMaster) store4<__nv_bfloat16>(T.copy, i, have, now.copy[j]);
      store4<typename B::S>(T.m, i, have, now.m[j]);
      store4<typename B::S>(T.v, i, have, now.v[j]);
    }
    if (EIGHT && lane == 0) {
      T.ms[last] = now.ms;
      T.vs[last] = now.vs;
    }
  }
}

// The values that 8-bit states stand for: four per thread and array, four times.
__global__ void __launch_bounds__(256) k_adamw_values(int64_t n, const uint8_t* m8, const float* ms, const uint8_t* v8,
                                                      const float* vs, float* m_out, float* v_out) {
  griddep_launch_dependents();
  griddep_wait();
  const int64_t base = static_cast<int64_t>(blockIdx.x) * 4096 + threadIdx.x * 4;
  uint32_t mc[4], vc[4];
  float sm[4], sv[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int64_t i = base + k * 1024;
    if (i >= n) continue;
    const int have = static_cast<int>(min(n - i, int64_t(4)));
    mc[k] = load4<uint8_t>(m8, i, n, have);
    vc[k] = load4<uint8_t>(v8, i, n, have);
    sm[k] = ms[i / kBlock];
    sv[k] = vs[i / kBlock];
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int64_t i = base + k * 1024;
    if (i >= n) continue;
    const int have = static_cast<int>(min(n - i, int64_t(4)));
    f2 m[2], v[2];
    decode(mc[k], vc[k], f2_dup(unit_m(sm[k])), f2_dup(unit_v(sv[k])), m, v);
    store4<float>(m_out, i, have, raw_f32(m));
    store4<float>(v_out, i, have, raw_f32(v));
  }
}

template <int PARAM, typename G, bool EIGHT, int CAP>
cudaError_t launch(const AdamArgs& a, const Scalars& s, int64_t from, int64_t to, cudaStream_t st) {
  Batch<CAP> b;
  int64_t blocks = 0;
  for (int64_t i = from; i < to; ++i) blocks += ceil_div(a.tensors[i].n, kBlock);
  // chunks of one block per warp, up to 16 times that where every SM still gets
  // several CTAs
  b.iters = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(16, blocks / (kWarps * 40 * num_sms()))));
  int64_t chunks = 0;
  b.count = 0;
  for (int64_t i = from; i < to; ++i) {
    const AdamTensor& t = a.tensors[i];
    if (t.n == 0) continue;
    b.t[b.count] = t;
    b.first[b.count++] = static_cast<int32_t>(chunks);
    chunks += ceil_div(ceil_div(t.n, kBlock), kWarps * b.iters);
  }
  if (b.count == 0) return cudaSuccess;
  if (chunks > INT32_MAX) return cudaErrorInvalidConfiguration;
  b.s = s;
  b.has_scale = a.scale != nullptr;
  b.has_clock = a.clock != nullptr;
  // never a NULL pointer behind a flag: any readable address
  b.clock = a.clock ? reinterpret_cast<const float*>(a.clock + 2) : reinterpret_cast<const float*>(b.t[0].p);
  b.scale = a.scale ? a.scale : reinterpret_cast<const float*>(b.t[0].p);
  auto kernel = k_adamw<PARAM, G, EIGHT, CAP>;
  constexpr uint32_t smem = kAheadBlocks<EIGHT> * Place<PARAM, G, EIGHT>::kStage;
  const cudaError_t e = set_smem(kernel, smem);
  if (e != cudaSuccess) return e;
  ProfScope prof(QLORA_KC_AUX, st);
  return launch_pdl(kernel, dim3(static_cast<unsigned>(chunks)), dim3(32 * kWarps), smem, st, nullptr, b);
}

template <int PARAM, typename G, bool EIGHT>
cudaError_t run(const AdamArgs& a, const Scalars& s, cudaStream_t st) {
  // few tensors: a launch with few parameters (29 KB of them cost a
  // call 1.1 us more: 14 tensors 6.3 us, 5.2 with the small list)
  constexpr int64_t kMany = 400, kFew = 16;
  if (a.count <= kFew) return launch<PARAM, G, EIGHT, kFew>(a, s, 0, a.count, st);
  for (int64_t at = 0; at < a.count; at += kMany) {
    const cudaError_t e = launch<PARAM, G, EIGHT, kMany>(a, s, at, std::min(a.count, at + kMany), st);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

template <int PARAM, typename G>
cudaError_t by_state(const AdamArgs& a, const Scalars& s, cudaStream_t st) {
  return a.bits == 8 ? run<PARAM, G, true>(a, s, st) : run<PARAM, G, false>(a, s, st);
}

template <int PARAM>
cudaError_t by_grad(const AdamArgs& a, const Scalars& s, cudaStream_t st) {
  return a.grad_dtype == QLORA_DT_BF16 ? by_state<PARAM, __nv_bfloat16>(a, s, st) : by_state<PARAM, float>(a, s, st);
}

}  // namespace

cudaError_t launch_adamw(const AdamArgs& a, cudaStream_t st) {
  Scalars s{};
  s.b1 = static_cast<float>(a.beta1);
  s.c1 = static_cast<float>(1.0 - a.beta1);
  s.b2 = static_cast<float>(a.beta2);
  s.c2 = static_cast<float>(1.0 - a.beta2);
  s.eps = static_cast<float>(a.eps);
  if (a.clock) {
    ProfScope prof(QLORA_KC_AUX, st);
    const cudaError_t e = launch_pdl(k_adamw_clock, dim3(1), dim3(1), 0, st, nullptr, a.clock, a.beta1, a.beta2, a.wd);
    if (e != cudaSuccess) return e;
  } else {
    const double t = static_cast<double>(a.step);
    s.decay = static_cast<float>(1.0 - a.lr * a.wd);
    s.size = static_cast<float>(a.lr / (1.0 - std::pow(a.beta1, t)));
    s.rbc2 = static_cast<float>(1.0 / std::sqrt(1.0 - std::pow(a.beta2, t)));
  }
  if (a.param_dtype == QLORA_DT_BF16) return by_grad<kParamBf16>(a, s, st);
  return a.copies ? by_grad<kParamMaster>(a, s, st) : by_grad<kParamF32>(a, s, st);
}

cudaError_t launch_adamw_values(int64_t n, const uint8_t* m8, const float* ms, const uint8_t* v8, const float* vs,
                                float* m_out, float* v_out, cudaStream_t st) {
  ProfScope prof(QLORA_KC_AUX, st);
  return launch_pdl(k_adamw_values, dim3(static_cast<unsigned>(ceil_div(n, 4096))), dim3(256), 0, st, nullptr, n, m8, ms,
                    v8, vs, m_out, v_out);
}

}  // namespace qlora
