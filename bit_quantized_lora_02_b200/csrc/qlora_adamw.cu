// qlora_adamw.cu -- one AdamW step (Loshchilov and Hutter, "Decoupled Weight
// Decay Regularization", ICLR 2019) over many tensors at once: the adapters' A
// and B of every projection.
//
//     g  = grad_scale grad
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
// p' is computed from m' and v' before they are coded.  Every operation on the
// way to a stored moment is one fp32 operation rounded on its own (no fused
// multiply-add), so the states are bit-reproducible from this definition.
//
// Bound: HBM.  bf16 parameters with fp32 gradients and 8-bit states move 12 bytes
// per value, fp32 masters with bf16 copies and 32-bit states 30.  A warp holds one
// block of 256 values, 8 to a lane; the block's maxima are one redux each.
// Tensors, their pointers and the chunk where each starts travel as kernel
// parameters (up to 28 KB): nothing has to be copied to the device before the
// launch, and a captured graph keeps them.
#include <cmath>

#include "qlora_device.cuh"
#include "qlora_internal.h"
#include "qlora_vec.cuh"

namespace qlora {

namespace {

constexpr int kBlock = 256;

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

// 8 values of a lane, at element i of an array of n; `have` of them exist.  At the
// array's end every load's address is clamped into it.
template <typename T>
__device__ __forceinline__ void load8(const void* base, int64_t i, int64_t n, int have, float (&f)[8]) {
  const T* p = reinterpret_cast<const T*>(base) + i;
  if (have == 8) {
    constexpr int N = Vec<T>::N;
    uint4 q[8 / N];
#pragma unroll
    for (int h = 0; h < 8 / N; ++h) q[h] = reinterpret_cast<const uint4*>(p)[h];
#pragma unroll
    for (int h = 0; h < 8 / N; ++h) {
      float x[N];
      Vec<T>::unpack(q[h], x);
#pragma unroll
      for (int k = 0; k < N; ++k) f[h * N + k] = x[k];
    }
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float x = to_f32(reinterpret_cast<const T*>(base)[min(i + k, n - 1)]);
      f[k] = k < have ? x : 0.0f;
    }
  }
}

template <typename T>
__device__ __forceinline__ void store8(void* base, int64_t i, int have, const float (&f)[8]) {
  T* p = reinterpret_cast<T*>(base) + i;
  if (have == 8) {
    constexpr int N = Vec<T>::N;
#pragma unroll
    for (int h = 0; h < 8 / N; ++h) {
      float x[N];
#pragma unroll
      for (int k = 0; k < N; ++k) x[k] = f[h * N + k];
      reinterpret_cast<uint4*>(p)[h] = Vec<T>::pack(x);
    }
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < have) p[k] = from_f32<T>(f[k]);
  }
}

// 8 byte codes, the first in the low byte of x
__device__ __forceinline__ uint2 load8b(const void* base, int64_t i, int64_t n, int have) {
  const uint8_t* p = reinterpret_cast<const uint8_t*>(base);
  if (have == 8) return *reinterpret_cast<const uint2*>(p + i);
  uint2 v = make_uint2(0u, 0u);
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const uint32_t x = p[min(i + k, n - 1)];
    const uint32_t b = k < have ? x << (8 * (k & 3)) : 0u;
    if (k < 4)
      v.x |= b;
    else
      v.y |= b;
  }
  return v;
}
__device__ __forceinline__ void store8b(void* base, int64_t i, int have, uint2 v) {
  uint8_t* p = reinterpret_cast<uint8_t*>(base) + i;
  if (have == 8) {
    *reinterpret_cast<uint2*>(p) = v;
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < have) p[k] = static_cast<uint8_t>((k < 4 ? v.x : v.y) >> (8 * (k & 3)));
  }
}

// m and v of 8 codes each (scales: the block's largest |m|, largest fourth root)
__device__ __forceinline__ void decode(uint2 mc, uint2 vc, float ms, float vs, float (&m)[8], float (&v)[8]) {
  const f2 dm = f2_dup(__fmul_rn(ms, 1.0f / 448.0f)), dv = f2_dup(__fmul_rn(vs, 1.0f / 255.0f));
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    const uint32_t mw = h < 2 ? mc.x : mc.y, vw = h < 2 ? vc.x : vc.y;
    uint32_t half2;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(half2) : "h"(static_cast<uint16_t>(mw >> (16 * (h & 1)))));
    float lo, hi;
    asm("{\n\t.reg .f16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
        : "=f"(lo), "=f"(hi)
        : "r"(half2));
    f2_get(f2_mul(f2_make(lo, hi), dm), m[2 * h], m[2 * h + 1]);
    // a byte b as 2^23 + b, so that one exact subtraction gives the float
    const float a = __uint_as_float(prmt(vw, 0x4B000000u, (h & 1) ? 0x7442u : 0x7440u)) - 8388608.0f;
    const float b = __uint_as_float(prmt(vw, 0x4B000000u, (h & 1) ? 0x7443u : 0x7441u)) - 8388608.0f;
    f2 t = f2_mul(f2_make(a, b), dv);
    t = f2_mul(t, t);
    f2_get(f2_mul(t, t), v[2 * h], v[2 * h + 1]);
  }
}

enum { kParamBf16 = 0, kParamF32 = 1, kParamMaster = 2 };   // master: fp32 and a bf16 copy

template <int PARAM, typename G, bool EIGHT, int CAP>
__global__ void __launch_bounds__(256) k_adamw(const __grid_constant__ Batch<CAP> b) {
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
  griddep_wait();
  Scalars s = b.s;
  if (b.has_clock) {
    s.decay = b.clock[0];
    s.size = b.clock[1];
    s.rbc2 = b.clock[2];
  }
  const float gs = b.has_scale ? *b.scale : 1.0f;
  const f2 gs2 = f2_dup(gs), b1 = f2_dup(s.b1), c1 = f2_dup(s.c1), b2 = f2_dup(s.b2), c2 = f2_dup(s.c2);
  int64_t block = static_cast<int64_t>(chunk - b.first[lo]) * 8 * b.iters + (threadIdx.x >> 5);
  for (int it = 0; it < b.iters; ++it, block += 8) {
    const int64_t i = block * kBlock + lane * 8;
    if (block * kBlock >= n) break;
    const int have = static_cast<int>(min(max(n - i, int64_t(0)), int64_t(8)));
    float p[8], g[8], m[8], v[8], r[8];
    load8<G>(T.g, i, n, have, g);
    if constexpr (PARAM == kParamBf16)
      load8<__nv_bfloat16>(T.p, i, n, have, p);
    else
      load8<float>(T.p, i, n, have, p);
    if constexpr (EIGHT) {
      const uint2 mc = load8b(T.m, i, n, have), vc = load8b(T.v, i, n, have);
      decode(mc, vc, T.ms[block], T.vs[block], m, v);
    } else {
      load8<float>(T.m, i, n, have, m);
      load8<float>(T.v, i, n, have, v);
    }
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      f2 q = f2_make(g[2 * h], g[2 * h + 1]);
      if (b.has_scale) q = f2_mul(q, gs2);
      // packed products, but scalar sums: the compiler fuses a packed product
      // into the packed sum behind it, which would round once instead of twice
      float a0, a1, q0, q1;
      f2_get(f2_mul(f2_make(m[2 * h], m[2 * h + 1]), b1), a0, a1);
      f2_get(f2_mul(q, c1), q0, q1);
      m[2 * h] = __fadd_rn(a0, q0);
      m[2 * h + 1] = __fadd_rn(a1, q1);
      f2_get(f2_mul(f2_make(v[2 * h], v[2 * h + 1]), b2), a0, a1);
      f2_get(f2_mul(f2_mul(q, q), c2), q0, q1);
      v[2 * h] = __fadd_rn(a0, q0);
      v[2 * h + 1] = __fadd_rn(a1, q1);
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      r[k] = __fsqrt_rn(v[k]);
      p[k] = p[k] * s.decay - __fdividef(m[k] * s.size, fmaf(r[k], s.rbc2, s.eps));
    }
    if constexpr (PARAM == kParamBf16) {
      store8<__nv_bfloat16>(T.p, i, have, p);
    } else {
      store8<float>(T.p, i, have, p);
      if constexpr (PARAM == kParamMaster) store8<__nv_bfloat16>(T.copy, i, have, p);
    }
    if constexpr (EIGHT) {
      uint32_t mm = 0, um = 0;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        r[k] = __fsqrt_rn(r[k]);
        mm = max(mm, __float_as_uint(m[k]) & 0x7FFFFFFFu);   // magnitudes order as integers (NaN above infinity)
        um = max(um, __float_as_uint(r[k]) & 0x7FFFFFFFu);
      }
      float ms = __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, mm));
      const float vs = __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, um));
      if (ms < 0x1p-100f) ms = 0.0f;
      const float im = ms > 0.0f ? __fdiv_rn(448.0f, ms) : 0.0f;
      const float iv = vs > 0.0f ? __fdiv_rn(255.0f, vs) : 0.0f;
      uint32_t mw[2], vw[2];
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        uint16_t e[2];
        uint32_t c[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          // adding 1.5 * 2^23 rounds to an integer (ties to even) in the low byte
          const float y = __fadd_rn(__fmul_rn(r[4 * q + k], iv), 12582912.0f);
          c[k] = max(__float_as_uint(y) & 0xFFu, v[4 * q + k] > 0.0f ? 1u : 0u);
        }
#pragma unroll
        for (int k = 0; k < 2; ++k)
          asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;"
              : "=h"(e[k])
              : "f"(__fmul_rn(m[4 * q + 2 * k + 1], im)), "f"(__fmul_rn(m[4 * q + 2 * k], im)));
        mw[q] = static_cast<uint32_t>(e[0]) | (static_cast<uint32_t>(e[1]) << 16);
        vw[q] = prmt(prmt(c[0], c[1], 0x0040u), prmt(c[2], c[3], 0x0040u), 0x5410u);
      }
      store8b(T.m, i, have, make_uint2(mw[0], mw[1]));
      store8b(T.v, i, have, make_uint2(vw[0], vw[1]));
      if (lane == 0) {
        T.ms[block] = ms;
        T.vs[block] = vs;
      }
    } else {
      store8<float>(T.m, i, have, m);
      store8<float>(T.v, i, have, v);
    }
  }
}

// The values that 8-bit states stand for.
__global__ void __launch_bounds__(256) k_adamw_values(int64_t n, const uint8_t* m8, const float* ms, const uint8_t* v8,
                                                      const float* vs, float* m_out, float* v_out) {
  griddep_launch_dependents();
  griddep_wait();
  const int64_t i = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * 8;
  if (i >= n) return;
  const int have = static_cast<int>(min(n - i, int64_t(8)));
  float m[8], v[8];
  decode(load8b(m8, i, n, have), load8b(v8, i, n, have), ms[i / kBlock], vs[i / kBlock], m, v);
  store8<float>(m_out, i, have, m);
  store8<float>(v_out, i, have, v);
}

template <int PARAM, typename G, bool EIGHT, int CAP>
cudaError_t launch(const AdamArgs& a, const Scalars& s, int64_t from, int64_t to, cudaStream_t st) {
  Batch<CAP> b;
  int64_t blocks = 0;
  for (int64_t i = from; i < to; ++i) blocks += ceil_div(a.tensors[i].n, kBlock);
  // chunks of 8 blocks (one per warp), up to four times that where every SM
  // still gets several CTAs
  b.iters = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(4, blocks / (8 * 16 * num_sms()))));
  int64_t chunks = 0;
  b.count = 0;
  for (int64_t i = from; i < to; ++i) {
    const AdamTensor& t = a.tensors[i];
    if (t.n == 0) continue;
    b.t[b.count] = t;
    b.first[b.count++] = static_cast<int32_t>(chunks);
    chunks += ceil_div(ceil_div(t.n, kBlock), 8 * b.iters);
  }
  if (b.count == 0) return cudaSuccess;
  if (chunks > INT32_MAX) return cudaErrorInvalidConfiguration;
  b.s = s;
  b.has_scale = a.scale != nullptr;
  b.has_clock = a.clock != nullptr;
  // never a NULL pointer behind a flag: any readable address
  b.clock = a.clock ? reinterpret_cast<const float*>(a.clock + 2) : reinterpret_cast<const float*>(b.t[0].p);
  b.scale = a.scale ? a.scale : reinterpret_cast<const float*>(b.t[0].p);
  ProfScope prof(QLORA_KC_AUX, st);
  return launch_pdl(k_adamw<PARAM, G, EIGHT, CAP>, dim3(static_cast<unsigned>(chunks)), dim3(256), 0, st, nullptr, b);
}

template <int PARAM, typename G, bool EIGHT>
cudaError_t run(const AdamArgs& a, const Scalars& s, cudaStream_t st) {
  // few tensors: a launch with few parameters (29 KB of them cost 2 us more)
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
  return launch_pdl(k_adamw_values, dim3(static_cast<unsigned>(ceil_div(n, 2048))), dim3(256), 0, st, nullptr, n, m8, ms,
                    v8, vs, m_out, v_out);
}

}  // namespace qlora
