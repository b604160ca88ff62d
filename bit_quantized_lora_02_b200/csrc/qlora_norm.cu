// qlora_norm.cu -- layer norm in front of the projections: forward with the
// residual add in front of it, backward with the weight's gradient.
//
// Per row of D values, with S = X (+ R, rounded to X's type):
//     mean = sum(S) / D  (rms: 0),   rstd = 1 / sqrt(sum((S - mean)^2) / D + eps),
//     Y = (S - mean) rstd w + b.
// Backward, with xh = (S - mean) rstd and g = dY w:
//     dX = rstd (g - sum(g) / D - xh sum(g xh) / D) (+ dS),   (rms: no sum(g) / D)
//     dw = sum over rows of dY xh,   db = sum over rows of dY.
// All of it is held in fp32; Y, S and dX are rounded once to the activations'
// type (bf16: nearest even), S before it is normalised, so that the backward
// pass, which reads S, sees the values that were normalised.
//
// Bound: HBM.  Every activation is read and written once: the forward keeps a row
// in registers between its reductions, the backward reads its two inputs a second
// time from shared memory.  8192 x 8192 bf16, rms with residual (537 MB each way):
// forward 83 us, the measured rate of a plain copy; backward 93 to 99 us (84 to
// 90% of it), of which about 5 are the reduction of 296 rows of partial sums.  Without a
// residual the forward moves half as much: rms 44 us (94%); with a mean and a bias
// 50 us (84%), where the second barrier of a row's sums shows.
#include "qlora_device.cuh"
#include "qlora_internal.h"
#include "qlora_vec.cuh"

namespace qlora {

namespace {

// Both kernels walk over rows gridDim apart.  A row is held by a CTA, or by one
// of its four warps where it is short (WARP), CH windows of 16 bytes to a thread;
// the CTA has as many warps as the row needs at CH windows each.  A thread has the
// same columns in every row: the weight stays in registers, and the backward pass
// sums its gradient there.  Rows that do not start on 16-byte boundaries shift the
// windows; the grid is then a multiple of the 8 (fp32: 4) rows after which the
// shift repeats, so that the columns still never change.
//
// The rows' loads run ahead through a ring of a.stages rows in shared memory
// (cp.async): what is in flight then depends neither on registers nor on how
// many CTAs are resident.  Each thread reads back only the 16-byte slots that it
// filled itself, so the ring needs no barrier; the barriers belong to the rows'
// sums.  32 values per thread, where the row is long enough: the shuffles,
// barriers and addresses of a row cost as much as 10 values' arithmetic.
template <typename T, bool WARP, int CH, bool ALIGNED>
struct Rows {
  static constexpr int N = Vec<T>::N;
  static constexpr int ROWS = WARP ? 4 : 1;
  int t, r, sh, D;
  int nt, tb;          // threads of the row, of the CTA
  int64_t row0, stride, M;
  uint32_t slot0, stage_bytes;

  __device__ __forceinline__ Rows(int64_t M_, int D_, void* ring, int arrays) : D(D_), M(M_) {
    tb = WARP ? 128 : blockDim.x;
    nt = WARP ? 32 : blockDim.x;
    t = WARP ? (threadIdx.x & 31) : threadIdx.x;
    r = WARP ? (threadIdx.x >> 5) : 0;
    row0 = static_cast<int64_t>(blockIdx.x) * ROWS + r;
    stride = static_cast<int64_t>(gridDim.x) * ROWS;
    sh = ALIGNED ? 0 : static_cast<int>((row0 * D) % N);
    slot0 = smem_u32(ring) + threadIdx.x * 16u;
    stage_bytes = static_cast<uint32_t>(arrays * CH * tb * 16);
  }
  // what window c can read: 16 bytes, fewer at the row's end, none past it
  __device__ __forceinline__ int bytes(int c) const {
    if constexpr (ALIGNED) return col(c) < D ? 16 : 0;
    return min(max(D - col(c), 0), N) * static_cast<int>(sizeof(T));
  }
  __device__ __forceinline__ int col(int c) const { return (t + c * nt) * N - sh; }
  // Start the loads of array k of a row (element offset `at`) into a stage.  A
  // window that starts in the row before reads that row's end too.
  __device__ __forceinline__ void copy(const void* base, int64_t at, int k, uint32_t stage) const {
    const T* p = reinterpret_cast<const T*>(base) + at - sh;
    uint32_t dst = slot0 + stage + static_cast<uint32_t>(k * CH * tb * 16);
#pragma unroll
    for (int c = 0; c < CH; ++c, dst += tb * 16) {
      const int n = bytes(c);
      cp_async16(dst, p + (n ? (t + c * nt) * N : 0), n);
    }
  }
  __device__ __forceinline__ uint4 get(int k, int c, uint32_t stage) const {
    return lds128(slot0 + stage + static_cast<uint32_t>((k * CH + c) * tb * 16));
  }
  // whether element i of window c belongs to the row
  __device__ __forceinline__ bool in(int c, int i) const {
    return ALIGNED ? col(c) < D : (col(c) + i >= 0 && col(c) + i < D);
  }
};

// Sums of one or two values over the row's threads: one barrier.  The caller
// alternates between two scratches, so a fast warp's next partial sums cannot
// meet a slow warp's reads.  Slots of warps that the CTA does not have stay zero
// (MAXW is the most it can have); every thread adds the slots in the same order.
template <bool WARP, int MAXW>
__device__ __forceinline__ f2 row_sum2(float a, float b, float4* scratch) {
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    a += __shfl_xor_sync(0xffffffffu, a, o);
    b += __shfl_xor_sync(0xffffffffu, b, o);
  }
  f2 v = f2_make(a, b);
  if constexpr (!WARP) {
    if ((threadIdx.x & 31) == 0) reinterpret_cast<float2*>(scratch)[threadIdx.x >> 5] = make_float2(a, b);
    __syncthreads();
    v = 0;
#pragma unroll
    for (int w = 0; w < MAXW / 2; ++w) {
      const float4 q = scratch[w];
      v = f2_add(f2_add(v, f2_make(q.x, q.y)), f2_make(q.z, q.w));
    }
  }
  return v;
}
template <bool WARP, int MAXW>
__device__ __forceinline__ float row_sum(float a, float4* scratch) {
  a = warp_sum(a);
  if constexpr (!WARP) {
    if ((threadIdx.x & 31) == 0) reinterpret_cast<float*>(scratch)[threadIdx.x >> 5] = a;
    __syncthreads();
    f2 v = 0, u = 0;
#pragma unroll
    for (int w = 0; w < MAXW / 4; ++w) {
      const float4 q = scratch[w];
      v = f2_add(v, f2_make(q.x, q.y));
      u = f2_add(u, f2_make(q.z, q.w));
    }
    a = f2_sum(f2_add(v, u));
  }
  return a;
}

constexpr float kLargest = 3.402823466e38f;   // the largest finite fp32 value

// CTAs of nt threads per SM at 128 registers per thread.
constexpr int norm_ctas(int nt) { return nt <= 512 ? 512 / nt : 1; }

// Columns col .. col + N - 1 of the weight or bias (bf16 or fp32, the same for
// all threads; base 16-byte aligned).  Zero outside [0, D).
template <int N>
__device__ __forceinline__ void load_w(const void* w, bool bf16, int col, int D, f2 (&out)[N / 2]) {
  float f[N];
#pragma unroll
  for (int i = 0; i < N; ++i) f[i] = 0.0f;
  if (col >= 0 && col + N <= D && (col & 3) == 0) {
    if (bf16) {
      const uint2* p = reinterpret_cast<const uint2*>(reinterpret_cast<const __nv_bfloat16*>(w) + col);
#pragma unroll
      for (int h = 0; h < N / 4; ++h) {
        const uint2 v = p[h];
        f[4 * h] = bf16_lo(v.x); f[4 * h + 1] = bf16_hi(v.x); f[4 * h + 2] = bf16_lo(v.y); f[4 * h + 3] = bf16_hi(v.y);
      }
    } else {
      const float4* p = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(w) + col);
#pragma unroll
      for (int h = 0; h < N / 4; ++h) {
        const float4 v = p[h];
        f[4 * h] = v.x; f[4 * h + 1] = v.y; f[4 * h + 2] = v.z; f[4 * h + 3] = v.w;
      }
    }
  } else if (col < D && col > -N) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int j = min(max(col + i, 0), D - 1);
      const float x = bf16 ? to_f32(reinterpret_cast<const __nv_bfloat16*>(w)[j]) : reinterpret_cast<const float*>(w)[j];
      f[i] = (col + i >= 0 && col + i < D) ? x : 0.0f;
    }
  }
#pragma unroll
  for (int i = 0; i < N / 2; ++i) out[i] = f2_make(f[2 * i], f[2 * i + 1]);
}

// ---------------------------------------------------------------------------
// Forward.
// ---------------------------------------------------------------------------
template <typename T, int MAXT, int CH, bool ALIGNED>
__global__ void __launch_bounds__(MAXT, norm_ctas(MAXT)) k_norm_fwd(NormArgs a) {
  constexpr int H = Vec<T>::N / 2, MAXW = MAXT / 32;
  constexpr bool WARP = MAXT == 128;
  __shared__ float4 scratch[2][MAXW / 4];
  extern __shared__ __align__(16) uint8_t ring[];
  if constexpr (!WARP) {
    for (int i = threadIdx.x; i < 2 * MAXW; i += blockDim.x) reinterpret_cast<float*>(scratch)[i] = 0.0f;
    __syncthreads();
  }
  const Rows<T, WARP, CH, ALIGNED> R(a.M, a.D, ring, 1 + a.has_r);
  const bool wbf16 = a.wdtype == QLORA_DT_BF16;
  griddep_launch_dependents();
  griddep_wait();
  auto issue = [&](int64_t row, uint32_t stage) {
    if (row < a.M) {
      R.copy(a.X, row * a.D, 0, stage);
      if (a.has_r) R.copy(a.R, row * a.D, 1, stage);
    }
    cp_async_commit();
  };
  for (int s = 0; s < a.stages; ++s) issue(R.row0 + s * R.stride, s * R.stage_bytes);
  f2 w[CH][H], b[CH][H];
#pragma unroll
  for (int c = 0; c < CH; ++c) load_w<2 * H>(a.w, wbf16, R.col(c), a.D, w[c]);
  if (a.has_b) {
#pragma unroll
    for (int c = 0; c < CH; ++c) load_w<2 * H>(a.b, wbf16, R.col(c), a.D, b[c]);
  } else {
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int i = 0; i < H; ++i) b[c][i] = 0;
  }
  int stage = 0, buf = 0;
  float mean = 0.0f;
  int64_t row = R.row0;
#pragma unroll 1
  while (true) {
#pragma unroll 1
    for (; row < a.M; row += R.stride) {
      const int64_t at = row * a.D;
      const uint32_t here = stage * R.stage_bytes;
      cp_async_wait(a.stages - 1);
      stage = stage + 1 == a.stages ? 0 : stage + 1;
      f2 v[CH][H];
#pragma unroll
      for (int c = 0; c < CH; ++c) unpack2(R.get(0, c, here), v[c], T());
      if (a.has_r) {
        T* s = reinterpret_cast<T*>(a.S) + at;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
          f2 q[H];
          unpack2(R.get(1, c, here), q, T());
#pragma unroll
          for (int i = 0; i < H; ++i) v[c][i] = f2_add(v[c][i], q[i]);
          const uint4 packed = pack2(v[c], T());
          unpack2(packed, v[c], T());
          store_raw<T, ALIGNED>(s, R.col(c), a.D, packed);
        }
      }
      issue(row + a.stages * R.stride, here);
      if constexpr (!ALIGNED) {
        if (R.col(0) < 0) {   // values of the row before
          float lo, hi;
#pragma unroll
          for (int i = 0; i < H; ++i) {
            f2_get(v[0][i], lo, hi);
            v[0][i] = f2_make(2 * i < R.sh ? 0.0f : lo, 2 * i + 1 < R.sh ? 0.0f : hi);
          }
        }
      }
      if (!a.rms) {
        f2 sum = 0;
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
          for (int i = 0; i < H; ++i) sum = f2_add(sum, v[c][i]);
        mean = row_sum<WARP, MAXW>(f2_sum(sum), scratch[buf]) / static_cast<float>(a.D);
        buf ^= 1;
        const f2 minus = f2_dup(-mean);
#pragma unroll
        for (int c = 0; c < CH; ++c) {
#pragma unroll
          for (int i = 0; i < H; ++i) v[c][i] = f2_add(v[c][i], minus);
          if (ALIGNED ? R.bytes(c) == 0 : R.bytes(c) < 16 || R.col(c) < 0) {   // outside the row: no share of the variance
            float lo, hi;
#pragma unroll
            for (int i = 0; i < H; ++i) {
              f2_get(v[c][i], lo, hi);
              v[c][i] = f2_make(R.in(c, 2 * i) ? lo : 0.0f, R.in(c, 2 * i + 1) ? hi : 0.0f);
            }
          }
        }
      }
      f2 sq = 0;
#pragma unroll
      for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int i = 0; i < H; ++i) sq = f2_fma(v[c][i], v[c][i], sq);
      const float squares = row_sum<WARP, MAXW>(f2_sum(sq), scratch[buf]);
      buf ^= 1;
      if (!(squares <= kLargest)) break;   // the same for all of the row's threads
      const float rstd = 1.0f / sqrtf(squares / static_cast<float>(a.D) + a.eps);
      if (R.t == 0) {
        if (a.mean_out) a.mean_out[row] = mean;
        if (a.rstd_out) a.rstd_out[row] = rstd;
      }
      T* y = reinterpret_cast<T*>(a.Y) + at;
      const f2 scale = f2_dup(rstd);
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        f2 o[H];
#pragma unroll
        for (int i = 0; i < H; ++i) o[i] = f2_fma(f2_mul(v[c][i], scale), w[c][i], b[c][i]);
        store_raw<T, ALIGNED>(y, R.col(c), a.D, pack2(o, T()));
      }
    }
    if (row >= a.M) break;
    // A row whose squares pass the range of fp32 (values of 1e17 to 1e19 and more,
    // by its length), from memory again: squares 2^-192 as large reach at most 2^64,
    // and what they lose below 2^-149 is no share of their sum.  Infinite again or
    // NaN: the row holds such a value, and all of it becomes NaN.  Outside the loop
    // over ordinary rows, which keeps its registers that way: 8192 x 8192 bf16 takes
    // 88 us with the residual, L2 flushed, as without this part, and 92 with it inside.
    const T* s = reinterpret_cast<const T*>(a.has_r ? a.S : a.X) + row * a.D;
    float sq = 0.0f;
#pragma unroll 1
    for (int c = 0; c < CH; ++c) {
      float x[2 * H];
      Vec<T>::unpack(load_raw<T, ALIGNED>(s, R.col(c), a.D), x);
#pragma unroll
      for (int i = 0; i < 2 * H; ++i) {
        const float d = (x[i] - mean) * 0x1p-96f;
        if (R.in(c, i)) sq = fmaf(d, d, sq);
      }
    }
    const float squares = row_sum<WARP, MAXW>(sq, scratch[buf]);
    buf ^= 1;
    const float rstd = squares <= kLargest
                           ? 0x1p-96f / sqrtf(squares / static_cast<float>(a.D) + a.eps * 0x1p-96f * 0x1p-96f)
                           : __uint_as_float(0x7FC00000u);
    if (R.t == 0) {
      if (a.mean_out) a.mean_out[row] = mean;
      if (a.rstd_out) a.rstd_out[row] = rstd;
    }
#pragma unroll 1
    for (int c = 0; c < CH; ++c) {
      float x[2 * H];
      f2 wl[H], bl[H], o[H];
      Vec<T>::unpack(load_raw<T, ALIGNED>(s, R.col(c), a.D), x);
      load_w<2 * H>(a.w, wbf16, R.col(c), a.D, wl);
      load_w<2 * H>(a.b, wbf16, R.col(c), a.D, bl);
#pragma unroll
      for (int i = 0; i < H; ++i)
        o[i] = f2_fma(f2_make((x[2 * i] - mean) * rstd, (x[2 * i + 1] - mean) * rstd), wl[i], a.has_b ? bl[i] : 0);
      store_raw<T, ALIGNED>(reinterpret_cast<T*>(a.Y) + row * a.D, R.col(c), a.D, pack2(o, T()));
    }
    row += R.stride;
  }
  cp_async_wait(0);
}

// ---------------------------------------------------------------------------
// Backward.  Each CTA leaves the weight's gradient of its rows as one row of
// partial sums; k_norm_reduce adds those in a fixed order.  With the bias's
// gradient in registers as well, the weight moves to shared memory.
// ---------------------------------------------------------------------------
template <typename T, int MAXT, int CH, bool ALIGNED, bool DB>
__global__ void __launch_bounds__(MAXT, norm_ctas(MAXT)) k_norm_bwd(NormArgs a) {
  constexpr int N = Vec<T>::N, H = N / 2;
  constexpr int WV = N / 4;                   // 16-byte slots of a window's fp32 weights
  constexpr int MAXW = MAXT / 32;
  constexpr bool WARP = MAXT == 128;
  using Row = Rows<T, WARP, CH, ALIGNED>;
  __shared__ float4 scratch[2][MAXW / 2];
  extern __shared__ __align__(16) uint8_t ring[];
  if constexpr (!WARP) {
    for (int i = threadIdx.x; i < 4 * MAXW; i += blockDim.x) reinterpret_cast<float*>(scratch)[i] = 0.0f;
    __syncthreads();
  }
  const Row R(a.M, a.D, ring, 2 + a.ring_ds);
  const bool wbf16 = a.wdtype == QLORA_DT_BF16;
  const uint32_t wslot = R.slot0 + a.stages * R.stage_bytes;
  griddep_launch_dependents();
  griddep_wait();
  auto issue = [&](int64_t row, uint32_t stage) {
    if (row < a.M) {
      R.copy(a.X, row * a.D, 0, stage);
      R.copy(a.dY, row * a.D, 1, stage);
      if (a.ring_ds) R.copy(a.dS, row * a.D, 2, stage);
    }
    cp_async_commit();
  };
  for (int s = 0; s < a.stages; ++s) issue(R.row0 + s * R.stride, s * R.stage_bytes);
  f2 dw[CH][H], db[DB ? CH : 1][H], w[DB ? 1 : CH][H];
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    f2 q[H];
    load_w<N>(a.w, wbf16, R.col(c), a.D, q);
#pragma unroll
    for (int i = 0; i < H; ++i) {
      dw[c][i] = 0;
      if constexpr (DB)
        db[c][i] = 0;
      else
        w[c][i] = q[i];
    }
    if constexpr (DB)
#pragma unroll
      for (int k = 0; k < WV; ++k) {
        const f2 p[2] = {q[2 * k], q[2 * k + 1]};
        sts128(wslot + (c * WV + k) * R.tb * 16, pack2(p, 0.0f));
      }
  }
  auto weight = [&](int c, f2 (&q)[H]) {
#pragma unroll
    for (int k = 0; k < WV; ++k) {
      f2 p[2];
      unpack2(lds128(wslot + (c * WV + k) * R.tb * 16), p, 0.0f);
      q[2 * k] = p[0];
      q[2 * k + 1] = p[1];
    }
  };

  const float inv_d = 1.0f / static_cast<float>(a.D);
  float mean = 0.0f, rstd = 0.0f;
  if (R.row0 < a.M) {
    mean = a.mean_in[R.row0];
    rstd = a.rstd_in[R.row0];
  }
  int buf = 0, stage = 0;
#pragma unroll 1
  for (int64_t row = R.row0; row < a.M; row += R.stride, buf ^= 1) {
    const int64_t next = min(row + R.stride, a.M - 1);
    const float mean_next = a.mean_in[next], rstd_next = a.rstd_in[next];
    if (a.rms) mean = 0.0f;
    const uint32_t here = stage * R.stage_bytes;
    cp_async_wait(a.stages - 1);
    const f2 minus = f2_dup(-mean), scale = f2_dup(rstd);
    // xh and dY of window c
    auto take = [&](int c, f2 (&xh)[H], f2 (&dy)[H]) {
      unpack2(R.get(0, c, here), xh, T());
      unpack2(R.get(1, c, here), dy, T());
      if (!ALIGNED && c == 0 && R.col(0) < 0) {   // values of the row before
        float lo, hi;
#pragma unroll
        for (int i = 0; i < H; ++i) {
          f2_get(xh[i], lo, hi);
          xh[i] = f2_make(2 * i < R.sh ? 0.0f : lo, 2 * i + 1 < R.sh ? 0.0f : hi);
          f2_get(dy[i], lo, hi);
          dy[i] = f2_make(2 * i < R.sh ? 0.0f : lo, 2 * i + 1 < R.sh ? 0.0f : hi);
        }
      }
#pragma unroll
      for (int i = 0; i < H; ++i) xh[i] = f2_mul(f2_add(xh[i], minus), scale);
    };
    // Outside the row xh is -mean rstd, and where that is infinite the sum of g xh
    // becomes NaN.  But then xh is 0 throughout the row: one value next to the mean
    // would differ from it by 2^-24 |mean| at least, and rstd stay below
    // 2^24 sqrt(D) / |mean|.  (Asked here, ahead of the sums, this costs nothing; behind
    // them 8192 x 8192 bf16 takes 111 us instead of 101.)
    const bool constant = isinf(mean * rstd) && rstd <= kLargest;
    f2 c1 = 0, c2 = 0;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      f2 xh[H], dy[H], wl[H];
      take(c, xh, dy);
      if constexpr (DB) weight(c, wl);
#pragma unroll
      for (int i = 0; i < H; ++i) {
        // outside the row dY and w are zero, so whatever finite xh is there adds nothing
        dw[c][i] = f2_fma(dy[i], xh[i], dw[c][i]);
        if constexpr (DB) db[c][i] = f2_add(db[c][i], dy[i]);
        const f2 g = f2_mul(dy[i], DB ? wl[i] : w[DB ? 0 : c][i]);
        c1 = f2_add(c1, g);
        c2 = f2_fma(g, xh[i], c2);
      }
    }
    float m1, m2;
    f2_get(row_sum2<WARP, MAXW>(f2_sum(c1), f2_sum(c2), scratch[buf]), m1, m2);
    if (a.dX) {
      if (constant) m2 = 0.0f;
      const f2 off = f2_dup(a.rms ? 0.0f : -m1 * inv_d), along = f2_dup(-m2 * inv_d);
      T* dx = reinterpret_cast<T*>(a.dX) + row * a.D;
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        f2 xh[H], o[H], q[H];
        take(c, xh, o);
        if constexpr (DB) weight(c, q);
#pragma unroll
        for (int i = 0; i < H; ++i)
          o[i] = f2_fma(xh[i], along, f2_fma(o[i], DB ? q[i] : w[DB ? 0 : c][i], off));
        if (a.has_ds) {
          const T* ds = reinterpret_cast<const T*>(a.dS) + row * a.D;
          unpack2(a.ring_ds ? R.get(2, c, here) : load_raw<T, ALIGNED>(ds, R.col(c), a.D), q, T());
#pragma unroll
          for (int i = 0; i < H; ++i) o[i] = f2_fma(o[i], scale, q[i]);
        } else {
#pragma unroll
          for (int i = 0; i < H; ++i) o[i] = f2_mul(o[i], scale);
        }
        store_raw<T, ALIGNED>(dx, R.col(c), a.D, pack2(o, T()));
      }
    }
    issue(row + a.stages * R.stride, here);
    stage = stage + 1 == a.stages ? 0 : stage + 1;
    mean = mean_next;
    rstd = rstd_next;
  }
  cp_async_wait(0);
  // one row of partial sums per CTA
  float* part = a.part + static_cast<int64_t>(blockIdx.x) * a.D * (DB ? 2 : 1);
#pragma unroll
  for (int k = 0; k < (DB ? 2 : 1); ++k) {
    // the four warps' sums are added in order: the ring is free for them now
    float* comb = WARP ? reinterpret_cast<float*>(ring) : part + k * a.D;
    if constexpr (WARP) {
      __syncthreads();
      for (int j = threadIdx.x; j < a.D; j += 128) comb[j] = 0.0f;
    }
    for (int rr = 0; rr < Row::ROWS; ++rr) {
      if constexpr (WARP) __syncthreads();
      if (rr == R.r) {
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
          for (int i = 0; i < N; ++i) {
            float lo, hi;
            f2_get(k ? db[DB ? c : 0][i / 2] : dw[c][i / 2], lo, hi);
            const int col = R.col(c) + i;
            if (R.in(c, i)) comb[col] = (WARP ? comb[col] : 0.0f) + (i & 1 ? hi : lo);
          }
      }
    }
    if constexpr (WARP) {
      __syncthreads();
      for (int j = threadIdx.x; j < a.D; j += 128) part[k * a.D + j] = comb[j];
    }
  }
}

// Sum of P rows of partial sums: 32 columns x 32 groups of rows per CTA.
__global__ void __launch_bounds__(1024) k_norm_reduce(const float* part, int P, int64_t cols, int64_t D, float* dw,
                                                      float* db) {
  __shared__ float s[32][33];
  griddep_launch_dependents();
  griddep_wait();
  const int64_t j = static_cast<int64_t>(blockIdx.x) * 32 + (threadIdx.x & 31);
  const int g = threadIdx.x >> 5;
  float v = 0.0f;
  if (j < cols) {
#pragma unroll 10
    for (int p = g; p < P; p += 32) v += part[static_cast<int64_t>(p) * cols + j];
  }
  s[g][threadIdx.x & 31] = v;
  __syncthreads();
  // warp g adds column g of the tile; lane i holds group i's sum
  const int64_t col = static_cast<int64_t>(blockIdx.x) * 32 + g;
  const float sum = warp_sum(s[threadIdx.x & 31][g]);
  if ((threadIdx.x & 31) == 0 && col < cols) {
    if (col < D)
      dw[col] = sum;
    else
      db[col - D] = sum;
  }
}

struct Cfg {
  int maxt, e, nt;   // kernel variant (most threads; 128: a warp per row), values per thread, threads of the CTA
};

// 32 values per thread where the row is long enough, in as many warps as it
// takes, up to 8192 values; longer rows always have 512 threads, since an SM
// holds one such CTA.  (The last case: unaligned rows next to the limit.)  16
// values per thread where whole warps of 32 each would leave 15% of the CTA's
// places empty (32768 x 2049 bf16: forward 157 -> 115 us, L2 flushed, 123 with the
// rare rows' part in the kernel; backward 183 -> 134; at
// 4400 values, 9% empty, 96 -> 106 and 107 -> 136), and in a backward pass with
// the bias's gradient, whose sums and weight leave room for too few rows ahead
// (8192 x 4096 fp32 93 -> 77 us; bf16 16384 x 4096 89 -> 93, up to 2560 faster).  A
// forward pass over no more rows than SMs spreads a long row over 1024 threads,
// for latency.
Cfg norm_cfg(int64_t need, int64_t M, bool fwd, int n, bool dbias) {
  if (need <= 256) return {128, 8, 128};
  if (need <= 512) return {128, 16, 128};
  if (fwd && M <= num_sms() && need > 2048 && need <= 16384) return {1024, need <= 8192 ? 8 : 16, 1024};
  if (fwd && need <= 1024) return {128, 32, 128};   // backward: a warp could not hold both gradients' sums
  if (need <= 8192) {
    const int nt32 = static_cast<int>(align_up(ceil_div(need, 32), 32)), nt16 = static_cast<int>(align_up(ceil_div(need, 16), 32));
    const bool half = dbias ? n == 4 || need <= 2560 : 16 * nt16 * 100 <= 85 * 32 * nt32;
    return half ? Cfg{512, 16, nt16} : Cfg{512, 32, nt32};
  }
  return need <= 16384 ? Cfg{512, 32, 512} : Cfg{512, 40, 416};
}

// CTAs: what fits on the SMs, no more than there are rows.  The forward pass
// takes several times as many where a CTA still gets three rows: SMs differ in
// the bandwidth they get, and the SMs that are ahead then take more of the CTAs
// (8192 x 8192 bf16: with the residual 95 us at one wave, 85 at four, 82 at
// eight; without 53 at one, 52 at two, 60 at eight).  Unaligned rows with several
// rows per CTA: a multiple of 8, so that the rows that a CTA visits start at the
// same offset from a 16-byte boundary.
int norm_grid(int64_t M, int64_t D, int n, bool fwd, bool residual, bool dbias) {
  const Cfg c = norm_cfg(D + (D % n ? n - 1 : 0), M, fwd, n, dbias);
  const int64_t want = ceil_div(M, c.maxt == 128 ? 4 : 1);
  int64_t g = static_cast<int64_t>(num_sms()) * norm_ctas(c.nt);
  if (fwd) g *= std::max<int64_t>(1, std::min<int64_t>(residual ? 8 : 2, want / (3 * g)));
  if (D % n) g = std::max<int64_t>(8, g / 8 * 8);
  return static_cast<int>(std::max<int64_t>(1, std::min(want, g)));
}

constexpr uint32_t kNormRoom = 215u * 1024u;   // dynamic shared memory of an SM's CTAs together, 1 KB less each

// Rows ahead, as many as fit beside the SM's other CTAs, four at most; `fixed`
// bytes of shared memory follow the ring.
template <typename K>
cudaError_t launch_rows(K kernel, NormArgs a, int grid, int nt, uint32_t stage, uint32_t fixed, uint32_t least,
                        cudaStream_t st) {
  const uint32_t room = (kNormRoom + 1024u) / static_cast<uint32_t>(norm_ctas(nt)) - 1024u;
  a.stages = static_cast<int>(std::min(4u, std::max(1u, room > fixed ? (room - fixed) / stage : 0u)));
  const uint32_t smem = std::max(stage * a.stages + fixed, least);
  cudaError_t e = set_smem(kernel, smem);
  if (e != cudaSuccess) return e;
  ProfScope prof(QLORA_KC_AUX, st);
  return launch_pdl(kernel, dim3(grid), dim3(nt), smem, st, nullptr, a);
}

template <typename T, int MAXT, int E>
struct Fwd {
  static cudaError_t run(const NormArgs& a, int grid, int nt, cudaStream_t st) {
    constexpr int CH = E / Vec<T>::N;
    const uint32_t stage = static_cast<uint32_t>((1 + a.has_r) * CH * nt * 16);
    return launch_rows(a.D % Vec<T>::N == 0 ? k_norm_fwd<T, MAXT, CH, true> : k_norm_fwd<T, MAXT, CH, false>, a, grid,
                       nt, stage, 0, 0, st);
  }
};

template <typename T, int MAXT, int E>
struct Bwd {
  static cudaError_t run(const NormArgs& a, int grid, int nt, cudaStream_t st) {
    constexpr int CH = E / Vec<T>::N;
    NormArgs b = a;
    // fp32 rows above 8192 values: no room for dS in the ring
    const uint32_t array = static_cast<uint32_t>(CH * nt * 16), fixed = a.db ? nt * E * 4 : 0;
    b.ring_ds = a.has_ds && 3 * array + fixed <= (kNormRoom + 1024u) / norm_ctas(nt) - 1024u;
    const uint32_t stage = (2 + b.ring_ds) * array;
    const bool al = a.D % Vec<T>::N == 0;
    auto kernel = a.db ? (al ? k_norm_bwd<T, MAXT, CH, true, true> : k_norm_bwd<T, MAXT, CH, false, true>)
                       : (al ? k_norm_bwd<T, MAXT, CH, true, false> : k_norm_bwd<T, MAXT, CH, false, false>);
    return launch_rows(kernel, b, grid, nt, stage, fixed, MAXT == 128 ? static_cast<uint32_t>(a.D) * 4u : 0u, st);
  }
};

// the variants that both passes have
template <typename T, template <typename, int, int> class K>
cudaError_t pick(const Cfg& c, const NormArgs& a, int grid, cudaStream_t st) {
  if (c.maxt == 128) return c.e == 8 ? K<T, 128, 8>::run(a, grid, c.nt, st) : K<T, 128, 16>::run(a, grid, c.nt, st);
  return c.e == 32 ? K<T, 512, 32>::run(a, grid, c.nt, st) : K<T, 512, 40>::run(a, grid, c.nt, st);
}

template <typename T>
cudaError_t run_fwd(const NormArgs& a, cudaStream_t st) {
  constexpr int N = Vec<T>::N;
  const Cfg c = norm_cfg(a.D + (a.D % N ? N - 1 : 0), a.M, true, N, false);
  const int grid = norm_grid(a.M, a.D, N, true, a.has_r, false);
  if (c.maxt == 1024)
    return c.e == 8 ? Fwd<T, 1024, 8>::run(a, grid, c.nt, st) : Fwd<T, 1024, 16>::run(a, grid, c.nt, st);
  if (c.maxt == 128 && c.e == 32) return Fwd<T, 128, 32>::run(a, grid, c.nt, st);
  if (c.maxt == 512 && c.e == 16) return Fwd<T, 512, 16>::run(a, grid, c.nt, st);
  return pick<T, Fwd>(c, a, grid, st);
}

cudaError_t reduce(const NormArgs& a, int parts, cudaStream_t st) {
  const int64_t cols = static_cast<int64_t>(a.D) * (a.db ? 2 : 1);
  ProfScope prof(QLORA_KC_AUX, st);
  return launch_pdl(k_norm_reduce, dim3(static_cast<unsigned>(ceil_div(cols, 32))), dim3(1024), 0, st, nullptr,
                    static_cast<const float*>(a.part), parts, cols, static_cast<int64_t>(a.D), a.dw, a.db);
}

template <typename T>
cudaError_t run_bwd(const NormArgs& a, cudaStream_t st) {
  constexpr int N = Vec<T>::N;
  const int grid = norm_grid(a.M, a.D, N, false, false, a.db != nullptr);
  const Cfg c = norm_cfg(a.D + (a.D % N ? N - 1 : 0), a.M, false, N, a.db != nullptr);
  cudaError_t e = c.maxt == 512 && c.e == 16 ? Bwd<T, 512, 16>::run(a, grid, c.nt, st) : pick<T, Bwd>(c, a, grid, st);
  return e != cudaSuccess ? e : reduce(a, grid, st);
}

}  // namespace

size_t norm_workspace_bytes(int64_t M, int64_t D, int dtype, bool dbias) {
  if (M == 0) return 0;
  return align_up(static_cast<size_t>(norm_grid(M, D, dtype == QLORA_DT_BF16 ? 8 : 4, false, false, dbias)) * D * (dbias ? 2 : 1) * 4,
                  256);
}

cudaError_t launch_norm_fwd(const NormArgs& a, cudaStream_t st) {
  return a.dtype == QLORA_DT_BF16 ? run_fwd<__nv_bfloat16>(a, st) : run_fwd<float>(a, st);
}

cudaError_t launch_norm_bwd(const NormArgs& a, cudaStream_t st) {
  if (a.M == 0) return reduce(a, 0, st);   // no rows: the sums are zero
  return a.dtype == QLORA_DT_BF16 ? run_bwd<__nv_bfloat16>(a, st) : run_bwd<float>(a, st);
}

}  // namespace qlora
