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
// Bound: HBM.  Both passes keep a row in registers between its reductions, so
// every activation is read and written once.
#include "qlora_device.cuh"
#include "qlora_internal.h"
#include "qlora_vec.cuh"

namespace qlora {

namespace {

// A reduction over the CTA's threads: one barrier each.  The caller alternates
// `buf` between two halves of the scratch, so a fast warp's next partial sums
// cannot meet a slow warp's reads.  Every thread adds the warps' sums in the
// same order.
template <int NT>
__device__ __forceinline__ float cta_sum(float v, float* scratch, int buf) {
  v = warp_sum(v);
  if constexpr (NT == 32) return v;
  constexpr int NW = NT / 32;
  float* s = scratch + buf * 32;
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
  __syncthreads();
  float t = 0.0f;
#pragma unroll
  for (int w = 0; w < NW; ++w) t += s[w];
  return t;
}

// Columns col .. col + N - 1 of the weight or bias (bf16 or fp32, the same for
// all threads; base 16-byte aligned).  Zero outside [0, D).
template <int N>
__device__ __forceinline__ void load_w(const void* w, bool bf16, int col, int D, float (&f)[N]) {
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
}

// ---------------------------------------------------------------------------
// Forward.  NT threads hold one row, CH windows each; a warp holds a row of up
// to 1024 values by itself (4 rows per CTA).  ALIGNED: every row starts on a
// 16-byte boundary and ends on one, so no element needs a bounds check.
// ---------------------------------------------------------------------------
template <typename T, int NT, int CH, bool ALIGNED>
__global__ void __launch_bounds__(NT == 32 ? 128 : NT) k_norm_fwd(NormArgs a) {
  constexpr int N = Vec<T>::N;
  constexpr int ROWS = NT == 32 ? 4 : 1;
  __shared__ float scratch[64];
  const int t = NT == 32 ? (threadIdx.x & 31) : threadIdx.x;
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * ROWS + (NT == 32 ? (threadIdx.x >> 5) : 0);
  griddep_launch_dependents();
  griddep_wait();
  for (int64_t row = row0; row < a.M; row += static_cast<int64_t>(gridDim.x) * ROWS) {
    const int64_t at = row * a.D;
    const int sh = ALIGNED ? 0 : static_cast<int>(at % N);
    const T* x = reinterpret_cast<const T*>(a.X) + at;
    float v[CH][N];
#pragma unroll
    for (int c = 0; c < CH; ++c) load_window(x, (t + c * NT) * N - sh, a.D, 0.0f, v[c]);
    if (a.has_r) {
      const T* r = reinterpret_cast<const T*>(a.R) + at;
      T* s = reinterpret_cast<T*>(a.S) + at;
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int col = (t + c * NT) * N - sh;
        float q[N];
        load_window(r, col, a.D, 0.0f, q);
#pragma unroll
        for (int i = 0; i < N; ++i) v[c][i] = to_f32(from_f32<T>(v[c][i] + q[i]));
        store_window(s, col, a.D, v[c]);
      }
    }
    float mean = 0.0f;
    if (!a.rms) {
      float sum = 0.0f;
#pragma unroll
      for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int i = 0; i < N; ++i) sum += v[c][i];
      mean = cta_sum<NT>(sum, scratch, 0) / static_cast<float>(a.D);
    }
    float sq = 0.0f;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int col = (t + c * NT) * N - sh;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const bool in = ALIGNED ? col < a.D : (col + i >= 0 && col + i < a.D);
        v[c][i] = in ? v[c][i] - mean : 0.0f;
        sq = fmaf(v[c][i], v[c][i], sq);
      }
    }
    const float rstd = 1.0f / sqrtf(cta_sum<NT>(sq, scratch, 1) / static_cast<float>(a.D) + a.eps);
    if (t == 0) {
      if (a.mean_out) a.mean_out[row] = mean;
      if (a.rstd_out) a.rstd_out[row] = rstd;
    }
    T* y = reinterpret_cast<T*>(a.Y) + at;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int col = (t + c * NT) * N - sh;
      if (col >= a.D) continue;
      float w[N];
      load_w<N>(a.w, a.wdtype == QLORA_DT_BF16, col, a.D, w);
#pragma unroll
      for (int i = 0; i < N; ++i) v[c][i] = v[c][i] * rstd * w[i];
      if (a.has_b) {
        load_w<N>(a.b, a.wdtype == QLORA_DT_BF16, col, a.D, w);
#pragma unroll
        for (int i = 0; i < N; ++i) v[c][i] += w[i];
      }
      store_window(y, col, a.D, v[c]);
    }
    if constexpr (NT != 32) {
      // rms uses one reduction per row: keep the next row's from this row's reads
      if (a.rms) __syncthreads();
    }
  }
}

// ---------------------------------------------------------------------------
// Backward.  A CTA (or warp) walks over rows gridDim apart.  Its threads keep
// the same columns for every row, so the weight's gradient is summed in
// registers and leaves them once, as one row of partial sums per CTA;
// k_norm_reduce adds those in a fixed order.  Rows that do not start on 16-byte
// boundaries shift the windows; the grid is then a multiple of N rows apart, so
// a thread's columns still never change.
// ---------------------------------------------------------------------------
template <typename T, int NT, int CH, bool ALIGNED, bool DB>
__global__ void __launch_bounds__(NT == 32 ? 128 : NT) k_norm_bwd(NormArgs a) {
  constexpr int N = Vec<T>::N;
  constexpr int ROWS = NT == 32 ? 4 : 1;
  __shared__ float scratch[128];
  extern __shared__ float comb[];
  const int t = NT == 32 ? (threadIdx.x & 31) : threadIdx.x;
  const int r = NT == 32 ? (threadIdx.x >> 5) : 0;
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * ROWS + r;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * ROWS;
  griddep_launch_dependents();
  griddep_wait();
  const int sh = ALIGNED ? 0 : static_cast<int>((row0 * a.D) % N);
  float dw[CH][N], db[DB ? CH : 1][N], w[CH][N];
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    load_w<N>(a.w, a.wdtype == QLORA_DT_BF16, (t + c * NT) * N - sh, a.D, w[c]);
#pragma unroll
    for (int i = 0; i < N; ++i) dw[c][i] = 0.0f;
    if constexpr (DB)
#pragma unroll
      for (int i = 0; i < N; ++i) db[c][i] = 0.0f;
  }
  const float inv_d = 1.0f / static_cast<float>(a.D);
  int buf = 0;
  for (int64_t row = row0; row < a.M; row += stride, buf ^= 1) {
    const int64_t at = row * a.D;
    const T* x = reinterpret_cast<const T*>(a.X) + at;
    const T* dy = reinterpret_cast<const T*>(a.dY) + at;
    const float mean = a.rms ? 0.0f : a.mean_in[row], rstd = a.rstd_in[row];
    float xh[CH][N], g[CH][N];
    float c1 = 0.0f, c2 = 0.0f;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int col = (t + c * NT) * N - sh;
      load_window(x, col, a.D, mean, xh[c]);
      load_window(dy, col, a.D, 0.0f, g[c]);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        xh[c][i] = (xh[c][i] - mean) * rstd;
        dw[c][i] = fmaf(g[c][i], xh[c][i], dw[c][i]);
        if constexpr (DB) db[c][i] += g[c][i];
        g[c][i] *= w[c][i];
        c1 += g[c][i];
        c2 = fmaf(g[c][i], xh[c][i], c2);
      }
    }
    if constexpr (NT == 32) {
      c1 = warp_sum(c1);
      c2 = warp_sum(c2);
    } else {
      constexpr int NW = NT / 32;
      c1 = warp_sum(c1);
      c2 = warp_sum(c2);
      float* s = scratch + buf * 64;
      if ((threadIdx.x & 31) == 0) {
        s[threadIdx.x >> 5] = c1;
        s[32 + (threadIdx.x >> 5)] = c2;
      }
      __syncthreads();
      c1 = c2 = 0.0f;
#pragma unroll
      for (int i = 0; i < NW; ++i) {
        c1 += s[i];
        c2 += s[32 + i];
      }
    }
    c1 = a.rms ? 0.0f : c1 * inv_d;
    c2 *= inv_d;
    if (a.dX) {
      T* dx = reinterpret_cast<T*>(a.dX) + at;
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int col = (t + c * NT) * N - sh;
        if (col >= a.D) continue;
        float o[N];
#pragma unroll
        for (int i = 0; i < N; ++i) o[i] = rstd * (g[c][i] - c1 - xh[c][i] * c2);
        if (a.has_ds) {
          float q[N];
          load_window(reinterpret_cast<const T*>(a.dS) + at, col, a.D, 0.0f, q);
#pragma unroll
          for (int i = 0; i < N; ++i) o[i] += q[i];
        }
        store_window(dx, col, a.D, o);
      }
    }
  }
  // one row of partial sums per CTA
  float* part = a.part + static_cast<int64_t>(blockIdx.x) * a.D * (DB ? 2 : 1);
#pragma unroll
  for (int k = 0; k < (DB ? 2 : 1); ++k) {
    if constexpr (NT == 32) {
      for (int j = threadIdx.x; j < a.D; j += 128) comb[j] = 0.0f;
      for (int rr = 0; rr < ROWS; ++rr) {
        __syncthreads();
        if (rr == r) {
#pragma unroll
          for (int c = 0; c < CH; ++c)
#pragma unroll
            for (int i = 0; i < N; ++i) {
              const int col = (t + c * NT) * N - sh + i;
              if (col >= 0 && col < a.D) comb[col] += k ? db[DB ? c : 0][i] : dw[c][i];
            }
        }
      }
      __syncthreads();
      for (int j = threadIdx.x; j < a.D; j += 128) part[k * a.D + j] = comb[j];
      __syncthreads();
    } else {
#pragma unroll
      for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const int col = (t + c * NT) * N - sh + i;
          if (col >= 0 && col < a.D) part[k * a.D + col] = k ? db[DB ? c : 0][i] : dw[c][i];
        }
    }
  }
}

// Sum of P rows of partial sums: 32 columns x 8 groups of rows per CTA.
__global__ void __launch_bounds__(256) k_norm_reduce(const float* __restrict__ part, int P, int64_t cols, int64_t D,
                                                     float* __restrict__ dw, float* __restrict__ db) {
  __shared__ float s[8][33];
  griddep_launch_dependents();
  griddep_wait();
  const int64_t j = static_cast<int64_t>(blockIdx.x) * 32 + (threadIdx.x & 31);
  const int g = threadIdx.x >> 5;
  float v = 0.0f;
  if (j < cols)
    for (int p = g; p < P; p += 8) v += part[static_cast<int64_t>(p) * cols + j];
  s[g][threadIdx.x & 31] = v;
  __syncthreads();
  if (g == 0 && j < cols) {
#pragma unroll
    for (int i = 1; i < 8; ++i) v += s[i][threadIdx.x & 31];
    if (j < D)
      dw[j] = v;
    else
      db[j - D] = v;
  }
}

struct Cfg {
  int nt, e;   // threads per row, values per thread
};

// Forward: as few threads per row as hold it with 16 to 32 values each, so that
// several rows are in flight on an SM; for no more rows than SMs the row is
// spread over up to 1024 threads, for latency.
Cfg fwd_cfg(int64_t need, int64_t M) {
  if (need <= 256) return {32, 8};
  if (M <= num_sms()) {
    if (need <= 8192) return {1024, 8};
    return {1024, 17};
  }
  if (need <= 512) return {32, 16};
  if (need <= 1024) return {32, 32};
  if (need <= 2048) return {128, 16};
  if (need <= 4096) return {256, 16};
  if (need <= 8192) return {256, 32};
  return {544, 32};
}

Cfg bwd_cfg(int64_t need) {
  if (need <= 256) return {32, 8};
  if (need <= 512) return {32, 16};
  if (need <= 1024) return {32, 32};
  if (need <= 2048) return {128, 16};
  if (need <= 4096) return {256, 16};
  if (need <= 8192) return {512, 16};
  return {544, 32};
}

template <typename T, int NT, int E>
cudaError_t run_fwd(const NormArgs& a, bool aligned, cudaStream_t st) {
  constexpr int CH = (E + Vec<T>::N - 1) / Vec<T>::N;
  constexpr int ROWS = NT == 32 ? 4 : 1;
  const dim3 block(NT == 32 ? 128 : NT);
  const dim3 grid(static_cast<unsigned>(std::min<int64_t>(ceil_div(a.M, ROWS), int64_t(1) << 30)));
  ProfScope prof(QLORA_KC_AUX, st);
  return aligned ? launch_pdl(k_norm_fwd<T, NT, CH, true>, grid, block, 0, st, nullptr, a)
                 : launch_pdl(k_norm_fwd<T, NT, CH, false>, grid, block, 0, st, nullptr, a);
}

template <typename T>
cudaError_t pick_fwd(const NormArgs& a, cudaStream_t st) {
  const bool aligned = a.D % Vec<T>::N == 0;
  const Cfg c = fwd_cfg(a.D + (aligned ? 0 : Vec<T>::N - 1), a.M);
  switch (c.nt * 64 + c.e) {
    case 32 * 64 + 8: return run_fwd<T, 32, 8>(a, aligned, st);
    case 32 * 64 + 16: return run_fwd<T, 32, 16>(a, aligned, st);
    case 32 * 64 + 32: return run_fwd<T, 32, 32>(a, aligned, st);
    case 128 * 64 + 16: return run_fwd<T, 128, 16>(a, aligned, st);
    case 256 * 64 + 16: return run_fwd<T, 256, 16>(a, aligned, st);
    case 256 * 64 + 32: return run_fwd<T, 256, 32>(a, aligned, st);
    case 1024 * 64 + 8: return run_fwd<T, 1024, 8>(a, aligned, st);
    case 1024 * 64 + 17: return run_fwd<T, 1024, 17>(a, aligned, st);
    default: return run_fwd<T, 544, 32>(a, aligned, st);
  }
}

template <typename T, int NT, int E, bool ALIGNED, bool DB>
cudaError_t run_bwd3(const NormArgs& a, int grid, cudaStream_t st) {
  constexpr int CH = E / Vec<T>::N;
  const dim3 block(NT == 32 ? 128 : NT);
  const size_t smem = NT == 32 ? static_cast<size_t>(a.D) * 4 : 0;
  ProfScope prof(QLORA_KC_AUX, st);
  return launch_pdl(k_norm_bwd<T, NT, CH, ALIGNED, DB>, dim3(grid), block, smem, st, nullptr, a);
}

template <typename T, int NT, int E>
cudaError_t run_bwd(const NormArgs& a, bool aligned, int grid, cudaStream_t st) {
  if (a.db) return aligned ? run_bwd3<T, NT, E, true, true>(a, grid, st) : run_bwd3<T, NT, E, false, true>(a, grid, st);
  return aligned ? run_bwd3<T, NT, E, true, false>(a, grid, st) : run_bwd3<T, NT, E, false, false>(a, grid, st);
}

// CTAs of the backward pass: one or more per SM, no more than there are rows.
// Unaligned rows with several rows per CTA: a multiple of 8, so that rows a CTA
// visits start at the same offset from a 16-byte boundary.
int bwd_grid(int64_t M, int64_t D, int n) {
  const Cfg c = bwd_cfg(D + (D % n ? n - 1 : 0));
  const int rows = c.nt == 32 ? 4 : 1;
  const int64_t want = ceil_div(M, rows);
  int64_t g = static_cast<int64_t>(num_sms()) * (c.nt == 32 ? 4 : c.nt <= 256 ? 2 : 1);
  if (D % n) g = g / 8 * 8;
  return static_cast<int>(std::max<int64_t>(1, std::min(want, g)));
}

template <typename T>
cudaError_t pick_bwd(const NormArgs& a, cudaStream_t st) {
  const bool aligned = a.D % Vec<T>::N == 0;
  const Cfg c = bwd_cfg(a.D + (aligned ? 0 : Vec<T>::N - 1));
  const int grid = bwd_grid(a.M, a.D, Vec<T>::N);
  cudaError_t e;
  switch (c.nt * 64 + c.e) {
    case 32 * 64 + 8: e = run_bwd<T, 32, 8>(a, aligned, grid, st); break;
    case 32 * 64 + 16: e = run_bwd<T, 32, 16>(a, aligned, grid, st); break;
    case 32 * 64 + 32: e = run_bwd<T, 32, 32>(a, aligned, grid, st); break;
    case 128 * 64 + 16: e = run_bwd<T, 128, 16>(a, aligned, grid, st); break;
    case 256 * 64 + 16: e = run_bwd<T, 256, 16>(a, aligned, grid, st); break;
    case 512 * 64 + 16: e = run_bwd<T, 512, 16>(a, aligned, grid, st); break;
    default: e = run_bwd<T, 544, 32>(a, aligned, grid, st); break;
  }
  if (e != cudaSuccess) return e;
  const int64_t cols = a.D * (a.db ? 2 : 1);
  ProfScope prof(QLORA_KC_AUX, st);
  return launch_pdl(k_norm_reduce, dim3(static_cast<unsigned>(ceil_div(cols, 32))), dim3(256), 0, st, nullptr,
                    static_cast<const float*>(a.part), grid, cols, static_cast<int64_t>(a.D), a.dw, a.db);
}

}  // namespace

size_t norm_workspace_bytes(int64_t M, int64_t D, int dtype, bool dbias) {
  if (M == 0) return 0;
  return align_up(static_cast<size_t>(bwd_grid(M, D, dtype == QLORA_DT_BF16 ? 8 : 4)) * D * (dbias ? 2 : 1) * 4, 256);
}

cudaError_t launch_norm_fwd(const NormArgs& a, cudaStream_t st) {
  return a.dtype == QLORA_DT_BF16 ? pick_fwd<__nv_bfloat16>(a, st) : pick_fwd<float>(a, st);
}

cudaError_t launch_norm_bwd(const NormArgs& a, cudaStream_t st) {
  if (a.M == 0) {   // no rows: the sums are zero
    const int64_t cols = static_cast<int64_t>(a.D) * (a.db ? 2 : 1);
    ProfScope prof(QLORA_KC_AUX, st);
    return launch_pdl(k_norm_reduce, dim3(static_cast<unsigned>(ceil_div(cols, 32))), dim3(256), 0, st, nullptr,
                      static_cast<const float*>(nullptr), 0, cols, static_cast<int64_t>(a.D), a.dw, a.db);
  }
  return a.dtype == QLORA_DT_BF16 ? pick_bwd<__nv_bfloat16>(a, st) : pick_bwd<float>(a, st);
}

}  // namespace qlora
