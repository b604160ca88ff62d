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
// Rows in flight hide the loads: registers are held to what lets about 96 KB of
// loads be outstanding on an SM.
constexpr int fwd_ctas(int nt, int e) { return nt == 32 ? (e > 16 ? 5 : 8) : nt * e <= 2048 ? 8 : nt * e <= 4096 ? 4 : nt * e <= 8192 ? (nt > 512 ? 1 : 3) : 1; }

template <typename T, int NT, int CH, bool ALIGNED>
__global__ void __launch_bounds__(NT == 32 ? 128 : NT, fwd_ctas(NT, CH * Vec<T>::N)) k_norm_fwd(NormArgs a) {
  constexpr int N = Vec<T>::N;
  constexpr int ROWS = NT == 32 ? 4 : 1;
  __shared__ float scratch[64];
  const int t = NT == 32 ? (threadIdx.x & 31) : threadIdx.x;
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * ROWS + (NT == 32 ? (threadIdx.x >> 5) : 0);
  griddep_launch_dependents();
  griddep_wait();
#pragma unroll 1
  for (int64_t row = row0; row < a.M; row += static_cast<int64_t>(gridDim.x) * ROWS) {
    const int64_t at = row * a.D;
    const int sh = ALIGNED ? 0 : static_cast<int>(at % N);
    const T* x = reinterpret_cast<const T*>(a.X) + at;
    // all of the row's loads before their first use: S may be R's memory, so the
    // compiler would keep a window's load behind the store of the one before
    float v[CH][N];
    uint4 raw[CH];
#pragma unroll
    for (int c = 0; c < CH; ++c) raw[c] = load_raw<T, ALIGNED>(x, (t + c * NT) * N - sh, a.D);
    if (a.has_r) {
      const T* r = reinterpret_cast<const T*>(a.R) + at;
      T* s = reinterpret_cast<T*>(a.S) + at;
      uint4 q[CH];
#pragma unroll
      for (int c = 0; c < CH; ++c) q[c] = load_raw<T, ALIGNED>(r, (t + c * NT) * N - sh, a.D);
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        float f[N];
        Vec<T>::unpack(raw[c], v[c]);
        Vec<T>::unpack(q[c], f);
#pragma unroll
        for (int i = 0; i < N; ++i) v[c][i] += f[i];
        raw[c] = Vec<T>::pack(v[c]);
        store_raw<T, ALIGNED>(s, (t + c * NT) * N - sh, a.D, raw[c]);
      }
    }
#pragma unroll
    for (int c = 0; c < CH; ++c) Vec<T>::unpack(raw[c], v[c]);
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
      store_raw<T, ALIGNED>(y, col, a.D, Vec<T>::pack(v[c]));
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
//
// The rows' loads run a.stages rows ahead through a ring in shared memory
// (cp.async): registers hold the gradient's sums and cannot hold rows in
// flight as well.  Each thread reads back only the 16-byte slots that it filled
// itself, so the ring needs no barrier; the one barrier per row belongs to the
// row's two sums.  Rows above 8192 values are held by a pair of CTAs (a cluster
// of two SMs), which exchange those sums through each other's shared memory: one
// CTA of 1024 threads would have 64 registers per thread and spill the sums.
// ---------------------------------------------------------------------------
constexpr int bwd_ctas(int nt, int e) { return nt == 32 ? (e > 8 ? 4 : 6) : nt == 64 ? 8 : nt == 128 ? 4 : nt == 256 ? 2 : 1; }

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// a float into this CTA's shared memory and into the pair's other CTA's
__device__ __forceinline__ void st_pair(float* p, float v, uint32_t other) {
  *p = v;
  uint32_t remote;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(smem_u32(p)), "r"(other));
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(remote), "f"(v) : "memory");
}

template <typename T, int NT, int CH, bool ALIGNED, bool DB, bool PAIR>
__global__ void __launch_bounds__(NT == 32 ? 128 : NT, bwd_ctas(NT, CH * Vec<T>::N)) k_norm_bwd(NormArgs a) {
  constexpr int N = Vec<T>::N;
  constexpr int ROWS = NT == 32 ? 4 : 1;
  constexpr int TB = NT == 32 ? 128 : NT;     // threads of the CTA
  constexpr int STEP = PAIR ? 2 * NT : NT;    // threads of a row
  __shared__ float scratch[128];
  extern __shared__ __align__(16) uint8_t ring[];
  const int half = PAIR ? (blockIdx.x & 1) : 0;
  const int t = NT == 32 ? (threadIdx.x & 31) : threadIdx.x + half * NT;
  const int r = NT == 32 ? (threadIdx.x >> 5) : 0;
  const int64_t row0 = static_cast<int64_t>(PAIR ? blockIdx.x >> 1 : blockIdx.x) * ROWS + r;
  const int64_t stride = static_cast<int64_t>(PAIR ? gridDim.x >> 1 : gridDim.x) * ROWS;
  const uint32_t slot0 = smem_u32(ring) + threadIdx.x * 16u;
  const int arrays = 2 + a.has_ds;
  const uint32_t stage_bytes = static_cast<uint32_t>(arrays * CH * TB * 16);
  griddep_launch_dependents();
  griddep_wait();
  const int sh = ALIGNED ? 0 : static_cast<int>((row0 * a.D) % N);
  const bool wbf16 = a.wdtype == QLORA_DT_BF16;

  // window c of the row: what it can read of the row (a window past the row's
  // end reads nothing, one that starts in the row before reads that too)
  auto issue = [&](int64_t row, uint32_t stage) {
    if (row < a.M) {
      const int64_t at = row * a.D;
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int col = (t + c * STEP) * N - sh;
        const int bytes = min(max(a.D - col, 0), N) * static_cast<int>(sizeof(T));
        const int64_t src = at + (bytes ? col : 0);
        const uint32_t dst = slot0 + stage + static_cast<uint32_t>(c * TB * 16);
        cp_async16(dst, reinterpret_cast<const T*>(a.X) + (bytes ? src : at - sh), bytes);
        cp_async16(dst + CH * TB * 16, reinterpret_cast<const T*>(a.dY) + (bytes ? src : at - sh), bytes);
        if (a.has_ds)
          cp_async16(dst + 2 * CH * TB * 16, reinterpret_cast<const T*>(a.dS) + (bytes ? src : at - sh), bytes);
      }
    }
    cp_async_commit();
  };

  float dw[CH][N], db[DB ? CH : 1][N], w[CH][N];
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    load_w<N>(a.w, wbf16, (t + c * STEP) * N - sh, a.D, w[c]);
#pragma unroll
    for (int i = 0; i < N; ++i) dw[c][i] = 0.0f;
    if constexpr (DB)
#pragma unroll
      for (int i = 0; i < N; ++i) db[c][i] = 0.0f;
  }
  for (int s = 0; s < a.stages; ++s) issue(row0 + s * stride, s * stage_bytes);
  if constexpr (PAIR) cluster_sync();   // both CTAs run before either writes to the other

  const float inv_d = 1.0f / static_cast<float>(a.D);
  float mean = 0.0f, rstd = 0.0f;
  if (row0 < a.M) {
    mean = a.mean_in[row0];
    rstd = a.rstd_in[row0];
  }
  int buf = 0, stage = 0;
#pragma unroll 1
  for (int64_t row = row0; row < a.M; row += stride, buf ^= 1) {
    const int64_t next = min(row + stride, a.M - 1);
    const float mean_next = a.mean_in[next], rstd_next = a.rstd_in[next];
    if (a.rms) mean = 0.0f;
    const uint32_t slot = slot0 + stage * stage_bytes;
    cp_async_wait(a.stages - 1);
    // xh and g = dY w of window c
    auto take = [&](int c, float (&xh)[N], float (&dy)[N]) {
      Vec<T>::unpack(lds128(slot + c * TB * 16), xh);
      Vec<T>::unpack(lds128(slot + (CH + c) * TB * 16), dy);
      if (!ALIGNED && c == 0 && t * N - sh < 0) {   // values of the row before
#pragma unroll
        for (int i = 0; i < N; ++i)
          if (i < sh) xh[i] = dy[i] = 0.0f;
      }
#pragma unroll
      for (int i = 0; i < N; ++i) xh[i] = (xh[i] - mean) * rstd;
    };
    float c1 = 0.0f, c2 = 0.0f;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      float xh[N], dy[N];
      take(c, xh, dy);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        // outside the row dY and w are zero, so whatever xh is there adds nothing
        dw[c][i] = fmaf(dy[i], xh[i], dw[c][i]);
        if constexpr (DB) db[c][i] += dy[i];
        const float g = dy[i] * w[c][i];
        c1 += g;
        c2 = fmaf(g, xh[i], c2);
      }
    }
    c1 = warp_sum(c1);
    c2 = warp_sum(c2);
    if constexpr (NT != 32) {
      constexpr int NW = STEP / 32;
      float* s = scratch + buf * 64;
      if ((threadIdx.x & 31) == 0) {
        const int at = t >> 5;
        if constexpr (PAIR) {
          st_pair(s + at, c1, half ^ 1);
          st_pair(s + 32 + at, c2, half ^ 1);
        } else {
          s[at] = c1;
          s[32 + at] = c2;
        }
      }
      if constexpr (PAIR) {
        __syncwarp();
        cluster_sync();
      } else {
        __syncthreads();
      }
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
      T* dx = reinterpret_cast<T*>(a.dX) + row * a.D;
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int col = (t + c * STEP) * N - sh;
        float xh[N], o[N];
        take(c, xh, o);
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const float g = o[i] * w[c][i];
          o[i] = rstd * (g - c1 - xh[i] * c2);
        }
        if (a.has_ds) {
          float q[N];
          Vec<T>::unpack(lds128(slot + (2 * CH + c) * TB * 16), q);
#pragma unroll
          for (int i = 0; i < N; ++i) o[i] += q[i];
        }
        store_raw<T, ALIGNED>(dx, col, a.D, Vec<T>::pack(o));
      }
    }
    issue(row + a.stages * stride, stage * stage_bytes);
    stage = stage + 1 == a.stages ? 0 : stage + 1;
    mean = mean_next;
    rstd = rstd_next;
  }
  cp_async_wait(0);
  __syncwarp();
  if constexpr (PAIR) cluster_sync();   // neither CTA leaves while the other may still write to it
  // one row of partial sums per CTA (or pair)
  float* part = a.part + static_cast<int64_t>(PAIR ? blockIdx.x >> 1 : blockIdx.x) * a.D * (DB ? 2 : 1);
#pragma unroll
  for (int k = 0; k < (DB ? 2 : 1); ++k) {
    if constexpr (NT == 32) {
      // the four warps' sums, added in order: the ring is free for them now
      float* comb = reinterpret_cast<float*>(ring);
      __syncthreads();
      for (int j = threadIdx.x; j < a.D; j += 128) comb[j] = 0.0f;
      for (int rr = 0; rr < ROWS; ++rr) {
        __syncthreads();
        if (rr == r) {
#pragma unroll
          for (int c = 0; c < CH; ++c)
#pragma unroll
            for (int i = 0; i < N; ++i) {
              const int col = (t + c * STEP) * N - sh + i;
              if (col >= 0 && col < a.D) comb[col] += k ? db[DB ? c : 0][i] : dw[c][i];
            }
        }
      }
      __syncthreads();
      for (int j = threadIdx.x; j < a.D; j += 128) part[k * a.D + j] = comb[j];
    } else {
#pragma unroll
      for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const int col = (t + c * STEP) * N - sh + i;
          if (col >= 0 && col < a.D) part[k * a.D + col] = k ? db[DB ? c : 0][i] : dw[c][i];
        }
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
#pragma unroll 4
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
  if (need <= 1024) return {64, 16};
  if (need <= 2048) return {128, 16};
  if (need <= 4096) return {256, 16};
  if (need <= 8192) return {512, 16};
  if (need <= 16384) return {1024, 16};   // a pair of 512
  return {1024, 17};
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

template <typename T, int NTROW, int E, bool ALIGNED, bool DB>
cudaError_t run_bwd3(NormArgs a, int grid, cudaStream_t st) {
  constexpr bool PAIR = NTROW == 1024;
  constexpr int NT = PAIR ? 512 : NTROW;
  constexpr int CH = (E + Vec<T>::N - 1) / Vec<T>::N;
  constexpr int TB = NT == 32 ? 128 : NT;
  // as many rows ahead as fit beside the SM's other CTAs, four at most
  const uint32_t stage = static_cast<uint32_t>((2 + a.has_ds) * CH * TB * 16);
  const uint32_t room = 200u * 1024u / bwd_ctas(NT, CH * Vec<T>::N);
  a.stages = static_cast<int>(std::min(4u, std::max(1u, room / stage)));
  const uint32_t smem = std::max(stage * a.stages, NT == 32 ? static_cast<uint32_t>(a.D) * 4u : 0u);
  auto kernel = k_norm_bwd<T, NT, CH, ALIGNED, DB, PAIR>;
  cudaError_t e = set_smem(kernel, smem);
  if (e != cudaSuccess) return e;
  ProfScope prof(QLORA_KC_AUX, st);
  const dim3 pair(2, 1, 1);
  return launch_pdl(kernel, dim3(PAIR ? 2 * grid : grid), dim3(TB), smem, st, PAIR ? &pair : nullptr, a);
}

template <typename T, int NT, int E>
cudaError_t run_bwd(const NormArgs& a, bool aligned, int grid, cudaStream_t st) {
  if (a.db) return aligned ? run_bwd3<T, NT, E, true, true>(a, grid, st) : run_bwd3<T, NT, E, false, true>(a, grid, st);
  return aligned ? run_bwd3<T, NT, E, true, false>(a, grid, st) : run_bwd3<T, NT, E, false, false>(a, grid, st);
}

// CTAs (or pairs) of the backward pass: what fits on the SMs, no more than there
// are rows; each leaves one row of partial sums.
// Unaligned rows with several rows per CTA: a multiple of 8, so that the rows a
// CTA visits start at the same offset from a 16-byte boundary.
int bwd_grid(int64_t M, int64_t D, int n) {
  const Cfg c = bwd_cfg(D + (D % n ? n - 1 : 0));
  const int rows = c.nt == 32 ? 4 : 1;
  const int64_t want = ceil_div(M, rows);
  int64_t g = c.nt == 1024 ? num_sms() / 2 : static_cast<int64_t>(num_sms()) * bwd_ctas(c.nt, c.e);
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
    case 64 * 64 + 16: e = run_bwd<T, 64, 16>(a, aligned, grid, st); break;
    case 128 * 64 + 16: e = run_bwd<T, 128, 16>(a, aligned, grid, st); break;
    case 256 * 64 + 16: e = run_bwd<T, 256, 16>(a, aligned, grid, st); break;
    case 512 * 64 + 16: e = run_bwd<T, 512, 16>(a, aligned, grid, st); break;
    case 1024 * 64 + 16: e = run_bwd<T, 1024, 16>(a, aligned, grid, st); break;
    default: e = run_bwd<T, 1024, 17>(a, aligned, grid, st); break;
  }
  if (e != cudaSuccess) return e;
  const int64_t cols = a.D * (a.db ? 2 : 1);
  ProfScope prof(QLORA_KC_AUX, st);
  return launch_pdl(k_norm_reduce, dim3(static_cast<unsigned>(ceil_div(cols, 32))), dim3(1024), 0, st, nullptr,
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
    return launch_pdl(k_norm_reduce, dim3(static_cast<unsigned>(ceil_div(cols, 32))), dim3(1024), 0, st, nullptr,
                      static_cast<const float*>(nullptr), 0, cols, static_cast<int64_t>(a.D), a.dw, a.db);
  }
  return a.dtype == QLORA_DT_BF16 ? pick_bwd<__nv_bfloat16>(a, st) : pick_bwd<float>(a, st);
}

}  // namespace qlora
