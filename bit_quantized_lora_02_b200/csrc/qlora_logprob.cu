// qlora_logprob.cu -- log probabilities of given tokens from logits, with the
// entropy and the top alternatives, and their gradient.
//
// Per row of V logits z, with m = max z and S = sum exp(z - m):
//     lse = m + log S,   logp = z_t - lse,
//     H = log S - G / S,   G = sum exp(z - m) (z - m),
//     dz = dlogp (1[j = t] - p) - dH p (log p + H),   p = exp(z - lse).
// H is summed from terms of one sign, so nothing cancels where one token has
// nearly all of the probability.  Everything is held in fp32.
//
// Forward, one pass over the row: each thread keeps a running maximum with S and
// G relative to it and rescales them when a batch of 4 x 16 bytes raises the
// maximum; the threads' triples are then merged.  Few rows are split over
// clusters of up to 8 CTAs, whose results meet in the first one's shared memory.
//
// Top alternatives without a second pass over memory: the threads' maxima give
// those of 32 groups of threads, and the top-th largest of these is a bound T
// that at least `top` logits reach.  Only threads whose own maximum reaches T
// look through their logits again (L2) and list what reaches it: about
// 32 log(32 / (32 - top)) logits of distinct values.  A rank count over the list orders it,
// equal logits by their index.  Lists that overflow (rows with few distinct
// values, as under a mask) take `collect_many`.
//
// Bound: HBM in the backward pass (read and write once) and, in bf16, the issue
// rate in the forward pass: 2 bytes per logit leave 11 instructions for each.
#include "qlora_device.cuh"
#include "qlora_internal.h"
#include "qlora_vec.cuh"

namespace qlora {

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLowest = -3.402823466e38f;
constexpr int kCap = 1024;        // entries of the candidate list
constexpr int kBatch = 4;         // windows per batch
constexpr int kGroups = 32;       // groups of threads that bound the top logits

__device__ const int64_t g_no_target = -1;   // read where no tokens are given

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// -infinity in every element of a packed vector
template <typename T>
__device__ __forceinline__ uint32_t minus_inf_word();
template <>
__device__ __forceinline__ uint32_t minus_inf_word<float>() { return 0xFF800000u; }
template <>
__device__ __forceinline__ uint32_t minus_inf_word<__nv_bfloat16>() { return 0xFF80FF80u; }

// A row of V logits seen through aligned 16-byte windows (qlora_vec.cuh);
// outside the row they read as -infinity.
template <typename T>
struct Row {
  static constexpr int N = Vec<T>::N;
  const T* p;
  int V, sh;
  __device__ __forceinline__ Row(const T* p_, int V_) : p(p_), V(V_) {
    sh = static_cast<int>((reinterpret_cast<uintptr_t>(p) & 15) / sizeof(T));
  }
  __device__ __forceinline__ int windows() const { return (V + sh + N - 1) / N; }
  __device__ __forceinline__ int col(int w) const { return w * N - sh; }
  __device__ __forceinline__ uint4 load(int w) const {
    const int c = col(w);
    if (c >= 0 && c + N <= V) return *reinterpret_cast<const uint4*>(p + c);
    const uint32_t f = minus_inf_word<T>();
    uint4 v = make_uint4(f, f, f, f);
    if (c < V && c > -N) {
      float x[N];
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float y = to_f32(p[min(max(c + i, 0), V - 1)]);
        x[i] = (c + i >= 0 && c + i < V) ? y : __uint_as_float(0xFF800000u);
      }
      v = Vec<T>::pack(x);
    }
    return v;
  }
};

__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// Largest logit of a batch (NaN does not count: the sums carry it)
template <typename T, int B>
__device__ __forceinline__ float batch_max(const uint4 (&v)[B]) {
  if constexpr (sizeof(T) == 2) {
    uint32_t m = max_bf16x2(max_bf16x2(v[0].x, v[0].y), max_bf16x2(v[0].z, v[0].w));
#pragma unroll
    for (int b = 1; b < B; ++b) m = max_bf16x2(m, max_bf16x2(max_bf16x2(v[b].x, v[b].y), max_bf16x2(v[b].z, v[b].w)));
    return fmaxf(bf16_lo(m), bf16_hi(m));
  } else {
    float m = __uint_as_float(v[0].x);
#pragma unroll
    for (int b = 0; b < B; ++b)
      m = fmaxf(fmaxf(fmaxf(m, __uint_as_float(v[b].x)), fmaxf(__uint_as_float(v[b].y), __uint_as_float(v[b].z))),
                __uint_as_float(v[b].w));
    return m;
  }
}

// m, S and G of some logits; m starts at the lowest finite value, so that
// differences from it stay defined for logits of -infinity.
struct Sums {
  float m, s, g;
  static __device__ __forceinline__ Sums none() { return {kLowest, 0.0f, 0.0f}; }
  // relative to a maximum M >= m
  __device__ __forceinline__ void rebase(float M, bool ent) {
    const float d = m - M, f = ex2(d * kLog2e);
    if (ent) g = f > 0.0f ? f * fmaf(s, d, g) : s * f;   // no 0 * infinity
    s *= f;
    m = M;
  }
};

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

__device__ __forceinline__ Sums warp_merge(Sums a, bool ent) {
  const float M = warp_max(a.m);
  a.rebase(M, ent);
  a.s = warp_sum(a.s);
  if (ent) a.g = warp_sum(a.g);
  return a;
}

// Logits in the order of their values as unsigned integers (-0 and 0 alike, NaN
// above all), and back.
__device__ __forceinline__ uint32_t key_of(float z) {
  if (z != z) return 0xFFFFFFFFu;
  const uint32_t u = __float_as_uint(z + 0.0f);
  return u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t k) {
  if (k == 0xFFFFFFFFu) return __uint_as_float(0x7FC00000u);
  return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

struct Entry {
  uint32_t key;
  int32_t idx;
};
__device__ __forceinline__ bool before(const Entry& a, const Entry& b) {
  return a.key > b.key || (a.key == b.key && a.idx < b.idx);
}

struct Shared {
  Sums part[32];
  uint32_t group[kGroups];
  Entry list[kCap];
  Entry best[kGroups];
  int count;
  uint32_t bound;
  // what the cluster's CTAs send to its first
  Sums all[8];
  Entry bests[8 * kGroups];
};

// Every logit of this thread's windows whose key is >= T (or > T) into the list.
template <typename T, int NT>
__device__ __forceinline__ void list_own(const Row<T>& row, int w0, int w1, uint32_t T_, bool strict, Shared& sm) {
  for (int w = w0 + threadIdx.x; w < w1; w += NT) {
    float x[Row<T>::N];
    Vec<T>::unpack(row.load(w), x);
#pragma unroll
    for (int i = 0; i < Row<T>::N; ++i) {
      const uint32_t k = key_of(x[i]);
      const int c = row.col(w) + i;
      if ((strict ? k > T_ : k >= T_) && c >= 0 && c < row.V) {
        const int at = atomicAdd(&sm.count, 1);
        if (at < kCap) sm.list[at] = {k, c};
      }
    }
  }
}

// The list's `n` entries in order into `best` (the first `top` of them).
template <int NT>
__device__ __forceinline__ void rank_list(int n, int top, const Entry* list, Entry* best) {
  for (int i = threadIdx.x; i < n; i += NT) {
    const Entry e = list[i];
    int r = 0;
    for (int j = 0; j < n && r < top; ++j) r += before(list[j], e);
    if (r < top) best[r] = e;
  }
}

// The top logits of a row with more than kCap that reach the bound: list those
// above it instead.  While these are too many as well, raise the bound to the
// top-th largest of those that fitted; then fill up with logits equal to the
// bound, in order of their index.
template <typename T, int NT>
__device__ __noinline__ void collect_many(const Row<T>& row, int w0, int w1, int top, uint32_t bound, float mine,
                                          Shared& sm) {
  int n;
  while (true) {
    __syncthreads();
    if (threadIdx.x == 0) sm.count = 0;
    __syncthreads();
    if (key_of(mine) >= bound) list_own<T, NT>(row, w0, w1, bound, true, sm);
    __syncthreads();
    n = sm.count;
    if (n <= kCap) break;
    rank_list<NT>(kCap, top, sm.list, sm.best);
    __syncthreads();
    bound = sm.best[top - 1].key;
  }
  rank_list<NT>(n, top, sm.list, sm.best);
  if (n >= top) return;
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    for (int w = w0; w < w1 && n < top; w += 32) {
      uint32_t hits = 0;
      if (w + lane < w1) {
        float x[Row<T>::N];
        Vec<T>::unpack(row.load(w + lane), x);
#pragma unroll
        for (int i = 0; i < Row<T>::N; ++i) {
          const int c = row.col(w + lane) + i;
          if (key_of(x[i]) == bound && c >= 0 && c < row.V) hits |= 1u << i;
        }
      }
      int sum = __popc(hits);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += y;
      }
      int at = n + sum - __popc(hits);
      for (uint32_t h = hits; h && at < top; h &= h - 1, ++at) sm.best[at] = {bound, row.col(w + lane) + __ffs(h) - 1};
      n += __shfl_sync(0xffffffffu, sum, 31);
    }
  }
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// a word into the cluster's first CTA's shared memory
__device__ __forceinline__ void st_first(void* p, uint32_t v) {
  uint32_t remote;
  asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(remote) : "r"(smem_u32(p)));
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(remote), "r"(v) : "memory");
}

template <typename T, int NT, bool ENT, bool TOP>
__global__ void __launch_bounds__(NT) k_logp_fwd(LogpArgs a) {
  constexpr int N = Vec<T>::N;
  __shared__ Shared sm;
  const int parts = a.split;
  const int part = parts > 1 ? static_cast<int>(cluster_rank()) : 0;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  griddep_launch_dependents();
  griddep_wait();
  if (parts > 1) cluster_sync();   // every CTA runs before one writes to another
  for (int64_t r = static_cast<int64_t>(blockIdx.x) / parts; r < a.N; r += gridDim.x / parts) {
    const Row<T> row(reinterpret_cast<const T*>(a.logits) + r * a.ld, a.V);
    const int nw = row.windows();
    const int per = (nw + parts - 1) / parts;
    const int w0 = part * per, w1 = min(nw, w0 + per);
    // the given token's logit, early
    float zt = 0.0f;
    bool counts = false;
    if (threadIdx.x == 0 && part == 0) {
      const int64_t* given = a.targets ? a.targets + r : &g_no_target;
      const int64_t t = *given;
      counts = t >= 0 && t < a.V;
      if (counts) zt = to_f32(row.p[t]);
    }
    if (TOP && threadIdx.x == 0) sm.count = 0;
    if (TOP && threadIdx.x < kGroups) sm.best[threadIdx.x] = {0u, 0};   // rows with NaN may not fill it

    Sums acc = Sums::none();
    f2 s2 = 0, g2 = 0;
    for (int w = w0 + threadIdx.x; w < w1; w += NT * kBatch) {
      uint4 v[kBatch];
      const uint32_t f = minus_inf_word<T>();
#pragma unroll
      for (int b = 0; b < kBatch; ++b) v[b] = w + b * NT < w1 ? row.load(w + b * NT) : make_uint4(f, f, f, f);
      const float top = batch_max<T>(v);
      if (top > acc.m) {
        acc.s = f2_sum(s2);
        if (ENT) acc.g = f2_sum(g2);
        acc.rebase(top, ENT);
        s2 = f2_make(acc.s, 0.0f);
        if (ENT) g2 = f2_make(acc.g, 0.0f);
      }
      const f2 minus = f2_dup(-acc.m), l2e = f2_dup(kLog2e);
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        f2 z[N / 2];
        unpack2(v[b], z, T());
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
          f2 d = f2_add(z[i], minus);
          float x0, x1;
          f2_get(f2_mul(d, l2e), x0, x1);
          const f2 e = f2_make(ex2(x0), ex2(x1));
          s2 = f2_add(s2, e);
          if (ENT) {
            f2_get(d, x0, x1);
            d = f2_make(fmaxf(x0, -1e4f), fmaxf(x1, -1e4f));   // 0 * -infinity counts as 0
            g2 = f2_fma(e, d, g2);
          }
        }
      }
    }
    acc.s = f2_sum(s2);
    if (ENT) acc.g = f2_sum(g2);
    const float mine = acc.m;   // no logit of this thread is larger

    if (TOP) {
      // the largest of this thread's group; a thread that saw nothing above the
      // lowest finite value may have seen nothing at all
      constexpr int PER = NT / kGroups;
      uint32_t k = mine > kLowest ? key_of(mine) : 0u;
#pragma unroll
      for (int o = PER / 2; o; o >>= 1) k = max(k, __shfl_xor_sync(0xffffffffu, k, o));
      if (threadIdx.x % PER == 0) sm.group[threadIdx.x / PER] = k;
    }
    acc = warp_merge(acc, ENT);
    if (lane == 0) sm.part[warp] = acc;
    __syncthreads();
    Sums all = Sums::none();
    if (lane < NT / 32) all = sm.part[lane];
    all = warp_merge(all, ENT);

    if (TOP) {
      const uint32_t g = sm.group[lane];
      int rank = 0;
#pragma unroll
      for (int j = 0; j < kGroups; ++j) {
        const uint32_t o = __shfl_sync(0xffffffffu, g, j);
        rank += o > g || (o == g && j < lane);
      }
      const uint32_t who = __ballot_sync(0xffffffffu, rank == a.top - 1);
      const uint32_t bound = __shfl_sync(0xffffffffu, g, __ffs(who) - 1);
      if (key_of(mine) >= bound) list_own<T, NT>(row, w0, w1, bound, false, sm);
      __syncthreads();
      const int n = sm.count;
      if (n <= kCap)
        rank_list<NT>(n, a.top, sm.list, sm.best);
      else
        collect_many<T, NT>(row, w0, w1, a.top, bound, mine, sm);
      __syncthreads();
    }

    if (parts > 1) {
      if (threadIdx.x == 0) {
        st_first(&sm.all[part].m, __float_as_uint(all.m));
        st_first(&sm.all[part].s, __float_as_uint(all.s));
        st_first(&sm.all[part].g, __float_as_uint(all.g));
      }
      if (TOP && threadIdx.x < a.top) {
        Entry* to = &sm.bests[part * a.top + threadIdx.x];
        st_first(&to->key, sm.best[threadIdx.x].key);
        st_first(&to->idx, static_cast<uint32_t>(sm.best[threadIdx.x].idx));
      }
      __syncwarp();
      cluster_sync();
      if (part == 0) {
        all = Sums::none();
        if (lane < parts) all = sm.all[lane];
        all = warp_merge(all, ENT);
        if (TOP) {
          rank_list<NT>(parts * a.top, a.top, sm.bests, sm.best);
          __syncthreads();
        }
      }
    }
    if (part == 0) {
      const bool empty = all.s == 0.0f;   // every logit is -infinity
      const float ls = logf(all.s), ninf = __uint_as_float(0xFF800000u);
      if (threadIdx.x == 0) {
        a.lse[r] = empty ? ninf : all.m + ls;
        if (a.targets) a.logp[r] = counts ? (empty ? ninf : (zt - all.m) - ls) : 0.0f;
        if (ENT) a.entropy[r] = empty ? 0.0f : ls - all.g / all.s;
      }
      if (TOP && threadIdx.x < a.top) {
        const Entry e = sm.best[threadIdx.x];
        a.top_ids[r * a.top + threadIdx.x] = e.idx;
        a.top_logp[r * a.top + threadIdx.x] = empty ? ninf : (value_of(e.key) - all.m) - ls;
      }
    }
    // the next row's results must not meet this row's readers
    if (parts > 1) {
      __syncwarp();
      cluster_sync();
    } else {
      __syncthreads();
    }
  }
}

// ---------------------------------------------------------------------------
// Backward: a CTA takes 256 x 4 windows of a row.
// ---------------------------------------------------------------------------
template <typename T, bool ENT>
__global__ void __launch_bounds__(256) k_logp_bwd(LogpArgs a, int tiles) {
  constexpr int N = Vec<T>::N;
  griddep_launch_dependents();
  griddep_wait();
  for (int64_t item = blockIdx.x; item < a.N * tiles; item += gridDim.x) {
    const int64_t r = item / tiles;
    const int w0 = static_cast<int>(item - r * tiles) * 256 * kBatch + threadIdx.x;
    const Row<T> row(reinterpret_cast<const T*>(a.logits) + r * a.ld, a.V);
    T* out = reinterpret_cast<T*>(a.dlogits) + r * a.ldd;
    uint4 v[kBatch];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) v[b] = row.load(w0 + b * 256);
    const float lse = a.lse_in[r];
    const int64_t t = a.targets[r];
    const bool counts = t >= 0 && t < a.V;
    const bool empty = lse == __uint_as_float(0xFF800000u);
    const float dl = counts && !empty ? a.dlogp[r] : 0.0f;
    float dh = 0.0f, base = dl;
    if (ENT) {
      dh = empty ? 0.0f : a.dentropy[r];
      base = fmaf(dh, a.entropy_in[r], dl);
    }
    const f2 minus = f2_dup(-lse), l2e = f2_dup(kLog2e), scale = f2_dup(-base), along = f2_dup(-dh);
    // the windows of the gradient's row are those of the logits' row when both
    // start at the same offset from a 16-byte boundary
    const bool same = (reinterpret_cast<uintptr_t>(out) & 15) / sizeof(T) == static_cast<uintptr_t>(row.sh);
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int col = row.col(w0 + b * 256);
      if (col >= a.cols) continue;
      f2 z[N / 2];
      unpack2(v[b], z, T());
      float o[N];
#pragma unroll
      for (int i = 0; i < N / 2; ++i) {
        const f2 d = f2_add(z[i], minus);
        float x0, x1;
        f2_get(f2_mul(d, l2e), x0, x1);
        const f2 p = f2_make(ex2(x0), ex2(x1));
        f2 f = scale;
        if (ENT) {
          f2_get(d, x0, x1);
          f = f2_fma(f2_make(fmaxf(x0, -1e4f), fmaxf(x1, -1e4f)), along, scale);
        }
        f2_get(f2_mul(p, f), o[2 * i], o[2 * i + 1]);
      }
      const int hit = static_cast<int>(t - col);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        if (counts && t >= col && hit == i) o[i] += dl;
        if (empty) o[i] = 0.0f;
      }
      if (col + N > a.V) {   // past the vocabulary: zero
#pragma unroll
        for (int i = 0; i < N; ++i)
          if (col + i >= a.V) o[i] = 0.0f;
      }
      if (same && col >= 0 && col + N <= a.cols) {
        *reinterpret_cast<uint4*>(out + col) = Vec<T>::pack(o);
      } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
          if (col + i >= 0 && col + i < a.cols) out[col + i] = from_f32<T>(o[i]);
      }
    }
  }
}

// CTAs of a cluster per row, so that few rows still fill the SMs, with at least
// 8192 logits for each CTA.
int split_of(int64_t N, int64_t V) {
  int s = 1;
  while (s < 8 && N * s * 2 <= num_sms() && V >= 8192 * 2 * s) s *= 2;
  return s;
}

template <typename T, int NT, bool ENT, bool TOP>
cudaError_t run_fwd(LogpArgs a, cudaStream_t st) {
  const int64_t rows = std::min<int64_t>(a.N, int64_t(1) << 27);
  ProfScope prof(QLORA_KC_AUX, st);
  const dim3 cluster(static_cast<unsigned>(a.split), 1, 1);
  return launch_pdl(k_logp_fwd<T, NT, ENT, TOP>, dim3(static_cast<unsigned>(rows * a.split)), dim3(NT), 0, st,
                    a.split > 1 ? &cluster : nullptr, a);
}

template <typename T, int NT>
cudaError_t pick_fwd(const LogpArgs& a, cudaStream_t st) {
  if (a.top) return a.entropy ? run_fwd<T, NT, true, true>(a, st) : run_fwd<T, NT, false, true>(a, st);
  return a.entropy ? run_fwd<T, NT, true, false>(a, st) : run_fwd<T, NT, false, false>(a, st);
}

template <typename T>
cudaError_t by_size(LogpArgs a, cudaStream_t st) {
  const int64_t windows = a.V / Vec<T>::N;
  a.split = split_of(a.N, a.V);
  if (windows > 2048 && a.N * a.split <= 2 * num_sms()) return pick_fwd<T, 1024>(a, st);
  if (windows > 2048) return pick_fwd<T, 512>(a, st);
  if (windows > 256) return pick_fwd<T, 256>(a, st);
  return pick_fwd<T, 128>(a, st);
}

template <typename T>
cudaError_t run_bwd(const LogpArgs& a, cudaStream_t st) {
  const int64_t windows = ceil_div(a.cols + Vec<T>::N - 1, Vec<T>::N);
  const int tiles = static_cast<int>(ceil_div(windows, 256 * kBatch));
  const unsigned grid = static_cast<unsigned>(std::min<int64_t>(a.N * tiles, int64_t(1) << 30));
  ProfScope prof(QLORA_KC_AUX, st);
  return a.dentropy ? launch_pdl(k_logp_bwd<T, true>, dim3(grid), dim3(256), 0, st, nullptr, a, tiles)
                    : launch_pdl(k_logp_bwd<T, false>, dim3(grid), dim3(256), 0, st, nullptr, a, tiles);
}

}  // namespace

cudaError_t launch_logp_fwd(const LogpArgs& a, cudaStream_t st) {
  return a.dtype == QLORA_DT_BF16 ? by_size<__nv_bfloat16>(a, st) : by_size<float>(a, st);
}

cudaError_t launch_logp_bwd(const LogpArgs& a, cudaStream_t st) {
  return a.dtype == QLORA_DT_BF16 ? run_bwd<__nv_bfloat16>(a, st) : run_bwd<float>(a, st);
}

}  // namespace qlora
