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
// maximum; the threads' triples are then merged.  (Folding the difference and the
// factor log2 e into one fused multiply-add saved no time and cost the exact 0 of
// a certain token's logp.)  Few rows are split over clusters of up to 8 CTAs,
// whose results meet in the first one's shared memory.
//
// Top alternatives without a second pass over memory: the threads' maxima give
// those of 32 groups of threads, and the top-th largest of these is a bound that
// at least `top` logits reach.  (Of random distinct ones about 32 (H(32) - H(32 -
// top)) do, H the harmonic numbers: drawing by size until `top` of 32 groups are hit;
// 31 for 20, 130 for 32.)
// Only threads whose own maximum reaches it have such logits: their windows are
// shared out over the CTA and loaded again (from L2), those that reach the bound
// are shared out by element, and a rank count orders the list, equal logits by
// their index.  Lists that overflow (rows with few distinct values, as under a
// mask) take `collect_many`.
//
// Bound: HBM in the backward pass (read and write once: 4096 x 32000 bf16 in 89 us,
// 92% of a copy's measured rate; fp32 99%) and in the fp32 forward (2048 x 32000 in
// 41 us, 99%).  In the bf16 forward (4096 x 32000 with the entropy: 51 us back to
// back, 80%; 54 with outputs allocated) 2 bytes per logit leave
// 11 issue slots for each, of which it takes 9, and the exponential's pipe is two
// thirds busy.  20 alternatives of each of 4096 rows take 30 us more; one row of
// 131072 takes 5.6 us, with 8 of them 8.8.
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
// outside the row they count as -infinity.
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

// m, S and G of some logits.  m starts at the lowest finite value, so that
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
  a.rebase(warp_max(a.m), ent);
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
constexpr uint32_t kInfKey = 0x007FFFFFu;   // of -infinity, the lowest
__device__ __forceinline__ float value_of(uint32_t k) {
  if (k == 0xFFFFFFFFu) return __uint_as_float(0x7FC00000u);
  return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

// A logit in the list of candidates: its key above the complement of its index,
// so that a larger entry comes first.
using Entry = uint64_t;
__device__ __forceinline__ Entry entry(uint32_t key, int idx) {
  return (static_cast<uint64_t>(key) << 32) | static_cast<uint32_t>(~idx);
}
__device__ __forceinline__ uint32_t entry_key(Entry e) { return static_cast<uint32_t>(e >> 32); }
__device__ __forceinline__ int entry_idx(Entry e) { return static_cast<int>(~static_cast<uint32_t>(e)); }

struct SharedTop {
  uint32_t group[kGroups];
  Entry list[kCap];
  Entry best[kGroups];
  Entry bests[8 * kGroups];   // what the cluster's CTAs send to its first
  int count;
  int threads, windows;       // entries of the two lists below
  uint16_t thread[1024];      // whose maximum reaches the bound
  int window[kCap];           // of theirs, that reach it
};
struct SharedSums {
  Sums part[2][32];
  Sums all[8];                // what the cluster's CTAs send to its first
};

// The logits of one window whose keys are >= least into the list.
template <typename T>
__device__ __noinline__ void list_window(uint4 v, int col, int V, uint32_t least, SharedTop* sm) {
  float z[Row<T>::N];
  Vec<T>::unpack(v, z);
#pragma unroll
  for (int i = 0; i < Row<T>::N; ++i) {
    const uint32_t k = key_of(z[i]);
    if (k >= least && col + i >= 0 && col + i < V) {
      const int at = atomicAdd(&sm->count, 1);
      if (at < kCap) sm->list[at] = entry(k, col + i);
    }
  }
}

// Every logit of this thread's windows whose key is >= bound (strict: > bound,
// which is never the largest key).  Eight windows are loaded at a time; most are
// dismissed by their largest logit.
template <typename T, int NT>
__device__ __forceinline__ void list_own(const Row<T>& row, int w0, int w1, uint32_t bound, bool strict, SharedTop& sm) {
  const uint32_t least = strict ? bound + 1 : bound;
  for (int w = w0 + threadIdx.x; w < w1; w += 8 * NT) {
    uint4 v[8];
    const uint32_t f = minus_inf_word<T>();
#pragma unroll
    for (int b = 0; b < 8; ++b) v[b] = w + b * NT < w1 ? row.load(w + b * NT) : make_uint4(f, f, f, f);
#pragma unroll
    for (int b = 0; b < 8; ++b) {
      const uint4 one[1] = {v[b]};
      if (w + b * NT < w1 && key_of(batch_max<T>(one)) >= least) list_window<T>(v[b], row.col(w + b * NT), row.V, least, &sm);
    }
  }
}

// The first `top` of the list's `n` entries, in order, into `best`.
template <int NT>
__device__ __forceinline__ void rank_list(int n, int top, const Entry* list, Entry* best) {
  for (int i = threadIdx.x; i < n; i += NT) {
    const Entry e = list[i];
    int r = 0;
#pragma unroll 8
    for (int j = 0; j < n; ++j) r += list[j] > e;
    if (r < top) best[r] = e;
  }
}

// The top logits of a row with more than kCap that reach the bound: list those
// above it instead.  While these are too many as well, raise the bound to the
// top-th largest of those that fitted; then fill up with logits equal to the
// bound, in order of their index.
template <typename T, int NT>
__device__ __noinline__ void collect_many(const Row<T>& row, int w0, int w1, int top, uint32_t bound, float mine,
                                          SharedTop& sm) {
  int n;
  while (true) {
    __syncthreads();
    if (threadIdx.x == 0) sm.count = 0;
    __syncthreads();
    if (bound != 0xFFFFFFFFu && key_of(mine) >= bound) list_own<T, NT>(row, w0, w1, bound, true, sm);
    __syncthreads();
    n = sm.count;
    if (n <= kCap) break;
    rank_list<NT>(kCap, top, sm.list, sm.best);
    __syncthreads();
    bound = entry_key(sm.best[top - 1]);
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
      for (uint32_t h = hits; h && at < top; h &= h - 1, ++at) sm.best[at] = entry(bound, row.col(w + lane) + __ffs(h) - 1);
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

constexpr int logp_ctas(int nt) { return nt >= 1024 ? 1 : nt == 32 ? 16 : 1024 / nt; }   // CTAs per SM, by registers
constexpr int kStages = 2;       // batches that a thread's loads run ahead (three leave too little L1: 2 to 13% slower)

// CTAs walk over rows gridDim apart; `split` CTAs of a cluster share a row.  The
// loads run ahead, from one row into the next, through a ring in shared memory
// (cp.async) in which each thread reads back only what it copied itself: so the
// end of a row, its merges and its top list, passes while the next row arrives.
template <typename T, int NT, bool ENT, bool TOP>
__global__ void __launch_bounds__(NT, logp_ctas(NT)) k_logp_fwd(LogpArgs a) {
  constexpr int N = Vec<T>::N;
  constexpr uint32_t kStage = kBatch * NT * 16;
  extern __shared__ __align__(16) uint8_t smem[];
  SharedSums& sums = *reinterpret_cast<SharedSums*>(smem + kStages * kStage);
  SharedTop& tops = *reinterpret_cast<SharedTop*>(smem + kStages * kStage + sizeof(SharedSums));   // only with TOP
  const int parts = a.split;
  const int part = parts > 1 ? static_cast<int>(cluster_rank()) : 0;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t first = blockIdx.x >> a.split_log2, stride = gridDim.x >> a.split_log2;
  const uint32_t slot = smem_u32(smem) + threadIdx.x * 16u;
  const uint32_t ninf = minus_inf_word<T>();
  griddep_launch_dependents();
  griddep_wait();
  if (parts > 1) cluster_sync();   // every CTA runs before one writes to another

  auto row_at = [&](int64_t r) { return Row<T>(reinterpret_cast<const T*>(a.logits) + r * a.ld, a.V); };
  auto windows_of = [&](const Row<T>& row, int& w0, int& w1) {
    const int nw = row.windows(), per = (nw + parts - 1) >> a.split_log2;
    w0 = part * per;
    w1 = min(nw, w0 + per);
  };
  auto has_edges = [&](const Row<T>& row) { return row.sh != 0 || (row.V + row.sh) % N != 0; };
  // what is copied next: batch `bw` (its first window) of row `br`
  int64_t br = first;
  Row<T> brow = row_at(br < a.N ? br : 0);
  int bw, bw1;
  windows_of(brow, bw, bw1);
  bool bedges = has_edges(brow);
  auto issue = [&](uint32_t stage) {
    if (br < a.N) {
      const T* src = brow.p + brow.col(bw + threadIdx.x);
      if (!bedges && bw + kBatch * NT <= bw1) {
#pragma unroll
        for (int b = 0; b < kBatch; ++b) cp_async16(slot + stage + b * NT * 16, src + b * NT * N, 16);
      } else {
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
          const int w = bw + b * NT + threadIdx.x;
          const uint32_t dst = slot + stage + b * NT * 16;
          if (w < bw1) {
            // a window that starts ahead of the row reads what lies there too
            cp_async16(dst, src + b * NT * N, min(a.V - brow.col(w), N) * static_cast<int>(sizeof(T)));
          } else {
            sts128(dst, make_uint4(ninf, ninf, ninf, ninf));
          }
        }
      }
      bw += kBatch * NT;
      if (bw >= bw1) {
        br += stride;
        brow = row_at(br < a.N ? br : 0);
        windows_of(brow, bw, bw1);
        bedges = has_edges(brow);
      }
    }
    cp_async_commit();
  };
  for (int k = 0; k < kStages; ++k) issue(k * kStage);

  uint32_t stage = 0;
  int buf = 0;
  for (int64_t r = first; r < a.N; r += stride, buf ^= 1) {
    const Row<T> row = row_at(r);
    int w0, w1;
    windows_of(row, w0, w1);
    const bool edges = has_edges(row);
    // the given token's logit, early
    float zt = 0.0f;
    bool counts = false;
    if (threadIdx.x == 0 && part == 0) {
      const int64_t* given = a.targets ? a.targets + r : &g_no_target;
      const int64_t t = *given;
      counts = t >= 0 && t < a.V;
      if (counts) zt = to_f32(row.p[t]);
    }
    if (TOP && threadIdx.x == 0) tops.count = tops.threads = tops.windows = 0;
    if (TOP && threadIdx.x < kGroups) tops.best[threadIdx.x] = entry(0u, 0);   // rows with NaN may not fill it

    Sums acc = Sums::none();
    f2 s2 = 0, g2 = 0;
    for (int w = w0; w < w1; w += NT * kBatch) {
      uint4 v[kBatch];
      cp_async_wait(kStages - 1);
#pragma unroll
      for (int b = 0; b < kBatch; ++b) v[b] = lds128(slot + stage + b * NT * 16);
      if (edges) {
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
          const int c = row.col(w + b * NT + threadIdx.x);
          if (c < 0 || (c < row.V && c + N > row.V)) {   // values outside the row
            float x[N];
            Vec<T>::unpack(v[b], x);
#pragma unroll
            for (int i = 0; i < N; ++i)
              if (c + i < 0 || c + i >= row.V) x[i] = __uint_as_float(0xFF800000u);
            v[b] = Vec<T>::pack(x);
          }
        }
      }
      issue(stage);
      stage = stage == (kStages - 1) * kStage ? 0 : stage + kStage;
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
      // the largest of this thread's group; -infinity for a thread that saw nothing
      // else or nothing at all (then m is where it started and S is 0)
      constexpr int PER = NT / kGroups;
      uint32_t k = mine > kLowest || acc.s > 0.0f ? key_of(mine) : kInfKey;
#pragma unroll
      for (int o = PER / 2; o; o >>= 1) k = max(k, __shfl_xor_sync(0xffffffffu, k, o));
      if (threadIdx.x % PER == 0) tops.group[threadIdx.x / PER] = k;
    }
    Sums all = warp_merge(acc, ENT);
    if (NT > 32) {
      // two scratches in turn: the next row's partial results cannot meet this row's readers
      if (lane == 0) sums.part[buf][warp] = all;
      __syncthreads();
      if (TOP || parts > 1 || warp == 0) {
        all = Sums::none();
        if (lane < NT / 32) all = sums.part[buf][lane];
        all = warp_merge(all, ENT);
      }
    } else {
      __syncwarp();
    }

    if (TOP) {
      const uint32_t g = tops.group[lane];
      int rank = 0;
#pragma unroll
      for (int j = 0; j < kGroups; ++j) {
        const uint32_t o = __shfl_sync(0xffffffffu, g, j);
        rank += o > g || (o == g && j < lane);
      }
      const uint32_t who = __ballot_sync(0xffffffffu, rank == a.top - 1);
      const uint32_t bound = __shfl_sync(0xffffffffu, g, __ffs(who) - 1);
      if (key_of(mine) >= bound) tops.thread[atomicAdd(&tops.threads, 1)] = static_cast<uint16_t>(threadIdx.x);
      __syncthreads();
      // every thread reaches a bound that separates nothing, as under a mask: the
      // list would overflow (one row of 131072, half masked: 51 us, else 14;
      // 1024 x 32000 with 5 logits left: 420 us, else 52)
      const int found = tops.threads;
      const bool even = NT > kGroups && found == NT && (w1 - w0) * N > kCap;
      // their windows, one per thread
      const int rounds = (w1 - w0 + NT - 1) / NT, todo = even ? 0 : found * rounds;
      for (int k = threadIdx.x; k < todo; k += NT) {
        const int w = w0 + tops.thread[k / rounds] + k % rounds * NT;
        if (w >= w1) continue;
        const uint4 one[1] = {row.load(w)};
        if (key_of(batch_max<T>(one)) >= bound) {
          const int at = atomicAdd(&tops.windows, 1);
          if (at < kCap) tops.window[at] = w;
        }
      }
      __syncthreads();
      // the elements of those that reach the bound, one per thread
      const int hits = tops.windows;
      for (int k = threadIdx.x; k < min(hits, kCap) * N; k += NT) {
        const int c = row.col(tops.window[k / N]) + k % N;
        if (c < 0 || c >= row.V) continue;
        const uint32_t key = key_of(to_f32(row.p[c]));
        if (key >= bound) {
          const int at = atomicAdd(&tops.count, 1);
          if (at < kCap) tops.list[at] = entry(key, c);
        }
      }
      __syncthreads();
      const int n = !even && hits <= kCap ? tops.count : kCap + 1;
      if (n <= kCap)
        rank_list<NT>(n, a.top, tops.list, tops.best);
      else
        collect_many<T, NT>(row, w0, w1, a.top, bound, mine, tops);
      __syncthreads();
    }

    if (parts > 1) {
      if (threadIdx.x == 0) {
        st_first(&sums.all[part].m, __float_as_uint(all.m));
        st_first(&sums.all[part].s, __float_as_uint(all.s));
        st_first(&sums.all[part].g, __float_as_uint(all.g));
      }
      if (TOP && threadIdx.x < a.top) {
        const Entry e = tops.best[threadIdx.x];
        uint32_t* to = reinterpret_cast<uint32_t*>(&tops.bests[part * a.top + threadIdx.x]);
        st_first(to, static_cast<uint32_t>(e));
        st_first(to + 1, static_cast<uint32_t>(e >> 32));
      }
      __syncwarp();
      cluster_sync();
      if (part == 0) {
        all = Sums::none();
        if (lane < parts) all = sums.all[lane];
        all = warp_merge(all, ENT);
        if (TOP) {
          rank_list<NT>(parts * a.top, a.top, tops.bests, tops.best);
          __syncthreads();
        }
      }
    }
    if (part == 0 && warp == 0) {
      const bool empty = all.s == 0.0f;   // every logit is -infinity
      const float ls = logf(all.s), none = __uint_as_float(0xFF800000u);
      if (lane == 0) {
        a.lse[r] = empty ? none : all.m + ls;
        if (a.targets) a.logp[r] = counts ? (empty ? none : (zt - all.m) - ls) : 0.0f;
        if (ENT) a.entropy[r] = empty ? 0.0f : ls - all.g / all.s;
      }
      if (TOP && lane < a.top) {
        const Entry e = tops.best[lane];
        a.top_ids[r * a.top + lane] = entry_idx(e);
        a.top_logp[r * a.top + lane] = empty ? none : (value_of(entry_key(e)) - all.m) - ls;
      }
    }
    // the next row's results must not meet this row's readers
    if (parts > 1) {
      __syncwarp();
      cluster_sync();
    } else if (TOP) {
      __syncthreads();
    }
  }
  cp_async_wait(0);
}

// ---------------------------------------------------------------------------
// Backward: 256 threads (or a warp) take 4 windows each of a row at a time.
// ---------------------------------------------------------------------------
// lse in fp32 is off by up to 2^-24 |lse|, and p by that as a factor.  Beyond this
// size (2^-16) the row is measured again, where probabilities would be wrong
// altogether if a mask of -1e9 or of the type's lowest value left nothing else.
constexpr float kExactLse = 256.0f;

// What a row's gradient takes: p = exp(z - m) / S, log p = z - m - ls.
struct RowGrad {
  float m, ls, inv_s;   // m and ls: lse and 0, or the largest logit and log S
  float dl, dh, h;      // gradients of logp and entropy, the entropy
  int64_t t;            // the given token, -1 where it does not count
};

template <bool ENT>
__device__ __forceinline__ RowGrad row_grad(const LogpArgs& a, int64_t r) {
  RowGrad g = {a.lse_in[r], 0.0f, 1.0f, a.dlogp[r], ENT ? a.dentropy[r] : 0.0f, ENT ? a.entropy_in[r] : 0.0f,
               a.targets[r]};
  if (g.t < 0 || g.t >= a.V) {
    g.t = -64;   // in no window, the row's first included
    g.dl = 0.0f;
  }
  // a row of -infinity only: measured from 0, its probabilities come out as 0
  if (g.m == __uint_as_float(0xFF800000u)) g.m = g.dl = g.dh = 0.0f;
  return g;
}

// Gradient of one window (what load() gave for its columns col ..) into `out`;
// `same`: the window is a 16-byte one of the gradient's row as well.
template <typename T, bool ENT>
__device__ __forceinline__ void grad_window(const RowGrad& g, const uint4& v, int col, int V, int cols, bool same, T* out) {
  constexpr int N = Vec<T>::N;
  const float unit = -g.inv_s;
  const f2 minus = f2_dup(-g.m), l2e = f2_dup(kLog2e), along = f2_dup(g.dh * unit),
           scale = f2_dup((ENT ? fmaf(g.dh, g.h - g.ls, g.dl) : g.dl) * unit);
  f2 z[N / 2], o[N / 2];
  unpack2(v, z, T());
#pragma unroll
  for (int i = 0; i < N / 2; ++i) {
    f2 d = f2_add(z[i], minus);
    float x0, x1;
    f2_get(f2_mul(d, l2e), x0, x1);
    const f2 p = f2_make(ex2(x0), ex2(x1));
    if (ENT) {
      f2_get(d, x0, x1);
      d = f2_make(fmaxf(x0, -1e4f), fmaxf(x1, -1e4f));   // 0 * -infinity counts as 0
    }
    o[i] = f2_mul(p, ENT ? f2_fma(d, along, scale) : scale);
  }
  if (g.t >= col && g.t < col + N) {
    const int hit = static_cast<int>(g.t - col);
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      float x0, x1;
      f2_get(o[i], x0, x1);
      o[i] = f2_make(hit == 2 * i ? x0 + g.dl : x0, hit == 2 * i + 1 ? x1 + g.dl : x1);
    }
  }
  if (same && col >= 0 && col + N <= V) {
    *reinterpret_cast<uint4*>(out + col) = pack2(o, T());
  } else {   // zeros past the vocabulary
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float x0, x1;
      f2_get(o[i / 2], x0, x1);
      const float x = col + i < V ? (i & 1 ? x1 : x0) : 0.0f;
      if (col + i >= 0 && col + i < cols) out[col + i] = from_f32<T>(x);
    }
  }
}

// A whole row by its threads (all of the CTA or one warp), measured before any
// of it is written (the gradient may be in place).
template <typename T, bool ENT, int TPR>
__device__ __forceinline__ void grad_large(const Row<T>& row, RowGrad g, int nw, int cols, bool same, T* out) {
  __shared__ float part[8];
  const int tid = threadIdx.x % TPR, own = row.windows();
  float m = kLowest, s = 0.0f;
#pragma unroll 1
  for (int w = tid; w < own; w += TPR) {
    const uint4 one[1] = {row.load(w)};
    m = fmaxf(m, batch_max<T>(one));
  }
  m = warp_max(m);
  if (TPR > 32) {
    __syncthreads();
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, part[i]);
  }
#pragma unroll 1
  for (int w = tid; w < own; w += TPR) {
    float z[Row<T>::N];
    Vec<T>::unpack(row.load(w), z);
#pragma unroll
    for (int i = 0; i < Row<T>::N; ++i) s += ex2((z[i] - m) * kLog2e);
  }
  s = warp_sum(s);
  if (TPR > 32) {
    __syncthreads();
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = s;
    __syncthreads();
    s = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) s += part[i];
  } else {
    __syncwarp();
  }
  g.m = m;
  g.ls = logf(s);
  g.inv_s = 1.0f / s;
#pragma unroll 1
  for (int w = tid; w < nw; w += TPR) grad_window<T, ENT>(g, row.load(w), row.col(w), row.V, cols, same, out);
}

// TPR threads to a row: 256, or 32 for short rows.
template <typename T, bool ENT, int TPR>
__global__ void __launch_bounds__(256, 5) k_logp_bwd(LogpArgs a) {
  constexpr int N = Vec<T>::N, ROWS = 256 / TPR;
  griddep_launch_dependents();
  griddep_wait();
  for (int64_t r = static_cast<int64_t>(blockIdx.x) * ROWS + threadIdx.x / TPR; r < a.N;
       r += static_cast<int64_t>(gridDim.x) * ROWS) {
    const Row<T> row(reinterpret_cast<const T*>(a.logits) + r * a.ld, a.V);
    T* out = reinterpret_cast<T*>(a.dlogits) + r * a.ldd;
    // the windows of the gradient's row are those of the logits' row when both
    // start at the same offset from a 16-byte boundary
    const bool same = (reinterpret_cast<uintptr_t>(out) & 15) / sizeof(T) == static_cast<uintptr_t>(row.sh);
    const int nw = (a.cols + row.sh + N - 1) / N;
    bool large = false;
    for (int w0 = blockIdx.y * TPR * kBatch + threadIdx.x % TPR; w0 < nw; w0 += gridDim.y * TPR * kBatch) {
      uint4 v[kBatch];
#pragma unroll
      for (int b = 0; b < kBatch; ++b) v[b] = row.load(w0 + b * TPR);
      const RowGrad g = row_grad<ENT>(a, r);
      large = fabsf(g.m) > kExactLse;
      if (large) break;
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const int col = row.col(w0 + b * TPR);
        if (col < a.cols) grad_window<T, ENT>(g, v[b], col, a.V, a.cols, same, out);
      }
    }
    // the first CTA of a row takes it all when it is measured again
    const bool again = TPR > 32 ? __syncthreads_or(large) : __any_sync(0xFFFFFFFFu, large);
    if (blockIdx.y == 0 && again) grad_large<T, ENT, TPR>(row, row_grad<ENT>(a, r), nw, a.cols, same, out);
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
  constexpr uint32_t smem = kStages * kBatch * NT * 16 + sizeof(SharedSums) + (TOP ? sizeof(SharedTop) : 0);
  // what fits on an SM: with alternatives shared memory allows 6 CTAs of 128 threads
  // and 10 of a warp (a grid of 8 and 16 left a quarter of the CTAs their whole share
  // for a second wave)
  constexpr int64_t per_sm = std::min<int64_t>(logp_ctas(NT), 228 * 1024 / (smem + 1024));
  // two waves of CTAs where each still gets several rows: SMs differ in the
  // bandwidth they get, and the ones that are ahead take more of the second
  const int64_t fit = std::max<int64_t>(1, static_cast<int64_t>(num_sms()) * per_sm / a.split);
  const int64_t rows = std::min<int64_t>(a.N, a.N >= 6 * fit ? 2 * fit : fit);
  auto kernel = k_logp_fwd<T, NT, ENT, TOP>;
  const cudaError_t e = set_smem(kernel, smem);
  if (e != cudaSuccess) return e;
  ProfScope prof(QLORA_KC_AUX, st);
  const dim3 cluster(static_cast<unsigned>(a.split), 1, 1);
  return launch_pdl(kernel, dim3(static_cast<unsigned>(rows * a.split)), dim3(NT), smem, st,
                    a.split > 1 ? &cluster : nullptr, a);
}

template <typename T, int NT>
cudaError_t pick_fwd(const LogpArgs& a, cudaStream_t st) {
  if (a.top) return a.entropy ? run_fwd<T, NT, true, true>(a, st) : run_fwd<T, NT, false, true>(a, st);
  return a.entropy ? run_fwd<T, NT, true, false>(a, st) : run_fwd<T, NT, false, false>(a, st);
}

// Threads per row: one batch of windows each for short rows; for long ones 256
// where that gives every CTA several rows (4096 x 32000 bf16: 52 us, 63 us with
// 512), 512 where it does not (1024 x 131072 bf16: 53 us, 48 us with 512), and
// 1024 where there are fewer rows than SMs.
template <typename T>
cudaError_t by_size(LogpArgs a, cudaStream_t st) {
  const int64_t windows = a.V / Vec<T>::N;
  a.split = split_of(a.N, a.V);
  for (a.split_log2 = 0; (1 << a.split_log2) < a.split;) ++a.split_log2;
  if (windows > 1024 && a.N * a.split <= num_sms()) return pick_fwd<T, 1024>(a, st);
  if (windows > 1024 && a.N < 6 * num_sms() * logp_ctas(256)) return pick_fwd<T, 512>(a, st);
  if (windows > 1024) return pick_fwd<T, 256>(a, st);
  if (windows > 32 * kBatch) return pick_fwd<T, 128>(a, st);
  return pick_fwd<T, 32>(a, st);
}

template <typename T>
cudaError_t run_bwd(const LogpArgs& a, cudaStream_t st) {
  const int64_t windows = ceil_div(a.cols + Vec<T>::N - 1, Vec<T>::N);
  ProfScope prof(QLORA_KC_AUX, st);
  if (windows <= 1024 && a.N >= 8 * num_sms()) {
    const dim3 grid(static_cast<unsigned>(std::min<int64_t>(ceil_div(a.N, 8), INT32_MAX)));
    return a.dentropy ? launch_pdl(k_logp_bwd<T, true, 32>, grid, dim3(256), 0, st, nullptr, a)
                      : launch_pdl(k_logp_bwd<T, false, 32>, grid, dim3(256), 0, st, nullptr, a);
  }
  const dim3 grid(static_cast<unsigned>(std::min<int64_t>(a.N, INT32_MAX)),
                  static_cast<unsigned>(std::min<int64_t>(ceil_div(windows, 256 * kBatch), 65535)));
  return a.dentropy ? launch_pdl(k_logp_bwd<T, true, 256>, grid, dim3(256), 0, st, nullptr, a)
                    : launch_pdl(k_logp_bwd<T, false, 256>, grid, dim3(256), 0, st, nullptr, a);
}

}  // namespace

cudaError_t launch_logp_fwd(const LogpArgs& a, cudaStream_t st) {
  return a.dtype == QLORA_DT_BF16 ? by_size<__nv_bfloat16>(a, st) : by_size<float>(a, st);
}

cudaError_t launch_logp_bwd(const LogpArgs& a, cudaStream_t st) {
  return a.dtype == QLORA_DT_BF16 ? run_bwd<__nv_bfloat16>(a, st) : run_bwd<float>(a, st);
}

}  // namespace qlora
