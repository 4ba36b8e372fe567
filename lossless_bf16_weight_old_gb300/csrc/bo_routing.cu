// bo_routing.cu -- the experts of each token of a mixture, their weights, per-expert counts and the
// balance loss, and the gradient of the router's logits (include/ops/bf16ops.h has the formulas).
//
// Selection orders whole numbers that no two experts share (keys), so it needs no rule for equal logits.
// A token's logits are a few hundred bytes: few tokens are bounded by latency, many by the selection's
// arithmetic, and only the gradient of many by HBM.
#include <cooperative_groups.h>

#include "bo_internal.cuh"

namespace bo {
namespace {

namespace cg = cooperative_groups;


constexpr uint32_t kThreads = 256, kWarps = kThreads / 32;
constexpr uint32_t kMaxCluster = 8;
constexpr uint32_t kMaxBlocks = 640;     // of the forward pass (its partial sums)
constexpr uint32_t kJoinThreads = 1024;   // (at least the experts)
constexpr uint32_t kLane = 16;           // experts that a lane holds
constexpr uint32_t kAll = 0xffffffffu;
constexpr float kLog2e = 1.44269504088896340736f;

struct RouteArgs {
  const uint8_t* x;
  uint64_t ld;            // bytes
  const uint8_t* mask;    // may be NULL
  uint64_t mask_stride;
  uint32_t tokens, experts, k, normalize;
  uint32_t lanes;         // that share a token (a power of two)
  uint32_t rounds;        // of a warp's tokens: a power of two, at most `lanes`
  uint32_t vec;           // their parts of a row are whole, aligned words of 32 bytes
  uint32_t joined;        // the grid is one cluster, which writes the results itself
  float* weights;
  int32_t* chosen;
  float* sums;            // of p: one row of `experts` for each block
  int32_t* counts;        // likewise
  int32_t* real;          // one for each block
  float* out_probs;
  int32_t* out_counts;
  float* out_loss;
  int32_t* out_real;
};
struct RouteGradArgs {
  const uint8_t* x;
  uint64_t ld;            // bytes
  uint8_t* dx;
  uint64_t ld_dx;         // bytes
  const float* gw;        // may be NULL
  uint64_t gw_stride, gw_choice;
  const float* gloss;     // may be NULL
  float loss;
  uint32_t tokens, experts, k, normalize;
  uint32_t lanes, vec, vec_dx;
  const int32_t* chosen;
  const int32_t* counts;
  const int32_t* real;
};

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float rcp(float x) {   // off by one step at most
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ void ld32(uint32_t* w, const void* p) {
  asm volatile("ld.global.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]),
                 "=r"(w[7])
               : "l"(p)
               : "memory");
}
__device__ __forceinline__ void st32(void* p, const uint32_t* w) {
  asm volatile("st.global.L1::no_allocate.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(w[0]),
               "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(kAll, v, d);
  return v;
}
// Among the lanes that share a token, at most 2^STEPS; steps past them go to the lane itself, without
// a branch.
template <int STEPS>
struct Lanes {
  uint32_t with[STEPS];
  float count[STEPS];
  __device__ __forceinline__ explicit Lanes(uint32_t lanes) {
#pragma unroll
    for (int i = 0; i < STEPS; i++) {
      with[i] = 1u << i < lanes ? 1u << i : 0;
      count[i] = with[i] ? 1.f : 0.f;
    }
  }
  __device__ __forceinline__ float sum(float v) const {
#pragma unroll
    for (int i = 0; i < STEPS; i++) v = fmaf(__shfl_xor_sync(kAll, v, with[i]), count[i], v);
    return v;
  }
  __device__ __forceinline__ float max(float v) const {
#pragma unroll
    for (int i = 0; i < STEPS; i++) v = max_nan(v, __shfl_xor_sync(kAll, v, with[i]));
    return v;
  }
};
template <bool F32>
__device__ __forceinline__ float element(const uint8_t* row, uint32_t e) {
  return F32 ? reinterpret_cast<const float*>(row)[e]
             : __uint_as_float((uint32_t) reinterpret_cast<const uint16_t*>(row)[e] << 16);
}

// N experts' logits from expert e0 on, as they lie in memory; -infinity past the last expert.
template <bool F32, int N>
struct Logits {
  static constexpr int kWords = F32 ? N : N / 2;
  uint32_t w[kWords];

  __device__ __forceinline__ void load(const uint8_t* row, uint32_t e0, uint32_t experts, bool vec) {
    if (vec && e0 < experts) {
#pragma unroll
      for (int i = 0; i < kWords; i += 8) ld32(w + i, row + (uint64_t)e0 * (F32 ? 4 : 2) + i * 4);
      return;
    }
#pragma unroll
    for (int i = 0; i < kWords; i++) {
      if (F32) {
        w[i] = e0 + i < experts ? reinterpret_cast<const uint32_t*>(row)[e0 + i] : 0xFF800000u;
      } else {
        const uint16_t* p = reinterpret_cast<const uint16_t*>(row);
        const uint32_t e = e0 + 2 * i;
        w[i] = e < experts ? p[e] : 0xFF80u;
        w[i] |= (e + 1 < experts ? (uint32_t)p[e + 1] : 0xFF80u) << 16;
      }
    }
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < kWords; i++) w[i] = 0;
  }
  __device__ __forceinline__ float2 pair(int i) const {   // elements 2 i and 2 i + 1
    return F32 ? make_float2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]))
               : make_float2(bf16_lo(w[i]), bf16_hi(w[i]));
  }
  __device__ __forceinline__ float max() const {
    if (F32) {
      float m = __uint_as_float(w[0]);
#pragma unroll
      for (int i = 1; i < kWords; i++) m = max_nan(m, __uint_as_float(w[i]));
      return m;
    }
    uint32_t m = w[0];
#pragma unroll
    for (int i = 1; i < kWords; i++) m = max_bf16x2(m, w[i]);
    return max_nan(bf16_lo(m), bf16_hi(m));
  }
};

// ------------------------------------------------------------------------------------- keys
// A whole number that orders logits, and equal ones by their expert, the lowest first: the bits of
// the logit as a signed number orders them, above the expert's complement.  NaN is above all others
// and -0 is 0.  32 bits hold a BF16 logit and its expert, 64 an FP32 one.
template <bool F32>
struct Keys;
template <>
struct Keys<false> {
  typedef int32_t T;
  static constexpr T kNone = INT32_MIN;
  static __device__ __forceinline__ T make(float x, uint32_t e) {
    const int32_t s = x != x ? 0x7FFF0000 : __float_as_int(x + 0.f);
    return (s ^ ((s >> 31) & 0x7FFF0000)) | (int32_t)(0xFFFFu - e);
  }
  static __device__ __forceinline__ float value(T k) {
    const int32_t s = k & (int32_t)0xFFFF0000;
    return __int_as_float(s ^ ((s >> 31) & 0x7FFF0000));
  }
  static __device__ __forceinline__ uint32_t expert(T k) { return 0xFFFFu - (uint32_t)(k & 0xFFFF); }
  static __device__ __forceinline__ T warp_max(T k) { return __reduce_max_sync(kAll, k); }
};
template <>
struct Keys<true> {
  typedef long long T;
  static constexpr T kNone = INT64_MIN;
  static __device__ __forceinline__ T make(float x, uint32_t e) {
    const int32_t s = x != x ? 0x7FFFFFFF : __float_as_int(x + 0.f);
    return (T)((unsigned long long)(uint32_t)(s ^ ((s >> 31) & 0x7FFFFFFF)) << 32 | (uint32_t)~e);
  }
  static __device__ __forceinline__ float value(T k) {
    const int32_t s = (int32_t)(k >> 32);
    return __int_as_float(s ^ ((s >> 31) & 0x7FFFFFFF));
  }
  static __device__ __forceinline__ uint32_t expert(T k) { return ~(uint32_t)k; }
  static __device__ __forceinline__ T warp_max(T k) {
    const int32_t hi = __reduce_max_sync(kAll, (int32_t)(k >> 32));
    const uint32_t lo = __reduce_max_sync(kAll, (int32_t)(k >> 32) == hi ? (uint32_t)k : 0u);
    return (T)((unsigned long long)(uint32_t)hi << 32 | lo);
  }
};
// The warp's k greatest of NV keys a lane; lane i gets the i-th.  first: the greatest.
template <bool F32, int NV>
__device__ __forceinline__ typename Keys<F32>::T choose(typename Keys<F32>::T (&key)[NV],
                                                        typename Keys<F32>::T first, uint32_t k, uint32_t lane) {
  typename Keys<F32>::T best = first, mine = 0;
  for (uint32_t i = 0;;) {
    if (lane == i) mine = best;
    if (++i == k) return mine;
    typename Keys<F32>::T next = Keys<F32>::kNone;
#pragma unroll
    for (int j = 0; j < NV; j++) {
      if (key[j] == best) key[j] = Keys<F32>::kNone;
      next = ::max(key[j], next);
    }
    best = Keys<F32>::warp_max(next);
  }
}

// k_route_many's keys: 32 bits in which the expert (at most 256) takes the lowest 8.  Of an FP32 logit
// the lowest 8 bits have to go: keys that differ there alone say nothing about the order.
template <bool F32>
struct Short {
  static constexpr uint32_t kExpertBits = 0xFFu;
  // of a lane's logits, from expert e0 on.  (What stands in place of experts past the last one,
  // -infinity, is below every expert's key, and k are chosen of at least as many.)
  static __device__ __forceinline__ void make(const Logits<F32, kLane>& x, int32_t* k) {
    if (F32) {
#pragma unroll
      for (int i = 0; i < (int)kLane; i++) {
        const int32_t s = __float_as_int(__fadd_rn(__uint_as_float(x.w[i]), 0.f));   // one zero, one NaN
        k[i] = ((s ^ ((s >> 31) & 0x7FFFFFFF)) & ~0xFF) | (15 - i);
      }
    } else {
#pragma unroll
      for (int i = 0; i < (int)kLane / 2; i++) {
        uint32_t v, sign;
        asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(v) : "r"(x.w[i]), "r"(0u));   // one zero, one NaN
        asm("prmt.b32 %0, %1, %1, 0xBB99;" : "=r"(sign) : "r"(v));          // all ones where negative
        v ^= sign & 0x7FFF7FFFu;
        k[2 * i] = (int32_t)__byte_perm(v, 15 - 2 * i, 0x1054);
        k[2 * i + 1] = (int32_t)__byte_perm(v, 14 - 2 * i, 0x3254);
      }
    }
  }
  // what is to be added to a lane's keys for its first expert e0
  static __device__ __forceinline__ int32_t base(uint32_t e0) { return (int32_t)(240 - e0); }
  static __device__ __forceinline__ uint32_t expert(int32_t k) { return 255 - ((uint32_t)k & 0xFF); }
  static __device__ __forceinline__ float value(int32_t k) { return Keys<false>::value(k); }   // BF16 alone
};

// Sorting networks, greatest first.
template <class T>
__device__ __forceinline__ void order(T& a, T& b) {
  const T hi = ::max(a, b), lo = ::min(a, b);
  a = hi;
  b = lo;
}
template <class T>
__device__ __forceinline__ void sort4(T* k) {
  order(k[0], k[1]), order(k[2], k[3]), order(k[0], k[2]), order(k[1], k[3]), order(k[1], k[2]);
}
template <class T>
__device__ __forceinline__ void sort8(T* k) {   // (K. Batcher, "Sorting networks and their applications", 1968)
  sort4(k), sort4(k + 4);
  order(k[0], k[4]), order(k[1], k[5]), order(k[2], k[6]), order(k[3], k[7]);
  order(k[2], k[4]), order(k[3], k[5]), order(k[1], k[2]), order(k[3], k[4]), order(k[5], k[6]);
}
template <int N, class T>
__device__ __forceinline__ void clean(T* k) {   // of a bitonic sequence
#pragma unroll
  for (int s = N / 2; s; s /= 2)
#pragma unroll
    for (int i = 0; i < N; i++)
      if (!(i & s)) order(k[i], k[i + s]);
}
// the N greatest of two sorted lists, in a
template <int N, class T>
__device__ __forceinline__ void merge(T* a, const T* b) {
#pragma unroll
  for (int i = 0; i < N; i++) a[i] = ::max(a[i], b[N - 1 - i]);
  clean<N>(a);
}
// The largest of what merge<N>(a, b) leaves out.
template <int N>
__device__ __forceinline__ int32_t left_out(const int32_t* a, const int32_t* b) {
  int32_t m = INT32_MIN;
#pragma unroll
  for (int i = 0; i < N; i++) m = ::max(m, ::min(a[i], b[N - 1 - i]));
  return m;
}

// The N greatest of 16, in the first places; with LAST, the greatest of the others is returned.
template <bool LAST, int N>
__device__ __forceinline__ int32_t best_of_16(int32_t* k) {
  int32_t last = INT32_MIN;
  if (N <= 4) {
    sort4(k), sort4(k + 4), sort4(k + 8), sort4(k + 12);
    if (LAST) last = ::max(left_out<4>(k, k + 4), left_out<4>(k + 8, k + 12));
    merge<4>(k, k + 4), merge<4>(k + 8, k + 12);
    if (LAST) last = ::max(last, left_out<4>(k, k + 8));
    merge<4>(k, k + 8);
  } else if (N <= 8) {
    sort8(k), sort8(k + 8);
    if (LAST) last = left_out<8>(k, k + 8);
    merge<8>(k, k + 8);
  } else {
    sort8(k), sort8(k + 8);
#pragma unroll
    for (int i = 0; i < 8; i++) order(k[i], k[15 - i]);
    clean<8>(k), clean<8>(k + 8);
  }
  return last;
}

// ------------------------------------------------------------------- a block's sums and counts
// In shared memory: counts of each expert, then sums of each warp, and in a grid that is one cluster, a
// place for each of its blocks' sums and counts.  There each block leaves its own with the first one, which
// writes the results; else for k_route_join.
__device__ __forceinline__ void finish(const RouteArgs& P, const int32_t* counts, float* sums, int32_t* reals,
                                       float* parts) {
  const uint32_t E = P.experts, threads = blockDim.x, warps = threads / 32, C = gridDim.x, c = blockIdx.x;
  const cg::cluster_group cluster = cg::this_cluster();
  float* all_sums = sums + warps * E;                                    // C x E, then as many counts
  int32_t* all_counts = reinterpret_cast<int32_t*>(all_sums + C * E);    // (if P.joined)
  __shared__ int32_t all_reals[kMaxCluster];
  __syncthreads();
  if (P.joined) {
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");   // (the first block is there)
    all_sums = cluster.map_shared_rank(all_sums + c * E, 0);
    all_counts = cluster.map_shared_rank(all_counts + c * E, 0);
  }
  for (uint32_t e = threadIdx.x; e < E; e += threads) {
    float s = 0.f;
    for (uint32_t i = 0; i < warps; i++) s += sums[i * E + e];
    if (P.joined) {
      all_sums[e] = s;
      all_counts[e] = counts[e];
    } else {
      P.sums[(uint64_t)c * E + e] = s;
      P.counts[(uint64_t)c * E + e] = counts[e];
    }
  }
  if (threadIdx.x == 0) {
    int32_t n = 0;
    for (uint32_t i = 0; i < warps; i++) n += reals[i];
    if (P.joined) *cluster.map_shared_rank(&all_reals[c % kMaxCluster], 0) = n;
    else P.real[c] = n;
  }
  if (!P.joined) return;
  cluster.sync();
  if (c != 0) return;
  int32_t N = 0;
  for (uint32_t b = 0; b < C; b++) N += all_reals[b];
  float share = 0.f;
  for (uint32_t e = threadIdx.x; e < E; e += threads) {
    float s = 0.f;
    int32_t n = 0;
    for (uint32_t b = 0; b < C; b++) s += all_sums[b * E + e], n += all_counts[b * E + e];
    const float p = N > 0 ? s / (float)N : 0.f;
    P.out_probs[e] = p;
    P.out_counts[e] = n;
    share += p * (float)n;
  }
  share = warp_sum(share);
  if (threadIdx.x % 32 == 0) parts[threadIdx.x / 32] = share;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (uint32_t i = 1; i < warps; i++) share += parts[i];
    *P.out_loss = N > 0 ? share / (float)N * ((float)E / (float)P.k) : 0.f;
    *P.out_real = N;
  }
}

// Joins the blocks' sums and counts.  Each block of the one cluster takes a part of the experts; its
// threads read as many slices of the blocks' rows at a time as there is room for, and a warp joins the
// slices of an expert.  Every sum has a fixed order.  (In FP32: with FP64, of which an SM does a few
// operations a cycle, 304 rows of 128 experts took 32 us.)
__global__ void __launch_bounds__(kJoinThreads) k_route_join(const RouteArgs P, uint32_t blocks) {
  __shared__ float sums[2 * kJoinThreads];
  __shared__ int32_t counts[2 * kJoinThreads];
  __shared__ float parts[kJoinThreads / 32], shares[kMaxCluster];
  __shared__ int32_t reals[kJoinThreads / 32];
  after_previous();
  asm volatile("barrier.cluster.arrive.relaxed.aligned;");   // (before another block's memory is written)
  const cg::cluster_group cluster = cg::this_cluster();
  const uint32_t E = P.experts, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const uint32_t C = gridDim.x, width = (E + C - 1) / C, first = blockIdx.x * width;
  const uint32_t slices = kJoinThreads / width, slice = threadIdx.x / width, col = threadIdx.x % width;
  float s = 0.f;
  int32_t c = 0, r = 0;
  if (slice < slices && first + col < E) {
#pragma unroll 8
    for (uint32_t b = slice; b < blocks; b += slices) {
      s += P.sums[(uint64_t)b * E + first + col];
      c += P.counts[(uint64_t)b * E + first + col];
    }
  }
  for (uint32_t b = threadIdx.x; b < blocks; b += kJoinThreads) r += P.real[b];
  if (slice < slices) {
    sums[slice * (width + 1) + col] = s;   // (a column's entries fall into different banks)
    counts[slice * (width + 1) + col] = c;
  }
  r = __reduce_add_sync(kAll, r);
  if (lane == 0) reals[warp] = r;
  __syncthreads();
  const int32_t N = __reduce_add_sync(kAll, reals[lane]);
  float share = 0.f;
  for (uint32_t i = warp; i < width && first + i < E; i += kJoinThreads / 32) {
    s = 0.f;
    c = 0;
    for (uint32_t j = lane; j < slices; j += 32) s += sums[j * (width + 1) + i], c += counts[j * (width + 1) + i];
    s = warp_sum(s);
    c = __reduce_add_sync(kAll, c);
    const float p = N > 0 ? s / (float)N : 0.f;
    if (lane == 0) {
      P.out_probs[first + i] = p;
      P.out_counts[first + i] = c;
    }
    share += p * (float)c;
  }
  if (lane == 0) parts[warp] = share;
  __syncthreads();
  asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
  if (warp == 0) {
    share = warp_sum(parts[lane]);
    if (lane == 0) *cluster.map_shared_rank(&shares[blockIdx.x], 0) = share;
  }
  cluster.sync();
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    share = shares[0];
    for (uint32_t b = 1; b < C; b++) share += shares[b];
    *P.out_loss = N > 0 ? share / (float)N * ((float)E / (float)P.k) : 0.f;
    *P.out_real = N;
  }
}

// ------------------------------------------------------------------------------ forward pass
// One warp a token, for few tokens, or more experts or choices than k_route_many takes: lane l holds
// experts l, l + 32, ...; a choice is a maximum over the warp, which the hardware finds in one
// instruction (FP32 keys: two).  64 tokens of 128 experts take 3.4 us, launch to end, in one cluster of
// eight blocks that also writes the counts and the loss; 2000 tokens 6.8 us, 3 of them k_route_join.
template <bool F32, int NV>
__global__ void __launch_bounds__(kThreads) k_route(const RouteArgs P) {
  extern __shared__ uint32_t sh[];
  int32_t* counts = reinterpret_cast<int32_t*>(sh);
  float* sums = reinterpret_cast<float*>(sh + P.experts);
  __shared__ int32_t reals[kWarps];
  __shared__ float parts[kWarps];
  typedef Keys<F32> K;
  typedef typename K::T Key;
  after_previous();
  if (P.joined) asm volatile("barrier.cluster.arrive.relaxed.aligned;");   // (waited for in `finish`)
  const uint32_t warp = threadIdx.x / 32, lane = threadIdx.x % 32, E = P.experts;
  for (uint32_t e = threadIdx.x; e < E; e += kThreads) counts[e] = 0;
  __syncthreads();
  float total[NV];
#pragma unroll
  for (int j = 0; j < NV; j++) total[j] = 0.f;
  int32_t real = 0;
  for (uint64_t t = (uint64_t)warp * gridDim.x + blockIdx.x; t < P.tokens; t += (uint64_t)gridDim.x * kWarps) {
    const uint8_t* row = P.x + t * P.ld;
    bool use = !P.mask || P.mask[t * P.mask_stride] != 0;
    Key key[NV], mine = 0;   // lane i: the i-th choice
    float p[NV], sum = 0.f, w = 0.f;
    if (use) {
      Key top = K::kNone;
#pragma unroll
      for (int j = 0; j < NV; j++) {
        const uint32_t e = lane + 32 * j;
        p[j] = e < E ? element<F32>(row, e) : __int_as_float(0xFF800000);
        key[j] = e < E ? K::make(p[j], e) : K::kNone;
        top = ::max(key[j], top);
      }
      const Key best = K::warp_max(top);
      const float max = K::value(best);
      use = max != __int_as_float(0xFF800000);
      if (use) {
#pragma unroll
        for (int j = 0; j < NV; j++) {
          p[j] = ex2((p[j] - max) * kLog2e);
          sum += p[j];
        }
        sum = warp_sum(sum);
        const float inv = 1.f / sum;
#pragma unroll
        for (int j = 0; j < NV; j++) total[j] += p[j] * inv;
        mine = choose<F32, NV>(key, best, P.k, lane);
        w = lane < P.k ? ex2((K::value(mine) - max) * kLog2e) : 0.f;
        w *= P.normalize ? 1.f / warp_sum(w) : inv;
        if (lane < P.k) atomicAdd(&counts[K::expert(mine)], 1);
        real++;
      }
    }
    if (lane < P.k) {
      P.weights[t * P.k + lane] = use ? w : 0.f;
      P.chosen[t * P.k + lane] = use ? (int32_t)K::expert(mine) : -1;
    }
  }
#pragma unroll
  for (int j = 0; j < NV; j++) {
    const uint32_t e = lane + 32 * j;
    if (e < E) sums[warp * E + e] = total[j];
  }
  if (lane == 0) reals[warp] = real;
  finish(P, counts, sums, reals, parts);
}

// A warp takes up to 32 tokens at a time.  `lanes` lanes share a token, 16 experts each, and it takes
// rounds of 32 / lanes tokens; in each, a lane finds the KL greatest of its 16 keys.  Lanes join their
// lists in pairs as soon as two rounds have one each: one of the two lanes goes on with the first
// round's token, the other with the second's.  After `lanes` rounds each lane has the whole list of one
// token: a join costs each list once, and not each lane.  Lists that wait lie in shared memory.  With
// fewer rounds, where there are too few tokens for all warps, lanes that no round brought together join
// their lists twice, once in each.
//
// The ALU pipe bounds it (73% of its rate; 1000000 tokens of 128 experts in 144 us): 62 of a token's 105
// instructions are minima, maxima, selections and permutations, 34 of them the sorting networks'.  HBM
// is at a third.  A third block an SM does not help (51 us for 262144 tokens, with two 50).
template <bool F32, int KL>
struct Lists {
  int4 key[KL / 4][32];
  int32_t out[F32 ? 32 : 1];   // the greatest key that is not in the list
};
template <bool F32, int KL>
__device__ __forceinline__ void put(Lists<F32, KL>& l, uint32_t lane, const int32_t* k, int32_t out) {
#pragma unroll
  for (int i = 0; i < KL / 4; i++) l.key[i][lane] = make_int4(k[4 * i], k[4 * i + 1], k[4 * i + 2], k[4 * i + 3]);
  if (F32) l.out[lane] = out;
}
template <bool F32, int KL>
__device__ __forceinline__ int32_t get(const Lists<F32, KL>& l, uint32_t lane, int32_t* k) {
#pragma unroll
  for (int i = 0; i < KL / 4; i++) {
    const int4 v = l.key[i][lane];
    k[4 * i] = v.x, k[4 * i + 1] = v.y, k[4 * i + 2] = v.z, k[4 * i + 3] = v.w;
  }
  return F32 ? l.out[lane] : 0;
}
constexpr uint32_t kLevels = 4;   // 16 lanes a token at most: 256 experts
template <bool F32, int KL>
struct Many {
  static constexpr uint32_t kMostWarps = !F32 && KL <= 8 ? 9 : 8;   // two blocks of them an SM (10 would fit: 262144 tokens 47.1 us, with 9 46.7)
  static constexpr uint32_t kWarpBytes = (kLevels + 1) * (uint32_t)sizeof(Lists<F32, KL>);
};

template <bool F32, int KL>
__global__ void __launch_bounds__((Many<F32, KL>::kMostWarps * 32), 2) k_route_many(const RouteArgs P) {
  extern __shared__ int4 sh4[];
  typedef Lists<F32, KL> L;
  typedef Short<F32> S;
  int32_t* counts = reinterpret_cast<int32_t*>(reinterpret_cast<uint8_t*>(sh4) + blockDim.x / 32 * Many<F32, KL>::kWarpBytes);
  float* sums = reinterpret_cast<float*>(counts + P.experts);
  __shared__ int32_t reals[Many<F32, KL>::kMostWarps];
  __shared__ float parts[Many<F32, KL>::kMostWarps];
  after_previous();
  const uint32_t warp = threadIdx.x / 32, lane = threadIdx.x % 32, E = P.experts, G = P.lanes, R = P.rounds;
  const uint32_t g = lane % G, q = lane / G, e0 = g * kLane, own = g % R, per = 32 / G * R;
  const Lanes<kLevels> lanes(G);
  L* const wait = reinterpret_cast<L*>(sh4) + warp * (kLevels + 1);
  for (uint32_t e = threadIdx.x; e < E; e += blockDim.x) counts[e] = 0;
  __syncthreads();
  const uint32_t units = (P.tokens + per - 1) / per, step = gridDim.x * (blockDim.x / 32);
  float2 total[kLane / 2];
#pragma unroll
  for (int j = 0; j < (int)kLane / 2; j++) total[j] = make_float2(0.f, 0.f);
  int32_t real = 0;
  Logits<F32, kLane> ahead;
  bool use_ahead = false;
  auto fetch = [&](uint32_t unit, uint32_t round) {
    const uint64_t t = (uint64_t)unit * per + q * R + round;
    use_ahead = t < P.tokens && (!P.mask || P.mask[t * P.mask_stride] != 0);
    if (use_ahead) ahead.load(P.x + t * P.ld, e0, E, P.vec);
    else ahead.clear();
  };
  uint32_t unit = warp * gridDim.x + blockIdx.x;
  if (unit < units) fetch(unit, 0);
  for (; unit < units; unit += step) {
    float sum_mine = 0.f, max_mine = 0.f;
    bool use_mine = false;
    int32_t list[kLane], out = INT32_MIN;
#pragma unroll 1
    for (uint32_t round = 0; round < R; round++) {
      const Logits<F32, kLane> x = ahead;
      bool use = use_ahead;
      if (round + 1 < R) fetch(unit, round + 1);
      else if (unit + step < units) fetch(unit + step, 0);
      float max = lanes.max(x.max());
      if (max == __int_as_float(0xFF800000)) use = false, max = 0.f;
      float2 e[kLane / 2], s = make_float2(0.f, 0.f);
#pragma unroll
      for (int j = 0; j < (int)kLane / 2; j++) {
        const float2 d = __fmul2_rn(__fadd2_rn(x.pair(j), make_float2(-max, -max)), make_float2(kLog2e, kLog2e));
        e[j] = make_float2(ex2(d.x), ex2(d.y));
        s = __fadd2_rn(s, e[j]);
      }
      const float sum = lanes.sum(s.x + s.y);
      const float inv = use ? rcp(sum) : 0.f;
#pragma unroll
      for (int j = 0; j < (int)kLane / 2; j++) total[j] = __ffma2_rn(e[j], make_float2(inv, inv), total[j]);
      if (round == own) sum_mine = sum, max_mine = max, use_mine = use;
      S::make(x, list);
      out = best_of_16<F32, KL>(list);
#pragma unroll
      for (int i = 0; i < KL; i++) list[i] += S::base(e0);
      if (F32) out += S::base(e0);
      // join as many times as the round's number ends in ones, then wait
      uint32_t level = 0;
#pragma unroll 1
      for (; (round >> level & 1) != 0; level++) {
        put(wait[kLevels], lane, list, out);
        __syncwarp();
        const L& from = lane >> level & 1 ? wait[kLevels] : wait[level];
        int32_t other[KL];
        const int32_t out1 = get(from, lane, list), out2 = get(from, lane ^ (1u << level), other);
        if (F32) out = ::max(::max(out1, out2), left_out<KL>(list, other));
        merge<KL>(list, other);
        __syncwarp();
      }
      if (round + 1 < R) put(wait[level], lane, list, out);
    }
    // lanes whose parts no round brought together: each of two joins both lists
#pragma unroll 1
    for (uint32_t d = R; d < G; d *= 2) {
      int32_t other[KL];
#pragma unroll
      for (int i = 0; i < KL; i++) other[i] = __shfl_xor_sync(kAll, list[i], d);
      if (F32) out = ::max(::max(out, __shfl_xor_sync(kAll, out, d)), left_out<KL>(list, other));
      merge<KL>(list, other);
    }
    const uint64_t t = (uint64_t)unit * per + q * R + own;
    const bool mine = g < R && t < P.tokens;   // (the token is this lane's to write)
    if (!mine) use_mine = false;
    real += __popc(__ballot_sync(kAll, use_mine));
    uint32_t expert[KL];
    float x[KL];
#pragma unroll
    for (int i = 0; i < KL; i++) {
      expert[i] = S::expert(list[i]);
      x[i] = F32 ? 0.f : S::value(list[i]);
    }
    if (F32) {
      const float* row = reinterpret_cast<const float*>(P.x + t * P.ld);
      bool unsure = false;
      if (use_mine) {
#pragma unroll
        for (int i = 0; i < KL; i++)
          if (i < (int)P.k) x[i] = row[expert[i]];
        // keys that are alike but for the expert: in order by the whole logits, or to be done again
#pragma unroll
        for (int i = 0; i < KL; i++) {
          const int32_t next = i + 1 < KL ? list[i + 1 < KL ? i + 1 : i] : out;
          if (i < (int)P.k && ((uint32_t)list[i] ^ (uint32_t)next) <= S::kExpertBits)
            if (i + 1 >= (int)P.k || !(x[i] >= x[i + 1 < KL ? i + 1 : i])) unsure = true;
        }
      }
      for (uint32_t who = __ballot_sync(kAll, unsure); who; who &= who - 1) {
        const uint32_t src = __ffs(who) - 1;
        const uint8_t* again = P.x + __shfl_sync(kAll, t, src) * P.ld;
        typedef Keys<F32> K;
        typename K::T key[kLane / 2], top = K::kNone;
#pragma unroll
        for (int j = 0; j < (int)kLane / 2; j++) {
          const uint32_t e = lane + 32 * j;
          key[j] = e < E ? K::make(element<F32>(again, e), e) : K::kNone;
          top = ::max(top, key[j]);
        }
        const typename K::T best = choose<F32, (int)kLane / 2>(key, K::warp_max(top), P.k, lane);
#pragma unroll
        for (int i = 0; i < KL; i++) {
          const uint32_t ei = __shfl_sync(kAll, K::expert(best), i);
          const float xi = __shfl_sync(kAll, K::value(best), i);
          if (lane == src && i < (int)P.k) expert[i] = ei, x[i] = xi;
        }
      }
    }
    if (mine) {
      float w[KL], s[KL];
#pragma unroll
      for (int i = 0; i < KL; i++) {
        w[i] = ex2((x[i] - max_mine) * kLog2e);
        s[i] = i < (int)P.k ? w[i] : 0.f;
      }
#pragma unroll
      for (int n = KL / 2; n; n /= 2)   // (as warp_sum does: a token's normalized weights are k_route's)
#pragma unroll
        for (int i = 0; i < n; i++) s[i] += s[i + n];
      const float inv = 1.f / (P.normalize ? s[0] : sum_mine);
      float* to = P.weights + t * P.k;
      int32_t* at = P.chosen + t * P.k;
      uint32_t wo[KL];
#pragma unroll
      for (int i = 0; i < KL; i++) {
        wo[i] = use_mine ? __float_as_uint(w[i] * inv) : 0u;
        if (use_mine && i < (int)P.k) atomicAdd(&counts[expert[i]], 1);
        if (!use_mine) expert[i] = 0xffffffffu;
      }
      if (KL == 8 && P.k == 8) {
        st32(to, wo);
        st32(at, expert);
      } else {
#pragma unroll
        for (int i = 0; i < KL; i++)
          if (i < (int)P.k) to[i] = __uint_as_float(wo[i]), at[i] = (int32_t)expert[i];
      }
    }
  }
#pragma unroll
  for (int j = 0; j < (int)kLane / 2; j++) {
    for (uint32_t d = G; d < 32; d *= 2) {
      total[j].x += __shfl_xor_sync(kAll, total[j].x, d);
      total[j].y += __shfl_xor_sync(kAll, total[j].y, d);
    }
    if (q == 0 && e0 + 2 * j < E) sums[warp * E + e0 + 2 * j] = total[j].x;
    if (q == 0 && e0 + 2 * j + 1 < E) sums[warp * E + e0 + 2 * j + 1] = total[j].y;
  }
  if (lane == 0) reals[warp] = real;
  finish(P, counts, sums, reals, parts);
}

// ----------------------------------------------------------------------------- backward pass
// `lanes` lanes share a token, N experts each and at most one of its choices each.  The choices'
// logits get their gradient on top of the others' a second time, from the lanes that hold them: the
// other way, handing each choice to the lane that holds its expert, costs an instruction for each of
// a lane's experts and choices.  1000000 tokens of 128 FP32 logits take 206 us, 5.3 TB/s (HBM); 32768 8 us.
template <bool F32, int N>
__global__ void __launch_bounds__(kThreads, 2) k_route_grad(const RouteGradArgs P) {
  extern __shared__ float share[];   // how often each expert was chosen
  __shared__ long long parts[kWarps];
  after_previous();
  const uint32_t warp = threadIdx.x / 32, lane = threadIdx.x % 32, E = P.experts, G = P.lanes;
  const uint32_t g = lane % G, q = lane / G, e0 = g * N, per = 32 / G;
  const Lanes<5> lanes(G);
  const uint64_t groups = ((uint64_t)P.tokens + per - 1) / per, step = (uint64_t)gridDim.x * kWarps;
  uint64_t n = (uint64_t)warp * gridDim.x + blockIdx.x;
  Logits<F32, N> x;
  int32_t mine;
  float gw;
  auto fetch = [&]() {
    const uint64_t t = n * per + q;
    const bool choose = t < P.tokens && g < P.k;
    mine = choose ? P.chosen[t * P.k + g] : -1;
    gw = choose && P.gw ? P.gw[t * P.gw_stride + g * P.gw_choice] : 0.f;
    if (t < P.tokens) x.load(P.x + t * P.ld, e0, E, P.vec);
    else x.clear();
  };
  if (n < groups) fetch();   // (under way while the experts' shares are worked out)
  long long sum = 0;
  for (uint32_t e = threadIdx.x; e < E; e += kThreads) {
    const int32_t m = P.counts[e];
    share[e] = (float)m;
    sum += m;
  }
#pragma unroll
  for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(kAll, sum, d);
  if (lane == 0) parts[warp] = sum;
  __syncthreads();
  sum = 0;
#pragma unroll
  for (uint32_t i = 0; i < kWarps; i++) sum += parts[i];
  const int32_t real = *P.real;
  const float gl = P.gloss ? *P.gloss : P.loss;
  const float unit = sum > 0 && real > 0 ? gl * ((float)E / (float)real) / (float)sum : 0.f;
  float2 c[N / 2];
#pragma unroll
  for (int j = 0; j < N / 2; j++)
    c[j] = make_float2(e0 + 2 * j < E ? unit * share[e0 + 2 * j] : 0.f, e0 + 2 * j + 1 < E ? unit * share[e0 + 2 * j + 1] : 0.f);
  for (; n < groups; n += step) {
    const uint64_t t = n * per + q;
    const bool there = t < P.tokens;
    const uint8_t* row = P.x + t * P.ld;
    uint8_t* out = P.dx + t * P.ld_dx;
    if (step <= n) fetch();
    if ((uint32_t)mine >= E) mine = -1;   // (the caller may have written there)
    const float xm = mine >= 0 ? element<F32>(row, (uint32_t)mine) : 0.f;
    const bool use = __shfl_sync(kAll, mine, q * G) >= 0;
    const float max = lanes.max(x.max());
    float2 p[N / 2], s = make_float2(0.f, 0.f);
#pragma unroll
    for (int j = 0; j < N / 2; j++) {
      const float2 d = __fmul2_rn(__fadd2_rn(x.pair(j), make_float2(-max, -max)), make_float2(kLog2e, kLog2e));
      p[j] = make_float2(ex2(d.x), ex2(d.y));
      s = __fadd2_rn(s, p[j]);
    }
    const float inv = rcp(lanes.sum(s.x + s.y));
    float2 dots = make_float2(0.f, 0.f);
#pragma unroll
    for (int j = 0; j < N / 2; j++) {
      p[j] = __fmul2_rn(p[j], make_float2(inv, inv));
      dots = __ffma2_rn(p[j], c[j], dots);
    }
    float dot = dots.x + dots.y;       // of p and dL/dp
    const float pm = mine >= 0 ? ex2((xm - max) * kLog2e) * inv : 0.f;
    float add;                         // what the choice adds to its logit
    if (P.normalize) {
      const float w = pm / lanes.sum(pm);   // (1 of a single choice, whose gradient cancels)
      add = w * (gw - lanes.sum(mine >= 0 ? w * gw : 0.f));
    } else {
      add = pm * gw;
      dot += mine >= 0 ? add : 0.f;
    }
    dot = lanes.sum(dot);
    __syncwarp();   // (the rows are read: their gradients may take their place)
    if (there) {
      uint32_t o[Logits<F32, N>::kWords];
#pragma unroll
      for (int j = 0; j < N / 2; j++) {
        float2 d = __fmul2_rn(p[j], __fadd2_rn(c[j], make_float2(-dot, -dot)));
        if (!use) d = make_float2(0.f, 0.f);
        if (F32) o[2 * j] = __float_as_uint(d.x), o[2 * j + 1] = __float_as_uint(d.y);
        else o[j] = pack_bf16(d.x, d.y);
      }
      if (P.vec_dx && e0 < E) {
#pragma unroll
        for (int i = 0; i < Logits<F32, N>::kWords; i += 8) st32(out + (uint64_t)e0 * (F32 ? 4 : 2) + i * 4, o + i);
      } else {
#pragma unroll
        for (int i = 0; i < N; i++) {
          if (e0 + i >= E) continue;
          if (F32) reinterpret_cast<uint32_t*>(out)[e0 + i] = o[i];
          else reinterpret_cast<uint16_t*>(out)[e0 + i] = (uint16_t)(o[i / 2] >> (16 * (i & 1)));
        }
      }
    }
    __syncwarp();
    if (mine >= 0) {
      const float d = pm * (unit * share[mine] - dot) + add;
      if (F32) reinterpret_cast<float*>(out)[mine] = d;
      else reinterpret_cast<uint16_t*>(out)[mine] = (uint16_t)pack_bf16(d, 0.f);
    }
  }
}

// --------------------------------------------------------------------------------- host side
struct Layout {
  uint64_t weights, experts, counts, probs, loss, real, partials, total;
};
bool layout(uint32_t tokens, uint32_t experts, uint32_t k, Layout& L) {
  if (tokens > BO_ROUTING_MAX_TOKENS || experts == 0 || experts > BO_ROUTING_MAX_EXPERTS || k == 0 ||
      k > experts || k > BO_ROUTING_MAX_K)
    return false;
  uint64_t off = 0;
  auto take = [&](uint64_t bytes) {
    const uint64_t at = off;
    off = up(off + bytes, 256);
    return at;
  };
  L.weights = take((uint64_t)tokens * k * 4);
  L.experts = take((uint64_t)tokens * k * 4);
  L.counts = take((uint64_t)experts * 4);
  L.probs = take((uint64_t)experts * 4);
  L.loss = take(4);
  L.real = take(4);
  L.partials = take((uint64_t)kMaxBlocks * (experts * 2 + 1) * 4);
  L.total = off;
  return true;
}
bool valid(const bo_routing* h) {
  Layout L;
  return h && h->d_weights && h->d_experts && h->d_counts && h->d_probs && h->d_loss && h->d_real &&
         h->d_partials && h->normalize <= 1 && layout(h->tokens, h->experts, h->k, L);
}
Region results(const bo_routing* h) {
  Layout L;
  layout(h->tokens, h->experts, h->k, L);
  return Region(h->d_weights, 1, 0, L.total, 1);
}
bool matrix(const void* p, uint64_t ld, uint64_t rows, uint64_t width, uint64_t size) {
  return p && aligned(p, size) && ld <= (1ull << 40) && (rows <= 1 || ld >= width);
}
uint32_t power_of_two(uint32_t n) {   // the least that is not below n
  uint32_t p = 1;
  while (p < n) p *= 2;
  return p;
}
// rows whose parts of `each` elements are whole, aligned words of 32 bytes
bool whole(const void* p, uint64_t ld, uint32_t width, uint32_t each) {   // (ld in bytes)
  return aligned(p, 32) && ld % 32 == 0 && width % each == 0;
}
template <bool F32, int KL>
int route_many(const RouteArgs& P, uint32_t grid, cudaStream_t s) {
  // Of the numbers of warps a block, the one that leaves the fewest without work in the last turn: 262144
  // tokens are 27 turns of 304 blocks' warps, 3 of 9 (0.9 us less) and not 4 of 8.
  const uint32_t per = 32 / P.lanes * P.rounds, turns = ((P.tokens + per - 1) / per + grid - 1) / grid;   // of a block with one warp
  uint32_t warps = Many<F32, KL>::kMostWarps, least = ~0u;
  for (uint32_t w = warps; w >= 4; w--) {
    const uint32_t all = (turns + w - 1) / w * w;
    if (all < least) least = all, warps = w;
  }
  return check(launch(k_route_many<F32, KL>, dim3(grid), warps * 32,
                      warps * Many<F32, KL>::kWarpBytes + P.experts * (1 + warps) * 4, 1, s, P));
}
template <bool F32>
int route(RouteArgs& P, uint32_t sms, cudaStream_t s) {
  const uint32_t smem = P.experts * (1 + kWarps) * 4;
  const uint32_t nv = (P.experts + 31) / 32;
  auto one = nv <= 1 ? k_route<F32, 1> : nv <= 2 ? k_route<F32, 2> : nv <= 4 ? k_route<F32, 4>
           : nv <= 8 ? k_route<F32, 8> : nv <= 16 ? k_route<F32, 16> : k_route<F32, 32>;
  if (P.tokens <= kMaxCluster * kWarps * 2) {   // one launch
    const uint32_t grid = P.tokens <= kWarps ? 1 : P.tokens <= 2 * kWarps ? 2 : P.tokens <= 4 * kWarps ? 4 : kMaxCluster;
    P.joined = 1;
    return check(launch(one, dim3(grid), kThreads, smem + grid * P.experts * 8, grid, s, P));
  }
  P.joined = 0;
  const uint32_t lanes = power_of_two((P.experts + kLane - 1) / kLane);
  uint32_t grid;
  int rc;
  // One bound for all numbers of experts, near where the two forms meet: 6000 tokens in the first one and 6001
  // in the second take 7.4 and 7.5 us of 16 experts (FP32 7.3 and 8.2), 9.9 and 9.3 of 128 (12.0 and 10.6), 13.2
  // and 12.7 of 256 (17.2 and 15.3).  With 256 experts they meet at 3000 already.
  if (P.tokens > 6000 && lanes <= 1u << kLevels && P.k <= 16) {
    P.lanes = lanes;
    P.vec = whole(P.x, P.ld, P.experts, kLane);
    // As many rounds as leave most warps some (128 experts: 20000 tokens take 12.5 us with 2 rounds
    // and 14.6 with 8, 262144 tokens 58 and 48).
    P.rounds = lanes;
    while (P.rounds > 1 && P.tokens / (32 / lanes * P.rounds) < sms * 12) P.rounds /= 2;
    const uint32_t per = 32 / lanes * P.rounds;
    grid = std::min({(P.tokens + per - 1) / per, sms * 2, kMaxBlocks});
    rc = P.k <= 4 ? route_many<F32, 4>(P, grid, s) : P.k <= 8 ? route_many<F32, 8>(P, grid, s) : route_many<F32, 16>(P, grid, s);
  } else {
    grid = std::min({(P.tokens + kWarps - 1) / kWarps, sms * 3, kMaxBlocks});
    rc = check(launch(one, dim3(grid), kThreads, smem, 1, s, P));
  }
  if (rc) return rc;
  const uint32_t C = std::min(power_of_two((P.experts + 7) / 8), kMaxCluster);
  return check(launch(k_route_join, dim3(C), kJoinThreads, 0, C, s, P, grid));
}
template <bool F32>
int route_grad(RouteGradArgs& P, uint32_t sms, cudaStream_t s) {
  const uint32_t each = P.experts <= 32 * kLane ? kLane : 2 * kLane;
  P.lanes = power_of_two(std::max((P.experts + each - 1) / each, P.k));
  P.vec = whole(P.x, P.ld, P.experts, each);
  P.vec_dx = whole(P.dx, P.ld_dx, P.experts, each);
  const uint64_t groups = ((uint64_t)P.tokens * P.lanes + 31) / 32;
  const uint32_t grid = (uint32_t)std::min<uint64_t>((groups + kWarps - 1) / kWarps, sms * 2);
  return check(launch(each == kLane ? k_route_grad<F32, kLane> : k_route_grad<F32, 2 * kLane>, dim3(grid), kThreads,
                      P.experts * 4, 1, s, P));
}

}  // namespace
}  // namespace bo

using namespace bo;

extern "C" {

uint64_t bo_routing_size(uint32_t tokens, uint32_t experts, uint32_t k) {
  Layout L;
  return layout(tokens, experts, k, L) ? L.total : 0;
}

int bo_routing_init(uint32_t tokens, uint32_t experts, uint32_t k, uint32_t normalize, void* d_mem,
                    uint64_t mem_bytes, bo_routing* h_out, void* stream) {
  Layout L;
  if (!h_out || !layout(tokens, experts, k, L) || normalize > 1 || !d_mem || !aligned(d_mem, 256) ||
      mem_bytes < L.total)
    return BD_ERR_INVALID_ARG;
  uint8_t* p = static_cast<uint8_t*>(d_mem);
  bo_routing h = {};
  h.d_weights = reinterpret_cast<float*>(p + L.weights);
  h.d_experts = reinterpret_cast<int32_t*>(p + L.experts);
  h.d_counts = reinterpret_cast<int32_t*>(p + L.counts);
  h.d_probs = reinterpret_cast<float*>(p + L.probs);
  h.d_loss = reinterpret_cast<float*>(p + L.loss);
  h.d_real = reinterpret_cast<int32_t*>(p + L.real);
  h.d_partials = p + L.partials;
  h.tokens = tokens;
  h.experts = experts;
  h.k = k;
  h.normalize = normalize;
  int rc;
  if ((rc = check(cudaGetDevice(&h.device)))) return rc;
  if ((rc = check(cudaMemsetAsync(d_mem, 0, L.total, static_cast<cudaStream_t>(stream))))) return rc;
  *h_out = h;
  return BD_OK;
}

int bo_routing_forward(const bo_routing* h, const void* d_logits, uint32_t dtype, uint64_t ld,
                       uint32_t tokens, const uint8_t* d_mask, uint64_t mask_stride, void* stream) {
  if (!valid(h) || dtype > BO_FP32 || tokens > h->tokens || mask_stride > (1ull << 40))
    return BD_ERR_INVALID_ARG;
  const uint64_t size = dtype == BO_FP32 ? 4 : 2;
  if (tokens > 0) {
    if (!matrix(d_logits, ld, tokens, h->experts, size)) return BD_ERR_INVALID_ARG;
    const Region out = results(h);
    if (meet(out, Region(d_logits, tokens, ld, h->experts, size)) ||
        meet(out, Region(d_mask, mask_stride ? tokens : 1, mask_stride, 1, 1)))
      return BD_ERR_INVALID_ARG;
  }
  int sms = 0;
  if (const int rc = sm_count(h->device, sms)) return rc;
  RouteArgs P = {};
  P.x = static_cast<const uint8_t*>(d_logits);
  P.ld = ld * size;
  P.mask = d_mask;
  P.mask_stride = mask_stride;
  P.tokens = tokens;
  P.experts = h->experts;
  P.k = h->k;
  P.normalize = h->normalize;
  P.weights = h->d_weights;
  P.chosen = h->d_experts;
  P.sums = static_cast<float*>(h->d_partials);
  P.counts = static_cast<int32_t*>(h->d_partials) + (uint64_t)kMaxBlocks * h->experts;
  P.real = P.counts + (uint64_t)kMaxBlocks * h->experts;
  P.out_probs = h->d_probs;
  P.out_counts = h->d_counts;
  P.out_loss = h->d_loss;
  P.out_real = h->d_real;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return dtype == BO_FP32 ? route<true>(P, (uint32_t)sms, s) : route<false>(P, (uint32_t)sms, s);
}

int bo_routing_backward(const bo_routing* h, const void* d_logits, uint32_t dtype, uint64_t ld,
                        uint32_t tokens, const float* d_grad_weights, uint64_t grad_stride,
                        uint64_t grad_choice_stride, float grad_loss, const float* d_grad_loss,
                        const int32_t* d_counts, void* d_grad_logits, uint64_t ld_grad, void* stream) {
  if (!valid(h) || dtype > BO_FP32 || tokens > h->tokens || grad_stride > (1ull << 40) ||
      grad_choice_stride > (1ull << 34) || !aligned(d_grad_weights, 4) || !aligned(d_grad_loss, 4) ||
      !aligned(d_counts, 4))
    return BD_ERR_INVALID_ARG;
  const uint64_t size = dtype == BO_FP32 ? 4 : 2;
  if (tokens > 0) {
    if (!matrix(d_logits, ld, tokens, h->experts, size) ||
        !matrix(d_grad_logits, ld_grad, tokens, h->experts, size))
      return BD_ERR_INVALID_ARG;
    const Region out(d_grad_logits, tokens, ld_grad, h->experts, size);
    const bool in_place = d_grad_logits == d_logits && (ld == ld_grad || tokens == 1);
    const uint64_t span = (tokens - 1) * grad_stride + (h->k - 1) * grad_choice_stride + 1;
    if ((!in_place && meet(out, Region(d_logits, tokens, ld, h->experts, size))) ||
        meet(out, results(h)) || meet(out, Region(d_grad_weights, 1, 0, span, 4)) ||
        meet(out, Region(d_grad_loss, 1, 0, 1, 4)) || meet(out, Region(d_counts, 1, 0, h->experts, 4)))
      return BD_ERR_INVALID_ARG;
  }
  int sms = 0;
  if (const int rc = sm_count(h->device, sms)) return rc;
  if (tokens == 0) return BD_OK;
  RouteGradArgs P = {};
  P.x = static_cast<const uint8_t*>(d_logits);
  P.ld = ld * size;
  P.dx = static_cast<uint8_t*>(d_grad_logits);
  P.ld_dx = ld_grad * size;
  P.gw = d_grad_weights;
  P.gw_stride = grad_stride;
  P.gw_choice = grad_choice_stride;
  P.gloss = d_grad_loss;
  P.loss = grad_loss;
  P.tokens = tokens;
  P.experts = h->experts;
  P.k = h->k;
  P.normalize = h->normalize;
  P.chosen = h->d_experts;
  P.counts = d_counts ? d_counts : h->d_counts;
  P.real = h->d_real;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return dtype == BO_FP32 ? route_grad<true>(P, (uint32_t)sms, s) : route_grad<false>(P, (uint32_t)sms, s);
}

}  // extern "C"
