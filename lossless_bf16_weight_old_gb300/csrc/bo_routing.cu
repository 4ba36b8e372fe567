// bo_routing.cu -- the experts of each token of a mixture, their weights, per-expert counts and the
// balance loss, and the gradient of the router's logits (include/ops/bf16ops.h has the formulas).
#include <cfloat>
#include <cmath>

#include "bo_internal.cuh"

namespace bo {
namespace {

constexpr uint32_t kThreads = 256, kWarps = kThreads / 32;
constexpr uint32_t kMaxBlocks = 304;   // of the forward pass (its partial sums)
constexpr uint32_t kJoinThreads = 1024;
constexpr uint32_t kAll = 0xffffffffu;
constexpr float kLog2e = 1.44269504088896340736f;

struct RouteArgs {
  const uint8_t* x;
  uint64_t ld;            // bytes
  const uint8_t* mask;    // may be NULL
  uint64_t mask_stride;
  uint32_t tokens, experts, k, normalize;
  float* weights;
  int32_t* chosen;
  float* sums;            // of p: one row of `experts` for each block
  int32_t* counts;        // likewise
  int32_t* real;          // one for each block
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
  const int32_t* chosen;
  const int32_t* counts;
  const int32_t* real;
};

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// A whole number that orders values: NaN above all, -0 as 0; 0 is below every one.
__device__ __forceinline__ uint32_t order_of(float x) {
  if (x != x) return 0xFFFFFFFFu;
  const uint32_t u = __float_as_uint(x + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t o) {
  return __uint_as_float(o & 0x80000000u ? o & 0x7FFFFFFFu : ~o);
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(kAll, v, d);
  return v;
}
template <bool F32>
__device__ __forceinline__ float element(const uint8_t* row, uint32_t e) {
  return F32 ? reinterpret_cast<const float*>(row)[e]
             : __uint_as_float((uint32_t) reinterpret_cast<const uint16_t*>(row)[e] << 16);
}

// One warp a token: lane l holds experts l, l + 32, ...
template <bool F32, int NV>
__global__ void __launch_bounds__(kThreads) k_route(const RouteArgs P) {
  extern __shared__ uint32_t sh[];   // experts counts, then experts sums of each warp
  int32_t* counts = reinterpret_cast<int32_t*>(sh);
  float* sums = reinterpret_cast<float*>(sh + P.experts);
  __shared__ int32_t reals[kWarps];
  after_previous();
  const uint32_t warp = threadIdx.x / 32, lane = threadIdx.x % 32, E = P.experts;
  for (uint32_t e = threadIdx.x; e < E; e += kThreads) counts[e] = 0;
  __syncthreads();
  float total[NV];
#pragma unroll
  for (int j = 0; j < NV; j++) total[j] = 0.f;
  int32_t real = 0;
  for (uint64_t t = (uint64_t)blockIdx.x * kWarps + warp; t < P.tokens; t += (uint64_t)gridDim.x * kWarps) {
    const uint8_t* row = P.x + t * P.ld;
    bool use = !P.mask || P.mask[t * P.mask_stride] != 0;
    uint32_t o[NV];
    float p[NV], sum = 0.f, w = 0.f;
    uint32_t mine = 0;       // lane i: the i-th choice
    if (use) {
      uint32_t top = 0;
#pragma unroll
      for (int j = 0; j < NV; j++) {
        const uint32_t e = lane + 32 * j;
        const float x = e < E ? element<F32>(row, e) : __int_as_float(0xFF800000);
        p[j] = x;
        o[j] = e < E ? order_of(x) : 0;
        top = max(top, o[j]);
      }
      top = __reduce_max_sync(kAll, top);
      const float max = value_of(top);
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
        float x_mine = max;
        for (uint32_t i = 0; i < P.k; i++) {
          uint32_t best = 0;
#pragma unroll
          for (int j = 0; j < NV; j++) best = ::max(best, o[j]);
          best = __reduce_max_sync(kAll, best);
          uint32_t at = 0xffffffffu;
#pragma unroll
          for (int j = NV - 1; j >= 0; j--)
            if (o[j] == best) at = lane + 32 * j;
          at = __reduce_min_sync(kAll, at);
#pragma unroll
          for (int j = 0; j < NV; j++)
            if (at == lane + 32 * j) o[j] = 0;
          if (lane == i) {
            mine = at;
            x_mine = value_of(best);
          }
        }
        w = lane < P.k ? ex2((x_mine - max) * kLog2e) : 0.f;
        w *= P.normalize ? 1.f / warp_sum(w) : inv;
        if (lane < P.k) atomicAdd(&counts[mine], 1);
        real++;
      }
    }
    if (lane < P.k) {
      P.weights[t * P.k + lane] = use ? w : 0.f;
      P.chosen[t * P.k + lane] = use ? (int32_t)mine : -1;
    }
  }
#pragma unroll
  for (int j = 0; j < NV; j++) {
    const uint32_t e = lane + 32 * j;
    if (e < E) sums[warp * E + e] = total[j];
  }
  if (lane == 0) reals[warp] = real;
  __syncthreads();
  for (uint32_t e = threadIdx.x; e < E; e += kThreads) {
    float s = 0.f;
    for (uint32_t i = 0; i < kWarps; i++) s += sums[i * E + e];
    P.sums[(uint64_t)blockIdx.x * E + e] = s;
    P.counts[(uint64_t)blockIdx.x * E + e] = counts[e];
  }
  if (threadIdx.x == 0) {
    int32_t n = 0;
    for (uint32_t i = 0; i < kWarps; i++) n += reals[i];
    P.real[blockIdx.x] = n;
  }
}

// Joins the blocks' sums and counts, in their order.
__global__ void __launch_bounds__(kJoinThreads) k_route_join(const float* sums, const int32_t* counts,
                                                             const int32_t* reals, uint32_t blocks,
                                                             uint32_t E, uint32_t k, float* probs,
                                                             int32_t* n, float* loss, int32_t* real) {
  __shared__ double part[kJoinThreads];
  __shared__ int32_t total;
  after_previous();
  if (threadIdx.x == 0) {
    int32_t r = 0;
    for (uint32_t b = 0; b < blocks; b++) r += reals[b];
    total = r;
    *real = r;
  }
  __syncthreads();
  const int32_t N = total;
  double share = 0;
  for (uint32_t e = threadIdx.x; e < E; e += kJoinThreads) {
    double s = 0;
    int32_t c = 0;
    for (uint32_t b = 0; b < blocks; b++) {
      s += sums[(uint64_t)b * E + e];
      c += counts[(uint64_t)b * E + e];
    }
    const double p = N > 0 ? s / N : 0;
    probs[e] = (float)p;
    n[e] = c;
    share += p * c;
  }
  part[threadIdx.x] = share;
  __syncthreads();
  for (uint32_t d = kJoinThreads / 2; d; d /= 2) {
    if (threadIdx.x < d) part[threadIdx.x] += part[threadIdx.x + d];
    __syncthreads();
  }
  if (threadIdx.x == 0) *loss = N > 0 ? (float)(part[0] * E / ((double)N * k)) : 0.f;
}

template <bool F32, int NV>
__global__ void __launch_bounds__(kThreads) k_route_grad(const RouteGradArgs P) {
  __shared__ long long parts[kWarps];
  after_previous();
  const uint32_t warp = threadIdx.x / 32, lane = threadIdx.x % 32, E = P.experts;
  long long sum = 0;
  for (uint32_t e = threadIdx.x; e < E; e += kThreads) sum += P.counts[e];
#pragma unroll
  for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(kAll, sum, d);
  if (lane == 0) parts[warp] = sum;
  __syncthreads();
  sum = 0;
  for (uint32_t i = 0; i < kWarps; i++) sum += parts[i];
  const int32_t N = *P.real;
  const float gl = P.gloss ? *P.gloss : P.loss;
  // dL/dp of expert e is unit * counts[e]
  const float unit = sum > 0 && N > 0 ? (float)((double)gl * E / ((double)sum * N)) : 0.f;
  for (uint64_t t = (uint64_t)blockIdx.x * kWarps + warp; t < P.tokens; t += (uint64_t)gridDim.x * kWarps) {
    uint8_t* out = P.dx + t * P.ld_dx;
    const int32_t mine = lane < P.k ? P.chosen[t * P.k + lane] : 0;
    const bool use = __shfl_sync(kAll, mine, 0) >= 0;
    float d[NV];
#pragma unroll
    for (int j = 0; j < NV; j++) d[j] = 0.f;
    if (use) {
      const uint8_t* row = P.x + t * P.ld;
      float x[NV], max = -FLT_MAX, s = 0.f;
#pragma unroll
      for (int j = 0; j < NV; j++) {
        const uint32_t e = lane + 32 * j;
        x[j] = e < E ? element<F32>(row, e) : __int_as_float(0xFF800000);
        max = fmaxf(max, x[j]);
      }
#pragma unroll
      for (int i = 16; i; i >>= 1) max = fmaxf(max, __shfl_xor_sync(kAll, max, i));
#pragma unroll
      for (int j = 0; j < NV; j++) {
        x[j] = ex2((x[j] - max) * kLog2e);
        s += x[j];
      }
      const float inv = 1.f / warp_sum(s);
      const float gw = P.gw && lane < P.k ? P.gw[t * P.gw_stride + lane * P.gw_choice] : 0.f;
      const float pm = lane < P.k ? ex2((element<F32>(row, (uint32_t)mine) - max) * kLog2e) * inv : 0.f;
      float dot = 0.f;   // sum of p dL/dp
#pragma unroll
      for (int j = 0; j < NV; j++) {
        const uint32_t e = lane + 32 * j;
        x[j] *= inv;
        d[j] = e < E ? unit * P.counts[e] : 0.f;
        dot = fmaf(x[j], d[j], dot);
      }
      float add;         // what the choice adds to its logit
      if (P.normalize) {
        const float w = pm / warp_sum(pm);
        add = w * (gw - warp_sum(w * gw));
      } else {
        add = pm * gw;
        dot += add;
      }
      dot = warp_sum(dot);
#pragma unroll
      for (int j = 0; j < NV; j++) d[j] = x[j] * (d[j] - dot);
      for (uint32_t i = 0; i < P.k; i++) {
        const uint32_t e = (uint32_t)__shfl_sync(kAll, mine, i);
        const float a = __shfl_sync(kAll, add, i);
#pragma unroll
        for (int j = 0; j < NV; j++)
          if (e == lane + 32 * j) d[j] += a;
      }
    }
    __syncwarp();   // (the row is read: its gradient may take its place)
#pragma unroll
    for (int j = 0; j < NV; j++) {
      const uint32_t e = lane + 32 * j;
      if (e >= E) continue;
      if (F32) reinterpret_cast<float*>(out)[e] = d[j];
      else reinterpret_cast<uint16_t*>(out)[e] = (uint16_t)pack_bf16(d[j], 0.f);
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
// the smallest of 1, 2, 4, ... 32 experts a lane
template <bool F32, class A, class F>
int by_experts(uint32_t experts, const F& f) {
  const uint32_t nv = (experts + 31) / 32;
  return nv <= 1 ? f(std::integral_constant<int, 1>()) : nv <= 2 ? f(std::integral_constant<int, 2>())
       : nv <= 4 ? f(std::integral_constant<int, 4>()) : nv <= 8 ? f(std::integral_constant<int, 8>())
       : nv <= 16 ? f(std::integral_constant<int, 16>()) : f(std::integral_constant<int, 32>());
}
template <bool F32>
int route(const RouteArgs& P, uint32_t grid, cudaStream_t s) {
  return by_experts<F32, RouteArgs>(P.experts, [&](auto nv) {
    return check(launch(k_route<F32, decltype(nv)::value>, dim3(grid), kThreads,
                        P.experts * (1 + kWarps) * 4, 1, s, P));
  });
}
template <bool F32>
int route_grad(const RouteGradArgs& P, uint32_t grid, cudaStream_t s) {
  return by_experts<F32, RouteGradArgs>(P.experts, [&](auto nv) {
    return check(launch(k_route_grad<F32, decltype(nv)::value>, dim3(grid), kThreads, 0, 1, s, P));
  });
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
  RouteArgs P;
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
  const uint32_t want = (tokens + kWarps - 1) / kWarps;
  const uint32_t grid = std::max(1u, std::min({want, (uint32_t)sms * 2, kMaxBlocks}));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (const int rc = dtype == BO_FP32 ? route<true>(P, grid, s) : route<false>(P, grid, s)) return rc;
  return check(launch(k_route_join, dim3(1), kJoinThreads, 0, 1, s, (const float*)P.sums,
                      (const int32_t*)P.counts, (const int32_t*)P.real, grid, h->experts, h->k,
                      h->d_probs, h->d_counts, h->d_loss, h->d_real));
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
  RouteGradArgs P;
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
  const uint32_t want = (tokens + kWarps - 1) / kWarps;
  const uint32_t grid = std::min(want, (uint32_t)sms * 8);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return dtype == BO_FP32 ? route_grad<true>(P, grid, s) : route_grad<false>(P, grid, s);
}

}  // extern "C"
