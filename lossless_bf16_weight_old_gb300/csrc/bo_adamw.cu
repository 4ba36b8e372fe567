// bo_adamw.cu -- AdamW over many tensors at once, with 32-bit or 8-bit moments, and the global
// gradient norm (include/ops/bf16ops.h has the formulas and the layout of the state).
//
// One table entry per 2048 elements carries everything a block needs, so a launch covers any
// number of tensors and a block's work is one 48-byte load away.  The step moves 28 bytes per
// element (BF16 gradients, FP32 master, 32-bit moments; 16 with 8-bit moments), the norm 2.  HBM
// bounds all but the step with 8-bit moments, which arithmetic bounds.  Measured rates stand at
// the kernels, beside the 6.77 TB/s of a copy.
#include <cmath>
#include <cstring>
#include <memory>
#include <new>
#include <vector>

#include "bo_internal.cuh"

namespace bo {
namespace {

constexpr uint32_t kThreads = 256;
constexpr uint32_t kChunkElems = 2048;   // eight elements a thread; eight 8-bit blocks
constexpr uint32_t kMaxGrid = 152 * 8;   // most blocks of the norm (its partial sums)
constexpr uint64_t kGamma = 0x9E3779B97F4A7C15ull;

struct alignas(16) Chunk {
  const void* w;    // weights of the chunk's first element (nullptr with a master)
  void* out;
  const void* g;
  uint64_t e0;      // its element in the arenas
  float wd;
  uint32_t count;   // elements, at most kChunkElems
  uint64_t pad;
};
static_assert(sizeof(Chunk) == 48, "three 16-byte words");

__device__ __forceinline__ Chunk load_chunk(const Chunk* p) {
  Chunk c;
  const uint4* s = reinterpret_cast<const uint4*>(p);
  uint4* d = reinterpret_cast<uint4*>(&c);
  d[0] = __ldg(s);
  d[1] = __ldg(s + 1);
  d[2] = __ldg(s + 2);
  return c;
}

// ------------------------------------------------------------------------------- the table
struct alignas(16) DevItem {
  const uint8_t* w;
  uint8_t* out;
  const uint8_t* g;
  uint64_t n;
  uint64_t first_block;
  uint64_t chunk0;   // chunks before this item
  float wd;
  uint32_t pad;
  uint64_t pad2;
};
static_assert(sizeof(DevItem) % 16 == 0, "uploaded in 16-byte words");

__global__ void k_build_chunks(const DevItem* __restrict__ items, uint32_t k, uint64_t chunks,
                               Chunk* __restrict__ table, uint32_t wsize, uint32_t gsize,
                               uint32_t osize) {
  const uint64_t c = (uint64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (c >= chunks) return;
  uint32_t lo = 0, hi = k;   // the last item whose chunk0 <= c
  while (hi - lo > 1) {
    const uint32_t mid = (lo + hi) / 2;
    if (items[mid].chunk0 <= c) lo = mid; else hi = mid;
  }
  const DevItem it = items[lo];
  const uint64_t at = (c - it.chunk0) * kChunkElems;
  Chunk ch;
  ch.w = it.w ? it.w + at * wsize : nullptr;
  ch.out = it.out + at * osize;
  ch.g = it.g + at * gsize;
  ch.e0 = it.first_block * BO_BLOCK_ELEMS + at;
  ch.wd = it.wd;
  const uint64_t left = it.n - at;
  ch.count = left < kChunkElems ? (uint32_t)left : kChunkElems;
  ch.pad = 0;
  table[c] = ch;
}

__global__ void k_init_control(bo_adamw_control* ctl, int64_t step) {
  ctl->step = step;
  ctl->norm = 0.f;
  ctl->coef = 1.f;
  ctl->status = BD_OK;
  ctl->ticket[0] = ctl->ticket[1] = ctl->ticket[2] = 0;
}

// ------------------------------------------------------------------- eight elements of a kind
template <bool F32>
__device__ __forceinline__ void load8(const void* p, uint32_t i, float (&x)[8]) {
  if (F32) {
    const uint4 a = ld16(static_cast<const float*>(p) + i);
    const uint4 b = ld16(static_cast<const float*>(p) + i + 4);
    x[0] = __uint_as_float(a.x); x[1] = __uint_as_float(a.y);
    x[2] = __uint_as_float(a.z); x[3] = __uint_as_float(a.w);
    x[4] = __uint_as_float(b.x); x[5] = __uint_as_float(b.y);
    x[6] = __uint_as_float(b.z); x[7] = __uint_as_float(b.w);
  } else {
    const uint4 a = ld16(static_cast<const uint16_t*>(p) + i);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int j = 0; j < 4; j++) {
      x[2 * j] = bf16_lo(w[j]);
      x[2 * j + 1] = bf16_hi(w[j]);
    }
  }
}
template <bool F32>
__device__ __forceinline__ float load1(const void* p, uint32_t i) {
  return F32 ? static_cast<const float*>(p)[i]
             : __uint_as_float((uint32_t) static_cast<const uint16_t*>(p)[i] << 16);
}

// ------------------------------------------------------------------------------ random bits
__device__ __forceinline__ uint64_t mix64(uint64_t z) {   // SplitMix64 (Steele, Lea & Flood 2014)
  z = (z ^ (z >> 30)) * 0xBF58476D1CE4E5B9ull;
  z = (z ^ (z >> 27)) * 0x94D049BB133111EBull;
  return z ^ (z >> 31);
}
// the 32 bits of each of the N elements from e0 on (both even)
template <int N>
__device__ __forceinline__ void noise(uint64_t key, uint64_t e0, uint32_t (&r)[N]) {
  uint64_t z = key + ((e0 >> 1) + 1) * kGamma;
#pragma unroll
  for (int j = 0; j < N / 2; j++) {
    const uint64_t h = mix64(z);
    r[2 * j] = (uint32_t)h;
    r[2 * j + 1] = (uint32_t)(h >> 32);
    z += kGamma;
  }
}
// BF16 bits of x in the upper half: away from zero when the cut-off part plus 16 random bits
// carries.  (Of a NaN the carry may reach the sign: see nan_of.)
__device__ __forceinline__ uint32_t bf16_carry(float x, uint32_t r) {
  return __float_as_uint(x) + (r & 0xFFFFu);
}
__device__ __forceinline__ uint32_t bf16_stochastic(float x, uint32_t r) {
  return isnan(x) ? 0x7FFFu : bf16_carry(x, r) >> 16;
}
// NaN if one of them is not finite, else 0: one instruction each
template <int N>
__device__ __forceinline__ float nan_of(const float (&p)[N]) {
  float s = 0.f;
#pragma unroll
  for (int j = 0; j < N; j++) s = fmaf(p[j], 0.f, s);
  return s;
}

// ----------------------------------------------------------------------------- the formula
constexpr float kTinyEps = 0x1p-39f;   // below it the root is taken of denormal numbers too

struct Rates {      // per launch
  float b1, c1, b2, c2;      // beta and 1 - beta
  float inv_bc1, inv_bc2;    // 1 / (1 - beta^t)
  float lr, eps, coef;
  float rate;                // -lr / (1 - beta1^t)
};

struct StepParams {
  const Chunk* table;
  uint64_t chunks;
  bo_adamw_state st;
  bo_adamw_control* ctl;
  const float* d_lr;
  float lr, b1, c1, b2, c2, log_b1, log_b2, eps;
  uint32_t clip;
  uint32_t stochastic;
  uint64_t seed;
};

// Reads what the step depends on, once per block; false: the step is skipped.  The step count
// is written only after every block has passed here (finish_step).
__device__ __forceinline__ bool begin_step(const StepParams& P, Rates& R, uint64_t& key) {
  __shared__ float sh[4];
  __shared__ unsigned long long sh_key;
  if (threadIdx.x == 0) {
    const int64_t t = *reinterpret_cast<volatile int64_t*>(&P.ctl->step) + 1;
    // 1 - beta^t without cancellation (beta = 0: log is -inf and the factor 1)
    sh[0] = 1.f / -expm1f((float)t * P.log_b1);
    sh[1] = 1.f / -expm1f((float)t * P.log_b2);
    sh[2] = P.d_lr ? *P.d_lr : P.lr;
    float coef = 1.f;
    if (P.clip) {
      const float norm = P.ctl->norm;
      coef = isfinite(norm) ? P.ctl->coef : -1.f;
    }
    sh[3] = coef;
    sh_key = mix64(P.seed ^ ((uint64_t)t * kGamma));
  }
  __syncthreads();
  R.b1 = P.b1; R.c1 = P.c1; R.b2 = P.b2; R.c2 = P.c2; R.eps = P.eps;
  R.inv_bc1 = sh[0];
  R.inv_bc2 = sh[1];
  R.lr = sh[2];
  R.coef = sh[3];
  R.rate = -(R.lr * sh[0]);
  key = sh_key;
  return sh[3] >= 0.f;
}

// The last block to finish counts the step.
__device__ __forceinline__ void finish_step(const StepParams& P, bool taken) {
  __syncthreads();
  if (threadIdx.x == 0) {
    if (atomicInc(&P.ctl->ticket[1], gridDim.x - 1) == gridDim.x - 1) {
      if (taken) P.ctl->step = P.ctl->step + 1;
      P.ctl->status = taken ? BD_OK : BO_SKIPPED_NONFINITE;
    }
  }
}

// Within 2^-22 or so of the root and the reciprocal; denormal numbers count as 0.
__device__ __forceinline__ float sqrt_fast(float x) {
  float r;
  asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float sqrt_full(float x) {   // ... and the root of denormal numbers
  float r;
  asm("sqrt.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float rsqrt_fast(float x) {
  float r;
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float rcp_fast(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// m / (sqrt(v) + eps), v with its bias correction.  The root and the quotient are the hardware's
// approximations, a few units in the last place of a term that lr scales down before it meets p.
// TINY: eps is so small that a v below 2^-126 counts (its root is below 2^-63, and beside a larger
// eps nothing).  The ratio of two small moments is the step then: an element with a gradient of
// 1e-20 moves as far as one with 1.  Where the denominator is 0, v having underflowed, nothing is
// known of the ratio, and it counts as 0.  (A denormal denominator, of a denormal eps, counts as
// 2^-126.)
template <bool TINY>
__device__ __forceinline__ float quotient(float m, float v, float eps) {
  if (!TINY) return m * rcp_fast(sqrt_fast(v) + eps);
  const float den = sqrt_full(v) + eps, q = m * rcp_fast(fmaxf(den, 0x1p-126f));
  return den == 0.f ? 0.f : q;
}

// One element: updates m, v and p.  (For any eps: HBM bounds the step that this is for.)
__device__ __forceinline__ void update(const Rates& R, float keep, float g, float& m, float& v,
                                       float& p) {
  g *= R.coef;
  m = fmaf(R.b1, m, R.c1 * g);
  v = fmaf(R.b2, v, R.c2 * g * g);
  p = fmaf(p, keep, R.rate * quotient<true>(m, v * R.inv_bc2, R.eps));
}

// BF16 words of weights p, rounded to nearest or by the random bits
template <int N>
__device__ __forceinline__ void weight_words(const float (&p)[N], bool stochastic,
                                             const uint32_t (&r)[N], uint32_t* w) {
#pragma unroll
  for (int j = 0; j < N / 2; j++)
    w[j] = stochastic ? __byte_perm(bf16_carry(p[2 * j], r[2 * j]),
                                    bf16_carry(p[2 * j + 1], r[2 * j + 1]), 0x7632)
                      : pack_bf16(p[2 * j], p[2 * j + 1]);
  if (stochastic && isnan(nan_of(p))) {
#pragma unroll
    for (int j = 0; j < N / 2; j++)
      w[j] = bf16_stochastic(p[2 * j], r[2 * j]) | bf16_stochastic(p[2 * j + 1], r[2 * j + 1]) << 16;
  }
}
// Eight new weights from p: the FP32 ones, or the master and the words of its rounding, or the
// words alone.
template <int WK>
__device__ __forceinline__ void store_weights(const Chunk& c, uint32_t i, float* master,
                                              const float (&p)[8], const uint32_t (&w)[4]) {
  if (WK == BO_WEIGHT_FP32) {
    float4* o = reinterpret_cast<float4*>(static_cast<float*>(c.out) + i);
    o[0] = make_float4(p[0], p[1], p[2], p[3]);
    o[1] = make_float4(p[4], p[5], p[6], p[7]);
    return;
  }
  if (WK == BO_WEIGHT_MASTER) {
    Float8 q;
#pragma unroll
    for (int j = 0; j < 8; j++) q.v[j] = p[j];
    st8(master, q);
  }
  *reinterpret_cast<uint4*>(static_cast<uint16_t*>(c.out) + i) = make_uint4(w[0], w[1], w[2], w[3]);
}
template <int WK>
__device__ __forceinline__ void store_weight1(const Chunk& c, uint32_t i, float* master, float p,
                                              bool stochastic, uint32_t r) {
  if (WK == BO_WEIGHT_FP32) {
    static_cast<float*>(c.out)[i] = p;
    return;
  }
  if (WK == BO_WEIGHT_MASTER) *master = p;
  static_cast<uint16_t*>(c.out)[i] =
      (uint16_t)((WK == BO_WEIGHT_BF16 && stochastic) ? bf16_stochastic(p, r)
                                                       : pack_bf16(p, 0.f) & 0xFFFFu);
}

// ------------------------------------------------------------------------ 32-bit moments
template <int WK, bool GF32>
struct Eight {   // a thread's elements
  float g[8], p[8];
  Float8 m, v;
  __device__ __forceinline__ void load(const StepParams& P, const Chunk& c, uint32_t i) {
    const uint64_t e = c.e0 + i;
    load8<GF32>(c.g, i, g);
    m = ld8(static_cast<float*>(P.st.d_m) + e);
    v = ld8(static_cast<float*>(P.st.d_v) + e);
    if (WK == BO_WEIGHT_MASTER) {
      const Float8 q = ld8(P.st.d_master + e);
#pragma unroll
      for (int j = 0; j < 8; j++) p[j] = q.v[j];
    } else {
      load8<WK == BO_WEIGHT_FP32>(c.w, i, p);
    }
  }
};

// Eight elements a thread, all loads of a chunk in flight at once: 625M elements (BF16 gradients,
// FP32 master) in 2542 us, 6.9 TB/s; the smallest step, fourteen tensors, 4.2 us a call.  The
// moments and p are rounded to FP32 once an operation, a BF16 weight once from FP32.
template <int WK, bool GF32>
__global__ void __launch_bounds__(kThreads, 4) k_step32(const StepParams P) {
  after_previous();
  Rates R;
  uint64_t key;
  // Backwards after a norm: it has left the last gradients in L2.
  const Chunk* const table = P.clip ? P.table + P.chunks - 1 : P.table;
  const int64_t dir = P.clip ? -1 : 1;
  const uint32_t i = threadIdx.x * 8;
  Chunk next;
  next.count = 0;
  if (blockIdx.x < P.chunks) next = load_chunk(table + dir * (int64_t)blockIdx.x);
  // the first elements are on their way while the rates are worked out
  Eight<WK, GF32> x;
  bool loaded = i + 8 <= next.count;
  if (loaded) x.load(P, next, i);
  const bool taken = begin_step(P, R, key);
  if (taken) {
    float* const am = static_cast<float*>(P.st.d_m);
    float* const av = static_cast<float*>(P.st.d_v);
    for (uint64_t ci = blockIdx.x; ci < P.chunks; ci += gridDim.x) {
      const Chunk c = next;
      if (ci + gridDim.x < P.chunks)
        next = load_chunk(table + dir * (int64_t)(ci + gridDim.x));
      const float keep = 1.f - R.lr * c.wd;
      const uint64_t e = c.e0 + i;
      float* const pm = WK == BO_WEIGHT_MASTER ? P.st.d_master + e : nullptr;
      if (i + 8 <= c.count) {
        if (!loaded) x.load(P, c, i);
        loaded = false;
#pragma unroll
        for (int j = 0; j < 8; j++) update(R, keep, x.g[j], x.m.v[j], x.v.v[j], x.p[j]);
        st8(am + e, x.m);
        st8(av + e, x.v);
        uint32_t r[8] = {}, w[4] = {};
        if (WK == BO_WEIGHT_BF16 && P.stochastic) noise(key, e, r);
        if (WK != BO_WEIGHT_FP32)
          weight_words(x.p, WK == BO_WEIGHT_BF16 && P.stochastic, r, w);
        store_weights<WK>(c, i, pm, x.p, w);
      } else if (i < c.count) {   // a tensor's last elements
        uint32_t r[8] = {};
        if (WK == BO_WEIGHT_BF16 && P.stochastic) noise(key, e, r);
#pragma unroll
        for (uint32_t j = 0; j < 8; j++) {
          if (i + j >= c.count) break;
          const float g = load1<GF32>(c.g, i + j);
          float m = am[e + j], v = av[e + j];
          float p = WK == BO_WEIGHT_MASTER ? pm[j] : load1<WK == BO_WEIGHT_FP32>(c.w, i + j);
          update(R, keep, g, m, v, p);
          am[e + j] = m;
          av[e + j] = v;
          store_weight1<WK>(c, i + j, pm + (WK == BO_WEIGHT_MASTER ? j : 0), p, P.stochastic, r[j]);
        }
      }
    }
  }
  finish_step(P, taken);
}

// ------------------------------------------------------------------------- 8-bit moments
// Here arithmetic counts as much as HBM: about eighty instructions an element, a tenth of them for
// the random bits, against the eighty-five that 16 bytes an element leave time for.  So additions,
// products and their sums are taken two elements at a time (the packed FP32 instructions).
//
// A code feeds the next step, so where a moment lies next to the bound between two codes, the last
// bit of its arithmetic decides between states that differ by a whole code.  Everything between
// the old code and the new one is therefore the correctly rounded FP32 operation, one for each
// operation of the formula and in its order: a step has one right result.
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
__device__ __forceinline__ float2 add2(float2 a, float2 b) { return __fadd2_rn(a, b); }
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }

// Integers and floats meet in the low bits of a float near a power of two: the converting
// instructions run at an eighth of the rate of an addition, and there would be five an element.
// Bytes j and j + 1, by 2^-8, and as signed numbers (w80 = w ^ 0x80808080), by 2^-7:
__device__ __forceinline__ float2 bytes_u(uint32_t w, uint32_t j) {
  return add2(make_float2(__uint_as_float(__byte_perm(w, 0x47000000u, 0x7650 | j)),
                          __uint_as_float(__byte_perm(w, 0x47000000u, 0x7651 | j))),
              both(-32768.f));
}
__device__ __forceinline__ float2 bytes_s(uint32_t w80, uint32_t j) {
  return add2(make_float2(__uint_as_float(__byte_perm(w80, 0x47800000u, 0x7650 | j)),
                          __uint_as_float(__byte_perm(w80, 0x47800000u, 0x7651 | j))),
              both(-65537.f));
}
__device__ __forceinline__ float max_nan(float a, float b) {   // NaN if either is
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float warp_max(float x) {
  float r;
  asm("redux.sync.max.NaN.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
  return r;
}
// An infinite scale would read as infinity or NaN by the code: NaN throughout marks the block.
__device__ __forceinline__ float finite_or_nan(float x) {
  return isfinite(x) ? x : __int_as_float(0x7FFFFFFF);
}
// 1 / scale; a scale next to the ends of the FP32 range comes with a power of two `pre` that
// brings it and its block's values into the middle.
__device__ __forceinline__ float inverse_scale(float scale, float& pre) {
  pre = scale < 0x1p-100f ? 0x1p80f : scale > 0x1p100f ? 0x1p-80f : 1.f;
  return scale > 0.f ? 1.f / (scale * pre) : 0.f;   // (under a NaN scale every code reads NaN)
}
// A code's value is m: (c |c| / 127^2) scale and v: (c / 255)^4 scale; the codes come divided by
// 128 and 256, which the factors make good without another rounding.
constexpr float kMUnit = (1.f / 16129.f) * 16384.f;
constexpr float kVUnit = (1.f / 255.f) * 256.f;
__device__ __forceinline__ float2 m_values(float2 c) {
  return mul2(make_float2(c.x * fabsf(c.x), c.y * fabsf(c.y)), both(kMUnit));
}
__device__ __forceinline__ float2 v_values(float2 c) {
  const float2 y = mul2(c, both(kVUnit)), y2 = mul2(y, y);
  return mul2(y2, y2);
}
// (The compiler joins a packed product and a packed sum into one operation with one rounding.)
__device__ __forceinline__ float2 sum2(float2 a, float2 b) {
  return make_float2(__fadd_rn(a.x, b.x), __fadd_rn(a.y, b.y));
}
// Two elements' update (the formula of `update`; the moments as said above).
template <bool TINY>
__device__ __forceinline__ void update2(const Rates& R, float keep, float2 g, float2& m, float2& v,
                                        float2& p) {
  g = mul2(g, both(R.coef));
  m = sum2(mul2(m, both(R.b1)), mul2(g, both(R.c1)));
  v = sum2(mul2(v, both(R.b2)), mul2(mul2(g, g), both(R.c2)));
  const float2 t = mul2(v, both(R.inv_bc2));
  float2 q;
  if (TINY) {
    q = make_float2(quotient<true>(m.x, t.x, R.eps), quotient<true>(m.y, t.y, R.eps));
  } else {
    const float2 den = add2(make_float2(sqrt_fast(t.x), sqrt_fast(t.y)), both(R.eps));
    q = mul2(m, make_float2(rcp_fast(den.x), rcp_fast(den.y)));
  }
  p = fma2(p, both(keep), mul2(both(R.rate), q));
}
// x / scale, rounded once: the product with the (correctly rounded) reciprocal, put right by its
// remainder, which one fused operation gives exactly (P. Markstein, "Computation of elementary
// functions on the IBM RISC System/6000 processor", 1990; the root in m_codes likewise)
__device__ __forceinline__ float2 ratio2(float2 x, float scale, float inv) {
  const float2 q = mul2(x, both(inv));
  return fma2(fma2(q, both(-scale), x), both(inv), q);
}
// the codes in the low bytes
__device__ __forceinline__ float2 m_codes(float2 m, float scale, float inv) {
  const float2 q = ratio2(m, scale, inv);
  const float2 x = make_float2(fmaxf(fabsf(q.x), 0x1p-100f), fmaxf(fabsf(q.y), 0x1p-100f));
  // the root, rounded once: x / sqrt(x), put right by its remainder
  const float2 h = make_float2(rsqrt_fast(x.x), rsqrt_fast(x.y)), y = mul2(x, h);
  const float2 e = fma2(mul2(y, both(-1.f)), y, x);
  const float2 r = mul2(fma2(e, mul2(h, both(0.5f)), y), both(127.f));
  return add2(make_float2(copysignf(r.x, m.x), copysignf(r.y, m.y)), both(12582912.f));
}
// Of the two codes whose values enclose v / scale, the upper one with the chance that makes the
// expected value v / scale; never 0 for v > 0 (a root of 0 under a moment that is not 0 is a
// step of m / eps).
__device__ __forceinline__ float2 v_codes(float2 v, float scale, float inv, uint32_t r0, uint32_t r1) {
  const float2 x = ratio2(v, scale, inv);
  // floor of 255 times x's fourth root, by rounding down at 2^23, where the code stays in the low
  // byte.  (One more or less next to a whole number makes the same code: its chance is 1 or 0.)
  float2 at = __ffma2_rd(make_float2(sqrt_fast(sqrt_fast(x.x)), sqrt_fast(sqrt_fast(x.y))), both(255.f),
                         both(8388608.f));
  at = make_float2(fminf(at.x, 8388862.f), fminf(at.y, 8388862.f));
  const float2 up = add2(at, both(1.f)), low = add2(at, both(-8388608.f));
  const float2 ya = mul2(low, both(1.f / 255.f)), yb = mul2(add2(low, both(1.f)), both(1.f / 255.f));
  const float2 a2 = mul2(ya, ya), b2 = mul2(yb, yb), a = mul2(a2, a2), b = mul2(b2, b2);
  const float2 u = add2(make_float2(__uint_as_float(0x3F800000u | (r0 >> 16) << 7),
                                    __uint_as_float(0x3F800000u | (r1 >> 16) << 7)),
                        both(-1.f));
  // u (upper - lower) < v / scale - lower
  const float2 l = mul2(u, fma2(a, both(-1.f), b)), h = fma2(a, both(-1.f), x);
  return make_float2(fmaxf(l.x < h.x ? up.x : at.x, v.x > 0.f ? 8388609.f : 8388608.f),
                     fmaxf(l.y < h.y ? up.y : at.y, v.y > 0.f ? 8388609.f : 8388608.f));
}
// the low bytes of four
__device__ __forceinline__ uint32_t low_bytes(float2 a, float2 b) {
  return __byte_perm(__byte_perm(__float_as_uint(a.x), __float_as_uint(a.y), 0x0040),
                     __byte_perm(__float_as_uint(b.x), __float_as_uint(b.y), 0x0040), 0x5410);
}

// One warp per block of 256: its eight elements a lane stay in registers while the block's
// maxima are found, so each byte is read and written once.  202M elements (BF16 gradients, FP32
// master) take 605 us, 5.3 TB/s: 85 instructions an element keep the FP32 pipes busy, and HBM is
// not the bound.  Four blocks an SM at 64 registers: three have room for more and take 775 us.
// Fetching the next chunk ahead through shared memory does not help either (711 us, of BF16
// weights 134 us for 40M elements with and without).
template <int WK, bool GF32>
__global__ void __launch_bounds__(kThreads, 4) k_step8(const StepParams P) {
  after_previous();
  Rates R;
  uint64_t key;
  // Backwards after a norm: it has left the last gradients in L2.
  const Chunk* const table = P.clip ? P.table + P.chunks - 1 : P.table;
  const int64_t dir = P.clip ? -1 : 1;
  const bool taken = begin_step(P, R, key);
  if (taken) {
    uint8_t* const am = static_cast<uint8_t*>(P.st.d_m);
    uint8_t* const av = static_cast<uint8_t*>(P.st.d_v);
    const uint32_t lane = threadIdx.x & 31;
    for (uint64_t ci = blockIdx.x; ci < P.chunks; ci += gridDim.x) {
      const Chunk c = load_chunk(table + dir * (int64_t)ci);   // (no registers for the one after)
      const uint32_t i = threadIdx.x * 8;
      if ((threadIdx.x & ~31u) * 8 >= c.count) continue;   // (the whole warp)
      const float keep = 1.f - R.lr * c.wd;
      const uint64_t e = c.e0 + i, blk = e / BO_BLOCK_ELEMS;
      float* const pm = WK == BO_WEIGHT_MASTER ? P.st.d_master + e : nullptr;
      const uint32_t cnt = c.count > i ? min(c.count - i, 8u) : 0u;
      float g[8] = {}, p[8] = {};
      uint2 cm = *reinterpret_cast<const uint2*>(am + e);
      cm = make_uint2(cm.x ^ 0x80808080u, cm.y ^ 0x80808080u);
      const uint2 cv = *reinterpret_cast<const uint2*>(av + e);
      const float sm = P.st.d_m_scale[blk], sv = P.st.d_v_scale[blk];
      if (cnt == 8) {
        load8<GF32>(c.g, i, g);
        if (WK == BO_WEIGHT_MASTER) {
          const Float8 q = ld8(pm);
#pragma unroll
          for (int j = 0; j < 8; j++) p[j] = q.v[j];
        } else {
          load8<WK == BO_WEIGHT_FP32>(c.w, i, p);
        }
      } else {
#pragma unroll
        for (uint32_t j = 0; j < 8; j++)
          if (j < cnt) {
            g[j] = load1<GF32>(c.g, i + j);
            p[j] = WK == BO_WEIGHT_MASTER ? pm[j] : load1<WK == BO_WEIGHT_FP32>(c.w, i + j);
          }
      }
      float2 m[4], v[4];
      float mm = 0.f, mv = 0.f;
#pragma unroll
      for (uint32_t j = 0; j < 4; j++) {
        m[j] = mul2(m_values(bytes_s(j < 2 ? cm.x : cm.y, 2 * j & 3)), both(sm));
        v[j] = mul2(v_values(bytes_u(j < 2 ? cv.x : cv.y, 2 * j & 3)), both(sv));
        float2 q = make_float2(p[2 * j], p[2 * j + 1]);
        const float2 gj = make_float2(g[2 * j], g[2 * j + 1]);
        if (P.eps < kTinyEps) update2<true>(R, keep, gj, m[j], v[j], q);
        else update2<false>(R, keep, gj, m[j], v[j], q);
        p[2 * j] = q.x;
        p[2 * j + 1] = q.y;
      }
      if (cnt < 8) {   // padding behind the tensor's end
#pragma unroll
        for (uint32_t j = 0; j < 4; j++) {
          if (2 * j >= cnt) m[j].x = v[j].x = 0.f;
          if (2 * j + 1 >= cnt) m[j].y = v[j].y = 0.f;
        }
      }
#pragma unroll
      for (uint32_t j = 0; j < 4; j++) {
        mm = max_nan(max_nan(mm, fabsf(m[j].x)), fabsf(m[j].y));
        mv = max_nan(max_nan(mv, v[j].x), v[j].y);
      }
      mm = finite_or_nan(warp_max(mm));
      mv = finite_or_nan(warp_max(mv));
      float mpre, vpre;
      const float minv = inverse_scale(mm, mpre), vinv = inverse_scale(mv, vpre);
      if (mpre != 1.f || vpre != 1.f) {
#pragma unroll
        for (uint32_t j = 0; j < 4; j++) {
          m[j] = mul2(m[j], both(mpre));
          v[j] = mul2(v[j], both(vpre));
        }
      }
      uint32_t r[8], w[4] = {};
      noise(key, e, r);
      float2 a[4], b[4];
#pragma unroll
      for (uint32_t j = 0; j < 4; j++) {
        a[j] = m_codes(m[j], mm * mpre, minv);
        b[j] = v_codes(v[j], mv * vpre, vinv, r[2 * j], r[2 * j + 1]);
      }
      *reinterpret_cast<uint2*>(am + e) = make_uint2(low_bytes(a[0], a[1]), low_bytes(a[2], a[3]));
      *reinterpret_cast<uint2*>(av + e) = make_uint2(low_bytes(b[0], b[1]), low_bytes(b[2], b[3]));
      if (lane == 0) {
        P.st.d_m_scale[blk] = mm;
        P.st.d_v_scale[blk] = mv;
      }
      if (cnt == 8) {
        if (WK != BO_WEIGHT_FP32)
          weight_words(p, WK == BO_WEIGHT_BF16 && P.stochastic, r, w);
        store_weights<WK>(c, i, pm, p, w);
      } else {
#pragma unroll
        for (uint32_t j = 0; j < 8; j++)
          if (j < cnt)
            store_weight1<WK>(c, i + j, pm + (WK == BO_WEIGHT_MASTER ? j : 0), p[j], P.stochastic,
                              r[j]);
      }
    }
  }
  finish_step(P, taken);
}

// Codes to values, one lane per eight elements of the arenas; either output may be missing.
template <bool F32>
__device__ __forceinline__ void put8(void* out, uint64_t t, const float (&x)[8]) {
  if (F32) {
    float4* o = static_cast<float4*>(out) + 2 * t;
    o[0] = make_float4(x[0], x[1], x[2], x[3]);
    o[1] = make_float4(x[4], x[5], x[6], x[7]);
  } else {
    static_cast<uint4*>(out)[t] = make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]),
                                             pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
  }
}
// 6 bytes an element with BF16 values: 202M elements in 190 us, 6.4 TB/s.
template <bool F32>
__global__ void __launch_bounds__(kThreads) k_moments(const bo_adamw_state st,
                                                       void* __restrict__ out_m,
                                                       void* __restrict__ out_v) {
  after_previous();
  const uint64_t stride = (uint64_t)gridDim.x * blockDim.x;
  for (uint64_t t = (uint64_t)blockIdx.x * blockDim.x + threadIdx.x; t < st.blocks * 32;
       t += stride) {
    float x[8];
    if (out_m) {
      const uint2 c = static_cast<const uint2*>(st.d_m)[t];
      const float s = st.d_m_scale[t >> 5];
#pragma unroll
      for (int j = 0; j < 8; j += 2) {
        const float2 y = mul2(m_values(bytes_s((j < 4 ? c.x : c.y) ^ 0x80808080u, j & 3)), both(s));
        x[j] = y.x;
        x[j + 1] = y.y;
      }
      put8<F32>(out_m, t, x);
    }
    if (out_v) {
      const uint2 c = static_cast<const uint2*>(st.d_v)[t];
      const float s = st.d_v_scale[t >> 5];
#pragma unroll
      for (int j = 0; j < 8; j += 2) {
        // fewer roundings than the step's: (c / 256)^2 is exact
        const float2 a = bytes_u(j < 4 ? c.x : c.y, j & 3), b = mul2(a, a);
        const float2 y = mul2(mul2(mul2(b, b), both(4294967296.f / 4228250625.f)), both(s));
        x[j] = y.x;
        x[j + 1] = y.y;
      }
      put8<F32>(out_v, t, x);
    }
  }
}

// --------------------------------------------------------------------------- gradient norm
// Sums in a fixed order: eight FP32 sums a thread over its elements, joined in FP64 over the
// block, and the blocks' sums by the last block to finish.  202M BF16 gradients in 74 us, 5.5 TB/s
// (reads alone, and the join at the end; with twice the blocks it is slower).
template <bool GF32>
__global__ void __launch_bounds__(kThreads, 8) k_norm(const Chunk* __restrict__ table,
                                                      uint64_t chunks, double* __restrict__ part,
                                                      bo_adamw_control* ctl, float max_norm) {
  after_previous();
  float s[8] = {};
  if (blockIdx.x < chunks) {
    Chunk next = load_chunk(table + blockIdx.x);
    for (uint64_t ci = blockIdx.x; ci < chunks; ci += gridDim.x) {
      const Chunk c = next;
      if (ci + gridDim.x < chunks) next = load_chunk(table + ci + gridDim.x);
      const uint32_t i = threadIdx.x * 8;
      if (i + 8 <= c.count) {
        float g[8];
        load8<GF32>(c.g, i, g);
#pragma unroll
        for (int j = 0; j < 8; j++) s[j] = fmaf(g[j], g[j], s[j]);
      } else {
        for (uint32_t j = i; j < c.count; j++) {
          const float g = load1<GF32>(c.g, j);
          s[0] = fmaf(g, g, s[0]);
        }
      }
    }
  }
  __shared__ double sh[kThreads];
  __shared__ bool last;
  sh[threadIdx.x] = (double)(((s[0] + s[1]) + (s[2] + s[3])) + ((s[4] + s[5]) + (s[6] + s[7])));
  __syncthreads();
  for (uint32_t d = kThreads / 2; d; d >>= 1) {
    if (threadIdx.x < d) sh[threadIdx.x] += sh[threadIdx.x + d];
    __syncthreads();
  }
  if (threadIdx.x == 0) {
    part[blockIdx.x] = sh[0];
    __threadfence();
    last = atomicInc(&ctl->ticket[0], gridDim.x - 1) == gridDim.x - 1;
  }
  __syncthreads();
  if (!last) return;
  __threadfence();
  double t = 0;
  for (uint32_t b = threadIdx.x; b < gridDim.x; b += kThreads) t += __ldcg(part + b);
  sh[threadIdx.x] = t;
  __syncthreads();
  for (uint32_t d = kThreads / 2; d; d >>= 1) {
    if (threadIdx.x < d) sh[threadIdx.x] += sh[threadIdx.x + d];
    __syncthreads();
  }
  if (threadIdx.x == 0) {
    const float norm = (float)sqrt(sh[0]);
    ctl->norm = norm;
    ctl->coef = max_norm > 0.f ? fminf(1.f, max_norm / (norm + 1e-6f)) : 1.f;
  }
}

// ------------------------------------------------------------------------------- host side
struct PlanLayout {
  uint64_t control, partials, items, table, total, chunks;
};

bool plan_layout(const bo_adamw_item* items, uint32_t k, PlanLayout& L) {
  if (k > 0 && !items) return false;
  L.chunks = 0;
  for (uint32_t i = 0; i < k; i++) {
    if (items[i].n > BD_MAX_ELEMS) return false;
    L.chunks += (items[i].n + kChunkElems - 1) / kChunkElems;
  }
  if (L.chunks > (1ull << 36)) return false;
  L.control = 0;
  L.partials = up(sizeof(bo_adamw_control), 256);
  L.items = L.partials + up((uint64_t)kMaxGrid * sizeof(double), 256);
  L.table = L.items + up((uint64_t)k * sizeof(DevItem), 256);
  L.total = L.table + up(L.chunks * sizeof(Chunk), 256);
  return true;
}

bool valid(const bo_adamw* h) {
  return h && h->d_control && h->d_chunks && h->d_partials && h->weight_kind <= BO_WEIGHT_FP32 &&
         h->grad_dtype <= BO_FP32 && (h->state_bits == 8 || h->state_bits == 32);
}

int launch_norm(const bo_adamw* h, float max_norm, int sms, cudaStream_t s) {
  const uint64_t want = h->chunks < 1 ? 1 : h->chunks;
  const uint32_t most = (uint32_t)sms * 8 < kMaxGrid ? (uint32_t)sms * 8 : kMaxGrid;
  const uint32_t grid = (uint32_t)(want < most ? want : most);
  const Chunk* table = static_cast<const Chunk*>(h->d_chunks);
  return check(launch(h->grad_dtype == BO_FP32 ? k_norm<true> : k_norm<false>, dim3(grid), kThreads,
                      0, 1, s, table, h->chunks, h->d_partials, h->d_control, max_norm));
}

template <int WK, bool GF32>
cudaError_t launch_step(bool bits8, uint32_t grid, const StepParams& P, cudaStream_t s) {
  return launch(bits8 ? k_step8<WK, GF32> : k_step32<WK, GF32>, dim3(grid), kThreads, 0, 1, s, P);
}

}  // namespace

constexpr uint32_t kBlobWords = 30 * 1024 / 16;
struct Blob {
  uint32_t words;
  uint32_t pad[3];
  uint4 data[kBlobWords];
};
static_assert(sizeof(Blob) <= 32000, "kernel parameter limit");

__global__ void k_put(const __grid_constant__ Blob b, uint4* __restrict__ dst) {
  const uint32_t i = blockIdx.x * blockDim.x + threadIdx.x;
  if (i < b.words) dst[i] = b.data[i];
}

cudaError_t upload(const void* host, uint64_t bytes, void* dst, cudaStream_t s) {
  const uint64_t words = bytes / 16;
  std::unique_ptr<Blob> b(new (std::nothrow) Blob);
  if (!b) return cudaErrorMemoryAllocation;
  for (uint64_t w0 = 0; w0 < words; w0 += kBlobWords) {
    const uint32_t cnt = (uint32_t)(words - w0 < kBlobWords ? words - w0 : kBlobWords);
    b->words = cnt;
    std::memcpy(b->data, static_cast<const uint8_t*>(host) + w0 * 16, (size_t)cnt * 16);
    k_put<<<(cnt + 127) / 128, 128, 0, s>>>(*b, static_cast<uint4*>(dst) + w0);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace bo

using namespace bo;

extern "C" {

uint64_t bo_adamw_plan_size(const bo_adamw_item* h_items, uint32_t k) {
  PlanLayout L;
  return plan_layout(h_items, k, L) ? L.total : 0;
}

int bo_adamw_plan(const bo_adamw_item* h_items, uint32_t k, const bo_adamw_state* state,
                  uint32_t weight_kind, uint32_t grad_dtype, uint32_t state_bits, uint32_t flags,
                  int64_t step, void* d_plan, uint64_t plan_bytes, bo_adamw* h_out,
                  void* stream) {
  PlanLayout L;
  if (!state || !h_out || !plan_layout(h_items, k, L)) return BD_ERR_INVALID_ARG;
  if (weight_kind > BO_WEIGHT_FP32 || grad_dtype > BO_FP32 || (state_bits != 8 && state_bits != 32) ||
      (flags & ~BO_ADAMW_STOCHASTIC) || step < 0)
    return BD_ERR_INVALID_ARG;
  if ((flags & BO_ADAMW_STOCHASTIC) && weight_kind != BO_WEIGHT_BF16) return BD_ERR_INVALID_ARG;
  if (!d_plan || !aligned(d_plan, 256) || plan_bytes < L.total) return BD_ERR_INVALID_ARG;
  const bool master = weight_kind == BO_WEIGHT_MASTER;
  if (state->blocks > BD_MAX_ELEMS / BO_BLOCK_ELEMS) return BD_ERR_INVALID_ARG;
  if (state->blocks > 0) {
    if (!state->d_m || !state->d_v || !aligned(state->d_m, 256) || !aligned(state->d_v, 256) ||
        (master && (!state->d_master || !aligned(state->d_master, 256))) ||
        (state_bits == 8 && (!state->d_m_scale || !state->d_v_scale ||
                             !aligned(state->d_m_scale, 256) || !aligned(state->d_v_scale, 256))))
      return BD_ERR_INVALID_ARG;
  }
  const uint64_t wsize = weight_kind == BO_WEIGHT_FP32 ? 4 : 2, gsize = grad_dtype == BO_FP32 ? 4 : 2;
  const uint64_t elems = state->blocks * BO_BLOCK_ELEMS, msize = state_bits == 8 ? 1 : 4;
  std::unique_ptr<DevItem[]> dev(new (std::nothrow) DevItem[k ? k : 1]);
  std::unique_ptr<Span[]> memory(new (std::nothrow) Span[3 * (size_t)k + 6]);
  std::unique_ptr<Span[]> arena(new (std::nothrow) Span[(size_t)k + 1]);
  if (!dev || !memory || !arena) return BD_ERR_INVALID_ARG;
  size_t spans = 0;
  auto uses = [&](const void* p, uint64_t bytes, bool write) {
    const uint64_t at = reinterpret_cast<uintptr_t>(p);
    memory[spans++] = Span{at, at + bytes, write};
  };
  uses(d_plan, L.total, true);
  uses(state->d_m, elems * msize, true);
  uses(state->d_v, elems * msize, true);
  if (state_bits == 8) {
    uses(state->d_m_scale, state->blocks * 4, true);
    uses(state->d_v_scale, state->blocks * 4, true);
  }
  if (master) uses(state->d_master, elems * 4, true);
  uint64_t chunk0 = 0;
  for (uint32_t i = 0; i < k; i++) {
    const bo_adamw_item& it = h_items[i];
    const uint64_t blocks = (it.n + BO_BLOCK_ELEMS - 1) / BO_BLOCK_ELEMS;
    if (it.reserved != 0 || it.first_block > state->blocks ||
        blocks > state->blocks - it.first_block)
      return BD_ERR_INVALID_ARG;
    arena[i] = Span{it.first_block, it.first_block + blocks, true};
    if (it.n > 0) {
      if (!it.d_out || !it.d_grad || !aligned(it.d_out, 16) || !aligned(it.d_grad, 16))
        return BD_ERR_INVALID_ARG;
      if (!master && (!it.d_weight || !aligned(it.d_weight, 16))) return BD_ERR_INVALID_ARG;
      uses(it.d_out, it.n * wsize, true);
      uses(it.d_grad, it.n * gsize, false);
      if (!master && it.d_weight != it.d_out) uses(it.d_weight, it.n * wsize, false);
    }
    DevItem& d = dev[i];
    std::memset(&d, 0, sizeof(d));
    d.w = master ? nullptr : static_cast<const uint8_t*>(it.d_weight);
    d.out = static_cast<uint8_t*>(it.d_out);
    d.g = static_cast<const uint8_t*>(it.d_grad);
    d.n = it.n;
    d.first_block = it.first_block;
    d.chunk0 = chunk0;
    d.wd = it.weight_decay;
    chunk0 += (it.n + kChunkElems - 1) / kChunkElems;
  }
  if (!disjoint(memory.get(), spans) || !disjoint(arena.get(), k)) return BD_ERR_INVALID_ARG;
  uint8_t* p = static_cast<uint8_t*>(d_plan);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  bo_adamw h;
  std::memset(&h, 0, sizeof(h));
  h.state = *state;
  h.d_control = reinterpret_cast<bo_adamw_control*>(p + L.control);
  h.d_partials = reinterpret_cast<double*>(p + L.partials);
  h.d_chunks = p + L.table;
  h.chunks = L.chunks;
  h.weight_kind = weight_kind;
  h.grad_dtype = grad_dtype;
  h.state_bits = state_bits;
  h.flags = flags;
  int rc;
  if ((rc = check(cudaGetDevice(&h.device)))) return rc;
  k_init_control<<<1, 1, 0, s>>>(h.d_control, step);
  if ((rc = check(cudaGetLastError()))) return rc;
  if (L.chunks > 0) {
    if ((rc = check(upload(dev.get(), (uint64_t)k * sizeof(DevItem), p + L.items, s)))) return rc;
    k_build_chunks<<<(uint32_t)((L.chunks + 255) / 256), 256, 0, s>>>(
        reinterpret_cast<const DevItem*>(p + L.items), k, L.chunks,
        reinterpret_cast<Chunk*>(p + L.table), (uint32_t)wsize, (uint32_t)gsize, (uint32_t)wsize);
    if ((rc = check(cudaGetLastError()))) return rc;
  }
  *h_out = h;
  return BD_OK;
}

int bo_adamw_norm(const bo_adamw* h, float max_norm, void* stream) {
  if (!valid(h) || !(max_norm >= 0.f)) return BD_ERR_INVALID_ARG;
  int sms = 0;
  if (const int rc = sm_count(h->device, sms)) return rc;
  return launch_norm(h, max_norm, sms, static_cast<cudaStream_t>(stream));
}

int bo_adamw_step(const bo_adamw* h, const bo_adamw_step_args* a, void* stream) {
  if (!valid(h) || !a) return BD_ERR_INVALID_ARG;
  if (!(a->beta1 >= 0 && a->beta1 < 1 && a->beta2 >= 0 && a->beta2 < 1) || !(a->eps >= 0.f) ||
      !(a->max_norm >= 0.f) || (a->d_lr && !aligned(a->d_lr, 4)) ||
      (!a->d_lr && !std::isfinite(a->lr)))
    return BD_ERR_INVALID_ARG;
  int sms = 0;
  if (const int rc = sm_count(h->device, sms)) return rc;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (a->max_norm > 0.f) {
    const int rc = launch_norm(h, a->max_norm, sms, s);
    if (rc) return rc;
  }
  StepParams P;
  P.table = static_cast<const Chunk*>(h->d_chunks);
  P.chunks = h->chunks;
  P.st = h->state;
  P.ctl = h->d_control;
  P.d_lr = a->d_lr;
  P.lr = a->lr;
  P.b1 = (float)a->beta1;
  P.c1 = (float)(1.0 - a->beta1);
  P.b2 = (float)a->beta2;
  P.c2 = (float)(1.0 - a->beta2);
  P.log_b1 = (float)std::log(a->beta1);
  P.log_b2 = (float)std::log(a->beta2);
  P.eps = a->eps;
  P.clip = a->max_norm > 0.f;
  P.stochastic = (h->flags & BO_ADAMW_STOCHASTIC) != 0;
  P.seed = a->seed;
  const uint64_t want = h->chunks < 1 ? 1 : h->chunks;
  const bool b8 = h->state_bits == 8;
  // A block of the 32-bit step takes a few chunks only: blocks that start in order keep the arenas'
  // pages open (625M parameters: 2.75 ms with 4 blocks an SM taking all chunks in turn, 2.54 ms
  // with 64; 8-bit moments, which arithmetic bounds, do not care).
  const uint32_t most = (uint32_t)sms * (b8 ? 4 : 64);
  const uint32_t grid = (uint32_t)(want < most ? want : most);
  cudaError_t e;
  switch (h->weight_kind * 2 + h->grad_dtype) {
    case BO_WEIGHT_MASTER * 2 + BO_BF16: e = launch_step<BO_WEIGHT_MASTER, false>(b8, grid, P, s); break;
    case BO_WEIGHT_MASTER * 2 + BO_FP32: e = launch_step<BO_WEIGHT_MASTER, true>(b8, grid, P, s); break;
    case BO_WEIGHT_BF16 * 2 + BO_BF16: e = launch_step<BO_WEIGHT_BF16, false>(b8, grid, P, s); break;
    case BO_WEIGHT_BF16 * 2 + BO_FP32: e = launch_step<BO_WEIGHT_BF16, true>(b8, grid, P, s); break;
    case BO_WEIGHT_FP32 * 2 + BO_BF16: e = launch_step<BO_WEIGHT_FP32, false>(b8, grid, P, s); break;
    default: e = launch_step<BO_WEIGHT_FP32, true>(b8, grid, P, s); break;
  }
  return check(e);
}

int bo_adamw_moments(const bo_adamw* h, uint32_t dtype, void* d_m, void* d_v, void* stream) {
  if (!valid(h) || h->state_bits != 8 || dtype > BO_FP32 || !aligned(d_m, 16) || !aligned(d_v, 16))
    return BD_ERR_INVALID_ARG;
  int sms = 0;
  if (const int rc = sm_count(h->device, sms)) return rc;
  const uint64_t blocks = h->state.blocks;
  if (blocks == 0) return BD_OK;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const uint64_t want = (blocks * 32 + kThreads - 1) / kThreads;
  const uint32_t grid = (uint32_t)(want < (uint64_t)sms * 8 ? want : (uint64_t)sms * 8);
  return check(launch(dtype == BO_FP32 ? k_moments<true> : k_moments<false>, dim3(grid), kThreads, 0,
                      1, s, h->state, d_m, d_v));
}

const char* bo_status_string(int code) {
  switch (code) {
    case BD_OK: return "ok";
    case BD_ERR_INVALID_ARG: return "invalid argument";
    case BD_ERR_CUDA: return "CUDA error";
    case BO_SKIPPED_NONFINITE: return "step skipped: the gradient norm is not finite";
    default: return "unknown status";
  }
}

}  // extern "C"
