// bo_logprobs.cu -- log probabilities of given tokens with entropy and top alternatives, and the
// logits' gradient (include/ops/bf16ops.h has the formulas).
//
// A row is read once, in windows of 64 bytes that are aligned whatever the row's own alignment is:
// the first and the last may lie partly outside the row, and are read by the element.  HBM bounds both
// passes where there are many rows; measured rates stand at the kernels, beside the 6.77 TB/s of a copy.
#include <cfloat>
#include <cmath>
#include <type_traits>
#include <cooperative_groups.h>

#include "bo_internal.cuh"

namespace bo {
namespace {

namespace cg = cooperative_groups;


constexpr uint32_t kThreads = 256;
constexpr uint32_t kMaxLogCluster = 3;
constexpr uint32_t kWindow = 64;                 // bytes
constexpr uint32_t kSegment = 8192;              // windows whose maxima are kept at once
constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;

// What the backward pass takes from the forward one, of each row.
struct alignas(32) Saved {
  float shift;      // p_j = 2^(x_j scale - shift) / sum, or, with `careful`, 2^((x_j - shift) / T log2 e) / sum
  float sum;
  float log2_sum;
  float entropy;
  float inv_t;      // 1 / T; NaN for a row without a valid token or temperature
  int32_t token;    // -1: the gradient is 0
  int32_t careful;
  float temp;       // T; NaN as inv_t is
};
static_assert(sizeof(Saved) == 32, "one sector");

struct ScoreArgs {
  const uint8_t* x;
  uint64_t ld;            // bytes
  const uint8_t* tokens;
  uint64_t token_stride;  // bytes
  const float* temps;     // may be NULL
  uint64_t temp_stride;   // elements
  float temp;
  uint32_t token_bytes, rows, vocab, top, log_cluster;
  float* logprobs;
  float* entropy;
  float* top_logprobs;
  int32_t* top_tokens;
  Saved* saved;
};

struct GradArgs {
  const uint8_t* x;
  uint64_t ld;            // bytes
  uint8_t* dx;
  uint64_t ld_dx;         // bytes
  const float* g;
  uint64_t g_stride;
  const float* h;
  uint64_t h_stride;
  uint32_t rows, vocab, pieces;
  const Saved* saved;
};

__device__ __forceinline__ float ex2(float x) {   // 2^x, 0 below 2^-126
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ void ld32(uint32_t (&w)[8], const void* p) {
  asm volatile("ld.global.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]),
                 "=r"(w[7])
               : "l"(p)
               : "memory");
}
__device__ __forceinline__ void st32(void* p, const uint32_t (&w)[8]) {
  asm volatile("st.global.L1::no_allocate.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(w[0]),
               "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}
// (x - max) / T for any of them, as two products: (x - max) 2^n by one fused operation, and with 1 / (T 2^n).
// The power keeps both in FP32's range: T may be so small that 1 / T is not, or a difference so large that it
// is not by itself.  (A small T gets none where max is 2^60 or more, and a 1 / T of 1e38 at most, whose product
// with log2 e is finite: there x is max, or 2^37 and more below it.)
struct OverT {
  float pow, from, inv;
  __device__ __forceinline__ OverT(float p, float f, float i) : pow(p), from(f), inv(i) {}
  __device__ __forceinline__ OverT(float max, float t) {
    pow = t > 0x1p64f ? 0x1p-64f : t < 0x1p-64f && fabsf(max) < 0x1p60f ? 0x1p64f : 1.f;
    from = max * pow;
    inv = 1.f / (t * pow);
    if (inv > 1e38f) inv = 1e38f;
  }
  __device__ __forceinline__ float far(float x) const { return fmaf(x, pow, -from); }
  __device__ __forceinline__ float operator()(float x) const { return far(x) * inv; }
};
template <bool F32>
__device__ __forceinline__ float element(const uint8_t* p) {
  return F32 ? *reinterpret_cast<const float*>(p)
             : __uint_as_float((uint32_t) * reinterpret_cast<const uint16_t*>(p) << 16);
}

// A key orders values and, of equal ones, places (the lowest first); 0 is below every key.
typedef unsigned long long Key;
__device__ __forceinline__ uint32_t order_of(float x) {
  if (x != x) return 0xFFFFFFFFu;
  const uint32_t u = __float_as_uint(x + 0.f);   // (-0 is 0)
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t o) {
  return __uint_as_float(o & 0x80000000u ? o & 0x7FFFFFFFu : ~o);
}
__device__ __forceinline__ Key key_of(uint32_t order, uint32_t place) {
  return (Key)order << 32 | (uint32_t)~place;
}
__device__ __forceinline__ uint32_t place_of(Key k) { return ~(uint32_t)k; }


// The windows of a row.
template <bool F32>
struct Windows {
  static constexpr uint32_t kSize = F32 ? 4 : 2, kElems = kWindow / kSize;
  const uint8_t* row;
  const uint8_t* base;   // of the first window
  uint32_t off, count;   // elements of the first window that lie before the row; windows
  uint32_t vocab;
  __device__ __forceinline__ Windows(const uint8_t* r, uint32_t v) : row(r), vocab(v) {
    const uint32_t skip = (uint32_t)(reinterpret_cast<uintptr_t>(r) & (kWindow - 1));
    base = r - skip;
    off = skip / kSize;
    count = (uint32_t)(((uint64_t)off + v + kElems - 1) / kElems);
  }
  // the row's element that begins window w (negative or past its end: outside)
  __device__ __forceinline__ int32_t first(uint32_t w) const { return (int32_t)(w * kElems) - (int32_t)off; }
  __device__ __forceinline__ bool whole(uint32_t w) const {
    return first(w) >= 0 && first(w) + kElems <= vocab;
  }
  // The lane's element of a window (any of the row's where it lies outside), without a branch, so that
  // several are under way at once; and its key, 0 outside the row.
  __device__ __forceinline__ float lane_value(uint32_t w, uint32_t lane) const {
    const int32_t e = min(max(first(w) + (int32_t)lane, 0), (int32_t)vocab - 1);
    return element<F32>(row + (int64_t)e * kSize);
  }
  __device__ __forceinline__ Key lane_key(float x, uint32_t w, uint32_t lane) const {
    const int32_t e = first(w) + (int32_t)lane;
    return lane < kElems && e >= 0 && e < (int32_t)vocab ? key_of(order_of(x), (uint32_t)e) : 0;
  }
  // the words of a window that is not whole; -infinity outside the row
  __device__ __forceinline__ void load_edge(uint32_t w, uint32_t (&lo)[8], uint32_t (&hi)[8]) const {
    const int32_t e0 = first(w);
#pragma unroll
    for (int i = 0; i < 16; i++) {
      uint32_t v;
      if (F32) {
        const int32_t e = e0 + i;
        v = e >= 0 && e < (int32_t)vocab ? __float_as_uint(element<true>(row + (int64_t)e * 4)) : 0xFF800000u;
      } else {
        const int32_t e = e0 + 2 * i;
        const uint16_t* p = reinterpret_cast<const uint16_t*>(row);
        v = e >= 0 && e < (int32_t)vocab ? p[e] : 0xFF80u;
        v |= (e + 1 >= 0 && e + 1 < (int32_t)vocab ? (uint32_t)p[e + 1] : 0xFF80u) << 16;
      }
      if (i < 8) lo[i] = v; else hi[i - 8] = v;
    }
  }
};

// has the L2 fetch whole windows of [begin, end), 256 KB of them at most
template <bool F32>
__device__ __forceinline__ void ahead(const Windows<F32>& W, uint32_t begin, uint32_t end) {
  if (begin < end && !W.whole(begin)) begin++;
  if (begin < end && !W.whole(end - 1)) end--;
  end = min(end, begin + 4096);
  if (begin < end)
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(W.base + (uint64_t)begin * kWindow),
                 "r"((end - begin) * kWindow)
                 : "memory");
}

// ---------------------------------------------------------------------------- online softmax
// Of the values so far: their maximum; `shift`, its product with the scale; the sum of e = 2^d over
// d = x scale - shift, and the sum of e d, in four parts each.  So d is one fused operation with one
// rounding, whose d of the maximum is the rounding of the shift.  That holds while the shift stays between
// -2^21 and 2^22 (kLeast, kMost): the rows whose maximum does not are read again (careful_sums).  The
// shift starts below all of them, so that -infinity has e = 0; its d is kept finite, so that e d is 0 and
// not NaN.  The floor that does so has to be far below the maximum at any scale and its product with the
// scale finite: rows of scales outside kLeastScale (with entropy, which alone has the floor) and kMostScale
// are read again too, and of maxima that differences from could pass FP32's range.
constexpr float kLeast = -2097152.f, kMost = 4194304.f;
constexpr uint32_t kFloorBf16 = 0xF149F149u;   // -1e30, twice
constexpr float kFloor = -1e30f, kLeastScale = 1e-23f, kMostScale = 1e8f;

struct Joined {
  float max, shift, s, t;
  // Those of all lanes: the greatest shift, then sums of the same scale.
  __device__ __forceinline__ void join_warp() {
    float to = shift;
    asm("redux.sync.max.f32 %0, %0, 0xffffffff;" : "+f"(max));
    asm("redux.sync.max.f32 %0, %0, 0xffffffff;" : "+f"(to));
    const float d = shift - to, f = d == 0.f ? 1.f : ex2(d);
    t = f * fmaf(s, d, t);
    s = f * s;
    shift = to;
#pragma unroll
    for (int i = 16; i; i >>= 1) {
      s += __shfl_xor_sync(0xffffffffu, s, i);
      t += __shfl_xor_sync(0xffffffffu, t, i);
    }
  }
};
__device__ __forceinline__ Joined nothing() {
  return Joined{-INFINITY, -kMost, 0.f, 0.f};
}
template <bool ENT>
struct Sums {
  float max = -INFINITY, shift = -kMost;
  float2 s[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
  float2 t[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};

  __device__ __forceinline__ void raise(float to, float scale) {   // (not called for a NaN)
    max = to;
    const float up = fminf(to * scale, kMost);
    if (!(up > shift)) return;
    const float d = shift - up, f = ex2(d);
    shift = up;
#pragma unroll
    for (int i = 0; i < 2; i++) {
      if (ENT) t[i] = make_float2(f * fmaf(s[i].x, d, t[i].x), f * fmaf(s[i].y, d, t[i].y));
      s[i] = make_float2(f * s[i].x, f * s[i].y);
    }
  }
  __device__ __forceinline__ void add(float2 x, float scale, int i) {
    const float2 d = __ffma2_rn(x, make_float2(scale, scale), make_float2(-shift, -shift));
    const float2 e = make_float2(ex2(d.x), ex2(d.y));
    s[i] = __fadd2_rn(s[i], e);
    if (ENT) t[i] = __ffma2_rn(e, d, t[i]);
  }
  __device__ __forceinline__ Joined joined() const {
    return Joined{max, shift, (s[0].x + s[0].y) + (s[1].x + s[1].y), (t[0].x + t[0].y) + (t[1].x + t[1].y)};
  }
};
template <bool F32>
__device__ __forceinline__ float window_max(const uint32_t (&lo)[8], const uint32_t (&hi)[8]) {
  if constexpr (F32) {
    float m[8];
#pragma unroll
    for (int i = 0; i < 8; i++) m[i] = max_nan(__uint_as_float(lo[i]), __uint_as_float(hi[i]));
#pragma unroll
    for (int n = 4; n; n >>= 1)
#pragma unroll
      for (int i = 0; i < n; i++) m[i] = max_nan(m[i], m[i + n]);
    return m[0];
  } else {
    uint32_t m[8];
#pragma unroll
    for (int i = 0; i < 8; i++) m[i] = max_bf16x2(lo[i], hi[i]);
#pragma unroll
    for (int n = 4; n; n >>= 1)
#pragma unroll
      for (int i = 0; i < n; i++) m[i] = max_bf16x2(m[i], m[i + n]);
    return max_nan(bf16_lo(m[0]), bf16_hi(m[0]));
  }
}
template <bool F32, bool ENT>
__device__ __forceinline__ void add_window(Sums<ENT>& a, const uint32_t (&lo)[8], const uint32_t (&hi)[8],
                                           float scale) {
#pragma unroll
  for (int i = 0; i < 8; i++) {
    if (F32) {
      const uint32_t* w = i < 4 ? lo : hi;
      const int j = 2 * (i & 3);
      float2 x = make_float2(__uint_as_float(w[j]), __uint_as_float(w[j + 1]));
      if (ENT) x = make_float2(max_nan(x.x, kFloor), max_nan(x.y, kFloor));
      a.add(x, scale, i & 1);
    } else {
      const uint32_t u = ENT ? max_bf16x2(lo[i], kFloorBf16) : lo[i], v = ENT ? max_bf16x2(hi[i], kFloorBf16) : hi[i];
      a.add(make_float2(bf16_lo(u), bf16_hi(u)), scale, 0);
      a.add(make_float2(bf16_lo(v), bf16_hi(v)), scale, 1);
    }
  }
}

// The sums of a whole row for any values and temperatures: d = (x - max) / T log2 e with the row's own maximum
// (OverT), kept above -200, where e is 0, so that e d is 0 and not NaN.  The maximum is taken as the lowest
// finite number at least: a row of -infinity has the sum 0.  For a block; every thread of warp 0 has the result.
template <uint32_t TH, bool F32>
__device__ __noinline__ Joined careful_sums(const Windows<F32>& W, float max, float temp, Joined* parts) {
  const uint32_t warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  max = fmaxf(max, -FLT_MAX);
  const OverT by(max, temp);
  const float scale = by.inv * kLog2e;
  float s = 0.f, t = 0.f;
  for (uint32_t e = threadIdx.x; e < W.vocab; e += TH) {
    const float x = element<F32>(W.row + (uint64_t)e * Windows<F32>::kSize);
    const float d = max_nan(by.far(x) * scale, -200.f), p = ex2(d);
    s += p;
    t = fmaf(p, d, t);
  }
#pragma unroll
  for (int d = 16; d; d >>= 1) {
    s += __shfl_xor_sync(0xffffffffu, s, d);
    t += __shfl_xor_sync(0xffffffffu, t, d);
  }
  if (lane == 0) parts[warp] = Joined{max, max, s, t};
  __syncthreads();
  s = lane < TH / 32 ? parts[lane].s : 0.f;
  t = lane < TH / 32 ? parts[lane].t : 0.f;
#pragma unroll
  for (int d = 16; d; d >>= 1) {
    s += __shfl_xor_sync(0xffffffffu, s, d);
    t += __shfl_xor_sync(0xffffffffu, t, d);
  }
  return Joined{max, max, s, t};
}

// ------------------------------------------------------------------------------- top tokens
__device__ __forceinline__ Key step(Key v, uint32_t stride, bool keep_max) {
  const Key o = __shfl_xor_sync(0xffffffffu, v, stride);
  return (v > o) == keep_max ? v : o;
}
// the lanes' keys in descending order
__device__ __forceinline__ Key sorted(Key v, uint32_t lane) {
#pragma unroll
  for (uint32_t size = 2; size <= 32; size *= 2)
#pragma unroll
    for (uint32_t stride = size / 2; stride; stride /= 2)
      v = step(v, stride, ((lane & stride) == 0) == ((lane & size) == 0));
  return v;
}
// the 32 greatest of two descending lists, in descending order; b reversed: lane 31 - i has its i-th
__device__ __forceinline__ Key merged_reversed(Key a, Key b, uint32_t lane) {
  Key v = a > b ? a : b;
#pragma unroll
  for (uint32_t stride = 16; stride; stride /= 2) v = step(v, stride, (lane & stride) == 0);
  return v;
}
__device__ __forceinline__ Key merged(Key a, Key b, uint32_t lane) {
  return merged_reversed(a, __shfl_sync(0xffffffffu, b, 31 - lane), lane);
}
// The warps' lists joined in lists[0].
template <uint32_t TH>
__device__ __forceinline__ void join_lists(Key mine, Key (*lists)[32], uint32_t warp, uint32_t lane) {
  lists[warp][lane] = mine;
  __syncthreads();
  for (uint32_t half = (TH / 32) / 2; half; half /= 2) {
    if (warp < half) {
      mine = merged_reversed(mine, lists[warp + half][31 - lane], lane);
      lists[warp][lane] = mine;
    }
    __syncthreads();
  }
}
// the same of the numbers that order values alone
__device__ __forceinline__ uint32_t step(uint32_t v, uint32_t stride, bool keep_max) {
  const uint32_t o = __shfl_xor_sync(0xffffffffu, v, stride);
  return keep_max ? max(v, o) : min(v, o);
}
__device__ __forceinline__ uint32_t sorted(uint32_t v, uint32_t lane) {
#pragma unroll
  for (uint32_t size = 2; size <= 32; size *= 2)
#pragma unroll
    for (uint32_t stride = size / 2; stride; stride /= 2)
      v = step(v, stride, ((lane & stride) == 0) == ((lane & size) == 0));
  return v;
}

// A window's maximum as it is kept: as the logits are.
template <bool F32>
using Max = typename std::conditional<F32, float, uint16_t>::type;
__device__ __forceinline__ void put_max(float* to, float m) { *to = m; }
__device__ __forceinline__ void put_max(uint16_t* to, float m) { *to = (uint16_t)(__float_as_uint(m) >> 16); }
__device__ __forceinline__ float max_value(float m) { return m; }
__device__ __forceinline__ float max_value(uint16_t m) { return __uint_as_float((uint32_t)m << 16); }

// Shared memory of the search for top tokens.
template <uint32_t TH>
struct TopSearch {
  static constexpr uint32_t kKeys = TH < 128 ? 128 : TH;          // that are sorted by their places at most
  static constexpr uint32_t kWindows = TH < 128 ? 4096 / TH : 32; // that a warp lists at most
  Key lists[TH / 32 + 1][32];     // the last one: of the segments so far
  uint32_t values[TH / 32][32];
  uint32_t windows[TH / 32][kWindows];
  Key keys[kKeys];
  uint32_t nkeys;
};
// Of a segment of windows [w0, w1) with their maxima in maxima[], its 32 greatest elements in T.lists[0],
// whatever values are alike.  The k greatest elements lie in the k windows with the greatest maxima (each
// of those that precede an element's window has one that precedes the element), and those windows are
// among the windows of the k threads with the greatest maxima.
template <uint32_t TH, bool F32>
__device__ __noinline__ void segment_top_of_alike(const Windows<F32>& W, uint32_t w0, uint32_t w1, uint32_t top,
                                                  const Max<F32>* maxima, TopSearch<TH>& T) {
  const uint32_t warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  Key best = 0, mine = 0;
  for (uint32_t w = w0 + threadIdx.x; w < w1; w += TH) best = max(best, key_of(order_of(max_value(maxima[w - w0])), w));
  join_lists<TH>(sorted(best, lane), T.lists, warp, lane);
  for (uint32_t i = warp; i < top; i += TH / 32) {
    const Key k = T.lists[0][i];
    if (!k) break;
    uint32_t w = w0 + (place_of(k) - w0) % TH + lane * TH;   // the thread's windows
    for (uint32_t n = 0; n < kSegment; n += 32 * TH, w += 32 * TH)
      mine = merged(mine, sorted(w < w1 ? key_of(order_of(max_value(maxima[w - w0])), w) : 0, lane), lane);
  }
  __syncthreads();
  join_lists<TH>(mine, T.lists, warp, lane);
  mine = 0;
  for (uint32_t i = warp; i < top; i += TH / 32) {
    const Key k = T.lists[0][i];
    if (!k) break;
    mine = merged(mine, sorted(W.lane_key(W.lane_value(place_of(k), lane), place_of(k), lane), lane), lane);
  }
  __syncthreads();
  join_lists<TH>(mine, T.lists, warp, lane);
}
// The same, much sooner where few values are alike.  best: the greatest maximum of this thread's windows.
// At least `top` elements are as great as the one of these that is the top-th of all threads' (the floor),
// so lesser ones do not count.  Each warp lists its windows with such elements, then their elements, and
// each of those goes to the place that the number of greater ones is.  (A floor from each warp by itself
// takes fewer steps and lets so many more through that one row took 1.3 us longer.)
template <uint32_t TH, bool F32>
__device__ __forceinline__ void segment_top(const Windows<F32>& W, uint32_t w0, uint32_t w1, uint32_t top, float best,
                                            const Max<F32>* maxima, TopSearch<TH>& T) {
  constexpr uint32_t kKeys = TopSearch<TH>::kKeys, kWindows = TopSearch<TH>::kWindows;
  const uint32_t warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const uint32_t best_order = threadIdx.x < w1 - w0 ? order_of(best) : 0;
  uint32_t v = sorted(best_order, lane);
  T.values[warp][lane] = v;
  if (warp == 0) T.lists[0][lane] = 0;
  if (threadIdx.x == 0) T.nkeys = 0;
  __syncthreads();   // (the maxima are there, too)
  for (uint32_t half = TH / 64; half; half /= 2) {
    if (warp < half) {
      v = max(v, T.values[warp + half][31 - lane]);
#pragma unroll
      for (uint32_t stride = 16; stride; stride /= 2) v = step(v, stride, (lane & stride) == 0);
      T.values[warp][lane] = v;
    }
    __syncthreads();
  }
  const uint32_t floor = T.values[0][top - 1];
  uint32_t nw = 0;
  const uint32_t threads = __ballot_sync(0xffffffffu, best_order >= floor && best_order > 0);
  if (threads) {
    const float least = value_of(floor);   // (NaN, which is only NaN's floor: then all are listed)
    auto look = [&](uint32_t w) {
      const bool in = w < w1 && !(max_value(maxima[min(w, w1 - 1) - w0]) < least);
      const uint32_t who = __ballot_sync(0xffffffffu, in);
      const uint32_t at = nw + __popc(who & ((1u << lane) - 1));
      if (in && at < kWindows) T.windows[warp][at] = w;
      nw += __popc(who);
    };
    // a step for each of the threads' windows, or for each such thread (1000 rows of 151936, top 5: 58 and 54
    // us; one row, top 20: 7.1 and 7.9)
    if (2 * __popc(threads) >= (w1 - w0) / TH) {
#pragma unroll 4
      for (uint32_t w = w0 + threadIdx.x; w - lane < w1; w += TH) look(w);
    } else {
      for (uint32_t left = threads; left; left &= left - 1)
        for (uint32_t first = w0 + warp * 32 + __ffs(left) - 1; first < w1; first += 32 * TH) look(first + lane * TH);
    }
    __syncwarp();
    constexpr uint32_t kAtOnce = 8;   // windows that are read at once
    const uint32_t listed = min(nw, kWindows);
    for (uint32_t i0 = 0; i0 < listed; i0 += kAtOnce) {
      float x[kAtOnce];
#pragma unroll
      for (uint32_t j = 0; j < kAtOnce; j++) x[j] = W.lane_value(T.windows[warp][min(i0 + j, listed - 1)], lane);
      uint32_t n = 0, at = 0;
      Key k[kAtOnce];
#pragma unroll
      for (uint32_t j = 0; j < kAtOnce; j++) {
        k[j] = i0 + j < listed ? W.lane_key(x[j], T.windows[warp][min(i0 + j, listed - 1)], lane) : 0;
        if ((uint32_t)(k[j] >> 32) < floor) k[j] = 0;
        n += k[j] != 0;
      }
      // (each lane's to places of its own)
      if (__any_sync(0xffffffffu, n > 0)) {
        if (n) at = atomicAdd(&T.nkeys, n);
#pragma unroll
        for (uint32_t j = 0; j < kAtOnce; j++)
          if (k[j]) {
            if (at < kKeys) T.keys[at] = k[j];
            at++;
          }
      }
    }
  }
  const bool fits = __syncthreads_and(nw <= kWindows);
  const uint32_t n = T.nkeys;
  if (fits && n <= kKeys) {
    for (uint32_t j = threadIdx.x; j < n; j += TH) {
      const Key k = T.keys[j];
      uint32_t greater = 0;
#pragma unroll 8
      for (uint32_t i = 0; i < n; i++) greater += T.keys[i] > k;
      if (greater < 32) T.lists[0][greater] = k;
    }
    __syncthreads();
    return;
  }
  __syncthreads();
  segment_top_of_alike<TH, F32>(W, w0, w1, top, maxima, T);
}

// ------------------------------------------------------------------------------ forward pass
// The blocks of a cluster share a row: each takes its part of the windows, and the first one joins
// their sums and lists.
//
// 8192 rows of 151936 BF16 logits with entropy take 354 to 360 us, 7.0 TB/s, at 4 instructions a logit (half of
// what the SMs issue).  Fetching windows ahead gains nothing, as other blocks read while one waits: by the
// L2 388 us against 365, into registers (and so with fewer blocks) 1639 rows of 32000 in 22.8 us against
// 21.8.  Those rows' 105 MB, at 4.6 TB/s, are as much as a launch of 23 us reads: PyTorch's maximum over as
// many bytes takes 25.
// The search for top tokens adds to each row some 2.5 us in which its block reads little: 4000 rows of
// 32000 take 45 us without, 61 with 20.  One row of 151936 with 20 takes 7.2 us (4.8 without): launch,
// token, logits, search, the cluster's meeting and the results are trips one after the other.
template <uint32_t TH, bool F32, bool ENT, bool TOP>
__global__ void __launch_bounds__(TH, (TOP || TH <= 128 ? 1024 : 1536) / TH) k_score(const ScoreArgs P) {
  extern __shared__ float dynamic[];
  Max<F32>* const maxima = reinterpret_cast<Max<F32>*>(dynamic);
  __shared__ TopSearch<TH> tops[1];
  constexpr uint32_t kBlocks = TH == 256 ? 1u << kMaxLogCluster : 1;   // of a cluster (of blocks of 256 threads)
  __shared__ Joined parts[TH / 32], sums[kBlocks];
  __shared__ Key keys[TOP ? kBlocks : 1][32];
  static_assert(sizeof(tops) + sizeof(parts) + sizeof(sums) + sizeof(keys) + kSegment * sizeof(float) <= kDefaultSmem,
                "no allowance");
  TopSearch<TH>& T = tops[0];
  after_previous();
  const cg::cluster_group cluster = cg::this_cluster();
  const uint32_t log_c = P.log_cluster, C = 1u << log_c, c = blockIdx.x & (C - 1);
  const uint32_t row = blockIdx.x >> log_c, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const Windows<F32> W(P.x + row * P.ld, P.vocab);
  const uint32_t begin = W.count * c >> log_c, end = W.count * (c + 1) >> log_c;   // (2^20 windows at most)
  if (C > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;");   // (before another block's memory is written)
  // (few rows: the L2 may as well have the block's part on its way while the token is looked up)
  if (C > 1 && threadIdx.x == 0) ahead(W, begin, end);
  const uint8_t* at = P.tokens + row * P.token_stride;
  const int64_t token = P.token_bytes == 8 ? *reinterpret_cast<const int64_t*>(at)
                                           : *reinterpret_cast<const int32_t*>(at);
  const float temp = P.temps ? P.temps[row * P.temp_stride] : P.temp;
  if (token < 0) {   // (the whole cluster)
    if (C > 1) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
    if (c == 0) {
      if (threadIdx.x == 0) {
        P.logprobs[row] = 0.f;
        if (P.entropy) P.entropy[row] = 0.f;
        P.saved[row].token = -1;
      }
      if (TOP && threadIdx.x < P.top) {
        P.top_logprobs[(uint64_t)row * P.top + threadIdx.x] = 0.f;
        P.top_tokens[(uint64_t)row * P.top + threadIdx.x] = -1;
      }
    }
    return;
  }
  const float inv_t = temp > 0.f && temp <= FLT_MAX ? 1.f / temp : __int_as_float(0x7FFFFFFF);   // (infinite below 2^-128)
  const float scale = inv_t * kLog2e;
  const bool valid = token < (int64_t)P.vocab;
  float given = 0.f;   // the token's logit, under way while the row is read
  if (c == 0 && warp == 0 && valid) given = element<F32>(W.row + token * Windows<F32>::kSize);

  Sums<ENT> a;
  if (TOP && warp == 0) T.lists[TH / 32][lane] = 0;
  // windows [begin, end) but for the first and last ones of the row, where they are not whole
  const uint32_t edge0 = W.whole(0) ? 0 : 1, edge1 = W.count > 1 && !W.whole(W.count - 1) ? W.count - 1 : W.count;
  for (uint32_t w0 = begin; w0 < end; w0 += kSegment) {
    const uint32_t w1 = TOP ? min(end, w0 + kSegment) : end;
    float best = -INFINITY;
    auto take = [&](uint32_t w, const uint32_t (&lo)[8], const uint32_t (&hi)[8]) {
      const float m = window_max<F32>(lo, hi);
      if (TOP) {
        put_max(maxima + (w - w0), m);
        best = max_nan(best, m);
      }
      if (m > a.max) a.raise(m, scale);
      add_window<F32, ENT>(a, lo, hi, scale);
    };
    // thread i takes the segment's windows i, i + TH, ...
#pragma unroll 1
    for (uint32_t i = 0; i < 2; i++) {
      const uint32_t edge = i ? edge1 : 0;
      if ((i ? edge < W.count : edge0 > 0) && edge >= w0 && edge < w1 && (edge - w0) % TH == threadIdx.x) {
        uint32_t lo[8], hi[8];
        W.load_edge(edge, lo, hi);
        take(edge, lo, hi);
      }
    }
    uint32_t w = w0 + threadIdx.x;
    if (w < edge0) w += TH;
    const uint32_t stop = min(w1, edge1);
#pragma unroll 1
    for (const uint8_t* p = W.base + (uint64_t)w * kWindow; w < stop; w += TH, p += TH * kWindow) {
      uint32_t lo[8], hi[8];
      ld32(lo, p);
      ld32(hi, p + 32);
      take(w, lo, hi);
    }
    if (!TOP) break;
    segment_top<TH, F32>(W, w0, w1, P.top, best, maxima, T);
    if (warp == 0) T.lists[TH / 32][lane] = w0 == begin ? T.lists[0][lane] : merged(T.lists[TH / 32][lane], T.lists[0][lane], lane);
    __syncthreads();
  }

  Joined j = a.joined();
  j.join_warp();
  if (lane == 0) parts[warp] = j;
  __syncthreads();
  // (every warp has the block's sums, and of the first block the cluster's)
  j = lane < TH / 32 ? parts[lane] : nothing();
  j.join_warp();
  if (C > 1) {   // each block leaves its sums and its list with the first one
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
    if (threadIdx.x == 0) *cluster.map_shared_rank(&sums[kBlocks > 1 ? c : 0], 0) = j;
    if (TOP && warp == 0) cluster.map_shared_rank(&keys[kBlocks > 1 ? c : 0][0], 0)[lane] = T.lists[TH / 32][lane];
    cluster.sync();
    if (c == 0) {
      j = lane < C ? sums[lane] : nothing();
      j.join_warp();
      if (TOP) join_lists<TH>(warp < C ? keys[warp][lane] : 0, T.lists, warp, lane);
    }
  }
  if (c == 0) {
    const float far = j.max * scale;
    const bool careful = !(far >= kLeast && far <= kMost && scale <= kMostScale && j.max <= -kFloor) ||
                         (ENT && !(scale >= kLeastScale));
    if (careful) {
      __syncthreads();   // (parts is read)
      j = careful_sums<TH, F32>(W, j.max, inv_t == inv_t ? temp : inv_t, parts);
    }
    if (warp == 0) {
      const bool empty = careful && j.s == 0.f;             // nothing but -infinity
      const float inf = __int_as_float(0x7F800000), nan = __int_as_float(0x7FFFFFFF);
      // The sum over the greatest term of it, whose own error then cancels: near 1 for a row with one
      // likely token, whose entropy and -lp are small.
      const float top_d = careful ? 0.f : fmaf(j.max, scale, -j.shift);
      const float log_sum = logf(j.s / (careful ? 1.f : ex2(top_d)));
      // (x - max) / T - ln sum e^((x - max) / T): no part is larger than the result, wherever the row lies.
      // (Multiplied by 1 / T: divided by T, which is half a step better, one row took 7.5 us, so 7.2.)
      // (One form for all rows: a second one in log_p left the loop over windows with more spills, 300 rows of
      // 151936 without entropy 12.2 us, so 11.6.)
      OverT by{1.f, j.max, inv_t};
      if (careful) by = OverT(j.max, inv_t == inv_t ? temp : inv_t);
      auto log_p = [&](float x) {
        if (empty) return -inf * inv_t;   // (NaN for a temperature that is none)
        return min_nan(by(x) - log_sum, 0.f);
      };
      if (lane == 0) {
        const float entropy = empty ? 0.f : max_nan(log_sum - kLn2 * (j.t / j.s - top_d), 0.f);
        P.logprobs[row] = valid ? log_p(given) : nan;
        if (ENT) P.entropy[row] = entropy;
        Saved sv = {};
        sv.shift = j.shift;
        sv.sum = j.s;
        sv.log2_sum = log2f(j.s);
        sv.entropy = entropy;
        sv.inv_t = valid ? inv_t : nan;
        sv.token = empty && valid && inv_t == inv_t ? -1 : (int32_t)(valid ? token : 0);
        sv.careful = careful;
        sv.temp = valid && inv_t == inv_t ? temp : nan;
        P.saved[row] = sv;
      }
      if (TOP && lane < P.top) {
        const Key k = T.lists[C > 1 ? 0 : TH / 32][lane];
        P.top_logprobs[(uint64_t)row * P.top + lane] = log_p(value_of((uint32_t)(k >> 32)));
        P.top_tokens[(uint64_t)row * P.top + lane] = (int32_t)place_of(k);
      }
    }
  }
}

// ----------------------------------------------------------------------------- backward pass
// dx_j = p_j (a + b log2 p_j) + [j = v] at, with p_j = 2^d / sum:  2^d (A + B d).
struct RowGrad {
  float scale, shift, A, B, at;
  bool careful, plain;   // plain: B is 0
  __device__ __forceinline__ RowGrad(const Saved& sv, float g, float h) {
    const float unit = sv.careful ? 1.f : sv.inv_t;   // (CarefulGrad divides by T at the end)
    const float a = -(h == 0.f ? g : g + h * sv.entropy) * unit, b = -h * kLn2 * unit, inv = 1.f / sv.sum;
    scale = sv.inv_t * kLog2e;
    shift = sv.shift;
    A = inv * (a - b * sv.log2_sum);
    B = inv * b;
    at = g * unit;
    careful = sv.careful;
    plain = h == 0.f;
  }
  // an element, and whether it is the given token, of a row that is not `careful`
  __device__ __forceinline__ float operator()(float x, bool given) const {
    const float d = max_nan(fmaf(x, scale, -shift), -200.f);
    return ex2(d) * fmaf(B, d, A) + (given ? at : 0.f);
  }
  template <bool PLAIN>
  __device__ __forceinline__ float2 two(float2 x) const {        // a row that is not `careful`
    float2 d = __ffma2_rn(x, make_float2(scale, scale), make_float2(-shift, -shift));
    if (PLAIN) return __fmul2_rn(make_float2(ex2(d.x), ex2(d.y)), make_float2(A, A));
    d = make_float2(max_nan(d.x, -200.f), max_nan(d.y, -200.f));
    return __fmul2_rn(make_float2(ex2(d.x), ex2(d.y)), __ffma2_rn(d, make_float2(B, B), make_float2(A, A)));
  }
};
// The same of a careful row.  1 / T is the last factor, in two products: by the least of T, parts of the sum
// would be infinite where it is 0.
struct CarefulGrad {
  const RowGrad& R;
  OverT by, end;
  __device__ __forceinline__ CarefulGrad(const RowGrad& r, float temp) : R(r), by(r.shift, temp), end(0.f, temp) {}
  __device__ __forceinline__ float operator()(float x, bool given) const {
    const float d = max_nan(by.far(x) * (by.inv * kLog2e), -200.f);
    return (ex2(d) * fmaf(R.B, d, R.A) + (given ? R.at : 0.f)) * end.inv * end.pow;
  }
};
template <bool F32, bool PLAIN>
__device__ __forceinline__ void grad_words(const RowGrad& R, uint32_t (&q)[8]) {
#pragma unroll
  for (int i = 0; i < (F32 ? 4 : 8); i++) {
    if (F32) {
      const float2 v = R.two<PLAIN>(make_float2(__uint_as_float(q[2 * i]), __uint_as_float(q[2 * i + 1])));
      q[2 * i] = __float_as_uint(v.x);
      q[2 * i + 1] = __float_as_uint(v.y);
    } else {
      const float2 v = R.two<PLAIN>(make_float2(bf16_lo(q[i]), bf16_hi(q[i])));
      q[i] = pack_bf16(v.x, v.y);
    }
  }
}
// One window a thread, read and written in words of 32 bytes.  4096 rows of 151936 BF16 logits with
// entropy take 348 us, 7.1 TB/s (HBM); 2048 rows of 32000, a quarter left out, 34.7 us, 6.6 TB/s; 333 odd
// FP32 rows of 32001 13.6 us, 6.0 TB/s.  Rows of the gradient that begin otherwise than the logits' take
// up to twice the time (4096 rows of 1000: 13.6 us, alike 7.2), careful ones three times.
template <bool F32>
__global__ void __launch_bounds__(kThreads) k_grad(const GradArgs P) {
  after_previous();
  const uint32_t row = blockIdx.x / P.pieces, piece = blockIdx.x % P.pieces;
  const Saved sv = P.saved[row];
  const float g = P.g ? P.g[row * P.g_stride] : 0.f, h = P.h ? P.h[row * P.h_stride] : 0.f;
  const Windows<F32> W(P.x + row * P.ld, P.vocab);
  uint8_t* out = P.dx + row * P.ld_dx;
  const bool zero = sv.token < 0 || (g == 0.f && h == 0.f);
  const RowGrad R(sv, g, h);
  constexpr uint32_t E = Windows<F32>::kElems, S = Windows<F32>::kSize;
  auto one = [&](int32_t e, const auto& value) {   // an element by itself
    if (e < 0 || e >= (int32_t)P.vocab) return;
    const float v = zero ? 0.f : value(element<F32>(W.row + (int64_t)e * S), e == sv.token);
    if (F32) reinterpret_cast<float*>(out)[e] = v;
    else reinterpret_cast<uint16_t*>(out)[e] = (uint16_t)pack_bf16(v, 0.f);
  };
  // Where the two rows begin differently within 32 bytes, or the row has to be worked out carefully:
  // elements side by side.
  const int32_t off = (int32_t)W.off * (int32_t)S;
  if ((reinterpret_cast<uintptr_t>(out - off) & 31) != 0 || (R.careful && !zero)) {
    const int32_t first = W.first(piece * kThreads) + (int32_t)threadIdx.x;
    if (R.careful) {
      const CarefulGrad careful(R, sv.temp);
#pragma unroll 4
      for (uint32_t i = 0; i < E; i++) one(first + (int32_t)(i * kThreads), careful);
    } else {
#pragma unroll 4
      for (uint32_t i = 0; i < E; i++) one(first + (int32_t)(i * kThreads), R);
    }
    return;
  }
  const uint32_t w = piece * kThreads + threadIdx.x, last = W.count - 1;
  if (w <= last && W.whole(w)) {
    const int32_t e0 = W.first(w);
    uint8_t* o = out + (int64_t)e0 * S;
    uint32_t lo[8], hi[8];
    const uint32_t v = (uint32_t)(sv.token - e0);   // the token's place, when below E
    float at = 0.f;
    if (zero) {
#pragma unroll
      for (int i = 0; i < 8; i++) lo[i] = hi[i] = 0;
    } else {
      const uint8_t* p = W.base + (uint64_t)w * kWindow;
      ld32(lo, p);
      ld32(hi, p + 32);
      if (v < E) at = R(element<F32>(W.row + (int64_t)sv.token * S), true);
      if (R.plain) grad_words<F32, true>(R, lo), grad_words<F32, true>(R, hi);
      else grad_words<F32, false>(R, lo), grad_words<F32, false>(R, hi);
    }
    st32(o, lo);
    st32(o + 32, hi);
    if (!zero && v < E) {
      if (F32) *reinterpret_cast<float*>(o + v * S) = at;
      else *reinterpret_cast<uint16_t*>(o + v * S) = (uint16_t)pack_bf16(at, 0.f);
    }
  }
  // the windows that are not whole: a warp each
  const uint32_t warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  if (lane < E) {
    if (warp == 0 && piece == 0 && !W.whole(0)) one(W.first(0) + (int32_t)lane, R);
    if (warp == 1 && piece == last / kThreads && last > 0 && !W.whole(last)) one(W.first(last) + (int32_t)lane, R);
  }
}

// --------------------------------------------------------------------------------- host side
struct Layout {
  uint64_t logprobs, entropy, top_logprobs, top_tokens, saved, total;
};
bool layout(uint32_t rows, uint32_t vocab, uint32_t top, uint32_t entropy, Layout& L) {
  if (rows > BO_LOGPROBS_MAX_ROWS || vocab == 0 || vocab > BO_LOGPROBS_MAX_VOCAB || top > vocab ||
      top > BO_LOGPROBS_MAX_TOP || entropy > 1)
    return false;
  uint64_t off = 0;
  auto take = [&](uint64_t bytes) {
    const uint64_t at = off;
    off = up(off + bytes, 256);
    return at;
  };
  L.logprobs = take((uint64_t)rows * 4);
  L.entropy = take(entropy ? (uint64_t)rows * 4 : 0);
  L.top_logprobs = take((uint64_t)rows * top * 4);
  L.top_tokens = take((uint64_t)rows * top * 4);
  L.saved = take((uint64_t)rows * sizeof(Saved));
  L.total = off ? off : 256;
  return true;
}
bool valid(const bo_logprobs* h) {
  return h && h->d_logprobs && h->d_saved && h->vocab > 0 && h->vocab <= BO_LOGPROBS_MAX_VOCAB &&
         h->rows <= BO_LOGPROBS_MAX_ROWS && h->top <= BO_LOGPROBS_MAX_TOP && h->top <= h->vocab &&
         (h->top == 0 || (h->d_top_logprobs && h->d_top_tokens));
}
// The results' memory, from the first to the last byte.
Region results(const bo_logprobs* h) {
  Layout L;
  layout(h->rows, h->vocab, h->top, h->d_entropy != nullptr, L);
  return Region(h->d_logprobs, 1, 0, L.total, 1);
}
// Numbers of `size` bytes, one a row, which may all be the same one.
Region column(const void* p, uint64_t rows, uint64_t stride, uint64_t size) {
  return Region(p, stride ? rows : std::min<uint64_t>(rows, 1), stride, 1, size);
}
bool matrix(const void* p, uint64_t ld, uint64_t rows, uint64_t width, uint64_t size) {
  return p && aligned(p, size) && ld <= (1ull << 40) && (rows <= 1 || ld >= width);
}
bool strided(const void* p, uint64_t stride, uint64_t size) {
  return aligned(p, size) && stride <= (1ull << 40);
}

template <uint32_t TH, bool F32>
cudaError_t score(const ScoreArgs& P, cudaStream_t s) {
  const uint32_t cluster = 1u << P.log_cluster;
  const bool ent = P.entropy != nullptr, top = P.top > 0;
  auto k = ent ? (top ? k_score<TH, F32, true, true> : k_score<TH, F32, true, false>)
               : (top ? k_score<TH, F32, false, true> : k_score<TH, F32, false, false>);
  // (a window more than a row fills where it begins inside one, and than its part of a cluster's)
  const uint64_t windows = ((uint64_t)P.vocab * (F32 ? 4 : 2) / kWindow + 2) / cluster + 1;
  const uint32_t smem = top ? (uint32_t)std::min<uint64_t>(kSegment, windows) * sizeof(Max<F32>) : 0;
  return launch(k, dim3(P.rows * cluster), TH, smem, cluster, s, P);
}

}  // namespace
}  // namespace bo

using namespace bo;

extern "C" {

uint64_t bo_logprobs_size(uint32_t rows, uint32_t vocab, uint32_t top, uint32_t entropy) {
  Layout L;
  return layout(rows, vocab, top, entropy, L) ? L.total : 0;
}

int bo_logprobs_init(uint32_t rows, uint32_t vocab, uint32_t top, uint32_t entropy, void* d_mem,
                     uint64_t mem_bytes, bo_logprobs* h_out, void* stream) {
  Layout L;
  if (!h_out || !layout(rows, vocab, top, entropy, L) || !d_mem || !aligned(d_mem, 256) ||
      mem_bytes < L.total)
    return BD_ERR_INVALID_ARG;
  uint8_t* p = static_cast<uint8_t*>(d_mem);
  bo_logprobs h = {};
  h.d_logprobs = reinterpret_cast<float*>(p + L.logprobs);
  h.d_entropy = entropy ? reinterpret_cast<float*>(p + L.entropy) : nullptr;
  h.d_top_logprobs = reinterpret_cast<float*>(p + L.top_logprobs);
  h.d_top_tokens = reinterpret_cast<int32_t*>(p + L.top_tokens);
  h.d_saved = p + L.saved;
  h.rows = rows;
  h.vocab = vocab;
  h.top = top;
  int rc;
  if ((rc = check(cudaGetDevice(&h.device)))) return rc;
  if ((rc = check(cudaMemsetAsync(d_mem, 0, L.total, static_cast<cudaStream_t>(stream))))) return rc;
  *h_out = h;
  return BD_OK;
}

int bo_logprobs_forward(const bo_logprobs* h, const void* d_logits, uint32_t dtype, uint64_t ld,
                        uint32_t rows, const void* d_tokens, uint32_t token_bytes,
                        uint64_t token_stride, float temperature, const float* d_temperature,
                        uint64_t temperature_stride, void* stream) {
  if (!valid(h) || dtype > BO_FP32 || rows > h->rows || (token_bytes != 4 && token_bytes != 8) ||
      (!d_temperature && !(temperature > 0.f && temperature <= FLT_MAX)))
    return BD_ERR_INVALID_ARG;
  const uint64_t size = dtype == BO_FP32 ? 4 : 2;
  if (rows > 0) {
    if (!matrix(d_logits, ld, rows, h->vocab, size) || !d_tokens ||
        !strided(d_tokens, token_stride, token_bytes) || !strided(d_temperature, temperature_stride, 4))
      return BD_ERR_INVALID_ARG;
    const Region out = results(h);
    if (meet(out, Region(d_logits, rows, ld, h->vocab, size)) ||
        meet(out, column(d_tokens, rows, token_stride, token_bytes)) ||
        meet(out, column(d_temperature, rows, temperature_stride, 4)))
      return BD_ERR_INVALID_ARG;
  }
  int sms = 0;
  if (const int rc = sm_count(h->device, sms)) return rc;
  if (rows == 0) return BD_OK;
  ScoreArgs P = {};
  P.x = static_cast<const uint8_t*>(d_logits);
  P.ld = ld * size;
  P.tokens = static_cast<const uint8_t*>(d_tokens);
  P.token_stride = token_stride * token_bytes;
  P.temps = d_temperature;
  P.temp_stride = temperature_stride;
  P.temp = temperature;
  P.token_bytes = token_bytes;
  P.rows = rows;
  P.vocab = h->vocab;
  P.top = h->top;
  P.logprobs = h->d_logprobs;
  P.entropy = h->d_entropy;
  P.top_logprobs = h->d_top_logprobs;
  P.top_tokens = h->d_top_tokens;
  P.saved = static_cast<Saved*>(h->d_saved);
  // Where rows are fewer than SMs, several blocks share one: up to eight, with a window a thread at least
  // (64 rows of 151936: four blocks 6.4 us, one 20).  From there on the largest blocks that the SMs
  // hold at once (300 rows of 151936: 512 threads 18.2 us, 256 22.8, 128 33; 1500 rows of 32000: 64
  // threads 19.4, 128 22.2).  Rows of up to 2048 windows (65536 BF16 logits) are too short for 512 (300 rows of
  // 32000: 5.6 us, with 256 4.9), and where there are more rows than that, 256 windows and fewer take 32
  // threads (20000 rows of 8000: 57.7 us, with 64 61.5, with 128 70.8), longer ones 64 (20000 rows of 32000:
  // 193 us, with 128 195), the longest 128 (8192 rows of 151936: 354 us, with 64 380).  With top tokens, whose
  // search takes shared memory, 128 begin at 1024 windows (1125 rows of 2001: 29 us, with 64 36).
  const uint64_t windows = (uint64_t)h->vocab * size / kWindow;
  while (P.log_cluster < kMaxLogCluster && (uint64_t)rows << P.log_cluster < (uint64_t)sms * 3 / 2 &&
         windows >> P.log_cluster >= 2 * 256)
    P.log_cluster++;
  const uint64_t held = (uint64_t)sms * (h->top ? 1024 : 1536), held_small = (uint64_t)sms * 1024;   // threads at once
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool f32 = dtype == BO_FP32;
  cudaError_t e;
  if (P.log_cluster == 0 && (uint64_t)rows * 512 <= held && windows > 2048)
    e = f32 ? score<512, true>(P, s) : score<512, false>(P, s);
  else if (P.log_cluster > 0 || (uint64_t)rows * 256 <= held)
    e = f32 ? score<256, true>(P, s) : score<256, false>(P, s);
  else if ((uint64_t)rows * 128 <= held_small)
    e = f32 ? score<128, true>(P, s) : score<128, false>(P, s);
  else if (windows <= 256)
    e = f32 ? score<32, true>(P, s) : score<32, false>(P, s);
  else if (windows <= (h->top ? 1024 : 2048) || (!h->top && (uint64_t)rows * 64 <= held_small))
    e = f32 ? score<64, true>(P, s) : score<64, false>(P, s);
  else
    e = f32 ? score<128, true>(P, s) : score<128, false>(P, s);
  return check(e);
}

int bo_logprobs_backward(const bo_logprobs* h, const void* d_logits, uint32_t dtype, uint64_t ld,
                         uint32_t rows, const float* d_grad_logprobs, uint64_t grad_logprobs_stride,
                         const float* d_grad_entropy, uint64_t grad_entropy_stride,
                         void* d_grad_logits, uint64_t ld_grad, void* stream) {
  if (!valid(h) || dtype > BO_FP32 || rows > h->rows || (d_grad_entropy && !h->d_entropy))
    return BD_ERR_INVALID_ARG;
  const uint64_t size = dtype == BO_FP32 ? 4 : 2;
  if (rows > 0) {
    if (!matrix(d_logits, ld, rows, h->vocab, size) ||
        !matrix(d_grad_logits, ld_grad, rows, h->vocab, size) || (!d_grad_logprobs && !d_grad_entropy) ||
        !strided(d_grad_logprobs, grad_logprobs_stride, 4) || !strided(d_grad_entropy, grad_entropy_stride, 4))
      return BD_ERR_INVALID_ARG;
    const Region out(d_grad_logits, rows, ld_grad, h->vocab, size);
    const bool in_place = d_grad_logits == d_logits && (ld == ld_grad || rows == 1);
    if ((!in_place && meet(out, Region(d_logits, rows, ld, h->vocab, size))) || meet(out, results(h)) ||
        meet(out, column(d_grad_logprobs, rows, grad_logprobs_stride, 4)) ||
        meet(out, column(d_grad_entropy, rows, grad_entropy_stride, 4)))
      return BD_ERR_INVALID_ARG;
  }
  int sms = 0;
  if (const int rc = sm_count(h->device, sms)) return rc;
  if (rows == 0) return BD_OK;
  GradArgs P = {};
  P.x = static_cast<const uint8_t*>(d_logits);
  P.ld = ld * size;
  P.dx = static_cast<uint8_t*>(d_grad_logits);
  P.ld_dx = ld_grad * size;
  P.g = d_grad_logprobs;
  P.g_stride = grad_logprobs_stride;
  P.h = d_grad_entropy;
  P.h_stride = grad_entropy_stride;
  P.rows = rows;
  P.vocab = h->vocab;
  // (one window more than a row fills where it begins inside one)
  P.pieces = (uint32_t)(((uint64_t)h->vocab * size / kWindow + 2 + kThreads - 1) / kThreads);
  P.saved = static_cast<const Saved*>(h->d_saved);
  const uint64_t blocks = (uint64_t)rows * P.pieces;
  if (blocks > 0x7FFFFFFFull) return BD_ERR_INVALID_ARG;
  return check(launch(dtype == BO_FP32 ? k_grad<true> : k_grad<false>, dim3((uint32_t)blocks), kThreads, 0,
                      1, static_cast<cudaStream_t>(stream), P));
}

}  // extern "C"
