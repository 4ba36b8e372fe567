// bo_adapter.cu -- low-rank adapters of many requests beside a shared projection: forward and
// backward (include/ops/bf16ops.h has the formulas).
//
// At ranks up to 128 a row's products take 2 r (hidden + out) operations for 2 hidden + 4 out
// bytes: below 100 operations a byte against the 280 that the tensor cores and HBM balance at,
// so every kernel here is built to stream x, y and the gradients once.
//
//   k_rows_*      group the rows of a batch by adapter (once per model step)
//   k_apply16     one launch for low = s A x and y += B low over tiles of 16 rows: the serving
//                 form, factors straight from global memory into the fragments
//   k_apply64     the same over tiles of 64 rows, factors and x through shared memory
//   k_low         low alone (bo_adapter_tc.cu), and
//   k_expand      y += B low alone: the two for many rows
//   k_transpose   the factors' transposes, with which the backward pass is the forward kernels:
//                 dlow = s B^T dy, dx += A^T dlow
//   k_wgrad_tc    dA and dB, sums over the rows of an adapter (bo_adapter_tc.cu); k_wgrad the same
//                 for rows and strides off the 16-byte boundary
//
// A tile of rows belongs to one adapter.  The thread blocks of a cluster share a tile: each takes
// a slice of the first product's long sum, the slices' sums meet through distributed shared
// memory in a fixed order, and each block then writes a slice of the second product's columns.
#include <cooperative_groups.h>
#include <algorithm>
#include <cstring>
#include <memory>
#include <new>

#include "bo_adapter.cuh"

namespace cg = cooperative_groups;

namespace bo {
namespace {

constexpr uint32_t kThreads = 256;   // eight warps

// ------------------------------------------------------------------------ grouping the rows
// One block per adapter counts its rows, then one block per adapter places them in order: the
// grouping is stable, so every later sum over an adapter's rows has one order.  Latency and the
// number of adapters bound it, since each reads the whole index: 64 rows of 64 adapters 1.8 + 2.7
// us, 16384 of 8 3.3 + 8.9 us, 131072 of 16 18 + 58 us.  A model step groups once for all layers.
__global__ void __launch_bounds__(kThreads) k_rows_count(const int32_t* __restrict__ index,
                                                         uint32_t rows, uint32_t k,
                                                         int32_t* __restrict__ counts,
                                                         int32_t* __restrict__ status) {
  after_previous();
  const int32_t a = (int32_t)blockIdx.x;
  int32_t c = 0, bad = 0;
  for (uint32_t t = threadIdx.x; t < rows; t += kThreads) {
    const int32_t v = index[t];
    c += v == a;
    bad |= v < -1 || v >= (int32_t)k;
  }
  __shared__ int32_t sh[2];
  if (threadIdx.x < 2) sh[threadIdx.x] = 0;
  __syncthreads();
  c = __reduce_add_sync(0xFFFFFFFFu, c);
  bad = __any_sync(0xFFFFFFFFu, bad);
  if ((threadIdx.x & 31) == 0) {
    atomicAdd(&sh[0], c);
    if (bad) atomicOr(&sh[1], 1);
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    counts[a] = sh[0];
    if (a == 0 && status) *status = sh[1] ? BD_ERR_INVALID_ARG : BD_OK;
  }
}

__device__ __forceinline__ int32_t block_sum(int32_t v, int32_t* sh) {   // sh: 8 words
  v = __reduce_add_sync(0xFFFFFFFFu, v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
  __syncthreads();
  int32_t s = 0;
  for (uint32_t w = 0; w < kThreads / 32; w++) s += sh[w];
  return s;
}

__global__ void __launch_bounds__(kThreads) k_rows_place(
    const int32_t* __restrict__ index, uint32_t rows, uint32_t k,
    const int32_t* __restrict__ counts, int32_t* __restrict__ perm, int32_t* __restrict__ offsets,
    Tile* __restrict__ tiles16, Tile* __restrict__ tiles64, Tile* __restrict__ tiles128,
    int32_t* __restrict__ ntiles, int32_t* __restrict__ blocks) {
  after_previous();
  __shared__ int32_t sh[kThreads / 32];
  const uint32_t a = blockIdx.x;
  int32_t c0 = 0, c16 = 0, c64 = 0, c128 = 0, cb = 0;
  for (uint32_t b = threadIdx.x; b < a; b += kThreads) {
    const int32_t c = counts[b];
    c0 += c;
    c16 += (c + 15) / 16;
    c64 += (c + 63) / 64;
    c128 += (c + 127) / 128;
    cb += max((c + 63) / 64, kLeast);
  }
  c0 = block_sum(c0, sh);
  c16 = block_sum(c16, sh);
  c64 = block_sum(c64, sh);
  c128 = block_sum(c128, sh);
  cb = block_sum(cb, sh);
  const int32_t mine = counts[a];
  const int32_t n16 = (mine + 15) / 16, n64 = (mine + 63) / 64, n128 = (mine + 127) / 128;
  if (threadIdx.x == 0) {
    offsets[a] = c0;
    blocks[a] = cb;
    if (a == k - 1) {
      offsets[k] = c0 + mine;
      blocks[k] = cb + max(n64, kLeast);
      ntiles[0] = c16 + n16;
      ntiles[1] = c64 + n64;
      ntiles[2] = c128 + n128;
    }
  }
  for (int32_t i = threadIdx.x; i < n16; i += kThreads)
    tiles16[c16 + i] = Tile{(int32_t)a, c0 + 16 * i, min(16, mine - 16 * i), c16 + n16};
  for (int32_t i = threadIdx.x; i < n64; i += kThreads)
    tiles64[c64 + i] = Tile{(int32_t)a, c0 + 64 * i, min(64, mine - 64 * i), c64 + n64};
  for (int32_t i = threadIdx.x; i < n128; i += kThreads)
    tiles128[c128 + i] = Tile{(int32_t)a, c0 + 128 * i, min(128, mine - 128 * i), c128 + n128};
  if (mine == 0) return;
  // four consecutive rows a thread, in order
  const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int32_t at = c0;
  const int32_t end = c0 + mine;
  for (uint32_t t0 = 0; t0 < rows && at < end; t0 += 4 * kThreads) {
    const uint32_t t = t0 + 4 * threadIdx.x;
    uint32_t hit = 0;
#pragma unroll
    for (uint32_t j = 0; j < 4; j++)
      if (t + j < rows && index[t + j] == (int32_t)a) hit |= 1u << j;
    const int32_t n = __popc(hit);
    int32_t incl = n;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int32_t o = __shfl_up_sync(0xFFFFFFFFu, incl, d);
      if ((int)lane >= d) incl += o;
    }
    __syncthreads();
    if (lane == 31) sh[warp] = incl;
    __syncthreads();
    int32_t before = 0, all = 0;
    for (uint32_t w = 0; w < kThreads / 32; w++) {
      if (w < warp) before += sh[w];
      all += sh[w];
    }
    int32_t p = at + before + incl - n;
#pragma unroll
    for (uint32_t j = 0; j < 4; j++)
      if (hit >> j & 1) perm[p++] = (int32_t)(t + j);
    at += all;
  }
}

// ------------------------------------------------------------------------------ building blocks
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void sts16(uint32_t dst, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(dst), "r"(v.x), "r"(v.y), "r"(v.z),
               "r"(v.w)
               : "memory");
}

__device__ __forceinline__ uint4 lds16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a)
               : "memory");
  return v;
}
__device__ __forceinline__ uint2 lds8(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
  return v;
}

// Eight values from p, of which the first n exist (n <= 0: none); the others are 0.  Off the
// 16-byte boundary they come as the 4-byte words that they fill, and the ends, without a branch:
// several of them wait for memory together (in branches each waits by itself: 8192 rows, x of 4095
// columns, rank 16, take 109 us, not 92).
__device__ __forceinline__ uint4 gather8(const uint16_t* p, int32_t n) {
  const int32_t odd = (int32_t)(reinterpret_cast<uintptr_t>(p) >> 1 & 1);
  n = min(n, 8);
  uint32_t t[5];
#pragma unroll
  for (int32_t j = 0; j < 5; j++) {   // values 2 j - odd and the next
    const int32_t e = 2 * j - odd;
    const bool front = j == 0 && odd;
    const uint32_t two = !front && e + 1 < n, one = front ? n > 0 : e + 1 == n;
    asm volatile(
        "{\n\t.reg .pred a, b;\n\tsetp.ne.u32 a, %2, 0;\n\tsetp.ne.u32 b, %3, 0;\n\t"
        "mov.b32 %0, 0;\n\t@a ld.global.b32 %0, [%1];\n\t@b ld.global.u16 %0, [%1];\n\t}"
        : "=&r"(t[j])
        : "l"(p + (front ? 0 : e)), "r"(two), "r"(one));
  }
  t[0] <<= 16 * odd;
  return make_uint4(__funnelshift_r(t[0], t[1], 16 * odd), __funnelshift_r(t[1], t[2], 16 * odd),
                    __funnelshift_r(t[2], t[3], 16 * odd), __funnelshift_r(t[3], t[4], 16 * odd));
}
// How rows of a matrix may be read: 16 bytes at a time, 4 bytes, or 2.
enum : uint32_t { kWide = 2, kEven = 1, kAny = 0 };
__device__ __forceinline__ uint32_t row_access(const uint16_t* base, uint64_t ld, bool vec) {
  return vec ? kWide : ((uint32_t)reinterpret_cast<uintptr_t>(base) | (uint32_t)ld * 2) & 3 ? kAny : kEven;
}
__device__ __forceinline__ uint4 load8(const uint16_t* p, int32_t n, bool vec) {
  if (vec) return n > 0 ? ld16(p) : make_uint4(0, 0, 0, 0);   // (n is a multiple of 8)
  return gather8(p, n);
}
// The same for the factors, which other blocks read too (n may be anything).
template <bool VEC = false>   // (whole words only)
__device__ __forceinline__ uint4 load8w(const uint16_t* p, int32_t n, bool vec) {
  if (VEC || (vec && (n >= 8 || n <= 0)))
    return n > 0 ? __ldg(reinterpret_cast<const uint4*>(p)) : make_uint4(0, 0, 0, 0);
  return gather8(p, n);
}
// ... N of them into shared memory.  Rows of even widths are copied without waiting too (8192 rows
// of 4094 and 4098, rank 16: forward 100 us, with loads and stores 128).
template <int N>
__device__ __forceinline__ void fill8(const uint32_t (&dst)[N], const uint16_t* const (&p)[N],
                                      const int32_t (&n)[N], const uint16_t* base, uint32_t access) {
  if (access == kWide) {
#pragma unroll
    for (int i = 0; i < N; i++) cp16n(dst[i], n[i] > 0 ? p[i] : base, n[i]);
  } else if (access == kEven) {
#pragma unroll
    for (int i = 0; i < N; i++)
#pragma unroll
      for (int j = 0; j < 4; j++) {
        const int32_t bytes = max(0, min(2 * n[i] - 4 * j, 4));
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst[i] + 4 * j),
                     "l"(bytes > 0 ? p[i] + 2 * j : base), "r"(bytes)
                     : "memory");
      }
  } else {
    uint4 v[N];
#pragma unroll
    for (int i = 0; i < N; i++) v[i] = gather8(p[i], n[i]);
#pragma unroll
    for (int i = 0; i < N; i++) sts16(dst[i], v[i]);
  }
}
__device__ __forceinline__ void store8(uint16_t* p, uint4 v, int32_t n, bool vec) {
  if (vec) {
    if (n > 0) *reinterpret_cast<uint4*>(p) = v;
    return;
  }
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  if (n >= 8) {
    const uint32_t odd = (uint32_t)reinterpret_cast<uintptr_t>(p) >> 1 & 1;
#pragma unroll
    for (int j = 0; j < 3; j++)
      *reinterpret_cast<uint32_t*>(p + odd + 2 * j) = __funnelshift_r(w[j], w[j + 1], 16 * odd);
    if (odd) {
      p[0] = (uint16_t)w[0];
      p[7] = (uint16_t)(w[3] >> 16);
    } else {
      *reinterpret_cast<uint32_t*>(p + 6) = w[3];
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < 8; j++)
    if (j < n) p[j] = (uint16_t)(w[j >> 1] >> (16 * (j & 1)));
}

// ... of rows that will not be read again soon
__device__ __forceinline__ void store8_stream(uint16_t* p, uint4 v) {
  asm volatile("st.global.cs.v4.u32 [%0], {%1,%2,%3,%4};" ::"l"(p), "r"(v.x), "r"(v.y), "r"(v.z),
               "r"(v.w)
               : "memory");
}

// Columns of the second product are dealt out so that a thread ends with eight neighbours: of a
// group of 32 columns, column 8 (i / 2) + 2 j + i % 2 is column i of the j-th mma tile, and the
// fragment's columns 2 q, 2 q + 1 over the four tiles are 8 q .. 8 q + 7.
__device__ __forceinline__ uint32_t dealt(uint32_t i, uint32_t j) {
  return 8 * (i >> 1) + 2 * j + (i & 1);
}
// Byte address in a tile of factor rows (RP columns) that are read in that order: the slots of
// rows 0, 1, 8, 9, 16, 17, 24, 25 (+ 2 j) have to differ.
template <int RP>
__device__ __forceinline__ uint32_t swz_dealt(uint32_t row, uint32_t chunk) {
  const uint32_t byte = row * (RP * 2) + chunk * 16, r = row >> 3;
  const uint32_t x = RP >= 64 ? ((r & 3) << 1 | (row & 1)) : RP == 32 ? (r & 3)
                                                                       : ((r & 1) | (r & 2) << 1);
  return byte ^ (x << 4);
}

// ---------------------------------------------------------------------- tiles of 16 rows
// The sum's index may be dealt to the threads in any order as long as both factors agree, so a
// thread reads 16 bytes (eight consecutive values) of each row and feeds them to two mma steps:
// the fragments come straight from global memory, every load of a warp independent of the
// others.  low enters the second product as two BF16 numbers, its rounding and what that cut
// off: with few rows the rounding errors of low would not average out in y, and the products
// cost nothing beside the latency of the loads.  What bounds it is the chain from the row's number
// to the stores, five trips to memory and one across the cluster: one row of rank 16 takes 4.6 us
// (4096 x 4096), 64 rows of 48 adapters 7.2 us (4096 x 11008, whose bytes take 3.9 us).
template <int RP>
struct Apply16 {
  static constexpr uint32_t kULd = RP + 8;
  static constexpr uint32_t kSmem = 9 * 16 * RP * 4 + 2 * 16 * kULd * 2;
};

// VEC: all rows, of the factors too, are whole 16-byte words; the code for others would be in the
// way of so short a kernel (one row of rank 16 5.3 us a call with it, 4.6 without; of rank 64 and
// 4096 x 11008 15.6 and 10.7).
template <int RP, bool VEC>
__global__ void __launch_bounds__(kThreads) k_apply16(const ApplyArgs P) {
  using L = Apply16<RP>;
  extern __shared__ __align__(1024) uint8_t smem[];
  float* const red = reinterpret_cast<float*>(smem);                 // [8][16][RP]
  float* const part = red + 8 * 16 * RP;                             // [16][RP]
  uint16_t* const us = reinterpret_cast<uint16_t*>(part + 16 * RP);  // [2][16][kULd]
  const cg::cluster_group cluster = cg::this_cluster();
  const uint32_t C = cluster.num_blocks(), c = cluster.block_rank();
  const uint32_t tile = blockIdx.x / C;
  after_previous();
  const Tile T = P.tiles[tile];              // (of the table's capacity, so within it)
  if (tile >= (uint32_t)*P.ntiles) return;   // (the whole cluster)
  const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, q = lane & 3;
  const int32_t r0 = (int32_t)g < T.count ? P.perm[T.start + g] : -1;
  const int32_t r1 = (int32_t)g + 8 < T.count ? P.perm[T.start + g + 8] : -1;
  const DevAdapter A = P.table[T.adapter];
  const int32_t rank = (int32_t)A.rank;
  const uint32_t first = c * 8 + warp, step = C * 8;

  // a group of 32 columns of y, and (of a small rank) its rows of B: loaded ahead of the sum
  constexpr int KS = RP >= 32 ? 32 : 16;
  constexpr bool kAhead = RP <= 32;
  uint4 y0, y1, w[4];
  auto load_w = [&](uint32_t gc, int ks, int j) {
    const uint32_t o = gc * 32 + dealt(g, j);
    const int32_t k = KS == 32 ? ks * 32 + 8 * (int32_t)q : 4 * (int32_t)q;
    const uint16_t* src = A.up + (uint64_t)o * A.ld_up + k;
    const int32_t n = o < P.N ? rank - k : 0;
    if (KS == 32) return load8w<VEC>(src, n, A.vec_up);
    uint2 t = make_uint2(0, 0);   // rank at most 16: four values a thread make one mma step
    if (VEC || A.vec_up) {
      if (n >= (VEC ? 1 : 4)) t = __ldg(reinterpret_cast<const uint2*>(src));
    }
    if (!VEC && (!A.vec_up || (n > 0 && n < 4))) {
      const uint4 f = gather8(src, min(n, 4));
      t = make_uint2(f.x, f.y);
    }
    return make_uint4(t.x, t.y, 0, 0);
  };
  auto load_group = [&](uint32_t gc) {
    const uint32_t col = gc * 32 + 8 * q;
    const int32_t n = (int32_t)P.N - (int32_t)col;
    y0 = load8(P.y + (int64_t)r0 * P.ldy + col, r0 >= 0 ? n : 0, VEC || P.vec_y);
    y1 = load8(P.y + (int64_t)r1 * P.ldy + col, r1 >= 0 ? n : 0, VEC || P.vec_y);
    if (kAhead) {
#pragma unroll
      for (int j = 0; j < 4; j++) w[j] = load_w(gc, 0, j);
    }
  };
  const bool any = P.y && first * 32 < P.N;
  if (any) load_group(first);

  float acc[RP / 8][4];
#pragma unroll
  for (int j = 0; j < RP / 8; j++) acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0.f;
#pragma unroll(RP <= 32 ? 4 : 1)
  for (uint32_t kc = first; kc * 32 < P.K; kc += step) {
    const uint32_t k = kc * 32 + 8 * q;
    const int32_t n = (int32_t)P.K - (int32_t)k;
    const uint4 xa = load8(P.x + (int64_t)r0 * P.ldx + k, r0 >= 0 ? n : 0, VEC || P.vec_x);
    const uint4 xb = load8(P.x + (int64_t)r1 * P.ldx + k, r1 >= 0 ? n : 0, VEC || P.vec_x);
#pragma unroll
    for (int j = 0; j < RP / 8; j++) {
      const int32_t row = j * 8 + g;
      const uint4 b = load8w<VEC>(A.down + (uint64_t)row * A.ld_down + k, row < rank ? n : 0, A.vec_down);
      mma16816(acc[j], xa.x, xb.x, xa.y, xb.y, b.x, b.y);
      mma16816(acc[j], xa.z, xb.z, xa.w, xb.w, b.z, b.w);
    }
  }
#pragma unroll
  for (int j = 0; j < RP / 8; j++) {
    float* d = red + (warp * 16 + g) * RP + j * 8 + 2 * q;
    *reinterpret_cast<float2*>(d) = make_float2(acc[j][0], acc[j][1]);
    *reinterpret_cast<float2*>(d + 8 * RP) = make_float2(acc[j][2], acc[j][3]);
  }
  __syncthreads();
  for (uint32_t e = threadIdx.x; e < 16 * RP; e += kThreads) {
    float s = 0.f;
#pragma unroll
    for (uint32_t v = 0; v < 8; v++) s += red[v * 16 * RP + e];
    part[e] = s;
  }
  cluster.sync();
  for (uint32_t e = threadIdx.x; e < 16 * RP; e += kThreads) {
    float v[kMaxCluster], s = 0.f;   // (all blocks' at once: each is a trip across the cluster)
#pragma unroll
    for (uint32_t b = 0; b < kMaxCluster; b++) v[b] = b < C ? cluster.map_shared_rank(part, b)[e] : 0.f;
#pragma unroll
    for (uint32_t b = 0; b < kMaxCluster; b++) s += v[b];
    const int32_t row = e / RP, col = e % RP;
    // columns past the rank are 0 whatever x holds (an infinity times a padded 0 is not)
    s = col < rank ? s * A.scale : 0.f;
    const uint32_t hi = pack_bf16(s, 0.f);
    const float rest = isfinite(bf16_lo(hi)) ? s - bf16_lo(hi) : 0.f;   // (s may round to infinity)
    us[row * L::kULd + col] = (uint16_t)hi;
    us[(16 + row) * L::kULd + col] = (uint16_t)pack_bf16(rest, 0.f);
    if (P.low && c == 0 && row < T.count)
      P.low[(int64_t)P.perm[T.start + row] * RP + col] = (uint16_t)hi;
  }
  __syncthreads();
  cg::cluster_group::arrival_token token = cluster.barrier_arrive();

  if (any) {
    for (uint32_t gc = first; gc * 32 < P.N; gc += step) {
      const uint32_t col = gc * 32 + 8 * q;
      const int32_t n = (int32_t)P.N - (int32_t)col;
      const uint32_t ya[4] = {y0.x, y0.y, y0.z, y0.w}, yb[4] = {y1.x, y1.y, y1.z, y1.w};
      uint4 wc[4];
      float d[4][4];   // y is the sum's first term
#pragma unroll
      for (int j = 0; j < 4; j++) {
        d[j][0] = bf16_lo(ya[j]);
        d[j][1] = bf16_hi(ya[j]);
        d[j][2] = bf16_lo(yb[j]);
        d[j][3] = bf16_hi(yb[j]);
        if (kAhead) wc[j] = w[j];
      }
      if ((gc + step) * 32 < P.N) load_group(gc + step);
#pragma unroll
      for (int ks = 0; ks < RP / KS; ks++) {
        if (ks * KS >= rank) break;
        if (!kAhead) {
#pragma unroll
          for (int j = 0; j < 4; j++) wc[j] = load_w(gc, ks, j);
        }
#pragma unroll
        for (int half = 0; half < 2; half++) {
          const uint16_t* u = us + (16 * half + g) * L::kULd;
          if (KS == 32) {
            const uint4 a = *reinterpret_cast<const uint4*>(u + ks * 32 + 8 * q);
            const uint4 b = *reinterpret_cast<const uint4*>(u + 8 * L::kULd + ks * 32 + 8 * q);
#pragma unroll
            for (int j = 0; j < 4; j++) {
              mma16816(d[j], a.x, b.x, a.y, b.y, wc[j].x, wc[j].y);
              mma16816(d[j], a.z, b.z, a.w, b.w, wc[j].z, wc[j].w);
            }
          } else {
            const uint2 a = *reinterpret_cast<const uint2*>(u + 4 * q);
            const uint2 b = *reinterpret_cast<const uint2*>(u + 8 * L::kULd + 4 * q);
#pragma unroll
            for (int j = 0; j < 4; j++) mma16816(d[j], a.x, b.x, a.y, b.y, wc[j].x, wc[j].y);
          }
        }
      }
      if (r0 >= 0)
        store8(P.y + (int64_t)r0 * P.ldy + col,
               make_uint4(pack_bf16(d[0][0], d[0][1]), pack_bf16(d[1][0], d[1][1]),
                          pack_bf16(d[2][0], d[2][1]), pack_bf16(d[3][0], d[3][1])),
               n, VEC || P.vec_y);
      if (r1 >= 0)
        store8(P.y + (int64_t)r1 * P.ldy + col,
               make_uint4(pack_bf16(d[0][2], d[0][3]), pack_bf16(d[1][2], d[1][3]),
                          pack_bf16(d[2][2], d[2][3]), pack_bf16(d[3][2], d[3][3])),
               n, VEC || P.vec_y);
    }
  }
  cluster.barrier_wait(std::move(token));   // the others may still read `part`
}

// ---------------------------------------------------------------------- tiles of 64 rows
// x and the factors through a ring of stages, two blocks an SM.  2048 rows of rank 16 (4096 x 4096)
// take 14.2 us for 50 MB: 1.1 us until the rows are known, 5.3 us of reading (at 6.3 TB/s, y
// included), 2.5 us for the sums to meet, 2.9 us of storing; with all tiles on the SMs at once
// nothing overlaps the middle.  A third block an SM would need 80 registers: the loads then sink
// to their uses (16384 rows, rank 64: 246 us became 378).
constexpr uint32_t kBK = 64;     // values of the first sum per stage
constexpr uint32_t kBN = 128;    // columns of the second product per step
constexpr uint32_t kStages = 4;

template <int RP>
struct Apply64 {
  static constexpr uint32_t kXBytes = 64 * kBK * 2, kWBytes = RP * kBK * 2;
  static constexpr uint32_t kStage = kXBytes + kWBytes;
  static constexpr uint32_t kRing = kStages * kStage;
  static constexpr uint32_t kPart = 64 * RP * 4;               // over the ring, after the sum
  // steps of B's rows (as many as fit over the ring) and of y that are there or on their way
  static constexpr uint32_t kUp = kBN * RP * 2, kUps = RP <= 32 ? 4 : RP == 64 ? 3 : 2;
  static constexpr uint32_t kY = 64 * kBN * 2, kYs = RP == 32 ? 3 : RP == 64 ? 2 : 4;
  // groups of copies that may be on their way at a step: those after its B, and after its y
  static constexpr int kAfterUp = 2 * (int)kUps - 3, kAfterY = 2 * (int)kYs - 2;
  static constexpr int kPending = kAfterUp < kAfterY ? kAfterUp : kAfterY;
  static constexpr uint32_t kULd = RP + 8;
  static constexpr uint32_t kU = 64 * kULd * 2;
  static constexpr uint32_t kFirst = kRing > kPart + kUps * kUp ? kRing : kPart + kUps * kUp;
  static constexpr uint32_t kRows = kFirst + kU, kYRing = kRows + 64 * 4;
  static constexpr uint32_t kSmem = kYRing + kYs * kY;
  // Of the sum a warp takes 32 rows and a quarter of a stage, so that a fragment of A serves two
  // tiles of rows; of rank 128, whose sums fill the registers, 16 rows and a half.
  static constexpr int kMR = RP <= 64 ? 2 : 1;
};

// VEC: every row of x, y and of the first factors can be read 16 bytes at a time.  (Rows of the
// second, of any rank, are read as they lie.)
template <int RP, bool VEC>
__global__ void __launch_bounds__(kThreads, RP <= 64 ? 2 : 1) k_apply64(const ApplyArgs P) {
  using L = Apply64<RP>;
  extern __shared__ __align__(1024) uint8_t smem[];
  float* const part = reinterpret_cast<float*>(smem);
  uint16_t* const us = reinterpret_cast<uint16_t*>(smem + L::kFirst);
  int32_t* const srow = reinterpret_cast<int32_t*>(smem + L::kRows);
  const cg::cluster_group cluster = cg::this_cluster();
  const uint32_t C = cluster.num_blocks(), c = cluster.block_rank();
  const uint32_t tile = blockIdx.x / C;
  after_previous();
  const Tile T = P.tiles[tile];              // (of the table's capacity, so within it)
  if (tile >= (uint32_t)*P.ntiles) return;   // (the whole cluster)
  const uint32_t tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, q = lane & 3;
  const uint32_t wr = warp & 3, wh = warp >> 2;   // 16 rows; half of a stage, of a step's columns
  // rows past the tile's end take its first row's place in loads and are never stored
  const int32_t row_a = P.perm[T.start];
  if (tid < 64) srow[tid] = (int32_t)tid < T.count ? P.perm[T.start + tid] : -1;
  const DevAdapter A = P.table[T.adapter];
  const int32_t rank = (int32_t)A.rank;
  __syncthreads();

  // ---- this block's steps of the columns of y.  A thread fetches the pieces that it will add to
  // by itself, ahead of the sum's end; (of rows off the 16-byte boundary one step ahead, into
  // registers).
  const uint32_t steps = P.y ? (P.N + kBN - 1) / kBN : 0;
  const uint32_t todo = steps > c ? (steps - c + C - 1) / C : 0;
  const int32_t r0 = srow[wr * 16 + g], r1 = srow[wr * 16 + g + 8];
  uint16_t* const yp0 = P.y + (int64_t)(r0 >= 0 ? r0 : row_a) * P.ldy + wh * 64 + 8 * q;
  uint16_t* const yp1 = P.y + (int64_t)(r1 >= 0 ? r1 : row_a) * P.ldy + wh * 64 + 8 * q;
  const int32_t left = (int32_t)P.N - (int32_t)(wh * 64 + 8 * q);
  uint4 y0[2], y1[2];
  const uint32_t yring = smem_addr(smem + L::kYRing) + tid * 16;
  auto load_y = [&](uint32_t i) {
#pragma unroll
    for (uint32_t h = 0; h < 2; h++) {
      const uint32_t at = (c + i * C) * kBN + h * 32;
      const int32_t n = left - (int32_t)at;
      if (VEC) {
        const uint32_t dst = yring + i % L::kYs * L::kY + h * 2 * kThreads * 16;
        if (r0 >= 0 && n > 0) cp16_ahead(dst, yp0 + at);
        if (r1 >= 0 && n > 0) cp16_ahead(dst + kThreads * 16, yp1 + at);
      } else {
        y0[h] = load8(yp0 + at, n, P.vec_y);
        y1[h] = load8(yp1 + at, n, P.vec_y);
      }
    }
  };

  // ---- low = s A x: this block's stages of the sum
  const uint32_t stages = (P.K + kBK - 1) / kBK;
  const uint32_t mine = stages > c ? (stages - c + C - 1) / C : 0;
  const uint32_t ring = smem_addr(smem);
  {
    const uint32_t xrow = tid >> 3, xch = tid & 7;   // rows xrow and xrow + 32, one 16-byte slot
    const int32_t s0 = srow[xrow], s1 = srow[xrow + 32];
    const uint16_t* const xp0 = P.x + (int64_t)(s0 >= 0 ? s0 : row_a) * P.ldx + xch * 8;
    const uint16_t* const xp1 = P.x + (int64_t)(s1 >= 0 ? s1 : row_a) * P.ldx + xch * 8;
    const uint16_t* const wp = A.down + xch * 8;
    const uint32_t x_access = row_access(P.x, P.ldx, P.vec_x);
    const uint32_t w_access = row_access(A.down, A.ld_down, A.vec_down);
    const uint32_t sx = swz(xrow * 128 + xch * 16);   // (32 rows on: the same slot, 4096 bytes on)
    auto load_stage = [&](uint32_t i) {
      const uint32_t k0 = (c + i * C) * kBK, at = ring + (i % kStages) * L::kStage + sx;
      const int32_t n = (int32_t)P.K - (int32_t)(k0 + xch * 8);
      const uint32_t k = n > 0 ? k0 : 0;   // (nothing is read past a row's end)
      if (VEC) {
        cp16z(at, xp0 + k, s0 >= 0 && n > 0);
        cp16z(at + 4096, xp1 + k, s1 >= 0 && n > 0);
#pragma unroll
        for (uint32_t r = 0; r < RP; r += 32) {
          const uint32_t row = r + xrow;
          if (RP < 32 && row >= RP) break;
          const bool there = (int32_t)row < rank;
          cp16z(at + L::kXBytes + r * 128, wp + (there ? (uint64_t)row * A.ld_down : 0) + k,
                there && n > 0);
        }
      } else {
        const uint32_t xd[2] = {at, at + 4096};
        const uint16_t* const xs[2] = {xp0 + k, xp1 + k};
        const int32_t xn[2] = {s0 >= 0 ? n : 0, s1 >= 0 ? n : 0};
        fill8(xd, xs, xn, P.x, x_access);
        constexpr uint32_t W = (RP + 31) / 32;
        if (RP < 32 && xrow >= RP) return;
        uint32_t wd[W];
        const uint16_t* ws[W];
        int32_t wn[W];
#pragma unroll
        for (uint32_t i = 0; i < W; i++) {
          const uint32_t row = i * 32 + xrow;
          const bool there = (int32_t)row < rank;
          wd[i] = at + L::kXBytes + i * 4096;
          ws[i] = wp + (there ? (uint64_t)row * A.ld_down : 0) + k;
          wn[i] = there ? n : 0;
        }
        fill8(wd, ws, wn, A.down, w_access);
      }
    };
    constexpr int MR = L::kMR;
    const uint32_t rg = warp % (4 / MR), kq = warp / (4 / MR);   // rows 16 MR rg ..; part of a stage
    float acc[MR][RP / 8][4];
#pragma unroll
    for (int m = 0; m < MR; m++)
#pragma unroll
      for (int j = 0; j < RP / 8; j++)
        acc[m][j][0] = acc[m][j][1] = acc[m][j][2] = acc[m][j][3] = 0.f;
    for (uint32_t i = 0; i < kStages - 1; i++) {
      if (i < mine) load_stage(i);
      cp_commit();
    }
    // behind the last stage, which iteration `tail` no longer finds to fetch, come the first y
    const uint32_t y_steps = todo < L::kYs ? todo : L::kYs;
    const uint32_t tail = mine > kStages - 1 ? mine - (kStages - 1) : 0;
    for (uint32_t i = 0; i < mine; i++) {
      cp_wait<kStages - 2>();
      __syncthreads();
      const uint32_t ahead = i + kStages - 1;
      if (ahead < mine) load_stage(ahead);
      else if (VEC && i - tail < y_steps) load_y(i - tail);
      cp_commit();
      const uint32_t xs = ring + (i % kStages) * L::kStage, ws = xs + L::kXBytes;
#pragma unroll
      for (uint32_t kk = 0; kk < 2 / MR; kk++) {
        const uint32_t kb = (kq * (2 / MR) + kk) * 32;   // byte of the 16-value step in a row
        uint32_t a[MR][4];
#pragma unroll
        for (int m = 0; m < MR; m++)
          ldsm4(a[m], xs + swz(((rg * MR + m) * 16 + (lane & 15)) * 128 + kb + (lane >> 4) * 16));
#pragma unroll
        for (int j = 0; j < RP / 16; j++) {
          uint32_t b[4];
          ldsm4(b, ws + swz(((lane >> 4) * 8 + (lane & 7)) * 128 + kb + ((lane >> 3) & 1) * 16) +
                       j * 2048);
#pragma unroll
          for (int m = 0; m < MR; m++) {
            mma16816(acc[m][2 * j], a[m][0], a[m][1], a[m][2], a[m][3], b[0], b[1]);
            mma16816(acc[m][2 * j + 1], a[m][0], a[m][1], a[m][2], a[m][3], b[2], b[3]);
          }
        }
      }
    }
    // (the last stage was waited for with everything before it; on their way are pieces of y)
    if (VEC)
      for (uint32_t i = mine - tail; i < y_steps; i++) {
        load_y(i);
        cp_commit();
      }
    // join the parts of every stage, in one order
    __syncthreads();
#pragma unroll
    for (int m = 0; m < MR; m++)
#pragma unroll
      for (int j = 0; j < RP / 8; j++)
#pragma unroll
        for (int h = 0; h < 2; h++)
          *reinterpret_cast<float2*>(part + kq * 64 * RP + ((rg * MR + m) * 16 + h * 8 + g) * RP +
                                     j * 8 + 2 * q) =
              make_float2(acc[m][j][2 * h], acc[m][j][2 * h + 1]);
    __syncthreads();
    for (uint32_t e = tid * 2; e < 64 * RP; e += kThreads * 2) {
      float2 s = *reinterpret_cast<const float2*>(part + e);
#pragma unroll
      for (uint32_t z = 1; z < 2 * MR; z++) {
        const float2 v = *reinterpret_cast<const float2*>(part + z * 64 * RP + e);
        s.x += v.x;
        s.y += v.y;
      }
      *reinterpret_cast<float2*>(part + e) = s;
    }
  }

  // ---- y += B low: this block's steps of the columns, the first one's loads ahead of the join
  constexpr uint32_t per = RP / 8, span = kThreads / per;   // 16-byte slots in a row; rows at once
  const uint32_t urow = tid / per, uch = tid % per;
  const uint32_t up0 = ring + L::kPart;
  const uint16_t* const upp = A.up + (uint64_t)urow * A.ld_up + uch * 8;
  const int32_t un = rank - (int32_t)uch * 8;
  const uint32_t up_access = row_access(A.up, A.ld_up, A.vec_up);
  auto load_up = [&](uint32_t i) {
    const uint32_t o0 = (c + i * C) * kBN, at = up0 + i % L::kUps * L::kUp;
    constexpr uint32_t W = kBN / span;
    uint32_t ud[W];
    const uint16_t* us[W];
    int32_t ns[W];
#pragma unroll
    for (uint32_t r = 0; r < W; r++) {
      const uint32_t o = o0 + r * span;
      ud[r] = at + swz_dealt<RP>(r * span + urow, uch);
      us[r] = upp + (uint64_t)o * A.ld_up;
      ns[r] = o + urow < P.N ? un : 0;
    }
    fill8(ud, us, ns, A.up, up_access);
  };
  // join the sums of the cluster's blocks: each joins some of the rows and hands them to all
  cluster.sync();
  if (!VEC && todo > 0) load_y(0);
#pragma unroll
  for (uint32_t i = 0; i + 1 < L::kUps; i++) {
    if (i < todo) load_up(i);
    cp_commit();
    cp_commit();   // (in the place of a y: every step has two groups)
  }
  {
    const uint32_t rows = 64 / C;
    for (uint32_t e = tid * 2; e < rows * RP; e += kThreads * 2) {
      const uint32_t row = c * rows + e / RP, col = e % RP;
      float2 v[kMaxCluster], s = make_float2(0.f, 0.f);   // (all blocks' at once)
#pragma unroll
      for (uint32_t b = 0; b < kMaxCluster; b++)
        v[b] = b < C ? *reinterpret_cast<const float2*>(cluster.map_shared_rank(part, b) + row * RP + col)
                     : make_float2(0.f, 0.f);
#pragma unroll
      for (uint32_t b = 0; b < kMaxCluster; b++) {
        s.x += v[b].x;
        s.y += v[b].y;
      }
      // columns past the rank are 0 whatever x holds (an infinity times a padded 0 is not)
      const uint32_t u = pack_bf16((int32_t)col < rank ? s.x * A.scale : 0.f,
                                   (int32_t)col + 1 < rank ? s.y * A.scale : 0.f);
#pragma unroll
      for (uint32_t b = 0; b < kMaxCluster; b++)
        if (b < C) *reinterpret_cast<uint32_t*>(cluster.map_shared_rank(us, b) + row * L::kULd + col) = u;
      if (P.low && srow[row] >= 0)
        *reinterpret_cast<uint32_t*>(P.low + (int64_t)srow[row] * RP + col) = u;
    }
  }
  cluster.sync();   // low is complete, and nobody reads another block's memory after this

  for (uint32_t i = 0; i < todo; i++) {
    cp_wait<L::kPending>();
    __syncthreads();
    if (i + L::kUps - 1 < todo) load_up(i + L::kUps - 1);
    cp_commit();
    if (VEC) {
#pragma unroll
      for (uint32_t h = 0; h < 2; h++) {
        const uint32_t src = yring + i % L::kYs * L::kY + h * 2 * kThreads * 16;
        y0[h] = lds16(src);
        y1[h] = lds16(src + kThreads * 16);
      }
    }
    float d[2][4][4];   // y is the sum's first term
#pragma unroll
    for (int h = 0; h < 2; h++) {
      const uint32_t a[4] = {y0[h].x, y0[h].y, y0[h].z, y0[h].w};
      const uint32_t b[4] = {y1[h].x, y1[h].y, y1[h].z, y1[h].w};
#pragma unroll
      for (int j = 0; j < 4; j++) {
        d[h][j][0] = bf16_lo(a[j]);
        d[h][j][1] = bf16_hi(a[j]);
        d[h][j][2] = bf16_lo(b[j]);
        d[h][j][3] = bf16_hi(b[j]);
      }
    }
    if (VEC ? i + L::kYs < todo : i + 1 < todo) load_y(VEC ? i + L::kYs : i + 1);
    cp_commit();
    const uint32_t at = up0 + i % L::kUps * L::kUp;
#pragma unroll
    for (int ks = 0; ks < RP / 16; ks++) {
      if (ks * 16 >= rank) break;
      uint32_t a[4];
      ldsm4(a, smem_addr(us + (wr * 16 + (lane & 15)) * L::kULd + ks * 16 + (lane >> 4) * 8));
#pragma unroll
      for (int h = 0; h < 2; h++)
#pragma unroll
        for (int jj = 0; jj < 2; jj++) {
          uint32_t b[4];
          const uint32_t row = wh * 64 + h * 32 + dealt(lane & 7, 2 * jj + (lane >> 4));
          ldsm4(b, at + swz_dealt<RP>(row, ks * 2 + ((lane >> 3) & 1)));
          mma16816(d[h][2 * jj], a[0], a[1], a[2], a[3], b[0], b[1]);
          mma16816(d[h][2 * jj + 1], a[0], a[1], a[2], a[3], b[2], b[3]);
        }
    }
#pragma unroll
    for (uint32_t h = 0; h < 2; h++) {
      const uint32_t col = (c + i * C) * kBN + h * 32;
      const int32_t n = left - (int32_t)col;
      if (r0 >= 0)
        store8(yp0 + col, make_uint4(pack_bf16(d[h][0][0], d[h][0][1]), pack_bf16(d[h][1][0], d[h][1][1]),
                                     pack_bf16(d[h][2][0], d[h][2][1]), pack_bf16(d[h][3][0], d[h][3][1])),
               n, VEC || P.vec_y);
      if (r1 >= 0)
        store8(yp1 + col, make_uint4(pack_bf16(d[h][0][2], d[h][0][3]), pack_bf16(d[h][1][2], d[h][1][3]),
                                     pack_bf16(d[h][2][2], d[h][2][3]), pack_bf16(d[h][3][2], d[h][3][3])),
               n, VEC || P.vec_y);
    }
  }
}

// ------------------------------------------------------- y += B low, for many rows of an adapter
// With low known, the blocks take equal shares of (columns, rows): a block keeps 256 columns' rows
// of B in shared memory and runs down the adapter's rows, each warp by itself over 32 rows at a
// time and 32 columns a step, so that B is read once per block and nothing waits for another
// warp.  A thread's own pieces of y come through a ring of asynchronous copies four steps deep,
// which fetch 256 bytes of L2 at once; the stores are streamed (186, 176 and 172 us without, with
// the one and with both).  16384 rows of rank 64 and 14336 columns: 172 us for 940 MB, 5.5 TB/s;
// issue is active half of the time, and reads and writes of the same pages take turns.
template <int RP>
struct Expand {
  static constexpr uint32_t kN = RP <= 64 ? 256 : 128;   // columns of a block
  static constexpr uint32_t kB = kN * RP * 2;
  static constexpr uint32_t kDepth = 4;
  static constexpr uint32_t kSlot = 4 * kThreads * 16;   // 64 bytes a thread
  static constexpr uint32_t kSmem = kB + kDepth * kSlot;
  // byte address of a factor row's 16-byte slot: the rows that a quarter warp reads together
  // (two neighbours; of rank 16 also those 8 further on) fall into different banks
  static __device__ __forceinline__ uint32_t at(uint32_t row, uint32_t byte) {
    const uint32_t a = row * (RP * 2) + byte;
    return RP >= 64 ? a ^ (row & 1) << 6 : RP == 16 ? a ^ (row >> 3 & 1) << 6 : a;
  }
};

// (At rank 128 low takes 64 registers: two blocks an SM spill, 130 us at 16384 rows of 4096 x 4096,
// one does not, 119 us.)
template <int RP>
__global__ void __launch_bounds__(kThreads, RP <= 64 ? 2 : 1) k_expand(const ApplyArgs P) {
  using L = Expand<RP>;
  constexpr int KS = RP >= 32 ? RP / 32 : 1;
  extern __shared__ __align__(1024) uint8_t smem[];
  after_previous();
  const uint32_t tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, q = lane & 3;
  const uint32_t nt = (uint32_t)*P.ntiles, chunks = (P.N + L::kN - 1) / L::kN;
  const uint64_t all = (uint64_t)nt * chunks;
  uint64_t at = all * blockIdx.x / gridDim.x;
  const uint64_t end = all * (blockIdx.x + 1) / gridDim.x;
  const uint32_t bs = smem_addr(smem), ring = bs + L::kB + tid * 16;
  while (at < end) {
    // the block's tiles of one adapter and one piece of the columns
    const uint32_t t0 = (uint32_t)(at % nt), n0 = (uint32_t)(at / nt) * L::kN;
    const Tile T = P.tiles[t0];
    const uint64_t left = end - at;
    const uint32_t t1 = left < (uint32_t)T.end - t0 ? t0 + (uint32_t)left : (uint32_t)T.end;
    const Tile Z = P.tiles[t1 - 1];
    at += t1 - t0;
    const DevAdapter A = P.table[T.adapter];
    const int32_t rank = (int32_t)A.rank, r_end = Z.start + Z.count;
    __syncthreads();   // every warp is done with the B before
    const uint32_t access = row_access(A.up, A.ld_up, A.vec_up);
    constexpr uint32_t W = 4;
    for (uint32_t s0 = tid; s0 < L::kN * (RP / 8); s0 += kThreads * W) {
      uint32_t dst[W];
      const uint16_t* src[W];
      int32_t ns[W];
#pragma unroll
      for (uint32_t i = 0; i < W; i++) {
        const uint32_t s = s0 + i * kThreads, row = s / (RP / 8), ch = s % (RP / 8);
        if (L::kN * (RP / 8) % (kThreads * W) != 0 && s >= L::kN * (RP / 8)) {
          dst[i] = dst[0];   // (once more the same)
          src[i] = src[0];
          ns[i] = ns[0];
          continue;
        }
        dst[i] = bs + L::at(row, ch * 16);
        src[i] = A.up + (uint64_t)(n0 + row) * A.ld_up + ch * 8;
        ns[i] = n0 + row < P.N ? rank - (int32_t)ch * 8 : 0;
      }
      fill8(dst, src, ns, A.up, access);
    }
    cp_commit();   // (waited for below, with the first pieces of y on their way too)

    const int32_t n_left = (int32_t)(P.N - n0);
    const uint32_t groups = (uint32_t)((n_left < (int32_t)L::kN ? n_left : (int32_t)L::kN) + 31) / 32;
    const int32_t units = (r_end - T.start + 31) / 32;
    const int32_t mine = units > (int32_t)warp ? (units - (int32_t)warp + 7) / 8 : 0;   // (may be 0)
    auto row_of = [&](int32_t u, int i) {   // the thread's i-th row of its u-th unit, or -1
      const int32_t r = T.start + ((int32_t)warp + u * 8) * 32 + (int32_t)g + 8 * i;
      return u < mine && r < r_end ? P.perm[r] : -1;
    };
    const int64_t base = (int64_t)n0 + 8 * q;
    // the copies run ahead: their unit, step and rows
    int32_t pu = 0;
    uint32_t pg = 0;
    int32_t prow[4], pnext[4], row[4], next[4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
      row[i] = prow[i] = row_of(0, i);
      next[i] = pnext[i] = row_of(1, i);
    }
    uint32_t issued = 0, total = (uint32_t)mine * groups;
    auto issue = [&]() {
      if (issued < total) {
        const uint32_t dst = ring + (issued % L::kDepth) * L::kSlot;
        const bool there = (int32_t)(pg * 32 + 8 * q) < n_left;
#pragma unroll
        for (int i = 0; i < 4; i++)
          if (prow[i] >= 0 && there)
            cp16_ahead(dst + i * kThreads * 16, P.y + (int64_t)prow[i] * P.ldy + base + pg * 32);
        if (++pg == groups) {
          pg = 0;
          pu++;
#pragma unroll
          for (int i = 0; i < 4; i++) {
            prow[i] = pnext[i];
            pnext[i] = row_of(pu + 1, i);
          }
        }
        issued++;
      }
      cp_commit();
    };
#pragma unroll
    for (uint32_t i = 0; i < L::kDepth - 1; i++) issue();
    cp_wait<L::kDepth - 1>();
    __syncthreads();   // B is there
    uint32_t step = 0;
    for (int32_t u = 0; u < mine; u++) {
      uint4 a[4][KS];   // low: rows g, g + 8, g + 16, g + 24
#pragma unroll
      for (int i = 0; i < 4; i++) {
        const uint16_t* src = P.low + (int64_t)(row[i] >= 0 ? row[i] : 0) * RP;
#pragma unroll
        for (int ks = 0; ks < KS; ks++) {
          if (RP >= 32) {
            a[i][ks] = ld16(src + ks * 32 + 8 * q);
          } else {
            const uint2 t = *reinterpret_cast<const uint2*>(src + 4 * q);
            a[i][ks] = make_uint4(t.x, t.y, 0, 0);
          }
        }
      }
      for (uint32_t gi = 0; gi < groups; gi++, step++) {
        issue();
        cp_wait<L::kDepth - 1>();
        const int32_t n = n_left - (int32_t)(gi * 32 + 8 * q);
        float d[2][4][4];   // y is the sum's first term
#pragma unroll
        for (int i = 0; i < 4; i++) {
          const uint4 y = lds16(ring + (step % L::kDepth) * L::kSlot + i * kThreads * 16);
          const uint32_t w[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
          for (int j = 0; j < 4; j++) {
            d[i >> 1][j][2 * (i & 1)] = bf16_lo(w[j]);
            d[i >> 1][j][2 * (i & 1) + 1] = bf16_hi(w[j]);
          }
        }
#pragma unroll
        for (int ks = 0; ks < KS; ks++)
#pragma unroll
          for (int j = 0; j < 4; j++) {
            const uint32_t o = gi * 32 + dealt(g, j);
            if (RP >= 32) {
              const uint4 b = lds16(bs + L::at(o, ks * 64 + q * 16));
#pragma unroll
              for (int m = 0; m < 2; m++) {
                const uint4 &lo = a[2 * m][ks], &hi = a[2 * m + 1][ks];
                mma16816(d[m][j], lo.x, hi.x, lo.y, hi.y, b.x, b.y);
                mma16816(d[m][j], lo.z, hi.z, lo.w, hi.w, b.z, b.w);
              }
            } else {
              const uint2 b = lds8(bs + L::at(o, q * 8));
#pragma unroll
              for (int m = 0; m < 2; m++)
                mma16816(d[m][j], a[2 * m][0].x, a[2 * m + 1][0].x, a[2 * m][0].y,
                         a[2 * m + 1][0].y, b.x, b.y);
            }
          }
#pragma unroll
        for (int i = 0; i < 4; i++) {
          const int m = i >> 1, h = 2 * (i & 1);
          if (row[i] >= 0 && n > 0)
            store8_stream(P.y + (int64_t)row[i] * P.ldy + base + gi * 32,
                          make_uint4(pack_bf16(d[m][0][h], d[m][0][h + 1]),
                                     pack_bf16(d[m][1][h], d[m][1][h + 1]),
                                     pack_bf16(d[m][2][h], d[m][2][h + 1]),
                                     pack_bf16(d[m][3][h], d[m][3][h + 1])));
        }
      }
#pragma unroll
      for (int i = 0; i < 4; i++) {
        row[i] = next[i];
        next[i] = row_of(u + 2, i);
      }
    }
    cp_wait<0>();
  }
}

// ---------------------------------------------------------------- transposes of the factors
// down (rank x hidden) to hidden x RP and up (out x rank) to RP x out8, both zero-padded, and a
// table entry that has them in the other's place.  4.8 us for four adapters of rank 64 (4096 and
// 11008 features, 15 MB), mostly latency; the factors change with every step of training, so the
// transposes are made in every call.
constexpr uint32_t kTF = 64;   // features a block turns at a time
template <int RP>
__global__ void __launch_bounds__(kThreads) k_transpose(const DevAdapter* __restrict__ table,
                                                        uint32_t hidden, uint32_t out,
                                                        uint32_t out8, uint16_t* __restrict__ buf,
                                                        DevAdapter* __restrict__ swapped,
                                                        uint32_t* __restrict__ counters,
                                                        uint32_t slices) {
  constexpr uint32_t kLd = RP + 2;
  __shared__ uint16_t sh[kTF * kLd];   // [feature][rank]
  after_previous();
  const DevAdapter A = table[blockIdx.y];
  uint16_t* const at = buf + (uint64_t)blockIdx.y * RP * ((uint64_t)hidden + out8);
  uint16_t* const bt = at + (uint64_t)hidden * RP;
  const uint32_t ht = (hidden + kTF - 1) / kTF;
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    DevAdapter S = A;
    S.down = bt;
    S.ld_down = out8;
    S.up = at;
    S.ld_up = RP;
    S.vec_down = S.vec_up = 1;
    swapped[blockIdx.y] = S;
  }
  for (uint32_t i = blockIdx.x * kThreads + threadIdx.x; i < slices; i += gridDim.x * kThreads)
    counters[(uint64_t)blockIdx.y * slices + i] = 0;   // of k_wgrad
  const bool first = blockIdx.x < ht;
  const uint32_t f0 = (first ? blockIdx.x : blockIdx.x - ht) * kTF;
  const int32_t rank = (int32_t)A.rank;
  for (uint32_t s = threadIdx.x; s < kTF * RP / 8; s += kThreads) {
    if (first) {   // eight features of a row of A
      const uint32_t r = s / (kTF / 8), f = s % (kTF / 8) * 8;
      const uint4 v = load8w(A.down + (uint64_t)r * A.ld_down + f0 + f,
                             (int32_t)r < rank ? (int32_t)hidden - (int32_t)(f0 + f) : 0, A.vec_down);
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int j = 0; j < 8; j++) sh[(f + j) * kLd + r] = (uint16_t)(w[j >> 1] >> (16 * (j & 1)));
    } else {       // eight columns of a row of B
      const uint32_t f = s / (RP / 8), r = s % (RP / 8) * 8;
      const uint4 v = load8w(A.up + (uint64_t)(f0 + f) * A.ld_up + r,
                             f0 + f < out ? rank - (int32_t)r : 0, A.vec_up);
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int j = 0; j < 4; j++) *reinterpret_cast<uint32_t*>(sh + f * kLd + r + 2 * j) = w[j];
    }
  }
  __syncthreads();
  for (uint32_t s = threadIdx.x; s < kTF * RP / 8; s += kThreads) {
    uint32_t w[4];
    if (first) {
      const uint32_t f = s / (RP / 8), r = s % (RP / 8) * 8;
#pragma unroll
      for (int j = 0; j < 4; j++) w[j] = *reinterpret_cast<const uint32_t*>(sh + f * kLd + r + 2 * j);
      if (f0 + f < hidden)
        *reinterpret_cast<uint4*>(at + (uint64_t)(f0 + f) * RP + r) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
      const uint32_t r = s / (kTF / 8), f = s % (kTF / 8) * 8;
#pragma unroll
      for (int j = 0; j < 4; j++)
        w[j] = sh[(f + 2 * j) * kLd + r] | (uint32_t)sh[(f + 2 * j + 1) * kLd + r] << 16;
      if (f0 + f < out8)
        *reinterpret_cast<uint4*>(bt + (uint64_t)r * out8 + f0 + f) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

// ------------------------------------------------------------------------ weight gradients
// A piece is 128 features of x (for dA) or dy (for dB) of one adapter, a sum over the adapter's
// rows in stages of 64.  The blocks take equal shares of all stages of all pieces, so none waits
// while another works; a piece that several blocks share is joined by the one that ends last, in
// the order of the blocks, from their sums in the workspace.
// This form, on mma.sync, takes what the other's 16-byte copies cannot: 8192 rows of 4095 and 4097
// features, rank 64, take 142 us; of 4096, there, 38 us.
constexpr uint32_t kWStages = 3;
template <int RP>
struct Wgrad {
  static constexpr uint32_t kQ = 64 * kFeat * 2, kPb = 64 * RP * 2, kStage = kQ + kPb;
  static constexpr uint32_t kLd = RP + 2;   // of the sums in shared memory, read along both ways
  static constexpr uint32_t kRing = kWStages * kStage, kPart = kFeat * kLd * 4;
  static constexpr uint32_t kSmem = kRing > kPart ? kRing : kPart;
  // 32 features a warp, so that a fragment of low serves two tiles; the warps' other half then
  // takes the other half of the rows (of rank 128 the sums alone fill the registers: 16)
  static constexpr int kMF = RP <= 64 ? 2 : 1;
};

template <int RP>
__global__ void __launch_bounds__(kThreads, 2) k_wgrad(const WgradArgs P) {
  using L = Wgrad<RP>;
  constexpr int MF = L::kMF;
  extern __shared__ __align__(1024) uint8_t smem[];
  float* const part = reinterpret_cast<float*>(smem);   // [feature][kLd], after a piece's stages
  __shared__ uint32_t sh_last;
  after_previous();
  const uint32_t hs = (P.hidden + kFeat - 1) / kFeat, slices = hs + (P.out + kFeat - 1) / kFeat;
  const uint32_t tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, q = lane & 3;
  const uint32_t fw = MF == 2 ? warp & 3 : warp, th = MF == 2 ? warp >> 2 : 0;
  const uint32_t ring = smem_addr(smem);
  const uint32_t qch = tid & 15, qrow = tid >> 4;
  constexpr uint32_t per = RP / 8, span = kThreads / per, PN = (64 + span - 1) / span;
  const uint32_t pch = tid % per, prow = tid / per;

  const Shares sh((uint64_t)P.blocks[P.k] * slices, gridDim.x);
  if (blockIdx.x >= sh.G) return;
  const uint64_t s_begin = sh.begin(blockIdx.x);
  for (Piece Q(P, slices, s_begin, sh.begin(blockIdx.x + 1)); !Q.over(); Q.next(P, slices)) {
    const uint32_t mine = Q.mine;
    const DevAdapter A = P.table[Q.adapter];
    const bool down = Q.slice < hs;
    const uint32_t f0 = (down ? Q.slice : Q.slice - hs) * kFeat, F = down ? P.hidden : P.out;
    const uint64_t lds = down ? P.ldx : P.lddy;
    const uint32_t access = down ? row_access(P.x, P.ldx, P.vec_x) : row_access(P.dy, P.lddy, P.vec_dy);
    const uint16_t* const pr = down ? P.dlow : P.low;
    const int32_t start = Q.row0 + (int32_t)Q.first * 64, end = Q.row1;
    const int32_t qn = (int32_t)F - (int32_t)(f0 + qch * 8);
    const uint16_t* const qsrc = (down ? P.x : P.dy) + (qn > 0 ? f0 + qch * 8 : 0);

    // A thread's slots of a stage: four rows of x or dy, up to four of low; their row numbers
    // are read one stage ahead of the rows.
    int32_t tq[4], tp[PN];
    auto load_rows = [&](uint32_t i) {
      const int32_t t0 = start + (int32_t)i * 64;
#pragma unroll
      for (uint32_t j = 0; j < 4; j++) {
        const int32_t t = t0 + (int32_t)(qrow + 16 * j);
        tq[j] = t < end ? P.perm[t] : -1;
      }
#pragma unroll
      for (uint32_t j = 0; j < PN; j++) {
        const uint32_t r = prow + span * j;
        const int32_t t = t0 + (int32_t)r;
        tp[j] = r < 64 && t < end ? P.perm[t] : -1;
      }
    };
    auto load_stage = [&](uint32_t i) {
      const uint32_t to = ring + (i % kWStages) * L::kStage;
      uint32_t dst[4];
      const uint16_t* src[4];
      int32_t ns[4];
#pragma unroll
      for (uint32_t j = 0; j < 4; j++) {
        dst[j] = to + (qch >> 3) * 8192 + swz((qrow + 16 * j) * 128 + (qch & 7) * 16);
        src[j] = qsrc + (int64_t)(tq[j] >= 0 ? tq[j] : 0) * lds;
        ns[j] = tq[j] >= 0 ? qn : 0;
      }
      fill8(dst, src, ns, qsrc, access);
#pragma unroll
      for (uint32_t j = 0; j < PN; j++) {
        const uint32_t r = prow + span * j;
        if (r < 64)
          cp16z(to + L::kQ + swz(r * (RP * 2) + pch * 16),
                pr + (int64_t)(tp[j] >= 0 ? tp[j] : 0) * RP + pch * 8, tp[j] >= 0);
      }
    };
    float acc[MF][RP / 8][4];
#pragma unroll
    for (int m = 0; m < MF; m++)
#pragma unroll
      for (int j = 0; j < RP / 8; j++)
        acc[m][j][0] = acc[m][j][1] = acc[m][j][2] = acc[m][j][3] = 0.f;
    __syncthreads();   // the piece before is done with the ring
    load_rows(0);
    for (uint32_t i = 0; i < kWStages - 1; i++) {
      if (i < mine) load_stage(i);
      if (i + 1 < mine) load_rows(i + 1);
      cp_commit();
    }
    for (uint32_t i = 0; i < mine; i++) {
      cp_wait<kWStages - 2>();
      __syncthreads();
      if (i + kWStages - 1 < mine) load_stage(i + kWStages - 1);
      if (i + kWStages < mine) load_rows(i + kWStages);
      cp_commit();
      const uint32_t qs = ring + (i % kWStages) * L::kStage, ps = qs + L::kQ;
#pragma unroll
      for (uint32_t kk = 0; kk < 4 / MF; kk++) {   // 16 rows of the batch
        const uint32_t kt = th * 2 + kk;
        uint32_t a[MF][4];
#pragma unroll
        for (int m = 0; m < MF; m++) {
          const uint32_t f = (fw * MF + m) * 16;
          ldsm4t(a[m], qs + (f >> 6) * 8192 +
                           swz((kt * 16 + (lane >> 4) * 8 + (lane & 7)) * 128 + (f & 63) * 2 +
                               ((lane >> 3) & 1) * 16));
        }
#pragma unroll
        for (int j = 0; j < RP / 16; j++) {
          uint32_t b[4];
          ldsm4t(b, ps + swz((kt * 16 + ((lane >> 3) & 1) * 8 + (lane & 7)) * (RP * 2) + j * 32 +
                             (lane >> 4) * 16));
#pragma unroll
          for (int m = 0; m < MF; m++) {
            mma16816(acc[m][2 * j], a[m][0], a[m][1], a[m][2], a[m][3], b[0], b[1]);
            mma16816(acc[m][2 * j + 1], a[m][0], a[m][1], a[m][2], a[m][3], b[2], b[3]);
          }
        }
      }
    }
    cp_wait<0>();
#pragma unroll
    for (int pass = 0; pass < MF; pass++) {   // join the two halves of every stage
      __syncthreads();
      if ((int)th == pass) {
#pragma unroll
        for (int m = 0; m < MF; m++)
#pragma unroll
          for (int j = 0; j < RP / 8; j++)
#pragma unroll
            for (int h = 0; h < 2; h++) {
              float2* d = reinterpret_cast<float2*>(
                  part + ((fw * MF + m) * 16 + h * 8 + g) * L::kLd + j * 8 + 2 * q);
              const float2 v = make_float2(acc[m][j][2 * h], acc[m][j][2 * h + 1]);
              *d = pass == 0 ? v : make_float2(d->x + v.x, d->y + v.y);
            }
      }
    }
    __syncthreads();
    bool write = true;
    uint32_t b0 = 0, b1 = 0;   // the blocks that share the piece, when several do
    if (mine < Q.stages) {
      float* const to = P.sums + (2 * (uint64_t)blockIdx.x + (Q.at != s_begin)) * (kFeat * RP);
      for (uint32_t e = tid * 2; e < kFeat * RP; e += kThreads * 2)
        __stcg(reinterpret_cast<float2*>(to + e),
               *reinterpret_cast<const float2*>(part + e / RP * L::kLd + e % RP));
      // the blocks of the piece's first and last stage
      const uint64_t p_last = Q.begin + Q.stages - 1;
      b0 = sh.owner(Q.begin);
      b1 = sh.owner(p_last);
      __threadfence();
      __syncthreads();
      if (tid == 0)
        sh_last = atomicInc(P.counters + (uint64_t)Q.adapter * slices + Q.slice, b1 - b0) == b1 - b0;
      __syncthreads();
      write = sh_last != 0;
      __threadfence();
    }
    if (write && mine < Q.stages) {   // the blocks' sums, in their order, many at once
      constexpr uint32_t U = RP >= 64 ? 8 : RP / 8;
      for (uint32_t e = tid * 4; e < kFeat * RP; e += kThreads * 4 * U) {
        float4 v[U];
#pragma unroll
        for (uint32_t u = 0; u < U; u++) v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
        for (uint32_t b = b0; b <= b1; b++) {   // a block's first piece, or its last
          const float* const from =
              P.sums + (2 * (uint64_t)b + (sh.begin(b) < Q.begin)) * (kFeat * RP) + e;
#pragma unroll
          for (uint32_t u = 0; u < U; u++) {
            const float4 w = __ldcg(reinterpret_cast<const float4*>(from + u * kThreads * 4));
            v[u].x += w.x;
            v[u].y += w.y;
            v[u].z += w.z;
            v[u].w += w.w;
          }
        }
#pragma unroll
        for (uint32_t u = 0; u < U; u++) {
          const uint32_t at = e + u * kThreads * 4;
          float2* const d = reinterpret_cast<float2*>(part + at / RP * L::kLd + at % RP);
          d[0] = make_float2(v[u].x, v[u].y);
          d[1] = make_float2(v[u].z, v[u].w);
        }
      }
      __syncthreads();
    }
    if (write) {
      for (uint32_t e = tid; e < kFeat * RP; e += kThreads) {
        // neighbours in memory to neighbouring threads: along the features for dA, the rank for dB
        const uint32_t fl = down ? e % kFeat : e / RP, r = down ? e / kFeat : e % RP;
        if (f0 + fl >= F || r >= A.rank) continue;
        const float v = part[fl * L::kLd + r];
        if (down)
          put_grad(A.gdown, (uint64_t)r * A.ld_gdown + f0 + fl, v, P.grad_f32, P.accumulate);
        else
          put_grad(A.gup, (uint64_t)(f0 + fl) * A.ld_gup + r, v, P.grad_f32, P.accumulate);
      }
    }
  }
}

// ------------------------------------------------------------------------------- host side
template <int RP>
cudaError_t launch_apply(bool small, bool vec, uint32_t tiles, uint32_t C, const ApplyArgs& P,
                         cudaStream_t s) {
  if constexpr (RP <= 64) {
    if (small)
      return launch(vec && P.vec_ups ? k_apply16<RP, true> : k_apply16<RP, false>, dim3(tiles * C),
                    kThreads, Apply16<RP>::kSmem, C, s, P);
  }
  return launch(vec ? k_apply64<RP, true> : k_apply64<RP, false>, dim3(tiles * C), kThreads,
                Apply64<RP>::kSmem, C, s, P);
}
template <int RP>
cudaError_t launch_expand(uint32_t grid, const ApplyArgs& P, cudaStream_t s) {
  return launch(k_expand<RP>, dim3(grid), kThreads, Expand<RP>::kSmem, 1, s, P);
}
template <int RP>
cudaError_t launch_wgrad(uint32_t grid, const WgradArgs& P, cudaStream_t s) {
  return launch(k_wgrad<RP>, dim3(grid), kThreads, Wgrad<RP>::kSmem, 1, s, P);
}

// Blocks of a cluster that share a tile: as many as the SMs hold at once, `slots` of them (`slots8`
// of clusters of 8, which not every corner of the GPU takes).
uint32_t cluster_for(uint64_t tiles, uint64_t slots, uint64_t slots8) {
  uint32_t c = 1;
  while (c < kMaxCluster && tiles * c * 2 <= (c == 4 ? slots8 : slots)) c *= 2;
  return c;
}

// Low and the second product are two launches from this many bytes of rows on.  One launch keeps
// low on the SM and is ahead below (1024 rows of 4096 x 4096, rank 16: 10.7 us against 14.9 us);
// two have better kernels for each half (16384 rows: 84 us against 75 us; of rank 64 and 4096 x
// 11008: 193 us against 171 us).
constexpr uint64_t kSplitBytes = 200000000;
uint64_t row_bytes(uint32_t K, uint32_t N) { return 2 * ((uint64_t)K + 2 * (uint64_t)N); }

uint32_t tile_bound(uint32_t rows, uint32_t k, uint32_t high) {
  const uint64_t b = (uint64_t)rows / high + k;
  return (uint32_t)(b < rows ? b : rows);
}
// ... as many as to expect: an adapter's last tile is there in two cases of three.
uint32_t tile_guess(uint32_t rows, uint32_t k, uint32_t high) {
  return tile_bound(rows, 2 * k / 3 + 1, high);
}

int apply(uint32_t RP, const bo_adapter_rows* R, ApplyArgs& P, int sms, cudaStream_t s) {
  const uint32_t rows = R->rows, k = R->k;
  P.perm = R->d_perm;
  P.status = R->d_status;
  const bool vec = P.vec_x && P.vec_factors && (!P.y || P.vec_y);
  if (vec && P.low && rows * row_bytes(P.K, P.N) >= kSplitBytes) {
    const uint32_t tiles = tile_bound(rows, k, 128);
    P.tiles = static_cast<const Tile*>(R->d_tiles[2]);
    P.ntiles = R->d_ntiles + 2;
    const int rc = check(tc_low(RP, tiles, cluster_for(tiles, sms, sms), P, s));
    if (rc || !P.y) return rc;
    P.tiles = static_cast<const Tile*>(R->d_tiles[1]);
    P.ntiles = R->d_ntiles + 1;
    const uint32_t grid = (RP <= 64 ? 2 : 1) * sms;
    switch (RP) {
      case 16: return check(launch_expand<16>(grid, P, s));
      case 32: return check(launch_expand<32>(grid, P, s));
      case 64: return check(launch_expand<64>(grid, P, s));
      default: return check(launch_expand<128>(grid, P, s));
    }
  }
  // Tiles of 16 rows have the shorter way to a result, tiles of 64 read the factors less often and
  // carry less in registers.  Measured at two widths (us, tiles of 16 / of 64; the bounds are where most
  // of these change sides, and miss by up to 6% beside them: rank 64, 512 rows of 8):
  //   rank 16, 4096 x 4096:   16 rows of 16 adapters 5.1 / 8.8, 512 of 8 6.1 / 8.0, 1024 of 8 9.3 / 10.6,
  //                           1024 of 64 9.7 / 15.0, 2048 of 64 19.9 / 18.6
  //   rank 64, 4096 x 11008:  64 of 1 11.7 / 17.8, 64 of 64 31.6 / 41.4, 256 of 32 22.6 / 26.3,
  //                           512 of 8 20.5 / 19.3, 1024 of 32 34 / 29
  //   rank 128, 4096 x 4096:  1 row 18.6 / 16.0, 64 of 64 114 / 48
  // and, where rows do not end with whole words, of rank 16 as above up to 512 rows, of rank 64
  //                           128 of 1 16.0 / 19.1, 64 of 64 47 / 41, 256 of 8 20 / 18.
  const uint32_t few = RP <= 32 && vec && P.vec_ups ? 1024 : 512;
  const bool small = RP == 128                        ? false
                     : RP <= 32 || (vec && P.vec_ups) ? rows <= few || rows / k < 24
                                                      : tile_guess(rows, k, 16) <= 16;
  const uint32_t high = small ? 16 : 64;
  const uint32_t tiles = tile_bound(rows, k, high), guess = tile_guess(rows, k, high);
  P.tiles = static_cast<const Tile*>(R->d_tiles[small ? 0 : 1]);
  P.ntiles = R->d_ntiles + (small ? 0 : 1);
  // Blocks of 64 rows fit twice on an SM (of rank 128 once), of 16 rows three times.  Past that a
  // second round waits for the first: 64 tiles of 16 rows with 4 / 8 blocks each take 8.5 / 12.3 us,
  // 32 of them 8.0 / 6.6 us; 64 tiles of 64 rows with 2 / 4 / 8 28.5 / 20.2 / 25.1 us (rank 16).
  const uint64_t n = (uint64_t)sms;
  const uint32_t C = small       ? cluster_for(guess, 3 * n, n * 12 / 5)
                     : RP == 128 ? cluster_for(guess, n, n * 2 / 3)
                                 : cluster_for(guess, 2 * n, 2 * n);
  switch (RP) {
    case 16: return check(launch_apply<16>(small, vec, tiles, C, P, s));
    case 32: return check(launch_apply<32>(small, vec, tiles, C, P, s));
    case 64: return check(launch_apply<64>(small, vec, tiles, C, P, s));
    default: return check(launch_apply<128>(small, vec, tiles, C, P, s));
  }
}

struct RowsLayout {
  uint64_t counts, offsets, blocks, ntiles, perm, tiles16, tiles64, tiles128, total;
};
bool rows_layout(uint32_t rows, uint32_t k, RowsLayout& L) {
  if (k == 0 || k > BO_ADAPTER_MAX_COUNT || rows > BO_ADAPTER_MAX_ROWS) return false;
  uint64_t off = 0;
  auto take = [&](uint64_t bytes) {
    const uint64_t at = off;
    off = up(off + bytes, 256);
    return at;
  };
  L.counts = take((uint64_t)k * 4);
  L.offsets = take(((uint64_t)k + 1) * 4);
  L.blocks = take(((uint64_t)k + 1) * 4);
  L.ntiles = take(12);
  L.perm = take((uint64_t)rows * 4);
  L.tiles16 = take(((uint64_t)rows / 16 + k) * sizeof(Tile));
  L.tiles64 = take(((uint64_t)rows / 64 + k) * sizeof(Tile));
  L.tiles128 = take(((uint64_t)rows / 128 + k) * sizeof(Tile));
  L.total = off;
  return true;
}

bool valid(const bo_adapter_set* s) {
  return s && s->d_table && s->k > 0 && s->hidden > 0 && s->out > 0 &&
         (s->rank == 16 || s->rank == 32 || s->rank == 64 || s->rank == 128);
}
bool valid(const bo_adapter_rows* r) {
  return r && r->d_perm && r->d_offsets && r->d_blocks && r->d_tiles[0] && r->d_tiles[1] &&
         r->d_tiles[2] && r->d_ntiles;
}
bool wide(const void* p, uint64_t ld, uint64_t width) {
  return aligned(p, 16) && ld % 8 == 0 && width % 8 == 0;
}
// Whether a set's gradients lie apart from one another and from its factors.  Sorts the regions.  Of
// matrices that lie between one another's rows every pair is looked at, a few million at most (all
// of 65535 adapters' factors as columns of one buffer would take a minute).
bool apart(Region* r, uint64_t n) {
  std::sort(r, r + n, [](const Region& a, const Region& b) { return a.at < b.at; });
  uint64_t left = 1u << 24;
  for (uint64_t i = 0; i < n; i++)
    for (uint64_t j = i + 1; j < n && r[j].at < r[i].end() && left; j++, left--)
      if ((r[i].write || r[j].write) && meet(r[i], r[j])) return false;
  return true;
}
uint64_t up8(uint64_t x) { return (x + 7) / 8 * 8; }

uint32_t wgrad_slices(const bo_adapter_set* set) {
  return (set->hidden + kFeat - 1) / kFeat + (set->out + kFeat - 1) / kFeat;
}
constexpr uint32_t kMaxSms = 256;   // (that a workspace is sized for)
struct BackwardLayout {
  uint64_t dlow, table, counters, sums, buf, total;
};
BackwardLayout backward_layout(const bo_adapter_set* set, uint32_t rows) {
  BackwardLayout L;
  L.dlow = 0;
  L.table = up((uint64_t)rows * set->rank * 2, 256);
  L.counters = L.table + up((uint64_t)set->k * sizeof(DevAdapter), 256);
  L.sums = L.counters + up((uint64_t)set->k * wgrad_slices(set) * 4, 256);
  L.buf = L.sums + (uint64_t)2 * 2 * kMaxSms * kFeat * set->rank * 4;
  L.total = L.buf + up((uint64_t)set->k * set->rank * ((uint64_t)set->hidden + up8(set->out)) * 2, 256);
  return L;
}

}  // namespace
}  // namespace bo

using namespace bo;

extern "C" {

uint64_t bo_adapter_set_size(uint32_t k) {
  return k == 0 || k > BO_ADAPTER_MAX_COUNT ? 0 : up((uint64_t)k * sizeof(DevAdapter), 256);
}

int bo_adapter_set_init(const bo_adapter* h_items, uint32_t k, uint32_t hidden, uint32_t out,
                        uint32_t grad_dtype, void* d_set, uint64_t set_bytes,
                        bo_adapter_set* h_out, void* stream) {
  const uint64_t need = bo_adapter_set_size(k);
  if (!h_items || !h_out || need == 0 || !d_set || !aligned(d_set, 256) || set_bytes < need ||
      grad_dtype > BO_FP32 || hidden == 0 || hidden > BO_ADAPTER_MAX_WIDTH || out == 0 ||
      out > BO_ADAPTER_MAX_WIDTH)
    return BD_ERR_INVALID_ARG;
  std::unique_ptr<DevAdapter[]> dev(new (std::nothrow) DevAdapter[k]);
  std::unique_ptr<Region[]> memory(new (std::nothrow) Region[4 * (size_t)k]);
  if (!dev || !memory) return BD_ERR_INVALID_ARG;
  uint64_t regions = 0;
  const uintptr_t gsize = grad_dtype == BO_FP32 ? 4 : 2;
  uint32_t most = 1;
  const bool grads = h_items[0].d_grad_down != nullptr;
  bool all_wide = true, ups_whole = true;
  for (uint32_t i = 0; i < k; i++) {
    const bo_adapter& a = h_items[i];
    if (!a.d_down || !a.d_up || !aligned(a.d_down, 2) || !aligned(a.d_up, 2) || a.rank < 1 ||
        a.rank > BO_ADAPTER_MAX_RANK || a.ld_down < hidden || a.ld_up < a.rank ||
        a.ld_down > (1ull << 40) || a.ld_up > (1ull << 40))
      return BD_ERR_INVALID_ARG;
    if (!a.d_grad_down == grads || !a.d_grad_up == grads) return BD_ERR_INVALID_ARG;
    if (grads && (!aligned(a.d_grad_down, gsize) || !aligned(a.d_grad_up, gsize) ||
                  a.ld_grad_down < hidden || a.ld_grad_up < a.rank || a.ld_grad_down > (1ull << 40) ||
                  a.ld_grad_up > (1ull << 40)))
      return BD_ERR_INVALID_ARG;
    if (grads) {
      memory[regions++] = Region(a.d_down, a.rank, a.ld_down, hidden);
      memory[regions++] = Region(a.d_up, out, a.ld_up, a.rank);
      memory[regions++] = Region(a.d_grad_down, a.rank, a.ld_grad_down, hidden, gsize);
      memory[regions++] = Region(a.d_grad_up, out, a.ld_grad_up, a.rank, gsize);
      memory[regions - 2].write = memory[regions - 1].write = true;
    }
    DevAdapter& d = dev[i];
    d.down = a.d_down;
    d.up = a.d_up;
    d.ld_down = a.ld_down;
    d.ld_up = a.ld_up;
    d.gdown = a.d_grad_down;
    d.gup = a.d_grad_up;
    d.ld_gdown = a.ld_grad_down;
    d.ld_gup = a.ld_grad_up;
    d.rank = a.rank;
    d.scale = a.scale;
    d.vec_down = wide(a.d_down, a.ld_down, hidden);
    d.vec_up = wide(a.d_up, a.ld_up, 8);   // (a rank's last 16 bytes are read in part)
    d.vec_gup = a.d_grad_up && wide(a.d_grad_up, a.ld_grad_up, a.rank);
    d.pad[0] = d.pad[1] = d.pad[2] = 0;
    if (!d.vec_down) all_wide = false;
    if (!d.vec_up || a.rank % 8 != 0) ups_whole = false;
    if (a.rank > most) most = a.rank;
  }
  if (!apart(memory.get(), regions)) return BD_ERR_INVALID_ARG;
  int device = 0;
  int rc = check(cudaGetDevice(&device));
  if (rc) return rc;
  rc = check(upload(dev.get(), (uint64_t)k * sizeof(DevAdapter), d_set,
                    static_cast<cudaStream_t>(stream)));
  if (rc) return rc;
  h_out->rank = most <= 16 ? 16 : most <= 32 ? 32 : most <= 64 ? 64 : 128;
  h_out->d_table = d_set;
  h_out->k = k;
  h_out->hidden = hidden;
  h_out->out = out;
  h_out->grad_dtype = grad_dtype;
  h_out->has_grads = grads;
  h_out->wide = (all_wide ? 1u : 0u) | (ups_whole ? 2u : 0u);
  h_out->device = device;
  return BD_OK;
}

uint64_t bo_adapter_rows_size(uint32_t rows, uint32_t k) {
  RowsLayout L;
  return rows_layout(rows, k, L) ? L.total : 0;
}

int bo_adapter_rows_init(const int32_t* d_index, uint32_t rows, uint32_t k, void* d_rows,
                         uint64_t rows_bytes, bo_adapter_rows* h_out, int32_t* d_status,
                         void* stream) {
  RowsLayout L;
  if (!h_out || !rows_layout(rows, k, L) || !d_rows || !aligned(d_rows, 256) ||
      rows_bytes < L.total || (rows > 0 && (!d_index || !aligned(d_index, 4))) ||
      (d_status && !aligned(d_status, 4)) || overlaps(d_index, (uint64_t)rows * 4, d_rows, L.total))
    return BD_ERR_INVALID_ARG;
  uint8_t* p = static_cast<uint8_t*>(d_rows);
  int32_t* counts = reinterpret_cast<int32_t*>(p + L.counts);
  int32_t* offsets = reinterpret_cast<int32_t*>(p + L.offsets);
  int32_t* blocks = reinterpret_cast<int32_t*>(p + L.blocks);
  int32_t* ntiles = reinterpret_cast<int32_t*>(p + L.ntiles);
  int32_t* perm = reinterpret_cast<int32_t*>(p + L.perm);
  Tile* t16 = reinterpret_cast<Tile*>(p + L.tiles16);
  Tile* t64 = reinterpret_cast<Tile*>(p + L.tiles64);
  Tile* t128 = reinterpret_cast<Tile*>(p + L.tiles128);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int device = 0;
  int rc = check(cudaGetDevice(&device));
  if (rc) return rc;
  rc = check(launch(k_rows_count, dim3(k), kThreads, 0, 1, s, d_index, rows, k, counts, d_status));
  if (rc) return rc;
  rc = check(launch(k_rows_place, dim3(k), kThreads, 0, 1, s, d_index, rows, k, counts, perm, offsets,
                    t16, t64, t128, ntiles, blocks));
  if (rc) return rc;
  h_out->d_perm = perm;
  h_out->d_offsets = offsets;
  h_out->d_blocks = blocks;
  h_out->d_tiles[0] = t16;
  h_out->d_tiles[1] = t64;
  h_out->d_tiles[2] = t128;
  h_out->d_status = d_status;
  h_out->d_ntiles = ntiles;
  h_out->rows = rows;
  h_out->k = k;
  h_out->device = device;
  return BD_OK;
}

int bo_adapter_forward(const bo_adapter_set* set, const bo_adapter_rows* rows, const uint16_t* d_x,
                       uint64_t ldx, uint16_t* d_y, uint64_t ldy, uint16_t* d_low, void* stream) {
  if (!valid(set) || !valid(rows) || rows->k != set->k || rows->device != set->device)
    return BD_ERR_INVALID_ARG;
  if (rows->rows == 0) return BD_OK;
  if (!d_x || !d_y || !aligned(d_x, 2) || !aligned(d_y, 2) || ldx < set->hidden ||
      ldy < set->out || ldx > (1ull << 40) || ldy > (1ull << 40) || !aligned(d_low, 16) ||
      (!d_low && rows->rows >= bo_adapter_low_rows(set)))
    return BD_ERR_INVALID_ARG;
  const Region x(d_x, rows->rows, ldx, set->hidden), y(d_y, rows->rows, ldy, set->out);
  const Region low(d_low, rows->rows, set->rank, set->rank);
  if (meet(x, y) || meet(low, y) || meet(low, x)) return BD_ERR_INVALID_ARG;
  int sms = 0;
  if (const int rc = sm_count(set->device, sms)) return rc;
  ApplyArgs P = {};
  P.table = static_cast<const DevAdapter*>(set->d_table);
  P.x = d_x;
  P.ldx = ldx;
  P.y = d_y;
  P.ldy = ldy;
  P.low = d_low;
  P.K = set->hidden;
  P.N = set->out;
  P.vec_x = wide(d_x, ldx, set->hidden);
  P.vec_y = wide(d_y, ldy, set->out);
  P.vec_factors = set->wide & 1;
  P.vec_ups = set->wide >> 1 & 1;
  P.stall = set->wide & BO_ADAPTER_DEBUG_STALL;
  return apply(set->rank, rows, P, sms, static_cast<cudaStream_t>(stream));
}

uint64_t bo_adapter_backward_workspace_size(const bo_adapter_set* set, uint32_t rows) {
  return valid(set) && rows <= BO_ADAPTER_MAX_ROWS ? backward_layout(set, rows).total : 0;
}

int bo_adapter_backward(const bo_adapter_set* set, const bo_adapter_rows* rows,
                        const uint16_t* d_x, uint64_t ldx, const uint16_t* d_dy, uint64_t lddy,
                        const uint16_t* d_low, uint16_t* d_dx, uint64_t lddx, int32_t accumulate,
                        void* d_ws, uint64_t ws_bytes, void* stream) {
  if (!valid(set) || !valid(rows) || rows->k != set->k || rows->device != set->device)
    return BD_ERR_INVALID_ARG;
  const BackwardLayout L = backward_layout(set, rows->rows);
  if (!d_ws || !aligned(d_ws, 256) || ws_bytes < L.total) return BD_ERR_INVALID_ARG;
  if (rows->rows > 0) {
    if (!d_x || !d_dy || !d_low || !aligned(d_x, 2) || !aligned(d_dy, 2) || !aligned(d_dx, 2) ||
        !aligned(d_low, 16) || ldx < set->hidden || lddy < set->out ||
        (d_dx && lddx < set->hidden) || ldx > (1ull << 40) || lddy > (1ull << 40) ||
        (d_dx && lddx > (1ull << 40)))
      return BD_ERR_INVALID_ARG;
    const Region x(d_x, rows->rows, ldx, set->hidden), dy(d_dy, rows->rows, lddy, set->out);
    const Region low(d_low, rows->rows, set->rank, set->rank), ws(d_ws, 1, L.total, L.total, 1);
    const Region dx(d_dx, rows->rows, lddx, set->hidden);
    if (meet(dx, x) || meet(dx, dy) || meet(dx, low) || meet(ws, x) || meet(ws, dy) ||
        meet(ws, low) || meet(ws, dx))
      return BD_ERR_INVALID_ARG;
  }
  int sms = 0;
  if (const int rc = sm_count(set->device, sms)) return rc;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  uint8_t* w = static_cast<uint8_t*>(d_ws);
  uint16_t* dlow = reinterpret_cast<uint16_t*>(w + L.dlow);
  DevAdapter* swapped = reinterpret_cast<DevAdapter*>(w + L.table);
  uint16_t* buf = reinterpret_cast<uint16_t*>(w + L.buf);
  const uint32_t out8 = (uint32_t)up8(set->out);
  uint32_t* counters = reinterpret_cast<uint32_t*>(w + L.counters);
  const uint32_t slices = wgrad_slices(set);
  const dim3 turn_grid((set->hidden + kTF - 1) / kTF + (out8 + kTF - 1) / kTF, set->k);
  auto* turn = set->rank == 16 ? k_transpose<16> : set->rank == 32 ? k_transpose<32>
               : set->rank == 64 ? k_transpose<64> : k_transpose<128>;
  int rc = check(launch(turn, turn_grid, kThreads, 0, 1, s, static_cast<const DevAdapter*>(set->d_table),
                        set->hidden, set->out, out8, buf, swapped, counters, slices));
  if (rc) return rc;
  if (rows->rows > 0) {
    ApplyArgs P = {};
    P.table = swapped;
    P.x = d_dy;
    P.ldx = lddy;
    P.y = d_dx;
    P.ldy = lddx;
    P.low = dlow;
    P.K = set->out;
    P.N = set->hidden;
    P.vec_x = wide(d_dy, lddy, set->out);
    P.vec_y = d_dx && wide(d_dx, lddx, set->hidden);
    P.vec_factors = P.vec_ups = 1;
    P.stall = set->wide & BO_ADAPTER_DEBUG_STALL;
    if ((rc = apply(set->rank, rows, P, sms, s))) return rc;
  }
  if (!set->has_grads) return BD_OK;
  WgradArgs G = {};
  G.table = static_cast<const DevAdapter*>(set->d_table);
  G.perm = rows->d_perm;
  G.offsets = rows->d_offsets;
  G.x = d_x;
  G.ldx = ldx;
  G.dy = d_dy;
  G.lddy = lddy;
  G.low = d_low;
  G.dlow = dlow;
  if (rows->rows == 0) G.x = G.dy = G.low = dlow;   // (nothing is read, but pointers are formed)
  G.hidden = set->hidden;
  G.out = set->out;
  G.vec_x = wide(d_x, ldx, set->hidden);
  G.vec_dy = wide(d_dy, lddy, set->out);
  G.grad_f32 = set->grad_dtype == BO_FP32;
  G.accumulate = accumulate != 0;
  G.blocks = rows->d_blocks;
  G.sums = reinterpret_cast<float*>(w + L.sums);
  G.counters = counters;
  G.k = set->k;
  const bool vec = G.vec_x && G.vec_dy;
  G.status = rows->d_status;
  G.stall = set->wide & BO_ADAPTER_DEBUG_STALL;
  const uint64_t stages = ((uint64_t)rows->rows / 64 + set->k) * slices;   // at most
  const uint64_t slots = sms < (int)kMaxSms ? sms : (int)kMaxSms;
  if (vec && rows->rows > 0)   // a block an SM
    return check(tc_wgrad(set->rank, (uint32_t)(stages < slots ? stages : slots), G, s));
  const uint32_t grid = (uint32_t)(stages < 2 * slots ? stages : 2 * slots);
  switch (set->rank) {
    case 16: return check(launch_wgrad<16>(grid, G, s));
    case 32: return check(launch_wgrad<32>(grid, G, s));
    case 64: return check(launch_wgrad<64>(grid, G, s));
    default: return check(launch_wgrad<128>(grid, G, s));
  }
}

uint32_t bo_adapter_low_rows(const bo_adapter_set* set) {
  if (!valid(set)) return 0;
  const uint64_t b = row_bytes(set->hidden, set->out);
  const uint64_t n = (kSplitBytes + b - 1) / b;
  return (uint32_t)(n < BO_ADAPTER_MAX_ROWS ? n : BO_ADAPTER_MAX_ROWS);
}

}  // extern "C"
