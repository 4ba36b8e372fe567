// bo_adapter.cu -- low-rank adapters of many requests beside a shared projection: forward and
// backward (include/ops/bf16ops.h has the formulas).
//
// At ranks up to 128 a row's products take 2 r (hidden + out) operations for 2 hidden + 4 out
// bytes: below 100 operations a byte against the 280 that the tensor cores and HBM balance at,
// so every kernel here is built to stream x, y and the gradients once, through registers or a
// ring of shared-memory tiles, with mma.sync on BF16 tiles beside it.
//
//   k_rows_*      group the rows of a batch by adapter (once per model step)
//   k_apply16     one launch for low = s A x and y += B low over tiles of 16 rows: the serving
//                 form, factors straight from global memory into the fragments
//   k_apply64     the same over tiles of 64 rows, factors and x through shared memory
//   k_transpose   the factors' transposes, with which the backward pass is the forward kernel:
//                 dlow = s B^T dy, dx += A^T dlow
//   k_wgrad       dA and dB, sums over the rows of an adapter
//
// A tile of rows belongs to one adapter.  The thread blocks of a cluster share a tile: each takes
// a slice of the first product's long sum, the slices' sums meet through distributed shared
// memory in a fixed order, and each block then writes a slice of the second product's columns.
#include <cooperative_groups.h>
#include <cstring>
#include <memory>
#include <new>

#include "bo_internal.cuh"

namespace cg = cooperative_groups;

namespace bo {
namespace {

constexpr uint32_t kThreads = 256;   // eight warps
constexpr uint32_t kMaxCluster = 8;

struct alignas(16) DevAdapter {
  const uint16_t* down;
  const uint16_t* up;
  uint64_t ld_down, ld_up;
  void* gdown;
  void* gup;
  uint64_t ld_gdown, ld_gup;
  uint32_t rank;
  float scale;
  uint32_t vec_down, vec_up;   // rows may be read 16 bytes at a time
};
static_assert(sizeof(DevAdapter) % 16 == 0, "uploaded in 16-byte words");

struct Tile {
  int32_t adapter, start, count, pad;
};

// ------------------------------------------------------------------------ grouping the rows
// One block per adapter counts its rows, then one block per adapter places them in order: the
// grouping is stable, so every later sum over an adapter's rows has one order.
__global__ void __launch_bounds__(kThreads) k_rows_count(const int32_t* __restrict__ index,
                                                         uint32_t rows, uint32_t k,
                                                         int32_t* __restrict__ counts,
                                                         int32_t* __restrict__ status) {
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
    Tile* __restrict__ tiles16, Tile* __restrict__ tiles64, int32_t* __restrict__ ntiles) {
  __shared__ int32_t sh[kThreads / 32];
  const uint32_t a = blockIdx.x;
  int32_t c0 = 0, c16 = 0, c64 = 0;
  for (uint32_t b = threadIdx.x; b < a; b += kThreads) {
    const int32_t c = counts[b];
    c0 += c;
    c16 += (c + 15) / 16;
    c64 += (c + 63) / 64;
  }
  c0 = block_sum(c0, sh);
  c16 = block_sum(c16, sh);
  c64 = block_sum(c64, sh);
  const int32_t mine = counts[a];
  const int32_t n16 = (mine + 15) / 16, n64 = (mine + 63) / 64;
  if (threadIdx.x == 0) {
    offsets[a] = c0;
    if (a == k - 1) {
      offsets[k] = c0 + mine;
      ntiles[0] = c16 + n16;
      ntiles[1] = c64 + n64;
    }
  }
  for (int32_t i = threadIdx.x; i < n16; i += kThreads)
    tiles16[c16 + i] = Tile{(int32_t)a, c0 + 16 * i, min(16, mine - 16 * i), 0};
  for (int32_t i = threadIdx.x; i < n64; i += kThreads)
    tiles64[c64 + i] = Tile{(int32_t)a, c0 + 64 * i, min(64, mine - 64 * i), 0};
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
__device__ __forceinline__ uint32_t smem_addr(const void* p) {
  return (uint32_t)__cvta_generic_to_shared(p);
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
__device__ __forceinline__ void cp16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
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

// Eight values from p, of which the first n exist (n <= 0: none); the others are 0.
__device__ __forceinline__ uint4 gather8(const uint16_t* p, int32_t n) {
  uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
  for (int j = 0; j < 8; j++)
    if (j < n) w[j >> 1] |= (uint32_t)p[j] << (16 * (j & 1));
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ uint4 load8(const uint16_t* p, int32_t n, bool vec) {
  if (vec) return n > 0 ? ld16(p) : make_uint4(0, 0, 0, 0);   // (n is a multiple of 8)
  return gather8(p, n);
}
// The same for the factors, which other blocks read too.
__device__ __forceinline__ uint4 load8w(const uint16_t* p, int32_t n, bool vec) {
  if (vec) return n > 0 ? __ldg(reinterpret_cast<const uint4*>(p)) : make_uint4(0, 0, 0, 0);
  return gather8(p, n);
}
// ... into shared memory
__device__ __forceinline__ void fill8(uint32_t dst, const uint16_t* p, int32_t n, bool vec) {
  if (vec && n > 0) cp16(dst, p);
  else sts16(dst, vec ? make_uint4(0, 0, 0, 0) : gather8(p, n));
}
__device__ __forceinline__ void store8(uint16_t* p, uint4 v, int32_t n, bool vec) {
  if (vec) {
    if (n > 0) *reinterpret_cast<uint4*>(p) = v;
    return;
  }
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int j = 0; j < 8; j++)
    if (j < n) p[j] = (uint16_t)(w[j >> 1] >> (16 * (j & 1)));
}
// y + acc, rounded once, for a packed pair
__device__ __forceinline__ uint32_t add_pair(uint32_t y, float a, float b) {
  return pack_bf16(bf16_lo(y) + a, bf16_hi(y) + b);
}

// Byte address in a tile of rows that fill 128-byte lines: the 16-byte slots of a line are
// permuted by the line's number, so that eight consecutive rows at one column (ldmatrix) fall
// into different banks.
__device__ __forceinline__ uint32_t swz(uint32_t byte) { return byte ^ (((byte >> 7) & 7) << 4); }

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

struct ApplyArgs {
  const DevAdapter* table;
  const Tile* tiles;
  const int32_t* ntiles;
  const int32_t* perm;
  const uint16_t* x;      // rows of K values
  uint64_t ldx;
  uint16_t* y;            // rows of N values, may be NULL
  uint64_t ldy;
  uint16_t* low;          // may be NULL
  uint32_t K, N;
  uint32_t vec_x, vec_y;
};

// ---------------------------------------------------------------------- tiles of 16 rows
// The sum's index may be dealt to the threads in any order as long as both factors agree, so a
// thread reads 16 bytes (eight consecutive values) of each row and feeds them to two mma steps:
// the fragments come straight from global memory, every load of a warp independent of the
// others.
template <int RP>
__global__ void __launch_bounds__(kThreads) k_apply16(const ApplyArgs P) {
  extern __shared__ __align__(1024) uint8_t smem[];
  float* const red = reinterpret_cast<float*>(smem);                 // [8][16][RP]
  float* const part = red + 8 * 16 * RP;                             // [16][RP]
  uint16_t* const us = reinterpret_cast<uint16_t*>(part + 16 * RP);  // [16][RP + 8]
  const cg::cluster_group cluster = cg::this_cluster();
  const uint32_t C = cluster.num_blocks(), c = cluster.block_rank();
  const uint32_t tile = blockIdx.x / C;
  if (tile >= (uint32_t)*P.ntiles) return;   // (the whole cluster)
  const Tile T = P.tiles[tile];
  const DevAdapter A = P.table[T.adapter];
  const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, q = lane & 3;
  const int32_t r0 = (int32_t)g < T.count ? P.perm[T.start + g] : -1;
  const int32_t r1 = (int32_t)g + 8 < T.count ? P.perm[T.start + g + 8] : -1;
  const int32_t rank = (int32_t)A.rank;

  float acc[RP / 8][4];
#pragma unroll
  for (int j = 0; j < RP / 8; j++) acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0.f;
  const uint32_t first = c * 8 + warp, step = C * 8;
#pragma unroll(RP <= 32 ? 4 : 1)
  for (uint32_t kc = first; kc * 32 < P.K; kc += step) {
    const uint32_t k = kc * 32 + 8 * q;
    const int32_t n = (int32_t)P.K - (int32_t)k;
    const uint4 xa = load8(P.x + (int64_t)r0 * P.ldx + k, r0 >= 0 ? n : 0, P.vec_x);
    const uint4 xb = load8(P.x + (int64_t)r1 * P.ldx + k, r1 >= 0 ? n : 0, P.vec_x);
#pragma unroll
    for (int j = 0; j < RP / 8; j++) {
      const int32_t row = j * 8 + g;
      const uint4 b = load8w(A.down + (uint64_t)row * A.ld_down + k, row < rank ? n : 0, A.vec_down);
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
    for (uint32_t w = 0; w < 8; w++) s += red[w * 16 * RP + e];
    part[e] = s;
  }
  cluster.sync();
  for (uint32_t e = threadIdx.x; e < 16 * RP; e += kThreads) {
    float s = 0.f;
    for (uint32_t b = 0; b < C; b++) s += cluster.map_shared_rank(part, b)[e];
    const int32_t row = e / RP, col = e % RP;
    // columns past the rank are 0 whatever x holds (an infinity times a padded 0 is not)
    const uint16_t u = col < rank ? (uint16_t)pack_bf16(s * A.scale, 0.f) : 0;
    us[row * (RP + 8) + col] = u;
    if (P.low && c == 0 && row < T.count)
      P.low[(int64_t)P.perm[T.start + row] * RP + col] = u;
  }
  __syncthreads();
  cg::cluster_group::arrival_token token = cluster.barrier_arrive();

  if (P.y) {
    for (uint32_t gc = first; gc * 32 < P.N; gc += step) {
      const uint32_t col = gc * 32 + 8 * q;
      const int32_t n = (int32_t)P.N - (int32_t)col;
      uint16_t* const p0 = P.y + (int64_t)r0 * P.ldy + col;
      uint16_t* const p1 = P.y + (int64_t)r1 * P.ldy + col;
      const uint4 y0 = load8(p0, r0 >= 0 ? n : 0, P.vec_y);
      const uint4 y1 = load8(p1, r1 >= 0 ? n : 0, P.vec_y);
      float d[4][4];
#pragma unroll
      for (int j = 0; j < 4; j++) d[j][0] = d[j][1] = d[j][2] = d[j][3] = 0.f;
      constexpr int KS = RP >= 32 ? 32 : 16;
#pragma unroll
      for (int ks = 0; ks < RP / KS; ks++) {
        if (ks * KS >= rank) break;
#pragma unroll
        for (int j = 0; j < 4; j++) {
          const uint32_t o = gc * 32 + dealt(g, j);
          if (KS == 32) {
            const int32_t k = ks * 32 + 8 * q;
            const uint4 a = *reinterpret_cast<const uint4*>(us + g * (RP + 8) + k);
            const uint4 b = *reinterpret_cast<const uint4*>(us + (g + 8) * (RP + 8) + k);
            const uint4 w = load8w(A.up + (uint64_t)o * A.ld_up + k, o < P.N ? rank - k : 0, A.vec_up);
            mma16816(d[j], a.x, b.x, a.y, b.y, w.x, w.y);
            mma16816(d[j], a.z, b.z, a.w, b.w, w.z, w.w);
          } else {
            const int32_t k = 4 * q;   // four values a thread: one mma step
            const uint2 a = *reinterpret_cast<const uint2*>(us + g * (RP + 8) + k);
            const uint2 b = *reinterpret_cast<const uint2*>(us + (g + 8) * (RP + 8) + k);
            uint2 w = make_uint2(0, 0);
            const uint16_t* src = A.up + (uint64_t)o * A.ld_up + k;
            if (o < P.N && k < rank) {
              if (A.vec_up) {
                w = __ldg(reinterpret_cast<const uint2*>(src));
              } else {
                const uint4 t = gather8(src, min(rank - k, 4));
                w = make_uint2(t.x, t.y);
              }
            }
            mma16816(d[j], a.x, b.x, a.y, b.y, w.x, w.y);
          }
        }
      }
      if (r0 >= 0)
        store8(p0, make_uint4(add_pair(y0.x, d[0][0], d[0][1]), add_pair(y0.y, d[1][0], d[1][1]),
                              add_pair(y0.z, d[2][0], d[2][1]), add_pair(y0.w, d[3][0], d[3][1])),
               n, P.vec_y);
      if (r1 >= 0)
        store8(p1, make_uint4(add_pair(y1.x, d[0][2], d[0][3]), add_pair(y1.y, d[1][2], d[1][3]),
                              add_pair(y1.z, d[2][2], d[2][3]), add_pair(y1.w, d[3][2], d[3][3])),
               n, P.vec_y);
    }
  }
  cluster.barrier_wait(std::move(token));   // the others may still read `part`
}

// ---------------------------------------------------------------------- tiles of 64 rows
constexpr uint32_t kBK = 64;     // values of the first sum per stage
constexpr uint32_t kBN = 128;    // columns of the second product per step
constexpr uint32_t kStages = 4;

template <int RP>
struct Apply64 {
  static constexpr uint32_t kXBytes = 64 * kBK * 2, kWBytes = RP * kBK * 2;
  static constexpr uint32_t kStage = kXBytes + kWBytes;
  static constexpr uint32_t kRing = kStages * kStage;
  static constexpr uint32_t kPart = 64 * RP * 4;               // over the ring, after the sum
  static constexpr uint32_t kUp = kBN * RP * 2;                // two of them
  static constexpr uint32_t kULd = RP + 8;
  static constexpr uint32_t kU = 64 * kULd * 2;
  static constexpr uint32_t kFirst = kRing > kPart + 2 * kUp ? kRing : kPart + 2 * kUp;
  static constexpr uint32_t kSmem = kFirst + kU + 64 * 4;
};

template <int RP>
__global__ void __launch_bounds__(kThreads) k_apply64(const ApplyArgs P) {
  using L = Apply64<RP>;
  extern __shared__ __align__(1024) uint8_t smem[];
  float* const part = reinterpret_cast<float*>(smem);
  uint8_t* const upt = smem + L::kPart;
  uint16_t* const us = reinterpret_cast<uint16_t*>(smem + L::kFirst);
  int32_t* const srow = reinterpret_cast<int32_t*>(smem + L::kFirst + L::kU);
  const cg::cluster_group cluster = cg::this_cluster();
  const uint32_t C = cluster.num_blocks(), c = cluster.block_rank();
  const uint32_t tile = blockIdx.x / C;
  if (tile >= (uint32_t)*P.ntiles) return;   // (the whole cluster)
  const Tile T = P.tiles[tile];
  const DevAdapter A = P.table[T.adapter];
  const uint32_t tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, q = lane & 3;
  const uint32_t wr = warp & 3, wh = warp >> 2;   // 16 rows; half of a stage, of a step's columns
  const int32_t rank = (int32_t)A.rank;
  if (tid < 64) srow[tid] = (int32_t)tid < T.count ? P.perm[T.start + tid] : -1;
  __syncthreads();

  // ---- low = s A x: this block's stages of the sum
  const uint32_t stages = (P.K + kBK - 1) / kBK;
  const uint32_t mine = stages > c ? (stages - c + C - 1) / C : 0;
  const uint32_t xrow = tid >> 3, xch = tid & 7;   // rows xrow and xrow + 32, one 16-byte slot
  const int32_t s0 = srow[xrow], s1 = srow[xrow + 32];
  const uint32_t ring = smem_addr(smem);
  auto load_stage = [&](uint32_t i) {
    const uint32_t k = (c + i * C) * kBK + xch * 8, at = ring + (i % kStages) * L::kStage;
    const int32_t n = (int32_t)P.K - (int32_t)k;
    fill8(at + swz(xrow * 128 + xch * 16), P.x + (int64_t)s0 * P.ldx + k, s0 >= 0 ? n : 0, P.vec_x);
    fill8(at + swz((xrow + 32) * 128 + xch * 16), P.x + (int64_t)s1 * P.ldx + k, s1 >= 0 ? n : 0,
          P.vec_x);
#pragma unroll
    for (uint32_t r = 0; r < RP; r += 32) {
      const uint32_t row = r + xrow;
      if (RP >= 32 || row < RP)
        fill8(at + L::kXBytes + swz(row * 128 + xch * 16), A.down + (uint64_t)row * A.ld_down + k,
              (int32_t)row < rank ? n : 0, A.vec_down);
    }
  };
  float acc[RP / 8][4];
#pragma unroll
  for (int j = 0; j < RP / 8; j++) acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0.f;
  for (uint32_t i = 0; i < kStages - 1; i++) {
    if (i < mine) load_stage(i);
    cp_commit();
  }
  for (uint32_t i = 0; i < mine; i++) {
    cp_wait<kStages - 2>();
    __syncthreads();
    if (i + kStages - 1 < mine) load_stage(i + kStages - 1);
    cp_commit();
    const uint32_t xs = ring + (i % kStages) * L::kStage, ws = xs + L::kXBytes;
#pragma unroll
    for (uint32_t kk = 0; kk < 2; kk++) {
      const uint32_t kb = wh * 64 + kk * 32;   // byte of the 16-value step in a row
      uint32_t a[4];
      ldsm4(a, xs + swz((wr * 16 + (lane & 15)) * 128 + kb + (lane >> 4) * 16));
#pragma unroll
      for (int j = 0; j < RP / 16; j++) {
        uint32_t b[4];
        ldsm4(b, ws + swz((j * 16 + (lane >> 4) * 8 + (lane & 7)) * 128 + kb + ((lane >> 3) & 1) * 16));
        mma16816(acc[2 * j], a[0], a[1], a[2], a[3], b[0], b[1]);
        mma16816(acc[2 * j + 1], a[0], a[1], a[2], a[3], b[2], b[3]);
      }
    }
  }
  cp_wait<0>();
  __syncthreads();
  // join the two halves of every stage, then the blocks of the cluster
  if (wh == 1) {
#pragma unroll
    for (int j = 0; j < RP / 8; j++) {
      float* d = part + (wr * 16 + g) * RP + j * 8 + 2 * q;
      *reinterpret_cast<float2*>(d) = make_float2(acc[j][0], acc[j][1]);
      *reinterpret_cast<float2*>(d + 8 * RP) = make_float2(acc[j][2], acc[j][3]);
    }
  }
  __syncthreads();
  if (wh == 0) {
#pragma unroll
    for (int j = 0; j < RP / 8; j++) {
      float2* d = reinterpret_cast<float2*>(part + (wr * 16 + g) * RP + j * 8 + 2 * q);
      float2* e = reinterpret_cast<float2*>(part + (wr * 16 + g + 8) * RP + j * 8 + 2 * q);
      *d = make_float2(d->x + acc[j][0], d->y + acc[j][1]);
      *e = make_float2(e->x + acc[j][2], e->y + acc[j][3]);
    }
  }
  cluster.sync();
  {
    const uint32_t rows = 64 / C;   // this block joins these rows and hands them to all
    for (uint32_t e = tid * 2; e < rows * RP; e += kThreads * 2) {
      const uint32_t row = c * rows + e / RP, col = e % RP;
      float2 s = make_float2(0.f, 0.f);
      for (uint32_t b = 0; b < C; b++) {
        const float2 v =
            *reinterpret_cast<const float2*>(cluster.map_shared_rank(part, b) + row * RP + col);
        s.x += v.x;
        s.y += v.y;
      }
      // columns past the rank are 0 whatever x holds (an infinity times a padded 0 is not)
      const uint32_t u = pack_bf16((int32_t)col < rank ? s.x * A.scale : 0.f,
                                   (int32_t)col + 1 < rank ? s.y * A.scale : 0.f);
      for (uint32_t b = 0; b < C; b++)
        *reinterpret_cast<uint32_t*>(cluster.map_shared_rank(us, b) + row * L::kULd + col) = u;
      if (P.low && srow[row] >= 0)
        *reinterpret_cast<uint32_t*>(P.low + (int64_t)srow[row] * RP + col) = u;
    }
  }
  cluster.sync();   // low is complete, and nobody reads another block's memory after this
  if (!P.y) return;

  // ---- y += B low: this block's steps of the columns
  const uint32_t steps = (P.N + kBN - 1) / kBN;
  const uint32_t todo = steps > c ? (steps - c + C - 1) / C : 0;
  const uint32_t up0 = smem_addr(upt);
  auto load_up = [&](uint32_t i) {
    const uint32_t o0 = (c + i * C) * kBN, at = up0 + (i & 1) * L::kUp;
    constexpr uint32_t per = RP / 8;   // 16-byte slots in a row
#pragma unroll
    for (uint32_t s = tid; s < kBN * per; s += kThreads) {
      const uint32_t row = s / per, ch = s % per, o = o0 + row;
      fill8(at + swz_dealt<RP>(row, ch), A.up + (uint64_t)o * A.ld_up + ch * 8,
            o < P.N ? rank - (int32_t)ch * 8 : 0, A.vec_up);
    }
  };
  const int32_t r0 = srow[wr * 16 + g], r1 = srow[wr * 16 + g + 8];
  uint4 y0[2], y1[2];
  auto load_y = [&](uint32_t i) {
#pragma unroll
    for (uint32_t h = 0; h < 2; h++) {
      const uint32_t col = (c + i * C) * kBN + wh * 64 + h * 32 + 8 * q;
      const int32_t n = (int32_t)P.N - (int32_t)col;
      y0[h] = load8(P.y + (int64_t)r0 * P.ldy + col, r0 >= 0 ? n : 0, P.vec_y);
      y1[h] = load8(P.y + (int64_t)r1 * P.ldy + col, r1 >= 0 ? n : 0, P.vec_y);
    }
  };
  if (todo > 0) {
    load_up(0);
    cp_commit();
    load_y(0);
  }
  for (uint32_t i = 0; i < todo; i++) {
    cp_wait<0>();
    __syncthreads();
    if (i + 1 < todo) load_up(i + 1);
    cp_commit();
    uint4 c0[2] = {y0[0], y0[1]}, c1[2] = {y1[0], y1[1]};
    if (i + 1 < todo) load_y(i + 1);
    const uint32_t at = up0 + (i & 1) * L::kUp;
    float d[2][4][4];
#pragma unroll
    for (int h = 0; h < 2; h++)
#pragma unroll
      for (int j = 0; j < 4; j++) d[h][j][0] = d[h][j][1] = d[h][j][2] = d[h][j][3] = 0.f;
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
      const uint32_t col = (c + i * C) * kBN + wh * 64 + h * 32 + 8 * q;
      const int32_t n = (int32_t)P.N - (int32_t)col;
      if (r0 >= 0)
        store8(P.y + (int64_t)r0 * P.ldy + col,
               make_uint4(add_pair(c0[h].x, d[h][0][0], d[h][0][1]),
                          add_pair(c0[h].y, d[h][1][0], d[h][1][1]),
                          add_pair(c0[h].z, d[h][2][0], d[h][2][1]),
                          add_pair(c0[h].w, d[h][3][0], d[h][3][1])),
               n, P.vec_y);
      if (r1 >= 0)
        store8(P.y + (int64_t)r1 * P.ldy + col,
               make_uint4(add_pair(c1[h].x, d[h][0][2], d[h][0][3]),
                          add_pair(c1[h].y, d[h][1][2], d[h][1][3]),
                          add_pair(c1[h].z, d[h][2][2], d[h][2][3]),
                          add_pair(c1[h].w, d[h][3][2], d[h][3][3])),
               n, P.vec_y);
    }
  }
}

// ---------------------------------------------------------------- transposes of the factors
// down (rank x hidden) to hidden x RP and up (out x rank) to RP x out8, both zero-padded, and a
// table entry that has them in the other's place.
__global__ void __launch_bounds__(kThreads) k_transpose(const DevAdapter* __restrict__ table,
                                                        uint32_t hidden, uint32_t out, uint32_t RP,
                                                        uint32_t out8, uint16_t* __restrict__ buf,
                                                        DevAdapter* __restrict__ swapped) {
  __shared__ uint16_t sh[32][33];
  const DevAdapter A = table[blockIdx.y];
  uint16_t* const at = buf + (uint64_t)blockIdx.y * RP * ((uint64_t)hidden + out8);
  uint16_t* const bt = at + (uint64_t)hidden * RP;
  const uint32_t tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  const uint32_t ht = (hidden + 31) / 32, ot = (out8 + 31) / 32;
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    DevAdapter S = A;
    S.down = bt;
    S.ld_down = out8;
    S.up = at;
    S.ld_up = RP;
    S.vec_down = S.vec_up = 1;
    swapped[blockIdx.y] = S;
  }
  for (uint32_t b = blockIdx.x; b < ht + ot; b += gridDim.x) {
    const bool first = b < ht;
    const uint32_t f0 = (first ? b : b - ht) * 32;
    for (uint32_t r0 = 0; r0 < RP; r0 += 32) {
      __syncthreads();
      for (uint32_t i = ty; i < 32; i += 8) {
        uint16_t v = 0;
        if (first) {   // rows r0 + i, columns f0 + tx
          if (r0 + i < A.rank && f0 + tx < hidden) v = A.down[(uint64_t)(r0 + i) * A.ld_down + f0 + tx];
        } else {       // rows f0 + i, columns r0 + tx
          if (f0 + i < out && r0 + tx < A.rank) v = A.up[(uint64_t)(f0 + i) * A.ld_up + r0 + tx];
        }
        sh[i][tx] = v;
      }
      __syncthreads();
      for (uint32_t i = ty; i < 32; i += 8) {
        const uint16_t v = sh[tx][i];
        if (first) {
          if (f0 + i < hidden && r0 + tx < RP) at[(uint64_t)(f0 + i) * RP + r0 + tx] = v;
        } else {
          if (r0 + i < RP && f0 + tx < out8) bt[(uint64_t)(r0 + i) * out8 + f0 + tx] = v;
        }
      }
    }
  }
}

// ------------------------------------------------------------------------ weight gradients
// A block takes 128 features of x (for dA) or dy (for dB) of one adapter; the blocks of a
// cluster split the adapter's rows in tiles of 64 and join their sums in a fixed order.
struct WgradArgs {
  const DevAdapter* table;
  const int32_t* perm;
  const int32_t* offsets;
  const uint16_t* x;
  uint64_t ldx;
  const uint16_t* dy;
  uint64_t lddy;
  const uint16_t* low;
  const uint16_t* dlow;
  uint32_t hidden, out, vec_x, vec_dy;
  uint32_t grad_f32, accumulate;
};

constexpr uint32_t kFeat = 128;
constexpr uint32_t kWStages = 3;
template <int RP>
struct Wgrad {
  static constexpr uint32_t kQ = 64 * kFeat * 2, kPb = 64 * RP * 2, kStage = kQ + kPb;
  static constexpr uint32_t kRing = kWStages * kStage, kPart = kFeat * RP * 4;
  static constexpr uint32_t kSmem = kRing > kPart ? kRing : kPart;
};

__device__ __forceinline__ void put_grad(void* base, uint64_t at, float v, bool f32, bool acc) {
  if (f32) {
    float* p = static_cast<float*>(base) + at;
    *p = acc ? *p + v : v;
  } else {
    uint16_t* p = static_cast<uint16_t*>(base) + at;
    const float s = acc ? __uint_as_float((uint32_t)*p << 16) + v : v;
    *p = (uint16_t)pack_bf16(s, 0.f);
  }
}

template <int RP>
__global__ void __launch_bounds__(kThreads) k_wgrad(const WgradArgs P) {
  using L = Wgrad<RP>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const cg::cluster_group cluster = cg::this_cluster();
  const uint32_t C = cluster.num_blocks(), c = cluster.block_rank();
  const uint32_t slice = blockIdx.x / C, hs = (P.hidden + kFeat - 1) / kFeat;
  const bool down = slice < hs;
  const uint32_t f0 = (down ? slice : slice - hs) * kFeat, F = down ? P.hidden : P.out;
  const uint16_t* const src = down ? P.x : P.dy;
  const uint64_t lds = down ? P.ldx : P.lddy;
  const bool vec = down ? P.vec_x : P.vec_dy;
  const uint16_t* const pr = down ? P.dlow : P.low;
  const int32_t start = P.offsets[blockIdx.y], end = P.offsets[blockIdx.y + 1];
  const uint32_t tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, q = lane & 3;
  const uint32_t tiles = (uint32_t)(end - start + 63) / 64;
  const uint32_t mine = tiles > c ? (tiles - c + C - 1) / C : 0;
  const uint32_t ring = smem_addr(smem);
  auto load_stage = [&](uint32_t i) {
    const int32_t t0 = start + (int32_t)((c + i * C) * 64);
    const uint32_t at = ring + (i % kWStages) * L::kStage;
#pragma unroll
    for (uint32_t s = tid; s < 64 * 16; s += kThreads) {
      const uint32_t row = s >> 4, ch = s & 15, f = f0 + ch * 8;
      const int32_t t = t0 + (int32_t)row < end ? P.perm[t0 + row] : -1;
      fill8(at + (ch >> 3) * 8192 + swz(row * 128 + (ch & 7) * 16), src + (int64_t)t * lds + f,
            t >= 0 ? (int32_t)F - (int32_t)f : 0, vec);
    }
    constexpr uint32_t per = RP / 8;
#pragma unroll
    for (uint32_t s = tid; s < 64 * per; s += kThreads) {
      const uint32_t row = s / per, ch = s % per;
      const int32_t t = t0 + (int32_t)row < end ? P.perm[t0 + row] : -1;
      fill8(at + L::kQ + swz(row * (RP * 2) + ch * 16), pr + (int64_t)t * RP + ch * 8,
            t >= 0 ? 8 : 0, true);
    }
  };
  float acc[RP / 8][4];
#pragma unroll
  for (int j = 0; j < RP / 8; j++) acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0.f;
  for (uint32_t i = 0; i < kWStages - 1; i++) {
    if (i < mine) load_stage(i);
    cp_commit();
  }
  for (uint32_t i = 0; i < mine; i++) {
    cp_wait<kWStages - 2>();
    __syncthreads();
    if (i + kWStages - 1 < mine) load_stage(i + kWStages - 1);
    cp_commit();
    const uint32_t qs = ring + (i % kWStages) * L::kStage + (warp >> 2) * 8192;
    const uint32_t ps = ring + (i % kWStages) * L::kStage + L::kQ;
#pragma unroll
    for (uint32_t kt = 0; kt < 4; kt++) {   // 16 rows of the batch
      uint32_t a[4];
      ldsm4t(a, qs + swz((kt * 16 + (lane >> 4) * 8 + (lane & 7)) * 128 + (warp & 3) * 32 +
                         ((lane >> 3) & 1) * 16));
#pragma unroll
      for (int j = 0; j < RP / 16; j++) {
        uint32_t b[4];
        ldsm4t(b, ps + swz((kt * 16 + ((lane >> 3) & 1) * 8 + (lane & 7)) * (RP * 2) + j * 32 +
                           (lane >> 4) * 16));
        mma16816(acc[2 * j], a[0], a[1], a[2], a[3], b[0], b[1]);
        mma16816(acc[2 * j + 1], a[0], a[1], a[2], a[3], b[2], b[3]);
      }
    }
  }
  cp_wait<0>();
  __syncthreads();
  float* const part = reinterpret_cast<float*>(smem);   // [feature][RP]
#pragma unroll
  for (int j = 0; j < RP / 8; j++) {
    float* d = part + (warp * 16 + g) * RP + j * 8 + 2 * q;
    *reinterpret_cast<float2*>(d) = make_float2(acc[j][0], acc[j][1]);
    *reinterpret_cast<float2*>(d + 8 * RP) = make_float2(acc[j][2], acc[j][3]);
  }
  cluster.sync();
  const DevAdapter A = P.table[blockIdx.y];
  const uint32_t feats = kFeat / C;
  for (uint32_t e = tid; e < feats * RP; e += kThreads) {
    // neighbours in memory to neighbouring threads: along the features for dA, the rank for dB
    const uint32_t fl = c * feats + (down ? e % feats : e / RP), r = down ? e / feats : e % RP;
    if (f0 + fl >= F || r >= A.rank) continue;
    float s = 0.f;
    for (uint32_t b = 0; b < C; b++) s += cluster.map_shared_rank(part, b)[fl * RP + r];
    if (down)
      put_grad(A.gdown, (uint64_t)r * A.ld_gdown + f0 + fl, s, P.grad_f32, P.accumulate);
    else
      put_grad(A.gup, (uint64_t)(f0 + fl) * A.ld_gup + r, s, P.grad_f32, P.accumulate);
  }
  cluster.sync();   // the others may still read `part`
}

// ------------------------------------------------------------------------------- host side
template <class F, class Args>
int launch_clusters(F* kernel, uint32_t grid_x, uint32_t grid_y, uint32_t cluster, uint32_t smem,
                    const Args& args, cudaStream_t s) {
  if (smem > 48 * 1024) {
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return BD_ERR_CUDA;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid_x * cluster, grid_y, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return check(cudaLaunchKernelEx(&cfg, kernel, args));
}

template <int RP>
int launch_apply(bool small, uint32_t tiles, uint32_t cluster, const ApplyArgs& P, cudaStream_t s) {
  if (small)
    return launch_clusters(k_apply16<RP>, tiles, 1, cluster,
                           (9 * 16 * RP) * 4 + 16 * (RP + 8) * 2, P, s);
  return launch_clusters(k_apply64<RP>, tiles, 1, cluster, Apply64<RP>::kSmem, P, s);
}

// Blocks of a cluster that share a piece of work: enough for about two blocks per SM.
uint32_t cluster_for(uint64_t pieces, int sms) {
  uint32_t c = 1;
  while (c < kMaxCluster && pieces * c < 2 * (uint64_t)sms) c *= 2;
  return c;
}

int apply(uint32_t RP, uint32_t rows, uint32_t k, const void* const* tiles, const int32_t* ntiles,
          ApplyArgs& P, int sms, cudaStream_t s) {
  // Tiles of 16 rows while the adapters have few rows each: a tile of 64 would be mostly empty.
  const bool small = rows <= 128 || rows / k < 24;
  const uint64_t bound0 = (uint64_t)rows / (small ? 16 : 64) + k;
  const uint32_t bound = (uint32_t)(bound0 < rows ? bound0 : rows);
  P.tiles = static_cast<const Tile*>(tiles[small ? 0 : 1]);
  P.ntiles = ntiles + (small ? 0 : 1);
  const uint32_t cluster = cluster_for(bound, sms);
  switch (RP) {
    case 16: return launch_apply<16>(small, bound, cluster, P, s);
    case 32: return launch_apply<32>(small, bound, cluster, P, s);
    case 64: return launch_apply<64>(small, bound, cluster, P, s);
    default: return launch_apply<128>(small, bound, cluster, P, s);
  }
}

struct RowsLayout {
  uint64_t counts, offsets, ntiles, perm, tiles16, tiles64, total;
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
  L.ntiles = take(8);
  L.perm = take((uint64_t)rows * 4);
  L.tiles16 = take(((uint64_t)rows / 16 + k) * sizeof(Tile));
  L.tiles64 = take(((uint64_t)rows / 64 + k) * sizeof(Tile));
  L.total = off;
  return true;
}

bool valid(const bo_adapter_set* s) {
  return s && s->d_table && s->k > 0 && s->hidden > 0 && s->out > 0 &&
         (s->rank == 16 || s->rank == 32 || s->rank == 64 || s->rank == 128);
}
bool valid(const bo_adapter_rows* r) {
  return r && r->d_perm && r->d_offsets && r->d_tiles[0] && r->d_tiles[1] && r->d_ntiles;
}
bool wide(const void* p, uint64_t ld, uint64_t width) {
  return aligned(p, 16) && ld % 8 == 0 && width % 8 == 0;
}
// bytes from the first to past the last value of `rows` rows
uint64_t extent(uint64_t rows, uint64_t ld, uint64_t width) {
  return rows == 0 ? 0 : 2 * ((rows - 1) * ld + width);
}
uint64_t up8(uint64_t x) { return (x + 7) / 8 * 8; }

struct BackwardLayout {
  uint64_t dlow, table, buf, total;
};
BackwardLayout backward_layout(const bo_adapter_set* set, uint32_t rows) {
  BackwardLayout L;
  L.dlow = 0;
  L.table = up((uint64_t)rows * set->rank * 2, 256);
  L.buf = L.table + up((uint64_t)set->k * sizeof(DevAdapter), 256);
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
  if (!dev) return BD_ERR_INVALID_ARG;
  const uintptr_t gsize = grad_dtype == BO_FP32 ? 4 : 2;
  uint32_t most = 1;
  bool grads = true;
  for (uint32_t i = 0; i < k; i++) {
    const bo_adapter& a = h_items[i];
    if (!a.d_down || !a.d_up || !aligned(a.d_down, 2) || !aligned(a.d_up, 2) || a.rank < 1 ||
        a.rank > BO_ADAPTER_MAX_RANK || a.ld_down < hidden || a.ld_up < a.rank ||
        a.ld_down > (1ull << 40) || a.ld_up > (1ull << 40))
      return BD_ERR_INVALID_ARG;
    if (!a.d_grad_down != !a.d_grad_up) return BD_ERR_INVALID_ARG;
    if (!a.d_grad_down) grads = false;
    else if (!aligned(a.d_grad_down, gsize) || !aligned(a.d_grad_up, gsize) ||
             a.ld_grad_down < hidden || a.ld_grad_up < a.rank || a.ld_grad_down > (1ull << 40) ||
             a.ld_grad_up > (1ull << 40))
      return BD_ERR_INVALID_ARG;
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
    d.vec_up = wide(a.d_up, a.ld_up, a.rank);
    if (a.rank > most) most = a.rank;
  }
  const int rc = check(upload(dev.get(), (uint64_t)k * sizeof(DevAdapter), d_set,
                              static_cast<cudaStream_t>(stream)));
  if (rc) return rc;
  h_out->d_table = d_set;
  h_out->k = k;
  h_out->hidden = hidden;
  h_out->out = out;
  h_out->rank = most <= 16 ? 16 : most <= 32 ? 32 : most <= 64 ? 64 : 128;
  h_out->grad_dtype = grad_dtype;
  h_out->has_grads = grads;
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
  int32_t* ntiles = reinterpret_cast<int32_t*>(p + L.ntiles);
  int32_t* perm = reinterpret_cast<int32_t*>(p + L.perm);
  Tile* t16 = reinterpret_cast<Tile*>(p + L.tiles16);
  Tile* t64 = reinterpret_cast<Tile*>(p + L.tiles64);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  k_rows_count<<<k, kThreads, 0, s>>>(d_index, rows, k, counts, d_status);
  int rc = check(cudaGetLastError());
  if (rc) return rc;
  k_rows_place<<<k, kThreads, 0, s>>>(d_index, rows, k, counts, perm, offsets, t16, t64, ntiles);
  if ((rc = check(cudaGetLastError()))) return rc;
  h_out->d_perm = perm;
  h_out->d_offsets = offsets;
  h_out->d_tiles[0] = t16;
  h_out->d_tiles[1] = t64;
  h_out->d_ntiles = ntiles;
  h_out->rows = rows;
  h_out->k = k;
  return BD_OK;
}

int bo_adapter_forward(const bo_adapter_set* set, const bo_adapter_rows* rows, const uint16_t* d_x,
                       uint64_t ldx, uint16_t* d_y, uint64_t ldy, uint16_t* d_low, void* stream) {
  if (!valid(set) || !valid(rows) || rows->k != set->k) return BD_ERR_INVALID_ARG;
  if (rows->rows == 0) return BD_OK;
  if (!d_x || !d_y || !aligned(d_x, 2) || !aligned(d_y, 2) || ldx < set->hidden ||
      ldy < set->out || ldx > (1ull << 40) || ldy > (1ull << 40) || !aligned(d_low, 16))
    return BD_ERR_INVALID_ARG;
  const uint64_t yb = extent(rows->rows, ldy, set->out);
  const uint64_t lb = d_low ? (uint64_t)rows->rows * set->rank * 2 : 0;
  if (overlaps(d_x, extent(rows->rows, ldx, set->hidden), d_y, yb) || overlaps(d_low, lb, d_y, yb) ||
      overlaps(d_low, lb, d_x, extent(rows->rows, ldx, set->hidden)))
    return BD_ERR_INVALID_ARG;
  const int sms = sm_count();
  if (sms <= 0) return BD_ERR_CUDA;
  ApplyArgs P = {};
  P.table = static_cast<const DevAdapter*>(set->d_table);
  P.perm = rows->d_perm;
  P.x = d_x;
  P.ldx = ldx;
  P.y = d_y;
  P.ldy = ldy;
  P.low = d_low;
  P.K = set->hidden;
  P.N = set->out;
  P.vec_x = wide(d_x, ldx, set->hidden);
  P.vec_y = wide(d_y, ldy, set->out);
  return apply(set->rank, rows->rows, set->k, rows->d_tiles, rows->d_ntiles, P, sms,
               static_cast<cudaStream_t>(stream));
}

uint64_t bo_adapter_backward_workspace_size(const bo_adapter_set* set, uint32_t rows) {
  return valid(set) && rows <= BO_ADAPTER_MAX_ROWS ? backward_layout(set, rows).total : 0;
}

int bo_adapter_backward(const bo_adapter_set* set, const bo_adapter_rows* rows,
                        const uint16_t* d_x, uint64_t ldx, const uint16_t* d_dy, uint64_t lddy,
                        const uint16_t* d_low, uint16_t* d_dx, uint64_t lddx, int32_t accumulate,
                        void* d_ws, uint64_t ws_bytes, void* stream) {
  if (!valid(set) || !valid(rows) || rows->k != set->k) return BD_ERR_INVALID_ARG;
  const BackwardLayout L = backward_layout(set, rows->rows);
  if (!d_ws || !aligned(d_ws, 256) || ws_bytes < L.total) return BD_ERR_INVALID_ARG;
  const uint64_t xb = extent(rows->rows, ldx, set->hidden), yb = extent(rows->rows, lddy, set->out);
  const uint64_t db = d_dx ? extent(rows->rows, lddx, set->hidden) : 0;
  if (rows->rows > 0) {
    if (!d_x || !d_dy || !d_low || !aligned(d_x, 2) || !aligned(d_dy, 2) || !aligned(d_dx, 2) ||
        !aligned(d_low, 16) || ldx < set->hidden || lddy < set->out ||
        (d_dx && lddx < set->hidden) || ldx > (1ull << 40) || lddy > (1ull << 40) ||
        (d_dx && lddx > (1ull << 40)))
      return BD_ERR_INVALID_ARG;
    if (overlaps(d_dx, db, d_x, xb) || overlaps(d_dx, db, d_dy, yb) ||
        overlaps(d_dx, db, d_low, (uint64_t)rows->rows * set->rank * 2) ||
        overlaps(d_dx, db, d_ws, L.total))
      return BD_ERR_INVALID_ARG;
  }
  const int sms = sm_count();
  if (sms <= 0) return BD_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  uint8_t* w = static_cast<uint8_t*>(d_ws);
  uint16_t* dlow = reinterpret_cast<uint16_t*>(w + L.dlow);
  DevAdapter* swapped = reinterpret_cast<DevAdapter*>(w + L.table);
  uint16_t* buf = reinterpret_cast<uint16_t*>(w + L.buf);
  const uint32_t out8 = (uint32_t)up8(set->out);
  int rc;
  if (rows->rows > 0) {
    const uint32_t pieces = (set->hidden + 31) / 32 + (out8 + 31) / 32;
    const uint32_t most = (uint32_t)((uint64_t)sms * 8 / set->k + 1);
    k_transpose<<<dim3(pieces < most ? pieces : most, set->k), kThreads, 0, s>>>(
        static_cast<const DevAdapter*>(set->d_table), set->hidden, set->out, set->rank, out8, buf,
        swapped);
    if ((rc = check(cudaGetLastError()))) return rc;
    ApplyArgs P = {};
    P.table = swapped;
    P.perm = rows->d_perm;
    P.x = d_dy;
    P.ldx = lddy;
    P.y = d_dx;
    P.ldy = lddx;
    P.low = dlow;
    P.K = set->out;
    P.N = set->hidden;
    P.vec_x = wide(d_dy, lddy, set->out);
    P.vec_y = d_dx && wide(d_dx, lddx, set->hidden);
    if ((rc = apply(set->rank, rows->rows, set->k, rows->d_tiles, rows->d_ntiles, P, sms, s)))
      return rc;
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
  G.hidden = set->hidden;
  G.out = set->out;
  G.vec_x = wide(d_x, ldx, set->hidden);
  G.vec_dy = wide(d_dy, lddy, set->out);
  G.grad_f32 = set->grad_dtype == BO_FP32;
  G.accumulate = accumulate != 0;
  const uint32_t slices = (set->hidden + kFeat - 1) / kFeat + (set->out + kFeat - 1) / kFeat;
  const uint32_t cluster = cluster_for((uint64_t)slices * set->k, sms);
  switch (set->rank) {
    case 16: return launch_clusters(k_wgrad<16>, slices, set->k, cluster, Wgrad<16>::kSmem, G, s);
    case 32: return launch_clusters(k_wgrad<32>, slices, set->k, cluster, Wgrad<32>::kSmem, G, s);
    case 64: return launch_clusters(k_wgrad<64>, slices, set->k, cluster, Wgrad<64>::kSmem, G, s);
    default: return launch_clusters(k_wgrad<128>, slices, set->k, cluster, Wgrad<128>::kSmem, G, s);
  }
}

}  // extern "C"
