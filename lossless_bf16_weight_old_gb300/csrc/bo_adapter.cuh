// bo_adapter.cuh -- what the adapter kernels share (bo_adapter.cu, bo_adapter_tc.cu).
#pragma once

#include "bo_internal.cuh"

namespace bo {

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
  uint32_t vec_gup, pad[3];    // rows of dB may be written 16 bytes at a time
};
static_assert(sizeof(DevAdapter) % 16 == 0, "uploaded in 16-byte words");

struct Tile {
  int32_t adapter, start, count;   // rows start .. start + count of the grouped order
  int32_t end;                     // the tile after the adapter's last
};

__device__ __forceinline__ uint32_t smem_addr(const void* p) {
  return (uint32_t)__cvta_generic_to_shared(p);
}
// (rows that are read from end to end, a piece at a time: HBM may as well send the piece after)
__device__ __forceinline__ void cp16_ahead(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// 16 bytes, or zeros in their place (src is not read then, but points at memory of the caller's)
__device__ __forceinline__ void cp16z(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(there ? 16 : 0)
               : "memory");
}
// The first n of eight values (none for n <= 0), and zeros in place of the others.
__device__ __forceinline__ void cp16n(uint32_t dst, const void* src, int32_t n) {
  const int32_t bytes = n >= 8 ? 16 : n > 0 ? 2 * n : 0;
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
// Byte address in a tile of rows that fill 128-byte lines: the 16-byte slots of a line are
// permuted by the line's number, so that eight consecutive rows at one column fall into
// different banks (the 128-byte swizzle of the tensor cores' and the copy engine's tiles).
__device__ __forceinline__ uint32_t swz(uint32_t byte) { return byte ^ (((byte >> 7) & 7) << 4); }

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
  uint32_t vec_x, vec_y;  // rows may be read 16 bytes at a time
  uint32_t vec_factors;   // ... of every adapter's first factor
  uint32_t vec_ups;       // ... of every second one, whose rows end with (or are 0 up to) whole words
  int32_t* status;        // BD_ERR_CUDA when a wait inside a kernel ran out; may be NULL
  uint32_t stall;         // the first stage is never reported
};

struct WgradArgs {
  const DevAdapter* table;
  const int32_t* perm;
  const int32_t* offsets;
  const int32_t* blocks;     // what a piece of each of the adapters before counts for, summed
  const uint16_t* x;
  uint64_t ldx;
  const uint16_t* dy;
  uint64_t lddy;
  const uint16_t* low;
  const uint16_t* dlow;
  float* sums;               // two of a block
  uint32_t* counters;        // one of a piece, 0 before and after
  uint32_t k, hidden, out, vec_x, vec_dy;
  uint32_t grad_f32, accumulate;
  int32_t* status;
  uint32_t stall;
};

constexpr uint32_t kFeat = 128;   // features of a piece of the weight gradients
constexpr int32_t kLeast = 4;     // stages that it counts for at least

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

// A block's share of all stages of all pieces, and the piece that a stage belongs to.
struct Shares {
  uint64_t all, each;
  uint32_t G, rest;   // blocks that have a share (none is empty, so those of a piece are consecutive)
  __device__ __forceinline__ Shares(uint64_t stages, uint32_t grid)
      : all(stages), G(grid < stages ? grid : (uint32_t)stages) {
    each = G ? all / G : 0;
    rest = (uint32_t)(all - each * G);
  }
  // all b / G (a grid has a few hundred blocks)
  __device__ __forceinline__ uint64_t begin(uint32_t b) const { return each * b + rest * b / G; }
  __device__ __forceinline__ uint32_t owner(uint64_t stage) const {
    uint32_t b = (uint32_t)(stage * G / all);
    while (begin(b + 1) <= stage) b++;
    return b;
  }
};
// Walks over the pieces of a block's share; only a new adapter is looked up.  A piece counts for at
// least kLeast stages, the time to carry it out: the 118 pieces of an adapter with four rows beside
// three with thousands (4096 + 11008 features) would else be one block's (195 us, not 62).
struct Piece {
  uint32_t adapter, slice, stages;   // its stages
  uint32_t first, mine;              // this block's
  uint64_t begin, at, end;           // its first stage among all, the block's, and the share's end
  int32_t row0, row1;                // the adapter's rows in the grouped order
  __device__ __forceinline__ Piece(const WgradArgs& P, uint32_t slices, uint64_t from, uint64_t to) {
    uint32_t lo = 0, hi = P.k;   // the last adapter whose stages begin at or before `from`
    while (hi - lo > 1) {
      const uint32_t mid = (lo + hi) / 2;
      if ((uint64_t)P.blocks[mid] * slices <= from) lo = mid; else hi = mid;
    }
    adapter = lo;
    at = from;
    end = to;
    const uint64_t a_begin = (uint64_t)P.blocks[lo] * slices;
    open(P);
    slice = (uint32_t)((at - a_begin) / units);
    begin = a_begin + (uint64_t)slice * units;
    part();
    if (mine == 0) next(P, slices);
  }
  __device__ __forceinline__ bool over() const { return at >= end; }
  __device__ __forceinline__ void next(const WgradArgs& P, uint32_t slices) {
    do {
      at += span;
      if (over()) return;
      begin += units;
      if (++slice == slices) {
        slice = 0;
        adapter++;
        open(P);
      }
      part();
    } while (mine == 0);
  }

 private:
  uint32_t units, span;              // what the piece counts for, and the share's part of that
  __device__ __forceinline__ void open(const WgradArgs& P) {
    units = (uint32_t)(P.blocks[adapter + 1] - P.blocks[adapter]);
    row0 = P.offsets[adapter];
    row1 = P.offsets[adapter + 1];
    stages = row1 > row0 ? (uint32_t)(row1 - row0 + 63) / 64 : 1;   // (at least one, of no rows)
  }
  __device__ __forceinline__ void part() {
    first = (uint32_t)(at - begin);
    const uint64_t p_end = begin + units;
    span = (uint32_t)((end < p_end ? end : p_end) - at);
    mine = first >= stages ? 0 : span < stages - first ? span : stages - first;
  }
};

// ---- bo_adapter_tc.cu: the forms on the tensor cores' own memory, for many rows.  rp: 16 to 128.
// All rows and factors can be read 16 bytes at a time.
cudaError_t tc_low(uint32_t rp, uint32_t tiles, uint32_t cluster, const ApplyArgs& P, cudaStream_t s);
cudaError_t tc_wgrad(uint32_t rp, uint32_t grid, const WgradArgs& P, cudaStream_t s);

}  // namespace bo
