// bo_internal.cuh -- definitions shared by the kernels of libbf16ops (include/ops/bf16ops.h).
#pragma once

#include <algorithm>
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "ops/bf16ops.h"

namespace bo {

inline bool aligned(const void* p, uintptr_t a) {
  return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}
// [a, a+na) and [b, b+nb) intersect
inline bool overlaps(const void* a, uint64_t na, const void* b, uint64_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return na > 0 && nb > 0 && x < y + nb && y < x + na;
}
// Memory (or anything numbered) that a call reads or writes.
struct Span {
  uint64_t begin, end;
  bool write;
};
// Whether nothing that is written meets anything else.  Sorts them.
inline bool disjoint(Span* s, size_t n) {
  std::sort(s, s + n, [](const Span& a, const Span& b) { return a.begin < b.begin; });
  uint64_t reads = 0, writes = 0;   // where those before end
  for (size_t i = 0; i < n; i++) {
    if (s[i].begin == s[i].end) continue;
    if (s[i].begin < writes || (s[i].write && s[i].begin < reads)) return false;
    uint64_t& most = s[i].write ? writes : reads;
    most = std::max(most, s[i].end);
  }
  return true;
}
// Memory of `rows` rows, in bytes.
struct Region {
  uint64_t at, ld, width, rows;
  bool write = false;
  Region() = default;
  Region(const void* p, uint64_t n, uint64_t stride, uint64_t columns, uint64_t size = 2)
      : at(reinterpret_cast<uintptr_t>(p)), ld(stride * size), width(columns * size), rows(p ? n : 0) {}
  uint64_t end() const { return rows ? at + (rows - 1) * ld + width : at; }
};
// Whether two of them have a byte in common.  Rows of the same stride may lie between one another's
// (columns of one buffer); of different strides they may not.
inline bool meet(const Region& a, const Region& b) {
  if (a.rows == 0 || b.rows == 0 || a.at >= b.end() || b.at >= a.end()) return false;
  if (a.at > b.at) return meet(b, a);
  if (a.rows == 1 || (b.rows > 1 && a.ld != b.ld)) return true;
  // b begins `off` bytes into row `skip` of a, which is not past a's last
  const uint64_t skip = (b.at - a.at) / a.ld, off = (b.at - a.at) % a.ld;
  return off < a.width || (skip + 1 < a.rows && off + b.width > a.ld);
}
inline uint64_t up(uint64_t x, uint64_t a) { return (x + a - 1) / a * a; }
inline int check(cudaError_t e) { return e == cudaSuccess ? BD_OK : BD_ERR_CUDA; }

// The SMs of the current device, which has to be the one that a handle was made on: its memory and
// the streams that go with it are not the others'.
inline int sm_count(int32_t device, int& sms) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return BD_ERR_CUDA;
  if (dev != device) return BD_ERR_INVALID_ARG;
  return check(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev));
}

// Copies `bytes` (a multiple of 16) of host memory to dst as kernel parameters: the host memory
// may go as soon as the call returns, and the call works during stream capture.
cudaError_t upload(const void* host, uint64_t bytes, void* dst, cudaStream_t s);

// Shared memory of a block: what the kernel declares itself and what its launch adds are together at most
// kDefaultSmem, unless the kernel was allowed more, and kMaxSmem then.  The allowance is the kernel's in
// the whole process, and the last one counts: every launch that may need it asks for all that there is, so
// that none takes away what a call on another thread is about to use.  Kernels that are launched with more
// than kDefaultSmem - kOwnSmem declare at most kOwnSmem.
constexpr uint32_t kDefaultSmem = 48 * 1024, kMaxSmem = 227 * 1024, kOwnSmem = 1024;

// Launches a kernel with programmatic stream serialization: it may be set up while the kernel
// before it on the stream ends (one row's adapter: 8.1 us a call without, 5.0 us with).  Every
// kernel launched this way first waits (after_previous) until all work before it is done and
// visible.  None lets the next one in before it ends: blocks that wait take places where the
// running kernel's next blocks, or clusters, would go (a training step of 2048 rows: 52 us against
// 59 us).  cluster > 1: thread-block clusters.
template <class... P, class... A>
cudaError_t launch(void (*kernel)(P...), dim3 grid, uint32_t threads, uint32_t smem,
                   uint32_t cluster, cudaStream_t s, const A&... args) {
  if (smem > kDefaultSmem - kOwnSmem) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (int)std::max(smem, kMaxSmem - kOwnSmem));
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}
// First in every kernel that launch() starts, in every thread.
__device__ __forceinline__ void after_previous() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
// ---- wide global memory accesses: each byte of a step or an adapter's rows is used once, so
// none of them takes a line of L1.
struct alignas(32) Float8 {
  float v[8];
};
__device__ __forceinline__ Float8 ld8(const float* p) {
  Float8 r;
  asm volatile("ld.global.L1::no_allocate.v8.f32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=f"(r.v[0]), "=f"(r.v[1]), "=f"(r.v[2]), "=f"(r.v[3]), "=f"(r.v[4]),
                 "=f"(r.v[5]), "=f"(r.v[6]), "=f"(r.v[7])
               : "l"(p)
               : "memory");
  return r;
}
__device__ __forceinline__ void st8(float* p, const Float8& r) {
  asm volatile("st.global.L1::no_allocate.v8.f32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p),
               "f"(r.v[0]), "f"(r.v[1]), "f"(r.v[2]), "f"(r.v[3]), "f"(r.v[4]), "f"(r.v[5]),
               "f"(r.v[6]), "f"(r.v[7])
               : "memory");
}
__device__ __forceinline__ uint4 ld16(const void* p) {
  uint4 r;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p)
               : "memory");
  return r;
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
// two floats rounded to nearest, the first in the low half
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

}  // namespace bo
