// bo_adapter_tc.cu -- the adapters' long sums on the fifth-generation tensor cores: low = s A x
// over 128 rows at a time, and the weight gradients' sums over an adapter's rows.
//
// Both are sums of thousands of terms into a narrow result, and what they cost is reading x (or
// dy) once.  With mma.sync the warps spend that time on fragments and barriers: 300 instructions
// a warp and stage, two thirds of the time waiting for one another.  Here eight warps do nothing
// but copy rows into a ring of stages (cp.async: 16 bytes of any row, so that rows need not be
// neighbours in the batch), laid out as the tensor cores read them, and one thread issues the
// products (tcgen05.mma, the sums in tensor memory).  No warp waits for another but through the
// stages' barriers: with one barrier for the block, what the copies, the products and the waits
// cost adds up (0.4 us a stage instead of 0.25).
//
// Every wait is bounded (about two seconds); past its bound a block sets the status, lets its own
// copies land and ends.
#include <cooperative_groups.h>

#include "bo_adapter.cuh"

namespace cg = cooperative_groups;

namespace bo {
namespace {


// ------------------------------------------------------------------------------------ barriers
__device__ __forceinline__ void bar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
// Waits until the barrier's phase of this parity is over; false: it was not within two seconds.
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity) {
  uint64_t t0 = 0;
  for (uint32_t i = 1;; i++) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(bar), "r"(parity)
        : "memory");
    if (done) return true;
    if ((i & 127) == 0) {
      uint64_t now;
      asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(now));
      if (t0 == 0) t0 = now;
      else if (now - t0 > 2000000000ull) return false;
    }
  }
}
// The same for a warp: one lane looks (each lane's look is an access of its own).
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity) {
  int32_t ok = 0;
  if ((threadIdx.x & 31) == 0) ok = bar_wait(bar, parity);
  return __shfl_sync(0xFFFFFFFFu, ok, 0) != 0;
}
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }
// makes copied stages visible to the tensor cores
__device__ __forceinline__ void copies_to_tensor() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// ------------------------------------------------------------------------------- tensor cores
__device__ __forceinline__ void tmem_alloc(uint32_t smem_dst, uint32_t cols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_dst),
               "r"(cols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t cols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols)
               : "memory");
}
__device__ __forceinline__ void tc_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_commit(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
      : "memory");
}
__device__ __forceinline__ void tc_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                       bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
      : "memory");
}
// 16 columns of this warp's 32 lanes, there after tmem_wait()
__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_wait() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

// Shared-memory matrix descriptors: address, the two strides between 8-row (or 8-step) groups and
// between swizzle-wide blocks, and the swizzle (2: 128 bytes, 4: 64, 6: 32).
__device__ __forceinline__ uint64_t matrix(uint32_t addr, uint32_t lead, uint32_t stride,
                                           uint32_t swizzle) {
  return (uint64_t)((addr >> 4) & 0x3FFF) | (uint64_t)((lead >> 4) & 0x3FFF) << 16 |
         (uint64_t)((stride >> 4) & 0x3FFF) << 32 | 1ull << 46 | (uint64_t)swizzle << 61;
}
// BF16 x BF16 into FP32, M = 128; mn: both operands run along their rows / columns (not the sum)
__host__ __device__ constexpr uint32_t instruction(uint32_t n, bool mn) {
  return 1u << 4 | 1u << 7 | 1u << 10 | (mn ? 3u << 15 : 0u) | (n >> 3) << 17 | (128u >> 4) << 24;
}

constexpr uint32_t kMaxStages = 8;
constexpr uint32_t kRingBudget = 200 * 1024;   // one block an SM
constexpr uint32_t kCopyWarps = 8;
constexpr uint32_t kHalves = 2;   // of a stage, each a swizzled line (64 values) wide or 64 rows high

struct alignas(8) Control {
  uint64_t full[kMaxStages], freed[kMaxStages], done[2], drained[2];
  uint32_t tmem, last, pad[2];
  float turn[4][32][17];   // 16 columns of dB of the four warps that write gradients
};

// A product waits for the one before it into the same sums (about 180 cycles, whatever its width),
// so the steps of a stage have sums of their own, as far as `sets` of them fit in tensor memory.
template <int RP, int SETS>
struct Sums {
  static constexpr uint32_t kN = 4 * RP * SETS <= 512 ? 4 : 2;
  static constexpr uint32_t kCols = RP * kN;
  static constexpr uint32_t kAlloc = kCols * SETS;
  // sixteen columns, joined
  static __device__ __forceinline__ void load(uint32_t from, uint32_t col, float (&v)[16]) {
    uint32_t w[kN][16];
#pragma unroll
    for (uint32_t z = 0; z < kN; z++) tmem_ld16(from + z * RP + col, w[z]);
    tmem_wait();
#pragma unroll
    for (int i = 0; i < 16; i++) {
      v[i] = __uint_as_float(w[0][i]);
#pragma unroll
      for (uint32_t z = 1; z < kN; z++) v[i] += __uint_as_float(w[z][i]);
    }
  }
};

__device__ __forceinline__ uint8_t* align1024(uint8_t* p) {
  return p + ((1024 - (smem_addr(p) & 1023)) & 1023);
}

// Barriers and tensor memory of a block; every thread calls it.
__device__ __forceinline__ uint32_t begin_block(Control* ctl, uint32_t stages, uint32_t cols) {
  if (threadIdx.x == 0) {
    for (uint32_t s = 0; s < stages; s++) {
      bar_init(smem_addr(&ctl->full[s]), 32 * kCopyWarps);
      bar_init(smem_addr(&ctl->freed[s]), 1);
    }
    for (uint32_t b = 0; b < 2; b++) {
      bar_init(smem_addr(&ctl->done[b]), 1);
      bar_init(smem_addr(&ctl->drained[b]), 128);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (threadIdx.x < 32) tmem_alloc(smem_addr(&ctl->tmem), cols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  return ctl->tmem;
}
__device__ __forceinline__ void end_block(uint32_t tmem, uint32_t cols) {
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (threadIdx.x < 32) tmem_free(tmem, cols);
}

// A copying warp's turn at stage i: waits for its place (of the ring's S) to be free ...
template <uint32_t S>
__device__ __forceinline__ bool stage_free(Control* ctl, uint32_t i) {
  return i < S || warp_wait(smem_addr(&ctl->freed[i % S]), (i / S + 1) & 1);
}
// ... and lets the stage's barrier know when what this thread has copied into it is there.  The
// copying warps never wait for their copies, and the fence between them and the tensor cores is
// the issuing thread's.  (With both in the copying warps and stages of half the size k_wgrad_tc
// takes 67.7 us instead of 61.3 (59 now) over 8191 rows of 4096 + 11008 features, k_low 33.0 instead of 32.0
// over 16384 rows of 4096; rank 64.)
template <uint32_t S>
__device__ __forceinline__ void stage_issued(Control* ctl, uint32_t i) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(
                   smem_addr(&ctl->full[i % S]))
               : "memory");
}

// ---------------------------------------------------------------------- low = s A x, 128 rows
// Half a stage is 64 values of the sum: 128 rows of x (16 KB) and the factor's rows.  The blocks of
// a cluster split the sum and join through distributed shared memory in a fixed order.  16384 rows
// of 4096, rank 64: 32 us for 134 MB, 4.2 TB/s.  Without the copies of x it is 17 us, without the
// products 31: reading bounds it, on 128 SMs (one tile each).
template <int RP>
struct Low {
  static constexpr uint32_t kThreads = 288;
  static constexpr uint32_t kX = 128 * 128, kHalf = kX + RP * 128, kStage = kHalves * kHalf;
  static constexpr uint32_t kS = kRingBudget / kStage < kMaxStages ? kRingBudget / kStage : kMaxStages;
  static constexpr uint32_t kLd = RP + 4;                            // of the sums in shared memory
  static constexpr uint32_t kPart = 128 * kLd * 4;                   // over the ring
  static constexpr uint32_t kRing = kS * kStage > kPart ? kS * kStage : kPart;
  static constexpr uint32_t kSmem = kRing + sizeof(Control) + 1024;
};

template <int RP>
__global__ void __launch_bounds__(288, 1) k_low(const ApplyArgs P) {
  using L = Low<RP>;
  using M = Sums<RP, 1>;
  constexpr uint32_t S = L::kS;
  extern __shared__ uint8_t raw[];
  uint8_t* const smem = align1024(raw);
  const uint32_t ring = smem_addr(smem);
  float* const part = reinterpret_cast<float*>(smem);
  Control* const ctl = reinterpret_cast<Control*>(smem + L::kRing);
  const cg::cluster_group cluster = cg::this_cluster();
  const uint32_t C = cluster.num_blocks(), c = cluster.block_rank();
  const uint32_t tile = blockIdx.x / C, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  after_previous();
  const Tile T = P.tiles[tile];              // (of the table's capacity, so within it)
  if (tile >= (uint32_t)*P.ntiles) return;   // (the whole cluster)
  const DevAdapter A = P.table[T.adapter];
  const int32_t rank = (int32_t)A.rank;
  const uint32_t all = (P.K + 64 * kHalves - 1) / (64 * kHalves);
  const uint32_t mine = all > c ? (all - c + C - 1) / C : 0;
  // a copying thread's 16-byte slots of a stage: four rows of x, and of the factor's rows
  const uint32_t ch = tid & 7, row0 = tid >> 3;
  const uint16_t* xp[4];
#pragma unroll
  for (int j = 0; j < 4; j++) {   // (past the tile's end: its first row, whose sum is not used)
    const int32_t t = (int32_t)row0 + 32 * j;
    xp[j] = P.x + (int64_t)P.perm[T.start + (t < T.count ? t : 0)] * P.ldx + ch * 8;
  }
  const uint32_t tmem = begin_block(ctl, S, M::kAlloc);
  bool ok = true;

  if (warp < kCopyWarps) {
    const uint32_t at = swz(row0 * 128 + ch * 16);
    for (uint32_t i = 0; i < mine; i++) {
      if (!(ok = stage_free<S>(ctl, i))) break;
#pragma unroll
      for (uint32_t h = 0; h < kHalves; h++) {
        const uint32_t k = ((c + i * C) * kHalves + h) * 64;
        const uint32_t to = ring + i % S * L::kStage + h * L::kHalf + at;
        const bool there = k + ch * 8 < P.K;
#pragma unroll
        for (int j = 0; j < 4; j++) cp16z(to + j * 4096, xp[j] + (there ? k : 0), there);
#pragma unroll
        for (uint32_t j = 0; j < RP; j += 32) {
          const uint32_t row = row0 + j;
          if (RP < 32 && row >= RP) break;
          const bool w = there && (int32_t)row < rank;
          cp16z(to + L::kX + j * 128, A.down + (w ? (uint64_t)row * A.ld_down + k + ch * 8 : 0), w);
        }
      }
      if (!P.stall || i > 0) stage_issued<S>(ctl, i);
    }
    copies_wait();
  } else {
    if (lane == 0) {
      for (uint32_t i = 0; i < mine; i++) {
        const uint32_t s = i % S;
        if (!(ok = bar_wait(smem_addr(&ctl->full[s]), (i / S) & 1))) break;
        copies_to_tensor();
        tc_fence_after();
#pragma unroll
        for (uint32_t h = 0; h < kHalves; h++) {
          const uint64_t a = matrix(ring + s * L::kStage + h * L::kHalf, 16, 1024, 2);
          const uint64_t b = matrix(ring + s * L::kStage + h * L::kHalf + L::kX, 16, 1024, 2);
#pragma unroll
          for (uint32_t k = 0; k < 4; k++)   // 16 values, 32 bytes, a step
            tc_mma(tmem + k % M::kN * RP, a + 2 * k, b + 2 * k, instruction(RP, false),
                   i > 0 || h > 0 || k >= M::kN);
        }
        tc_commit(smem_addr(&ctl->freed[s]));
      }
      tc_commit(smem_addr(&ctl->done[0]));
      // (given up: the others may have too, and nobody else sees that the block's last arrival is in)
      if (!ok) bar_wait(smem_addr(&ctl->done[0]), 0);
    }
    __syncwarp();
  }
  if (warp < kCopyWarps) {   // a warp: 32 rows, half the columns
    ok = warp_wait(smem_addr(&ctl->done[0]), 0) && ok;
    tc_fence_after();
    const uint32_t quarter = warp & 3, row = quarter * 32 + lane;   // tensor memory's lanes
    const uint32_t from = tmem + (quarter << 21);                   // lane in the upper half
    const bool real = (int32_t)row < T.count;
    uint16_t* const to = P.low + (real ? (int64_t)P.perm[T.start + row] * RP : 0);
    for (uint32_t col = (warp >> 2) * 16; col < RP; col += 32) {
      float v[16];
      M::load(from, col, v);
      if (mine == 0) {
#pragma unroll
        for (int i = 0; i < 16; i++) v[i] = 0.f;
      }
      if (C > 1) {
#pragma unroll
        for (int i = 0; i < 16; i += 4)
          *reinterpret_cast<float4*>(part + row * L::kLd + col + i) =
              make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
      } else if (real) {
        uint32_t w[8];
#pragma unroll
        for (int i = 0; i < 8; i++)   // past the rank 0, whatever x holds
          w[i] = pack_bf16((int32_t)col + 2 * i < rank ? v[2 * i] * A.scale : 0.f,
                           (int32_t)col + 2 * i + 1 < rank ? v[2 * i + 1] * A.scale : 0.f);
        *reinterpret_cast<uint4*>(to + col) = make_uint4(w[0], w[1], w[2], w[3]);
        *reinterpret_cast<uint4*>(to + col + 8) = make_uint4(w[4], w[5], w[6], w[7]);
      }
    }
  }
  if (!ok && P.status) *P.status = BD_ERR_CUDA;
  if (C > 1) {
    cluster.sync();
    const uint32_t rows = 128 / C;
    for (uint32_t e = tid * 4; e < rows * RP; e += L::kThreads * 4) {
      const uint32_t row = c * rows + e / RP, col = e % RP;
      if ((int32_t)row >= T.count) continue;
      float4 w[kMaxCluster];   // (all blocks' at once: each is a trip across the cluster)
#pragma unroll
      for (uint32_t b = 0; b < kMaxCluster; b++)
        w[b] = b < C ? *reinterpret_cast<const float4*>(cluster.map_shared_rank(part, b) +
                                                        row * L::kLd + col)
                     : make_float4(0.f, 0.f, 0.f, 0.f);
      float v[4] = {};
#pragma unroll
      for (uint32_t b = 0; b < kMaxCluster; b++) {
        v[0] += w[b].x;
        v[1] += w[b].y;
        v[2] += w[b].z;
        v[3] += w[b].w;
      }
#pragma unroll
      for (int i = 0; i < 4; i++) v[i] = (int32_t)col + i < rank ? v[i] * A.scale : 0.f;
      *reinterpret_cast<uint2*>(P.low + (int64_t)P.perm[T.start + row] * RP + col) =
          make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
    }
    cluster.sync();   // the others may still read `part`
  }
  end_block(tmem, M::kAlloc);
}

// ------------------------------------------------------------------------ weight gradients
// A piece is 128 features of x (for dA) or dy (for dB) of one adapter, a sum over the adapter's
// rows in stages of 64.  The blocks take equal shares of all stages of all pieces, so none waits
// while another works; a piece that several blocks share is joined by the one that ends last, in
// the order of the blocks, from their sums in the workspace.  Four warps carry a piece out while
// the next one's stages arrive and are multiplied into the other set of sums.  8191 rows of 4
// adapters, 4096 and 11008 features, rank 64: 59 us for 247 MB, 4.2 TB/s, of which 53 us are the
// reading and the rest its start and the last piece's join; 2048 rows of 4096 + 4096: 13.3 us.
template <int RP>
struct WgradTc {
  static constexpr uint32_t kThreads = 32 * (kCopyWarps + 1 + 4);
  static constexpr uint32_t kQ = 64 * kFeat * 2, kHalf = kQ + 64 * RP * 2, kStage = kHalves * kHalf;
  static constexpr uint32_t kBox = RP < 64 ? RP : 64;          // columns of low in a swizzled row
  static constexpr uint32_t kLine = kBox * 2;                  // its bytes
  static constexpr uint32_t kSwizzle = RP == 16 ? 6 : RP == 32 ? 4 : 2;
  static constexpr uint32_t kS = kRingBudget / kStage < kMaxStages ? kRingBudget / kStage : kMaxStages;
  static constexpr uint32_t kSmem = kS * kStage + sizeof(Control) + 1024;
  // address of a 16-byte slot of low's rows
  static __device__ __forceinline__ uint32_t at(uint32_t row, uint32_t slot) {
    const uint32_t byte = slot / 8 * 8192 + row * kLine + slot % 8 * 16;
    const uint32_t x = (byte >> 7) & (RP >= 64 ? 7 : RP == 32 ? 3 : 1);
    return byte ^ x << 4;
  }
};

template <int RP>
__global__ void __launch_bounds__(32 * (kCopyWarps + 5), 1) k_wgrad_tc(const WgradArgs P) {
  using L = WgradTc<RP>;
  using M = Sums<RP, 2>;
  constexpr uint32_t S = L::kS;
  extern __shared__ uint8_t raw[];
  uint8_t* const smem = align1024(raw);
  const uint32_t ring = smem_addr(smem);
  Control* const ctl = reinterpret_cast<Control*>(smem + S * L::kStage);
  const uint32_t tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  after_previous();
  const uint32_t hs = (P.hidden + kFeat - 1) / kFeat, slices = hs + (P.out + kFeat - 1) / kFeat;
  const Shares sh((uint64_t)P.blocks[P.k] * slices, gridDim.x);
  if (blockIdx.x >= sh.G) return;
  const uint64_t s_begin = sh.begin(blockIdx.x), s_end = sh.begin(blockIdx.x + 1);
  const uint32_t tmem = begin_block(ctl, S, M::kAlloc);
  bool ok = true;

  if (warp < kCopyWarps) {
    // a warp copies eight rows of a stage; a lane's 16-byte slots are four of x or dy, and of low
    const uint32_t qch = lane & 15, qrow = lane >> 4;
    constexpr uint32_t per = RP / 8, span = 32 / per > 8 ? 8 : 32 / per, PN = 8 / span;
    const uint32_t pch = lane % per, prow = lane / per;
    uint32_t i = 0;
    for (Piece Q(P, slices, s_begin, s_end); !Q.over() && ok; Q.next(P, slices)) {
      const bool down = Q.slice < hs;
      const uint32_t f = (down ? Q.slice : Q.slice - hs) * kFeat + qch * 8;
      const bool there = f < (down ? P.hidden : P.out);
      const uint16_t* const qsrc = (down ? P.x : P.dy) + (there ? f : 0);
      const uint16_t* const psrc = (down ? P.dlow : P.low) + pch * 8;
      const uint64_t ld = down ? P.ldx : P.lddy;
      // row numbers of four stages at once, a lane each, read four stages ahead
      const int32_t start = Q.row0 + (int32_t)(Q.first * 64 + warp * 8), stop = Q.row1;
      auto look = [&](uint32_t j) {   // of stages j .. j + 3
        const int32_t t = start + (int32_t)((j + (lane >> 3)) * 64 + (lane & 7));
        return t < stop ? P.perm[t] : -1;
      };
      int32_t rows = look(0), next = look(4);
      for (uint32_t j = 0; j < Q.mine; j += kHalves, i++) {
        if (j > 0 && j % 4 == 0) {
          rows = next;
          next = look(j + 4);
        }
        if (!(ok = stage_free<S>(ctl, i))) break;
#pragma unroll
        for (uint32_t h = 0; h < kHalves; h++) {
          if (j + h >= Q.mine) break;
          const uint32_t to = ring + i % S * L::kStage + h * L::kHalf, from = (j + h) % 4 * 8;
#pragma unroll
          for (uint32_t u = 0; u < 4; u++) {
            const uint32_t r = qrow + 2 * u;
            const int32_t t = __shfl_sync(0xFFFFFFFFu, rows, from + r);
            cp16z(to + (qch >> 3) * 8192 + swz((warp * 8 + r) * 128 + (qch & 7) * 16),
                  qsrc + (t >= 0 ? t : 0) * ld, t >= 0 && there);
          }
#pragma unroll
          for (uint32_t u = 0; u < PN; u++) {
            const uint32_t r = prow + span * u;
            const int32_t t = __shfl_sync(0xFFFFFFFFu, rows, from + (r & 7));
            if (r < 8)
              cp16z(to + L::kQ + L::at(warp * 8 + r, pch), psrc + (int64_t)(t >= 0 ? t : 0) * RP,
                    t >= 0);
          }
        }
        if (!P.stall || i > 0) stage_issued<S>(ctl, i);
      }
    }
    copies_wait();
  } else if (warp == kCopyWarps) {   // issues the products
    if (lane == 0) {
      uint32_t i = 0, piece = 0;
      for (Piece Q(P, slices, s_begin, s_end); !Q.over() && ok; Q.next(P, slices), piece++) {
        const uint32_t b = piece & 1, d = tmem + b * M::kCols;
        if (piece >= 2 && !(ok = bar_wait(smem_addr(&ctl->drained[b]), (piece / 2 + 1) & 1))) break;
        tc_fence_after();
        for (uint32_t j = 0; j < Q.mine; j += kHalves, i++) {
          const uint32_t s = i % S;
          if (!(ok = bar_wait(smem_addr(&ctl->full[s]), (i / S) & 1))) break;
          copies_to_tensor();
          tc_fence_after();
#pragma unroll
          for (uint32_t h = 0; h < kHalves; h++) {
            if (j + h >= Q.mine) break;
            const uint32_t at = ring + s * L::kStage + h * L::kHalf;
            const uint64_t a = matrix(at, 8192, 1024, 2);
            const uint64_t l = matrix(at + L::kQ, 8192, 8 * L::kLine, L::kSwizzle);
#pragma unroll
            for (uint32_t k = 0; k < 4; k++)   // 16 rows of the batch a step
              tc_mma(d + k % M::kN * RP, a + k * (2048 >> 4), l + k * ((16 * L::kLine) >> 4),
                     instruction(RP, true), j + h > 0 || k >= M::kN);
          }
          tc_commit(smem_addr(&ctl->freed[s]));
        }
        tc_commit(smem_addr(&ctl->done[b]));
        if (!ok) bar_wait(smem_addr(&ctl->done[b]), (piece / 2) & 1);   // (as in k_low)
      }
    }
    __syncwarp();
  } else {   // carries the sums out: a thread has a feature
    const uint32_t quarter = warp & 3, fl = quarter * 32 + lane, t = tid - 32 * (kCopyWarps + 1);
    float(&turn)[32][17] = ctl->turn[quarter];
    auto meet = [](bool yes) {   // of the four warps: whether all say yes
      uint32_t r;
      asm volatile(
          "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
          "barrier.cta.red.and.pred q, 1, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
          : "=r"(r)
          : "r"((uint32_t)yes)
          : "memory");
      return r != 0;
    };
    uint32_t piece = 0;
    DevAdapter A;
    uint32_t known = 0xFFFFFFFFu;
    for (Piece Q(P, slices, s_begin, s_end); !Q.over(); Q.next(P, slices), piece++) {
      const uint32_t b = piece & 1;
      if (Q.adapter != known) A = P.table[known = Q.adapter];
      const bool down = Q.slice < hs, whole = Q.mine == Q.stages;
      const uint32_t f = (down ? Q.slice : Q.slice - hs) * kFeat + fl;
      const bool real = f < (down ? P.hidden : P.out);
      // The parts of a piece are joined from the last block's to the first's.  As a rule the first
      // block ends last, by a long way: then it finds the others' parts while its own stages are
      // still being multiplied, and its own part never leaves the SM.
      uint32_t b0 = blockIdx.x, b1 = blockIdx.x;   // the blocks of the piece's first and last stage
      uint32_t* const count = P.counters + (uint64_t)Q.adapter * slices + Q.slice;
      if (!whole) {
        const uint64_t p_last = Q.begin + Q.stages - 1;
        if (Q.begin < s_begin) b0 = sh.owner(Q.begin);
        if (p_last >= s_end) b1 = sh.owner(p_last);
      }
      bool kept = whole;                           // this block's part stays in tensor memory
      auto look = [&]() {                          // whether the other parts are there
        meet(true);                                // (every warp has read `last` as it was)
        if (t == 0) {
          uint32_t seen;
          asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(seen) : "l"(count) : "memory");
          ctl->last = seen == b1 - b0;
        }
        meet(true);
        const bool r = ctl->last != 0;
        __threadfence();
        return r;
      };
      constexpr uint32_t W = RP < 32 ? RP : 32;    // columns joined at once (64 spill: 66 us, not 59)
      auto join = [&](uint32_t wide, uint32_t q, float (&sum)[W]) {   // block q's first piece, or its last
        const float* p =
            P.sums + (2 * (uint64_t)q + (sh.begin(q) < Q.begin)) * (kFeat * RP) + wide * kFeat + fl;
#pragma unroll
        for (uint32_t j = 0; j < W; j++) sum[j] += __ldcg(p + j * kFeat);
      };
      float sum[W];
#pragma unroll
      for (uint32_t j = 0; j < W; j++) sum[j] = 0.f;
      const bool early = !whole && b0 == blockIdx.x && look();
      if (early) {
        kept = true;
        for (uint32_t q = b1; q > b0; q--) join(0, q, sum);
      }
      if (!(ok = meet(warp_wait(smem_addr(&ctl->done[b]), (piece / 2) & 1)))) break;   // (all or none)
      tc_fence_after();
      const uint32_t from = tmem + b * M::kCols + (quarter << 21);
      bool write = true;
      if (!whole && !early) {
        kept = b0 == blockIdx.x && look();   // (the others are not expected to be last)
        if (!kept) {   // this part to the workspace; the last block to do so joins
          float* const to = P.sums + (2 * (uint64_t)blockIdx.x + (Q.at != s_begin)) * (kFeat * RP) + fl;
#pragma unroll 1
          for (uint32_t col = 0; col < RP; col += 16) {
            float v[16];
            M::load(from, col, v);
#pragma unroll
            for (int j = 0; j < 16; j++) __stcg(to + (col + j) * kFeat, v[j]);
          }
          __threadfence();
          meet(true);
          if (t == 0) ctl->last = atomicAdd(count, 1) == b1 - b0;
          meet(true);
          write = ctl->last != 0;
          __threadfence();
        }
      }
      if (write) {
        if (!whole && t == 0) *count = 0;
#pragma unroll 1
        for (uint32_t wide = 0; wide < RP; wide += W) {
          if (wide > 0) {
#pragma unroll
            for (uint32_t j = 0; j < W; j++) sum[j] = 0.f;
          }
          for (uint32_t q = b1 + 1; q-- > b0;) {
            if (q != blockIdx.x || !kept) {
              if (!early || wide > 0) join(wide, q, sum);
              continue;
            }
#pragma unroll
            for (uint32_t part = 0; part < W; part += 16) {
              float v[16];
              M::load(from, wide + part, v);
#pragma unroll
              for (uint32_t j = 0; j < 16; j++) sum[part + j] += v[j];
            }
          }
#pragma unroll
          for (uint32_t part = 0; part < W; part += 16) {
            const uint32_t col = wide + part;
            const float(&v)[16] = reinterpret_cast<const float(&)[16]>(sum[part]);
            if (col >= A.rank) continue;
            if (!down && (P.accumulate || P.grad_f32 || !A.vec_gup)) {
              // a row's values lie in one thread: handed out, so that sixteen lanes write a row
#pragma unroll
              for (uint32_t j = 0; j < 16; j++) turn[lane][j] = v[j];
              __syncwarp();
              const uint32_t j = lane & 15, row = f - lane + (lane >> 4);   // and every other one
              uint64_t o = (uint64_t)row * A.ld_gup + col + j;
              const uint32_t n = col + j < A.rank && row < P.out ? (P.out - row + 1) / 2 : 0;
#pragma unroll 2
              for (uint32_t r = 0; r < 16 && r < n; r++, o += 2 * (uint64_t)A.ld_gup)
                put_grad(A.gup, o, turn[(lane >> 4) + 2 * r][j], P.grad_f32, P.accumulate);
              __syncwarp();
              continue;
            }
            if (!real) continue;
            if (P.accumulate || P.grad_f32) {
#pragma unroll
              for (uint32_t j = 0; j < 16; j++) {
                if (col + j >= A.rank) break;
                put_grad(A.gdown, (uint64_t)(col + j) * A.ld_gdown + f, v[j], P.grad_f32, P.accumulate);
              }
            } else if (down) {   // neighbouring features in neighbouring lanes
              uint16_t* p = static_cast<uint16_t*>(A.gdown) + (uint64_t)col * A.ld_gdown + f;
#pragma unroll
              for (uint32_t j = 0; j < 16; j++, p += A.ld_gdown)
                if (col + j < A.rank) *p = (uint16_t)pack_bf16(v[j], 0.f);
            } else {   // (the rank is a multiple of 8 here)
              uint16_t* const p = static_cast<uint16_t*>(A.gup) + (uint64_t)f * A.ld_gup + col;
#pragma unroll
              for (uint32_t j = 0; j < 16; j += 8)
                if (col + j < A.rank)
                  *reinterpret_cast<uint4*>(p + j) =
                      make_uint4(pack_bf16(v[j], v[j + 1]), pack_bf16(v[j + 2], v[j + 3]),
                                 pack_bf16(v[j + 4], v[j + 5]), pack_bf16(v[j + 6], v[j + 7]));
            }
          }
        }
      }
      tc_fence_before();
      bar_arrive(smem_addr(&ctl->drained[b]));
    }
  }
  if (!ok && P.status) *P.status = BD_ERR_CUDA;
  end_block(tmem, M::kAlloc);
}

// ------------------------------------------------------------------------------- host side
template <int RP>
cudaError_t low(uint32_t blocks, uint32_t C, const ApplyArgs& P, cudaStream_t s) {
  return launch(k_low<RP>, dim3(blocks), Low<RP>::kThreads, Low<RP>::kSmem, C, s, P);
}
template <int RP>
cudaError_t wgrad(uint32_t grid, const WgradArgs& P, cudaStream_t s) {
  return launch(k_wgrad_tc<RP>, dim3(grid), WgradTc<RP>::kThreads, WgradTc<RP>::kSmem, 1, s, P);
}

}  // namespace

cudaError_t tc_low(uint32_t rp, uint32_t tiles, uint32_t C, const ApplyArgs& P, cudaStream_t s) {
  switch (rp) {
    case 16: return low<16>(tiles * C, C, P, s);
    case 32: return low<32>(tiles * C, C, P, s);
    case 64: return low<64>(tiles * C, C, P, s);
    default: return low<128>(tiles * C, C, P, s);
  }
}

cudaError_t tc_wgrad(uint32_t rp, uint32_t grid, const WgradArgs& P, cudaStream_t s) {
  switch (rp) {
    case 16: return wgrad<16>(grid, P, s);
    case 32: return wgrad<32>(grid, P, s);
    case 64: return wgrad<64>(grid, P, s);
    default: return wgrad<128>(grid, P, s);
  }
}

}  // namespace bo
