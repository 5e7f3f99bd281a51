// ssd_linear.cuh -- the cross entropy of a linear head and its gradients
// without stored logits (ssd_linear_ce, ssd_linear_ce_grad): one persistent
// tcgen05 matrix-product kernel in forms that differ in which operands
// they read and in what their epilogue does with a tile.
//
//   lse   z = H W^T            -> per row and vocabulary tile: max, sum exp(z - max); the target's logit
//   grad  G = s (softmax(z) - onehot)  in bf16, one piece of the vocabulary at a time
//   back  dH += G W            -> fp32, one slot per split of the piece
//         dW = G^T H           -> bf16; the tiles of both in one launch, or of one of them
// Measured at 4096 rows of 2048 over 128256 under the power cap: lse 1366
// TFLOP/s, grad 1202 (it writes 1 GB of G and forms the exponentials), dh and dw
// 1230-1330; cuBLAS sustains 1399.  At 64 rows the weight's bytes bound lse, grad
// and dh (5.3-6.4 TB/s) and the written gradient dw (5.3 TB/s).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "../../include/ssd.h"
#include "ssd_device.cuh"
#include "ssd_rows.cuh"

namespace ssd {

constexpr int kGemmThreads = 192;  // warp 0: copies, warp 1: products, warps 2-5: epilogue
constexpr int kAccCols = 256;      // TMEM columns of one accumulator
constexpr int kBlockK = 64;        // one 128-byte swizzle row of bf16
constexpr int kATile = 128 * kBlockK * 2;
constexpr int kOutBuf = 32 * 128;  // one epilogue warp's staging buffer: 32 rows of 128 bytes

// Limit of the product kernel's waits between its roles (a test build shortens it).
#ifndef SSD_GEMM_WAIT_NS
#define SSD_GEMM_WAIT_NS 2000000000ull
#endif
constexpr unsigned long long kGemmWaitNs = SSD_GEMM_WAIT_NS;

enum GemmOp { kOpLse = 0, kOpGrad = 1, kOpBack = 2, kOpDh = 3, kOpDw = 4 };
constexpr bool is_back(int op) { return op >= kOpBack; }

// A pair of CTAs (CG = 2) computes 256 x 256 tiles, each CTA staging half of
// either operand.  A single CTA, for up to 128 rows, where the weight's bytes
// bound the call, computes tiles of 128 x 128: narrow ones leave less of the
// last wave idle (64 rows over 128256: 7 waves of 128 columns against 4 of
// 256).  Its tiles of the back form are 128 x 256: dW, bound by what it writes,
// took 102 us in them against 117 in 128 x 128; dH alone, bound by the weights it
// reads, 82 us in narrow ones against 95.
template <int Op, int CG>
struct GemmShape {
  static constexpr int kTileM = 128 * CG;
  static constexpr int kTileN = Op == kOpBack || Op == kOpDw ? 256 : 128 * CG;
  static constexpr int kBRows = kTileN / CG;  // the CTA's share of the B tile
  static constexpr int kBTile = kBRows * kBlockK * 2;
  static constexpr int kStage = kATile + kBTile;
  static constexpr int kStages = kBRows == 128 ? 6 : 4;
  static constexpr int kSmem = kStages * kStage + 4 * 2 * kOutBuf + 1024;  // and the slack to align to 1 KB
};

// The head of the workspace.
struct LinearHdr {
  int32_t n_active, error;
  float scale_max;  // the largest magnitude among the active rows' scales
};

struct GemmArgs {
  const LinearHdr* hdr;
  int32_t* error;
  const int32_t* target;  // per active row
  const float* scale;
  const float* lse;
  float* zt;        // the target's logit per active row
  float2* part;     // [vocabulary tile][rows]
  int rows;         // padded row count: leading dimension of part, rows of one dh slot
  int V, D;
  int v0, v_count;  // the piece of the vocabulary
  int slots, first; // back: splits of the piece; whether it is the first piece
};

// ---------------------------------------------------------------------------
// tcgen05, tensor copies.
// ---------------------------------------------------------------------------
template <int CG>
__device__ __forceinline__ void tmem_alloc(uint32_t* out, uint32_t cols) {
  if (CG == 1)
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(out)), "r"(cols)
                 : "memory");
  else
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(out)), "r"(cols)
                 : "memory");
}
template <int CG>
__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t cols) {
  if (CG == 1) {
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols) : "memory");
  } else {
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols) : "memory");
  }
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// Shared-memory operand descriptor, 128-byte swizzle.  K-major (rows of 64 k):
// groups of 8 rows lie 1024 bytes apart.  MN-major (rows of 64 m or n, one per
// k): groups of 8 k lie 1024 bytes apart, the next 64 m or n 8192 bytes.
__device__ __forceinline__ uint64_t operand_desc(uint32_t addr, bool mn_major) {
  const uint64_t lbo = mn_major ? (8192u >> 4) : 1u;
  return static_cast<uint64_t>((addr & 0x3FFFFu) >> 4) | (lbo << 16) | (static_cast<uint64_t>(1024u >> 4) << 32) |
         (1ull << 46) | (2ull << 61);
}

template <int CG>
__device__ __forceinline__ void mma_bf16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  if (CG == 1)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc),
        "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc),
        "r"(accumulate)
        : "memory");
}

// Arrives on the barrier (in both CTAs of a pair) when the products issued so
// far have completed.
template <int CG>
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
  if (CG == 1)
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar))
                 : "memory");
  else
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_addr(bar)),
        "h"(static_cast<uint16_t>(3))
        : "memory");
}

// Tile load into this CTA's shared memory; the bytes are counted on the
// barrier at cluster address `bar` (the pair's first CTA when CG = 2).
template <int CG>
__device__ __forceinline__ void tma_load(void* dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  if (CG == 1)
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::
            "r"(smem_addr(dst)),
        "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, "
        "%3}], [%4];" ::"r"(smem_addr(dst)),
        "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void tma_store(const CUtensorMap* map, int x, int y, const void* src) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(map), "r"(x),
               "r"(y), "r"(smem_addr(src))
               : "memory");
}
__device__ __forceinline__ void tma_add(const CUtensorMap* map, int x, int y, const void* src) {
  asm volatile("cp.reduce.async.bulk.tensor.2d.global.shared::cta.add.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(map),
               "r"(x), "r"(y), "r"(smem_addr(src))
               : "memory");
}

// Starts the load of 32 consecutive accumulator columns of the warp's 32 lanes.
__device__ __forceinline__ void tmem_load32(uint32_t addr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr));
}
// The loads above have arrived: r has its values behind this.
__device__ __forceinline__ void tmem_wait(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                 "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                 "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}

// A wait of one of the kernel's roles.  Once one has given up, the kernel's
// other waits in this CTA give up too, and the call is flagged.
template <int CG>
struct GemmWait {
  volatile int* abort;
  int32_t* error;
  static __device__ __forceinline__ bool poll(uint64_t* bar, uint32_t parity) {
    return CG == 1 ? mbar_try_wait(bar, parity, kSuspendHintNs) : mbar_try_wait_cluster(bar, parity);
  }
  __device__ __forceinline__ bool operator()(uint64_t* bar, uint32_t parity) const {
    if (poll(bar, parity)) return true;
    const unsigned long long t0 = global_ns();
    for (uint32_t i = 0; i < (1u << 30); ++i) {
      if (poll(bar, parity)) return true;
      if (*abort || global_ns() - t0 > kGemmWaitNs) break;
    }
    *abort = 1;
    atomicExch(error, 1);
    return false;
  }
};

// One tile of a form's work list.
struct GemmTile {
  int m, n, slot, kb0, kb1;
  bool dw;  // back: of dW, else of dH
};

// The tiles of one group (a CTA, or a pair of them), `count` of them.  lse and
// grad: every step-th tile.  back: every step-th tile of dH, then dW's.  Groups
// that have one dH tile less take `ratio` dW tiles (that tile's cost) among
// themselves before all groups take them in turn, so neighbours in time share
// what they read.
template <int Op, int CG>
struct GemmWork {
  int m_tiles, n_tiles, k_blocks, all;   // dH's in the back form
  int n_dw, k_dw, more, ratio, n_dh;
  int group, step, count;
  __device__ __forceinline__ GemmWork(const GemmArgs& a, int n_active, int g, int groups) {
    const int na = max(n_active, 1);
    constexpr int TM = GemmShape<Op, CG>::kTileM, TN = GemmShape<Op, CG>::kTileN;
    group = g;
    step = groups;
    m_tiles = (na + TM - 1) / TM;
    n_tiles = ((is_back(Op) ? a.D : a.v_count) + TN - 1) / TN;
    k_blocks = ((is_back(Op) ? a.v_count : a.D) + kBlockK - 1) / kBlockK;
    all = !is_back(Op) ? m_tiles * n_tiles : Op != kOpDw ? m_tiles * n_tiles * a.slots : 0;
    count = n_dh = g < all ? (all - g + groups - 1) / groups : 0;
    if (is_back(Op)) {
      n_dw = n_tiles;
      k_dw = (na + kBlockK - 1) / kBlockK;
      const int total = Op != kOpDh ? (a.v_count + TM - 1) / TM * n_dw : 0;
      more = all % groups;  // the groups below have one dH tile more
      const int cost = dw_cost(k_dw), few = groups - more;
      ratio = Op == kOpBack ? min((k_blocks / a.slots + cost / 2) / cost, (total + few - 1) / few) : 0;
      const int own = total - ratio * few;  // tiles of the common turns; may be negative by less than `few`
      if (own >= 0)
        count += (g < more ? 0 : ratio) + (g < own ? (own - g + groups - 1) / groups : 0);
      else
        count += g < more ? 0 : ratio - (g - more >= few + own ? 1 : 0);
    }
  }
  // A dW tile's time in blocks of k: at least its epilogue's.
  static __host__ __device__ __forceinline__ int dw_cost(int k_dw) {
    const int least = CG == 1 ? 2 : 8;
    return k_dw > least ? k_dw : least;
  }
  // Neighbouring tiles share the operand that is dear: the weight tile (lse,
  // grad, dH), or the piece's columns (dW).
  __device__ __forceinline__ GemmTile at(const GemmArgs& a, int i) const {
    GemmTile r;
    r.slot = 0;
    r.kb0 = 0;
    r.dw = Op == kOpDw;
    if (is_back(Op) && i >= n_dh) {
      i -= n_dh;
      const int first = group < more ? 0 : ratio, few = step - more;
      const int t = i < first ? i * few + group - more : ratio * few + (i - first) * step + group;
      r.dw = true;
      r.n = t % n_dw;
      r.m = t / n_dw;
      r.kb1 = k_dw;
      return r;
    }
    int t = group + i * step;
    if (is_back(Op)) {
      r.slot = t / (m_tiles * n_tiles);
      t -= r.slot * m_tiles * n_tiles;
    }
    if (Op == kOpGrad) t = all - 1 - t;  // the forward call went upwards: its last weights may be in L2
    r.m = t % m_tiles;
    r.n = t / m_tiles;
    r.kb1 = k_blocks;
    if (is_back(Op)) {
      r.kb0 = static_cast<int>(static_cast<long long>(k_blocks) * r.slot / a.slots);
      r.kb1 = static_cast<int>(static_cast<long long>(k_blocks) * (r.slot + 1) / a.slots);
    }
    return r;
  }
};

// The tensor maps of a launch; the second set is dW's in the back form.
struct GemmMaps {
  CUtensorMap a, b, out, a2, b2, out2;
};

// r[i], by halving: registers have no index.
__device__ __forceinline__ uint32_t pick32(const uint32_t (&r)[32], int i) {
  uint32_t v[16];
#pragma unroll
  for (int j = 0; j < 16; ++j) v[j] = (i & 16) ? r[j + 16] : r[j];
#pragma unroll
  for (int w = 8; w > 0; w >>= 1)
#pragma unroll
    for (int j = 0; j < w; ++j) v[j] = (i & w) ? v[j + w] : v[j];
  return v[0];
}

// Stages 16 bytes of the lane's row (128 bytes, 128-byte swizzle).
__device__ __forceinline__ void stage16(char* buf, int lane, int chunk, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  *reinterpret_cast<uint4*>(buf + lane * 128 + ((chunk ^ (lane & 7)) << 4)) = make_uint4(x, y, z, w);
}

template <int Op, int CG>
__global__ void __launch_bounds__(kGemmThreads, 1)
    ssd_gemm_kernel(const __grid_constant__ GemmMaps maps, const GemmArgs a) {
  using S = GemmShape<Op, CG>;
  constexpr int kStages = S::kStages, kTileN = S::kTileN;
  constexpr bool kBMn = is_back(Op);
  extern __shared__ char smem_raw[];
  char* smem = reinterpret_cast<char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  char* out_buf = smem + kStages * S::kStage;
  __shared__ uint64_t full[kStages], empty[kStages], tfull[2], tempty[2];
  __shared__ uint32_t tmem_base;
  __shared__ int abort_flag;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = CG == 1 ? 0 : static_cast<int>(cg::this_cluster().block_rank());
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&tfull[i], 1);
      mbar_init(&tempty[i], 4 * CG);
    }
    abort_flag = 0;
    mbar_init_fence();
  }
  if (warp == 1) tmem_alloc<CG>(&tmem_base, 512);
  tc_fence_before();
  if (CG == 1)
    __syncthreads();
  else
    cg::this_cluster().sync();
  tc_fence_after();
  const uint32_t tmem = tmem_base;
  const GemmWait<CG> wait = {&abort_flag, a.error};
  stream_wait();
  const int n_active = a.hdr->n_active;
  const float scale_max = a.hdr->scale_max;
  const GemmWork<Op, CG> work(a, n_active, static_cast<int>(blockIdx.x) / CG, static_cast<int>(gridDim.x) / CG);

  if (warp == 0) {
    if (lane == 0) {
      int s = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int t = 0; ok && t < work.count; ++t) {
        const GemmTile tile = work.at(a, t);
        const int m0 = tile.m * S::kTileM + rank * 128, n0 = tile.n * kTileN + rank * S::kBRows;
        for (int kb = tile.kb0; kb < tile.kb1; ++kb) {
          if (!wait(&empty[s], phase ^ 1)) {
            ok = false;
            break;
          }
          char* pa = smem + s * S::kStage;
          char* pb = pa + kATile;
          const int k0 = kb * kBlockK;
          if (rank == 0) mbar_arrive_expect_tx(&full[s], S::kStage * CG);
          const uint32_t bar = CG == 1 ? smem_addr(&full[s]) : cluster_addr(&full[s], 0);
          if (is_back(Op) && tile.dw) {
            tma_load<CG>(pa, &maps.a2, m0, k0, bar);
            tma_load<CG>(pa + 8192, &maps.a2, m0 + 64, k0, bar);
          } else {
            tma_load<CG>(pa, &maps.a, k0, m0, bar);
          }
          if (kBMn) {
            const CUtensorMap* map = tile.dw ? &maps.b2 : &maps.b;
            const int y = k0 + (tile.dw ? 0 : a.v0);
#pragma unroll
            for (int j = 0; j < S::kBRows / 64; ++j) tma_load<CG>(pb + j * 8192, map, n0 + j * 64, y, bar);
          } else {
            tma_load<CG>(pb, &maps.b, k0, a.v0 + n0, bar);
          }
          if (++s == kStages) {
            s = 0;
            phase ^= 1;
          }
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) {
      // D fp32, A and B bf16, majorness, N / 8, M / 16
      constexpr uint32_t shape = (1u << 4) | (1u << 7) | (1u << 10) | (kBMn ? 1u << 16 : 0u) |
                                 (static_cast<uint32_t>(kTileN / 8) << 17) |
                                 (static_cast<uint32_t>(S::kTileM / 16) << 24);
      int s = 0, acc = 0;
      uint32_t phase = 0, acc_phase = 0;
      bool ok = true;
      for (int t = 0; ok && t < work.count; ++t) {
        const GemmTile tile = work.at(a, t);
        if (tile.kb0 == tile.kb1) continue;
        if (!wait(&tempty[acc], acc_phase ^ 1)) break;
        tc_fence_after();
        const uint32_t d = tmem + acc * kAccCols;
        const bool a_mn = is_back(Op) && tile.dw;
        const uint32_t idesc = shape | (a_mn ? 1u << 15 : 0u);
        const uint64_t a_step = (a_mn ? 2048 : 32) >> 4;
        for (int kb = tile.kb0; kb < tile.kb1; ++kb) {
          if (!wait(&full[s], phase)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t pa = smem_addr(smem + s * S::kStage);
          const uint64_t da = operand_desc(pa, a_mn), db = operand_desc(pa + kATile, kBMn);
#pragma unroll
          for (int k = 0; k < kBlockK / 16; ++k)
            mma_bf16<CG>(d, da + k * a_step,
                         db + static_cast<uint64_t>(k * ((kBMn ? 2048 : 32) >> 4)), idesc,
                         (kb > tile.kb0 || k > 0) ? 1u : 0u);
          mma_commit<CG>(&empty[s]);
          if (++s == kStages) {
            s = 0;
            phase ^= 1;
          }
        }
        if (ok) mma_commit<CG>(&tfull[acc]);
        acc ^= 1;
        if (acc == 0) acc_phase ^= 1;
      }
    }
  } else {
    // Epilogue: warp w reads the accumulator lanes 32 (w mod 4) .. + 31.
    const int quad = warp & 3;
    char* buf = out_buf + (warp - 2) * 2 * kOutBuf;
    int acc = 0, b = 0;
    uint32_t acc_phase = 0;
    for (int t = 0; t < work.count; ++t) {
      const GemmTile tile = work.at(a, t);
      if (tile.kb0 == tile.kb1) continue;
      const int row = tile.m * S::kTileM + rank * 128 + quad * 32 + lane;  // of the product
      const int row0 = row - lane;
      bool live = true;
      int target = -1;
      float scale = 0.f, shift = 0.f;
      if (Op == kOpLse || Op == kOpGrad) {
        live = row < n_active;
        if (live) target = a.target[row] - a.v0 - tile.n * kTileN;
        if (Op == kOpGrad && live) {
          scale = a.scale[row];
          shift = a.lse[row] * kLog2e;
        }
      }
      const int n_valid = a.v_count - tile.n * kTileN;  // lse, grad: columns inside the vocabulary
      // one decision for the warp: lanes that gave up alone would leave the others at its barriers
      if (!__all_sync(0xFFFFFFFFu, wait(&tfull[acc], acc_phase))) break;
      tc_fence_after();
      const uint32_t src = tmem + acc * kAccCols + (static_cast<uint32_t>(quad * 32) << 16);
      float mx = -INFINITY, sum = 0.f;
      const auto chunk = [&](auto of_dw, int c, uint32_t (&r)[32]) {
        constexpr bool kDw = decltype(of_dw)::value;
        if (Op == kOpLse) {
          if (c * 32 + 32 > n_valid) {
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (c * 32 + j >= n_valid) r[j] = 0xFF800000u;
          }
          float m = mx;
#pragma unroll
          for (int j = 0; j < 32; ++j) m = fmaxf(m, __uint_as_float(r[j]));
          const float ref = m > -INFINITY ? m : 0.f;
          float add[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int j = 0; j < 32; ++j) add[j & 3] += ex2((__uint_as_float(r[j]) - ref) * kLog2e);
          sum = sum * ex2((mx - ref) * kLog2e) + ((add[0] + add[1]) + (add[2] + add[3]));
          mx = m;
          if (target >= 0 && (target >> 5) == c) a.zt[row] = __uint_as_float(pick32(r, target & 31));
        } else if (Op == kOpGrad) {
          float g[32];
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            float p = ex2(fmaf(__uint_as_float(r[j]), kLog2e, -shift));
            if (target == c * 32 + j) p -= 1.f;
            g[j] = live && c * 32 + j < n_valid ? p * scale : 0.f;
          }
          const int half = c & 1;
          if (half == 0) {
            if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
            __syncwarp();
          }
#pragma unroll
          for (int q = 0; q < 4; ++q)
            stage16(buf + b * kOutBuf, lane, half * 4 + q, Elem<uint16_t>::pack2(g[q * 8], g[q * 8 + 1]),
                    Elem<uint16_t>::pack2(g[q * 8 + 2], g[q * 8 + 3]), Elem<uint16_t>::pack2(g[q * 8 + 4], g[q * 8 + 5]),
                    Elem<uint16_t>::pack2(g[q * 8 + 6], g[q * 8 + 7]));
          if (half == 1) {
            fence_proxy_async_shared();
            __syncwarp();
            if (lane == 0) {
              tma_store(&maps.out, tile.n * kTileN + (c >> 1) * 64, row0, buf + b * kOutBuf);
              asm volatile("cp.async.bulk.commit_group;" ::: "memory");
            }
            b ^= 1;
          }
        } else if (!kDw) {
          if (tile.n * kTileN + c * 32 < a.D) {  // uniform over the warp
            if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
            __syncwarp();
#pragma unroll
            for (int q = 0; q < 8; ++q)
              stage16(buf + b * kOutBuf, lane, q, r[q * 4], r[q * 4 + 1], r[q * 4 + 2], r[q * 4 + 3]);
            fence_proxy_async_shared();
            __syncwarp();
            if (lane == 0) {
              const int x = tile.n * kTileN + c * 32, y = tile.slot * a.rows + row0;
              if (a.first)
                tma_store(&maps.out, x, y, buf + b * kOutBuf);
              else
                tma_add(&maps.out, x, y, buf + b * kOutBuf);
              asm volatile("cp.async.bulk.commit_group;" ::: "memory");
            }
            b ^= 1;
          }
        } else {
          const int half = c & 1;
          if (tile.n * kTileN + (c >> 1) * 64 < a.D && a.v0 + row0 < a.V) {  // uniform over the warp
#pragma unroll
            for (int j = 0; j < 32; ++j) r[j] = __float_as_uint(__uint_as_float(r[j]) * scale_max);
            if (half == 0) {
              if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
              __syncwarp();
            }
#pragma unroll
            for (int q = 0; q < 4; ++q)
              stage16(buf + b * kOutBuf, lane, half * 4 + q,
                      Elem<uint16_t>::pack2(__uint_as_float(r[q * 8]), __uint_as_float(r[q * 8 + 1])),
                      Elem<uint16_t>::pack2(__uint_as_float(r[q * 8 + 2]), __uint_as_float(r[q * 8 + 3])),
                      Elem<uint16_t>::pack2(__uint_as_float(r[q * 8 + 4]), __uint_as_float(r[q * 8 + 5])),
                      Elem<uint16_t>::pack2(__uint_as_float(r[q * 8 + 6]), __uint_as_float(r[q * 8 + 7])));
            if (half == 1) {
              fence_proxy_async_shared();
              __syncwarp();
              if (lane == 0) {
                tma_store(&maps.out2, tile.n * kTileN + (c >> 1) * 64, a.v0 + row0, buf + b * kOutBuf);
                asm volatile("cp.async.bulk.commit_group;" ::: "memory");
              }
              b ^= 1;
            }
          }
        }
      };
      // 32 columns at a time, the next ones on their way
      const auto walk = [&](auto of_dw) {
        uint32_t r0[32], r1[32];
        tmem_load32(src, r0);
#pragma unroll 1
        for (int c = 0; c < kTileN / 32; c += 2) {
          tmem_wait(r0);
          tmem_load32(src + (c + 1) * 32, r1);
          chunk(of_dw, c, r0);
          tmem_wait(r1);
          if (c + 2 < kTileN / 32) tmem_load32(src + (c + 2) * 32, r0);
          chunk(of_dw, c + 1, r1);
        }
      };
      if (Op == kOpDw || (Op == kOpBack && tile.dw))
        walk(std::true_type());
      else
        walk(std::false_type());
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (CG == 1)
          asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];" ::"r"(smem_addr(&tempty[acc])) : "memory");
        else
          asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(
                           cluster_addr(&tempty[acc], 0))
                       : "memory");
      }
      acc ^= 1;
      if (acc == 0) acc_phase ^= 1;
      if (Op == kOpLse && live) a.part[static_cast<size_t>(tile.n) * a.rows + row] = make_float2(mx, sum);
    }
    if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  }
  __syncthreads();
  if (abort_flag) {  // copies and products may still be in flight: far longer than any of them takes
    const unsigned long long t0 = global_ns();
    for (int i = 0; i < 100000 && global_ns() - t0 < 20000000ull; ++i) __nanosleep(1000);
    __syncthreads();
  }
  if (CG == 2) cg::this_cluster().sync();  // the pair's barriers and accumulators are no longer used
  if (warp == 1) tmem_free<CG>(tmem, 512);
}

// ---------------------------------------------------------------------------
// Before and after the products.
// ---------------------------------------------------------------------------
struct PrepArgs {
  LinearHdr* hdr;
  RowsIn hidden;
  const int32_t* targets;
  const float* row_scale;  // gradient call only; may be NULL
  const float* lse;        // gradient call only
  int32_t* index;          // the active rows' places among the N
  int32_t* target;         // their targets, scales, log-normalisers
  float* scale;
  float* lse_c;
  uint16_t* h;             // their hidden states, dense; for the gradient with zero rows up to a whole block of k
  float* loss;             // forward call: what left-out rows get
  float* lse_out;
  uint16_t* grad_hidden;   // gradient call: likewise
  int32_t* status;         // may be NULL in the gradient call
  int N, V, D;
  int block_rows;          // rows of one block, at most kPrepRows
};
constexpr int kPrepRows = 256;

// Whether row n takes part, and its status where it does not.  A row whose
// log-normaliser or scale is not finite is left out of the gradient: its NaN
// would reach every row of the weight's gradient.
__device__ __forceinline__ bool row_active(const PrepArgs& a, int n, int32_t* status) {
  const int t = a.targets[n];
  *status = 0;
  if (t < 0) return false;
  if (a.row_scale && a.row_scale[n] == 0.f) return false;
  if (t >= a.V) {
    *status = SSD_ROW_BAD_TOKEN;
    return false;
  }
  if ((a.lse && !(fabsf(a.lse[n]) < INFINITY)) || (a.row_scale && !(fabsf(a.row_scale[n]) < INFINITY))) {
    *status = SSD_ROW_NONFINITE;
    return false;
  }
  return true;
}

__global__ void __launch_bounds__(kRowThreads) ssd_linear_prep_kernel(const PrepArgs a) {
  __shared__ int ired[kRowWarps];
  __shared__ float fred[kRowWarps];
  __shared__ int place[kPrepRows];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int n0 = static_cast<int>(blockIdx.x) * a.block_rows;
  stream_wait();
  // Every block counts the rows itself: one launch, and 4 bytes a row from L2.
  int before = 0, total = 0;
  float top = 0.f;
  int32_t st;
  for (int n = tid; n < a.N; n += kRowThreads) {
    const int on = row_active(a, n, &st) ? 1 : 0;
    total += on;
    if (n < n0) before += on;
    if (on && a.row_scale) top = fmaxf(top, fabsf(a.row_scale[n]));
  }
  before = block_reduce(before, ired, OpAdd());
  total = block_reduce(total, ired, OpAdd());
  if (a.scale) {
    // G is formed with each row's share of the largest scale, which itself
    // multiplies the 32-bit sums: equal scales, the usual case, add no rounding.
    top = a.row_scale ? block_reduce(top, fred, OpMax()) : 1.f;
    if (!(top > 0.f && top < INFINITY)) top = 1.f;
  }
  if (blockIdx.x == 0 && tid == 0) *a.hdr = LinearHdr{total, 0, top};
  for (int i0 = 0; warp == 0 && i0 < a.block_rows; i0 += 32) {
    const int i = i0 + lane, n = n0 + i;
    const bool in = i < a.block_rows && n < a.N;
    const bool on = in && row_active(a, n, &st);
    const uint32_t mask = __ballot_sync(0xFFFFFFFFu, on);
    const int at = before + __popc(mask & ((1u << lane) - 1u));
    before += __popc(mask);
    if (in) place[i] = on ? at : -1;
    if (on) {
      a.index[at] = n;
      a.target[at] = a.targets[n];
      if (a.scale) {
        a.scale[at] = a.row_scale ? a.row_scale[n] / top : 1.f;
        a.lse_c[at] = a.lse[n];
        if (a.status) a.status[n] = 0;
      }
    } else if (in) {
      if (a.status) a.status[n] = st;
      if (a.loss) {
        const float v = st ? __int_as_float(0x7FC00000) : 0.f;
        a.loss[n] = v;
        a.lse_out[n] = v;
      }
    }
  }
  __syncthreads();
  const int vecs = a.D / 8;
  for (int i = warp; i < a.block_rows && n0 + i < a.N; i += kRowWarps) {
    const int at = place[i];
    if (at >= 0) {
      const uint4* src = reinterpret_cast<const uint4*>(
          static_cast<const uint16_t*>(a.hidden.base) +
          row_offset(a.hidden.batch_stride, a.hidden.row_stride, a.hidden.rows_per_batch, n0 + i));
      uint4* dst = reinterpret_cast<uint4*>(a.h + static_cast<size_t>(at) * a.D);
      int v = lane;
      for (; v + 96 < vecs; v += 128) {  // four loads in flight
        const uint4 x0 = __ldg(src + v), x1 = __ldg(src + v + 32), x2 = __ldg(src + v + 64), x3 = __ldg(src + v + 96);
        dst[v] = x0, dst[v + 32] = x1, dst[v + 64] = x2, dst[v + 96] = x3;
      }
      for (; v < vecs; v += 32) dst[v] = __ldg(src + v);
    } else if (a.grad_hidden) {
      uint4* dst = reinterpret_cast<uint4*>(a.grad_hidden + static_cast<size_t>(n0 + i) * a.D);
      for (int v = lane; v < vecs; v += 32) dst[v] = make_uint4(0u, 0u, 0u, 0u);
    }
  }
  if (!a.grad_hidden) return;
  // zero rows behind the last active one: dW reads whole blocks of k rows
  const int end = (max(total, 1) + kBlockK - 1) / kBlockK * kBlockK;
  for (int r = total + static_cast<int>(blockIdx.x) * kRowWarps + warp; r < end; r += static_cast<int>(gridDim.x) * kRowWarps) {
    uint4* dst = reinterpret_cast<uint4*>(a.h + static_cast<size_t>(r) * a.D);
    for (int v = lane; v < vecs; v += 32) dst[v] = make_uint4(0u, 0u, 0u, 0u);
  }
}

constexpr int kJoinThreads = 1024;
constexpr int kJoinRows = 8;  // of one block: 128 threads share a row's tiles

// (maximum, sum of exponentials around it), joined.
struct MaxSum {
  float max;
  double sum;
};
__device__ __forceinline__ MaxSum join(const MaxSum& a, const MaxSum& b) {
  const float m = fmaxf(a.max, b.max);
  const float ref = m > -INFINITY ? m : 0.f;
  return MaxSum{m, a.sum * static_cast<double>(ex2((a.max - ref) * kLog2e)) +
                       b.sum * static_cast<double>(ex2((b.max - ref) * kLog2e))};
}

// Joins the vocabulary tiles' maxima and sums, in a fixed order.
__global__ void __launch_bounds__(kJoinThreads)
    ssd_linear_join_kernel(const LinearHdr* hdr, const float2* part, int rows, int tiles, const int32_t* index,
                           const float* zt, float* loss, float* lse, int32_t* status) {
  __shared__ float maxima[32][kJoinRows];
  __shared__ double sums[32][kJoinRows];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, r = tid % kJoinRows;
  const int row0 = static_cast<int>(blockIdx.x) * kJoinRows, row = row0 + r;
  stream_wait();
  const int n_active = hdr->n_active;
  if (row0 >= n_active) return;
  const bool live = row < n_active;
  MaxSum s = {-INFINITY, 0.0};
  constexpr int kStep = kJoinThreads / kJoinRows, kBatch = 8;  // loads in flight
  for (int t0 = tid / kJoinRows; live && t0 < tiles; t0 += kStep * kBatch) {
    float2 p[kBatch];
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int t = t0 + i * kStep;
      p[i] = t < tiles ? part[static_cast<size_t>(t) * rows + row] : make_float2(-INFINITY, 0.f);
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) m = fmaxf(m, p[i].x);
    const float ref = m > -INFINITY ? m : 0.f;
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < kBatch; ++i) sum += p[i].y * ex2((p[i].x - ref) * kLog2e);
    s = join(s, MaxSum{m, static_cast<double>(sum)});
  }
#pragma unroll
  for (int o = kJoinRows; o < 32; o <<= 1) {
    const MaxSum q = {__shfl_down_sync(0xFFFFFFFFu, s.max, o), __shfl_down_sync(0xFFFFFFFFu, s.sum, o)};
    s = join(s, q);
  }
  if (lane < kJoinRows) {
    maxima[warp][lane] = s.max;
    sums[warp][lane] = s.sum;
  }
  __syncthreads();
  if (warp >= kJoinRows) return;
  // a warp per row: lane w holds warp w's
  s = MaxSum{maxima[lane][warp], sums[lane][warp]};
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const MaxSum q = {__shfl_down_sync(0xFFFFFFFFu, s.max, o), __shfl_down_sync(0xFFFFFFFFu, s.sum, o)};
    s = join(s, q);
  }
  const int at = row0 + warp;
  if (lane == 0 && at < n_active) {
    const double l = static_cast<double>(s.max > -INFINITY ? s.max : 0.f) + log(s.sum);
    const int n = index[at];
    const double z = static_cast<double>(zt[at]);
    int32_t st = 0;
    if (!(fabs(l) < INFINITY) || !(fabs(z) < INFINITY)) st |= SSD_ROW_NONFINITE;
    if (hdr->error) st |= SSD_ROW_DEVICE_TIMEOUT;
    const float nan = __int_as_float(0x7FC00000);
    loss[n] = st ? nan : static_cast<float>(l - z);
    lse[n] = st ? nan : static_cast<float>(l);
    status[n] = st;
  }
}

constexpr int kDhThreads = 128;

// Sums dh's slots in order, scales and rounds once, and puts the rows in their
// places.  After a wait that gave up, both gradients are NaN: parts of the
// weight's may be unwritten, and it has no status of its own.
__global__ void __launch_bounds__(kDhThreads)
    ssd_linear_dh_kernel(const LinearHdr* hdr, const float* part, int rows, int slots, int D, const int32_t* index,
                         uint16_t* grad_hidden, uint4* grad_weight, size_t weight_vecs, int32_t* status) {
  const int r = static_cast<int>(blockIdx.x);
  const int d = (static_cast<int>(blockIdx.y) * kDhThreads + static_cast<int>(threadIdx.x)) * 4;
  stream_wait();
  const LinearHdr h = *hdr;
  if (h.error) {
    const size_t step = static_cast<size_t>(gridDim.x) * gridDim.y * kDhThreads;
    for (size_t i = (static_cast<size_t>(blockIdx.y) * gridDim.x + blockIdx.x) * kDhThreads + threadIdx.x;
         i < weight_vecs; i += step)
      grad_weight[i] = make_uint4(0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u);
  }
  if (r >= h.n_active || d >= D) return;
  const int n = index[r];
  if (h.error && status && d == 0) status[n] = SSD_ROW_DEVICE_TIMEOUT;
  const float* src = part + static_cast<size_t>(r) * D + d;
  const size_t step = static_cast<size_t>(rows) * D;
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
  for (int k = 0; k < slots; ++k) {
    const float4 v = *reinterpret_cast<const float4*>(src + k * step);
    s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
  }
  const float f = h.error ? __int_as_float(0x7FC00000) : h.scale_max;
  *reinterpret_cast<uint2*>(grad_hidden + static_cast<size_t>(n) * D + d) =
      make_uint2(Elem<uint16_t>::pack2(s.x * f, s.y * f), Elem<uint16_t>::pack2(s.z * f, s.w * f));
}

}  // namespace ssd
