// ssd_train.cu -- host side of the draft-training calls of include/ssd.h:
// ssd_teacher_top, ssd_distill (ssd_rows.cuh), ssd_linear_ce and
// ssd_linear_ce_grad (ssd_linear.cuh).
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <map>
#include <mutex>
#include <utility>

#include "../../include/ssd.h"
#include "ssd_device.cuh"
#include "ssd_linear.cuh"
#include "ssd_rows.cuh"

namespace ssd {

static std::mutex g_fn_mu;
static std::map<std::pair<const void*, int>, int> g_fn_smem;

// Raises a kernel's dynamic shared-memory limit on the current device, once.
// Nothing is thrown past the C entry points.
static cudaError_t allow_smem(const void* fn, int bytes) try {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::lock_guard<std::mutex> lock(g_fn_mu);
  int& have = g_fn_smem[std::make_pair(fn, dev)];
  if (have >= bytes) return cudaSuccess;
  e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) have = bytes;
  return e;
} catch (...) {
  return cudaErrorMemoryAllocation;
}

// Launches a kernel as a programmatic dependent of the one before it in the
// stream (it waits for that one itself), in clusters of `cluster` blocks.
template <typename... P, typename... A>
static ssd_status launch_dependent(void (*fn)(P...), dim3 grid, int threads, int smem, int cluster, cudaStream_t stream,
                                   const A&... args) {
  if (smem > 0 && allow_smem(reinterpret_cast<const void*>(fn), smem) != cudaSuccess) return SSD_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = stream;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  at[1].val.clusterDim.y = 1;
  at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = cluster > 0 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, fn, args...) == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

// ---------------------------------------------------------------------------
// Rows in cluster shared memory.
// ---------------------------------------------------------------------------
// Bytes of a row that one CTA stages.  Four such CTAs of the distillation fit an
// SM; of the top kernel, whose own shared memory is larger, four up to slices of
// 51,456 bytes (128256 bf16 gives 51,312) and three above.
constexpr long long kSliceTarget = 52 * 1024;
constexpr long long kSliceMin = 8 * 1024;      // do not split a row finer than this for the sake of few rows
constexpr long long kSliceMax = 200 * 1024;
constexpr int kSmCount = 148;
constexpr long long kRowOne = 66 * 1024;
constexpr int kRowFill = 2 * kSmCount;              // CTAs that fill the GPU

struct RowPlan {
  int cluster, slice_vecs, smem;
};

// CTAs per row and the 16-byte vectors of a slice; false when the row does
// not fit the cluster's shared memory.
static bool row_plan(long long rows, int V, int esize, RowPlan* p) {
  const long long vecs = (static_cast<long long>(V) * esize + 15) / 16 + 1;  // a row may start inside a vector
  const long long bytes = vecs * 16;
  long long c = (bytes + kSliceTarget - 1) / kSliceTarget;
  const long long fill = (kRowFill + rows - 1) / rows, by_len = bytes / kSliceMin;
  const long long extra = fill < by_len ? fill : by_len;
  if (c < extra) c = extra;
  // a block of its own for a short row, when there are enough of them: 384 rows
  // of 62 KB 18.5 us against 22.8 in pairs, 80 of them 12.3 against 10.3
  if (bytes <= kRowOne && rows >= kRowFill) c = 1;
  if (c > kMaxRowCluster) c = kMaxRowCluster;
  const long long sv = (vecs + c - 1) / c;
  if (sv * 16 > kSliceMax) return false;
  p->cluster = static_cast<int>(c);
  p->slice_vecs = static_cast<int>(sv);
  p->smem = static_cast<int>(sv * 16);
  return true;
}

// The top logits: slices of a row for as many CTAs, each row's own or joined.
struct TopPlan {
  int slices, slice_vecs, smem;
  size_t keys, total;  // workspace: the slices' records, then their sorted keys
};

static bool top_plan(long long rows, int V, int esize, TopPlan* p) {
  const long long vecs = (static_cast<long long>(V) * esize + 15) / 16 + 1;  // a row may start inside a vector
  const long long bytes = vecs * 16;
  long long n = (bytes + kSliceTarget - 1) / kSliceTarget;
  const long long fill = (kRowFill + rows - 1) / rows, by_len = bytes / kSliceMin;
  const long long extra = fill < by_len ? fill : by_len;
  if (n < extra) n = extra;
  // One slice, and no join, where that costs less: 384 rows of 62 KB 16.5 us
  // against 23.9; but 384 of 195 KB 43 against 33 (and 97 KB the same).  Few rows
  // in one slice against several, 64 logits kept: 1, 32 and 148 of 125 KB 13.9,
  // 15.0 and 17.0 us against 15.0, 19.4 and 18.8; of 199 KB bf16 16.0, 18.2 and
  // 21.5 against 14.7, 20.7 and 22.3 (fp32, and 200 kept: less in one).
  if (bytes <= kRowOne || (rows <= kSmCount && bytes <= kSliceMax)) n = 1;
  if (n > kTopSlices) n = kTopSlices;
  const long long need = (bytes + kSliceMax - 1) / kSliceMax;
  if (n < need) n = need;
  if (n > kMaxTopSlices || rows * n > 0x7FFFFFFFLL) return false;
  const long long sv = (vecs + n - 1) / n;
  p->slices = static_cast<int>(n);
  p->slice_vecs = static_cast<int>(sv);
  p->smem = static_cast<int>(n > 1 || sv * 16 > static_cast<long long>(sizeof(TopFinish)) ? sv * 16 : sizeof(TopFinish));
  p->keys = p->total = 0;
  if (n > 1) {
    p->keys = static_cast<size_t>(rows * n) * sizeof(TopSlice);
    p->total = p->keys + static_cast<size_t>(rows * n) * kPool * 8;
  }
  return true;
}

// Workspace that serves `rows` rows and every smaller number of them: few rows
// are cut into more slices, so a plan's own need is not monotone.  From kRowFill
// rows on the slices of a row no longer depend on their number.
static size_t top_workspace(long long rows, int V, int esize) {
  TopPlan p;
  if (!top_plan(rows, V, esize, &p)) return 0;
  size_t most = p.total;
  for (long long r = 1; r < rows && r <= kRowFill; ++r)
    if (top_plan(r, V, esize, &p) && p.total > most) most = p.total;
  return most;
}

// Checks common to the row calls.
static ssd_status check_rows(int dtype, int n_batch, int rows_per_batch, int V, int64_t batch_stride,
                             int64_t row_stride, float T, int M) {
  if (dtype != SSD_DTYPE_BF16 && dtype != SSD_DTYPE_FP32) return SSD_ERR_DTYPE;
  if (n_batch < 0 || rows_per_batch < 0 || V < 1 || M < 1 || M > SSD_MAX_TOP || M > V) return SSD_ERR_INVALID_ARG;
  if (!(T >= SSD_MIN_TRAIN_T && T <= SSD_MAX_TRAIN_T)) return SSD_ERR_INVALID_ARG;
  if (batch_stride < 0 || row_stride < 0) return SSD_ERR_INVALID_ARG;
  if (static_cast<long long>(n_batch) * rows_per_batch > 0x7FFFFFFFLL / kMaxRowCluster) return SSD_ERR_INVALID_ARG;
  return SSD_OK;
}

static bool aligned_to(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

// ---------------------------------------------------------------------------
// The linear head.
// ---------------------------------------------------------------------------
typedef CUresult (*EncodeTiled)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The driver's tensor-map encoder, looked up once (libcuda is not linked).
static EncodeTiled encode_tiled() {
  static EncodeTiled fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<EncodeTiled>(p);
  }();
  return fn;
}

// A row-major [rows, cols] matrix copied in boxes of 128-byte rows, swizzled.
static bool tile_map(CUtensorMap* m, const void* base, bool fp32, long long cols, long long rows, long long row_bytes,
                     int box_rows) {
  const EncodeTiled fn = encode_tiled();
  if (!fn) return false;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(row_bytes)};
  const cuuint32_t box[2] = {fp32 ? 32u : 64u, static_cast<cuuint32_t>(box_rows)};
  const cuuint32_t step[2] = {1u, 1u};
  return fn(m, fp32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base),
            dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr long long kPieceBytes = 256ll << 20;  // of the gradient's logits, kept at a time
constexpr long long kBothBytes = 128ll << 20;  // a piece of G that L2 holds
constexpr int kMaxSlots = 32;

// Sizes of one call, and where its workspace holds what.
struct LinearPlan {
  int cg;            // CTAs of one product tile
  int rows;          // N rounded up to whole tiles
  int tiles;         // vocabulary tiles of the forward call
  int piece;         // vocabulary of one piece of the gradient
  int slots;         // splits of a piece's k axis in dh
  bool both;         // dh and dw in one launch
  size_t hdr, index, target, scale, lse, zt, h, part, g, dh, total;
};

static LinearPlan linear_plan(int N, int D, int V, bool grad) {
  LinearPlan p = {};
  p.cg = N > 128 ? 2 : 1;
  const int tm = 128 * p.cg, tn = tm;
  p.rows = (N + tm - 1) / tm * tm;
  p.tiles = (V + tn - 1) / tn;
  const long long v_up = (V + 255ll) / 256 * 256;  // dw's tiles are 256 high
  const long long fit = kPieceBytes / (2ll * p.rows) / 256 * 256;
  p.piece = static_cast<int>(fit < 256 ? 256 : (fit > v_up ? v_up : fit));
  // One launch for dH and dW where L2 holds the piece of G that both read: both
  // gradients of 5 rows of 512 over 5003 22.6 us against 24.6, of 384 of 2048 over
  // 32000 171 against 176, most sizes within 1%; but 2048 of 2048 over 128256 (two
  // pieces of 256 MB) 2503 against 2328.  For single CTAs also where L2 holds the
  // weight (64 rows of 2048 over 128256 294 against 289).
  p.both = 2ll * p.rows * p.piece <= kBothBytes && (p.cg == 2 || 2ll * V * D <= kBothBytes);
  const long long dh_cols = p.both ? 256 : 128 * p.cg;
  const long long v_piece = V < p.piece ? V : p.piece, d_tiles = (D + dh_cols - 1) / dh_cols, groups = kSmCount / p.cg;
  const long long dh_tiles = p.rows / tm * d_tiles, dw_tiles = (v_piece + tm - 1) / tm * d_tiles;
  const long long blocks = (v_piece + kBlockK - 1) / kBlockK, dw_blocks = (N + kBlockK - 1) / kBlockK;
  p.slots = 1;
  if (p.both) {
    // splits of k in dH: the fewest that leave no dH tile with more than half of a group's work
    const long long least = p.cg == 1 ? GemmWork<kOpBack, 1>::dw_cost(static_cast<int>(dw_blocks))
                                      : GemmWork<kOpBack, 2>::dw_cost(static_cast<int>(dw_blocks));
    const long long half = (dh_tiles * blocks + dw_tiles * least) / (2 * groups);
    while (p.slots < kMaxSlots && blocks / (p.slots + 1) >= 8 && blocks > half * p.slots) ++p.slots;
  } else {
    // the fewest whole waves of tiles per split, few splits where they make no difference
    double best = 1e30;
    for (int k = 1; k <= kMaxSlots && (k == 1 || blocks / k >= 8); ++k) {
      const double waves = static_cast<double>((dh_tiles * k + groups - 1) / groups) / k * (1.0 + 0.01 * k);
      if (waves < best) {
        best = waves;
        p.slots = k;
      }
    }
  }
  size_t off = 0;
  const auto take = [&off](size_t bytes) {
    const size_t at = off;
    off += (bytes + 255) / 256 * 256;
    return at;
  };
  const size_t r = static_cast<size_t>(p.rows);
  p.hdr = take(sizeof(LinearHdr));
  p.index = take(r * 4);
  p.target = take(r * 4);
  p.h = take(r * static_cast<size_t>(D) * 2);
  if (grad) {
    p.scale = take(r * 4);
    p.lse = take(r * 4);
    p.g = take(r * static_cast<size_t>(p.piece) * 2);
    p.dh = take(r * static_cast<size_t>(p.slots) * static_cast<size_t>(D) * 4);
  } else {
    p.zt = take(r * 4);
    p.part = take(r * static_cast<size_t>(p.tiles) * 8);
  }
  p.total = off;
  return p;
}

// Workspace that serves N rows and every smaller number of them: splits and
// pieces jump with the row tiles, so a plan's own need is not monotone.  A plan
// changes at multiples of kBlockK rows only.
static size_t linear_workspace(int N, int D, int V, bool grad) {
  size_t most = linear_plan(N, D, V, grad).total;
  for (int n = kBlockK; n < N; n += kBlockK) {
    const size_t need = linear_plan(n, D, V, grad).total;
    if (need > most) most = need;
  }
  return most;
}

template <int Op, int CG>
static ssd_status launch_gemm(const GemmMaps& maps, const GemmArgs& a, long long most_tiles, cudaStream_t stream) {
  const long long fit = kSmCount / CG;
  const long long groups = most_tiles < fit ? most_tiles : fit;
  return launch_dependent(&ssd_gemm_kernel<Op, CG>, dim3(static_cast<unsigned>(groups * CG)), kGemmThreads,
                          GemmShape<Op, CG>::kSmem, CG, stream, maps, a);
}

static ssd_status check_linear(int dtype, int n_batch, int rows_per_batch, int D, int V, int64_t batch_stride,
                               int64_t row_stride, int64_t weight_stride) {
  if (dtype != SSD_DTYPE_BF16) return SSD_ERR_DTYPE;
  if (n_batch < 0 || rows_per_batch < 0 || D < 8 || D % 8 != 0 || D > SSD_MAX_LINEAR_D || V < 1 ||
      V > SSD_MAX_LINEAR_V)
    return SSD_ERR_INVALID_ARG;
  if (static_cast<long long>(n_batch) * rows_per_batch > SSD_MAX_LINEAR_N) return SSD_ERR_INVALID_ARG;
  if (batch_stride < 0 || row_stride < 0 || batch_stride % 8 != 0 || row_stride % 8 != 0) return SSD_ERR_INVALID_ARG;
  if (weight_stride < D || weight_stride % 8 != 0 || weight_stride >= (1ll << 38)) return SSD_ERR_INVALID_ARG;
  return SSD_OK;
}

// Whether a dense block shares a byte with rows of `len` bytes, `step` apart.
static bool overlaps(const void* block, size_t bytes, const void* base, long long rows, long long len, long long step) {
  const long long p = static_cast<long long>(reinterpret_cast<intptr_t>(block)),
                  b = static_cast<long long>(reinterpret_cast<intptr_t>(base));
  const long long r = p < b + len ? 0 : (step > 0 ? (p - b - len) / step + 1 : rows);  // the first row that ends behind p
  return r < rows && b + r * step < p + static_cast<long long>(bytes);
}

static void prep_args(PrepArgs* a, const LinearPlan& p, char* ws, const RowsIn& hidden, const int32_t* targets, int N,
                      int V, int D) {
  *a = PrepArgs{};
  a->hdr = reinterpret_cast<LinearHdr*>(ws + p.hdr);
  a->hidden = hidden;
  a->targets = targets;
  a->index = reinterpret_cast<int32_t*>(ws + p.index);
  a->target = reinterpret_cast<int32_t*>(ws + p.target);
  a->h = reinterpret_cast<uint16_t*>(ws + p.h);
  a->N = N;
  a->V = V;
  a->D = D;
}

// Few rows per block, so that the copies spread over the GPU; every block
// reads all targets, so no more than 1024 blocks.
static ssd_status launch_prep(PrepArgs& a, cudaStream_t stream) {
  static_assert(SSD_MAX_LINEAR_N <= 1024 * kPrepRows, "a block's rows");
  int rows = (a.N + 1023) / 1024;
  if (rows < kRowWarps) rows = kRowWarps;
  a.block_rows = rows;
  const int blocks = (a.N + rows - 1) / rows;
  const int zero = a.grad_hidden ? kBlockK / kRowWarps : 1;  // blocks that clear the rows behind the last
  return launch_dependent(&ssd_linear_prep_kernel, dim3(static_cast<unsigned>(blocks < zero ? zero : blocks)),
                          kRowThreads, 0, 0, stream, a);
}

static GemmArgs gemm_args(const LinearPlan& p, char* ws, int V, int D) {
  GemmArgs g = {};
  g.hdr = reinterpret_cast<const LinearHdr*>(ws + p.hdr);
  g.error = &reinterpret_cast<LinearHdr*>(ws + p.hdr)->error;
  g.target = reinterpret_cast<const int32_t*>(ws + p.target);
  g.rows = p.rows;
  g.V = V;
  g.D = D;
  return g;
}

template <int CG>
static ssd_status linear_forward(const LinearPlan& p, char* ws, const void* weight, long long ws_bytes_row, int N, int D,
                                 int V, float* loss, float* lse, int32_t* status, cudaStream_t stream) {
  GemmMaps maps = {};
  if (!tile_map(&maps.a, ws + p.h, false, D, N, 2ll * D, 128) ||
      !tile_map(&maps.b, weight, false, D, V, ws_bytes_row, GemmShape<kOpLse, CG>::kBRows))
    return SSD_ERR_CUDA;
  GemmArgs g = gemm_args(p, ws, V, D);
  g.v_count = V;
  g.zt = reinterpret_cast<float*>(ws + p.zt);
  g.part = reinterpret_cast<float2*>(ws + p.part);
  const long long most = static_cast<long long>(p.rows / GemmShape<kOpLse, CG>::kTileM) * p.tiles;
  const ssd_status st = launch_gemm<kOpLse, CG>(maps, g, most, stream);
  if (st != SSD_OK) return st;
  return launch_dependent(&ssd_linear_join_kernel, dim3(static_cast<unsigned>((N + kJoinRows - 1) / kJoinRows)),
                          kJoinThreads, 0, 0, stream, g.hdr, static_cast<const float2*>(g.part), p.rows, p.tiles,
                          reinterpret_cast<const int32_t*>(ws + p.index), static_cast<const float*>(g.zt), loss, lse,
                          status);
}

template <int CG>
static ssd_status linear_backward(const LinearPlan& p, char* ws, const void* weight, long long ws_bytes_row, int N,
                                  int D, int V, void* grad_hidden, void* grad_weight, int32_t* status,
                                  cudaStream_t stream) {
  using S = GemmShape<kOpGrad, CG>;
  using W = GemmShape<kOpBack, CG>;
  // The maps end at row N: what a tile reads behind it is zero and costs no traffic.
  GemmMaps grad = {}, back = {};
  if (!tile_map(&grad.a, ws + p.h, false, D, N, 2ll * D, 128) ||
      !tile_map(&grad.b, weight, false, D, V, ws_bytes_row, S::kBRows) ||
      !tile_map(&grad.out, ws + p.g, false, p.piece, N, 2ll * p.piece, 32) ||
      !tile_map(&back.a, ws + p.g, false, p.piece, N, 2ll * p.piece, 128) ||
      !tile_map(&back.b, weight, false, D, V, ws_bytes_row, 64) ||
      !tile_map(&back.out, ws + p.dh, true, D, static_cast<long long>(p.rows) * p.slots, 4ll * D, 32) ||
      !tile_map(&back.a2, ws + p.g, false, p.piece, N, 2ll * p.piece, 64) ||
      !tile_map(&back.b2, ws + p.h, false, D, N, 2ll * D, 64) ||
      !tile_map(&back.out2, grad_weight, false, D, V, 2ll * D, 32))
    return SSD_ERR_CUDA;
  GemmArgs g = gemm_args(p, ws, V, D);
  g.scale = reinterpret_cast<const float*>(ws + p.scale);
  g.lse = reinterpret_cast<const float*>(ws + p.lse);
  g.slots = p.slots;
  const long long m_tiles = p.rows / S::kTileM, d_tiles = (D + W::kTileN - 1) / W::kTileN;
  const long long dh_cols = p.both ? W::kTileN : GemmShape<kOpDh, CG>::kTileN;
  for (long long v0 = 0; v0 < V; v0 += p.piece) {
    g.v0 = static_cast<int>(v0);
    g.v_count = static_cast<int>(V - v0 < p.piece ? V - v0 : p.piece);
    g.first = v0 == 0;
    const long long v_tiles = (g.v_count + S::kTileN - 1) / S::kTileN;
    ssd_status st = launch_gemm<kOpGrad, CG>(grad, g, m_tiles * v_tiles, stream);
    const long long dh_most = m_tiles * p.slots * ((D + dh_cols - 1) / dh_cols);
    const long long dw_most = (g.v_count + W::kTileM - 1ll) / W::kTileM * d_tiles;
    if (st == SSD_OK)
      st = p.both ? launch_gemm<kOpBack, CG>(back, g, dh_most + dw_most, stream)
                  : launch_gemm<kOpDh, CG>(back, g, dh_most, stream);
    if (st == SSD_OK && !p.both) st = launch_gemm<kOpDw, CG>(back, g, dw_most, stream);
    if (st != SSD_OK) return st;
  }
  const dim3 grid(static_cast<unsigned>(N), static_cast<unsigned>((D / 4 + kDhThreads - 1) / kDhThreads));
  return launch_dependent(&ssd_linear_dh_kernel, grid, kDhThreads, 0, 0, stream, g.hdr,
                          reinterpret_cast<const float*>(ws + p.dh), p.rows, p.slots, D,
                          reinterpret_cast<const int32_t*>(ws + p.index), static_cast<uint16_t*>(grad_hidden),
                          static_cast<uint4*>(grad_weight), static_cast<size_t>(V) * D / 8, status);
}

}  // namespace ssd

using namespace ssd;

extern "C" {

size_t ssd_teacher_top_workspace_bytes(int rows, int V, int dtype, int M) {
  if (check_rows(dtype, 1, rows, V, 0, 0, 1.f, M) != SSD_OK || rows == 0) return 0;
  return top_workspace(rows, V, dtype == SSD_DTYPE_FP32 ? 4 : 2);
}

ssd_status ssd_teacher_top(const void* logits, int dtype, int n_batch, int rows_per_batch, int V, int64_t batch_stride,
                           int64_t row_stride, float T, int M, int32_t* tokens, float* values, float* lse, float* tail,
                           int32_t* status, void* workspace, size_t ws_bytes, void* stream) {
  const ssd_status st = check_rows(dtype, n_batch, rows_per_batch, V, batch_stride, row_stride, T, M);
  if (st != SSD_OK) return st;
  const long long rows = static_cast<long long>(n_batch) * rows_per_batch;
  if (rows == 0) return SSD_OK;
  if (!logits || !tokens || !values || !lse || !tail || !status) return SSD_ERR_INVALID_ARG;
  const int esize = dtype == SSD_DTYPE_FP32 ? 4 : 2;
  if (!aligned_to(logits, esize) || !aligned_to(workspace, 256)) return SSD_ERR_ALIGNMENT;
  TopPlan p;
  if (!top_plan(rows, V, esize, &p)) return SSD_ERR_UNSUPPORTED;
  if (p.total > 0 && (!workspace || ws_bytes < p.total)) return SSD_ERR_WORKSPACE;
  TopArgs a;
  const bool one = n_batch == 1 || batch_stride == row_stride * rows_per_batch;
  a.in = RowsIn{logits, batch_stride, row_stride, one ? 0 : rows_per_batch};
  a.tokens = tokens;
  a.values = values;
  a.lse = lse;
  a.tail = tail;
  a.status = status;
  a.slices = static_cast<TopSlice*>(workspace);
  a.keys = reinterpret_cast<unsigned long long*>(static_cast<char*>(workspace) + p.keys);
  a.V = V;
  a.M = M;
  a.slice_vecs = p.slice_vecs;
  a.n_slices = p.slices;
  a.inv_t = 1.0 / static_cast<double>(T);
  a.log2e_t = static_cast<float>(1.4426950408889634 * a.inv_t);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  void (*fn)(TopArgs) = dtype == SSD_DTYPE_BF16 ? &ssd_top_kernel<uint16_t> : &ssd_top_kernel<float>;
  const ssd_status done =
      launch_dependent(fn, dim3(static_cast<unsigned>(rows * p.slices)), kRowThreads, p.smem, 0, s, a);
  if (done != SSD_OK || p.slices == 1) return done;
  return launch_dependent(&ssd_top_join_kernel, dim3(static_cast<unsigned>(rows)), kRowThreads,
                          (p.slices * kPool + 2) * 8, 0, s, a);
}

ssd_status ssd_distill(const void* logits, int dtype, int n_batch, int rows_per_batch, int V, int64_t batch_stride,
                       int64_t row_stride, float T, int M, const int32_t* tokens, const float* values,
                       const float* tail, const float* row_scale, float* loss, int32_t* status, void* grad,
                       int64_t grad_batch_stride, int64_t grad_row_stride, void* stream) {
  const ssd_status st = check_rows(dtype, n_batch, rows_per_batch, V, batch_stride, row_stride, T, M);
  if (st != SSD_OK) return st;
  // rows of the gradient must not overlap
  if (grad && ((rows_per_batch > 1 && grad_row_stride < V) || (n_batch > 1 && grad_batch_stride < V)))
    return SSD_ERR_INVALID_ARG;
  const long long rows = static_cast<long long>(n_batch) * rows_per_batch;
  if (rows == 0) return SSD_OK;
  if (!logits || !tokens || !values || !loss || !status) return SSD_ERR_INVALID_ARG;
  const int esize = dtype == SSD_DTYPE_FP32 ? 4 : 2;
  if (!aligned_to(logits, esize) || !aligned_to(grad, esize)) return SSD_ERR_ALIGNMENT;
  RowPlan p;
  if (!row_plan(rows, V, esize, &p)) return SSD_ERR_UNSUPPORTED;
  DistillArgs a;
  // rows of one stride need no division by rows_per_batch
  const auto flat = [&](int64_t b, int64_t r) { return n_batch == 1 || b == r * rows_per_batch; };
  const bool one = flat(batch_stride, row_stride) && (!grad || flat(grad_batch_stride, grad_row_stride));
  a.in = RowsIn{logits, batch_stride, row_stride, one ? 0 : rows_per_batch};
  a.tokens = tokens;
  a.values = values;
  a.tail = tail;
  a.row_scale = row_scale;
  a.loss = loss;
  a.status = status;
  a.grad = grad;
  a.g_batch_stride = grad_batch_stride;
  a.g_row_stride = grad_row_stride;
  a.V = V;
  a.M = M;
  a.slice_vecs = p.slice_vecs;
  a.inv_t = 1.0 / static_cast<double>(T);
  a.log2e_t = static_cast<float>(1.4426950408889634 * a.inv_t);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  void (*fn)(DistillArgs) = dtype == SSD_DTYPE_BF16 ? &ssd_distill_kernel<uint16_t> : &ssd_distill_kernel<float>;
  return launch_dependent(fn, dim3(static_cast<unsigned>(rows * p.cluster)), kRowThreads, p.smem, p.cluster, s, a);
}

size_t ssd_linear_ce_workspace_bytes(int N, int D, int V, int grad) {
  if (N < 0 || N > SSD_MAX_LINEAR_N || D < 8 || D % 8 != 0 || D > SSD_MAX_LINEAR_D || V < 1 || V > SSD_MAX_LINEAR_V)
    return 0;
  return linear_workspace(N > 0 ? N : 1, D, V, grad != 0);
}

ssd_status ssd_linear_ce(const void* hidden, const void* weight, int dtype, int n_batch, int rows_per_batch, int D,
                         int V, int64_t batch_stride, int64_t row_stride, int64_t weight_stride,
                         const int32_t* targets, float* loss, float* lse, int32_t* status, void* workspace,
                         size_t ws_bytes, void* stream) {
  ssd_status st = check_linear(dtype, n_batch, rows_per_batch, D, V, batch_stride, row_stride, weight_stride);
  if (st != SSD_OK) return st;
  const int N = n_batch * rows_per_batch;
  if (N == 0) return SSD_OK;
  if (!hidden || !weight || !targets || !loss || !lse || !status) return SSD_ERR_INVALID_ARG;
  if (!aligned_to(hidden, 16) || !aligned_to(weight, 16) || !aligned_to(workspace, 256)) return SSD_ERR_ALIGNMENT;
  const LinearPlan p = linear_plan(N, D, V, false);
  if (!workspace || ws_bytes < p.total) return SSD_ERR_WORKSPACE;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  char* ws = static_cast<char*>(workspace);
  PrepArgs a;
  prep_args(&a, p, ws, RowsIn{hidden, batch_stride, row_stride, rows_per_batch}, targets, N, V, D);
  a.loss = loss;
  a.lse_out = lse;
  a.status = status;
  if ((st = launch_prep(a, s)) != SSD_OK) return st;
  return p.cg == 1 ? linear_forward<1>(p, ws, weight, 2ll * weight_stride, N, D, V, loss, lse, status, s)
                   : linear_forward<2>(p, ws, weight, 2ll * weight_stride, N, D, V, loss, lse, status, s);
}

ssd_status ssd_linear_ce_grad(const void* hidden, const void* weight, int dtype, int n_batch, int rows_per_batch, int D,
                              int V, int64_t batch_stride, int64_t row_stride, int64_t weight_stride,
                              const int32_t* targets, const float* lse, const float* row_scale, void* grad_hidden,
                              void* grad_weight, int32_t* status, void* workspace, size_t ws_bytes, void* stream) {
  ssd_status st = check_linear(dtype, n_batch, rows_per_batch, D, V, batch_stride, row_stride, weight_stride);
  if (st != SSD_OK) return st;
  const int N = n_batch * rows_per_batch;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (!grad_weight) return SSD_ERR_INVALID_ARG;
  if (!aligned_to(grad_weight, 16)) return SSD_ERR_ALIGNMENT;
  if (N == 0)  // no row: the weight's gradient is zero
    return cudaMemsetAsync(grad_weight, 0, 2ull * static_cast<size_t>(V) * D, s) == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
  if (!hidden || !weight || !targets || !lse || !grad_hidden) return SSD_ERR_INVALID_ARG;
  if (!aligned_to(hidden, 16) || !aligned_to(weight, 16) || !aligned_to(grad_hidden, 16) ||
      !aligned_to(workspace, 256))
    return SSD_ERR_ALIGNMENT;
  const LinearPlan p = linear_plan(N, D, V, true);
  if (!workspace || ws_bytes < p.total) return SSD_ERR_WORKSPACE;
  // The weight is read to the end, other rows' hidden states while rows that are left out get their zeros.
  const size_t gh_bytes = 2ull * static_cast<size_t>(N) * D, gw_bytes = 2ull * static_cast<size_t>(V) * D;
  if (overlaps(grad_weight, gw_bytes, weight, V, 2ll * D, 2 * weight_stride) ||
      overlaps(grad_hidden, gh_bytes, weight, V, 2ll * D, 2 * weight_stride) ||
      overlaps(grad_hidden, gh_bytes, grad_weight, 1, static_cast<long long>(gw_bytes), 0))
    return SSD_ERR_INVALID_ARG;
  const bool in_place = grad_hidden == hidden && (rows_per_batch == 1 || row_stride == D) &&
                        (n_batch == 1 || batch_stride == static_cast<int64_t>(rows_per_batch) * D);
  const long long extent = 2 * ((n_batch - 1) * batch_stride + (rows_per_batch - 1) * row_stride + D);
  const bool within = !in_place && overlaps(grad_hidden, gh_bytes, hidden, 1, extent, 0);
  for (int b = 0; within && b < (batch_stride > 0 ? n_batch : 1); ++b)
    if (overlaps(grad_hidden, gh_bytes, static_cast<const char*>(hidden) + 2 * b * batch_stride, rows_per_batch, 2ll * D,
                 2 * row_stride))
      return SSD_ERR_INVALID_ARG;
  char* ws = static_cast<char*>(workspace);
  PrepArgs a;
  prep_args(&a, p, ws, RowsIn{hidden, batch_stride, row_stride, rows_per_batch}, targets, N, V, D);
  a.row_scale = row_scale;
  a.lse = lse;
  a.scale = reinterpret_cast<float*>(ws + p.scale);
  a.lse_c = reinterpret_cast<float*>(ws + p.lse);
  a.grad_hidden = static_cast<uint16_t*>(grad_hidden);
  a.status = status;
  if ((st = launch_prep(a, s)) != SSD_OK) return st;
  return p.cg == 1
             ? linear_backward<1>(p, ws, weight, 2ll * weight_stride, N, D, V, grad_hidden, grad_weight, status, s)
             : linear_backward<2>(p, ws, weight, 2ll * weight_stride, N, D, V, grad_hidden, grad_weight, status, s);
}

}  // extern "C"
