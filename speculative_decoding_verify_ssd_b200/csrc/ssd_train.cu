// ssd_train.cu -- host side of the draft-training calls of include/ssd.h:
// ssd_teacher_top, ssd_distill (ssd_rows.cuh).
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <map>
#include <mutex>
#include <utility>

#include "../../include/ssd.h"
#include "ssd_device.cuh"
#include "ssd_rows.cuh"

namespace ssd {

static std::mutex g_fn_mu;
static std::map<std::pair<const void*, int>, int> g_fn_smem;

// Raises a kernel's dynamic shared-memory limit on the current device, once.
static cudaError_t allow_smem(const void* fn, int bytes) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::lock_guard<std::mutex> lock(g_fn_mu);
  int& have = g_fn_smem[std::make_pair(fn, dev)];
  if (have >= bytes) return cudaSuccess;
  e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) have = bytes;
  return e;
}

// ---------------------------------------------------------------------------
// Rows in cluster shared memory.
// ---------------------------------------------------------------------------
constexpr long long kSliceTarget = 66 * 1024;  // bytes of a row that one CTA stages: three CTAs fit an SM
constexpr long long kSliceMin = 8 * 1024;      // do not split a row finer than this for the sake of few rows
constexpr long long kSliceMax = 200 * 1024;
constexpr int kRowFill = 2 * 148;              // CTAs that fill the GPU

struct RowPlan {
  int cluster, slice_vecs, smem;
};

// CTAs per row and the 16-byte vectors of a slice; false when the row does
// not fit the cluster's shared memory.
static bool row_plan(long long rows, int V, int esize, int min_bytes, RowPlan* p) {
  const long long vecs = (static_cast<long long>(V) * esize + 15) / 16 + 1;  // a row may start inside a vector
  const long long bytes = vecs * 16;
  long long c = (bytes + kSliceTarget - 1) / kSliceTarget;
  const long long fill = (kRowFill + rows - 1) / rows, by_len = bytes / kSliceMin;
  const long long extra = fill < by_len ? fill : by_len;
  if (c < extra) c = extra;
  if (c > kMaxRowCluster) c = kMaxRowCluster;
  const long long sv = (vecs + c - 1) / c;
  if (sv * 16 > kSliceMax) return false;
  p->cluster = static_cast<int>(c);
  p->slice_vecs = static_cast<int>(sv);
  p->smem = static_cast<int>(sv * 16 > min_bytes ? sv * 16 : min_bytes);
  return true;
}

template <typename Args>
static ssd_status launch_rows(void (*fn)(Args), const Args& a, long long rows, const RowPlan& p, cudaStream_t stream) {
  if (allow_smem(reinterpret_cast<const void*>(fn), p.smem) != cudaSuccess) return SSD_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(rows * p.cluster));
  cfg.blockDim = dim3(kRowThreads);
  cfg.dynamicSmemBytes = static_cast<size_t>(p.smem);
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = static_cast<unsigned>(p.cluster);
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fn, a) == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
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

}  // namespace ssd

using namespace ssd;

extern "C" {

ssd_status ssd_teacher_top(const void* logits, int dtype, int n_batch, int rows_per_batch, int V, int64_t batch_stride,
                           int64_t row_stride, float T, int M, int32_t* tokens, float* values, float* lse, float* tail,
                           int32_t* status, void* stream) {
  const ssd_status st = check_rows(dtype, n_batch, rows_per_batch, V, batch_stride, row_stride, T, M);
  if (st != SSD_OK) return st;
  const long long rows = static_cast<long long>(n_batch) * rows_per_batch;
  if (rows == 0) return SSD_OK;
  if (!logits || !tokens || !values || !lse || !tail || !status) return SSD_ERR_INVALID_ARG;
  const int esize = dtype == SSD_DTYPE_FP32 ? 4 : 2;
  if (!aligned_to(logits, esize)) return SSD_ERR_ALIGNMENT;
  RowPlan p;
  if (!row_plan(rows, V, esize, kTopMinBytes, &p)) return SSD_ERR_UNSUPPORTED;
  TopArgs a;
  a.in = RowsIn{logits, batch_stride, row_stride, rows_per_batch};
  a.tokens = tokens;
  a.values = values;
  a.lse = lse;
  a.tail = tail;
  a.status = status;
  a.V = V;
  a.M = M;
  a.slice_vecs = p.slice_vecs;
  a.T = T;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  return dtype == SSD_DTYPE_BF16 ? launch_rows(&ssd_top_kernel<uint16_t>, a, rows, p, s)
                                 : launch_rows(&ssd_top_kernel<float>, a, rows, p, s);
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
  if (!row_plan(rows, V, esize, 0, &p)) return SSD_ERR_UNSUPPORTED;
  DistillArgs a;
  a.in = RowsIn{logits, batch_stride, row_stride, rows_per_batch};
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
  a.T = T;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  return dtype == SSD_DTYPE_BF16 ? launch_rows(&ssd_distill_kernel<uint16_t>, a, rows, p, s)
                                 : launch_rows(&ssd_distill_kernel<float>, a, rows, p, s);
}

}  // extern "C"
