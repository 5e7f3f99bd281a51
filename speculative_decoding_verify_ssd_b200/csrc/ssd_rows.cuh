// ssd_rows.cuh -- the vocabulary-row operators of draft training: the top
// logits of a row with the mass left outside them (ssd_teacher_top) and the
// distillation loss of a row against such a teacher with its gradient
// (ssd_distill).  One thread-block cluster holds one whole row in its CTAs'
// shared memory, so a row is read from HBM once however many passes the
// arithmetic takes over it.
#pragma once

#include <cooperative_groups.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/ssd.h"
#include "ssd_device.cuh"

namespace ssd {

constexpr int kRowThreads = 256;
constexpr int kRowWarps = kRowThreads / 32;
constexpr int kMaxRowCluster = 8;   // the portable cluster size
constexpr int kCandPerCta = 512;    // top candidates one CTA may contribute
constexpr int kCandTotal = 1024;    // candidates ranked at once
constexpr unsigned long long kRowWaitNs = 1000000000ull;  // limit of the wait for a slice's bytes

// Rows of a [n_batch, rows_per_batch, V] tensor, strides in elements.
struct RowsIn {
  const void* base;
  long long batch_stride, row_stride;
  int rows_per_batch;
};

__device__ __forceinline__ long long row_offset(long long batch_stride, long long row_stride, int rows_per_batch,
                                                int row) {
  const int b = row / rows_per_batch;
  return b * batch_stride + static_cast<long long>(row - b * rows_per_batch) * row_stride;
}

template <typename T>
struct Elem;
template <>
struct Elem<uint16_t> {
  static constexpr int kVec = 8;
  static __device__ __forceinline__ float to_float(uint16_t v) { return __uint_as_float(static_cast<uint32_t>(v) << 16); }
  static __device__ __forceinline__ uint16_t neg_inf() { return 0xFF80u; }
  // round to nearest even; the callers' values are finite
  static __device__ __forceinline__ uint16_t from_float(float f) {
    uint16_t h;
    asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(h) : "f"(f));
    return h;
  }
  static __device__ __forceinline__ void unpack(const uint4& v, float (&f)[8]) {
    f[0] = bf16_lo(v.x), f[1] = bf16_hi(v.x), f[2] = bf16_lo(v.y), f[3] = bf16_hi(v.y);
    f[4] = bf16_lo(v.z), f[5] = bf16_hi(v.z), f[6] = bf16_lo(v.w), f[7] = bf16_hi(v.w);
  }
  static __device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
  }
  static __device__ __forceinline__ uint4 pack(const float (&f)[8]) {
    return make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
  }
  // the largest element, NaN when any is
  static __device__ __forceinline__ float vec_max(const uint4& v) {
    const uint32_t m = bf16x2_max_nan(bf16x2_max_nan(v.x, v.y), bf16x2_max_nan(v.z, v.w));
    return fmax_nan(bf16_lo(m), bf16_hi(m));
  }
  static constexpr int kKeyBits = 16;  // an order key's low 16 bits are constant
};
template <>
struct Elem<float> {
  static constexpr int kVec = 4;
  static __device__ __forceinline__ float to_float(float v) { return v; }
  static __device__ __forceinline__ float neg_inf() { return -INFINITY; }
  static __device__ __forceinline__ float from_float(float f) { return f; }
  static __device__ __forceinline__ void unpack(const uint4& v, float (&f)[4]) {
    f[0] = __uint_as_float(v.x), f[1] = __uint_as_float(v.y), f[2] = __uint_as_float(v.z), f[3] = __uint_as_float(v.w);
  }
  static __device__ __forceinline__ uint4 pack(const float (&f)[4]) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
  }
  static __device__ __forceinline__ float vec_max(const uint4& v) {
    return fmax_nan(fmax_nan(__uint_as_float(v.x), __uint_as_float(v.y)),
                    fmax_nan(__uint_as_float(v.z), __uint_as_float(v.w)));
  }
  static constexpr int kKeyBits = 32;
};

// This CTA's part of a row: the 16-byte vectors [first, first + count) of the
// vectors that the row touches, counted from the one that holds element 0 at
// place `head`.  Vector first + i is staged at data[i]; the places of the edge
// vectors that lie outside the row hold -inf.
struct Slice {
  int head, first, count;
};

template <typename TIn>
__device__ __forceinline__ Slice slice_of(const TIn* row, int V, int slice_vecs, int rank) {
  constexpr int VE = Elem<TIn>::kVec;
  Slice s;
  s.head = static_cast<int>((reinterpret_cast<uintptr_t>(row) & 15u) / sizeof(TIn));
  const int n = (s.head + V + VE - 1) / VE;
  s.first = min(rank * slice_vecs, n);
  s.count = min(slice_vecs, n - s.first);
  return s;
}

// Starts the copies of the slice: whole vectors in bulk (one barrier phase),
// the row's ragged edge vectors element by element.
template <typename TIn>
__device__ __forceinline__ void slice_load(const TIn* row, int V, const Slice& s, uint4* data, uint64_t* bar) {
  constexpr int VE = Elem<TIn>::kVec;
  const int lo_edge = s.first == 0 && s.head != 0;                         // vector 0 starts before the row
  const int last = (s.head + V + VE - 1) / VE - 1;
  const int hi_edge = s.first + s.count - 1 == last && (s.head + V) % VE != 0;  // the last one ends behind it
  const int a = lo_edge ? 1 : 0;
  int b = s.count - (hi_edge ? 1 : 0);
  if (s.count == 0) b = 0;
  const int whole = max(b - a, 0);
  if (threadIdx.x == 0) {
    mbar_arrive_expect_tx(bar, static_cast<uint32_t>(whole) * 16u);
    const char* src = reinterpret_cast<const char*>(row) - s.head * static_cast<int>(sizeof(TIn)) +
                      (static_cast<long long>(s.first) + a) * 16;
    const uint64_t policy = l2_policy_evict_first();
    constexpr int kPiece = 1024;  // vectors of one copy
    for (int i = 0; i < whole; i += kPiece)
      bulk_copy_g2s_hint(data + a + i, src + static_cast<long long>(i) * 16,
                         static_cast<uint32_t>(min(kPiece, whole - i)) * 16u, bar, policy);
  }
  // at most two edge vectors, VE elements each
  if (threadIdx.x >= 32 && threadIdx.x < 32 + 2 * VE) {
    const int e = (threadIdx.x - 32) % VE;
    const bool second = threadIdx.x >= 32 + VE;
    const bool mine = s.count > 0 && (second ? hi_edge && !(lo_edge && s.count == 1) : (lo_edge != 0));
    if (mine) {
      const int i = second ? s.count - 1 : 0;
      const int v = (s.first + i) * VE - s.head + e;
      reinterpret_cast<TIn*>(data + i)[e] = v >= 0 && v < V ? row[v] : Elem<TIn>::neg_inf();
    }
  }
}

// Waits for the slice's bytes.  A wait that gives up waits once more (the
// copies still target this CTA's shared memory) before the row is flagged.
__device__ __forceinline__ int slice_wait(uint64_t* bar) {
  if (mbar_wait_bounded(bar, 0, kRowWaitNs)) return 0;
  (void)mbar_wait_bounded(bar, 0, kRowWaitNs);
  return SSD_ROW_DEVICE_TIMEOUT;
}

// ---------------------------------------------------------------------------
// Block reductions.  `red` holds one value per warp; every thread gets the
// result; a barrier stands on both sides of the exchange.
// ---------------------------------------------------------------------------
template <typename T, typename Op>
__device__ __forceinline__ T block_reduce(T v, T* red, Op op) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = op(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  T r = red[0];
#pragma unroll
  for (int w = 1; w < kRowWarps; ++w) r = op(r, red[w]);
  return r;
}
struct OpAdd {
  template <typename T>
  __device__ __forceinline__ T operator()(T a, T b) const {
    return a + b;
  }
};
struct OpMax {
  __device__ __forceinline__ float operator()(float a, float b) const { return fmaxf(a, b); }
  __device__ __forceinline__ double operator()(double a, double b) const { return fmax(a, b); }
};
struct OpMaxNan {
  __device__ __forceinline__ float operator()(float a, float b) const { return fmax_nan(a, b); }
};
struct OpOr {
  __device__ __forceinline__ int operator()(int a, int b) const { return a | b; }
};

// max + log(sum of exponentials) of two (reference, sum) pairs, natural units:
// each stands for sum * exp(ref).  A sum of 0 stands for nothing.
__device__ __forceinline__ double lse_of(double ref, double sum) { return sum > 0.0 ? ref + log(sum) : -INFINITY; }
__device__ __forceinline__ double lse_join(double a, double b) {
  const double m = fmax(a, b);
  if (!(m > -INFINITY)) return m;
  return m + log1p(exp(fmin(a, b) - m));
}

// What one CTA of a distillation row tells the others.
struct DistillPart {
  double tail_sum, atom_sum, numer;  // sums of exponentials around the maxima below; sum_m p_m (log p_m - z_m / T)
  float tail_max, atom_max;
  int flags;
};

// What the gradient needs of the joined row.
struct DistillJoin {
  double lse;
  float k, ref;  // gradient outside the atoms: k * exp((z - ref) / T)
  int bad;
};

struct DistillArgs {
  RowsIn in;
  const int32_t* tokens;   // [rows, M]
  const float* values;     // [rows, M]
  const float* tail;       // [rows] or NULL
  const float* row_scale;  // [rows] or NULL
  float* loss;             // [rows]
  int32_t* status;         // [rows]
  void* grad;              // or NULL
  long long g_batch_stride, g_row_stride;
  int V, M, slice_vecs;
  float T;
};

// ---------------------------------------------------------------------------
// Distillation.  With teacher weights p over M atoms and one tail, student
// q = softmax(z / T), q_tail the student's mass outside the atoms:
//   loss = sum_m p_m (log p_m - log q_m) + p_tail (log p_tail - log q_tail)
//   dloss/dz_v = (q_v - p_m) / T at v = id_m,
//                (q_tail - p_tail) / T * exp(z_v / T) / sum_tail elsewhere.
// The atoms' logits are taken out of the staged row (replaced by -inf) before
// the sums, so the tail's sum is formed without them and never by subtraction.
// ---------------------------------------------------------------------------
template <typename TIn>
__global__ void __launch_bounds__(kRowThreads) ssd_distill_kernel(const DistillArgs a) {
  constexpr int VE = Elem<TIn>::kVec;
  extern __shared__ __align__(128) uint4 data[];
  __shared__ uint64_t bar;
  __shared__ int32_t ids[SSD_MAX_TOP];
  __shared__ double dred[kRowWarps];
  __shared__ float fred[kRowWarps];
  __shared__ int ired[kRowWarps];
  __shared__ DistillPart part;
  __shared__ DistillJoin join;

  cg::cluster_group cluster = cg::this_cluster();
  const int rank = static_cast<int>(cluster.block_rank()), C = static_cast<int>(cluster.num_blocks());
  const int row = static_cast<int>(blockIdx.x) / C;
  const int tid = threadIdx.x;
  const TIn* src = static_cast<const TIn*>(a.in.base) +
                   row_offset(a.in.batch_stride, a.in.row_stride, a.in.rows_per_batch, row);
  TIn* dst = a.grad ? static_cast<TIn*>(a.grad) +
                          row_offset(a.g_batch_stride, a.g_row_stride, a.in.rows_per_batch, row)
                    : nullptr;
  const float scale = a.row_scale ? a.row_scale[row] : 1.f;
  const Slice s = slice_of(src, a.V, a.slice_vecs, rank);
  // the first element of the slice, and one past its last
  const int v0 = max(s.first * VE - s.head, 0), v1 = s.count > 0 ? min((s.first + s.count) * VE - s.head, a.V) : v0;

  if (scale == 0.f) {  // the whole cluster takes this path: the row has no part in the loss and is not read
    if (dst)
      for (int v = v0 + tid; v < v1; v += kRowThreads) dst[v] = Elem<TIn>::from_float(0.f);
    if (rank == 0 && tid == 0) {
      a.loss[row] = 0.f;
      a.status[row] = 0;
    }
    return;
  }

  if (tid == 0) {
    mbar_init(&bar, 1);
    mbar_init_fence();
  }
  __syncthreads();
  slice_load(src, a.V, s, data, &bar);

  // The teacher's weights, while the copies are in flight: one atom per thread.
  const double invT = 1.0 / static_cast<double>(a.T);
  int flags = 0;
  int id = -1;
  double log_p = -INFINITY;
  if (tid < a.M) {
    id = a.tokens[static_cast<long long>(row) * a.M + tid];
    const float t = a.values[static_cast<long long>(row) * a.M + tid];
    ids[tid] = id;
    if (id >= a.V || id < -1) flags |= SSD_ROW_BAD_TOKEN;
    if (id >= 0) {
      if (!(t < INFINITY)) flags |= SSD_ROW_NONFINITE;  // NaN or +inf
      log_p = static_cast<double>(t) * invT;
    }
  }
  double log_p_tail = a.tail ? static_cast<double>(a.tail[row]) : -INFINITY;
  if (!(log_p_tail < INFINITY)) flags |= SSD_ROW_NONFINITE;
  {
    const double top = fmax(block_reduce(log_p, dred, OpMax()), log_p_tail);  // the barriers also publish ids
    if (!(top > -INFINITY)) flags |= SSD_ROW_NONFINITE;                      // a teacher without any mass
    const double sum = block_reduce(log_p > -INFINITY ? exp(log_p - top) : 0.0, dred, OpAdd()) +
                       (log_p_tail > -INFINITY ? exp(log_p_tail - top) : 0.0);
    const double norm = top + log(sum);
    log_p -= norm;
    log_p_tail -= norm;
  }
  const double p = log_p > -INFINITY ? exp(log_p) : 0.0;
  const double p_tail = log_p_tail > -INFINITY ? exp(log_p_tail) : 0.0;
  if (id >= 0)
    for (int j = 0; j < tid; ++j)
      if (ids[j] == id) flags |= SSD_ROW_BAD_TOKEN;  // the same token twice

  flags |= slice_wait(&bar);
  __syncthreads();  // the edge elements are staged

  // Take this slice's atoms out of the staged row.
  const bool mine = id >= v0 && id < v1;
  float z_atom = -INFINITY;
  flags = block_reduce(flags, ired, OpOr());
  if (mine && flags == 0) {
    TIn* at = reinterpret_cast<TIn*>(data) + (id + s.head - s.first * VE);
    z_atom = Elem<TIn>::to_float(*at);
    *at = Elem<TIn>::neg_inf();
  }
  __syncthreads();

  const float c = static_cast<float>(1.4426950408889634 * invT);
  float m = -INFINITY;
  for (int i = tid; i < s.count; i += kRowThreads) m = fmax_nan(m, Elem<TIn>::vec_max(data[i]));
  m = block_reduce(m, fred, OpMaxNan());
  float za_max = block_reduce(mine ? z_atom : -INFINITY, fred, OpMaxNan());
  if (!(m < INFINITY) || !(za_max < INFINITY)) flags |= SSD_ROW_NONFINITE;
  const float ref = m > -INFINITY && m < INFINITY ? m : 0.f;
  float sum = 0.f;
  for (int i = tid; i < s.count; i += kRowThreads) {
    float f[VE];
    Elem<TIn>::unpack(data[i], f);
#pragma unroll
    for (int e = 0; e < VE; ++e) sum += ex2((f[e] - ref) * c);
  }
  const double tail_sum = block_reduce(static_cast<double>(sum), dred, OpAdd());
  const float za_ref = za_max > -INFINITY && za_max < INFINITY ? za_max : 0.f;
  const double atom_sum = block_reduce(
      z_atom > -INFINITY ? exp((static_cast<double>(z_atom) - static_cast<double>(za_ref)) * invT) : 0.0, dred, OpAdd());
  const double numer =
      block_reduce(mine && p > 0.0 ? p * (log_p - static_cast<double>(z_atom) * invT) : 0.0, dred, OpAdd());
  if (tid == 0) part = DistillPart{tail_sum, atom_sum, numer, ref, za_ref, flags};
  cluster.sync();

  // One warp of every CTA joins the parts, a lane each, in the same order, so
  // all hold the same bits.
  const double w = static_cast<double>(scale) * invT;
  if (tid < 32) {
    DistillPart q = {0.0, 0.0, 0.0, 0.f, 0.f, 0};
    if (tid < C) q = *cluster.map_shared_rank(&part, tid);
    double tail_max = q.tail_sum > 0.0 ? static_cast<double>(q.tail_max) : -INFINITY;
    double atom_max = q.atom_sum > 0.0 ? static_cast<double>(q.atom_max) : -INFINITY;
    int fl = q.flags;
#pragma unroll
    for (int o = kMaxRowCluster / 2; o > 0; o >>= 1) {
      tail_max = fmax(tail_max, __shfl_xor_sync(0xFFFFFFFFu, tail_max, o));
      atom_max = fmax(atom_max, __shfl_xor_sync(0xFFFFFFFFu, atom_max, o));
      fl |= __shfl_xor_sync(0xFFFFFFFFu, fl, o);
    }
    double tail = q.tail_sum > 0.0 ? q.tail_sum * exp((static_cast<double>(q.tail_max) - tail_max) * invT) : 0.0;
    double atom = q.atom_sum > 0.0 ? q.atom_sum * exp((static_cast<double>(q.atom_max) - atom_max) * invT) : 0.0;
    double num = q.numer;
#pragma unroll
    for (int o = kMaxRowCluster / 2; o > 0; o >>= 1) {
      tail += __shfl_xor_sync(0xFFFFFFFFu, tail, o);
      atom += __shfl_xor_sync(0xFFFFFFFFu, atom, o);
      num += __shfl_xor_sync(0xFFFFFFFFu, num, o);
    }
    if (tid == 0) {
      const double lse_tail = lse_of(tail_max * invT, tail);
      const double lse = lse_join(lse_tail, lse_of(atom_max * invT, atom));
      if (!(lse > -INFINITY)) fl |= SSD_ROW_NONFINITE;  // every logit is -inf
      const bool bad = (fl & SSD_ROW_INVALID) != 0;
      if (rank == 0) {
        double loss = num + (1.0 - p_tail) * lse;
        if (p_tail > 0.0) loss += p_tail * (log_p_tail - lse_tail + lse);
        if (!bad && !(loss < INFINITY)) fl |= SSD_ROW_ZERO_Q;
        a.loss[row] = bad ? __int_as_float(0x7FC00000) : static_cast<float>(loss);
        a.status[row] = fl;
      }
      join.lse = lse;
      join.k = bad || !(tail > 0.0) ? 0.f : static_cast<float>(w * (exp(lse_tail - lse) - p_tail) / tail);
      join.ref = tail > 0.0 ? static_cast<float>(tail_max) : 0.f;
      join.bad = bad;
    }
  }
  if (dst) {
    __syncthreads();
    const bool bad = join.bad;
    const float k = join.k, r0 = join.ref;
    // whole vectors only where the row's places in both tensors agree modulo 16 bytes
    const bool same = ((reinterpret_cast<uintptr_t>(dst) ^ reinterpret_cast<uintptr_t>(src)) & 15u) == 0;
    for (int i = tid; i < s.count; i += kRowThreads) {
      float f[VE];
      Elem<TIn>::unpack(data[i], f);
      const int v = (s.first + i) * VE - s.head;
#pragma unroll
      for (int e = 0; e < VE; ++e) f[e] = bad ? 0.f : k * ex2((f[e] - r0) * c);
      if (same && v >= 0 && v + VE <= a.V) {
        *reinterpret_cast<uint4*>(dst + v) = Elem<TIn>::pack(f);
      } else {
#pragma unroll
        for (int e = 0; e < VE; ++e)
          if (v + e >= 0 && v + e < a.V) dst[v + e] = Elem<TIn>::from_float(f[e]);
      }
    }
    __syncthreads();  // the atoms' places are written after the vectors that hold them
    if (mine && !bad) {
      const double q = z_atom > -INFINITY ? exp(static_cast<double>(z_atom) * invT - join.lse) : 0.0;
      dst[id] = Elem<TIn>::from_float(static_cast<float>(w * (q - p)));
    }
  }
  cluster.sync();  // no CTA leaves while another may read its part
}

// ---------------------------------------------------------------------------
// The top M logits of a row.
// ---------------------------------------------------------------------------
struct TopArgs {
  RowsIn in;
  int32_t* tokens;  // [rows, M]
  float* values;    // [rows, M]
  float* lse;       // [rows]
  float* tail;      // [rows]
  int32_t* status;  // [rows]
  int V, M, slice_vecs;
  float T;
};

struct TopPart {
  double sum;
  float max, ref;
  int count, flags;
};

// Rank 0 gathers the candidates where its slice was staged.
constexpr int kTopMinBytes = kCandTotal * (sizeof(unsigned long long) + sizeof(float));

// Keys of the cluster's thread maxima, kMaxima / C of them (a power of two)
// from each CTA: their M-th largest is a lower bound of the row's M-th
// largest logit, and few logits reach it.
constexpr int kMaxima = 1024;

// The key of a logit from its kKeyBits high bits: the bits below them are the
// complement of the mantissa's zeros in a negative logit's key.
template <typename TIn>
__device__ __forceinline__ uint32_t full_key(uint32_t k) {
  if (Elem<TIn>::kKeyBits == 16 && !(k & 0x80000000u)) k |= 0xFFFFu;
  return k;
}

template <typename TIn>
__global__ void __launch_bounds__(kRowThreads) ssd_top_kernel(const TopArgs a) {
  constexpr int VE = Elem<TIn>::kVec;
  extern __shared__ __align__(128) uint4 data[];
  __shared__ uint64_t bar;
  __shared__ uint32_t maxima[kRowThreads];
  __shared__ unsigned long long cand[kCandPerCta];
  __shared__ double dred[kRowWarps];
  __shared__ float fred[kRowWarps];
  __shared__ int ired[kRowWarps];
  __shared__ int counts[4];  // per-CTA counts exchanged by the exact select
  __shared__ int n_cand;
  __shared__ uint32_t tau_s;
  __shared__ TopPart part, part2;

  cg::cluster_group cluster = cg::this_cluster();
  const int rank = static_cast<int>(cluster.block_rank()), C = static_cast<int>(cluster.num_blocks());
  const int row = static_cast<int>(blockIdx.x) / C;
  const int tid = threadIdx.x, lane = tid & 31;
  const TIn* src = static_cast<const TIn*>(a.in.base) +
                   row_offset(a.in.batch_stride, a.in.row_stride, a.in.rows_per_batch, row);
  const Slice s = slice_of(src, a.V, a.slice_vecs, rank);
  const int base = s.first * VE - s.head;  // token id of the first staged place
  const double invT = 1.0 / static_cast<double>(a.T);
  const float c = static_cast<float>(1.4426950408889634 * invT);

  if (tid == 0) {
    mbar_init(&bar, 1);
    mbar_init_fence();
    n_cand = 0;
  }
  __syncthreads();
  slice_load(src, a.V, s, data, &bar);
  int flags = slice_wait(&bar);
  __syncthreads();

  float m = -INFINITY;
  for (int i = tid; i < s.count; i += kRowThreads) m = fmax_nan(m, Elem<TIn>::vec_max(data[i]));
  maxima[tid] = ord_key(m);
  m = block_reduce(m, fred, OpMaxNan());
  flags = block_reduce(flags, ired, OpOr());
  if (!(m < INFINITY)) flags |= SSD_ROW_NONFINITE;
  if (tid == 0) part = TopPart{0.0, m, 0.f, 0, flags};
  cluster.sync();

  int fl = 0;
  float row_max = -INFINITY;
  for (int r = 0; r < C; ++r) {
    const TopPart* q = cluster.map_shared_rank(&part, r);
    fl |= q->flags;
    row_max = fmax_nan(row_max, q->max);
  }
  if (!(row_max > -INFINITY)) fl |= SSD_ROW_NONFINITE;
  if (fl) {
    if (rank == 0) {
      for (int i = tid; i < a.M; i += kRowThreads) {
        a.tokens[static_cast<long long>(row) * a.M + i] = -1;
        a.values[static_cast<long long>(row) * a.M + i] = __int_as_float(0x7FC00000);
      }
      if (tid == 0) {
        a.lse[row] = a.tail[row] = __int_as_float(0x7FC00000);
        a.status[row] = fl;
      }
    }
    cluster.sync();
    return;
  }

  // The threshold tau.
  if (tid < 32) {
    uint32_t keys[kMaxima / 32];
    const int per = C <= 4 ? kRowThreads : kRowThreads / 2;  // maxima taken from each CTA
#pragma unroll
    for (int i = 0; i < kMaxima / 32; ++i) {
      const int k = i * 32 + lane, r = k / per, t = k % per;
      uint32_t v = 0u;
      if (r < C) {
        const uint32_t* q = cluster.map_shared_rank(&maxima[0], r);
        v = per == kRowThreads ? q[t] : max(q[t], q[t + per]);
      }
      keys[i] = v;
    }
    const uint32_t t = warp_kth_largest<kMaxima / 32>(keys, a.M, Elem<TIn>::kKeyBits);
    if (lane == 0) tau_s = t;
  }
  __syncthreads();
  const uint32_t tau_key = tau_s;
  // With fewer maxima than M, or M of them -inf, every logit is a candidate.
  const float tau = tau_key <= ord_key(-INFINITY) ? -INFINITY : key_to_float(full_key<TIn>(tau_key));
  const float ref = tau > -INFINITY ? tau : 0.f;
  float sum = 0.f;
  for (int i = tid; i < s.count; i += kRowThreads) {
    const uint4 v = data[i];
    float f[VE];
    Elem<TIn>::unpack(v, f);
    if (Elem<TIn>::vec_max(v) >= tau) {
#pragma unroll
      for (int e = 0; e < VE; ++e) {
        const int id = base + i * VE + e;
        if (f[e] >= tau) {
          if (id >= 0 && id < a.V) {
            const int at = atomicAdd(&n_cand, 1);
            if (at < kCandPerCta) cand[at] = rank_key(f[e], id);
          }
        } else {
          sum += ex2((f[e] - ref) * c);
        }
      }
    } else {
#pragma unroll
      for (int e = 0; e < VE; ++e) sum += ex2((f[e] - ref) * c);
    }
  }
  double below = block_reduce(static_cast<double>(sum), dred, OpAdd());
  if (tid == 0) {
    part2.sum = below;
    part2.count = n_cand;
  }
  cluster.sync();
  int total = 0;
  bool over = false;
  below = 0.0;
  for (int r = 0; r < C; ++r) {
    const TopPart* q = cluster.map_shared_rank(&part2, r);
    total += q->count;
    over |= q->count > kCandPerCta;
    below += q->sum;
  }
  over |= total > kCandTotal;
  double ref_d = static_cast<double>(ref);
  float limit = tau;  // the tail's logits are below it (or equal to it and counted apart)

  if (over) {
    // Exact select, for rows with many equal logits at the threshold: the
    // M-th largest key by two bits a pass over the staged row, then the equal
    // ones in token order.
    uint32_t prefix = 0u;
    int above = 0;  // elements with a larger key than the prefix's final value
    for (int bit = 30; bit >= 32 - Elem<TIn>::kKeyBits; bit -= 2) {
      const uint32_t c1 = prefix | (1u << bit), c2 = prefix | (2u << bit), c3 = prefix | (3u << bit);
      int n1 = 0, n2 = 0, n3 = 0;
      for (int i = tid; i < s.count; i += kRowThreads) {
        float f[VE];
        Elem<TIn>::unpack(data[i], f);
#pragma unroll
        for (int e = 0; e < VE; ++e) {
          const int id = base + i * VE + e;
          const uint32_t k = id >= 0 && id < a.V ? ord_key(f[e]) : 0u;
          n1 += k >= c1;
          n2 += k >= c2;
          n3 += k >= c3;
        }
      }
      n1 = block_reduce(n1, ired, OpAdd());
      n2 = block_reduce(n2, ired, OpAdd());
      n3 = block_reduce(n3, ired, OpAdd());
      if (tid == 0) counts[0] = n1, counts[1] = n2, counts[2] = n3;
      cluster.sync();
      n1 = n2 = n3 = 0;
      for (int r = 0; r < C; ++r) {
        const int* q = cluster.map_shared_rank(&counts[0], r);
        n1 += q[0], n2 += q[1], n3 += q[2];
      }
      cluster.sync();  // read before the next pass overwrites them
      prefix = n3 >= a.M ? c3 : (n2 >= a.M ? c2 : (n1 >= a.M ? c1 : prefix));
    }
    int gt = 0, eq = 0;
    const float kth = key_to_float(full_key<TIn>(prefix));
    const float kref = kth > -INFINITY ? kth : 0.f;
    if (tid == 0) n_cand = 0;
    __syncthreads();
    sum = 0.f;
    for (int i = tid; i < s.count; i += kRowThreads) {
      float f[VE];
      Elem<TIn>::unpack(data[i], f);
#pragma unroll
      for (int e = 0; e < VE; ++e) {
        const int id = base + i * VE + e;
        if (id < 0 || id >= a.V) continue;
        if (f[e] > kth) {
          ++gt;
          const int at = atomicAdd(&n_cand, 1);
          if (at < kCandPerCta) cand[at] = rank_key(f[e], id);  // fewer than M <= kCandPerCta in all
        } else if (f[e] == kth) {
          ++eq;
        } else {
          sum += ex2((f[e] - kref) * c);
        }
      }
    }
    below = block_reduce(static_cast<double>(sum), dred, OpAdd());
    gt = block_reduce(gt, ired, OpAdd());
    eq = block_reduce(eq, ired, OpAdd());
    if (tid == 0) {
      counts[0] = gt, counts[1] = eq;
      part2.sum = below;
    }
    cluster.sync();
    int eq_before = 0, eq_all = 0;
    below = 0.0;
    for (int r = 0; r < C; ++r) {
      const int* q = cluster.map_shared_rank(&counts[0], r);
      above += q[0];
      if (r < rank) eq_before += q[1];
      eq_all += q[1];
      below += cluster.map_shared_rank(&part2, r)->sum;
    }
    const int need = a.M - above;  // of the equal ones, in token order
    int taken = eq_before;
    __syncthreads();
    for (int i0 = 0; i0 < s.count && taken < need; i0 += kRowThreads) {  // uniform over the CTA
      const int i = i0 + tid;
      float f[VE];
      int n = 0;
      if (i < s.count) {
        Elem<TIn>::unpack(data[i], f);
#pragma unroll
        for (int e = 0; e < VE; ++e) {
          const int id = base + i * VE + e;
          n += id >= 0 && id < a.V && f[e] == kth;
        }
      }
      int inc = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xFFFFFFFFu, inc, o);
        if (lane >= o) inc += y;
      }
      __syncthreads();
      if (lane == 31) ired[tid >> 5] = inc;
      __syncthreads();
      int before = taken + inc - n, chunk = 0;
#pragma unroll
      for (int w = 0; w < kRowWarps; ++w) {
        if (w < (tid >> 5)) before += ired[w];
        chunk += ired[w];
      }
      if (n > 0) {
#pragma unroll
        for (int e = 0; e < VE; ++e) {
          const int id = base + i * VE + e;
          if (id >= 0 && id < a.V && f[e] == kth) {
            if (before < need) {
              const int at = atomicAdd(&n_cand, 1);
              if (at < kCandPerCta) cand[at] = rank_key(kth, id);
            }
            ++before;
          }
        }
      }
      taken += chunk;
    }
    __syncthreads();
    if (tid == 0) part2.count = n_cand;
    ref_d = static_cast<double>(kref);
    limit = kth;
    if (kth > -INFINITY) below += static_cast<double>(eq_all - need);
    cluster.sync();
    total = a.M;
  }

  // A tail far below the threshold: sum it again around its own maximum.
  if (total == a.M && a.V > a.M && below < 1e-18) {
    float tm = -INFINITY;
    for (int i = tid; i < s.count; i += kRowThreads) {
      float f[VE];
      Elem<TIn>::unpack(data[i], f);
#pragma unroll
      for (int e = 0; e < VE; ++e)
        if (f[e] < limit) tm = fmaxf(tm, f[e]);
    }
    tm = block_reduce(tm, fred, OpMax());
    if (tid == 0) part.max = tm;
    cluster.sync();
    tm = -INFINITY;
    for (int r = 0; r < C; ++r) tm = fmaxf(tm, cluster.map_shared_rank(&part, r)->max);
    sum = 0.f;
    if (tm > -INFINITY)
      for (int i = tid; i < s.count; i += kRowThreads) {
        float f[VE];
        Elem<TIn>::unpack(data[i], f);
#pragma unroll
        for (int e = 0; e < VE; ++e)
          if (f[e] < limit) sum += ex2((f[e] - tm) * c);
      }
    below = block_reduce(static_cast<double>(sum), dred, OpAdd());
    if (tid == 0) part2.sum = below;
    cluster.sync();
    below = 0.0;
    for (int r = 0; r < C; ++r) below += cluster.map_shared_rank(&part2, r)->sum;
    if (tm > -INFINITY) ref_d = static_cast<double>(tm);
  }

  if (rank == 0) {
    // Gather and rank the candidates; those past the M-th belong to the tail.
    // The sums run over the ranked order, whatever order the candidates came in.
    unsigned long long* pool = reinterpret_cast<unsigned long long*>(data);
    float* ranked = reinterpret_cast<float*>(pool + kCandTotal);
    __syncthreads();  // the staged logits are no longer read
    int off = 0;
    for (int r = 0; r < C; ++r) {
      const int n = min(cluster.map_shared_rank(&part2, r)->count, kCandPerCta);
      const unsigned long long* q = cluster.map_shared_rank(&cand[0], r);
      for (int i = tid; i < n && off + i < kCandTotal; i += kRowThreads) pool[off + i] = q[i];
      off = min(off + n, kCandTotal);
    }
    __syncthreads();
    for (int i = tid; i < off; i += kRowThreads) {
      const unsigned long long k = pool[i];
      int pos = 0;
      for (int j = 0; j < off; ++j) pos += pool[j] > k;
      const float z = key_to_float(static_cast<uint32_t>(k >> 32));
      ranked[pos] = z;
      if (pos < a.M) {
        a.tokens[static_cast<long long>(row) * a.M + pos] =
            static_cast<int32_t>(0xFFFFFFFFu - static_cast<uint32_t>(k & 0xFFFFFFFFull));
        a.values[static_cast<long long>(row) * a.M + pos] = z;
      }
    }
    __syncthreads();
    double top_sum = 0.0, rest = 0.0;
    for (int i = tid; i < off; i += kRowThreads) {
      const double z = static_cast<double>(ranked[i]);
      if (i < a.M)
        top_sum += exp((z - static_cast<double>(row_max)) * invT);
      else if (z > -INFINITY)
        rest += exp((z - ref_d) * invT);
    }
    top_sum = block_reduce(top_sum, dred, OpAdd());
    rest = block_reduce(rest, dred, OpAdd());
    if (tid == 0) {
      const double t = lse_of(ref_d * invT, below + rest);
      a.tail[row] = static_cast<float>(t);
      a.lse[row] = static_cast<float>(lse_join(t, lse_of(static_cast<double>(row_max) * invT, top_sum)));
      a.status[row] = 0;
    }
  }
  cluster.sync();  // rank 0 has read the others' candidates
}

}  // namespace ssd
