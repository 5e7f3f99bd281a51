// ssd_rows.cuh -- the vocabulary-row operators of draft training: the top
// logits of a row with the mass left outside them (ssd_teacher_top) and the
// distillation loss of a row against such a teacher with its gradient
// (ssd_distill).  A CTA stages a slice of a row in shared memory, so a row is
// read from HBM once however many passes the arithmetic takes over it.  The
// distillation, whose gradient needs the whole row's sums, holds the row in one
// thread-block cluster; the top logits of the slices are joined by a second,
// small kernel.
#pragma once

#include <cooperative_groups.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/ssd.h"
#include "ssd_device.cuh"

namespace ssd {

constexpr int kRowThreads = 256;
constexpr int kRowWarps = kRowThreads / 32;
constexpr int kMaxRowCluster = 8;   // the portable cluster size
constexpr int kPool = 448;          // top candidates ranked at once (even)
constexpr unsigned long long kRowWaitNs = 1000000000ull;  // limit of the wait for a slice's bytes

// The training kernels are launched as programmatic dependents: a kernel's
// blocks may be scheduled while the kernel before it in the stream still runs,
// and wait here until that one has completed, before they touch global memory.
// Behind the wait the next kernel may be scheduled in the same way.
__device__ __forceinline__ void stream_wait() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// Rows of a [n_batch, rows_per_batch, V] tensor, strides in elements.
struct RowsIn {
  const void* base;
  long long batch_stride, row_stride;
  int rows_per_batch;
};

__device__ __forceinline__ long long row_offset(long long batch_stride, long long row_stride, int rows_per_batch,
                                                int row) {
  if (rows_per_batch == 0) return row * row_stride;  // one stride reaches every row
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
  // round to nearest even
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
  static __device__ __forceinline__ void unpack2(const uint4& v, f32x2 (&f)[4]) {
    f[0] = f2_pack(bf16_lo(v.x), bf16_hi(v.x)), f[1] = f2_pack(bf16_lo(v.y), bf16_hi(v.y));
    f[2] = f2_pack(bf16_lo(v.z), bf16_hi(v.z)), f[3] = f2_pack(bf16_lo(v.w), bf16_hi(v.w));
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
  static __device__ __forceinline__ void unpack2(const uint4& v, f32x2 (&f)[2]) {
    f[0] = f2_pack(__uint_as_float(v.x), __uint_as_float(v.y));
    f[1] = f2_pack(__uint_as_float(v.z), __uint_as_float(v.w));
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
// the row's ragged edge vectors element by element.  One warp; the other
// threads see the barrier and the edges after the next barrier of the CTA.
template <typename TIn>
__device__ __forceinline__ void slice_load(const TIn* row, int V, const Slice& s, uint4* data, uint64_t* bar) {
  constexpr int VE = Elem<TIn>::kVec;
  const int lane = threadIdx.x & 31;
  const bool lo_edge = s.count > 0 && s.first == 0 && s.head != 0;  // vector 0 starts before the row
  const int last = (s.head + V + VE - 1) / VE - 1;
  const bool hi_edge =  // the last vector ends behind the row
      s.count > 0 && s.first + s.count - 1 == last && (s.head + V) % VE != 0 && !(lo_edge && s.count == 1);
  const int a = lo_edge ? 1 : 0;
  const int whole = max(s.count - a - (hi_edge ? 1 : 0), 0);
  if (lane == 0) {
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
  const int e = lane % VE;
  if (lane < 2 * VE && (lane < VE ? lo_edge : hi_edge)) {
    const int i = lane < VE ? 0 : s.count - 1;
    const int v = (s.first + i) * VE - s.head + e;
    reinterpret_cast<TIn*>(data + i)[e] = v >= 0 && v < V ? row[v] : Elem<TIn>::neg_inf();
  }
}

// The address of a shared-memory place in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t cluster_addr(const void* p, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(p)), "r"(rank));
  return a;
}

// mbar_try_wait whose acquire reaches the other CTAs of the cluster.
__device__ __forceinline__ bool mbar_try_wait_cluster(uint64_t* bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(smem_addr(bar)), "r"(parity), "r"(kSuspendHintNs)
      : "memory");
  return done != 0;
}

// Stores into another CTA's shared memory whose bytes are counted on that CTA's
// barrier: the receiver waits for them alone, and the sender for nothing.
__device__ __forceinline__ void st_async(uint32_t to, uint32_t bar, float a, float b, float c, float d) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(to),
               "f"(a), "f"(b), "f"(c), "f"(d), "r"(bar)
               : "memory");
}
__device__ __forceinline__ void st_async(uint32_t to, uint32_t bar, double a, double b) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.f64 [%0], {%1, %2}, [%3];" ::"r"(to), "d"(a),
               "d"(b), "r"(bar)
               : "memory");
}
__device__ __forceinline__ void st_async(uint32_t to, uint32_t bar, int a) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.b32 [%0], %1, [%2];" ::"r"(to), "r"(a), "r"(bar)
               : "memory");
}

// Waits for the slice's bytes; a barrier of the CTA (one warp polls, the others
// stand at the barrier).  A wait that gives up waits once more (the copies still
// target this CTA's shared memory) before the row is flagged.
__device__ __forceinline__ int slice_wait(uint64_t* bar, uint32_t parity) {
  int late = 0;
  if (threadIdx.x >= kRowThreads - 32) {
    late = mbar_wait_bounded(bar, parity, kRowWaitNs) ? 0 : SSD_ROW_DEVICE_TIMEOUT;
    if (late) (void)mbar_wait_bounded(bar, parity, kRowWaitNs);
  }
  return __syncthreads_or(late) ? SSD_ROW_DEVICE_TIMEOUT : 0;
}

// Waits for the cluster's parts.  Its limit is twice slice_wait's, the longest
// that another CTA of the cluster can be behind: a CTA that gives up here has
// no store still coming.
__device__ __forceinline__ int parts_wait(uint64_t* bar) {
  for (int i = 0; i < 4; ++i) {
    const unsigned long long t0 = global_ns();
    do {
      if (mbar_try_wait_cluster(bar, 0)) return i == 0 ? 0 : SSD_ROW_DEVICE_TIMEOUT;
    } while (global_ns() - t0 < kRowWaitNs);
  }
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

// The largest of a warp's values, NaN when any is (made the canonical one,
// whose key is the largest).
__device__ __forceinline__ float warp_max_nan(float v) {
  return key_to_float(__reduce_max_sync(0xFFFFFFFFu, ord_key(fmax_nan(v, v))));
}
__device__ __forceinline__ double warp_sum_d(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}
// The sum over lanes 0 to 7, in every lane; the other lanes' values do not count.
template <typename T>
__device__ __forceinline__ T warp_sum8(T v) {
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return __shfl_sync(0xFFFFFFFFu, v, 0);
}
__device__ __forceinline__ bool is_number(float v) { return v > -INFINITY && v < INFINITY; }

// The exponentials 2^((f - ref) * c) of a vector's elements, added to `acc`
// (element pairs apart).  The difference is formed first: scaled logits far
// from 0 would carry the rounding of c.
template <typename TIn>
__device__ __forceinline__ void exp_sum(const uint4& v, f32x2 minus_ref, f32x2 c, f32x2& acc) {
  f32x2 f[Elem<TIn>::kVec / 2];
  Elem<TIn>::unpack2(v, f);
#pragma unroll
  for (int i = 0; i < Elem<TIn>::kVec / 2; ++i) {
    float x, y;
    f2_unpack(f2_mul(f2_add(f[i], minus_ref), c), x, y);
    acc = f2_add(acc, f2_pack(ex2(x), ex2(y)));
  }
}

// The sum over a thread's vectors of the staged slice: i, i + kStride, ...
template <typename TIn, int kStride = kRowThreads>
__device__ __forceinline__ float slice_exp_sum(const uint4* data, int count, float ref, float c, int i = threadIdx.x) {
  const f32x2 r2 = f2_pack(-ref, -ref), c2 = f2_pack(c, c);
  f32x2 a0 = 0ull, a1 = 0ull;
  for (; i + kStride < count; i += 2 * kStride) {
    const uint4 u = data[i], w = data[i + kStride];
    exp_sum<TIn>(u, r2, c2, a0);
    exp_sum<TIn>(w, r2, c2, a1);
  }
  if (i < count) exp_sum<TIn>(data[i], r2, c2, a0);
  float x, y;
  f2_unpack(f2_add(a0, a1), x, y);
  return x + y;
}

template <typename TIn, int kStride = kRowThreads>
__device__ __forceinline__ float slice_max(const uint4* data, int count, int i = threadIdx.x) {
  float m = -INFINITY, m1 = -INFINITY;
  for (; i + kStride < count; i += 2 * kStride) {
    const uint4 u = data[i], w = data[i + kStride];
    m = fmax_nan(m, Elem<TIn>::vec_max(u));
    m1 = fmax_nan(m1, Elem<TIn>::vec_max(w));
  }
  if (i < count) m = fmax_nan(m, Elem<TIn>::vec_max(data[i]));
  return fmax_nan(m, m1);
}

// The gradient outside the atoms, k 2^((f - ref) c), of a staged vector.
//
// Rounded to bf16, |k| goes into the exponent (d = log2 |k|) and its sign into
// the conversion; where |ref c| is moderate (kFar false) so does -ref c: the
// product f c then carries c's rounding (2^-24 |f c|, below 2^-13).
struct GradScale {
  float k, d, ref, c;
};
template <typename TIn, bool kNegative, bool kFar>
__device__ __forceinline__ uint4 gradient_of(const uint4& v, const GradScale& g) {
  constexpr int kPairs = Elem<TIn>::kVec / 2;
  const f32x2 c2 = f2_pack(g.c, g.c), r2 = f2_pack(-g.ref, -g.ref);
  f32x2 f[kPairs];
  uint32_t out[4];
  Elem<TIn>::unpack2(v, f);
#pragma unroll
  for (int i = 0; i < kPairs; ++i) {
    float x, y;
    if (sizeof(TIn) == 2) {
      const f32x2 d2 = f2_pack(g.d, g.d);
      f2_unpack(f2_fma(kFar ? f2_add(f[i], r2) : f[i], c2, d2), x, y);
      out[i] = kNegative ? Elem<uint16_t>::pack2(-ex2(x), -ex2(y)) : Elem<uint16_t>::pack2(ex2(x), ex2(y));
    } else {
      const f32x2 k2 = f2_pack(g.k, g.k);
      f2_unpack(f2_mul(f2_add(f[i], r2), c2), x, y);
      f2_unpack(f2_mul(f2_pack(ex2(x), ex2(y)), k2), x, y);
      out[2 * i] = __float_as_uint(x);
      out[2 * i + 1] = __float_as_uint(y);
    }
  }
  return make_uint4(out[0], out[1], out[2], out[3]);
}

// The logit that the loss terms of some atoms are formed around: their largest,
// or 0 where 64 bits lose nothing by that (2^-29 of log p - log q).  In a row of
// nothing but the type's lowest value the differences are all that is left;
// taking the largest always cost 1.5% of the call, this 1.1% (384 rows of 128256
// bf16 44.7 us without either, 45.4 and 45.2 with them; small_weight below costs
// up to 0.6% more).
__device__ __forceinline__ float atom_ref(float atom_max, float c) {
  return atom_max > -INFINITY && fabsf(atom_max) * c > 16777216.f ? atom_max : 0.f;
}

// What one warp, and then one CTA, of a distillation row found: sums of
// exponentials of its tail logits and atoms around their maxima (tail_sum NaN:
// the row is void), and for the loss sum_m p_m ((t_m - top) - (z_m - r)) / T and
// sum_m p_m, with r = atom_ref(atom_max).
// (The loss takes the sum of the p_m as they were rounded: their errors then
// enter with the size of log p - log q, not of log q.)
struct __align__(16) DistillPart {
  float tail_max, tail_sum, atom_max, atom_sum;
  double numer, weight;
  int flags;
};

// Log-weights, relative to the largest, at and below which e^x is 0 in 64 bits:
// such a teacher's token has no weight.
constexpr double kNoWeight = -745.0;

// A weight below fp32's range, e^log_weight * inv_total.  It counts at logits this
// low: where q is 0 the loss is infinite, and the type's lowest value is large
// enough to be seen.
constexpr float kMasked = -1e30f;
__device__ __forceinline__ double small_weight(double log_weight, float inv_total) {
  const float e = ex2(fmaxf(static_cast<float>(log_weight * 1.4426950408889634) + 126.f, -126.f)) * inv_total;
  return static_cast<double>(e) * 1.1754943508222875e-38 + 1e-300;  // 2^-126
}

// The teacher's weights: p_m = exp((t_m - top) / T) / total, p_tail likewise.
struct DistillTeacher {
  double top, total;  // top in units of logits / T
  float inv_total, p_tail;
  int flags;
};

// The joined row, as the gradient needs it.
struct DistillJoin {
  GradScale scale;       // outside the atoms; k 0: none, or a void row
  float at_top, weight;  // on an atom: weight * (2^((z - at_top) c) / total - p)
  float total;
  int bad, far, late;
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
  double inv_t;   // 1 / T
  float log2e_t;  // log2(e) / T
};

// ---------------------------------------------------------------------------
// Distillation.  With teacher weights p over M atoms and one tail, student
// q = softmax(z / T), q_tail the student's mass outside the atoms:
//   loss = sum_m p_m (log p_m - log q_m) + p_tail (log p_tail - log q_tail)
//   dloss/dz_v = (q_v - p_m) / T at v = id_m,
//                (q_tail - p_tail) / T * exp(z_v / T) / sum_tail elsewhere.
// The atoms' logits are taken out of the staged row (replaced by -inf) before
// the sums, so the tail's sum is formed without them and never by subtraction.
// Exponentials and the sums of one CTA are 32-bit (relative error 2^-22 and
// below); log-weights, whose differences the loss is made of, and the loss are
// 64-bit.
// Each of a slice's phases (load, maximum, exponentials, exchange, exponentials
// again, store) is bound by something else, and they follow one another in a
// CTA: four CTAs of 52 KB slices per SM overlap part of them.  384 rows of
// 128256 bf16 with gradient take 45.4 us (4.4 TB/s of logits and gradient, 67%
// of the copy rate; issue 53%, exp2 pipe 53%), 2048 rows of 151936 252-262 us
// (4.8-5.0 TB/s).  Smaller slices (five to eight CTAs), clusters that stay and stage
// the next row, and a gradient stored in bulk all measured slower.
// ---------------------------------------------------------------------------
template <typename TIn>
__global__ void __launch_bounds__(kRowThreads, 4) ssd_distill_kernel(const DistillArgs a) {
  constexpr int VE = Elem<TIn>::kVec;
  extern __shared__ __align__(128) uint4 data[];
  __shared__ uint64_t bars[kRowWarps], parts_bar;
  __shared__ __align__(16) int32_t ids[SSD_MAX_TOP];
  __shared__ float atoms[SSD_MAX_TOP], logits[SSD_MAX_TOP];  // the teacher's and, of this slice's, the student's
  __shared__ DistillPart warps[kRowWarps];
  __shared__ DistillPart parts[kMaxRowCluster];  // the cluster's, written by their CTAs
  __shared__ DistillTeacher teacher;
  __shared__ DistillJoin join;

  cg::cluster_group cluster = cg::this_cluster();
  const int rank = static_cast<int>(cluster.block_rank()), C = static_cast<int>(cluster.num_blocks());
  const int row = static_cast<int>(blockIdx.x) / C;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const TIn* src = static_cast<const TIn*>(a.in.base) +
                   row_offset(a.in.batch_stride, a.in.row_stride, a.in.rows_per_batch, row);
  TIn* dst = a.grad ? static_cast<TIn*>(a.grad) +
                          row_offset(a.g_batch_stride, a.g_row_stride, a.in.rows_per_batch, row)
                    : nullptr;
  stream_wait();
  // All of the row's small inputs are asked for at once; one atom per thread.
  const float scale = a.row_scale ? a.row_scale[row] : 1.f;
  const float tail_in = a.tail ? a.tail[row] : -INFINITY;
  const int id = tid < a.M ? a.tokens[static_cast<long long>(row) * a.M + tid] : -1;
  const float t_in = tid < a.M ? a.values[static_cast<long long>(row) * a.M + tid] : -INFINITY;
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

  // The parts that this CTA waits for: everyone's sums where it forms a
  // gradient, the loss terms too in the first.
  const uint32_t parts_bytes = (rank == 0 ? 36u : (dst ? 16u : 0u)) * static_cast<uint32_t>(C);
  if (lane == 0) {
    mbar_init(&bars[warp], 1);
    if (warp == 0) mbar_init(&parts_bar, 1);
    mbar_init_fence();
    if (warp == 0) mbar_arrive_expect_tx(&parts_bar, parts_bytes);
  }
  __syncwarp();
  // This CTA runs and has its barrier: the others may write into it.  (Relaxed:
  // the barrier's own fence has published it.)
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  // Each warp loads, patches and sums a piece of the slice of its own, and starts
  // when that piece is there: 384 rows of 128256 bf16 45.3 us against 47.2 behind
  // one barrier for the whole slice, 2048 of 151936 256 against 250.
  const int each = (s.count + kRowWarps - 1) / kRowWarps, skip = min(warp * each, s.count);
  const Slice piece = {s.head, s.first + skip, min(each, s.count - skip)};
  uint4* const staged = data + skip;
  slice_load(src, a.V, piece, staged, &bars[warp]);
  const double invT = a.inv_t;
  const float c = a.log2e_t;
  const float t = id >= 0 ? t_in : -INFINITY;
  ids[tid] = id;
  atoms[tid] = t;
  int flags = 0;
  if (id >= a.V || id < -1) flags |= SSD_ROW_BAD_TOKEN;
  __syncthreads();

  if (warp == 0) {
    // The teacher's weights, while the slice's copies are in flight.
    float top = -INFINITY;
#pragma unroll 1
    for (int i = lane; i < a.M; i += 32) top = fmax_nan(top, atoms[i]);
    top = warp_max_nan(top);
    int f = 0;
    if (!(top < INFINITY) || !(tail_in < INFINITY)) f = SSD_ROW_NONFINITE;     // NaN or +inf
    if (!(top > -INFINITY) && !(tail_in > -INFINITY)) f = SSD_ROW_NONFINITE;  // a teacher without any mass
    const double at_top = fmax(static_cast<double>(top) * invT, static_cast<double>(tail_in));
    float sum = 0.f;
#pragma unroll 1
    for (int i = lane; i < a.M; i += 32)
      sum += ex2(static_cast<float>((static_cast<double>(atoms[i]) * invT - at_top) * 1.4426950408889634));
    const float e_tail = ex2(static_cast<float>((static_cast<double>(tail_in) - at_top) * 1.4426950408889634));
    sum = warp_sum(sum) + e_tail;
    if (lane == 0) teacher = DistillTeacher{at_top, static_cast<double>(sum), 1.f / sum, e_tail / sum, f};
  }
  // Is a token there twice?  The cluster's CTAs share the tokens out, and in each
  // the other warps look while the first is busy, every lane at four earlier ones.
  for (int m = (warp - 1) * C + rank; warp > 0 && m < a.M; m += (kRowWarps - 1) * C) {
    const int want = ids[m];
    bool twice = false;
    for (int j = 4 * lane; j < m; j += 128) {
      const int4 q = *reinterpret_cast<const int4*>(ids + j);
      twice |= q.x == want || (q.y == want && j + 1 < m) || (q.z == want && j + 2 < m) || (q.w == want && j + 3 < m);
    }
    if (twice && want >= 0) flags |= SSD_ROW_BAD_TOKEN;
  }
  __syncwarp();
  if (!mbar_wait_bounded(&bars[warp], 0, kRowWaitNs)) {
    flags |= SSD_ROW_DEVICE_TIMEOUT;
    (void)mbar_wait_bounded(&bars[warp], 0, kRowWaitNs);  // the copies still target this CTA's shared memory
  }
  __syncwarp();

  // Take the piece's atoms out of the staged row.
  const int w0 = max(piece.first * VE - piece.head, 0);
  const int w1 = piece.count > 0 ? min((piece.first + piece.count) * VE - piece.head, a.V) : w0;
#pragma unroll 1
  for (int i = lane; i < a.M; i += 32) {
    const int at = ids[i];
    if (at >= w0 && at < w1) {
      TIn* const e = reinterpret_cast<TIn*>(staged) + (at + piece.head - piece.first * VE);
      logits[i] = Elem<TIn>::to_float(*e);
      *e = Elem<TIn>::neg_inf();
    }
  }
  __syncwarp();
  const float m = warp_max_nan(slice_max<TIn, 32>(staged, piece.count, lane));
  const float ref = is_number(m) ? m : 0.f;
  float sum = slice_exp_sum<TIn, 32>(staged, piece.count, ref, c, lane);
  __syncthreads();

  const bool mine = id >= v0 && id < v1;
  const float z_atom = mine ? logits[tid] : -INFINITY;
  const double t_rel = static_cast<double>(t) * invT - teacher.top;
  const float p = ex2(static_cast<float>(t_rel * 1.4426950408889634)) * teacher.inv_total;
  {
    if (!(m < INFINITY)) flags |= SSD_ROW_NONFINITE;
    sum = warp_sum(sum);
    float am = -INFINITY, as = 0.f;
    double num = 0.0, weight = 0.0;
    if (warp * 32 < a.M) {
      am = warp_max_nan(z_atom);
      if (!(am < INFINITY)) flags |= SSD_ROW_NONFINITE;
      if (!is_number(am)) am = 0.f;
      as = warp_sum(ex2((z_atom - am) * c));
      weight = warp_sum_d(mine ? static_cast<double>(p) : 0.0);
      const float around = atom_ref(am, c);
      double z = static_cast<double>(z_atom);
      if (__any_sync(0xFFFFFFFFu, around != 0.f)) z -= static_cast<double>(around);  // a branch, rarely taken
      double term = mine && p > 0.f ? static_cast<double>(p) * (t_rel - z * invT) : 0.0;
      const bool small = mine && p == 0.f && z_atom < kMasked && t_rel > kNoWeight;
      if (__any_sync(0xFFFFFFFFu, small)) term = small ? small_weight(t_rel, teacher.inv_total) * (t_rel - z * invT) : term;
      num = warp_sum_d(term);
    }
    flags = __reduce_or_sync(0xFFFFFFFFu, flags) | teacher.flags;
    if (flags) sum = __int_as_float(0x7FC00000);
    if (lane == 0) warps[warp] = DistillPart{ref, sum, am, as, num, weight, flags};
  }
  __syncthreads();
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");  // every CTA runs
  if (warp == 0) {
    // The CTA's part, written into every CTA of the cluster (its loss terms only
    // into the first).  Reading the warps' parts remotely from every warp cost
    // more than the sums themselves; ordinary remote stores and a cluster barrier
    // cost a fence: 289 us for 2048 rows of 151936 bf16 against 257.
    DistillPart q = {};
    if (lane < kRowWarps) q = warps[lane];
    float tm = q.tail_sum > 0.f ? q.tail_max : -INFINITY, am = q.atom_sum > 0.f ? q.atom_max : -INFINITY;
    tm = warp_max_nan(tm);
    am = warp_max_nan(am);
    const int fl = __reduce_or_sync(0xFFFFFFFFu, q.flags);
    const float ts = warp_sum8(q.tail_sum > 0.f ? q.tail_sum * ex2((q.tail_max - tm) * c) : 0.f);
    const float as = warp_sum8(q.atom_sum > 0.f ? q.atom_sum * ex2((q.atom_max - am) * c) : 0.f);
    const float around = atom_ref(am, c), own = atom_ref(q.atom_max, c);
    if (__any_sync(0xFFFFFFFFu, own != around))
      q.numer -= q.weight * ((static_cast<double>(own) - static_cast<double>(around)) * invT);
    const double num = warp_sum8(q.numer), weight = warp_sum8(q.weight);
    const DistillPart out = {tm, fl ? __int_as_float(0x7FC00000) : ts, am, as, num, weight, fl};
    if (lane < C && (lane == 0 || dst)) {
      const uint32_t to = cluster_addr(&parts[rank], lane), on = cluster_addr(&parts_bar, lane);
      st_async(to, on, out.tail_max, out.tail_sum, out.atom_max, out.atom_sum);
      if (lane == 0) {
        st_async(to + offsetof(DistillPart, numer), on, out.numer, out.weight);
        st_async(to + offsetof(DistillPart, flags), on, out.flags);
      }
    }
  }
  if (!dst && rank != 0) return;  // nobody writes into this CTA

  // One warp joins the cluster's parts, in the same order in every CTA, in 32
  // bits: all the gradient needs.
  float4 q = make_float4(-INFINITY, 0.f, -INFINITY, 0.f);
  float tail_max = -INFINITY, atom_max = -INFINITY, at_top = -INFINITY;
  bool bad = false;
  int late = 0;
  if (warp == 0) {
    // one verdict for the warp: a part that only some lanes waited long enough for counts for none
    late = static_cast<int>(__reduce_or_sync(0xFFFFFFFFu, static_cast<unsigned>(parts_wait(&parts_bar))));
    if (lane < C) q = *reinterpret_cast<const float4*>(&parts[lane]);
    tail_max = warp_max_nan(q.x);
    atom_max = warp_max_nan(q.z);
    const float tail = warp_sum8(q.y == 0.f ? 0.f : q.y * ex2((q.x - tail_max) * c));  // NaN stays
    const float atom = warp_sum8(q.w == 0.f ? 0.f : q.w * ex2((q.z - atom_max) * c));
    at_top = fmaxf(tail_max, atom_max);
    const float tail_share = tail_max > -INFINITY ? tail * ex2((tail_max - at_top) * c) : 0.f;
    const float total = tail_share + (atom_max > -INFINITY ? atom * ex2((atom_max - at_top) * c) : 0.f);
    bad = !(tail >= 0.f) || !(total > 0.f) || late != 0;  // a void row; every logit -inf
    if (lane == 0) {
      const float w = scale * static_cast<float>(invT);
      const float k = bad || !(tail > 0.f) ? 0.f : w * (tail_share / total - teacher.p_tail) / tail;
      const float ref = tail > 0.f ? tail_max : 0.f;
      const bool far = !(fabsf(ref * c) <= 1024.f);
      join = DistillJoin{{k, log2f(fabsf(k)) - (far ? 0.f : ref * c), ref, c}, at_top, w, total, bad, far, late};
    }
  }
  if (dst) {
    __syncthreads();
    const DistillJoin j = join;
    // whole vectors only where the row's places in both tensors agree modulo 16 bytes
    const bool same = ((reinterpret_cast<uintptr_t>(dst) ^ reinterpret_cast<uintptr_t>(src)) & 15u) == 0;
    const int shift = s.first * VE - s.head;  // the token of the slice's first place
    const int whole0 = same ? (shift < 0 ? 1 : 0) : s.count, whole1 = same ? min(s.count, (a.V - shift) / VE) : s.count;
    // the vectors at the row's edges, or all of them
    const auto by_element = [&](int i, const uint4& g) {
      const TIn* e = reinterpret_cast<const TIn*>(&g);
#pragma unroll
      for (int n = 0; n < VE; ++n) {
        const int v = shift + i * VE + n;
        if (v >= 0 && v < a.V) dst[v] = e[n];
      }
    };
    const auto write = [&](auto value) {
#pragma unroll 2
      for (int i = whole0 + tid; i < whole1; i += kRowThreads) *reinterpret_cast<uint4*>(dst + shift + i * VE) = value(i);
      if (same) {
        if (tid == 0 && whole0 == 1 && s.count > 0) by_element(0, value(0));
        if (tid == 32 && whole1 < s.count && whole1 >= whole0) by_element(whole1, value(whole1));
      } else {
        for (int i = tid; i < s.count; i += kRowThreads) by_element(i, value(i));
      }
    };
    if (j.scale.k == 0.f) {  // also a void row, whose logits may be NaN
      // NaN (in either type) where only this CTA gave up: the first one's status need not tell
      const uint32_t w = j.late ? 0x7FC07FC0u : 0u;
      write([w](int) { return make_uint4(w, w, w, w); });
    } else if (sizeof(TIn) == 2 && j.far)
      j.scale.k < 0.f ? write([&](int i) { return gradient_of<TIn, true, true>(data[i], j.scale); })
                      : write([&](int i) { return gradient_of<TIn, false, true>(data[i], j.scale); });
    else if (sizeof(TIn) == 2 && j.scale.k < 0.f)
      write([&](int i) { return gradient_of<TIn, true, false>(data[i], j.scale); });
    else
      write([&](int i) { return gradient_of<TIn, false, false>(data[i], j.scale); });
    __syncthreads();  // the atoms' places are written after the vectors that hold them
    if (mine && !j.bad)
      dst[id] = Elem<TIn>::from_float(j.weight * (ex2((z_atom - j.at_top) * c) / j.total - p));
  }
  if (rank == 0 && warp == 0) {
    // The loss is made of differences of logarithms: 64 bits.
    const DistillPart* own = &parts[lane < C ? lane : 0];
    const bool on = lane < C;
    const double tail_d =
        warp_sum8(on && q.y > 0.f ? static_cast<double>(q.y) * static_cast<double>(ex2((q.x - tail_max) * c)) : 0.0);
    const double atom_d =
        warp_sum8(on && q.w > 0.f ? static_cast<double>(q.w) * static_cast<double>(ex2((q.z - atom_max) * c)) : 0.0);
    const double own_weight = on ? own->weight : 0.0;
    double numer = on ? own->numer : 0.0, top = static_cast<double>(at_top) * invT;  // top: what the terms leave to it
    if (__any_sync(0xFFFFFFFFu, atom_ref(q.z, c) != 0.f)) {
      if (on) numer -= own_weight * ((static_cast<double>(atom_ref(q.z, c)) - static_cast<double>(at_top)) * invT);
      top = 0.0;
    }
    const double num = warp_sum8(numer), weight = warp_sum8(own_weight);
    int fl = __reduce_or_sync(0xFFFFFFFFu, on ? own->flags : 0) | late;
    // Both around the larger maximum; the tail's own logarithm is kept where its share underflows.
    const float other = tail_max > atom_max ? atom_max : tail_max;
    const double factor = other > -INFINITY ? exp((static_cast<double>(other) - static_cast<double>(at_top)) * invT) : 0.0;
    const double total_d = tail_max > atom_max ? tail_d + atom_d * factor : tail_d * factor + atom_d;
    // three logarithms at once
    const double logs = log(lane == 0 ? total_d : (lane == 1 ? tail_d : teacher.total));
    const double lse = __shfl_sync(0xFFFFFFFFu, logs, 0), log_tail = __shfl_sync(0xFFFFFFFFu, logs, 1);  // around at_top, tail_max
    const double lse_tail =
        tail_d > 0.0 ? (static_cast<double>(tail_max) - static_cast<double>(at_top)) * invT + log_tail : -INFINITY;
    const double norm = __shfl_sync(0xFFFFFFFFu, logs, 2);
    if (lane == 0) {
      double p_tail = static_cast<double>(teacher.p_tail);
      double loss = num + weight * (lse + top - norm);
      const double t_tail = static_cast<double>(tail_in) - teacher.top;
      if (!(p_tail > 0.0) && lse_tail < kMasked && t_tail > kNoWeight) p_tail = small_weight(t_tail, teacher.inv_total);
      if (p_tail > 0.0) loss += p_tail * (t_tail - norm - lse_tail + lse);
      if (!(total_d > 0.0)) fl |= SSD_ROW_NONFINITE;
      if (!bad && !(loss < INFINITY)) fl |= SSD_ROW_ZERO_Q;
      a.loss[row] = bad ? __int_as_float(0x7FC00000) : static_cast<float>(loss);
      a.status[row] = fl;
    }
  }
}

// ---------------------------------------------------------------------------
// The top M logits of a row.  Each CTA lists the logits of its slice that can
// be among them (all at or above a threshold that at least M reach), and sums
// the exponentials of the others; a row of one slice is then done, else the
// join kernel ranks the slices' lists.  (One cluster per row, exchanging over
// distributed shared memory, took 54 us for 384 rows of 128256 bf16: its CTAs
// waited for one another three times a row.)  Those rows take 45 us, 36 of them
// here: 17 instructions per logit, of which 6 find the maxima and 6 sum, over
// bytes that alone take 15 us.  CTAs that stay and stage the next slice measured
// 66-69 us, 512 threads on 85 KB slices 53.
// ---------------------------------------------------------------------------
struct TopArgs {
  RowsIn in;
  int32_t* tokens;  // [rows, M]
  float* values;    // [rows, M]
  float* lse;       // [rows]
  float* tail;      // [rows]
  int32_t* status;  // [rows]
  struct TopSlice* slices;       // [rows, n_slices]
  unsigned long long* keys;      // [rows, n_slices, kPool]
  int V, M, slice_vecs, n_slices;
  double inv_t;
  float log2e_t;
};

// What one slice found: the largest key (which tells NaN and +inf), how many
// keys it lists, the 16 high bits of a key that M of them reach (0: of none),
// and the sum of the exponentials of its other logits around ref.
struct TopSlice {
  double sum;
  float ref;
  uint32_t top, cut;
  int count, timeout;
};

// Maxima of a slice: every thread's largest vector maximum, and for larger M its
// second largest too.  Their M-th largest is a lower bound of the slice's M-th
// largest logit, and few logits reach it.
constexpr int kMaxima = 2 * kRowThreads;
static_assert(kPool % 2 == 0 && kPool * sizeof(uint16_t) <= kMaxima * sizeof(uint32_t), "the maxima's place holds the vectors'");
static_assert(kMaxima >= 2 * SSD_MAX_TOP && kPool > SSD_MAX_TOP, "more maxima and places than logits asked for");

// The key of a logit from its kKeyBits high bits: the bits below them are the
// complement of the mantissa's zeros in a negative logit's key.
template <typename TIn>
__device__ __forceinline__ uint32_t full_key(uint32_t k) {
  if (Elem<TIn>::kKeyBits == 16 && !(k & 0x80000000u)) k |= 0xFFFFu;
  return k;
}

// A threshold that at least M of a warp's keys reach, and no more than about
// M / 4 above that, by quartering the range of the keys' 16 high bits; and the
// largest key.  One warp runs through it while the others wait, so it is a loop
// of few instructions: a search of all 16 bits took 3600 cycles, and 5900
// unrolled, since straight-line code waits for its instructions.
template <int kPerLane>
__device__ __forceinline__ uint2 threshold_and_top(const uint32_t* all, int M) {
  const int lane = threadIdx.x & 31;
  uint32_t keys[kPerLane], top = 0u, low = 0xFFFFFFFFu;
#pragma unroll
  for (int i = 0; i < kPerLane; ++i) {
    keys[i] = all[i * 32 + lane];
    top = max(top, keys[i]);
    low = min(low, keys[i]);
    keys[i] >>= 16;
  }
  top = __reduce_max_sync(0xFFFFFFFFu, top);
  low = __reduce_min_sync(0xFFFFFFFFu, low) >> 16;
  uint32_t high = (top >> 16) + 1u;  // fewer than M reach `high`, at least M reach `low`
#pragma unroll 1
  while (high - low > 1u) {
    const uint32_t d = high - low, m1 = low + (d + 3) / 4, m2 = low + (d + 1) / 2, m3 = low + (3 * d + 3) / 4;
    uint32_t k = 0u;  // three counts of at most kMaxima
#pragma unroll
    for (int i = 0; i < kPerLane; ++i)
      k += (keys[i] >= m1 ? 1u : 0u) + (keys[i] >= m2 ? 1u << 10 : 0u) + (keys[i] >= m3 ? 1u << 20 : 0u);
    k = __reduce_add_sync(0xFFFFFFFFu, k);
    const int n1 = k & 1023u, n2 = (k >> 10) & 1023u, n3 = k >> 20;
    const int reach = n3 >= M ? n3 : (n2 >= M ? n2 : n1);
    if (n3 >= M) {
      low = m3;
    } else if (n2 >= M) {
      low = m2;
      high = min(high, m3);
    } else if (n1 >= M) {
      low = m1;
      high = min(high, m2);
    } else {
      high = min(high, m1);
    }
    if (reach >= M && reach <= M + M / 4 + 4) break;
  }
  return make_uint2(low << 16, top);
}

// A thread's largest vectors by their largest element, and where the first two
// are: few threads hold more than two vectors with candidates.
struct TopVecs {
  float first, second, third;  // NaN in the third when any element is
  int at, at2;
};
template <typename TIn>
__device__ __forceinline__ TopVecs slice_top_vecs(const uint4* data, int count) {
  TopVecs m = {-INFINITY, -INFINITY, -INFINITY, 0, 0};
#pragma unroll 2
  for (int i = threadIdx.x; i < count; i += kRowThreads) {
    const float v = Elem<TIn>::vec_max(data[i]);
    if (v > m.second) {
      m.third = fmax_nan(m.third, m.second);
      const bool best = v > m.first;
      m.second = best ? m.first : v;
      m.at2 = best ? m.at : i;
      m.first = best ? v : m.first;
      m.at = best ? i : m.at;
    } else {
      m.third = fmax_nan(m.third, v);
    }
  }
  return m;
}

__device__ __forceinline__ int key_token(unsigned long long k) {
  return static_cast<int32_t>(0xFFFFFFFFu - static_cast<uint32_t>(k & 0xFFFFFFFFull));
}
__device__ __forceinline__ float key_logit(unsigned long long k) { return key_to_float(static_cast<uint32_t>(k >> 32)); }

// Outputs of a row that cannot be ranked.
__device__ __forceinline__ void top_void(const TopArgs& a, int row, int status) {
  for (int i = threadIdx.x; i < a.M; i += kRowThreads) {
    a.tokens[static_cast<long long>(row) * a.M + i] = -1;
    a.values[static_cast<long long>(row) * a.M + i] = __int_as_float(0x7FC00000);
  }
  if (threadIdx.x == 0) {
    a.lse[row] = a.tail[row] = __int_as_float(0x7FC00000);
    a.status[row] = status;
  }
}

// lse and tail of a row from the sum of the top's exponentials around the row's
// largest logit and the others' around ref.  One warp.
__device__ __forceinline__ void top_logs(const TopArgs& a, int row, float row_max, double top_sum, float ref,
                                         double others) {
  const double share = others > 0.0 ? others * static_cast<double>(ex2((ref - row_max) * a.log2e_t)) : 0.0;
  const int lane = threadIdx.x & 31;
  const double logs = log(lane == 0 ? others : top_sum + share);  // two logarithms at once
  if (lane == 0) {
    a.tail[row] = others > 0.0 ? static_cast<float>(static_cast<double>(ref) * a.inv_t + logs) : -INFINITY;
    a.status[row] = 0;
  }
  if (lane == 1) a.lse[row] = static_cast<float>(static_cast<double>(row_max) * a.inv_t + logs);
}

constexpr int kTopSlices = 16;     // slices of a row, as far as they hold it
constexpr int kMaxTopSlices = 32;  // of a row of more than 3.2 MB
constexpr int kShort = 512;  // keys of a row that are ranked from a list of their own (even)

// Shared memory of top_finish.
struct TopFinish {
  TopSlice slices[kMaxTopSlices];
  __align__(16) unsigned long long list[kShort];
  float ranked[SSD_MAX_TOP];
  float fred[kRowWarps];
  double dred[kRowWarps];
  unsigned long long ured[kRowWarps], last;
  int n_list;
};

// The outputs of a row from its n listed keys (with a 0 behind them: 0 is below
// every key) and its slices' sums.  Whatever order the keys stand in, the
// results are the same bits: ranks are exact, the top's sum runs over the ranks,
// and the other listed ones are summed in integers.
__device__ __forceinline__ void top_finish(const TopArgs& a, int row, unsigned long long* keys, int n, int S,
                                           TopFinish& f) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const float c = a.log2e_t;
  if (tid == 0) f.n_list = 0;
  __syncthreads();
  uint32_t top = 0u;
  int timeout = 0;
  float ref = -INFINITY;
  for (int s = 0; s < S; ++s) {
    top = max(top, f.slices[s].top);
    timeout |= f.slices[s].timeout;
    if (f.slices[s].sum > 0.0) ref = fmaxf(ref, f.slices[s].ref);
  }
  if (timeout || top >= ord_key(INFINITY) || top <= ord_key(-INFINITY)) {
    top_void(a, row, timeout ? SSD_ROW_DEVICE_TIMEOUT : SSD_ROW_NONFINITE);
    return;
  }
  const float row_max = key_to_float(top);

  // A cut at 16 bits that at least M keys reach, and not many more, by halving
  // from the slices' largest threshold: the barrier counts.
  const uint32_t* high = reinterpret_cast<const uint32_t*>(keys) + 1;  // the logit's half of a key
  uint32_t lo = 0u, hi = (top >> 16) + 1u;
  for (int s = 0; s < S; ++s) lo = max(lo, f.slices[s].cut);
  const uint32_t k0 = tid < n ? high[2 * tid] >> 16 : 0u, k1 = tid + kRowThreads < n ? high[2 * (tid + kRowThreads)] >> 16 : 0u;
#pragma unroll 1
  while (hi - lo > 1u) {
    const uint32_t mid = (lo + hi) >> 1;
    int k = __syncthreads_count(k0 >= mid);
    if (n > kRowThreads) k += __syncthreads_count(k1 >= mid);
    for (int i0 = 2 * kRowThreads; i0 < n; i0 += kRowThreads)
      k += __syncthreads_count(i0 + tid < n && (high[2 * (i0 + tid)] >> 16) >= mid);
    if (k >= a.M) {
      lo = mid;
      if (k <= a.M + a.M / 4 + 4) break;
    } else {
      hi = mid;
    }
  }
  const uint32_t cut = lo << 16;
  for (int i0 = warp * 32; i0 < n; i0 += kRowThreads) {
    const int i = i0 + lane;
    const bool on = i < n && high[2 * i] >= cut;
    const uint32_t who = __ballot_sync(0xFFFFFFFFu, on);
    int at = 0;
    if (lane == 0 && who) at = atomicAdd(&f.n_list, __popc(who));
    at = __shfl_sync(0xFFFFFFFFu, at, 0) + __popc(who & ((1u << lane) - 1u));
    if (on && at < kShort) f.list[at] = keys[i];
  }
  __syncthreads();
  const bool fits = f.n_list < kShort;
  const unsigned long long* list = fits ? f.list : keys;
  const int m = fits ? f.n_list : n;
  if (fits && tid == 0) f.list[m] = 0ull;
  __syncthreads();
  // A key's rank is the number of larger ones: four threads count for a key, or
  // two or one where there are many; two keys a load.
  float left = -INFINITY;  // the largest listed logit past the M-th
  const int share = m <= kRowThreads / 4 ? 4 : (m <= kRowThreads / 2 ? 2 : 1);
  for (int i0 = 0; i0 < m; i0 += kRowThreads / share) {
    const int i = i0 + tid / share;
    const unsigned long long k = i < m ? list[i] : ~0ull;
    int pos = 0;
    for (int j = 2 * (tid % share); j < m; j += 2 * share) {
      const ulonglong2 q = *reinterpret_cast<const ulonglong2*>(list + j);
      pos += (q.x > k ? 1 : 0) + (q.y > k ? 1 : 0);
    }
    if (share > 1) pos += __shfl_xor_sync(0xFFFFFFFFu, pos, 1);
    if (share > 2) pos += __shfl_xor_sync(0xFFFFFFFFu, pos, 2);
    if (i < m && tid % share == 0) {
      const float z = key_logit(k);
      if (pos < a.M) {
        a.tokens[static_cast<long long>(row) * a.M + pos] = key_token(k);
        a.values[static_cast<long long>(row) * a.M + pos] = z;
        f.ranked[pos] = z;
        if (pos == a.M - 1) f.last = k;
      }
    }
  }
  __syncthreads();
  const unsigned long long last = f.last;  // the M-th key
  for (int i = tid; i < n; i += kRowThreads)
    if (keys[i] < last) left = fmaxf(left, key_logit(keys[i]));
  left = warp_max_nan(left);
  if (lane == 0) f.fred[warp] = left;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kRowWarps; ++w) left = fmaxf(left, f.fred[w]);
  ref = fmaxf(ref, left);
  if (!(ref > -INFINITY)) ref = 0.f;
  if (!(left > -INFINITY)) left = 0.f;
  // The listed others in 2^-40 of their own largest: a slice's reference can lie
  // far above them.
  unsigned long long rest = 0ull;
  for (int i = tid; i < n; i += kRowThreads)
    if (keys[i] < last) rest += static_cast<unsigned long long>(ex2((key_logit(keys[i]) - left) * c) * 1099511627776.f);
  float top_sum = 0.f;
  for (int i = tid; i < a.M; i += kRowThreads) top_sum += ex2((f.ranked[i] - row_max) * c);
  top_sum = warp_sum(top_sum);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) rest += __shfl_xor_sync(0xFFFFFFFFu, rest, o);
  if (lane == 0) {
    f.dred[warp] = static_cast<double>(top_sum);
    f.ured[warp] = rest;
  }
  __syncthreads();
  if (warp != 0) return;
  double top_d = 0.0;
  rest = 0ull;
#pragma unroll
  for (int w = 0; w < kRowWarps; ++w) {
    top_d += f.dred[w];
    rest += f.ured[w];
  }
  double others = 0.0;
  if (lane < S && f.slices[lane].sum > 0.0)
    others = f.slices[lane].sum * static_cast<double>(ex2((f.slices[lane].ref - ref) * c));
  const double rest_d = static_cast<double>(rest) * 9.094947017729282e-13 * static_cast<double>(ex2((left - ref) * c));
  top_logs(a, row, row_max, top_d, ref, warp_sum_d(others) + (rest > 0ull ? rest_d : 0.0));
}

template <typename TIn>
__global__ void __launch_bounds__(kRowThreads, 4) ssd_top_kernel(const TopArgs a) {
  constexpr int VE = Elem<TIn>::kVec;
  extern __shared__ __align__(128) uint4 data[];
  __shared__ uint64_t bar;
  __shared__ uint32_t maxima[kMaxima];
  __shared__ __align__(16) unsigned long long pool[kPool + 2];  // candidates
  __shared__ double dred[kRowWarps];
  __shared__ int ired[kRowWarps];
  TopFinish& fin = *reinterpret_cast<TopFinish*>(data);  // over the staged slice, when that is done with
  __shared__ int n_pool, n_vecs;
  __shared__ uint2 tau_top;

  stream_wait();
  const int row = static_cast<int>(blockIdx.x) / a.n_slices, part = static_cast<int>(blockIdx.x) - row * a.n_slices;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const TIn* src = static_cast<const TIn*>(a.in.base) +
                   row_offset(a.in.batch_stride, a.in.row_stride, a.in.rows_per_batch, row);
  const Slice s = slice_of(src, a.V, a.slice_vecs, part);
  const int base = s.first * VE - s.head;  // token id of the first staged place
  const int v0 = max(base, 0), v1 = s.count > 0 ? min(base + s.count * VE, a.V) : v0;  // the slice's tokens
  const float c = a.log2e_t;

  if (warp == kRowWarps - 1) {
    if (lane == 0) {
      mbar_init(&bar, 1);
      mbar_init_fence();
    }
    __syncwarp();  // the other lanes poll the barrier too
    slice_load(src, a.V, s, data, &bar);
  }
  if (tid == 0) n_pool = n_vecs = 0;
  int timeout = slice_wait(&bar, 0);
  const TopVecs mine = slice_top_vecs<TIn>(data, s.count);
  const bool both = a.M > kMaxima / 4;  // with half of the maxima at or above the threshold, 1.4 M candidates
  // a NaN in the third is the slice's NaN whichever maxima count
  maxima[tid] = ord_key(mine.third == mine.third ? mine.first : mine.third);
  if (both) maxima[kRowThreads + tid] = ord_key(mine.second);
  __syncthreads();
  if (warp == 0) {
    const uint2 t = both ? threshold_and_top<kMaxima / 32>(maxima, a.M) : threshold_and_top<kMaxima / 64>(maxima, a.M);
    if (lane == 0) tau_top = t;
  }
  __syncthreads();
  const uint32_t top_key = tau_top.y;
  const bool ranked = top_key < ord_key(INFINITY) && !timeout;  // no NaN, no +inf
  // With fewer maxima than M, or M of them -inf, every logit is a candidate.
  const float tau = tau_top.x <= ord_key(-INFINITY) ? -INFINITY : key_to_float(full_key<TIn>(tau_top.x));
  float ref = tau > -INFINITY ? tau : 0.f;

  // A candidate goes to the pool, and out of the staged slice: what is left
  // there is the tail.  Past the pool's end nothing is kept, and the slice is
  // read again.
  const auto take = [&](int i, int e, float z) {
    const int at = atomicAdd(&n_pool, 1);
    if (at < kPool) pool[at] = rank_key(z, base + i * VE + e);
    reinterpret_cast<TIn*>(data + i)[e] = Elem<TIn>::neg_inf();
  };
  const auto real = [&](int i, int e) {  // a place of the row, not one beside its ends
    const int id = base + i * VE + e;
    return id >= 0 && id < a.V;
  };
  double below = 0.0;
  if (ranked && top_key <= ord_key(-INFINITY)) {
    // nothing but -inf: the first tokens, in order
    for (int i = tid; i < min(a.M, v1 - v0); i += kRowThreads) pool[i] = rank_key(-INFINITY, v0 + i);
    if (tid == 0) n_pool = min(a.M, v1 - v0);
    __syncthreads();
  } else if (ranked) {
    // The vectors that hold candidates, gathered first and then looked through
    // by all threads: done by each thread for its own, this step took half of
    // the kernel's time.
    uint16_t* vecs = reinterpret_cast<uint16_t*>(maxima);  // no longer used
    const auto note = [&](bool on, int i) {
      const uint32_t who = __ballot_sync(0xFFFFFFFFu, on);
      if (who == 0u) return;
      int at = 0;
      if (lane == 0) at = atomicAdd(&n_vecs, __popc(who));
      at = __shfl_sync(0xFFFFFFFFu, at, 0) + __popc(who & ((1u << lane) - 1u));
      if (on && at < kPool) vecs[at] = static_cast<uint16_t>(i);
    };
    if (!(tau > -INFINITY)) {  // every vector
      for (int i0 = tid - lane; i0 < s.count; i0 += kRowThreads) note(i0 + lane < s.count, i0 + lane);
    } else {
      note(mine.first >= tau, mine.at);
      note(mine.second >= tau, mine.at2);
      if (__any_sync(0xFFFFFFFFu, mine.third >= tau)) {
        for (int i0 = tid - lane; i0 < s.count; i0 += kRowThreads) {
          const int i = i0 + lane;
          note(i < s.count && mine.third >= tau && i != mine.at && i != mine.at2 &&
                   Elem<TIn>::vec_max(data[i]) >= tau,
               i);
        }
      }
    }
    __syncthreads();
    // A vector per thread: its candidates as a mask, their places by a prefix sum.
    const int listed = min(n_vecs, kPool);
    for (int j0 = tid - lane; j0 < listed; j0 += kRowThreads) {
      const int i = j0 + lane < listed ? vecs[j0 + lane] : 0;
      uint32_t on = 0u;
      if (j0 + lane < listed) {
        float f[VE];
        Elem<TIn>::unpack(data[i], f);
#pragma unroll
        for (int e = 0; e < VE; ++e) on |= f[e] >= tau && real(i, e) ? 1u << e : 0u;
      }
      const int k = __popc(on);
      int inc = k;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xFFFFFFFFu, inc, o);
        if (lane >= o) inc += y;
      }
      int at = 0;
      if (lane == 31) at = atomicAdd(&n_pool, inc);
      at = __shfl_sync(0xFFFFFFFFu, at, 31) + inc - k;
      for (; on; on &= on - 1u, ++at) {
        const int e = __ffs(static_cast<int>(on)) - 1;
        TIn* place = reinterpret_cast<TIn*>(data + i) + e;
        if (at < kPool) pool[at] = rank_key(Elem<TIn>::to_float(*place), base + i * VE + e);
        *place = Elem<TIn>::neg_inf();
      }
    }
    if (tid == 0 && n_vecs > kPool) n_pool = kPool + 1;
    __syncthreads();
    const float sum = slice_exp_sum<TIn>(data, s.count, ref, c);
    below = block_reduce(static_cast<double>(sum), dred, OpAdd());
  }
  int n = n_pool;

  if (n > kPool) {
    // Exact select, for slices with many equal logits at the threshold: stage
    // the slice again, find its M-th largest key by two bits a pass, then take
    // the larger ones, and the equal ones in token order.
    __syncthreads();
    if (warp == kRowWarps - 1) {
      fence_proxy_async_shared();
      slice_load(src, a.V, s, data, &bar);
    }
    if (tid == 0) n_pool = 0;
    timeout |= slice_wait(&bar, 1);
    uint32_t prefix = 0u;
#pragma unroll 1
    for (int bit = 30; bit >= 32 - Elem<TIn>::kKeyBits; bit -= 2) {
      const uint32_t c1 = prefix | (1u << bit), c2 = prefix | (2u << bit), c3 = prefix | (3u << bit);
      int n1 = 0, n2 = 0, n3 = 0;
      for (int i = tid; i < s.count; i += kRowThreads) {
        float f[VE];
        Elem<TIn>::unpack(data[i], f);
#pragma unroll
        for (int e = 0; e < VE; ++e) {
          const uint32_t k = real(i, e) ? ord_key(f[e]) : 0u;
          n1 += k >= c1;
          n2 += k >= c2;
          n3 += k >= c3;
        }
      }
      n1 = block_reduce(n1, ired, OpAdd());
      n2 = block_reduce(n2, ired, OpAdd());
      n3 = block_reduce(n3, ired, OpAdd());
      prefix = n3 >= a.M ? c3 : (n2 >= a.M ? c2 : (n1 >= a.M ? c1 : prefix));
    }
    const float kth = key_to_float(full_key<TIn>(prefix));
    int need = 0;  // of the equal ones, in token order
    for (int i = tid; i < s.count; i += kRowThreads) {
      float f[VE];
      Elem<TIn>::unpack(data[i], f);
#pragma unroll
      for (int e = 0; e < VE; ++e) need += real(i, e) && f[e] > kth;
    }
    need = a.M - block_reduce(need, ired, OpAdd());
    int taken = 0;
    for (int i0 = 0; i0 < s.count; i0 += kRowThreads) {
      const int i = i0 + tid;
      float f[VE];
      int eq = 0;
      if (i < s.count) {
        Elem<TIn>::unpack(data[i], f);
#pragma unroll
        for (int e = 0; e < VE; ++e) {
          if (!real(i, e)) f[e] = __int_as_float(0x7FC00000);  // equal to nothing
          eq += f[e] == kth;
        }
      }
      int inc = eq;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xFFFFFFFFu, inc, o);
        if (lane >= o) inc += y;
      }
      __syncthreads();
      if (lane == 31) ired[warp] = inc;
      __syncthreads();
      int before = taken + inc - eq, chunk = 0;
#pragma unroll
      for (int w = 0; w < kRowWarps; ++w) {
        if (w < warp) before += ired[w];
        chunk += ired[w];
      }
      if (i < s.count) {
#pragma unroll
        for (int e = 0; e < VE; ++e) {
          if (f[e] > kth) take(i, e, f[e]);
          if (f[e] == kth) {
            if (before < need) take(i, e, f[e]);
            ++before;
          }
        }
      }
      taken += chunk;
    }
    ref = kth > -INFINITY ? kth : 0.f;
    below = block_reduce(static_cast<double>(slice_exp_sum<TIn>(data, s.count, ref, c)), dred, OpAdd());
    n = a.M;
  }
  // Others far below the threshold: sum them again around their own maximum.
  if (ranked && n < v1 - v0 && below < 1e-18) {
    const float m = static_cast<float>(
        block_reduce(static_cast<double>(slice_max<TIn>(data, s.count)), dred, OpMax()));
    if (m > -INFINITY) {
      ref = m;
      below = block_reduce(static_cast<double>(slice_exp_sum<TIn>(data, s.count, ref, c)), dred, OpAdd());
    }
  }

  if (!ranked) n = 0;
  const uint32_t cut = n >= a.M ? tau_top.x >> 16 : 0u;
  if (a.n_slices > 1) {
    const size_t at = static_cast<size_t>(row) * a.n_slices + part;
    unsigned long long* out = a.keys + at * kPool;
    __syncthreads();  // the pool
    for (int i = tid; i < n; i += kRowThreads) out[i] = pool[i];
    if (tid == 0) a.slices[at] = TopSlice{below, ref, top_key, cut, n, timeout};
    return;
  }
  if (tid == 0) {
    fin.slices[0] = TopSlice{below, ref, top_key, cut, n, timeout};
    pool[n] = 0ull;
  }
  top_finish(a, row, pool, n, 1, fin);
}

// A CTA per row: the slices' lists, one after the other, then as above.
__global__ void __launch_bounds__(kRowThreads) ssd_top_join_kernel(const TopArgs a) {
  extern __shared__ __align__(128) uint4 staged[];
  unsigned long long* keys = reinterpret_cast<unsigned long long*>(staged);  // [n_slices * kPool + 2]
  __shared__ TopFinish fin;
  const int row = blockIdx.x, tid = threadIdx.x, S = a.n_slices;
  stream_wait();  // the slices' results
  if (tid < S) fin.slices[tid] = a.slices[static_cast<size_t>(row) * S + tid];
  __syncthreads();
  int n = 0;
  for (int s = 0; s < S; ++s) n += fin.slices[s].count;
  for (int s = tid >> 5; s < S; s += kRowWarps) {  // a warp per list
    const unsigned long long* in = a.keys + (static_cast<size_t>(row) * S + s) * kPool;
    const int count = fin.slices[s].count;
    int off = 0;
    for (int r = 0; r < s; ++r) off += fin.slices[r].count;
#pragma unroll 4
    for (int i = tid & 31; i < count; i += 32) keys[off + i] = __ldcg(in + i);
  }
  if (tid == 0) keys[n] = 0ull;
  top_finish(a, row, keys, n, S, fin);
}

}  // namespace ssd
