// distill.cu -- the loss that trains a draft on its teacher's most likely
// tokens, and its gradient (sm_103a).
//
// A row of the draft's logits x with z = x / T, s = softmax(z), and the teacher's
// list of K tokens with weights t_k: their probabilities, with one class more for
// the rest of the vocabulary, t_r = 1 - sum t_k, s_r = sum of the unlisted s_v
// (tail); or normalised over the list, t_r = 0.
//   L = sum t_k (ln t_k - ln s_k) + t_r (ln t_r - ln s_r)
//   dL/dz_v = s_v - t_v where v is listed, s_v (1 - t_r / s_r) elsewhere.
// The unlisted elements are summed apart from the listed ones, against their own
// reference m and sum l: s_r would be lost as 1 - sum s_k where the draft is sure
// of its list, and with them their gradient is 2^((x - m) k) (s_r - t_r) / l.
//
// Bound: a row is read once and its gradient written once, 4 to 8 operations on
// an element: memory.  A cluster of C CTAs takes a row.  With the gradient asked
// for, a CTA keeps its slice (64 KB at V = 128256) in shared memory: it is summed
// as it arrives, the cluster's sums are exchanged by one barrier, and the
// gradient is taken from the copy.  Slices beyond shared memory are read twice,
// and the loss alone streams through a ring.  Listed elements are found by a bit
// for each element, set before the first piece is summed; they are few, so their
// gradients are written one by one over the others', after a barrier.
#include <math.h>

#include "vocab_rows.cuh"

namespace sv {
namespace {

constexpr int kMaxList = 128;
constexpr int kRing = 3;          // groups of the ring that a slice streams through
constexpr int kResident = 10;     // groups of a slice that stays in shared memory, at most

struct DistillArgs {
  const void *logits;
  int64_t row_stride;
  const int32_t *token;
  const float *logprob, *weight;
  float4 *stat;
  int R, V, K, tail;
  float temperature, k;  // k = log2(e) / T
  float *loss;
  void *grad;
  int64_t grad_stride;
  uint32_t *status;
  int resident;  // groups' places in shared memory
};

// The teacher's list, by the CTA's first warps (thread i: entry i): weights t_k
// and their logarithms; what they add up to and what they leave.  Faults:
// entries outside [0, V) but -1 (an unused one), log probabilities that are NaN
// or +inf, and a list that adds up to more than 1 by more than rounding (tail).
struct List {
  int token[kMaxList];
  float t[kMaxList], log_t[kMaxList], x[kMaxList];
  float rest;       // t_r
  int used;         // entries
  uint32_t flags;
};
// Every thread of the CTA calls it; ends with a barrier.  x: the draft's logits
// of the listed tokens (0 for the unused).
template <typename T> __device__ void read_list(List &li, const DistillArgs &a, size_t r, const T *row) {
  const unsigned FULL = 0xffffffffu;
  constexpr int E = kMaxList / 32;
  const int lane = threadIdx.x & 31;
  if (threadIdx.x < 32) {
    float v[E], most = -INFINITY;
    int tok[E];
    uint32_t flags = 0;
    int used = 0;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int i = lane + 32 * e;
      tok[e] = i < a.K ? a.token[r * a.K + i] : -1;
      v[e] = tok[e] != -1 ? a.logprob[r * a.K + i] : -INFINITY;
      if (tok[e] < -1 || tok[e] >= a.V) {
        flags |= SV_ROW_BAD_TOKEN;
        tok[e] = -1;
      }
      if (!(v[e] < INFINITY)) flags |= SV_ROW_NAN;
      most = fmaxf(most, v[e]);
      used += tok[e] != -1;
    }
    float x[E];
#pragma unroll
    for (int e = 0; e < E; ++e) x[e] = tok[e] >= 0 ? RowElem<T>::load(row + tok[e]) : 0.0f;
    most = warp_max(most);
    // against 1 (the values are log probabilities) or against the list's sum
    const float ref = a.tail || most == -INFINITY ? 0.0f : most;
    // What the list leaves: 1 - exp of its largest value as one number, so that
    // a teacher who is almost sure keeps the digits of its doubt.
    int first = kMaxList;
#pragma unroll
    for (int e = E - 1; e >= 0; --e)
      if (v[e] == most) first = lane + 32 * e;
    first = __reduce_min_sync(FULL, first);
    float sum = 0.0f, left = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const float t = expf(v[e] - ref);
      sum += t;
      left -= lane + 32 * e == first ? expm1f(v[e]) : t;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      sum += __shfl_xor_sync(FULL, sum, o);
      left += __shfl_xor_sync(FULL, left, o);
    }
    const float shift = a.tail ? 0.0f : ref + (sum > 0.0f ? logf(sum) : 0.0f);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int i = lane + 32 * e;
      li.token[i] = tok[e];
      li.log_t[i] = v[e] - shift;
      li.t[i] = a.tail ? expf(v[e]) : sum > 0.0f ? expf(v[e] - ref) / sum : 0.0f;
      li.x[i] = x[e];
    }
    used = __reduce_add_sync(FULL, used);
    flags = __reduce_or_sync(FULL, flags);
    // a teacher's log probabilities are rounded numbers: their sum may pass 1
    if (a.tail && !(sum < 1.0f + 0x1p-8f)) flags |= SV_ROW_NAN;
    if (!a.tail && used && !(sum > 0.0f)) flags |= SV_ROW_NAN;  // nothing to normalise
    if (lane == 0) {
      li.rest = a.tail ? (used ? fmaxf(left, 0.0f) : 1.0f) : 0.0f;
      li.used = used;
      li.flags = flags;
    }
  }
  __syncthreads();
}

__device__ __forceinline__ float listed_grad(const List &li, int i, const float4 &st, float k, float w) {
  const float share = ex2_approx((li.x[i] - st.z) * k) * st.w;
  return (share - li.t[i]) * w;
}

// Gradient of the unlisted elements of piece w.
template <typename T>
__device__ __forceinline__ uint4 grad_piece(const uint4 &w, float m, float coef, float k) {
  constexpr int VEC = RowElem<T>::VEC;
  float x[VEC];
  RowElem<T>::unpack(w, x);
#pragma unroll
  for (int i = 0; i < VEC; i += 2) {
    const unsigned long long y = f2_mul(f2_add(f2_pack(x[i], x[i + 1]), f2_splat(-m)), f2_splat(k));
    float y0, y1;
    f2_unpack(y, y0, y1);
    f2_unpack(f2_mul(f2_pack(ex2_approx(y0), ex2_approx(y1)), f2_splat(coef)), x[i], x[i + 1]);
  }
  return RowElem<T>::pack(x);
}
template <typename T>
__device__ __forceinline__ float grad_of(float x, float m, float coef, float k) {
  return ex2_approx((x - m) * k) * coef;
}

// The slice's gradient in full but for the listed elements: pieces from
// `piece(g, j)` where the gradient's row lies on the 16-byte grid as the logits'
// does, single elements otherwise (those of the logits come from memory again:
// the two rows are different ones then).  coef 0: zeros, whatever the row holds.
template <typename T, typename F>
__device__ void write_grad(const T *row, T *grad, const RowSlice &s, uint32_t rank, float m, float coef, float k, F piece) {
  constexpr int VEC = RowElem<T>::VEC;
  const bool zero = coef == 0.0f;
  if (rank == 0 && (int)threadIdx.x < s.singles) {
    const int i = single_at<T>(s, threadIdx.x);
    grad[i] = RowElem<T>::store(zero ? 0.0f : grad_of<T>(RowElem<T>::load(row + i), m, coef, k));
  }
  if ((uintptr_t)row % 16 == (uintptr_t)grad % 16) {
    uint4 *out = (uint4 *)(grad + s.head);
    const int groups = row_groups(s);
    for (int g = 0; g < groups; ++g) {
      const int v0 = s.v0 + g * kGroupVecs + (int)threadIdx.x;
      uint4 w[kPieces];  // all on their way before the first is stored
#pragma unroll
      for (int j = 0; j < kPieces; ++j)
        if (v0 + j * kRowThreads < s.v1) w[j] = piece(g, j, v0 + j * kRowThreads);
#pragma unroll
      for (int j = 0; j < kPieces; ++j)
        if (v0 + j * kRowThreads < s.v1)
          out[v0 + j * kRowThreads] = zero ? make_uint4(0, 0, 0, 0) : grad_piece<T>(w[j], m, coef, k);
    }
  } else {
    const int lo = s.head + s.v0 * VEC, hi = s.head + s.v1 * VEC;
    for (int i = lo + threadIdx.x; i < hi; i += kRowThreads)
      grad[i] = RowElem<T>::store(zero ? 0.0f : grad_of<T>(RowElem<T>::load(row + i), m, coef, k));
  }
}

// Whether element i of the row is one of the slice's, or of the first CTA's singles.
template <typename T> __device__ __forceinline__ bool in_slice(const RowSlice &s, uint32_t rank, int i) {
  const int v = i - s.head;
  if (v < 0 || v >= s.vecs * RowElem<T>::VEC) return rank == 0;
  return v / RowElem<T>::VEC >= s.v0 && v / RowElem<T>::VEC < s.v1;
}

// waits until at most n of the groups asked for are on their way
__device__ __forceinline__ void wait_all_but(int n) {
  switch (n) {
    case 0: return group_wait<0>();
    case 1: return group_wait<1>();
    case 2: return group_wait<2>();
    case 3: return group_wait<3>();
    case 4: return group_wait<4>();
    case 5: return group_wait<5>();
    case 6: return group_wait<6>();
    case 7: return group_wait<7>();
    case 8: return group_wait<8>();
    default: return group_wait<9>();
  }
}
static_assert(kResident <= 10, "wait_all_but");

template <typename T, bool GRAD>
__global__ void __launch_bounds__(kRowThreads, 3) distill_kernel(DistillArgs a, unsigned C) {
  grid_dep_sync();
  constexpr int VEC = RowElem<T>::VEC;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const size_t r = blockIdx.x / C;
  const uint32_t rank = C > 1 ? cluster_rank() : 0;
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ List li;
  __shared__ RowPart s_part[kRowWarps];
  __shared__ unsigned long long s_all[kMaxRowCluster];  // reference and sum of each CTA
  __shared__ uint32_t s_flags[kMaxRowCluster];
  __shared__ uint32_t s_twice, s_singles;
  __shared__ float4 s_stat;
  if (C > 1) cluster_arrive_relaxed();
  const T *row = (const T *)a.logits + (int64_t)r * a.row_stride;
  const RowSlice s = row_slice(row, a.V, rank, C);
  const int groups = row_groups(s);
  const bool resident = GRAD && groups <= a.resident;
  const int ahead = resident ? groups : kRing - 1;
  // a byte for each piece of the slice, its bits the elements
  uint32_t *bits = (uint32_t *)(smem + (size_t)a.resident * kGroupBytes);
  const unsigned char *piece_bits = (const unsigned char *)bits;

  for (int g = 0; g < ahead; ++g) {
    if (g < groups) load_group(row, s, g, g, smem);
    group_commit();
  }
  for (int i = threadIdx.x; i < (s.v1 - s.v0 + 3) / 4; i += kRowThreads) bits[i] = 0;
  if (threadIdx.x == 0) s_twice = s_singles = 0;
  read_list(li, a, r, row);
  const bool skip = li.used == 0 && li.flags == 0;  // the same in every CTA
  const float k = a.k;
  const unsigned long long k2 = f2_splat(k);
  RowSums sums = row_sums();
  uint32_t flags = li.flags;
  if (!skip && !flags) {
    if ((int)threadIdx.x < a.K) {
      const int t = li.token[threadIdx.x];
      if (t >= 0 && in_slice<T>(s, rank, t)) {
        const int e = t - s.head;
        uint32_t was, bit;
        if (e < 0 || e >= s.vecs * VEC) {
          bit = 1u << (e < 0 ? t : t - s.vecs * VEC);
          was = atomicOr(&s_singles, bit);
        } else {
          const int v = e / VEC - s.v0;
          bit = 1u << (8 * (v & 3) + e % VEC);
          was = atomicOr(&bits[v >> 2], bit);
        }
        if (was & bit) s_twice = 1;
      }
    }
    __syncthreads();
    if (s_twice) flags |= SV_ROW_BAD_TOKEN;
    if (rank == 0 && (int)threadIdx.x < s.singles && !(s_singles >> threadIdx.x & 1))
      add_single<false>(sums, RowElem<T>::load(row + single_at<T>(s, threadIdx.x)), k);
    int slot = 0, slot_load = kRing - 1;
    for (int g = 0; g < groups; ++g) {
      if (resident) {
        wait_all_but(groups - 1 - g);
      } else {
        if (g + kRing - 1 < groups) load_group(row, s, g + kRing - 1, slot_load, smem);
        group_commit();
        group_wait<kRing - 1>();
      }
      const int at = resident ? g : slot;
      uint4 w[kPieces];
      uint32_t listed[kPieces], any = 0;
#pragma unroll
      for (int j = 0; j < kPieces; ++j) {
        w[j] = ring_piece(smem, at, j);
        const int v = g * kGroupVecs + j * kRowThreads + (int)threadIdx.x;
        listed[j] = v < s.v1 - s.v0 ? piece_bits[v] : 0;
        any |= listed[j];
      }
      if (any) {  // -inf in their places
#pragma unroll
        for (int j = 0; j < kPieces; ++j) {
          if (!listed[j]) continue;
          float x[VEC];
          RowElem<T>::unpack(w[j], x);
#pragma unroll
          for (int i = 0; i < VEC; ++i)
            if (listed[j] >> i & 1) x[i] = -INFINITY;
          w[j] = RowElem<T>::pack(x);
        }
      }
      float top = RowElem<T>::most(w[0]);
#pragma unroll
      for (int j = 1; j < kPieces; ++j) top = fmaxf(top, RowElem<T>::most(w[j]));
      if (top > sums.lim) raise<false>(sums, top, k);
#pragma unroll
      for (int j = 0; j < kPieces; ++j) add_piece<T, false>(sums, w[j], k2);
      slot = slot + 1 == kRing ? 0 : slot + 1;
      slot_load = slot_load + 1 == kRing ? 0 : slot_load + 1;
    }
  }
  group_wait<0>();

  // the CTA's sums, then the cluster's, to every CTA
  const RowPart mine = warp_join(part_of(sums), k);
  if (lane == 0) s_part[warp] = mine;
  __syncthreads();
  RowPart rest = warp_join(lane < kRowWarps ? s_part[lane] : RowPart{-INFINITY, 0.0f, 0.0f}, k);
  if (C > 1) {
    cluster_wait();
    if (warp == 0 && lane < (int)C) {
      cluster_st_u64(&s_all[rank], lane, (unsigned long long)__float_as_uint(rest.l) << 32 | __float_as_uint(rest.top));
      asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(cluster_addr(&s_flags[rank], lane)), "r"(flags) : "memory");
    }
    cluster_sync();
    RowPart p{-INFINITY, 0.0f, 0.0f};
    if (lane < (int)C) {
      p.top = __uint_as_float((uint32_t)s_all[lane]);
      p.l = __uint_as_float((uint32_t)(s_all[lane] >> 32));
    }
    rest = warp_join(p, k);
    flags = __reduce_or_sync(0xffffffffu, lane < (int)C ? s_flags[lane] : 0u);
  }
  if (warp == 0) {
    constexpr int E = kMaxList / 32;
    float top = rest.top;
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (li.token[lane + 32 * e] >= 0) top = fmaxf(top, li.x[lane + 32 * e]);
    top = warp_max(top);
    float sum = 0.0f;  // of the listed
    const float ref = top == -INFINITY ? 0.0f : top;
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (li.token[lane + 32 * e] >= 0) sum += ex2_approx((li.x[lane + 32 * e] - ref) * k);
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    const RowPart r_all = moved(rest, ref, k);
    const float l = sum + r_all.l;
    if (!(l > 0.0f)) flags |= SV_ROW_NAN;
    if (skip) flags = 0;
    const bool none = skip || flags;
    // ln s_v = (x_v - ref) / T - ln l, of the rest (rest.top - ref) / T + ln(rest.l / l)
    const float log_l = logf(l);
    float loss = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int i = lane + 32 * e;
      if (li.token[i] >= 0 && li.t[i] > 0.0f)
        loss += li.t[i] * (li.log_t[i] - ((li.x[i] - ref) / a.temperature - log_l));
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) loss += __shfl_xor_sync(0xffffffffu, loss, o);
    const bool has_rest = rest.top != -INFINITY;
    // a list of the whole vocabulary leaves nothing, but for its rounding
    const float t_rest = li.used == a.V ? 0.0f : li.rest;
    if (t_rest > 0.0f)
      loss += t_rest * (logf(t_rest) - (has_rest ? (rest.top - ref) / a.temperature + logf(rest.l) - log_l : -INFINITY));
    if (lane == 0) {
      const float coef = has_rest ? (r_all.l / l - t_rest) / rest.l : 0.0f;
      s_stat = none ? make_float4(__uint_as_float(flags), 0.0f, 0.0f, 0.0f)
                    : make_float4(has_rest ? rest.top : 0.0f, coef, ref, 1.0f / l);
      if (rank == 0) {
        if (a.stat) a.stat[r] = s_stat;
        a.loss[r] = skip ? 0.0f : flags ? __int_as_float(0x7fffffff) : loss;
        a.status[r] = flags;
      }
    }
  }
  if constexpr (GRAD) {
    __syncthreads();
    const float4 st = s_stat;
    const float w = (a.weight ? a.weight[r] : 1.0f) / a.temperature;
    T *grad = (T *)a.grad + (int64_t)r * a.grad_stride;
    // a row without a gradient has 0 for 1 / l
    const float coef = st.w == 0.0f ? 0.0f : st.y * w;
    if (resident)
      write_grad<T>(row, grad, s, rank, st.x, coef, k, [&](int g, int j, int) { return ring_piece(smem, g, j); });
    else
      write_grad<T>(row, grad, s, rank, st.x, coef, k, [&](int, int, int v) { return ((const uint4 *)(row + s.head))[v]; });
    if (st.w == 0.0f) return;
    __syncthreads();
    if ((int)threadIdx.x < a.K) {
      const int t = li.token[threadIdx.x];
      if (t >= 0 && in_slice<T>(s, rank, t)) grad[t] = RowElem<T>::store(listed_grad(li, threadIdx.x, st, k, w));
    }
  }
}

// The gradient from a forward pass's statistics: CTA `rank` of C of a row.
template <typename T>
__global__ void __launch_bounds__(kRowThreads, 4) distill_grad_kernel(DistillArgs a, unsigned C) {
  grid_dep_sync();
  const size_t r = blockIdx.x / C;
  const uint32_t rank = blockIdx.x % C;
  __shared__ List li;
  const T *row = (const T *)a.logits + (int64_t)r * a.row_stride;
  T *grad = (T *)a.grad + (int64_t)r * a.grad_stride;
  const RowSlice s = row_slice(row, a.V, rank, C);
  float4 st = a.stat[r];
  const float w = (a.weight ? a.weight[r] : 1.0f) / a.temperature;
  read_list(li, a, r, row);
  uint32_t flags = li.used == 0 ? li.flags : st.w == 0.0f ? __float_as_uint(st.x) | li.flags : li.flags;
  const bool none = st.w == 0.0f || flags || li.used == 0;
  write_grad<T>(row, grad, s, rank, st.x, none ? 0.0f : st.y * w, a.k,
                [&](int, int, int v) { return ((const uint4 *)(row + s.head))[v]; });
  __syncthreads();
  if (!none && (int)threadIdx.x < a.K) {
    const int t = li.token[threadIdx.x];
    if (t >= 0 && in_slice<T>(s, rank, t)) grad[t] = RowElem<T>::store(listed_grad(li, threadIdx.x, st, a.k, w));
  }
  if (rank == 0 && threadIdx.x == 0) a.status[r] = flags;
}

// CTAs to a row and groups' places of each: with a gradient slices of 64 KB, so
// that three CTAs fit an SM and one's sums hide behind the others' rows; smaller
// ones where a batch of few rows would leave SMs idle.
struct Shape {
  unsigned C;
  int resident;
  size_t smem;
};
Shape shape_of(int V, size_t es, long long R, bool grad) {
  const size_t row = (size_t)V * es;
  Shape z;
  z.C = 1;
  if (grad)
    while (z.C < kMaxRowCluster && (row > z.C * (size_t)65536 || (row > z.C * (size_t)16384 && R * z.C < 456))) z.C *= 2;
  else
    z.C = row_ctas(row, R, 16384, 1216);
  const long long vecs = (long long)(row / 16), per = (vecs + z.C - 1) / z.C;
  const long long groups = (per + kGroupVecs - 1) / kGroupVecs;
  z.resident = grad && groups > kRing && groups <= kResident ? (int)groups : kRing;
  z.smem = (size_t)z.resident * kGroupBytes + align_up((size_t)per, 4);
  return z;
}

template <typename T, bool GRAD> cudaError_t launch_loss(DistillArgs a, cudaStream_t st) {
  const Shape z = shape_of(a.V, sizeof(T), a.R, GRAD);
  a.resident = z.resident;
  static thread_local int set_dev = -1;
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev != set_dev) {  // as much as the longest rows take: a ring and a bit for each element
    const size_t bits = (size_t)SV_MAX_VOCAB * sizeof(T) / 16 / kMaxRowCluster;
    const size_t a0 = kRing * (size_t)kGroupBytes + bits, b0 = kResident * (size_t)(kGroupBytes + kGroupVecs);
    const cudaError_t e = cudaFuncSetAttribute(distill_kernel<T, GRAD>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (int)((GRAD && b0 > a0 ? b0 : a0) + 16));
    if (e != cudaSuccess) return e;
    set_dev = dev;
  }
  return launch_pdl_cluster(distill_kernel<T, GRAD>, dim3((unsigned)a.R * z.C), dim3(kRowThreads), z.C, z.smem, st, a, z.C);
}
template <typename T> cudaError_t launch_grad(const DistillArgs &a, cudaStream_t st) {
  // 64 KB of a row to a CTA
  const unsigned C = (unsigned)(((size_t)a.V * sizeof(T) + 65535) / 65536);
  return launch_pdl(distill_grad_kernel<T>, dim3((unsigned)a.R * C), dim3(kRowThreads), 0, st, a, C);
}

// What both calls check; fills `a` but for the outputs of one of them.
sv_status check_args(DistillArgs &a, const void *logits, int64_t row_stride, sv_dtype dt, const int32_t *token,
                     const float *logprob, const float *weight, int R, int V, int K, float temperature, int tail,
                     void *grad, int64_t grad_stride, uint32_t *status) {
  if (R < 0 || V < 1 || K < 1) return set_error(SV_ERR_INVALID_ARG, "need R >= 0, V >= 1, K >= 1");
  if (dt != SV_F32 && dt != SV_BF16 && dt != SV_F16)
    return set_error(SV_ERR_INVALID_ARG, "unknown dtype %d", (int)dt);
  if (K > V) return set_error(SV_ERR_INVALID_ARG, "K > V");
  if (K > kMaxList) return set_error(SV_ERR_UNSUPPORTED, "K > %d", kMaxList);
  if (V > SV_MAX_VOCAB) return set_error(SV_ERR_UNSUPPORTED, "V > %d", SV_MAX_VOCAB);
  if (tail != 0 && tail != 1) return set_error(SV_ERR_INVALID_ARG, "tail is 0 or 1");
  if (!(temperature > 0.0f) || !isfinite(temperature) || !isfinite(kLog2eF / temperature) ||
      !(kLog2eF / temperature > 0.0f))
    return set_error(SV_ERR_INVALID_ARG, "temperature must be > 0 and finite, its inverse too");
  if (R > (1 << 22)) return set_error(SV_ERR_UNSUPPORTED, "R > %d", 1 << 22);
  const int64_t most = INT64_MAX / 16;  // of any offset, in elements
  if (row_stride < 0 || (R > 0 && row_stride > most / R))
    return set_error(SV_ERR_INVALID_ARG, "negative or too large stride");
  if (grad && R > 1 && (grad_stride < V || grad_stride > most / R))
    return set_error(SV_ERR_INVALID_ARG, "the gradient's rows overlap, or its stride is too large");
  if (R == 0) return SV_OK;
  if (!logits || !token || !logprob || !status) return set_error(SV_ERR_INVALID_ARG, "null pointer");
  if (grad == logits && R > 1 && grad_stride != row_stride)
    return set_error(SV_ERR_INVALID_ARG, "a gradient in the logits' place needs their stride");
  const size_t es = dt == SV_F32 ? 4 : 2;
  if ((uintptr_t)logits % es || (uintptr_t)grad % es || (uintptr_t)token % 4 || (uintptr_t)logprob % 4 ||
      (uintptr_t)weight % 4 || (uintptr_t)status % 4)
    return set_error(SV_ERR_INVALID_ARG, "misaligned pointer");
  sv_status s;
  if ((s = map_arg(logits, "logits")) != SV_OK || (s = map_arg(token, "teacher_token")) != SV_OK ||
      (s = map_arg(logprob, "teacher_logprob")) != SV_OK || (s = map_arg(weight, "weight")) != SV_OK ||
      (s = map_arg(grad, "out_grad")) != SV_OK || (s = map_arg(status, "out_status")) != SV_OK)
    return s;
  a.logits = logits;
  a.row_stride = row_stride;
  a.token = token;
  a.logprob = logprob;
  a.weight = weight;
  a.stat = nullptr;
  a.R = R;
  a.V = V;
  a.K = K;
  a.tail = tail;
  a.temperature = temperature;
  a.k = kLog2eF / temperature;
  a.loss = nullptr;
  a.grad = grad;
  a.grad_stride = grad_stride;
  a.status = status;
  a.resident = 0;
  return SV_OK;
}

}  // namespace
}  // namespace sv

using namespace sv;

extern "C" sv_status sv_distill_loss(const void *logits, int64_t row_stride, sv_dtype dt,
                                     const int32_t *teacher_token, const float *teacher_logprob,
                                     const float *weight, int R, int V, int K, float temperature,
                                     int tail, float *out_loss, float *out_stat, void *out_grad,
                                     int64_t grad_stride, uint32_t *out_status, void *stream) {
  DistillArgs a;
  sv_status s = check_args(a, logits, row_stride, dt, teacher_token, teacher_logprob, weight, R, V, K, temperature,
                           tail, out_grad, grad_stride, out_status);
  if (s != SV_OK || R == 0) return s;
  if (!out_loss) return set_error(SV_ERR_INVALID_ARG, "null pointer");
  if ((uintptr_t)out_loss % 4 || (uintptr_t)out_stat % 16)
    return set_error(SV_ERR_INVALID_ARG, "misaligned pointer (out_stat needs 16 bytes)");
  if ((s = map_arg(out_loss, "out_loss")) != SV_OK || (s = map_arg(out_stat, "out_stat")) != SV_OK) return s;
  a.loss = out_loss;
  a.stat = (float4 *)out_stat;
  cudaStream_t st = (cudaStream_t)stream;
  LaunchScope ls("distill", st);
  cudaError_t e;
  if (out_grad)
    e = dt == SV_F32    ? launch_loss<float, true>(a, st)
        : dt == SV_BF16 ? launch_loss<__nv_bfloat16, true>(a, st)
                        : launch_loss<__half, true>(a, st);
  else
    e = dt == SV_F32    ? launch_loss<float, false>(a, st)
        : dt == SV_BF16 ? launch_loss<__nv_bfloat16, false>(a, st)
                        : launch_loss<__half, false>(a, st);
  return check_launch("distill", e);
}

extern "C" sv_status sv_distill_grad(const void *logits, int64_t row_stride, sv_dtype dt,
                                     const int32_t *teacher_token, const float *teacher_logprob,
                                     const float *stat, const float *weight, int R, int V, int K,
                                     float temperature, int tail, void *out_grad,
                                     int64_t grad_stride, uint32_t *out_status, void *stream) {
  DistillArgs a;
  sv_status s = check_args(a, logits, row_stride, dt, teacher_token, teacher_logprob, weight, R, V, K, temperature,
                           tail, out_grad, grad_stride, out_status);
  if (s != SV_OK || R == 0) return s;
  if (!stat || !out_grad) return set_error(SV_ERR_INVALID_ARG, "null pointer");
  if ((uintptr_t)stat % 16) return set_error(SV_ERR_INVALID_ARG, "misaligned pointer (stat needs 16 bytes)");
  if ((s = map_arg(stat, "stat")) != SV_OK) return s;
  a.stat = (float4 *)stat;
  cudaStream_t st = (cudaStream_t)stream;
  LaunchScope ls("distill_grad", st);
  return check_launch("distill_grad", dt == SV_F32    ? launch_grad<float>(a, st)
                                      : dt == SV_BF16 ? launch_grad<__nv_bfloat16>(a, st)
                                                      : launch_grad<__half>(a, st));
}
