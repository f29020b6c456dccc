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

// The teacher's list, an entry to each of the CTA's first threads: its token (-1:
// unused), value a_k and the draft's logit there.  Asked for before the row is gone
// through, so that the two ways to memory lie behind the row's.
struct Entry {
  int token;
  float value, x;
  uint32_t flags;  // of the entry: a token outside [0, V), a value that is NaN or +inf
};
constexpr int kListWarps = kMaxList / 32;
static_assert(kMaxList <= kRowThreads, "an entry to a thread");
template <typename T> __device__ __forceinline__ Entry read_entry(const DistillArgs &a, size_t r, const T *row) {
  Entry e{-1, -INFINITY, 0.0f, 0u};
  if ((int)threadIdx.x < a.K) {
    const size_t i = r * a.K + threadIdx.x;
    e.token = a.token[i];
    if (e.token != -1) {
      e.value = a.logprob[i];
      if (e.token < 0 || e.token >= a.V) {
        e.flags |= SV_ROW_BAD_TOKEN;
        e.token = -1;
      } else {
        e.x = RowElem<T>::load(row + e.token);
      }
      if (!(e.value < INFINITY)) e.flags |= SV_ROW_NAN;
    }
  }
  return e;
}
// What the list comes to, from a part of it for each of its warps: the largest value
// and its exponential's companions.  (1 - exp of the largest value is taken as one
// number, so that a teacher who is almost sure keeps the digits of its doubt.)
struct ListPart {
  float most, others;  // the largest value; sum of exp(value - ref) of all but it
  float top, sum;      // the draft's largest listed logit; sum of 2^((x - top) k)
  int used;
  uint32_t flags;
};
struct List {
  float shift, inv;  // t_k = exp(a_k - ref) inv, ln t_k = a_k - shift
  float ref;
  float rest;        // t_r
  float top, sum;    // as ListPart
  int used;
  uint32_t flags;
};
// One warp's part; ref 0 with tail, the warp's own largest value without.
__device__ __forceinline__ ListPart list_part(const Entry &e, int tail, float k) {
  const unsigned FULL = 0xffffffffu;
  ListPart p;
  p.most = warp_max(e.value);
  const unsigned who = __ballot_sync(FULL, e.value == p.most);
  const float ref = tail || p.most == -INFINITY ? 0.0f : p.most;
  p.others = who && (int)(threadIdx.x & 31) == __ffs(who) - 1 ? 0.0f : expf(e.value - ref);
  const bool there = e.token >= 0;
  p.top = warp_max(there ? e.x : -INFINITY);
  p.sum = there ? ex2_approx((e.x - (p.top == -INFINITY ? 0.0f : p.top)) * k) : 0.0f;
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    p.others += __shfl_xor_sync(FULL, p.others, o);
    p.sum += __shfl_xor_sync(FULL, p.sum, o);
  }
  p.used = __reduce_add_sync(FULL, there ? 1 : 0);
  p.flags = __reduce_or_sync(FULL, e.flags);
  return p;
}
__device__ __forceinline__ List list_of(const ListPart *parts, int tail, float k) {
  List li;
  float most = -INFINITY;
  li.top = -INFINITY;
  li.used = 0;
  li.flags = 0;
  int first = 0;
#pragma unroll
  for (int w = 0; w < kListWarps; ++w) {
    if (parts[w].most > most) {
      most = parts[w].most;
      first = w;
    }
    li.top = fmaxf(li.top, parts[w].top);
    li.used += parts[w].used;
    li.flags |= parts[w].flags;
  }
  li.ref = tail || most == -INFINITY ? 0.0f : most;
  const float top = li.top == -INFINITY ? 0.0f : li.top;
  float others = 0.0f;  // all but the largest
  li.sum = 0.0f;
#pragma unroll
  for (int w = 0; w < kListWarps; ++w) {
    const ListPart &p = parts[w];
    // with tail the parts' sums are taken against 0, as the list's is
    const float o = p.others + (w == first || p.most == -INFINITY ? 0.0f : expf(tail ? p.most : 0.0f));
    others += tail || p.most == -INFINITY ? o : o * expf(p.most - li.ref);
    li.sum += p.top == -INFINITY ? p.sum : p.sum * ex2_approx((p.top - top) * k);
  }
  const float sum = others + expf(most - li.ref);
  li.inv = tail ? 1.0f : sum > 0.0f ? 1.0f / sum : 0.0f;
  li.shift = tail ? 0.0f : li.ref + (sum > 0.0f ? logf(sum) : 0.0f);
  li.rest = tail ? (li.used ? fmaxf(-expm1f(most) - others, 0.0f) : 1.0f) : 0.0f;
  // a teacher's log probabilities are rounded numbers: their sum may pass 1
  if (tail && !(sum < 1.0f + 0x1p-8f)) li.flags |= SV_ROW_NAN;
  if (!tail && li.used && !(sum > 0.0f)) li.flags |= SV_ROW_NAN;  // nothing to normalise
  return li;
}
// an entry's gradient; st: the row's statistics
__device__ __forceinline__ float listed_grad(const Entry &e, const List &li, const float4 &st, float k, float w) {
  const float share = ex2_approx((e.x - st.z) * k) * st.w;
  return (share - expf(e.value - li.ref) * li.inv) * w;
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
  __shared__ ListPart s_list[kListWarps];
  __shared__ RowPart s_part[kRowWarps];
  __shared__ unsigned long long s_all[kMaxRowCluster];  // reference and sum of each CTA
  __shared__ uint32_t s_flags[kMaxRowCluster];
  __shared__ uint32_t s_twice, s_singles;
  __shared__ float s_loss[kListWarps];
  if (C > 1) cluster_arrive_relaxed();
  const T *row = (const T *)a.logits + (int64_t)r * a.row_stride;
  const RowSlice s = row_slice(row, a.V, rank, C);
  const int groups = row_groups(s);
  const bool resident = GRAD && groups <= a.resident;
  const int ahead = resident ? groups : kRing - 1;
  // a bit for each element of the slice: a byte for a piece, the four of a thread in
  // a group a word
  uint32_t *bits = (uint32_t *)(smem + (size_t)a.resident * kGroupBytes);

  for (int g = 0; g < ahead; ++g) {
    if (g < groups) load_group(row, s, g, g, smem);
    group_commit();
  }
  const Entry e = read_entry(a, r, row);
  const float single_x =
      rank == 0 && (int)threadIdx.x < s.singles ? RowElem<T>::load(row + single_at<T>(s, threadIdx.x)) : -INFINITY;
  for (int g = 0; g < groups; ++g) bits[g * kRowThreads + threadIdx.x] = 0;
  if (threadIdx.x == 0) s_twice = s_singles = 0;
  __syncthreads();
  if (e.token >= 0 && in_slice<T>(s, rank, e.token)) {
    const int i = e.token - s.head;
    uint32_t was, bit;
    if (i < 0 || i >= s.vecs * VEC) {
      bit = 1u << (i < 0 ? e.token : e.token - s.vecs * VEC);
      was = atomicOr(&s_singles, bit);
    } else {
      const int v = i / VEC - s.v0;
      bit = 1u << (v % kGroupVecs / kRowThreads * 8 + i % VEC);
      was = atomicOr(&bits[v / kGroupVecs * kRowThreads + v % kRowThreads], bit);
    }
    if (was & bit) s_twice = 1;
  }
  __syncthreads();
  const float k = a.k;
  const unsigned long long k2 = f2_splat(k);
  RowSums sums = row_sums();
  if ((int)threadIdx.x < s.singles && !(s_singles >> threadIdx.x & 1)) add_single<false>(sums, single_x, k);
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
#pragma unroll
    for (int j = 0; j < kPieces; ++j) w[j] = ring_piece(smem, at, j);
    const uint32_t listed = bits[g * kRowThreads + threadIdx.x];
    if (listed) {  // -inf in their places
#pragma unroll
      for (int j = 0; j < kPieces; ++j) {
        if (!(listed >> (8 * j) & 0xffu)) continue;
        float x[VEC];
        RowElem<T>::unpack(w[j], x);
#pragma unroll
        for (int i = 0; i < VEC; ++i)
          if (listed >> (8 * j + i) & 1) x[i] = -INFINITY;
        w[j] = RowElem<T>::pack(x);
      }
    }
    const float top = RowElem<T>::most4(w);
    if (top > sums.lim) raise<false>(sums, top, k);
#pragma unroll
    for (int j = 0; j < kPieces; ++j) add_piece<T, false>(sums, w[j], k2);
    slot = slot + 1 == kRing ? 0 : slot + 1;
    slot_load = slot_load + 1 == kRing ? 0 : slot_load + 1;
  }
  group_wait<0>();

  // the CTA's sums, then the cluster's, to every CTA; the list's in each
  const RowPart mine = warp_join(part_of(sums), k);
  if (lane == 0) s_part[warp] = mine;
  if (warp < kListWarps) {
    const ListPart p = list_part(e, a.tail, k);
    if (lane == 0) s_list[warp] = p;
  }
  __syncthreads();
  RowPart rest = warp_join(lane < kRowWarps ? s_part[lane] : RowPart{-INFINITY, 0.0f, 0.0f}, k);
  const uint32_t twice = s_twice ? SV_ROW_BAD_TOKEN : 0u;
  uint32_t flags = twice;
  if (C > 1) {
    cluster_wait();
    if (warp == 0 && lane < (int)C) {
      cluster_st_u64(&s_all[rank], lane, (unsigned long long)__float_as_uint(rest.l) << 32 | __float_as_uint(rest.top));
      asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(cluster_addr(&s_flags[rank], lane)), "r"(twice) : "memory");
    }
    asm volatile("barrier.cluster.arrive.release;" ::: "memory");
  }
  const List li = list_of(s_list, a.tail, k);
  if (C > 1) {
    cluster_wait();
    RowPart p{-INFINITY, 0.0f, 0.0f};
    if (lane < (int)C) {
      p.top = __uint_as_float((uint32_t)s_all[lane]);
      p.l = __uint_as_float((uint32_t)(s_all[lane] >> 32));
    }
    rest = warp_join(p, k);
    flags = __reduce_or_sync(0xffffffffu, lane < (int)C ? s_flags[lane] : 0u);
  }
  // every warp: the row's sum, and what the unlisted elements' gradient takes
  const bool skip = li.used == 0 && li.flags == 0;
  const bool has_rest = rest.top != -INFINITY;
  const float top = fmaxf(rest.top, li.top), ref = top == -INFINITY ? 0.0f : top;
  const RowPart all = moved(rest, ref, k);
  const float l = all.l + (li.top == -INFINITY ? 0.0f : li.sum * ex2_approx((li.top - ref) * k));
  flags |= li.flags;
  if (!(l > 0.0f)) flags |= SV_ROW_NAN;
  if (skip) flags = 0;
  // a list of the whole vocabulary leaves nothing, but for its rounding
  const float t_rest = li.used == a.V ? 0.0f : li.rest;
  const float coef = has_rest ? (all.l / l - t_rest) / rest.l : 0.0f;
  const float4 st = skip || flags ? make_float4(__uint_as_float(flags), 0.0f, 0.0f, 0.0f)
                                  : make_float4(has_rest ? rest.top : 0.0f, coef, ref, 1.0f / l);
  if (rank == 0 && warp < kListWarps) {
    // ln s_v = (x_v - ref) / T - ln l, of the rest (rest.top - ref) / T + ln(rest.l / l)
    const float log_l = logf(l), t = expf(e.value - li.ref) * li.inv;
    float loss = e.token >= 0 && t > 0.0f ? t * (e.value - li.shift - ((e.x - ref) / a.temperature - log_l)) : 0.0f;
#pragma unroll
    for (int o = 16; o; o >>= 1) loss += __shfl_xor_sync(0xffffffffu, loss, o);
    if (warp == 0 && t_rest > 0.0f)
      loss += t_rest * (logf(t_rest) - (has_rest ? (rest.top - ref) / a.temperature + logf(rest.l) - log_l : -INFINITY));
    if (lane == 0) s_loss[warp] = loss;
  }
  if constexpr (GRAD) {
    const float w = (a.weight ? a.weight[r] : 1.0f) / a.temperature;
    T *grad = (T *)a.grad + (int64_t)r * a.grad_stride;
    // a row without a gradient has 0 for 1 / l
    const float c = st.w == 0.0f ? 0.0f : st.y * w;
    if (resident)
      write_grad<T>(row, grad, s, rank, st.x, c, k, [&](int g, int j, int) { return ring_piece(smem, g, j); });
    else
      write_grad<T>(row, grad, s, rank, st.x, c, k, [&](int, int, int v) { return ((const uint4 *)(row + s.head))[v]; });
    __syncthreads();
    if (st.w != 0.0f && e.token >= 0 && in_slice<T>(s, rank, e.token))
      grad[e.token] = RowElem<T>::store(listed_grad(e, li, st, k, w));
  } else {
    __syncthreads();
  }
  if (rank == 0 && threadIdx.x == 0) {
    float loss = 0.0f;
#pragma unroll
    for (int i = 0; i < kListWarps; ++i) loss += s_loss[i];
    if (a.stat) a.stat[r] = st;
    a.loss[r] = skip ? 0.0f : flags ? __int_as_float(0x7fffffff) : loss;
    a.status[r] = flags;
  }
}

// The gradient from a forward pass's statistics: CTA `rank` of C of a row.
template <typename T>
__global__ void __launch_bounds__(kRowThreads, 4) distill_grad_kernel(DistillArgs a, unsigned C) {
  grid_dep_sync();
  const size_t r = blockIdx.x / C;
  const uint32_t rank = blockIdx.x % C;
  __shared__ ListPart s_list[kListWarps];
  const T *row = (const T *)a.logits + (int64_t)r * a.row_stride;
  T *grad = (T *)a.grad + (int64_t)r * a.grad_stride;
  const RowSlice s = row_slice(row, a.V, rank, C);
  const Entry e = read_entry(a, r, row);
  const float4 st = a.stat[r];
  const float w = (a.weight ? a.weight[r] : 1.0f) / a.temperature;
  if ((threadIdx.x >> 5) < kListWarps) {
    const ListPart p = list_part(e, a.tail, a.k);
    if ((threadIdx.x & 31) == 0) s_list[threadIdx.x >> 5] = p;
  }
  __syncthreads();
  const List li = list_of(s_list, a.tail, a.k);
  const uint32_t flags = li.flags | (li.used && st.w == 0.0f ? __float_as_uint(st.x) : 0u);
  const bool none = st.w == 0.0f || flags || li.used == 0;
  write_grad<T>(row, grad, s, rank, st.x, none ? 0.0f : st.y * w, a.k,
                [&](int, int, int v) { return ((const uint4 *)(row + s.head))[v]; });
  __syncthreads();
  if (!none && e.token >= 0 && in_slice<T>(s, rank, e.token))
    grad[e.token] = RowElem<T>::store(listed_grad(e, li, st, a.k, w));
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
  z.smem = (size_t)z.resident * kGroupBytes + (size_t)groups * kGroupVecs;
  return z;
}

template <typename T, bool GRAD> cudaError_t launch_loss(DistillArgs a, cudaStream_t st) {
  const Shape z = shape_of(a.V, sizeof(T), a.R, GRAD);
  a.resident = z.resident;
  static thread_local int set_dev = -1;
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev != set_dev) {  // as much as the longest rows take: a ring and a bit for each element
    const size_t bits = (size_t)SV_MAX_VOCAB * sizeof(T) / 16 / kMaxRowCluster + kGroupVecs;
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
