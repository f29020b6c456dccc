// distill.cu -- the loss that trains a draft on its teacher's most likely
// tokens, and its gradient (sm_103a).
//
// A row of the draft's logits x with z = x / T, s = softmax(z), and the teacher's
// list of K tokens with weights t_k: their probabilities, with one class more for
// the rest of the vocabulary, t_r = 1 - sum t_k, s_r = sum of the unlisted s_v
// (tail); or normalised over the list, t_r = 0.
//   L = sum t_k (ln t_k - ln s_k) + t_r (ln t_r - ln s_r)
//   dL/dz_v = s_v - t_v where v is listed, s_v (1 - t_r / s_r) elsewhere
// (s_v times sum t_k, where a teacher's rounded weights add up to more than 1).
// The unlisted elements are summed apart from the listed ones, against their own
// reference m and sum l: s_r would be lost as 1 - sum s_k where the draft is sure
// of its list, and with them their gradient is 2^((x - m) k) (s_r - t_r) / l.
//
// Bound: a row is read once and its gradient written once, 4 to 8 operations on
// an element: memory.  A cluster of C CTAs takes a row, each a slice that streams
// through a ring of shared memory; the cluster's sums are exchanged by one barrier.
// With the gradient asked for, a CTA then goes back through its slice: the last
// three groups are still in the ring, the others come from L2 (so that few rows are
// under way at once, some 80 KB of a row to a CTA), and the gradient is stored past the
// lines that are still to be read.  Listed elements are found by a bit for each
// element, set before the first piece is summed; they are few, so their gradients
// are written one by one over the others', after a barrier.
//
// 2048 rows of V = 128256 bf16, K = 64, loss and gradient: 195 us (5.4 TB/s, 0.79; some
// 8 % of the bytes read are read again), the loss alone 86 (0.90).  Slices kept in
// shared memory, 64 KB to a CTA: 236 us (a third of the CTAs' time stands at barriers);
// clusters that go from row to row with the next row's slice on its way: 301.
#include <math.h>

#include "vocab_rows.cuh"

namespace sv {
namespace {

constexpr int kMaxList = 128;
constexpr int kRing = 3;          // groups of the ring that a slice streams through
// What the teacher's values leave of 1 is rounding where it is less than kRounding: a
// value in 32 bits is off by some 2^-24 of itself, of ln l and of the exponentials that
// l comes from, all of a list's values together by up to (K + 48) 2^-24; below 2^-16 it
// is next to nothing.  A student without a share (below kNoShare: the rest is masked)
// there would have to pay for it with an infinite loss, or 10^-7 of a mask of -3e38.
constexpr float kRounding = 0x1p-16f, kNoShare = 0x1p-100f;

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
  int ring;  // bytes of shared memory that the groups stream through
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
  float total;       // sum of t_k and t_r: 1, or what a teacher's rounded values are above it
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
// The list's, by every warp: a lane to each part.
__device__ __forceinline__ List list_of(const ListPart *parts, int tail, float k) {
  const unsigned FULL = 0xffffffffu;
  const int lane = threadIdx.x & 31;
  ListPart p{-INFINITY, 0.0f, -INFINITY, 0.0f, 0, 0u};
  if (lane < kListWarps) p = parts[lane];
  List li;
  const float most = warp_max(p.most);
  li.top = warp_max(p.top);
  li.used = __reduce_add_sync(FULL, p.used);
  li.flags = __reduce_or_sync(FULL, p.flags);
  const int first = __ffs(__ballot_sync(FULL, p.most == most)) - 1;
  li.ref = tail || most == -INFINITY ? 0.0f : most;
  // all but the largest; with tail the parts' sums are taken against 0, as the list's
  // is, without against their own largest
  float others = 0.0f;
  if (p.most != -INFINITY) {
    others = p.others + (lane == first ? 0.0f : expf(tail ? p.most : 0.0f));
    if (!tail) others *= expf(p.most - li.ref);
  }
  li.sum = p.top == -INFINITY ? p.sum : p.sum * ex2_approx((p.top - li.top) * k);
#pragma unroll
  for (int o = kListWarps / 2; o; o >>= 1) {
    others += __shfl_xor_sync(FULL, others, o);
    li.sum += __shfl_xor_sync(FULL, li.sum, o);
  }
  others = __shfl_sync(FULL, others, 0);
  li.sum = __shfl_sync(FULL, li.sum, 0);
  const float sum = others + expf(most - li.ref);
  li.inv = tail ? 1.0f : sum > 0.0f ? 1.0f / sum : 0.0f;
  li.shift = tail ? 0.0f : li.ref + (sum > 0.0f ? logf(sum) : 0.0f);
  li.rest = tail ? (li.used ? fmaxf(-expm1f(most) - others, 0.0f) : 1.0f) : 0.0f;
  li.total = tail ? fmaxf(sum, 1.0f) : 1.0f;
  // a teacher's log probabilities are rounded numbers: their sum may pass 1
  if (tail && !(sum < 1.0f + 0x1p-8f)) li.flags |= SV_ROW_NAN;
  if (!tail && li.used && !(sum > 0.0f)) li.flags |= SV_ROW_NAN;  // nothing to normalise
  return li;
}
// an entry's gradient; st: the row's statistics
__device__ __forceinline__ float listed_grad(const Entry &e, const List &li, const float4 &st, float k, float w) {
  const float share = ex2_approx((e.x - st.z) * k) * st.w;
  return (share * li.total - expf(e.value - li.ref) * li.inv) * w;
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

// The slice's gradient in full but for the listed elements, by a CTA of THREADS:
// pieces from `piece(g, j, v)` where the gradient's row lies on the 16-byte grid as the logits'
// does, the last groups first; single elements otherwise (those of the logits come
// from memory again: the two rows are different ones then).  coef 0: zeros, whatever
// the row holds.
template <typename T, int THREADS, typename F>
__device__ __forceinline__ void write_grad(const T *row, T *grad, const RowSlice &s, uint32_t rank, float m, float coef, float k,
                                           F piece) {
  constexpr int VEC = RowElem<T>::VEC;
  const bool zero = coef == 0.0f;
  if (rank == 0 && (int)threadIdx.x < s.singles) {
    const int i = single_at<T>(s, threadIdx.x);
    grad[i] = RowElem<T>::store(zero ? 0.0f : grad_of<T>(RowElem<T>::load(row + i), m, coef, k));
  }
  if ((uintptr_t)row % 16 == (uintptr_t)grad % 16) {
    constexpr int kVecs = kGroupVecs<THREADS>;
    uint4 *out = (uint4 *)(grad + s.head);
    for (int g = row_groups<THREADS>(s) - 1; g >= 0; --g) {
      const int v0 = s.v0 + g * kVecs + (int)threadIdx.x;
      uint4 w[kPieces];  // all on their way before the first is stored
#pragma unroll
      for (int j = 0; j < kPieces; ++j)
        if (v0 + j * THREADS < s.v1) w[j] = piece(g, j, v0 + j * THREADS);
#pragma unroll
      for (int j = 0; j < kPieces; ++j)
        if (v0 + j * THREADS < s.v1)
          __stcs(out + v0 + j * THREADS, zero ? make_uint4(0, 0, 0, 0) : grad_piece<T>(w[j], m, coef, k));
    }
  } else {
    const int lo = s.head + s.v0 * VEC, hi = s.head + s.v1 * VEC;
    for (int i = lo + threadIdx.x; i < hi; i += THREADS)
      grad[i] = RowElem<T>::store(zero ? 0.0f : grad_of<T>(RowElem<T>::load(row + i), m, coef, k));
  }
}

// Whether element i of the row is one of the slice's, or of the first CTA's singles.
template <typename T> __device__ __forceinline__ bool in_slice(const RowSlice &s, uint32_t rank, int i) {
  const int v = i - s.head;
  if (v < 0 || v >= s.vecs * RowElem<T>::VEC) return rank == 0;
  return v / RowElem<T>::VEC >= s.v0 && v / RowElem<T>::VEC < s.v1;
}

// A byte for each piece of a slice, its bits the elements; the four of a thread in a
// group are a word.  Sets those of an entry's token; `twice` where it was set before.
struct ListedBits {
  uint32_t singles, twice;
};
template <typename T, int THREADS>
__device__ __forceinline__ void set_bit(uint32_t *bits, ListedBits &l, const RowSlice &s, uint32_t rank, int token) {
  constexpr int VEC = RowElem<T>::VEC;
  if (token < 0 || !in_slice<T>(s, rank, token)) return;
  const int i = token - s.head;
  uint32_t was, bit;
  if (i < 0 || i >= s.vecs * VEC) {
    bit = 1u << (i < 0 ? token : token - s.vecs * VEC);
    was = atomicOr(&l.singles, bit);
  } else {
    const int v = i / VEC - s.v0;
    bit = 1u << (v % kGroupVecs<THREADS> / THREADS * 8 + i % VEC);
    was = atomicOr(&bits[v / kGroupVecs<THREADS> * THREADS + v % THREADS], bit);
  }
  if (was & bit) l.twice = 1;
}
// The unlisted elements of a group's pieces into the sums.
template <typename T, int THREADS>
__device__ __forceinline__ void add_group(RowSums &sums, const unsigned char *ring, int at, uint32_t listed, float k,
                                          unsigned long long k2) {
  constexpr int VEC = RowElem<T>::VEC;
  uint4 w[kPieces];
#pragma unroll
  for (int j = 0; j < kPieces; ++j) w[j] = ring_piece<THREADS>(ring, at, j);
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
}
// A CTA's sums and faults to every CTA of the cluster: the beginning, which arrives
// at the cluster's barrier, and the end, which waits for it.
struct Exchange {
  unsigned long long part[kMaxRowCluster];  // reference and sum of each CTA
  uint32_t flags[kMaxRowCluster];
};
__device__ __forceinline__ void push(Exchange &x, const RowPart &p, uint32_t flags, uint32_t rank, unsigned C) {
  const int lane = threadIdx.x & 31;
  if (threadIdx.x < C) {
    cluster_st_u64(&x.part[rank], lane, (unsigned long long)__float_as_uint(p.l) << 32 | __float_as_uint(p.top));
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(cluster_addr(&x.flags[rank], lane)), "r"(flags) : "memory");
  }
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");
}
__device__ __forceinline__ RowPart pull(const Exchange &x, uint32_t &flags, unsigned C, float k) {
  const int lane = threadIdx.x & 31;
  cluster_wait();
  RowPart p{-INFINITY, 0.0f, 0.0f};
  if (lane < (int)C) {
    p.top = __uint_as_float((uint32_t)x.part[lane]);
    p.l = __uint_as_float((uint32_t)(x.part[lane] >> 32));
  }
  flags = __reduce_or_sync(0xffffffffu, lane < (int)C ? x.flags[lane] : 0u);
  return warp_join(p, k);
}
// What a row comes to, from the unlisted elements' sums and the list.
struct Row {
  float4 st;  // out_stat
  float ref, l, t_rest;
  uint32_t flags;
  bool skip, has_rest;
};
__device__ __forceinline__ Row row_of(const DistillArgs &a, const RowPart &rest, const List &li, uint32_t flags) {
  const float k = a.k;
  Row r;
  r.skip = li.used == 0 && li.flags == 0;
  r.has_rest = rest.top != -INFINITY;
  const float top = fmaxf(rest.top, li.top);
  r.ref = top == -INFINITY ? 0.0f : top;
  const RowPart all = moved(rest, r.ref, k);
  // (a list without a number above -inf has 0, or NaN from the data)
  r.l = all.l + (li.top == -INFINITY ? li.sum : li.sum * ex2_approx((li.top - r.ref) * k));
  r.flags = flags | li.flags;
  if (!(r.l > 0.0f)) r.flags |= SV_ROW_NAN;
  if (r.skip) r.flags = 0;
  r.t_rest = li.rest < kRounding && !(all.l >= r.l * kNoShare) ? 0.0f : li.rest;
  const float coef = r.has_rest ? (all.l / r.l * li.total - r.t_rest) / rest.l : 0.0f;
  r.st = r.skip || r.flags ? make_float4(__uint_as_float(r.flags), 0.0f, 0.0f, 0.0f)
                           : make_float4(r.has_rest ? rest.top : 0.0f, coef, r.ref, 1.0f / r.l);
  return r;
}
// A list warp's part of the loss; the first warp's has the rest's term.
__device__ __forceinline__ float loss_part(const DistillArgs &a, const Row &r, const RowPart &rest, const List &li,
                                           const Entry &e) {
  // ln s_v = (x_v - ref) / T - ln l, of the rest (rest.top - ref) / T + ln(rest.l / l)
  const float log_l = logf(r.l), t = expf(e.value - li.ref) * li.inv;
  float loss = e.token >= 0 && t > 0.0f ? t * (e.value - li.shift - ((e.x - r.ref) / a.temperature - log_l)) : 0.0f;
#pragma unroll
  for (int o = 16; o; o >>= 1) loss += __shfl_xor_sync(0xffffffffu, loss, o);
  if (threadIdx.x < 32 && r.t_rest > 0.0f)
    loss += r.t_rest *
            (logf(r.t_rest) - (r.has_rest ? (rest.top - r.ref) / a.temperature + logf(rest.l) - log_l : -INFINITY));
  return loss;
}
__device__ __forceinline__ void put_row(const DistillArgs &a, size_t r, const Row &row, const float *losses) {
  float loss = 0.0f;
#pragma unroll
  for (int i = 0; i < kListWarps; ++i) loss += losses[i];
  if (a.stat) a.stat[r] = row.st;
  a.loss[r] = row.skip ? 0.0f : row.flags ? __int_as_float(0x7fffffff) : loss;
  a.status[r] = row.flags;
}

// THREADS: the CTA's, of which as many stay on an SM as registers allow.
template <typename T, bool GRAD, int THREADS>
__global__ void __launch_bounds__(THREADS, THREADS == 128 ? 8 : 3) distill_kernel(DistillArgs a, unsigned C) {
  grid_dep_sync();
  static_assert(kMaxList <= THREADS, "an entry to a thread");
  constexpr int kWarps = THREADS / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const size_t r = blockIdx.x / C;
  const uint32_t rank = C > 1 ? cluster_rank() : 0;
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ ListPart s_list[kListWarps];
  __shared__ RowPart s_part[kWarps];
  __shared__ Exchange s_all;
  __shared__ ListedBits s_bits;
  __shared__ float s_loss[kListWarps];
  if (C > 1) cluster_arrive_relaxed();
  const T *row = (const T *)a.logits + (int64_t)r * a.row_stride;
  const RowSlice s = row_slice(row, a.V, rank, C);
  const int groups = row_groups<THREADS>(s);
  uint32_t *bits = (uint32_t *)(smem + a.ring);

#pragma unroll
  for (int g = 0; g < kRing - 1; ++g) {
    if (g < groups) load_group<THREADS>(row, s, g, g, smem);
    group_commit();
  }
  const Entry e = read_entry(a, r, row);
  const bool has_single = rank == 0 && (int)threadIdx.x < s.singles;
  const float single_x = has_single ? RowElem<T>::load(row + single_at<T>(s, threadIdx.x)) : -INFINITY;
  for (int g = 0; g < groups; ++g) bits[g * THREADS + threadIdx.x] = 0;
  if (threadIdx.x == 0) s_bits = ListedBits{0, 0};
  __syncthreads();
  set_bit<T, THREADS>(bits, s_bits, s, rank, e.token);
  __syncthreads();
  const float k = a.k;
  const unsigned long long k2 = f2_splat(k);
  RowSums sums = row_sums();
  if (has_single && !(s_bits.singles >> threadIdx.x & 1)) add_single<false>(sums, single_x, k);
  int slot = 0, slot_load = kRing - 1;
  for (int g = 0; g < groups; ++g) {
    if (g + kRing - 1 < groups) load_group<THREADS>(row, s, g + kRing - 1, slot_load, smem);
    group_commit();
    group_wait<kRing - 1>();
    add_group<T, THREADS>(sums, smem, slot, bits[g * THREADS + threadIdx.x], k, k2);
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
  RowPart rest = warp_join(lane < kWarps ? s_part[lane] : RowPart{-INFINITY, 0.0f, 0.0f}, k);
  uint32_t flags = s_bits.twice ? SV_ROW_BAD_TOKEN : 0u;
  if (C > 1) {
    cluster_wait();
    push(s_all, rest, flags, rank, C);
  }
  const List li = list_of(s_list, a.tail, k);
  if (C > 1) rest = pull(s_all, flags, C, k);
  const Row out = row_of(a, rest, li, flags);
  if (rank == 0 && warp < kListWarps) {
    const float loss = loss_part(a, out, rest, li, e);
    if (lane == 0) s_loss[warp] = loss;
  }
  if constexpr (GRAD) {
    const float w = (a.weight ? a.weight[r] : 1.0f) / a.temperature;
    T *grad = (T *)a.grad + (int64_t)r * a.grad_stride;
    // a row without a gradient has 0 for 1 / l
    const float c = out.st.w == 0.0f ? 0.0f : out.st.y * w;
    // (the logits may be the gradient's own place: a piece is read, by whoever writes
    // there, before it is written)
    write_grad<T, THREADS>(row, grad, s, rank, out.st.x, c, k, [&](int g, int j, int v) {
      return g >= groups - kRing ? ring_piece<THREADS>(smem, g % kRing, j) : ((const uint4 *)(row + s.head))[v];
    });
    __syncthreads();
    if (out.st.w != 0.0f && e.token >= 0 && in_slice<T>(s, rank, e.token))
      grad[e.token] = RowElem<T>::store(listed_grad(e, li, out.st, k, w));
  } else {
    __syncthreads();
  }
  if (rank == 0 && threadIdx.x == 0) put_row(a, r, out, s_loss);
}

// The gradient from a forward pass's statistics: CTA `rank` of C of a row.  It streams
// and no more, so that smaller CTAs, whose beginnings and ends lie apart, do best (2048
// rows of V = 128256 bf16: 163 us, 6.46 TB/s, by 128 threads, 171 by 256; 777 of 40001
// fp32: 44 and 47).
constexpr int kGradThreads = 128;
static_assert(kMaxList <= kGradThreads, "an entry to a thread");
template <typename T>
__global__ void __launch_bounds__(kGradThreads, 8) distill_grad_kernel(DistillArgs a, unsigned C) {
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
  const bool skip = li.used == 0 && li.flags == 0;  // as in the forward pass
  const uint32_t flags = skip ? 0u : li.flags | (st.w == 0.0f ? __float_as_uint(st.x) : 0u);
  const bool none = st.w == 0.0f || flags || skip;
  write_grad<T, kGradThreads>(row, grad, s, rank, st.x, none ? 0.0f : st.y * w, a.k,
                [&](int, int, int v) { return ((const uint4 *)(row + s.head))[v]; });
  __syncthreads();
  if (!none && e.token >= 0 && in_slice<T>(s, rank, e.token))
    grad[e.token] = RowElem<T>::store(listed_grad(e, li, st, a.k, w));
  if (rank == 0 && threadIdx.x == 0) a.status[r] = flags;
}

template <typename T, bool GRAD, int THREADS> cudaError_t launch_loss(DistillArgs a, unsigned C, cudaStream_t st) {
  // of a slice: its groups, as many of them as the ring has at once, and a bit for each
  // element in whole groups
  const size_t row = (size_t)a.V * sizeof(T);
  auto groups_of = [](size_t bytes, unsigned c) {
    return ((bytes / 16 + c - 1) / c + kGroupVecs<THREADS> - 1) / kGroupVecs<THREADS>;
  };
  const size_t groups = groups_of(row, C);
  a.ring = kGroupBytes<THREADS> * (int)(groups < (size_t)kRing ? groups : (size_t)kRing);
  static thread_local int set_dev = -1;
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev != set_dev) {  // as much as the longest rows take
    const size_t most = groups_of((size_t)SV_MAX_VOCAB * sizeof(T), kMaxRowCluster) * kGroupVecs<THREADS>;
    const cudaError_t e = cudaFuncSetAttribute(distill_kernel<T, GRAD, THREADS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               kRing * kGroupBytes<THREADS> + (int)most);
    if (e != cudaSuccess) return e;
    set_dev = dev;
  }
  return launch_pdl_cluster(distill_kernel<T, GRAD, THREADS>, dim3((unsigned)a.R * C), dim3(THREADS), C,
                            a.ring + groups * kGroupVecs<THREADS>, st, a, C);
}
template <typename T, bool GRAD> cudaError_t launch_loss(const DistillArgs &a, cudaStream_t st) {
  // CTAs to a row: with a gradient about 80 KB of it to each (2048 rows of 128256 bf16 by
  // 1 to 5 CTAs each: 226, 198, 192, 203 and 230 us; 1500 of 75000 fp32: 212, 179, 163,
  // 154 and 164), less of few rows, and more where that many run at once (200 rows by 2 and
  // 3: 24 and 29 us).  CTAs of 128 threads for short rows, whose time is the way
  // there and back, of which more are under way (4000 rows of 1000 fp32, loss: 18.5 us,
  // by 256 threads 31.9; with the gradient 21 and 36; of 32000 bf16 48 and 59, with the
  // gradient 98 and 96; of 50256 fp32 128 and 121, with the gradient 339 and 278)
  const size_t row = (size_t)a.V * sizeof(T);
  const bool small = row <= (GRAD ? 32768 : 131072);
  unsigned C = 1;
  if (GRAD) {
    const size_t slices = (row + 40960) / 81920, most = (row + 16383) / 16384, once = 456 / (size_t)a.R;
    size_t c = once < most ? once : most;
    if (c * 131072 < row) c = slices;
    C = c < 1 ? 1u : c > kMaxRowCluster ? kMaxRowCluster : (unsigned)c;
  } else {
    C = row_ctas(row, a.R, small ? 456 : 304);
  }
  while (C * 2 <= kMaxRowCluster && row > C * (size_t)262144) C *= 2;  // a slice's bits: 16 KB, of the longest rows 128
  return small ? launch_loss<T, GRAD, 128>(a, C, st) : launch_loss<T, GRAD, 256>(a, C, st);
}
template <typename T> cudaError_t launch_grad(const DistillArgs &a, cudaStream_t st) {
  // 64 KB of a row to a CTA, less of few rows: as many CTAs as run at once (50 rows of
  // 128256 bf16: 6.7 us, with 64 KB 10.5; 5 rows of 32000: 2.8 and 5.9)
  const size_t row = (size_t)a.V * sizeof(T);
  auto ctas = [&](size_t bytes) { return (row + bytes - 1) / bytes; };
  size_t bytes = 65536;
  while (bytes > 8192 && ctas(bytes / 2) * a.R <= 1216) bytes /= 2;
  const unsigned C = (unsigned)ctas(bytes);
  return launch_pdl(distill_grad_kernel<T>, dim3((unsigned)a.R * C), dim3(kGradThreads), 0, st, a, C);
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
