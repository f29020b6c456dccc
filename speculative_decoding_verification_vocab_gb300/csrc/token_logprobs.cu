// token_logprobs.cu -- log probabilities of given tokens, the entropy and the
// most likely alternatives of vocabulary rows (sm_103a).
//
// What a round answers with beside its tokens, and what a teacher leaves for its
// draft.  With z = x / T, m near max z and l = sum exp(z - m), in one pass over
// a row: log p(t) = z_t - m - ln l, H = ln l - sum exp(z - m) (z - m) / l, and
// the K largest x, equal ones in ascending token id.
//
// Bound: each row asked for is read once (V elements; 5 operations on each), and
// some 100 bytes are written: memory.  A cluster of C CTAs takes a row, each
// streaming its slice through shared memory; every CTA ends with its sums and
// its K best, stores them to the first CTA, which joins them.  One launch, no
// workspace.
//
// The K best of a slice cost the pass a maximum: a thread keeps, in shared memory,
// the largest of each run of its elements (32 and more; 8 runs), rounded up to 16
// bits.  In the end the threads' maxima give a value tau that K elements are known
// to reach (below), the runs that reach it (K and a few) are read again, from L2,
// and their elements of at least tau, K and some, are sorted.  A row of which too
// many elements reach tau (constant ones, say) goes through a list that is cut
// back to the K best whenever it is full.  (With that list filled in the pass, 16 KB
// by 16 KB between barriers, 4096 rows of V = 128256 bf16 took 378 us at K = 20 and
// 676 at K = 128.)
//
// 4096 rows of V = 128256 bf16: 155 us without alternatives (6.78 TB/s, all that memory
// gives), 191 at K = 20 (0.81), 266 at K = 128: behind its row a CTA has another 16000
// clocks of barriers and ways to L2, a third of its time, in which three others of the
// SM stream.  1000 rows of 50257 fp32, K = 64: 51 us, two waves of CTAs.  Five CTAs to
// an SM with two groups in the ring take 198 and 54, CTAs of 128 threads 191 and 62.
#include <math.h>

#include "vocab_rows.cuh"

namespace sv {
namespace {

typedef unsigned long long u64;
constexpr int kMaxTop = 128;
constexpr int kMaxima = 256;   // of a CTA's elements, one or two to a thread: they give the threshold
constexpr int kRing = 3;       // groups: one in work, two on their way
constexpr int kRuns = 8;       // of a thread's elements
constexpr int kList = 2048;    // keys, in the ring's place; a power of two
constexpr int kSlowList = 512; // of them, where the list is cut back: at least kMaxTop + THREADS
template <int THREADS>
constexpr bool kFits = kList * 8 + kRuns * THREADS * 2 <= kRing * kGroupBytes<THREADS> && kSlowList >= kMaxTop + THREADS;
static_assert(kFits<128> && kFits<256> && kMaxTop <= kMaxima, "lists");

struct LogArgs {
  const void *logits;
  int64_t seq_stride, row_stride;
  const int32_t *rows, *tokens;
  int T, P, V, K;
  float temperature, k;  // k = log2(e) / T
  float *logprob, *entropy;
  int32_t *top_token;
  float *top_logprob;
  uint32_t *status;
};

// Numbers in the order of the floats (-0 as +0), and back
__device__ __forceinline__ uint32_t order_of(float x) {
  const uint32_t b = __float_as_uint(__fadd_rn(x, 0.0f));
  return b >> 31 ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t order) {
  return __uint_as_float(order >> 31 ? order & 0x7fffffffu : ~order);
}
// Orders by value, then by the lower index; 0 is below every element's.
__device__ __forceinline__ u64 key_of(float x, int index) { return (u64)order_of(x) << 32 | (uint32_t)~index; }
__device__ __forceinline__ float value_of(u64 key) { return value_of((uint32_t)(key >> 32)); }
__device__ __forceinline__ int index_of(u64 key) { return (int)~(uint32_t)key; }

// The min(n, K) largest of keys[0, n), all different, in descending order at the
// front; keys has room for the next power of two.  Every thread of the CTA calls
// it with the keys visible, and finds them in place.
template <int THREADS> __device__ void keep_best(u64 *keys, int n, int K) {
  constexpr int M = kMaxima / THREADS;
  if (n <= kMaxima) {  // a thread counts what is above its keys
    const int i = threadIdx.x;
    u64 mine[M];
    int above[M];
#pragma unroll
    for (int m = 0; m < M; ++m) {
      mine[m] = i + m * THREADS < n ? keys[i + m * THREADS] : 0;
      above[m] = 0;
    }
    const ulonglong2 *two = (const ulonglong2 *)keys;
    auto count = [&](int of) {
#pragma unroll 4
      for (int j = 0; j < n / 2; ++j) {
        const ulonglong2 o = two[j];
#pragma unroll
        for (int m = 0; m < M; ++m)
          if (m < of) above[m] += (o.x > mine[m]) + (o.y > mine[m]);
      }
      if (n & 1) {
#pragma unroll
        for (int m = 0; m < M; ++m)
          if (m < of) above[m] += keys[n - 1] > mine[m];
      }
    };
    if (n > THREADS)
      count(M);
    else if ((i & ~31) < n)
      count(1);
    __syncthreads();
#pragma unroll
    for (int m = 0; m < M; ++m)
      if (i + m * THREADS < n && above[m] < K) keys[above[m]] = mine[m];
    __syncthreads();
    return;
  }
  int size = 2 * kMaxima;
  while (size < n) size *= 2;
  for (int i = n + threadIdx.x; i < size; i += THREADS) keys[i] = 0;
  for (int run = 2; run <= size; run *= 2)
    for (int step = run / 2; step; step /= 2) {
      __syncthreads();
      for (int i = threadIdx.x; i < size / 2; i += THREADS) {
        const int lo = 2 * i - (i & (step - 1)), hi = lo + step;
        const u64 a = keys[lo], b = keys[hi];
        if ((a < b) == ((lo & run) == 0)) {  // descending where the run's bit is clear
          keys[lo] = b;
          keys[hi] = a;
        }
      }
    }
  __syncthreads();
}

// The digit of the K-th largest of the numbers counted in bins[256], and how many of K
// are left for it (-1: fewer than K are counted); for every warp at once.
__device__ __forceinline__ int digit_of(const uint32_t *bins, int &K) {
  const unsigned FULL = 0xffffffffu;
  const int lane = threadIdx.x & 31;
  const uint4 lo = ((const uint4 *)bins)[2 * lane], hi = ((const uint4 *)bins)[2 * lane + 1];
  const int n[8] = {(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
  int own = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) own += n[i];
  int from = own;  // of this lane's bins and those above
#pragma unroll
  for (int o = 1; o < 32; o *= 2) {
    const int x = __shfl_down_sync(FULL, from, o);
    if (lane + o < 32) from += x;
  }
  const unsigned reach = __ballot_sync(FULL, from >= K);
  if (!reach) return -1;
  const int at = 31 - __clz(reach);
  int left = K - (from - own), digit = 8 * lane + 7;
#pragma unroll
  for (int i = 7; i > 0; --i)
    if (digit == 8 * lane + i && left > n[i]) {
      left -= n[i];
      --digit;
    }
  K = __shfl_sync(FULL, left, at);
  return __shfl_sync(FULL, digit, at);
}

// x rounded up to the upper 16 bits of a float
__device__ __forceinline__ uint16_t up16(float x) {
  const uint32_t b = __float_as_uint(x);
  return (uint16_t)((b >> 31 ? b : b + 0xffffu) >> 16);
}
// the slice's piece v
template <typename T> __device__ __forceinline__ uint4 piece_at(const T *row, const RowSlice &s, int v) {
  return __ldg((const uint4 *)(row + s.head) + v);
}

// The K best of a slice by a list that is cut back as it fills, a group of pieces
// after the other.  Every thread of the CTA calls it and finds the list's first
// min(K, elements) in order; returns their number.  s_n: a counter.
template <typename T, int THREADS>
__device__ __noinline__ int best_by_list(const T *row, const RowSlice &s, uint32_t rank, u64 *list, int K, int *s_n) {
  constexpr int VEC = RowElem<T>::VEC;
  float tau = -INFINITY;  // what an element has to reach, and its key to exceed
  u64 tau_key = 0;
  __syncthreads();
  if (threadIdx.x == 0) *s_n = 0;
  __syncthreads();
  auto offer = [&](float x, int index) {
    if (x >= tau && x > -INFINITY) {
      const u64 key = key_of(x, index);
      if (key > tau_key) {
        const int at = atomicAdd(s_n, 1);
        if (at < kSlowList) list[at] = key;
      }
    }
  };
  // after a barrier behind the last offer
  auto cut = [&](int n) {
    keep_best<THREADS>(list, n, K);
    if (n >= K) {
      tau_key = list[K - 1];
      tau = value_of(tau_key);
    }
    if (threadIdx.x == 0) *s_n = min(n, K);
    __syncthreads();
  };
  if (rank == 0 && (int)threadIdx.x < s.singles) {
    const int i = single_at<T>(s, threadIdx.x);
    offer(RowElem<T>::load(row + i), i);
  }
  __syncthreads();
  const int groups = row_groups<THREADS>(s);
  for (int g = 0; g < groups; ++g) {
    auto piece = [&](int j) { return s.v0 + g * kGroupVecs<THREADS> + j * THREADS + (int)threadIdx.x; };
    const int before = *s_n;  // settled by the barriers that ended the last group
    float most[kPieces], top = -INFINITY;
#pragma unroll
    for (int j = 0; j < kPieces; ++j) {
      most[j] = piece(j) < s.v1 ? RowElem<T>::most(piece_at(row, s, piece(j))) : -INFINITY;
      top = fmaxf(top, most[j]);
    }
    const bool some = top >= tau && top > -INFINITY;
    // (the votes' barrier stands behind every thread's look at the counter)
    if (!__syncthreads_or(some)) continue;
    if (some) {
      for (int j = 0; j < kPieces; ++j) {
        if (most[j] < tau || most[j] == -INFINITY) continue;
        float x[VEC];
        RowElem<T>::unpack(piece_at(row, s, piece(j)), x);
#pragma unroll
        for (int i = 0; i < VEC; ++i) offer(x[i], s.head + piece(j) * VEC + i);
      }
    }
    __syncthreads();
    int n = *s_n;
    __syncthreads();
    if (n > kSlowList) {  // again, an element of each thread at a time
      if (threadIdx.x == 0) *s_n = before;
      __syncthreads();
      n = before;
      for (int j = 0; j < kPieces; ++j) {
        for (int i = 0; i < VEC; ++i) {
          if (n > kSlowList - THREADS) cut(n);
          if (piece(j) < s.v1) {
            const int at = s.head + piece(j) * VEC + i;
            offer(RowElem<T>::load(row + at), at);
          }
          __syncthreads();
          n = *s_n;
          __syncthreads();
        }
      }
    }
    if (n >= 2 * K + 32) cut(n);
  }
  const int n = *s_n;
  keep_best<THREADS>(list, n, K);
  return min(n, K);
}

// THREADS: the CTA's, of which as many stay on an SM as registers allow.
template <typename T, bool TOP, int THREADS>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) token_logprobs_kernel(LogArgs a, unsigned C) {
  grid_dep_sync();
  constexpr int VEC = RowElem<T>::VEC;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const size_t item = blockIdx.x / C;
  const uint32_t rank = C > 1 ? cluster_rank() : 0;
  extern __shared__ __align__(16) unsigned char smem[];
  u64 *list = (u64 *)smem;                                         // [kList], when the ring is free
  uint16_t *hits = (uint16_t *)(list + kList);                     // [kRuns THREADS], as the list
  uint16_t *runs = (uint16_t *)(smem + kRing * kGroupBytes<THREADS>);  // [kRuns][THREADS]
  u64 *all = (u64 *)(smem + kRing * kGroupBytes<THREADS> + (TOP ? kRuns * THREADS * 2 : 0));  // [C][K], the first CTA's
  __shared__ RowPart s_part[THREADS / 32];
  __shared__ RowPart s_all[kMaxRowCluster];
  __shared__ int s_n, s_hits;
  __shared__ __align__(16) uint32_t s_bins[2][256];

  const int b = (int)(item / a.P);
  const int token = a.tokens ? a.tokens[item] : 0;
  const int r = a.rows ? a.rows[item] : (int)(item % a.P);
  const bool skip = (a.tokens && token == -1) || (a.rows && r == -1);
  if (skip || r < 0 || r >= a.T) {  // the same in every CTA of the cluster
    if (rank == 0) {
      const float nan = __int_as_float(0x7fffffff);
      if (threadIdx.x == 0) {
        if (a.logprob) a.logprob[item] = skip ? 0.0f : nan;
        a.entropy[item] = skip ? 0.0f : nan;
        a.status[item] = skip ? 0u : SV_ROW_BAD_ROW;
      }
      for (int i = threadIdx.x; i < a.K; i += THREADS) {
        a.top_token[item * a.K + i] = -1;
        a.top_logprob[item * a.K + i] = skip ? -INFINITY : nan;
      }
    }
    return;
  }
  // every CTA has started before another stores to its shared memory
  if (C > 1) cluster_arrive_relaxed();
  const T *row = (const T *)a.logits + b * a.seq_stride + r * a.row_stride;
  const RowSlice s = row_slice(row, a.V, rank, C);
  const int groups = row_groups<THREADS>(s);
#pragma unroll
  for (int g = 0; g < kRing - 1; ++g) {
    if (g < groups) load_group<THREADS>(row, s, g, g, smem);
    group_commit();
  }
  const bool known = token >= 0 && token < a.V;
  const float given = rank == 0 && a.tokens && known ? RowElem<T>::load(row + token) : 0.0f;
  const float k = a.k;
  const unsigned long long k2 = f2_splat(k);
  RowSums sums = row_sums();
  const bool has_single = rank == 0 && (int)threadIdx.x < s.singles;
  const int single = has_single ? single_at<T>(s, threadIdx.x) : 0;
  const float single_x = has_single ? RowElem<T>::load(row + single) : -INFINITY;
  if (has_single) add_single<true>(sums, single_x, k);
  if (TOP) {
    if (threadIdx.x == 0) s_n = s_hits = 0;
    for (int i = threadIdx.x; i < 512; i += THREADS) s_bins[0][i] = 0;
    __syncthreads();
  }

  // run i of a thread: its groups [i per, (i + 1) per)
  const int per = (groups + kRuns - 1) / kRuns;
  constexpr int M = kMaxima / THREADS;
  float tops[M];  // of the runs i with i % M, the first with the single
#pragma unroll
  for (int m = 0; m < M; ++m) tops[m] = m ? -INFINITY : single_x;
  int run = 0, slot = 0, slot_load = kRing - 1;
  for (int g = 0; g < groups; ++run) {
    float run_top = -INFINITY;
    for (const int end = min(g + per, groups); g < end; ++g) {
      if (g + kRing - 1 < groups) load_group<THREADS>(row, s, g + kRing - 1, slot_load, smem);
      group_commit();
      group_wait<kRing - 1>();
      uint4 w[kPieces];
#pragma unroll
      for (int j = 0; j < kPieces; ++j) w[j] = ring_piece<THREADS>(smem, slot, j);
      const float top = RowElem<T>::most4(w);
      if (top > sums.lim) raise<true>(sums, top, k);
#pragma unroll
      for (int j = 0; j < kPieces; ++j) add_piece<T, true>(sums, w[j], k2);
      if (TOP) run_top = fmaxf(run_top, top);
      slot = slot + 1 == kRing ? 0 : slot + 1;
      slot_load = slot_load + 1 == kRing ? 0 : slot_load + 1;
    }
    if (TOP) {
      runs[run * THREADS + threadIdx.x] = up16(run_top);
      if (M == 1 || run % 2 == 0)
        tops[0] = fmaxf(tops[0], run_top);
      else
        tops[M - 1] = fmaxf(tops[M - 1], run_top);
    }
  }
  group_wait<0>();

  // the upper 16 bits of the thread's maxima, as ordered numbers (0: none above -inf)
  uint32_t top_key[M];
  float thread_top = -INFINITY;
#pragma unroll
  for (int m = 0; m < M; ++m) {
    thread_top = fmaxf(thread_top, tops[m]);
    top_key[m] = TOP && tops[m] > -INFINITY ? order_of(tops[m]) >> 16 : 0u;
    if (top_key[m]) atomicAdd(&s_bins[0][top_key[m] >> 8], 1u);
  }
  const RowPart mine = warp_join(part_of(sums), k);
  if (lane == 0) s_part[warp] = mine;
  __syncthreads();  // the ring is free, too
  int n = 0;
  if (TOP) {
    // tau: the K-th largest of the CTA's maxima, to 16 bits (none: all above -inf), a
    // byte of it at a time.  K elements reach it, and a few more: in any order 1.04 K of
    // 128256 at K = 20, 1.4 K at 128.
    int left = a.K;
    const int high = digit_of(s_bins[0], left);
#pragma unroll
    for (int m = 0; m < M; ++m)
      if (high >= 0 && (int)(top_key[m] >> 8) == high) atomicAdd(&s_bins[1][top_key[m] & 255], 1u);
    __syncthreads();
    const float tau = high < 0 ? -INFINITY : value_of((uint32_t)(high << 8 | digit_of(s_bins[1], left)) << 16);
    auto offer = [&](float x, int index) {
      if (x >= tau && x > -INFINITY) {
        const int at = atomicAdd(&s_n, 1);
        if (at < kList) list[at] = key_of(x, index);
      }
    };
    if (has_single) offer(single_x, single);
    // the runs that reach it, then their pieces over all threads: one way to L2
    if (thread_top >= tau && thread_top > -INFINITY) {
#pragma unroll
      for (int i = 0; i < kRuns; ++i) {
        const float top = __uint_as_float((uint32_t)runs[i * THREADS + threadIdx.x] << 16);
        if (i < run && top >= tau) hits[atomicAdd(&s_hits, 1)] = (uint16_t)(i * THREADS + threadIdx.x);
      }
    }
    __syncthreads();
    const int of_run = per * kPieces, pieces = s_hits * of_run;
    for (int i = threadIdx.x; i < pieces; i += THREADS) {
      const int hit = hits[i / of_run], q = i % of_run;
      const int g = hit / THREADS * per + q / kPieces;
      const int v = s.v0 + g * kGroupVecs<THREADS> + q % kPieces * THREADS + hit % THREADS;
      if (g >= groups || v >= s.v1) continue;
      const uint4 w = piece_at(row, s, v);
      const float m = RowElem<T>::most(w);
      if (!(m >= tau) || m == -INFINITY) continue;
      float x[VEC];
      RowElem<T>::unpack(w, x);
#pragma unroll
      for (int e = 0; e < VEC; ++e) offer(x[e], s.head + v * VEC + e);
    }
    __syncthreads();
    n = s_n;
    if (n > kList) {
      n = best_by_list<T, THREADS>(row, s, rank, list, a.K, &s_n);
    } else {
      keep_best<THREADS>(list, n, a.K);
      n = min(n, a.K);
    }
  }
  auto join = [&](const RowPart *parts, int count) {
    return warp_join(lane < count ? parts[lane] : RowPart{-INFINITY, 0.0f, 0.0f}, k);
  };
  RowPart sum = join(s_part, THREADS / 32);
  if (C > 1) {
    cluster_wait();
    if (threadIdx.x == 0) {
      const u64 two = (u64)__float_as_uint(sum.l) << 32 | __float_as_uint(sum.top);
      const uint32_t at = cluster_addr(&s_all[rank], 0);
      asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(at), "r"((uint32_t)two) : "memory");
      asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(at + 4), "r"((uint32_t)(two >> 32)) : "memory");
      asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(at + 8), "r"(__float_as_uint(sum.s)) : "memory");
    }
    if (TOP)
      for (int i = threadIdx.x; i < a.K; i += THREADS) cluster_st_u64(all + rank * a.K + i, 0, i < n ? list[i] : 0);
    cluster_sync();
    if (rank != 0) return;
    sum = join(s_all, (int)C);
    if (TOP) {
      // lists that are not full hold zeros behind their keys; where the keys are
      // fewer than K in all, so does the first list behind their number
      keep_best<THREADS>(all, (int)C * a.K, a.K);
      list = all;
      n = a.K;
    }
  }
  // a sum that is NaN (a NaN or +inf among the elements) or 0 (all -inf)
  const bool bad = !(sum.l > 0.0f);
  const float nan = __int_as_float(0x7fffffff);
  const float log_l = logf(sum.l);
  auto logprob = [&](float x) { return (x - sum.top) / a.temperature - log_l; };
  if (threadIdx.x == 0) {
    uint32_t flags = bad ? SV_ROW_NAN : 0u;
    if (a.logprob) {
      if (!known) flags |= SV_ROW_BAD_TOKEN;
      a.logprob[item] = bad || !known ? nan : logprob(given);
    }
    // s is in log2 units
    a.entropy[item] = bad ? nan : fmaxf(log_l - sum.s / sum.l * 0.69314718055994531f, 0.0f);
    a.status[item] = flags;
  }
  if (TOP) {
    for (int i = threadIdx.x; i < a.K; i += THREADS) {
      const u64 key = i < n ? list[i] : 0;
      a.top_token[item * a.K + i] = bad || !key ? -1 : index_of(key);
      a.top_logprob[item * a.K + i] = bad ? nan : key ? logprob(value_of(key)) : -INFINITY;
    }
  }
}

template <typename T, bool TOP, int THREADS>
cudaError_t launch(const LogArgs &a, unsigned items, unsigned C, cudaStream_t st) {
  // dynamic memory beyond 48 KB has to be asked for, once for each device
  size_t keys = 0;
  if (TOP && C > 1) {
    keys = ((size_t)C * a.K + 1) / 2 * 2;
    if (keys > (size_t)kMaxima) {  // more than that keep_best sorts in a power of two
      keys = 2 * kMaxima;
      while (keys < (size_t)C * a.K) keys *= 2;
    }
  }
  const size_t smem = (size_t)kRing * kGroupBytes<THREADS> + (TOP ? kRuns * THREADS * 2 : 0) + keys * 8;
  static thread_local int set_dev = -1;
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev != set_dev) {
    const cudaError_t e = cudaFuncSetAttribute(token_logprobs_kernel<T, TOP, THREADS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               kRing * kGroupBytes<THREADS> + kRuns * THREADS * 2 + (int)kMaxRowCluster * kMaxTop * 8);
    if (e != cudaSuccess) return e;
    set_dev = dev;
  }
  return launch_pdl_cluster(token_logprobs_kernel<T, TOP, THREADS>, dim3(items * C), dim3(THREADS), C, smem, st, a, C);
}
// CTAs of 128 threads where rows are short, or the few best are asked for: what a CTA
// does behind its row lies apart from more others' (4000 rows, K = 20: V = 8192 bf16 35
// us, by 256 threads 54; 50257 bf16 86 and 105; 50256 fp32 149 and 146; K = 5: 128256
// bf16 171 and 186; K = 0: 50257 bf16 68 and 74, 128256 162 and 153).  Of many best a
// thread's share of the elements that reach the threshold is too large (K = 128, 50256
// fp32: 288 and 213).
bool small_ctas(size_t row_bytes, int K) { return K <= 32 && row_bytes <= (K > 0 && K <= 8 ? 262144 : 131072); }
template <typename T> cudaError_t launch(const LogArgs &a, unsigned items, cudaStream_t st) {
  const size_t row = (size_t)a.V * sizeof(T);
  const bool small = small_ctas(row, a.K);
  const unsigned C = row_ctas(row, items, small ? 456 : 304);
  if (small) return a.K ? launch<T, true, 128>(a, items, C, st) : launch<T, false, 128>(a, items, C, st);
  return a.K ? launch<T, true, 256>(a, items, C, st) : launch<T, false, 256>(a, items, C, st);
}

}  // namespace
}  // namespace sv

using namespace sv;

extern "C" sv_status sv_token_logprobs(const void *logits, int64_t seq_stride, int64_t row_stride,
                                       sv_dtype dt, const int32_t *rows, const int32_t *tokens,
                                       int B, int T, int P, int V, int K, float temperature,
                                       float *out_logprob, float *out_entropy,
                                       int32_t *out_top_token, float *out_top_logprob,
                                       uint32_t *out_status, void *stream) {
  if (B < 0 || T < 1 || P < 0 || V < 1 || K < 0)
    return set_error(SV_ERR_INVALID_ARG, "need B >= 0, T >= 1, P >= 0, V >= 1, K >= 0");
  if (dt != SV_F32 && dt != SV_BF16 && dt != SV_F16)
    return set_error(SV_ERR_INVALID_ARG, "unknown dtype %d", (int)dt);
  if (!rows && P > T) return set_error(SV_ERR_INVALID_ARG, "P > T without rows");
  if (K > V) return set_error(SV_ERR_INVALID_ARG, "K > V");
  if (K > kMaxTop) return set_error(SV_ERR_UNSUPPORTED, "K > %d", kMaxTop);
  if (V > SV_MAX_VOCAB) return set_error(SV_ERR_UNSUPPORTED, "V > %d", SV_MAX_VOCAB);
  if (!(temperature > 0.0f) || !isfinite(temperature) || !isfinite(kLog2eF / temperature) ||
      !(kLog2eF / temperature > 0.0f))
    return set_error(SV_ERR_INVALID_ARG, "temperature must be > 0 and finite, its inverse too");
  if ((long long)B * P > (1LL << 27)) return set_error(SV_ERR_UNSUPPORTED, "B P > 2^27");
  const int64_t most = INT64_MAX / 16;  // of any offset, in elements
  if (seq_stride < 0 || row_stride < 0 || (B > 0 && seq_stride > most / B) || row_stride > most / T)
    return set_error(SV_ERR_INVALID_ARG, "negative or too large stride");
  if (B == 0 || P == 0) return SV_OK;
  if (!logits || !out_entropy || !out_status || (tokens && !out_logprob) || (K > 0 && (!out_top_token || !out_top_logprob)))
    return set_error(SV_ERR_INVALID_ARG, "null pointer");
  if (!tokens) out_logprob = nullptr;
  if (K == 0) {
    out_top_token = nullptr;
    out_top_logprob = nullptr;
  }
  const size_t es = dt == SV_F32 ? 4 : 2;
  if ((uintptr_t)logits % es || (uintptr_t)rows % 4 || (uintptr_t)tokens % 4 || (uintptr_t)out_logprob % 4 ||
      (uintptr_t)out_entropy % 4 || (uintptr_t)out_top_token % 4 || (uintptr_t)out_top_logprob % 4 ||
      (uintptr_t)out_status % 4)
    return set_error(SV_ERR_INVALID_ARG, "misaligned pointer");
  sv_status s;
  if ((s = map_arg(logits, "logits")) != SV_OK || (s = map_arg(rows, "rows")) != SV_OK ||
      (s = map_arg(tokens, "tokens")) != SV_OK || (s = map_arg(out_logprob, "out_logprob")) != SV_OK ||
      (s = map_arg(out_entropy, "out_entropy")) != SV_OK ||
      (s = map_arg(out_top_token, "out_top_token")) != SV_OK ||
      (s = map_arg(out_top_logprob, "out_top_logprob")) != SV_OK ||
      (s = map_arg(out_status, "out_status")) != SV_OK)
    return s;
  LogArgs a;
  a.logits = logits;
  a.seq_stride = seq_stride;
  a.row_stride = row_stride;
  a.rows = rows;
  a.tokens = tokens;
  a.T = T;
  a.P = P;
  a.V = V;
  a.K = K;
  a.temperature = temperature;
  a.k = kLog2eF / temperature;
  a.logprob = out_logprob;
  a.entropy = out_entropy;
  a.top_token = out_top_token;
  a.top_logprob = out_top_logprob;
  a.status = out_status;
  cudaStream_t st = (cudaStream_t)stream;
  LaunchScope ls("token_logprobs", st);
  const unsigned items = (unsigned)(B * P);
  return check_launch("token_logprobs", dt == SV_F32    ? launch<float>(a, items, st)
                                        : dt == SV_BF16 ? launch<__nv_bfloat16>(a, items, st)
                                                        : launch<__half>(a, items, st));
}
