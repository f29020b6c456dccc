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
// The K best of a slice: a list in shared memory takes every element that is at
// least tau, a value that K elements are known to reach.  The first 4096 to 8192
// elements give a first tau without a sort (below), and whenever the list has
// grown to twice K it is cut back to the K best, whose last is the next tau.
// Elements in random order pass it K times a group at first and ever more seldom
// (K ln(n) in all); elements in ascending order overflow the list, and their
// group is gone through again 256 elements at a time.
#include <math.h>

#include "vocab_rows.cuh"

namespace sv {
namespace {

typedef unsigned long long u64;
constexpr int kMaxTop = 128;
constexpr int kRing = 3;       // groups: one in work, two on their way
constexpr int kList = 512;     // keys, a power of two of at least kMaxTop + kRowThreads

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

// Orders by value, then by the lower index; 0 is below every element's.
__device__ __forceinline__ u64 key_of(float x, int index) {
  const uint32_t b = __float_as_uint(__fadd_rn(x, 0.0f));  // -0 as +0
  return (u64)(b >> 31 ? ~b : b | 0x80000000u) << 32 | (uint32_t)~index;
}
__device__ __forceinline__ float value_of(u64 key) {
  const uint32_t b = (uint32_t)(key >> 32);
  return __uint_as_float(b >> 31 ? b & 0x7fffffffu : ~b);
}
__device__ __forceinline__ int index_of(u64 key) { return (int)~(uint32_t)key; }

// The min(n, K) largest of keys[0, n), all different, in descending order at the
// front; keys has room for the next power of two.  Every thread of the CTA calls
// it with the keys visible, and finds them in place.
__device__ void keep_best(u64 *keys, int n, int K) {
  if (n <= kRowThreads) {  // a thread counts what is above its key
    const int i = threadIdx.x;
    const u64 mine = i < n ? keys[i] : 0;
    int above = 0;
    if ((i & ~31) < n) {
      const ulonglong2 *two = (const ulonglong2 *)keys;
#pragma unroll 4
      for (int j = 0; j < n / 2; ++j) {
        const ulonglong2 o = two[j];
        above += (o.x > mine) + (o.y > mine);
      }
      if (n & 1) above += keys[n - 1] > mine;
    }
    __syncthreads();
    if (i < n && above < K) keys[above] = mine;
    __syncthreads();
    return;
  }
  int size = 2 * kRowThreads;
  while (size < n) size *= 2;
  for (int i = n + threadIdx.x; i < size; i += kRowThreads) keys[i] = 0;
  for (int run = 2; run <= size; run *= 2)
    for (int step = run / 2; step; step /= 2) {
      __syncthreads();
      for (int i = threadIdx.x; i < size / 2; i += kRowThreads) {
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

// The j-th largest of the warp's 32 numbers (1 <= j <= 32): a bitonic sort.
__device__ __forceinline__ float warp_jth(float x, int j) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int run = 2; run <= 32; run *= 2)
#pragma unroll
    for (int step = run / 2; step; step /= 2) {
      const float y = __shfl_xor_sync(0xffffffffu, x, step);
      const bool larger = ((lane & step) == 0) == ((lane & run) == 0);
      x = larger ? fmaxf(x, y) : fminf(x, y);
    }
  return __shfl_sync(0xffffffffu, x, j - 1);
}

template <typename T, bool TOP>
__global__ void __launch_bounds__(kRowThreads, 4) token_logprobs_kernel(LogArgs a, unsigned C) {
  grid_dep_sync();
  constexpr int VEC = RowElem<T>::VEC;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const size_t item = blockIdx.x / C;
  const uint32_t rank = C > 1 ? cluster_rank() : 0;
  extern __shared__ __align__(16) unsigned char smem[];
  u64 *list = (u64 *)(smem + kRing * kGroupBytes);  // [kList]
  u64 *all = list + kList;                          // [C][K], the first CTA's
  __shared__ RowPart s_part[kRowWarps];
  __shared__ RowPart s_all[kMaxRowCluster];
  __shared__ int s_n;
  __shared__ float s_warp[kRowWarps];

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
      for (int i = threadIdx.x; i < a.K; i += kRowThreads) {
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
  const int groups = row_groups(s);
#pragma unroll
  for (int g = 0; g < kRing - 1; ++g) {
    if (g < groups) load_group(row, s, g, g, smem);
    group_commit();
  }
  const bool known = token >= 0 && token < a.V;
  const float given = rank == 0 && a.tokens && known ? RowElem<T>::load(row + token) : 0.0f;
  float tau = -INFINITY;  // what an element has to reach, and its key to exceed
  u64 tau_key = 0;
  const float k = a.k;
  RowSums sums = row_sums();
  if (TOP) {
    if (threadIdx.x == 0) s_n = 0;
    __syncthreads();
  }
  auto offer = [&](float x, int index) {
    if (x >= tau && x > -INFINITY) {
      const u64 key = key_of(x, index);
      if (key > tau_key) {
        const int at = atomicAdd(&s_n, 1);
        if (at < kList) list[at] = key;
      }
    }
  };
  // every thread, after a barrier behind the last offer: the list's K best
  auto cut = [&](int n) {
    keep_best(list, n, a.K);
    if (n >= a.K) {
      tau_key = list[a.K - 1];
      tau = value_of(tau_key);
    }
    if (threadIdx.x == 0) s_n = min(n, a.K);
    __syncthreads();
  };
  if (rank == 0 && (int)threadIdx.x < s.singles) {
    const int i = single_at<T>(s, threadIdx.x);
    const float x = RowElem<T>::load(row + i);
    add_single<true>(sums, x, k);
    if (TOP) offer(x, i);
  }

  int slot = 0, slot_load = kRing - 1;
  for (int g = 0; g < groups; ++g) {
    if (g + kRing - 1 < groups) load_group(row, s, g + kRing - 1, slot_load, smem);
    group_commit();
    group_wait<kRing - 1>();
    uint4 w[kPieces];
    float most[kPieces];
#pragma unroll
    for (int j = 0; j < kPieces; ++j) w[j] = ring_piece(smem, slot, j);
#pragma unroll
    for (int j = 0; j < kPieces; ++j) most[j] = RowElem<T>::most(w[j]);
    const float top = fmaxf(fmaxf(most[0], most[1]), fmaxf(most[2], most[3]));
    if (top > sums.lim) raise<true>(sums, top, k);
#pragma unroll
    for (int j = 0; j < kPieces; ++j) add_piece<T, true>(sums, w[j], k);
    if (TOP) {
      // first element of this thread's piece j in the row
      auto first = [&](int j) { return s.head + (s.v0 + g * kGroupVecs + j * kRowThreads + (int)threadIdx.x) * VEC; };
      int before = 0;
      if (g == 0) {
        // In each of the W warps that have pieces, ceil(K / W) threads have an
        // element of at least the warp's ceil(K / W)-th largest maximum (-inf
        // where fewer threads have one): K elements reach the least of the
        // warps' numbers.
        const int W = min((s.v1 - s.v0 + 31) / 32, kRowWarps);
        const float mine = warp_jth(top, min((a.K + W - 1) / W, 32));
        if (lane == 0) s_warp[warp] = mine;
        __syncthreads();
        before = s_n;
        tau = s_warp[0];
        for (int i = 1; i < W; ++i) tau = fminf(tau, s_warp[i]);
        if (32 * W < a.K) tau = -INFINITY;
        __syncthreads();  // s_n is read by all before it grows
      } else {
        before = s_n;  // settled by the barriers that ended the last group
      }
      const bool some = top >= tau && top > -INFINITY;
      // a barrier with the votes: s_n is read above by all before it grows
      if (__syncthreads_or(some)) {
        if (some) {
#pragma unroll
          for (int j = 0; j < kPieces; ++j) {
            if (most[j] < tau) continue;
            float x[VEC];
            RowElem<T>::unpack(w[j], x);
#pragma unroll
            for (int i = 0; i < VEC; ++i) offer(x[i], first(j) + i);
          }
        }
        __syncthreads();
        int n = s_n;
        __syncthreads();
        if (n > kList) {  // again, an element of each thread at a time
          if (threadIdx.x == 0) s_n = before;
          __syncthreads();
          n = before;
          for (int j = 0; j < kPieces; ++j) {
            const uint4 again = ring_piece(smem, slot, j);
            float x[VEC];
            RowElem<T>::unpack(again, x);
            for (int i = 0; i < VEC; ++i) {
              if (n > kList - kRowThreads) {
                cut(n);
              }
              float xi = x[0];
#pragma unroll
              for (int e = 1; e < VEC; ++e) xi = e == i ? x[e] : xi;
              offer(xi, first(j) + i);
              __syncthreads();
              n = s_n;
              __syncthreads();
            }
          }
        }
        if (n >= 2 * a.K + 32) cut(n);
      }
    }
    slot = slot + 1 == kRing ? 0 : slot + 1;
    slot_load = slot_load + 1 == kRing ? 0 : slot_load + 1;
  }
  group_wait<0>();

  const RowPart mine = warp_join(part_of(sums), k);
  if (lane == 0) s_part[warp] = mine;
  __syncthreads();
  int n = 0;
  if (TOP) {
    n = s_n;
    keep_best(list, n, a.K);
    n = min(n, a.K);
  }
  auto join = [&](const RowPart *parts, int count) {
    return warp_join(lane < count ? parts[lane] : RowPart{-INFINITY, 0.0f, 0.0f}, k);
  };
  RowPart sum = join(s_part, kRowWarps);
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
      for (int i = threadIdx.x; i < a.K; i += kRowThreads) cluster_st_u64(all + rank * a.K + i, 0, i < n ? list[i] : 0);
    cluster_sync();
    if (rank != 0) return;
    sum = join(s_all, (int)C);
    if (TOP) {
      // lists that are not full hold zeros behind their keys; where the keys are
      // fewer than K in all, so does the first list behind their number
      keep_best(all, (int)C * a.K, a.K);
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
    for (int i = threadIdx.x; i < a.K; i += kRowThreads) {
      const u64 key = i < n ? list[i] : 0;
      a.top_token[item * a.K + i] = bad || !key ? -1 : index_of(key);
      a.top_logprob[item * a.K + i] = bad ? nan : key ? logprob(value_of(key)) : -INFINITY;
    }
  }
}

template <typename T, bool TOP>
cudaError_t launch(const LogArgs &a, unsigned items, unsigned C, cudaStream_t st) {
  // dynamic memory beyond 48 KB has to be asked for, once for each device
  size_t keys = TOP ? (size_t)kList : 0;
  if (TOP && C > 1) {
    size_t room = 2 * kRowThreads;  // keep_best sorts powers of two
    while (room < (size_t)C * a.K) room *= 2;
    keys += room;
  }
  const size_t smem = (size_t)kRing * kGroupBytes + keys * 8;
  static thread_local int set_dev = -1;
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev != set_dev) {
    const cudaError_t e = cudaFuncSetAttribute(token_logprobs_kernel<T, TOP>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               kRing * kGroupBytes + (kList + (int)kMaxRowCluster * kMaxTop) * 8);
    if (e != cudaSuccess) return e;
    set_dev = dev;
  }
  return launch_pdl_cluster(token_logprobs_kernel<T, TOP>, dim3(items * C), dim3(kRowThreads), C, smem, st, a, C);
}
template <typename T> cudaError_t launch(const LogArgs &a, unsigned items, unsigned C, cudaStream_t st) {
  return a.K ? launch<T, true>(a, items, C, st) : launch<T, false>(a, items, C, st);
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
  const unsigned C = row_ctas((size_t)V * es, (long long)B * P, 16384, 1216);
  cudaStream_t st = (cudaStream_t)stream;
  LaunchScope ls("token_logprobs", st);
  const unsigned items = (unsigned)(B * P);
  return check_launch("token_logprobs", dt == SV_F32    ? launch<float>(a, items, C, st)
                                        : dt == SV_BF16 ? launch<__nv_bfloat16>(a, items, C, st)
                                                        : launch<__half>(a, items, C, st));
}
