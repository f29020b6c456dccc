// kv_evict.cu -- eviction from a paged KV cache by accumulated attention
// weight (sm_103a).
//
// A cache under a budget ([Lesson] "Decodificação Especulativa e EAGLE-3",
// "Reversão de KV cache": a physical cache with a logical length): of the n
// slots of a (layer, sequence, KV head) the first `sinks`, the last `recent`
// and, of those between, the ones with the largest summed attention weight are
// kept, `budget` in all, in their order; slot k of the shorter cache is slot
// kept[k] of the longer.
//
// Two launches.  evict_select: a cluster of C CTAs per (layer, sequence, KV
// head) finds the weight of the last slot kept by a radix selection (four
// rounds of 8 bits, histograms added over the cluster's shared memory), then
// ranks the kept slots by a scan and writes their list and their weights.
// evict_move moves the rows in place: kept[k] >= k and strictly increasing, so
// in increasing k no write reaches a slot whose read is still to come; a CTA
// owns a column range of one (layer, K or V, sequence, KV head) and goes
// through the list in batches, all reads of a batch before its writes.
//
// Bound: the rows that move, read and written once: memory.
#include <math.h>

#include "common.cuh"

namespace sv {
namespace {

constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr unsigned kMaxCluster = 8;
constexpr int kMoveThreads = 256;
constexpr int kMaxSlots = 1 << 30;

struct EvictArgs {
  char *kv;
  int64_t layer_stride, kv_stride, page_stride;  // bytes
  const int32_t *table, *seq_len;
  const float *w;
  float *out_w;
  int L, B, H, page, max_pages, num_pages, cap, S;
  int row_bytes;  // of one head
  int64_t tok_bytes;  // from slot to slot in a page
  int budget, sinks, recent;
  int32_t *kept, *kv_len;
  uint32_t *status;
  // workspace
  float *w_stage;   // [L B H][budget]: the kept slots' weights
  int32_t *w_todo;  // [L B H]: slots to move (0: none), -1 on a fault
  int col_bytes, ncol;  // a move CTA's columns of a row, and how many such ranges
};

// A weight as an unsigned number in the order of eviction: larger is kept
// first; -0 with +0; NaN below everything.
__device__ __forceinline__ uint32_t order_key(float x) {
  if (x != x) return 0;
  const uint32_t b = __float_as_uint(__fadd_rn(x, 0.0f));
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(EvictArgs a, unsigned C) {
  grid_dep_sync();
  const unsigned FULL = 0xffffffffu;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int item = blockIdx.x / C;  // (layer, sequence, head)
  const int rank = C > 1 ? (int)cluster_rank() : 0;
  const int b = item / a.H % a.B;
  const int n = a.seq_len[b];
  const int m = a.budget;
  __shared__ uint32_t s_hist[256 * 33];
  __shared__ uint32_t s_sum[256];
  __shared__ uint32_t s_pick[2];
  __shared__ uint32_t s_cnt[2];  // this CTA's slots above the limit, and at it
  __shared__ uint32_t s_scan[kSelWarps][2];
  int32_t *kept = a.kept + (size_t)item * m;
  const bool writer = item < a.B * a.H && item % a.H == 0 && rank == 0;  // layer 0, head 0

  // faults: a length out of range, or a page of the sequence out of the pool
  uint32_t fault = n < 0 || n > a.cap ? SV_ROW_BAD_LEN : 0;
  if (!fault) {
    const int pages = (int)(((long long)n + a.page - 1) / a.page);
    bool bad = false;
    for (int i = threadIdx.x; i < pages; i += kSelThreads)
      bad |= (unsigned)a.table[(size_t)b * a.max_pages + i] >= (unsigned)a.num_pages;
    if (__syncthreads_or(bad)) fault = SV_ROW_BAD_PAGE;
  }
  if (writer && threadIdx.x == 0) {
    a.kv_len[b] = fault ? -1 : min(n, m);
    if (a.status) a.status[b] = fault;
  }
  const int me = rank * kSelThreads + threadIdx.x, all = (int)C * kSelThreads;
  if (fault || n <= m) {  // the same for every CTA of the cluster
    for (int k = me; k < m; k += all) kept[k] = !fault && k < n ? k : -1;
    if (me == 0) a.w_todo[item] = fault ? -1 : 0;
    return;
  }

  // the slots between the first and the last, and how many of them stay
  const float *w = a.w + (size_t)item * a.S;
  const int mid0 = a.sinks, mid1 = n - a.recent;
  uint32_t need = (uint32_t)(m - a.sinks - a.recent);
  const int per = (int)(((long long)(mid1 - mid0) + C - 1) / C);
  const int lo = min(mid0 + rank * per, mid1), hi = min(lo + per, mid1);

  // radix selection: `limit` is the key of the need-th largest; `need` ends as
  // the number of slots at the limit that stay
  uint32_t limit = 0, mask = 0;
  if (need > 0) {
    for (int shift = 24; shift >= 0; shift -= 8) {
      for (int i = threadIdx.x; i < 256 * 33; i += kSelThreads) s_hist[i] = 0;
      __syncthreads();
      // a column of bins per lane: no two lanes of a warp meet in one counter
      for (int i = lo + threadIdx.x; i < hi; i += kSelThreads) {
        const uint32_t key = order_key(w[i]);
        if ((key & mask) == limit) atomicAdd(&s_hist[(key >> shift & 255) * 33 + lane], 1u);
      }
      __syncthreads();
      if (threadIdx.x < 256) {
        uint32_t c = 0;
#pragma unroll
        for (int l = 0; l < 32; ++l) c += s_hist[threadIdx.x * 33 + l];
        s_sum[threadIdx.x] = c;
      }
      if (C > 1)
        cluster_sync();
      else
        __syncthreads();
      if (warp == 0) {  // lane l: the bins 255 - 8 l ... 248 - 8 l, from the top
        uint32_t c[8], sum = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          c[j] = 0;
          for (unsigned r = 0; r < C; ++r)
            c[j] += C > 1 ? cluster_ld_u32(&s_sum[255 - 8 * lane - j], r) : s_sum[255 - 8 * lane - j];
          sum += c[j];
        }
        uint32_t incl = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint32_t x = __shfl_up_sync(FULL, incl, o);
          if (lane >= o) incl += x;
        }
        uint32_t before = incl - sum;
        if (before < need && need <= incl) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            if (before < need && need <= before + c[j]) {
              s_pick[0] = 255 - 8 * lane - j;
              s_pick[1] = need - before;
            }
            before += c[j];
          }
        }
      }
      __syncthreads();
      limit |= s_pick[0] << shift;
      need = s_pick[1];
      mask |= 255u << shift;
      if (C > 1) cluster_sync();  // the counts are read: they may be written again
    }
  }

  // ranks: slots above the limit all stay, those at it while `need` lasts
  auto kind = [&](int i) -> uint32_t {
    if (m == a.sinks + a.recent) return 0;  // none of these stays
    const uint32_t key = order_key(w[i]);
    return key > limit ? 1 : key == limit ? 2 : 0;
  };
  // a warp's run of slots
  const int run = ((hi - lo + kSelWarps - 1) / kSelWarps + 31) / 32 * 32;
  const int r0 = min(lo + warp * run, hi), r1 = min(r0 + run, hi);
  uint32_t above = 0, at = 0;
  for (int i0 = r0; i0 < r1; i0 += 32) {
    const uint32_t k = i0 + lane < r1 ? kind(i0 + lane) : 0;
    above += __popc(__ballot_sync(FULL, k == 1));
    at += __popc(__ballot_sync(FULL, k == 2));
  }
  if (lane == 0) {
    s_scan[warp][0] = above;
    s_scan[warp][1] = at;
  }
  __syncthreads();
  uint32_t b_above = 0, b_at = 0, t_above = 0, t_at = 0;
  for (int j = 0; j < kSelWarps; ++j) {
    if (j < warp) {
      b_above += s_scan[j][0];
      b_at += s_scan[j][1];
    }
    t_above += s_scan[j][0];
    t_at += s_scan[j][1];
  }
  if (C > 1) {
    if (threadIdx.x == 0) {
      s_cnt[0] = t_above;
      s_cnt[1] = t_at;
    }
    cluster_sync();
    for (int r = 0; r < rank; ++r) {
      b_above += cluster_ld_u32(&s_cnt[0], (uint32_t)r);
      b_at += cluster_ld_u32(&s_cnt[1], (uint32_t)r);
    }
  }
  float *stage = a.w_stage + (size_t)item * m;
  for (int i0 = r0; i0 < r1; i0 += 32) {
    const int i = i0 + lane;
    const uint32_t k = i < r1 ? kind(i) : 0;
    const uint32_t ma = __ballot_sync(FULL, k == 1), me_ = __ballot_sync(FULL, k == 2);
    const uint32_t below = (1u << lane) - 1u;
    const uint32_t ra = b_above + __popc(ma & below), re = b_at + __popc(me_ & below);
    if (k == 1 || (k == 2 && re < need)) {
      const int pos = a.sinks + (int)(ra + min(re, need));
      kept[pos] = i;
      stage[pos] = w[i];
    }
    b_above += __popc(ma);
    b_at += __popc(me_);
  }
  for (int k = me; k < a.sinks; k += all) {
    kept[k] = k;
    stage[k] = w[k];
  }
  for (int k = me; k < a.recent; k += all) {
    kept[m - a.recent + k] = n - a.recent + k;
    stage[m - a.recent + k] = w[n - a.recent + k];
  }
  if (me == 0) a.w_todo[item] = m;
  if (C > 1) cluster_sync();  // no CTA leaves while its counts may still be read
}

// ---------------------------------------------------------------------------
// Moves: blockIdx.x = ((item, K or V), column range).  The CTAs of an item also
// put its weights in place.
constexpr int kBatchRows = 128;
template <typename V>
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(EvictArgs a) {
  grid_dep_sync();
  const int col = blockIdx.x % a.ncol;
  const int rest = blockIdx.x / a.ncol;
  const int which = rest & 1, item = rest >> 1;
  const int b = item / a.H % a.B, h = item % a.H, l = item / a.H / a.B;
  const int todo = a.w_todo[item];
  if (todo < 0) return;
  const int n = a.seq_len[b];
  {  // the weights, spread over the item's CTAs
    const float *w = a.w + (size_t)item * a.S;
    float *__restrict__ out = a.out_w + (size_t)item * a.S;
    const float *__restrict__ stage = a.w_stage + (size_t)item * a.budget;
    const int k0 = (which * a.ncol + col) * kMoveThreads + threadIdx.x, step = 2 * a.ncol * kMoveThreads;
    if (todo > 0) {
#pragma unroll 8
      for (int k = k0; k < todo; k += step) out[k] = stage[k];
#pragma unroll 8
      for (int k = todo + k0; k < n; k += step) out[k] = 0.0f;
    } else if (a.out_w != a.w) {
      for (int k = k0; k < n; k += step) out[k] = w[k];
    }
  }
  if (todo == 0) return;
  const int32_t *kept = a.kept + (size_t)item * a.budget;
  // the first slot that moves: kept[k] - k never falls
  int k0 = 0, k1 = todo;
  while (k0 < k1) {
    const int k = (k0 + k1) >> 1;
    if (kept[k] == k)
      k0 = k + 1;
    else
      k1 = k;
  }
  __shared__ long long s_src[kBatchRows], s_dst[kBatchRows];
  const int32_t *table = a.table + (size_t)b * a.max_pages;
  char *base = a.kv + l * a.layer_stride + which * a.kv_stride + (int64_t)h * a.row_bytes +
               (int64_t)col * a.col_bytes;
  const int words = min(a.col_bytes, a.row_bytes - col * a.col_bytes) / (int)sizeof(V);
  constexpr int U = 8;
  for (; k0 < todo; k0 += kBatchRows) {
    const int cnt = min(kBatchRows, todo - k0);
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * cnt; i += kMoveThreads) {
      const int r = i >> 1;
      const int slot = i & 1 ? kept[k0 + r] : k0 + r;
      const int pg = slot / a.page;
      const long long off = (long long)table[pg] * a.page_stride + (long long)(slot - pg * a.page) * a.tok_bytes;
      (i & 1 ? s_src : s_dst)[r] = off;
    }
    __syncthreads();
    const int total = cnt * words;
    for (int i0 = 0; i0 < total; i0 += kMoveThreads * U) {
      V v[U];
#pragma unroll
      for (int j = 0; j < U; ++j) {
        const int i = i0 + j * kMoveThreads + threadIdx.x;
        if (i < total) v[j] = *(const V *)(base + s_src[i / words] + (size_t)(i % words) * sizeof(V));
      }
      __syncthreads();  // every read of these rows before their writes
#pragma unroll
      for (int j = 0; j < U; ++j) {
        const int i = i0 + j * kMoveThreads + threadIdx.x;
        if (i < total) *(V *)(base + s_dst[i / words] + (size_t)(i % words) * sizeof(V)) = v[j];
      }
    }
  }
}

struct Sizes {
  long long items;
  size_t stage, todo, total;
};
bool sizes_of(Sizes &z, int L, int B, int H, int budget) {
  z.items = (long long)L * B * H;
  if (z.items > (1 << 24) || budget > kMaxSlots) return false;
  z.stage = 0;
  z.todo = align_up((size_t)z.items * budget * 4, 256);
  z.total = align_up(z.todo + (size_t)z.items * 4, 256);
  return true;
}

}  // namespace
}  // namespace sv

using namespace sv;

extern "C" size_t sv_kv_evict_workspace(int L, int B, int Hkv, int budget) {
  Sizes z;
  if (L < 1 || B < 0 || Hkv < 1 || budget < 1 || !sizes_of(z, L, B, Hkv, budget)) return 0;
  return z.total;
}

extern "C" sv_status sv_kv_evict(void *kv, int64_t layer_stride, int64_t kv_stride,
                                 int64_t page_stride, int elem_bytes, const int32_t *block_table,
                                 const int32_t *seq_len, const float *weight_sum,
                                 float *out_weight_sum, int L, int B, int Hkv, int D, int page,
                                 int max_pages, int num_pages, int S, int budget, int sinks,
                                 int recent, int32_t *out_kept, int32_t *out_kv_len,
                                 uint32_t *out_status, void *workspace, size_t workspace_bytes,
                                 void *stream) {
  if (L < 1 || B < 0 || Hkv < 1 || D < 1 || elem_bytes < 1 || page < 1 || max_pages < 1 || num_pages < 1)
    return set_error(SV_ERR_INVALID_ARG, "bad cache shape");
  if (budget < 1 || sinks < 0 || recent < 0 || (long long)sinks + recent > budget)
    return set_error(SV_ERR_INVALID_ARG, "need budget >= 1, sinks, recent >= 0 and sinks + recent <= budget");
  const long long cap = (long long)page * max_pages;
  Sizes z;
  if (cap > kMaxSlots || !sizes_of(z, L, B, Hkv, budget) || (long long)D * elem_bytes > (1 << 20))
    return set_error(SV_ERR_UNSUPPORTED,
                     "more than 2^30 slots a sequence, 2^24 (layer, sequence, head)s or 1 MiB a row");
  if (S < cap) return set_error(SV_ERR_INVALID_ARG, "weight sums have %d slots a head, the page table %lld", S, cap);
  const int row = D * elem_bytes;
  if (row % 4) return set_error(SV_ERR_UNSUPPORTED, "rows of %d bytes (a multiple of 4 is needed)", row);
  const int64_t inner = (int64_t)page * Hkv * row, limit = INT64_MAX / 4;
  if (page_stride > limit / elem_bytes / num_pages || page_stride * elem_bytes < inner || kv_stride < 1 ||
      kv_stride > limit / elem_bytes || layer_stride < 0 || layer_stride > limit / elem_bytes / L)
    return set_error(SV_ERR_INVALID_ARG, "page_stride must cover a page, kv_stride be positive, layer_stride >= 0");
  if (L > 1 && layer_stride < 1) return set_error(SV_ERR_INVALID_ARG, "layer_stride must be positive");
  if (B == 0) return SV_OK;
  if (!kv || !block_table || !seq_len || !weight_sum || !out_weight_sum || !out_kept || !out_kv_len || !workspace)
    return set_error(SV_ERR_INVALID_ARG, "null pointer");
  if ((uintptr_t)kv % 4 || (page_stride * elem_bytes) % 4 || (kv_stride * elem_bytes) % 4 ||
      (layer_stride * elem_bytes) % 4 || (uintptr_t)block_table % 4 || (uintptr_t)seq_len % 4 ||
      (uintptr_t)weight_sum % 4 || (uintptr_t)out_weight_sum % 4 || (uintptr_t)out_kept % 4 ||
      (uintptr_t)out_kv_len % 4 || (uintptr_t)out_status % 4 || (uintptr_t)workspace % 256)
    return set_error(SV_ERR_INVALID_ARG, "misaligned pointer or stride (4 bytes; the workspace 256)");
  if (workspace_bytes < z.total)
    return set_error(SV_ERR_INVALID_ARG, "workspace of %zu bytes, need %zu", workspace_bytes, z.total);
  sv_status s;
  if ((s = map_arg(kv, "kv")) != SV_OK || (s = map_arg(block_table, "block_table")) != SV_OK ||
      (s = map_arg(seq_len, "seq_len")) != SV_OK || (s = map_arg(weight_sum, "weight_sum")) != SV_OK ||
      (s = map_arg(out_weight_sum, "out_weight_sum")) != SV_OK ||
      (s = map_arg(out_kept, "out_kept")) != SV_OK || (s = map_arg(out_kv_len, "out_kv_len")) != SV_OK ||
      (s = map_arg(out_status, "out_status")) != SV_OK || (s = map_arg(workspace, "workspace")) != SV_OK)
    return s;
  EvictArgs a;
  a.kv = (char *)kv;
  a.layer_stride = layer_stride * elem_bytes;
  a.kv_stride = kv_stride * elem_bytes;
  a.page_stride = page_stride * elem_bytes;
  a.table = block_table;
  a.seq_len = seq_len;
  a.w = weight_sum;
  a.out_w = out_weight_sum;
  a.L = L;
  a.B = B;
  a.H = Hkv;
  a.page = page;
  a.max_pages = max_pages;
  a.num_pages = num_pages;
  a.cap = (int)cap;
  a.S = S;
  a.row_bytes = row;
  a.tok_bytes = (int64_t)Hkv * row;
  a.budget = budget;
  a.sinks = sinks;
  a.recent = recent;
  a.kept = out_kept;
  a.kv_len = out_kv_len;
  a.status = out_status;
  a.w_stage = (float *)((char *)workspace + z.stage);
  a.w_todo = (int32_t *)((char *)workspace + z.todo);
  const int items = (int)z.items;
  // CTAs of an item: one per 8192 slots, while the card has room for them
  unsigned C = 1;
  while (C < kMaxCluster && cap > (long long)C * 8192 && (long long)items * C * 2 <= 1216) C *= 2;
  cudaStream_t st = (cudaStream_t)stream;
  {
    LaunchScope ls("evict_select", st);
    s = check_launch("evict_select", launch_pdl_cluster(evict_select_kernel, dim3((unsigned)items * C),
                                                        dim3(kSelThreads), C, 0, st, a, C));
    if (s != SV_OK) return s;
  }
  const bool vec = row % 16 == 0 && (uintptr_t)kv % 16 == 0 && a.page_stride % 16 == 0 &&
                   a.kv_stride % 16 == 0 && a.layer_stride % 16 == 0;
  // columns of a row apart while the streams are few; 64 bytes keep whole sectors
  a.col_bytes = row;
  while (a.col_bytes > 64 && a.col_bytes % 128 == 0 && (long long)items * 2 * (row / a.col_bytes) < 608)
    a.col_bytes /= 2;
  a.ncol = row / a.col_bytes;
  const dim3 grid((unsigned)items * 2 * a.ncol);
  LaunchScope ls("evict_move", st);
  return check_launch("evict_move", vec ? launch_pdl(evict_move_kernel<uint4>, grid, dim3(kMoveThreads), 0, st, a)
                                        : launch_pdl(evict_move_kernel<uint32_t>, grid, dim3(kMoveThreads), 0, st, a));
}
