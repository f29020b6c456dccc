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
// One launch: a cluster of C CTAs per (layer, sequence, KV head), or one CTA
// while there are many, goes through
//   selection  the weight of the last slot kept, by a radix selection (rounds
//              of 11, 11 and 10 bits over keys kept in shared memory).  Up to
//              kLocal slots every CTA of the cluster selects by itself (an
//              exchange costs 2.5 us a round), beyond that each a part, the
//              counts added over the cluster's shared memory;
//   ranks      the kept slots in their order, by a scan over the warps: their
//              list, weights and where their rows lie;
//   moves      the rows in place, K and V together.  kept[k] >= k and strictly
//              increasing, so in increasing k no write reaches a slot whose
//              read is still to come: a ring of asynchronous copies runs ahead
//              of the stores, and a barrier per stage stands between a stage's
//              reads and its writes.
// Bound: the rows that move, read and written once: memory.  With many CTAs
// the selections of some run under the moves of others.  Measured (of the copy
// rate, 6788 GB/s): 2048 items of about 2100 slots to 1024, 346 us for 2.18 GB
// (0.93); 256 of 60000 to 16384, 847 us (0.77: keys that do not fit are read in
// each round); 16 of 131001 to 32768, 119 us for 0.56 GB (0.69: 29 us of
// selection and ranks with idle memory, then 86); 8 of 1101 to 1024, 14.5 us, of
// which 3.5 select, 4 rank and list, 4 move.
#include <math.h>

#include "cluster.cuh"

namespace sv {
namespace {

constexpr int kBins = 2048;
constexpr int kGather = 256;  // slots of a warp that are listed together, 8 of a lane
constexpr unsigned kMaxCluster = 8;
constexpr int kLocal = 8192;
constexpr int kMaxRowBytes = 2048;
constexpr int kMaxSlots = 1 << 30;

struct EvictArgs {
  char *kv;
  int64_t layer_stride, kv_stride, page_stride;  // bytes
  const int32_t *table, *seq_len;
  const float *w;
  float *out_w;
  int L, B, H, page, page_shift, max_pages, num_pages, cap, S;
  int row_bytes;      // of one head
  int64_t tok_bytes;  // from slot to slot in a page
  int budget, sinks, recent;
  int32_t *kept, *kv_len;
  uint32_t *status;
  int C;       // CTAs of a cluster
  int cached;  // keys of a CTA that fit its shared memory; longer parts are read again
  // workspace
  float *w_stage;    // [L B H][budget]: the kept slots' weights
  long long *w_src;  // [L B H][budget]: where their rows lie, in bytes from head 0
};

// A weight as an unsigned number in the order of eviction: larger is kept
// first; -0 with +0; NaN below everything.
__device__ __forceinline__ uint32_t order_key(float x) {
  if (x != x) return 0;
  const uint32_t b = __float_as_uint(__fadd_rn(x, 0.0f));
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

template <typename V>
__device__ __forceinline__ void cp_word(uint32_t dst, const void *src) {
  if constexpr (sizeof(V) == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}

// Shared memory: the ring; before the moves, two histograms and the keys.
template <typename V, int T> struct Layout {
  // Words of a thread in a stage: 64 KB stages where a cluster's barrier stands
  // between them (16 items of 131001 slots: 127 us; 136 with 32 KB ones and the
  // barrier's arrival a stage ahead), 16 KB ones where four CTAs share an SM.
  static constexpr int kWordsEach = T == 512 ? 8 : 4;
  static constexpr int kStageWords = T * kWordsEach;
  static constexpr int kStages = 3;
  static constexpr int kRing = kStages * kStageWords * (int)sizeof(V);
  static constexpr int kKeysAt = 2 * kBins * 4;
  // keys that make the block no larger than its ring, but not fewer than this
  static constexpr int kMostKeys = T == 512 ? 47104 : 8192;
  static constexpr int kPer = T / 4;  // rows of a stage, at most
  static constexpr int kOnePerSm = 208 * 1024;
  static int bytes(int cached) {
    const int select = kKeysAt + (cached + kGather) * 4;  // (the last lanes go past the keys)
    return select > kRing ? select : kRing;
  }
  static_assert(T / 32 * kGather * 4 <= kKeysAt, "the histograms hold what the warps gather");
  static_assert(kRing <= kOnePerSm && kKeysAt + (kMostKeys + kGather) * 4 <= kOnePerSm, "one CTA to an SM");
  static_assert(2 * kMaxRowBytes <= kStageWords * (int)sizeof(V), "a stage holds a row's K and V");
};

// T = 256: C = 1, many items; T = 512: few.
template <typename V, int T>
__global__ void __launch_bounds__(T, T == 256 ? 4 : 1) evict_kernel(EvictArgs a) {
  grid_dep_sync();
  using Lay = Layout<V, T>;
  constexpr int W = T / 32;
  constexpr int kStages = Lay::kStages, kWordsEach = Lay::kWordsEach;
  constexpr int PB = kBins / T;  // bins of a thread
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ long long s_from[kStages + 1][Lay::kPer], s_to[kStages + 1][Lay::kPer];
  __shared__ uint32_t s_part[W], s_pick[2];
  __shared__ uint32_t s_cnt[2];  // this CTA's slots above the limit, and at it
  __shared__ uint32_t s_scan[W][2];
  __shared__ int s_first;
  uint32_t *s_hist = (uint32_t *)smem;  // [2][kBins], used in turn
  uint32_t *s_keys = (uint32_t *)(smem + Lay::kKeysAt);
  const unsigned FULL = 0xffffffffu;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int C = T == 256 ? 1 : a.C;
  const int item = blockIdx.x / C;  // (layer, sequence, head)
  const int rank = C > 1 ? (int)cluster_rank() : 0;
  const int h = item % a.H, b = item / a.H % a.B, l = item / a.H / a.B;
  const int n = a.seq_len[b];
  const int m = a.budget;
  int32_t *kept = a.kept + (size_t)item * m;
  const int32_t *table = a.table + (size_t)b * a.max_pages;
  const float *w = a.w + (size_t)item * a.S;
  float *out_w = a.out_w + (size_t)item * a.S;

  // faults: a length out of range, or a page of the sequence out of the pool
  uint32_t fault = n < 0 || n > a.cap ? SV_ROW_BAD_LEN : 0;
  bool bad = false;
  if (!fault) {
    const int pages = (int)(((long long)n + a.page - 1) / a.page);
#pragma unroll 4
    for (int i = threadIdx.x; i < pages; i += T) bad |= (unsigned)table[i] >= (unsigned)a.num_pages;
  }
  for (int i = threadIdx.x; i < 2 * kBins; i += T) s_hist[i] = 0;
  if (threadIdx.x == 0) s_first = 0x7fffffff;
  if (__syncthreads_or(bad)) fault = SV_ROW_BAD_PAGE;
  if (l == 0 && h == 0 && rank == 0 && threadIdx.x == 0) {
    a.kv_len[b] = fault ? -1 : min(n, m);
    if (a.status) a.status[b] = fault;
  }
  const int me = rank * T + threadIdx.x, all = C * T;
  if (fault || n <= m) {  // the same for every CTA of the cluster
    for (int k = me; k < m; k += all) kept[k] = !fault && k < n ? k : -1;
    if (!fault && a.out_w != a.w)
      for (int k = me; k < n; k += all) out_w[k] = w[k];
    return;
  }

  // ------------------------------------------------------------ selection
  // the slots between the first and the last, and how many of them stay
  const int mid0 = a.sinks, mid1 = n - a.recent;
  uint32_t need = (uint32_t)(m - a.sinks - a.recent);
  const bool none = need == 0;
  const int P = mid1 - mid0 > kLocal ? C : 1;  // CTAs that select together
  const int part = P > 1 ? rank : 0;
  const int per = (int)(((long long)(mid1 - mid0) + P - 1) / P);
  const int lo = min(mid0 + part * per, mid1), hi = min(lo + per, mid1);
  const bool cached = hi - lo <= a.cached;
  // `limit` becomes the key of the need-th largest, `need` the number of slots
  // at the limit that stay
  uint32_t limit = 0, mask = 0;
  if (!none) {
#pragma unroll 1
    for (int round = 0; round < 3; ++round) {
      const int shift = round == 0 ? 21 : round == 1 ? 10 : 0;
      const uint32_t bins = round == 2 ? kBins / 2 : kBins;
      uint32_t *hist = s_hist + (round & 1) * kBins;
      if (round == 2)  // read in round 0, which every CTA has left
        for (int i = threadIdx.x; i < kBins; i += T) hist[i] = 0;
      __syncthreads();
      auto count = [&](bool in, uint32_t key) {
        // (equal digits of a warp cost no more than different ones)
        if (in && (key & mask) == limit) atomicAdd(&hist[key >> shift & (bins - 1)], 1u);
      };
      if (cached) {
        if (round == 0) {
          const uint32_t at = (uint32_t)__cvta_generic_to_shared(s_keys) - 4 * (uint32_t)lo;
          for (int i = lo + threadIdx.x; i < hi; i += T)
            asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(at + 4 * (uint32_t)i), "l"(w + i) : "memory");
          asm volatile("cp.async.wait_all;" ::: "memory");
          __syncthreads();
        }
        // four neighbouring keys of a thread, its own from here to the ranks
        for (int i = lo + 4 * (int)threadIdx.x; i < hi; i += 4 * T) {
          uint4 *at = (uint4 *)(s_keys + (i - lo)), x = *at;
          if (round == 0) {
            x.x = order_key(__uint_as_float(x.x));
            x.y = order_key(__uint_as_float(x.y));
            x.z = order_key(__uint_as_float(x.z));
            x.w = order_key(__uint_as_float(x.w));
            *at = x;
          }
          count(true, x.x);
          count(i + 1 < hi, x.y);
          count(i + 2 < hi, x.z);
          count(i + 3 < hi, x.w);
        }
      } else {  // too many to keep: read again each round
        constexpr int kMany = 16;  // loads of a thread in flight
        for (int i0 = lo + threadIdx.x; i0 < hi; i0 += T * kMany) {
          float x[kMany];
#pragma unroll
          for (int j = 0; j < kMany; ++j) x[j] = i0 + j * T < hi ? w[i0 + j * T] : 0.0f;
#pragma unroll
          for (int j = 0; j < kMany; ++j) count(i0 + j * T < hi, order_key(x[j]));
        }
      }
      if (P > 1)
        cluster_sync();
      else
        __syncthreads();
      // thread t: the bins from the top, PB t on
      const int low = (int)bins - PB * ((int)threadIdx.x + 1);
      uint32_t c[PB] = {}, sum = 0;
      if (low >= 0) {
        if (T == 256 || P == 1) {
#pragma unroll
          for (int j = 0; j < PB; ++j) c[j] = hist[low + PB - 1 - j];
        } else if constexpr (T == 512) {
          uint4 x[kMaxCluster];
#pragma unroll
          for (int r = 0; r < (int)kMaxCluster; ++r)
            x[r] = r < P ? cluster_ld_v4(&hist[low], (uint32_t)r) : make_uint4(0, 0, 0, 0);
#pragma unroll
          for (int r = 0; r < (int)kMaxCluster; ++r) {
            c[0] += x[r].w;
            c[1] += x[r].z;
            c[2] += x[r].y;
            c[3] += x[r].x;
          }
        }
#pragma unroll
        for (int j = 0; j < PB; ++j) sum += c[j];
      }
      uint32_t incl = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t x = __shfl_up_sync(FULL, incl, o);
        if (lane >= o) incl += x;
      }
      if (lane == 31) s_part[warp] = incl;
      __syncthreads();
      // (the warps' sums fit a warp)
      uint32_t before = incl - sum + __reduce_add_sync(FULL, lane < warp ? s_part[lane < W ? lane : 0] : 0);
      if (before < need && need <= before + sum) {
#pragma unroll
        for (int j = 0; j < PB; ++j) {
          if (before < need && need <= before + c[j]) {
            s_pick[0] = (uint32_t)(low + PB - 1 - j);
            s_pick[1] = need - before;
          }
          before += c[j];
        }
      }
      __syncthreads();
      limit |= s_pick[0] << shift;
      need = s_pick[1];
      mask |= (bins - 1) << shift;
    }
  }

  // ------------------------------------------------------------ ranks
  // Slots above the limit all stay, those at it while `need` lasts.  A warp
  // takes a run of slots.
  __syncthreads();
  const int run = ((hi - lo + W - 1) / W + 31) & ~31;
  const int r0 = min(lo + warp * run, hi), r1 = none ? r0 : min(r0 + run, hi);
  uint32_t b_above = 0, b_at = 0;  // in this warp's run, then before its next slots
  auto tally = [&](bool in, uint32_t key) {
    b_above += in && key > limit;
    b_at += in && key == limit;
  };
  if (cached) {
#pragma unroll 2
    for (int i = r0 + 4 * lane; i < r1; i += 128) {
      const uint4 x = *(const uint4 *)(s_keys + (i - lo));
      tally(true, x.x);
      tally(i + 1 < r1, x.y);
      tally(i + 2 < r1, x.z);
      tally(i + 3 < r1, x.w);
    }
  } else {
#pragma unroll 4
    for (int i = r0 + lane; i < r1; i += 32) tally(true, order_key(w[i]));
  }
  b_above = __reduce_add_sync(FULL, b_above);
  b_at = __reduce_add_sync(FULL, b_at);
  if (lane == 0) {
    s_scan[warp][0] = b_above;
    s_scan[warp][1] = b_at;
  }
  __syncthreads();
  const uint32_t of_warp[2] = {lane < W ? s_scan[lane < W ? lane : 0][0] : 0,
                               lane < W ? s_scan[lane < W ? lane : 0][1] : 0};
  b_above = __reduce_add_sync(FULL, lane < warp ? of_warp[0] : 0);
  b_at = __reduce_add_sync(FULL, lane < warp ? of_warp[1] : 0);
  const uint32_t t_above = __reduce_add_sync(FULL, of_warp[0]), t_at = __reduce_add_sync(FULL, of_warp[1]);
  if (P > 1) {
    if (threadIdx.x == 0) {
      s_cnt[0] = t_above;
      s_cnt[1] = t_at;
    }
    cluster_sync();
    uint32_t x = 0, y = 0;
    if (lane < rank) {
      x = cluster_ld_u32(&s_cnt[0], (uint32_t)lane);
      y = cluster_ld_u32(&s_cnt[1], (uint32_t)lane);
    }
    b_above += __reduce_add_sync(FULL, x);
    b_at += __reduce_add_sync(FULL, y);
  }
  // Positions of the list go round the cluster's CTAs, `each` at a time: a
  // stage of the ring, K and V of whole rows.  Where all select the same, each
  // lists its own; where each selects a part, what it finds.
  const int words = a.row_bytes / (int)sizeof(V);
  const int each = min(Lay::kPer, Lay::kStageWords / (2 * words));
  const int each_shift = (each & (each - 1)) ? -1 : __ffs(each) - 1;
  auto turn_of = [&](int k) { return each_shift >= 0 ? k >> each_shift : k / each; };
  float *stage = a.w_stage + (size_t)item * m;
  long long *src = a.w_src + (size_t)item * m;
  int first = 0x7fffffff;
  // entries k of the list, two at a time, are slots i (nothing below 0)
  auto list = [&](const int (&k)[2], const int (&i)[2]) {
    int id[2];
    float x[2];
#pragma unroll
    for (int j = 0; j < 2; ++j)
      if (k[j] >= 0) {
        id[j] = table[a.page_shift >= 0 ? i[j] >> a.page_shift : i[j] / a.page];
        x[j] = w[i[j]];
      }
#pragma unroll
    for (int j = 0; j < 2; ++j)
      if (k[j] >= 0) {
        const int in_page = a.page_shift >= 0 ? i[j] & (a.page - 1) : i[j] % a.page;
        kept[k[j]] = i[j];
        stage[k[j]] = x[j];
        src[k[j]] = id[j] * (long long)a.page_stride + in_page * (long long)a.tok_bytes;
        if (i[j] != k[j]) first = min(first, k[j]);
      }
  };
  // A warp gathers what stays of kGather slots in the histograms' place (their
  // positions follow one another) and lists it with all lanes.
  int *found = (int *)s_hist + warp * kGather;
  for (int i0 = r0; i0 < r1; i0 += kGather) {
    const int k0 = a.sinks + (int)(b_above + min(b_at, need));
    // 8 neighbouring slots of a lane, by two wide loads: counted, scanned over
    // the warp, gathered (a ballot and population counts for every 32 slots took
    // twice as long: the integer pipe bounds this)
    const uint32_t *from = s_keys + (i0 - lo);
    if (!cached) {
#pragma unroll
      for (int j = 0; j < kGather; j += 32) {
        const int i = i0 + j + lane;
        found[j + lane] = i < r1 ? (int)order_key(w[i]) : 0;
      }
      __syncwarp();
      from = (const uint32_t *)found;
    }
    const uint4 x0 = ((const uint4 *)from)[2 * lane], x1 = ((const uint4 *)from)[2 * lane + 1];
    uint32_t key[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
    const int i_mine = i0 + 8 * lane, behind = i0 + kGather - r1;  // slots of the next run, or none
    if (behind > 0) {
#pragma unroll
      for (int j = 0; j < 8; ++j) key[j] = i_mine + j < r1 ? key[j] : 0;
    }
    uint32_t c = 0;  // above the limit, and 2^16 times those at it
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (key[j] > limit) c += 1;
      if (key[j] == limit) c += 0x10000;
    }
    uint32_t incl = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t x = __shfl_up_sync(FULL, incl, o);
      if (lane >= o) incl += x;
    }
    const uint32_t total = __shfl_sync(FULL, incl, 31), at0 = min(b_at, need);
    __syncwarp();  // the keys may lie where the slots go
    if (total >> 16) {
      uint32_t at = b_at + ((incl - c) >> 16);
      int *to = found + ((incl - c) & 0xffff) + min(at, need) - at0;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const bool level = key[j] == limit;
        if (key[j] > limit || (level && at < need)) *to++ = i_mine + j;
        at += level;
      }
    } else {
      int *to = found + (incl - c);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (key[j] > limit) *to++ = i_mine + j;
    }
    b_above += total & 0xffff;
    b_at += total >> 16;
    if (limit == 0 && behind > 0) b_at -= behind;  // they came last
    const int n_found = (int)((total & 0xffff) + min(b_at, need) - at0);
    __syncwarp();
    for (int e = lane; e < n_found; e += 64) {
      int k[2], i[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        k[j] = k0 + e + 32 * j;
        if (e + 32 * j >= n_found || (P < C && turn_of(k[j]) % C != rank)) k[j] = -1;
        i[j] = k[j] >= 0 ? found[e + 32 * j] : 0;
      }
      list(k, i);
    }
    __syncwarp();
  }
  const int ends = a.sinks + a.recent;
  for (int e = me; e < ends; e += 2 * all) {
    int k[2], i[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int e_j = e + j * all;
      k[j] = e_j >= ends ? -1 : e_j < a.sinks ? e_j : m - ends + e_j;
      i[j] = e_j < a.sinks ? k[j] : n - m + k[j];
    }
    list(k, i);
  }
  first = __reduce_min_sync(FULL, first);
  if (lane == 0) atomicMin(&s_first, first);
  // No weight is read again, and the ring takes the keys' place.
  if (C > 1) {
    cluster_sync();
    first = 0x7fffffff;
    if (lane < C) first = (int)cluster_ld_u32(&s_first, (uint32_t)lane);
    first = __reduce_min_sync(FULL, first);
    cluster_sync();  // read by all: a CTA may leave
  } else {
    __syncthreads();
    first = s_first;
  }

  // ------------------------------------------------------------ moves
  char *base = a.kv + l * a.layer_stride + (int64_t)h * a.row_bytes;
  // Stage s: positions (s C + rank) each + 0 ... each - 1 of this CTA, from the
  // first stage with a row that moves.  This thread moves up to kWordsEach
  // words of it, at the same places in every stage, and looks up one row.
  const int stages = (int)((m + (long long)each * C - 1) / (each * C));
  const int s0 = min(first / (each * C), stages);
  auto start = [&](int s) { return (s * C + rank) * each; };
  int row[kWordsEach];
  long long off[kWordsEach];
#pragma unroll
  for (int j = 0; j < kWordsEach; ++j) {
    const int at = j * T + threadIdx.x, word = at % (2 * words);
    row[j] = at / (2 * words);
    off[j] = word < words ? word * (long long)sizeof(V) : (word - words) * (long long)sizeof(V) + a.kv_stride;
    if (row[j] >= each) row[j] = 0x40000000;  // no word
  }
  // Weights: each stage's with its rows, where a few CTAs have to keep the memory
  // busy (16 items of 131001 slots: 119 us, all before the first row moves 121);
  // before the moves where others move meanwhile (2048 items: 344 us, with the
  // moves 346; 256 of 20000 slots: 389 and 394).
  constexpr bool kWithMoves = T == 512;
  V *mine = (V *)smem + threadIdx.x;
  const uint32_t mine_at = (uint32_t)__cvta_generic_to_shared(mine);
  long long next_from = 0;
  int next_id = 0;
  float next_w = 0.0f;
  auto fetch = [&](int s) {  // what the look-up of stage s needs from memory
    const int k = start(s) + (int)threadIdx.x;
    if ((int)threadIdx.x < each && k < m) {
      next_from = src[k];
      if (kWithMoves) next_w = stage[k];
      next_id = table[a.page_shift >= 0 ? k >> a.page_shift : k / a.page];
    }
  };
  auto look_up = [&](int s, int at) {
    if ((int)threadIdx.x >= each) return;
    const int k = start(s) + (int)threadIdx.x;
    const int in_page = a.page_shift >= 0 ? k & (a.page - 1) : k % a.page;
    if (kWithMoves && k < m) out_w[k] = next_w;
    s_from[at][threadIdx.x] = next_from;
    s_to[at][threadIdx.x] = next_id * (long long)a.page_stride + in_page * (long long)a.tok_bytes;
  };
  auto load = [&](int s, int slot, int at) {
    const int left = m - start(s);
#pragma unroll
    for (int j = 0; j < kWordsEach; ++j)
      if (row[j] < left)
        cp_word<V>(mine_at + (slot * Lay::kStageWords + j * T) * (int)sizeof(V),
                   base + s_from[at][row[j]] + off[j]);
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  {  // the first look-ups side by side
    long long from[kStages];
    int id[kStages];
    float weight[kStages];
#pragma unroll
    for (int s = 0; s < kStages; ++s) {
      fetch(s0 + s);
      from[s] = next_from;
      id[s] = next_id;
      weight[s] = next_w;
    }
    fetch(s0 + kStages);
    const long long keep_from = next_from;
    const int keep_id = next_id;
    const float keep_w = next_w;
#pragma unroll
    for (int s = 0; s < kStages; ++s) {
      next_from = from[s];
      next_id = id[s];
      next_w = weight[s];
      look_up(s0 + s, s);
    }
    next_from = keep_from;
    next_id = keep_id;
    next_w = keep_w;
  }
  __syncthreads();
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) load(s0 + s, s, s);
  // (the first stages' weights stay where they are)
  const int before_moves = kWithMoves ? a.out_w == a.w ? 0 : (int)min((long long)s0 * each * C, (long long)m) : m;
  for (int k = me; k < before_moves; k += 4 * all) {
    float x[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = k + j * all < before_moves ? stage[k + j * all] : 0.0f;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (k + j * all < before_moves) out_w[k + j * all] = x[j];
  }
  int zero = m + me;  // the weights behind the list
  auto clear = [&](int end) {
#pragma unroll 4
    for (; zero < end; zero += all) out_w[zero] = 0.0f;
  };
  const long long zeros = (n - m) / max(stages - s0, 1) + all;  // of a stage
  if (!kWithMoves) clear(n);
  int slot = 0, place = 0;  // of stage s: (s - s0) mod kStages, mod (kStages + 1)
  for (int s = s0; s < stages; ++s) {
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
    // This stage's reads are done and its successors' rows looked up, by all
    // threads.  Over the cluster nothing has to be made visible: the copies
    // have arrived, and only then may the others write where they read from.
    if (C > 1) asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory");
    __syncthreads();
    const int before = place == 0 ? kStages : place - 1;
    load(s + kStages - 1, slot == 0 ? kStages - 1 : slot - 1, place >= 2 ? place - 2 : place + kStages - 1);
    if (C > 1) asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
    const int left = m - start(s);
    V v[kWordsEach];
#pragma unroll
    for (int j = 0; j < kWordsEach; ++j)
      if (row[j] < left) v[j] = mine[slot * Lay::kStageWords + j * T];
#pragma unroll
    for (int j = 0; j < kWordsEach; ++j)
      if (row[j] < left) *(V *)(base + s_to[place][row[j]] + off[j]) = v[j];
    look_up(s + kStages, before);  // in the place of stage s - 1
    fetch(s + kStages + 1);
    if (kWithMoves) clear((int)min((long long)n, m + (s - s0 + 1) * zeros));
    slot = slot + 1 == kStages ? 0 : slot + 1;
    place = place == kStages ? 0 : place + 1;
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  clear(n);
}

// How many clusters of C CTAs, one CTA to an SM, the device runs at once: GPCs
// of different sizes leave 15 clusters of 8, 23 of 6, 36 of 4 on 152 SMs.
int cluster_room(int C) {
  static thread_local int dev_of = -1, room[kMaxCluster + 1];
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev != dev_of) {
    for (int c = 1; c <= (int)kMaxCluster; ++c) {
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3((unsigned)c * 256);
      cfg.blockDim = dim3(512);
      cfg.dynamicSmemBytes = Layout<uint4, 512>::kOnePerSm;
      cudaLaunchAttribute at[1];
      at[0].id = cudaLaunchAttributeClusterDimension;
      at[0].val.clusterDim.x = (unsigned)c;
      at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
      cfg.attrs = at;
      cfg.numAttrs = 1;
      if (cudaOccupancyMaxActiveClusters(&room[c], evict_kernel<uint4, 512>, &cfg) != cudaSuccess) {
        cudaGetLastError();
        room[c] = c == 1 ? num_sms() : 0;
      }
    }
    dev_of = dev;
  }
  return room[C];
}

template <typename V, int T>
sv_status allow_smem() {
  static thread_local int set_dev = -1;
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev == set_dev) return SV_OK;
  const cudaError_t e = cudaFuncSetAttribute(
      evict_kernel<V, T>, cudaFuncAttributeMaxDynamicSharedMemorySize, Layout<V, T>::kOnePerSm);
  if (e != cudaSuccess) return check_launch("kv_evict", e);
  set_dev = dev;
  return SV_OK;
}

template <typename V, int T>
sv_status launch(EvictArgs &a, int items, cudaStream_t st) {
  using Lay = Layout<V, T>;
  // (up to kLocal slots a CTA holds them all)
  const long long part = a.cap > kLocal ? max(((long long)a.cap + a.C - 1) / a.C, (long long)kLocal) : a.cap;
  a.cached = (int)(part < Lay::kMostKeys ? part : Lay::kMostKeys);
  LaunchScope ls("kv_evict", st);
  return check_launch("kv_evict", launch_pdl_cluster(evict_kernel<V, T>, dim3((unsigned)(items * a.C)), dim3(T),
                                                     (unsigned)a.C, (size_t)Lay::bytes(a.cached), st, a));
}

struct Sizes {
  long long items;
  size_t stage, src, total;
};
bool sizes_of(Sizes &z, int L, int B, int H, int budget) {
  constexpr long long most = 1 << 24;
  if ((long long)L * B > most) return false;  // the product of three may pass 63 bits
  z.items = (long long)L * B * H;
  if (z.items > most || budget > kMaxSlots) return false;
  z.stage = 0;
  z.src = align_up((size_t)z.items * budget * 4, 256);
  z.total = align_up(z.src + (size_t)z.items * budget * 8, 256);
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
  if (cap > kMaxSlots || !sizes_of(z, L, B, Hkv, budget) || (long long)D * elem_bytes > kMaxRowBytes)
    return set_error(SV_ERR_UNSUPPORTED,
                     "more than 2^30 slots a sequence, 2^24 (layer, sequence, head)s or %d bytes a row",
                     kMaxRowBytes);
  if (S < cap) return set_error(SV_ERR_INVALID_ARG, "weight sums have %d slots a head, the page table %lld", S, cap);
  const int row = D * elem_bytes;
  if (row % 4) return set_error(SV_ERR_UNSUPPORTED, "rows of %d bytes (a multiple of 4 is needed)", row);
  const int64_t limit = INT64_MAX / 4;
  // (slots that a page has room for: a page's own bytes may pass 63 bits)
  if (page_stride < 1 || page_stride > limit / elem_bytes / num_pages ||
      page_stride * elem_bytes / row / Hkv < page || kv_stride < 1 || kv_stride > limit / elem_bytes ||
      layer_stride < 0 || layer_stride > limit / elem_bytes / L)
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
  const bool vec = row % 16 == 0 && (uintptr_t)kv % 16 == 0 && page_stride * elem_bytes % 16 == 0 &&
                   kv_stride * elem_bytes % 16 == 0 && layer_stride * elem_bytes % 16 == 0;
  if (workspace_bytes < z.total)
    return set_error(SV_ERR_INVALID_ARG, "workspace of %zu bytes, need %zu", workspace_bytes, z.total);
  // other CTAs still read what one writes
  auto overlap = [](const void *x, size_t nx, const void *y, size_t ny) {
    return (uintptr_t)x < (uintptr_t)y + ny && (uintptr_t)y < (uintptr_t)x + nx;
  };
  const size_t sums = (size_t)z.items * S * 4;
  if (out_weight_sum != weight_sum && overlap(weight_sum, sums, out_weight_sum, sums))
    return set_error(SV_ERR_INVALID_ARG, "out_weight_sum overlaps weight_sum (it may be the same)");
  if (overlap(out_kv_len, (size_t)B * 4, seq_len, (size_t)B * 4))
    return set_error(SV_ERR_INVALID_ARG, "out_kv_len overlaps seq_len");
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
  a.page_shift = -1;
  for (int i = 0; i < 31; ++i)
    if (page == 1 << i) a.page_shift = i;
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
  char *ws = (char *)workspace;
  a.w_stage = (float *)(ws + z.stage);
  a.w_src = (long long *)(ws + z.src);
  // Few items: large CTAs, one to an SM, and for each item the largest cluster
  // with which all run at once (16 items in clusters of 8, two of them
  // on the same SMs, took 175 us where clusters of 6 took 166).  Many: small
  // CTAs, 4 on an SM, which select under each other's moves (2048 items: 349 us;
  // in two launches, selection and moves, 400).
  const int items = (int)z.items;
  a.C = 1;
  cudaStream_t st = (cudaStream_t)stream;
  if (items <= 152) {
    if ((s = allow_smem<uint4, 512>()) != SV_OK || (s = allow_smem<uint32_t, 512>()) != SV_OK) return s;
    for (int c = (int)kMaxCluster; c > 1 && a.C == 1; --c)
      if (items <= cluster_room(c)) a.C = c;
    return vec ? launch<uint4, 512>(a, items, st) : launch<uint32_t, 512>(a, items, st);
  }
  if ((s = allow_smem<uint4, 256>()) != SV_OK || (s = allow_smem<uint32_t, 256>()) != SV_OK) return s;
  return vec ? launch<uint4, 256>(a, items, st) : launch<uint32_t, 256>(a, items, st);
}
