// paged_attn.cu -- attention of one new token per sequence over a paged KV
// cache, split over the cache's length and joined (sm_103a).
//
// The drafting side of a speculative step ([Lesson] "Decodificação Especulativa
// e EAGLE-3", Passo 3; [Blog] "投机解码发展", section 4): the draft model produces
// its tokens one at a time, each attending to the cached ones.  With s_j =
// scale <q, k_j> over the visible slots j, m = max s_j and l = sum exp(s_j - m):
// out = sum exp(s_j - m) v_j / l, lse = m + ln l.  Two disjoint parts of the
// slots join exactly: m = max(m1, m2), l = l1 2^(m1 - m) + l2 2^(m2 - m), and
// the same for the weighted sums of the values (scores are kept in log2 units).
//
// Bound: every visible K and V row is read once for 16 query heads of its KV
// head (4 D bytes a slot and KV head), 4 D G operations on it: memory up to G = 16;
// above, each further 16 heads read the rows again, mostly from L2.  The matrix
// products only have to keep up with HBM (45 GB/s per SM), so they run as
// m16n8k16 tensor instructions on registers, transposed: S^T = K Q^T with 16
// keys as rows and 8 (or 16) query heads as columns, O^T = V^T P^T with 16
// dimensions as rows.  With the keys on the long side no row of an instruction
// is spent on heads a model does not have (G = 1 to 8 costs the same), and S,
// P and O never leave a warp's registers.
//
// Work: a unit is a run of 64-key tiles of one (sequence, KV head, up to 16
// query heads); KV heads of the same tiles are neighbouring CTAs, so that the
// D-wide slices of one token's row are read at about the same time.  Units are
// cut from the lengths on the device (a scan over the batch): up to a few
// hundred sequences into as many equal shares of all tiles as are resident, a
// CTA going from one sequence to the next.  So the host never sees them and a
// captured graph follows them.  Within a unit each of the 4 warps owns 16 keys of
// every tile: it loads them (cp.async, 16 bytes a lane), multiplies, and keeps its
// own m, l and O; nothing but the last merge crosses warps, and no CTA barrier
// stands in the loop.
//
// Groups of 16 keys start at multiples of 16 slots, so with pages of a multiple
// of 16 slots one table entry serves a group; other page sizes look up every
// row.  Rows that are not visible are zero-filled in shared memory, not read.
//
// Measured (of the copy rate, 6788 GB/s): 128 sequences of 3585-4096 tokens, 64
// query heads on 8 KV heads of 128, 303 us for 2.02 GB (0.98; pages of 20 or of
// 1 slot: 330 us); one of 131001 tokens, 84 us (0.94); windows of 2048 at D =
// 64, 64 x 16 heads, 88 us (0.90); 24 ragged sequences with weight sums, 53 us of
// GPU time (0.66: the scores' way to memory and back, two launches), 54 to 61 in a
// stream of calls.  256 query heads on 8 KV heads, 468 us for the same batch (0.64),
// 512 on 8, 32 sequences, 191 us (0.40).  With queries on the long side of the
// products (heads padded to 16 rows) the first four took 342, 109, 106 and 83 us.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>

#include "common.cuh"

namespace sv {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = 4;
constexpr int kGroup = 16;                // keys of a warp in a tile
constexpr int kTile = kWarps * kGroup;    // keys of a CTA tile
constexpr int kRows = 16;                 // query heads of a unit, at most
// CTAs that are resident at once on 152 SMs (2 per SM at D = 128), and the
// fewest tiles of a unit: below that its fixed cost shows (one of 200 tokens: 8.4
// us of GPU time with 8, 12.4 with 2 and a join).
template <int D> constexpr int kSlots = D == 64 ? 608 : D == 128 ? 304 : 152;
constexpr int kMinTiles = 8;
constexpr int kMaxSlots = 1 << 30;
// The reference the exponentials are taken against follows the maximum only when
// a score is more than 2^kSlack above it: most tiles need no maximum over the
// warp, and sums and products are in 32 bits.  In fp16 the reference lies 2^kBias
// below the maximum it was set by, so that weights fill the type's range from the
// top (2^15 at most): numbers below 2^-24 round to nothing, and 20000 weights of
// 2^-25.5 beside one of 1 lost a quarter of their output with the reference at
// the maximum.  Now a weight is off by 2^-36 of the largest.  bf16 reaches 2^-126.
template <typename T> constexpr float kSlack = 8.0f;
template <typename T> constexpr float kBias = 0.0f;
template <> constexpr float kSlack<__half> = 4.0f;
template <> constexpr float kBias<__half> = 11.0f;
constexpr float kLn2 = 0.693147180559945309f, kLog2e = 1.4426950408889634f;

struct PagedArgs {
  const void *q, *kv;
  int64_t kv_stride, page_stride;  // elements from K to V, and from page to page
  const int32_t *table, *seq_len;
  int B, Hq, Hkv, G, gt, NH;  // gt groups of 16 query heads per KV head, NH = Hkv gt
  int page, page_shift, max_pages, num_pages;
  int window, sinks, cap;
  int units;   // aimed at
  int groups;  // the grid's groups of CTAs, one for each head group
  int finding;  // how a CTA finds its unit: one of the below
  float scale_log2;
  int rows;  // query heads of a unit: min(G, 16)
  int vis_max;
  float *weight_sum;
  int S;
  void *out;
  float *lse;
  uint32_t *status;
  // workspace
  int4 *w_map;       // [groups]: sequence (or -1), unit within it, its units, its length
  int2 *w_first;     // [B]: index of the sequence's first group, its units
  float *w_o;        // [units][rows][D]
  float2 *w_ml;      // [units][rows]: reference (log2 units) and sum
  uint32_t *w_flag;  // [units]
  float *w_score;    // [B][Hkv][vis_max][G], q.k
};

// The visible slots of a sequence: [0, first) and [lo, len), laid out one after
// the other from multiples of 16 slots, so that positions v, v + 1, ... of a
// group are slots of one aligned run of 16 (some of them not visible).
struct Visible {
  int len, lo, first;
  int split, shift;  // position v is slot v below split, v + shift from there
  int n;             // positions
  bool bad;
};
__device__ __forceinline__ Visible visible(const PagedArgs &a, int len) {
  Visible v;
  v.bad = len < 0 || len > a.cap;
  v.len = v.bad ? 0 : len;
  v.lo = a.window > 0 ? max(0, v.len - a.window) : 0;
  v.first = a.sinks;
  if (v.lo <= a.sinks) v.lo = v.first = 0;  // they meet: [0, len)
  v.split = (v.first + kGroup - 1) / kGroup * kGroup;
  v.shift = v.lo / kGroup * kGroup - v.split;
  v.n = v.len - v.shift;
  return v;
}
__device__ __forceinline__ int slot_of(const Visible &v, int pos) {
  return pos < v.split ? pos : pos + v.shift;
}
__device__ __forceinline__ bool seen(const Visible &v, int pos) {
  return pos < v.split ? pos < v.first : pos + v.shift >= v.lo && pos < v.n;
}
__device__ __forceinline__ int tiles_of(const Visible &v) { return (v.n + kTile - 1) / kTile; }

struct Plan {
  int b, i, n;   // sequence, unit within it, units of it
  int first;     // group index of the sequence's first unit
};
// How a CTA finds its unit.
//   kWhole  no sequence has room for two
//   kOne    a single sequence
//   kScan   a scan of the lengths in every CTA; sequences cut one by one
//   kShare  a scan too; an equal share of the batch's tiles, wherever the
//           sequences end
//   kMap    a map that a launch of its own has written; one by one
// Shares leave no CTA with less to do (sequences cut one by one in brackets): 24
// ragged sequences 51 us (54), 128 of 500-8000 tokens 355 (379), 32 of 500-20000
// 234 (240), 128 of 3585-4096 301 (310), windows of 2052 at D = 64 91 (95).  They
// cost a CTA the way to a first load once more where a sequence ends, and every
// CTA the scan: with more heads than kShareHeads to a resident CTA, or sequences
// than kShareBatch, the map is as good (1000 of 200-2000: 105 us, shares 109; 2000
// of 90-1110: 111 and 160), and sequences that are cut into 8 units and more each
// have equal ones anyway (4 of 700: 19 us, shares 21).
enum { kWhole, kOne, kScan, kShare, kMap };
constexpr int kShareHeads = 4, kShareBatch = 512;

// Units aimed at where sequences are cut one by one.  Into 8 and more for each
// (sequence, KV head) they are nearly equal, and one wave of as many as are
// resident is best (one of 131001 tokens: 84 us, in two waves 93).  Fewer units
// each leave them unequal: twice as many, so that the early ones make room.
// Rounding up adds half a unit to each (sequence, head); a batch of more of those
// than units is left whole.
int slots_of(int D) { return D == 64 ? kSlots<64> : D == 128 ? kSlots<128> : kSlots<256>; }
int units_for(int D, int B, int NH) {
  return 8LL * B * NH <= slots_of(D) ? slots_of(D) : 2 * slots_of(D);
}
// tiles that a unit may have at most, for a batch of that many tiles in all
__device__ __forceinline__ long long unit_tiles(const PagedArgs &a, long long tiles) {
  const long long room = max((long long)a.units / 2, a.B == 1 ? (long long)a.units : a.units - (long long)a.B * a.NH / 2);
  return min(max((long long)kMinTiles, (tiles * a.NH + room - 1) / room), (long long)kMaxSlots);
}
// units of a sequence of t tiles when a unit may have `most`
__device__ __forceinline__ int units_of(int t, long long most) {
  if (t <= kMinTiles) return 1;
  return ((unsigned)t + (unsigned)most - 1) / (unsigned)most;
}

// Cuts the batch into groups of units: calls out(b, first, n) for every
// sequence, each from one thread, and returns how many groups there are.  Every
// thread of the CTA calls it.  Lengths are read past L1 (paged_finish_kernel).
template <int THREADS, typename F>
__device__ int cut_batch(const PagedArgs &a, F out) {
  constexpr int W = THREADS / 32;
  __shared__ long long s_red[W];
  const unsigned FULL = 0xffffffffu;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // a run of k sequences to each thread
  const int k = (a.B + THREADS - 1) / THREADS;
  const int b0 = min((int)threadIdx.x * k, a.B), b1 = min(b0 + k, a.B);
  const int t0 = b0 < b1 ? tiles_of(visible(a, __ldcg(a.seq_len + b0))) : 0;  // read once where k = 1
  auto tiles_at = [&](int b) { return b == b0 ? t0 : tiles_of(visible(a, __ldcg(a.seq_len + b))); };
  long long tiles = 0;
  for (int b = b0; b < b1; ++b) tiles += tiles_at(b);
#pragma unroll
  for (int o = 16; o; o >>= 1) tiles += __shfl_xor_sync(FULL, tiles, o);
  if (lane == 0) s_red[warp] = tiles;
  __syncthreads();
  tiles = 0;
#pragma unroll
  for (int w = 0; w < W; ++w) tiles += s_red[w];
  __syncthreads();
  const long long most = unit_tiles(a, tiles);
  int mine = 0;
  for (int b = b0; b < b1; ++b) mine += units_of(tiles_at(b), most);
  int incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(FULL, incl, o);
    if (lane >= o) incl += x;
  }
  if (lane == 31) s_red[warp] = incl;
  __syncthreads();
  int at = incl - mine, all = 0;
#pragma unroll
  for (int w = 0; w < W; ++w) {
    if (w < warp) at += (int)s_red[w];
    all += (int)s_red[w];
  }
  for (int b = b0; b < b1; ++b) {
    const int n = units_of(tiles_at(b), most);
    out(b, at, n);
    at += n;
  }
  return all;
}

// The batch as one row of tiles, sequence after sequence (an empty one counts as
// a tile): calls out(b, first tile, tiles, tiles in all) for every sequence, each
// from one thread.  Every thread of the CTA calls it.
template <int THREADS, typename F>
__device__ void walk_batch(const PagedArgs &a, F out) {
  constexpr int W = THREADS / 32;
  __shared__ long long s_sum[W];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int k = (a.B + THREADS - 1) / THREADS;
  const int b0 = min((int)threadIdx.x * k, a.B), b1 = min(b0 + k, a.B);
  auto read = [&](int b) { return max(tiles_of(visible(a, __ldcg(a.seq_len + b))), 1); };
  const int t0 = b0 < b1 ? read(b0) : 0;  // read once where k = 1
  auto tiles_at = [&](int b) { return b == b0 ? t0 : read(b); };
  long long mine = 0;
  for (int b = b0; b < b1; ++b) mine += tiles_at(b);
  long long incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += x;
  }
  if (lane == 31) s_sum[warp] = incl;
  __syncthreads();
  long long at = incl - mine, all = 0;
#pragma unroll
  for (int w = 0; w < W; ++w) {
    if (w < warp) at += s_sum[w];
    all += s_sum[w];
  }
  for (int b = b0; b < b1; ++b) {
    const int t = tiles_at(b);
    out(b, at, t, all);
    at += t;
  }
}
// Group g of G takes the tiles from g all / G to (g + 1) all / G; a part of a
// sequence in a group is unit (group + sequence): with every part one or the other
// grows by one.
__device__ __forceinline__ long long share_groups(const PagedArgs &a, long long all) {
  return min((long long)a.groups, max(all / kMinTiles, 1LL));
}
struct Share {
  int b;
  long long first, at, end;  // the sequence's first tile; the group's tiles from `at` to `end`
};
template <int THREADS> __device__ Share find_share(const PagedArgs &a, int g) {
  __shared__ Share s_share;
  if (threadIdx.x == 0) s_share.b = -1;
  __syncthreads();
  walk_batch<THREADS>(a, [&](int b, long long first, int t, long long all) {
    const long long G = share_groups(a, all), at = g * all / G;
    if (g < G && first <= at && at < first + t) s_share = Share{b, first, at, (g + 1) * all / G};
  });
  __syncthreads();
  return s_share;
}

// The sequence and part that group g is (BY_GROUP; not for kShare), or the units
// of sequence g.  Every thread of the CTA calls it; b = -1: no such group.
template <int THREADS, bool BY_GROUP>
__device__ Plan find_plan(const PagedArgs &a, int g) {
  if (a.finding == kWhole) return Plan{g, 0, 1, g};
  if (a.finding == kOne) {
    const int t = tiles_of(visible(a, __ldcg(a.seq_len)));
    const int n = units_of(t, unit_tiles(a, t));
    return Plan{BY_GROUP && g >= n ? -1 : 0, BY_GROUP ? g : 0, n, 0};
  }
  if (a.finding == kMap) {
    if (BY_GROUP) {
      const int4 e = __ldcg(a.w_map + g);
      return Plan{e.x, e.y, e.z, g - e.y};
    }
    const int2 e = __ldcg(a.w_first + g);
    return Plan{g, 0, e.y, e.x};
  }
  __shared__ Plan s_plan;
  if (BY_GROUP || a.finding == kScan) {
    if (threadIdx.x == 0) s_plan.b = -1;
    __syncthreads();
    cut_batch<THREADS>(a, [&](int b, int first, int n) {
      if (BY_GROUP ? g >= first && g < first + n : b == g) s_plan = Plan{b, BY_GROUP ? g - first : 0, n, first};
    });
    __syncthreads();
    return s_plan;
  }
  walk_batch<THREADS>(a, [&](int b, long long first, int t, long long all) {
    if (b != g) return;
    const long long G = share_groups(a, all);
    const int g0 = (int)(((first + 1) * G - 1) / all), g1 = (int)(((first + t) * G - 1) / all);
    s_plan = Plan{b, 0, g1 - g0 + 1, g0 + b};
  });
  __syncthreads();
  return s_plan;
}

constexpr int kMapThreads = 1024;
__global__ void __launch_bounds__(kMapThreads) paged_map_kernel(PagedArgs a) {
  grid_dep_sync();
  const int all = cut_batch<kMapThreads>(a, [&](int b, int first, int n) {
    a.w_first[b] = make_int2(first, n);
    const int len = a.seq_len[b];
    for (int i = 0; i < n; ++i) a.w_map[first + i] = make_int4(b, i, n, len);
  });
  for (int g = all + threadIdx.x; g < a.groups; g += kMapThreads) a.w_map[g] = make_int4(-1, 0, 0, 0);
}

// ------------------------------------------------------------ element types
template <typename T> struct Pair;
template <> struct Pair<__nv_bfloat16> {
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *(const uint32_t *)&v;
  }
  static __device__ __forceinline__ float2 unpack(uint32_t v) { return make_float2(bf16_lo(v), bf16_hi(v)); }
  static __device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
};
template <> struct Pair<__half> {
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *(const uint32_t *)&v;
  }
  static __device__ __forceinline__ float2 unpack(uint32_t v) { return __half22float2(*(const __half2 *)&v); }
  static __device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
};

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// an 8 x 8 matrix of 16-bit elements, a row's pair per lane, transposed
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
// 16 bytes to shared memory; the second form writes zeros (and reads nothing)
// when `bytes` is 0
__device__ __forceinline__ void cp16(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp16(uint32_t dst, const void *src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <int D, int NT> struct Shape {
  static constexpr int kRowBytes = 2 * D;
  static constexpr int kPart = kGroup * kRowBytes;  // a group's K (or V) rows
  static constexpr int kStages = 3;
  static constexpr int kWarpBytes = kStages * 2 * kPart;
  static constexpr int kHeads = 8 * NT;
  // the query tile stays in registers but where the accumulators fill them
  static constexpr bool kQRegs = D * NT < 512;
  static constexpr int kQBytes = kQRegs ? 0 : kHeads * kRowBytes;
  static constexpr size_t kSmem = (size_t)kWarps * kWarpBytes + kQBytes + 512;  // + alignment
  // O of the warps for the last merge: rows 4 floats longer than D, so that the
  // 8 x 4 lanes of a store meet in no bank
  static constexpr int kMergeRow = D + 4;
  static_assert((size_t)kWarps * kHeads * kMergeRow * 4 <= (size_t)kWarps * kWarpBytes, "merge");
};

// SHARING: kShare; a kernel of its own, since its loop over the parts costs the
// other findings registers and a longer way to their first load (4 of 700: 19 us,
// in one kernel 21).
template <typename T, int D, int NT, bool SHARING>
__global__ void __launch_bounds__(kThreads, SHARING && D == 64 ? 4 : 0) paged_attn_kernel(PagedArgs a) {
  grid_dep_sync();
  using Sh = Shape<D, NT>;
  // the operands' rows are addressed by exclusive or: they start at 512 bytes
  extern __shared__ unsigned char smem_raw[];
  const uint32_t sm0 = ((uint32_t)__cvta_generic_to_shared(smem_raw) + 511) & ~511u;
  unsigned char *smem = smem_raw + (sm0 - (uint32_t)__cvta_generic_to_shared(smem_raw));
  const unsigned FULL = 0xffffffffu;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g4 = lane >> 2, t4 = lane & 3;
  const int unit = blockIdx.x;
  const int h = unit % a.NH;
  const int hkv = h / a.gt, head0 = hkv * a.G + (h % a.gt) * kRows;
  const int rows = min(kRows, a.G - (h % a.gt) * kRows);
  Share share;
  Plan plan;
  if constexpr (SHARING)
    share = find_share<kThreads>(a, unit / a.NH);
  else
    plan = find_plan<kThreads, true>(a, unit / a.NH);
  if ((SHARING ? share.b : plan.b) < 0) return;

  __shared__ float s_m[kWarps][kRows], s_l[kWarps][kRows];
  __shared__ uint32_t s_bad[kWarps];
  __shared__ long long s_row[kWarps][32];  // offsets of two groups' rows (pages not of 16)

  // one part of a sequence after the other (one only, unless CTAs share the batch)
  for (;;) {
    const int b = SHARING ? share.b : plan.b;
    const Visible vis = visible(a, a.finding == kMap ? __ldcg(&a.w_map[unit / a.NH].w) : __ldcg(a.seq_len + b));
    const int tiles = tiles_of(vis);
    int t0, t1;
    if constexpr (SHARING) {
      t0 = (int)(share.at - share.first);
      t1 = (int)min(share.end - share.first, (long long)tiles);
    } else {
      t0 = (int)((long long)tiles * plan.i / plan.n);
      t1 = (int)((long long)tiles * (plan.i + 1) / plan.n);
    }
    const bool whole = SHARING ? t0 == 0 && t1 == tiles : plan.n == 1;
    const size_t part = SHARING ? (size_t)(unit / a.NH + b) * a.NH + h : unit;

    // query heads as the right-hand operand: head g4 (+ 8), dimensions 2 t4 ...
    const T *q = (const T *)a.q + ((size_t)b * a.Hq + head0) * D;
    uint32_t qf[Sh::kQRegs ? D / 16 : 1][NT][2];
    const uint32_t sm_q = sm0 + kWarps * Sh::kWarpBytes;
    if (Sh::kQRegs) {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const uint32_t *r = (const uint32_t *)(q + (size_t)(g4 + 8 * n) * D + 2 * t4);
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          qf[k][n][0] = g4 + 8 * n < rows ? r[8 * k] : 0;
          qf[k][n][1] = g4 + 8 * n < rows ? r[8 * k + 4] : 0;
        }
      }
    } else {
      for (int i = threadIdx.x; i < Sh::kHeads * (D / 8); i += kThreads) {
        const int r = i / (D / 8), c = i % (D / 8);
        const uint4 v = r < rows ? *(const uint4 *)(q + (size_t)r * D + c * 8) : make_uint4(0, 0, 0, 0);
        *(uint4 *)(smem + kWarps * Sh::kWarpBytes + r * Sh::kRowBytes + ((c ^ (r & 7)) * 16)) = v;
      }
      __syncthreads();
    }

    // ------------------------------------------------------------ the loads
    // This warp's group i is the 16 positions from (t0 + i) kTile + 16 warp.
    const int groups = t1 - t0;
    auto pos_of = [&](int i) { return (t0 + i) * kTile + warp * kGroup; };
    const uint32_t sm_w = sm0 + warp * Sh::kWarpBytes;
    const int32_t *table = a.table + (size_t)b * a.max_pages;
    const T *kv = (const T *)a.kv + (int64_t)hkv * D;
    const int64_t row_elems = (int64_t)a.Hkv * D;
    constexpr int CPR = D / 8;     // 16-byte pieces of a row
    constexpr int RPI = 32 / CPR;  // rows of one round of the warp's copies
    const int lr = lane / CPR, lc = lane % CPR;
    const bool by_row = a.page % kGroup != 0;
    bool bad = false;
    // Lanes look rows up in parallel: lane l the first row of group i0 + l
    // (`ids` of 32 groups), or by_row the row l % 16 of group i0 + l / 16 (of 2).
    // The table entries are loaded a batch ahead; an offset is -1 where nothing
    // is visible, and odd where not all of the group's 16 slots are.
    const int batch = by_row ? 2 : 32;
    int next_id = 0;
    auto position = [&](int i0) { return by_row ? pos_of(i0 + (lane >> 4)) + (lane & 15) : pos_of(i0 + lane); };
    auto wanted = [&](int i0) {  // whether the lane's row or group has a slot to load
      const int i = i0 + (by_row ? lane >> 4 : lane), p = position(i0);
      return i < groups && (by_row ? seen(vis, p) : p < vis.n);
    };
    auto fetch_ids = [&](int i0) {
      if (wanted(i0)) {
        const int slot = slot_of(vis, position(i0));
        next_id = table[a.page_shift >= 0 ? slot >> a.page_shift : slot / a.page];
      }
    };
    auto offsets = [&](int i0) -> long long {
      if (!wanted(i0)) return -1;
      if ((unsigned)next_id >= (unsigned)a.num_pages) {
        bad = true;
        return -1;
      }
      const int p = position(i0), slot = slot_of(vis, p);
      const int in_page = a.page_shift >= 0 ? slot & (a.page - 1) : slot % a.page;
      const long long off = next_id * (long long)a.page_stride + in_page * (long long)row_elems;
      return by_row || (seen(vis, p) && seen(vis, p + kGroup - 1)) ? off : off | 1;
    };
    long long offs = -1;
    auto load_group = [&](int i, int stage) {
      if (i >= groups || pos_of(i) >= vis.n) return;  // nothing, and nothing after it
      if ((i & (batch - 1)) == 0) {
        offs = offsets(i);
        fetch_ids(i + batch);
        if (by_row) {
          __syncwarp();
          s_row[warp][lane] = offs;
          __syncwarp();
        }
      }
      const uint32_t dst = (sm_w + stage * 2 * Sh::kPart) + lr * Sh::kRowBytes + ((lc ^ lr) * 16);
      if (by_row) {
#pragma unroll
        for (int j = 0; j < kGroup / RPI; ++j) {
          const long long off = s_row[warp][(i & 1) * kGroup + j * RPI + lr];
          const uint32_t n = off >= 0 ? 16u : 0u;
          const T *src = kv + (off >= 0 ? off : 0) + lc * 8;
          const uint32_t d = (dst ^ ((j * RPI & 7) * 16)) + j * RPI * Sh::kRowBytes;
          cp16(d, src, n);
          cp16(d + Sh::kPart, src + a.kv_stride, n);
        }
        return;
      }
      const long long off = __shfl_sync(FULL, offs, i & 31);
      if (!(off & 1)) {  // all 16 rows
        const T *k = kv + off + lr * row_elems + lc * 8, *v = k + a.kv_stride;
#pragma unroll
        for (int j = 0; j < kGroup / RPI; ++j) {
          const uint32_t d = (dst ^ ((j * RPI & 7) * 16)) + j * RPI * Sh::kRowBytes;
          cp16(d, k);
          cp16(d + Sh::kPart, v);
          k += RPI * row_elems;
          v += RPI * row_elems;
        }
      } else {  // some, or none
        const int p = pos_of(i);
#pragma unroll 1
        for (int j = 0; j < kGroup / RPI; ++j) {
          const int r = j * RPI + lr;
          const uint32_t n = off >= 0 && seen(vis, p + r) ? 16u : 0u;
          const T *src = kv + (n ? (off ^ 1) + r * row_elems : 0) + lc * 8;
          const uint32_t d = (dst ^ ((j * RPI & 7) * 16)) + j * RPI * Sh::kRowBytes;
          cp16(d, src, n);
          cp16(d + Sh::kPart, src + a.kv_stride, n);
        }
      }
    };

    float o[D / 16][NT][4];
#pragma unroll
    for (int j = 0; j < D / 16; ++j)
#pragma unroll
      for (int n = 0; n < NT; ++n) o[j][n][0] = o[j][n][1] = o[j][n][2] = o[j][n][3] = 0.0f;
    // per head 2 t4 + e (+ 8 n): the reference m (log2 units), l, and the z that
    // is subtracted (m, or 0 while there is no finite score)
    float m[NT][2], z[NT][2], l[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        m[n][e] = -INFINITY;
        z[n][e] = l[n][e] = 0.0f;
      }
    const float sc = a.scale_log2;
    float *scores = a.w_score ? a.w_score + ((size_t)b * a.Hkv + hkv) * a.vis_max * a.G + (h % a.gt) * kRows
                              : nullptr;

    fetch_ids(0);
#pragma unroll
    for (int i = 0; i < Sh::kStages - 1; ++i) {
      load_group(i, i);
      cp_commit();
    }
    // addresses of this lane's rows of the operands: K's row (key) and V's
    const int ka = (((lane >> 3) & 1) << 3) + (lane & 7), kh = lane >> 4;
    const int va = ((lane >> 4) << 3) + (lane & 7), vh = (lane >> 3) & 1;
    const uint32_t k_lane = sm_w + ka * Sh::kRowBytes + ((kh ^ (ka & 7)) * 16);
    const uint32_t v_lane = sm_w + Sh::kPart + va * Sh::kRowBytes + ((vh ^ (va & 7)) * 16);
    int st_load = Sh::kStages - 1, st = 0;
    uint32_t partial = 0;  // of the 32 groups from i & ~31: those with slots that are not visible
    for (int i = 0; i < groups; ++i) {
      cp_wait<Sh::kStages - 2>();
      __syncwarp();
      load_group(i + Sh::kStages - 1, st_load);  // into the stage read last round
      cp_commit();
      const uint32_t k_at = k_lane + st * 2 * Sh::kPart, v_at = v_lane + st * 2 * Sh::kPart;
      st = st + 1 == Sh::kStages ? 0 : st + 1;
      st_load = st_load + 1 == Sh::kStages ? 0 : st_load + 1;
      if ((i & 31) == 0) {
        const int p = pos_of(i + lane);
        partial = __ballot_sync(FULL, !(seen(vis, p) && seen(vis, p + kGroup - 1)));
      }
      const int pos0 = pos_of(i);
      if (pos0 >= vis.n) continue;  // the last tile's groups past the end

      // S^T = K Q^T: 16 keys x 8 NT heads, even and odd steps apart
      float s[NT][4] = {}, s2[NT][4] = {};
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        uint32_t ak[4];
        ldsm4(ak, k_at ^ (k * 32));
        if (Sh::kQRegs) {
#pragma unroll
          for (int n = 0; n < NT; ++n) Pair<T>::mma(k & 1 ? s2[n] : s[n], ak, qf[k][n][0], qf[k][n][1]);
        } else {
          uint32_t bq[4];  // heads 0-7 and 8-15, 16 dimensions
          const int qr = (lane & 7) + ((lane >> 4) << 3), qh = (lane >> 3) & 1;
          ldsm4(bq, sm_q + qr * Sh::kRowBytes + (((2 * k + qh) ^ (qr & 7)) * 16));
#pragma unroll
          for (int n = 0; n < NT; ++n) Pair<T>::mma(k & 1 ? s2[n] : s[n], ak, bq[2 * n], bq[2 * n + 1]);
        }
      }
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[n][e] += s2[n][e];
      // keys pos0 + g4 and pos0 + g4 + 8 of this lane; whole groups need no test
      if (partial >> (i & 31) & 1) {
        const bool in0 = seen(vis, pos0 + g4), in1 = seen(vis, pos0 + g4 + 8);
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            s[n][e] = in0 ? s[n][e] : -INFINITY;
            s[n][2 + e] = in1 ? s[n][2 + e] : -INFINITY;
          }
      }
      if (scores) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            float *w = scores + (size_t)(pos0 + g4 + 8 * r) * a.G;
            const int c = 2 * t4 + 8 * n;
            if (pos0 + g4 + 8 * r < vis.n) {
              if (c < rows) w[c] = s[n][2 * r];
              if (c + 1 < rows) w[c + 1] = s[n][2 * r + 1];
            }
          }
      }
      // a score above the reference by more than the slack moves it
      bool up = false;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) up |= fmaxf(s[n][e], s[n][2 + e]) * sc > m[n][e] + (kBias<T> + kSlack<T>);
      if (__any_sync(FULL, up)) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float x = fmaxf(s[n][e], s[n][2 + e]) * sc;
#pragma unroll
            for (int w = 4; w < 32; w <<= 1) x = fmaxf(x, __shfl_xor_sync(FULL, x, w));
            x = fmaxf(x - kBias<T>, m[n][e]);
            // a head without a finite score yet has nothing to rescale
            const float f = x == -INFINITY ? 1.0f : ex2_approx(m[n][e] - x);
            m[n][e] = x;
            z[n][e] = x == -INFINITY ? 0.0f : x;
            l[n][e] *= f;
#pragma unroll
            for (int j = 0; j < D / 16; ++j) {
              o[j][n][e] *= f;
              o[j][n][2 + e] *= f;
            }
          }
      }
      // P^T as the sum of two 16-bit parts: the weights keep twice the type's
      // bits (one part alone would add a rounding as large as the output's own:
      // 2.2e-3 from 64 bits where bf16 rounds by 1.7e-3; it costs 1 % of the time)
      uint32_t ph[NT][2], pl[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const float x = ex2_approx(fmaf(s[n][2 * r], sc, -z[n][0]));
          const float y = ex2_approx(fmaf(s[n][2 * r + 1], sc, -z[n][1]));
          l[n][0] += x;
          l[n][1] += y;
          const uint32_t hi = Pair<T>::pack(x, y);
          const float2 back = Pair<T>::unpack(hi);
          ph[n][r] = transpose8(hi);
          pl[n][r] = transpose8(Pair<T>::pack(x - back.x, y - back.y));
        }
      // O^T += V^T P^T
#pragma unroll
      for (int j = 0; j < D / 16; ++j) {
        uint32_t av[4];
        ldsm4t(av, v_at ^ (j * 32));
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          Pair<T>::mma(o[j][n], av, ph[n][0], ph[n][1]);
          Pair<T>::mma(o[j][n], av, pl[n][0], pl[n][1]);
        }
      }
      __syncwarp();  // every lane is done with this stage before it is filled again
    }
    cp_wait<0>();

    // ------------------------------------------------------------ merge the warps
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int w = 4; w < 32; w <<= 1) l[n][e] += __shfl_xor_sync(FULL, l[n][e], w);
        if (g4 == 0) {
          s_m[warp][8 * n + 2 * t4 + e] = m[n][e];
          s_l[warp][8 * n + 2 * t4 + e] = l[n][e];
        }
      }
    bad = __any_sync(FULL, bad);
    if (lane == 0) s_bad[warp] = bad ? 1 : 0;
    __syncthreads();  // the ring is free too: O goes there
    float *mo = (float *)smem + (size_t)warp * Sh::kHeads * Sh::kMergeRow;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int c = 8 * n + 2 * t4 + e;
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) M = fmaxf(M, s_m[w][c]);
        const float f = m[n][e] == -INFINITY ? 0.0f : ex2_approx(m[n][e] - M);
#pragma unroll
        for (int j = 0; j < D / 16; ++j) {
          mo[c * Sh::kMergeRow + 16 * j + g4] = o[j][n][e] * f;
          mo[c * Sh::kMergeRow + 16 * j + 8 + g4] = o[j][n][2 + e] * f;
        }
      }
    uint32_t flag = vis.bad ? SV_ROW_BAD_LEN : 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w)
      if (s_bad[w]) flag |= SV_ROW_BAD_PAGE;
    __syncthreads();
    const float *mr = (const float *)smem;
    for (int i = threadIdx.x; i < rows * (D / 2); i += kThreads) {
      const int r = i / (D / 2), c = (i % (D / 2)) * 2;
      float x = 0.0f, y = 0.0f, sum = 0.0f, M = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float2 p = *(const float2 *)(mr + ((size_t)w * Sh::kHeads + r) * Sh::kMergeRow + c);
        x += p.x;
        y += p.y;
        M = fmaxf(M, s_m[w][r]);
      }
      // (a sum without a finite reference is 0, or NaN from the data: it stays)
#pragma unroll
      for (int w = 0; w < kWarps; ++w)
        sum += s_m[w][r] == -INFINITY ? s_l[w][r] : s_l[w][r] * ex2_approx(s_m[w][r] - M);
      if (whole) {
        const float nan = __int_as_float(0x7fffffff);
        const float inv = 1.0f / sum;
        x = flag ? nan : sum == 0.0f ? 0.0f : x * inv;
        y = flag ? nan : sum == 0.0f ? 0.0f : y * inv;
        *(uint32_t *)((T *)a.out + ((size_t)b * a.Hq + head0 + r) * D + c) = Pair<T>::pack(x, y);
        if (c == 0 && a.lse)
          a.lse[(size_t)b * a.Hq + head0 + r] =
              flag ? nan : sum == 0.0f ? -INFINITY : (M + log2f(sum)) * kLn2;
      } else {
        *(float2 *)(a.w_o + (part * a.rows + r) * D + c) = make_float2(x, y);
      }
      if (c == 0 && a.w_ml) a.w_ml[part * a.rows + r] = make_float2(M, sum);
    }
    if (threadIdx.x == 0) {
      if (a.w_flag) a.w_flag[part] = flag;
      if (whole && h == 0 && a.status) a.status[b] = flag;
    }
    if constexpr (!SHARING) return;
    share.first += max(tiles, 1);
    share.at = share.first;
    if (share.at >= share.end || ++share.b >= a.B) return;
    __syncthreads();  // the merge's rows are read: the ring is free
  }
}

// ---------------------------------------------------------------------------
// The end of a call that was split or sums weights.  CTAs below `joins`: the
// join, one query row of a (sequence, head group) with its units spread over
// the warps (wide), or a warp to each row (many sequences, few units each).
// The others: weight_sum += sum over the G query heads of 2^(s - m) / l, each
// visible slot by one thread, so no two add to one place; a thread has the scores
// of 4 slots on their way together (24 ragged sequences: 52.4 us, one after the
// other 53.6; 128 of 500-8000: 431 and 452).  Both find their units from the
// lengths (read past L1), and the sums so far, before they wait for the
// attention: it started after whatever wrote those had ended.
constexpr int kEndThreads = 256;
constexpr int kEndWarps = kEndThreads / 32;
constexpr int kSumKeys = 1024;  // positions of a CTA

// reference and sum of a row's units; every lane of the warp calls it
__device__ __forceinline__ float2 join_ml(const PagedArgs &a, const Plan &p, int h, int r, uint32_t &flag) {
  const unsigned FULL = 0xffffffffu;
  const int lane = threadIdx.x & 31;
  float M = -INFINITY, sum = 0.0f;
  flag = 0;
  for (int i = lane; i < p.n; i += 32) {
    const size_t u = (size_t)(p.first + i) * a.NH + h;
    const float2 ml = a.w_ml[u * a.rows + r];
    const float x = fmaxf(M, ml.x);
    sum = (M == -INFINITY ? sum : sum * ex2_approx(M - x)) + (ml.x == -INFINITY ? ml.y : ml.y * ex2_approx(ml.x - x));
    M = x;
    flag |= a.w_flag[u];
  }
  flag = __reduce_or_sync(FULL, flag);
  const float top = warp_max(M);
  sum = M == -INFINITY ? sum : sum * ex2_approx(M - top);
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(FULL, sum, o);
  return make_float2(top, sum);
}

template <typename T, int D>
__global__ void __launch_bounds__(kEndThreads) paged_finish_kernel(PagedArgs a, int joins, int wide, int key_ctas) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const float nan = __int_as_float(0x7fffffff);
  if ((int)blockIdx.x < joins) {
    const int at = wide ? blockIdx.x / a.rows : blockIdx.x;
    const int h = at % a.NH, b = at / a.NH;
    const Plan plan = find_plan<kEndThreads, false>(a, b);
    grid_dep_sync();
    if (plan.n == 1) return;  // written already
    const int hkv = h / a.gt, head0 = hkv * a.G + (h % a.gt) * kRows;
    const int rows = min(kRows, a.G - (h % a.gt) * kRows);
    __shared__ __align__(16) float s_o[kEndWarps][D];  // written in pairs
    constexpr int E = D / 32;
    for (int r = wide ? blockIdx.x % a.rows : warp; r < rows; r += wide ? kRows : kEndWarps) {
      uint32_t flag;
      const float2 ml = join_ml(a, plan, h, r, flag);
      float acc[E] = {};
#pragma unroll 4
      for (int i = wide ? warp : 0; i < plan.n; i += wide ? kEndWarps : 1) {
        const size_t u = (size_t)(plan.first + i) * a.NH + h;
        const float m = a.w_ml[u * a.rows + r].x;
        const float f = m == -INFINITY ? 0.0f : ex2_approx(m - ml.x);
        const float *src = a.w_o + (u * a.rows + r) * D + lane * 2;
#pragma unroll
        for (int e = 0; e < E; e += 2) {
          const float2 x = *(const float2 *)(src + e * 32);
          acc[e] += x.x * f;
          acc[e + 1] += x.y * f;
        }
      }
      const size_t row = (size_t)b * a.Hq + head0 + r;
      const float inv = 1.0f / ml.y;
      auto put = [&](int c, float x, float y) {
        x = flag ? nan : ml.y == 0.0f ? 0.0f : x * inv;
        y = flag ? nan : ml.y == 0.0f ? 0.0f : y * inv;
        *(uint32_t *)((T *)a.out + row * D + c) = Pair<T>::pack(x, y);
      };
      if (wide) {
#pragma unroll
        for (int e = 0; e < E; e += 2)
          *(float2 *)&s_o[warp][e * 32 + lane * 2] = make_float2(acc[e], acc[e + 1]);
        __syncthreads();
        for (int c = threadIdx.x * 2; c < D; c += kEndThreads * 2) {
          float x = 0.0f, y = 0.0f;
#pragma unroll
          for (int w = 0; w < kEndWarps; ++w) {
            x += s_o[w][c];
            y += s_o[w][c + 1];
          }
          put(c, x, y);
        }
      } else {
#pragma unroll
        for (int e = 0; e < E; e += 2) put(e * 32 + lane * 2, acc[e], acc[e + 1]);
      }
      if (lane == 0 && (!wide || warp == 0)) {
        if (a.lse) a.lse[row] = flag ? nan : ml.y == 0.0f ? -INFINITY : (ml.x + log2f(ml.y)) * kLn2;
        if (h == 0 && r == 0 && a.status) a.status[b] = flag;
      }
    }
    return;
  }
  const int at = blockIdx.x - joins;
  const int item = at / key_ctas, b = item / a.Hkv, hkv = item % a.Hkv;
  const Visible vis = visible(a, __ldcg(a.seq_len + b));
  int p0 = at % key_ctas * kSumKeys;
  if (vis.bad || p0 >= vis.n) {
    grid_dep_sync();
    return;
  }
  // the sums so far, before the wait too
  constexpr int kEach = kSumKeys / kEndThreads;  // slots of a thread
  float *sums = a.weight_sum + ((size_t)b * a.Hkv + hkv) * a.S;
  int to[kEach];
  float before[kEach];
  auto read_sums = [&]() {
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
      const int p = p0 + j * kEndThreads + (int)threadIdx.x;
      to[j] = p < vis.n && seen(vis, p) ? slot_of(vis, p) : -1;
      before[j] = to[j] >= 0 ? __ldcg(sums + to[j]) : 0.0f;
    }
  };
  read_sums();
  const Plan plan = find_plan<kEndThreads, false>(a, b);
  grid_dep_sync();
  // [G]: reference and 1 / sum of a row, apart: in one number, the log2 of the sum
  // of exponentials, a weight would be off by half a step of that number (2^-12 of
  // itself where scores lie about 4096; the output has no such error)
  extern __shared__ float2 s_ml[];
  __shared__ uint32_t s_flag;
  if (threadIdx.x == 0) s_flag = 0;
  __syncthreads();
  for (int g = warp; g < a.G; g += kEndWarps) {
    uint32_t flag;
    const float2 ml = join_ml(a, plan, hkv * a.gt + g / kRows, g % kRows, flag);
    if (lane == 0) {
      // without a finite score every exponential is 2^-inf: weights 0, or NaN from the data
      s_ml[g] = make_float2(ml.x == -INFINITY ? INFINITY : ml.x, ml.y == 0.0f ? 0.0f : 1.0f / ml.y);
      if (flag) s_flag = 1;
    }
  }
  __syncthreads();
  if (s_flag) return;
  for (;;) {
    float w[kEach] = {};
    const float *sc = a.w_score + (((size_t)b * a.Hkv + hkv) * a.vis_max + p0 + threadIdx.x) * a.G;
    for (int g = 0; g < a.G; g += a.G % 4 == 0 ? 4 : 1) {
      float4 x[kEach];
#pragma unroll
      for (int j = 0; j < kEach; ++j) {
        const float *at = sc + (size_t)j * kEndThreads * a.G + g;
        if (to[j] >= 0) x[j] = a.G % 4 == 0 ? *(const float4 *)at : make_float4(*at, 0.0f, 0.0f, 0.0f);
      }
#pragma unroll
      for (int j = 0; j < kEach; ++j) {
        if (to[j] < 0) continue;
        auto weight = [&](float s, const float2 &ml) { return ex2_approx(fmaf(s, a.scale_log2, -ml.x)) * ml.y; };
        w[j] += weight(x[j].x, s_ml[g]);
        if (a.G % 4 == 0)
          w[j] += weight(x[j].y, s_ml[g + 1]) + weight(x[j].z, s_ml[g + 2]) + weight(x[j].w, s_ml[g + 3]);
      }
    }
#pragma unroll
    for (int j = 0; j < kEach; ++j)
      if (to[j] >= 0) sums[to[j]] = before[j] + w[j];
    p0 += key_ctas * kSumKeys;
    if (p0 >= vis.n) return;
    read_sums();
  }
}

// ------------------------------------------------------------------ host side
struct Sizes {
  int G, gt, NH, rows, cap, vis_max;
  long long groups, units;  // of the grid; of the workspace, for all heads
  int finding;
  size_t map, first, o, ml, flag, score, total;
};

// false when the shape is beyond what the kernels index
bool sizes_of(Sizes &z, int B, int Hq, int Hkv, int D, int page, int max_pages, int window,
              int sinks, int weights) {
  z.G = Hq / Hkv;
  z.gt = (z.G + kRows - 1) / kRows;
  z.NH = Hkv * z.gt;
  z.rows = z.G < kRows ? z.G : kRows;
  const long long cap = (long long)page * max_pages;
  if (cap > kMaxSlots) return false;
  z.cap = (int)cap;
  // positions: a window and the first tokens start at multiples of 16 each
  long long most = cap;
  if (window > 0) {
    const long long w = ((long long)sinks + 2 * kGroup - 1) / kGroup * kGroup + window + kGroup;
    most = w < cap + 2 * kGroup ? w : cap + 2 * kGroup;
  }
  z.vis_max = (int)most;
  const long long tiles = (z.vis_max + kTile - 1) / kTile;
  const long long most_tiles = B * (tiles > 1 ? tiles : 1);
  const long long by_len = (long long)B * ((tiles + kMinTiles - 1) / kMinTiles);
  const long long by_units = (long long)B + units_for(D, B, z.NH) / z.NH;
  z.groups = by_len < by_units ? by_len : by_units;
  if (z.groups < B) z.groups = B;
  z.finding = z.groups == B ? kWhole : B == 1 ? kOne : 8LL * B * z.NH <= slots_of(D) ? kScan : kMap;
  z.units = z.groups * z.NH;
  if (z.finding == kMap && B <= kShareBatch && (long long)B * z.NH <= (long long)kShareHeads * slots_of(D) &&
      z.NH <= slots_of(D)) {
    z.finding = kShare;
    const long long by_slots = slots_of(D) / z.NH, by_tiles = most_tiles / kMinTiles;
    z.groups = by_tiles < 1 ? 1 : by_tiles < by_slots ? by_tiles : by_slots;
    z.units = (z.groups + B) * z.NH;
  }
  const long long rows = (long long)B * z.NH * kRows;  // CTAs of the join, at most
  if (z.units > 0x3fffffffLL || rows > 0x1fffffffLL || z.G > 8192) return false;
  const bool split = z.finding != kWhole;
  size_t at = 0;
  auto take = [&](size_t n) {
    const size_t r = at;
    at = align_up(at + n, 256);
    return r;
  };
  z.map = take(z.finding == kMap ? (size_t)z.groups * 16 : 0);
  z.first = take(z.finding == kMap ? (size_t)B * 8 : 0);
  z.o = take(split ? (size_t)z.units * z.rows * D * 4 : 0);
  z.ml = take(split || weights ? (size_t)z.units * z.rows * 8 : 0);
  z.flag = take(split || weights ? (size_t)z.units * 4 : 0);
  z.score = take(weights ? (size_t)B * Hq * z.vis_max * 4 : 0);
  z.total = at;
  return true;
}

template <typename T, int D, int NT, bool SHARING>
sv_status attend(const PagedArgs &a, const Sizes &z, cudaStream_t st) {
  static thread_local int set_dev = -1;
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev != set_dev) {
    const cudaError_t e =
        cudaFuncSetAttribute(paged_attn_kernel<T, D, NT, SHARING>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)Shape<D, NT>::kSmem);
    if (e != cudaSuccess) return check_launch("paged_attention", e);
    set_dev = dev;
  }
  LaunchScope ls("paged_attention", st);
  return check_launch("paged_attention",
                      launch_pdl(paged_attn_kernel<T, D, NT, SHARING>, dim3((unsigned)(z.groups * z.NH)),
                                 dim3(kThreads), Shape<D, NT>::kSmem, st, a));
}

template <typename T, int D>
sv_status run(const PagedArgs &a, const Sizes &z, bool weights, cudaStream_t st) {
  sv_status s = SV_OK;
  if (a.finding == kMap) {
    LaunchScope ls("paged_map", st);
    s = check_launch("paged_map", launch_pdl(paged_map_kernel, dim3(1), dim3(kMapThreads), 0, st, a));
    if (s != SV_OK) return s;
  }
  if (a.finding == kShare)
    s = z.rows <= 8 ? attend<T, D, 1, true>(a, z, st) : attend<T, D, 2, true>(a, z, st);
  else
    s = z.rows <= 8 ? attend<T, D, 1, false>(a, z, st) : attend<T, D, 2, false>(a, z, st);
  if (s != SV_OK) return s;
  const bool split = a.finding != kWhole;
  if (!split && !weights) return SV_OK;
  // a CTA to each row where a head has many units, spread over its warps (8
  // sequences of 8000: 53 us, with a warp to each 55); a warp to each row otherwise
  // (24 ragged ones: 51 us, with a CTA to each 53; 128 of 90-1110: 31 and 38)
  const int wide = 4LL * a.B * a.NH <= slots_of(D);
  const int joins = split ? a.B * a.NH * (wide ? a.rows : 1) : 0;
  // CTAs for a head's slots: as the table has room for, but no more in all than
  // the card runs a few times over (a table far longer than its sequences would
  // cost an empty CTA for each of its parts)
  const long long heads = (long long)a.B * a.Hkv, room = (4864 + heads - 1) / heads;
  const long long want = (z.vis_max + kSumKeys - 1) / kSumKeys;
  const int key_ctas = weights ? (int)(want < room ? want : room) : 0;
  const long long ctas = joins + key_ctas * heads;
  const size_t smem = weights ? (size_t)a.G * sizeof(float2) : 0;
  if (smem > 32 * 1024) {  // beside the join's 8 KB more than a kernel has unasked
    const cudaError_t e =
        cudaFuncSetAttribute(paged_finish_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return check_launch("paged_finish", e);
  }
  LaunchScope ls("paged_finish", st);
  return check_launch("paged_finish",
                      launch_pdl(paged_finish_kernel<T, D>, dim3((unsigned)ctas), dim3(kEndThreads),
                                 smem, st, a, joins, wide, key_ctas ? key_ctas : 1));
}

bool bad_shape(int B, int Hq, int Hkv, int D, int page, int max_pages, int window, int sinks) {
  return B < 0 || Hq < 1 || Hkv < 1 || Hq % Hkv || D < 1 || page < 1 || max_pages < 1 || window < 0 ||
         sinks < 0;
}

}  // namespace
}  // namespace sv

using namespace sv;

extern "C" size_t sv_paged_attention_workspace(int B, int Hq, int Hkv, int D, int page, int max_pages,
                                               int window, int sinks, int weights) {
  Sizes z;
  if (bad_shape(B, Hq, Hkv, D, page, max_pages, window, sinks) ||
      !sizes_of(z, B, Hq, Hkv, D, page, max_pages, window, sinks, weights))
    return 0;
  return z.total;
}

extern "C" sv_status sv_paged_attention(const void *q, const void *kv, int64_t kv_stride,
                                        int64_t page_stride, sv_dtype dt, const int32_t *block_table,
                                        const int32_t *seq_len, int B, int Hq, int Hkv, int D,
                                        int page, int max_pages, int num_pages, int window,
                                        int sinks, float scale, float *weight_sum, int S, void *out,
                                        float *out_lse, uint32_t *out_status, void *workspace,
                                        size_t workspace_bytes, void *stream) {
  if (bad_shape(B, Hq, Hkv, D, page, max_pages, window, sinks) || num_pages < 1)
    return set_error(SV_ERR_INVALID_ARG,
                     "need B >= 0, Hq a multiple of Hkv >= 1, page, max_pages, num_pages >= 1, "
                     "window >= 0 and sinks >= 0");
  if (dt != SV_BF16 && dt != SV_F16)
    return set_error(SV_ERR_INVALID_ARG, "the cache is SV_BF16 or SV_F16, not dtype %d", (int)dt);
  if (D != 64 && D != 128 && D != 256)
    return set_error(SV_ERR_UNSUPPORTED, "head dimension %d (64, 128 or 256)", D);
  if (!(scale > 0.0f) || !isfinite(scale * kLog2e))
    return set_error(SV_ERR_INVALID_ARG, "scale must be > 0 and finite");
  Sizes z;
  if (!sizes_of(z, B, Hq, Hkv, D, page, max_pages, window, sinks, weight_sum != nullptr))
    return set_error(SV_ERR_UNSUPPORTED, "more than 2^30 slots a sequence, or too many work units");
  const int64_t inner = (int64_t)page * Hkv * D;
  if (page_stride < inner || page_stride % 8 || kv_stride % 8 || kv_stride < 1 ||
      page_stride > INT64_MAX / 4 / num_pages || kv_stride > INT64_MAX / 4)
    return set_error(SV_ERR_INVALID_ARG,
                     "page_stride must cover a page (%lld elements), kv_stride be positive, and both "
                     "be multiples of 8",
                     (long long)inner);
  if (weight_sum && S < z.cap)
    return set_error(SV_ERR_INVALID_ARG, "weight_sum has %d slots a head, the page table %d", S, z.cap);
  if (B == 0) return SV_OK;
  if (!q || !kv || !block_table || !seq_len || !out)
    return set_error(SV_ERR_INVALID_ARG, "null pointer");
  if ((uintptr_t)q % 16 || (uintptr_t)kv % 16 || (uintptr_t)out % 16)
    return set_error(SV_ERR_INVALID_ARG, "q, kv and out need 16-byte alignment");
  if ((uintptr_t)block_table % 4 || (uintptr_t)seq_len % 4 || (uintptr_t)weight_sum % 4 ||
      (uintptr_t)out_lse % 4 || (uintptr_t)out_status % 4 || (uintptr_t)workspace % 256)
    return set_error(SV_ERR_INVALID_ARG, "misaligned pointer (the workspace needs 256 bytes)");
  if (workspace_bytes < z.total || (z.total && !workspace))
    return set_error(SV_ERR_INVALID_ARG, "workspace of %zu bytes, need %zu", workspace_bytes, z.total);
  if (!z.total) workspace = nullptr;
  sv_status s;
  if ((s = map_arg(q, "q")) != SV_OK || (s = map_arg(kv, "kv")) != SV_OK ||
      (s = map_arg(block_table, "block_table")) != SV_OK ||
      (s = map_arg(seq_len, "seq_len")) != SV_OK || (s = map_arg(out, "out")) != SV_OK ||
      (s = map_arg(weight_sum, "weight_sum")) != SV_OK ||
      (s = map_arg(out_lse, "out_lse")) != SV_OK || (s = map_arg(out_status, "out_status")) != SV_OK ||
      (s = map_arg(workspace, "workspace")) != SV_OK)
    return s;
  PagedArgs a;
  a.q = q;
  a.kv = kv;
  a.kv_stride = kv_stride;
  a.page_stride = page_stride;
  a.table = block_table;
  a.seq_len = seq_len;
  a.B = B;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.G = z.G;
  a.gt = z.gt;
  a.NH = z.NH;
  a.page = page;
  a.page_shift = -1;
  for (int i = 0; i < 31; ++i)
    if (page == 1 << i) a.page_shift = i;
  a.max_pages = max_pages;
  a.num_pages = num_pages;
  a.window = window;
  a.sinks = sinks;
  a.cap = z.cap;
  a.units = units_for(D, B, z.NH);
  a.scale_log2 = scale * kLog2e;
  a.rows = z.rows;
  a.vis_max = z.vis_max;
  a.weight_sum = weight_sum;
  a.S = S;
  a.out = out;
  a.lse = out_lse;
  a.status = out_status;
  char *w = (char *)workspace;
  const bool split = z.finding != kWhole, wt = weight_sum != nullptr;
  a.groups = (int)z.groups;
  a.finding = z.finding;
  a.w_map = z.finding == kMap ? (int4 *)(w + z.map) : nullptr;
  a.w_first = z.finding == kMap ? (int2 *)(w + z.first) : nullptr;
  a.w_o = split ? (float *)(w + z.o) : nullptr;
  a.w_ml = split || wt ? (float2 *)(w + z.ml) : nullptr;
  a.w_flag = split || wt ? (uint32_t *)(w + z.flag) : nullptr;
  a.w_score = wt ? (float *)(w + z.score) : nullptr;
  cudaStream_t st = (cudaStream_t)stream;
  if (dt == SV_BF16)
    return D == 64    ? run<__nv_bfloat16, 64>(a, z, wt, st)
           : D == 128 ? run<__nv_bfloat16, 128>(a, z, wt, st)
                      : run<__nv_bfloat16, 256>(a, z, wt, st);
  return D == 64    ? run<__half, 64>(a, z, wt, st)
         : D == 128 ? run<__half, 128>(a, z, wt, st)
                    : run<__half, 256>(a, z, wt, st);
}
