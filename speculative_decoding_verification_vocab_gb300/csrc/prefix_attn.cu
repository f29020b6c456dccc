// prefix_attn.cu -- attention of one new token per sequence for a batch whose
// sequences share long prefixes, each prefix read once for all (sm_103a).
//
// Many candidates of one prompt -- samples to choose from, drafts that are
// verified apart, users of one system prompt -- decode over the same first slots.
// With W sequences to a prefix and G = Hq / Hkv query heads to a KV head, W G
// query rows meet the same keys: a matrix product, on the 5th-generation tensor
// cores.  The slots of the prefix and a sequence's own ones are disjoint parts of
// its softmax, which join exactly: m = max(m1, m2), l = l1 2^(m1 - m) +
// l2 2^(m2 - m), and the same for the weighted sums of the values (scores in log2
// units).  Three launches: the prefixes' parts (here), the sequences' own slots
// (paged_attn.cu, its sums left unnormalised), the join.
//
// Bound: a slot of a prefix is 4 D bytes a KV head and 4 D W G operations: memory
// up to some 280 rows, above the tensor cores and the softmax's exponentials.
//
// Work: the query rows of a KV head (row r = sequence r / G, head r % G) are cut
// into columns of 256 (two tiles of 128), and a column's keys, of all prefixes and
// KV heads one after the other as a row of 128-key tiles, into equal shares, one for
// each of its CTAs: parts of a segment (prefix, KV head), whose sums go to the
// workspace.  The CTAs of the columns that have the same share are neighbours and
// read the same keys at the same time, once from memory (with a column's share
// beside the next column's instead, 7 times).  Shares are cut from the lengths on
// the device, so a captured launch follows growing prefixes.
// A CTA works on two S buffers in turn, so that the tensor cores have one while
// the softmax is at the other: those of the column's two query tiles with the
// same keys or, where the last column has one tile only, those of even and odd key
// tiles, which the join puts together like any two parts.
//   warps 0-1   producers, of K and of V: page table entries a tile ahead, TMA
//               boxes of 64 columns (128-byte swizzled) of as many rows as lie in a
//               page, a lane to each; pages behind the last are out of the map's
//               bounds and arrive as zeros.  Small pages and caches in host memory go
//               by asynchronous copies of 16 bytes (both warps both);
//   warps 2-3   MMA issuers, one to a buffer, so that one's waits lie behind the
//               other's products: S = Q K^T from shared memory, O += P V with P in
//               tensor memory, in the place of the S it comes from;
//   warps 4-11  softmax, four to a buffer, a row to a thread, 64 keys at a time: the
//               running maximum with a lazy rescale of O, P as 16-bit values (two for
//               each where there is one query tile); at a segment's end O, m and l to
//               the workspace.  The halves of a buffer take turns too: one is
//               multiplied and filled with the next tile's scores while the other is
//               worked on.
// Every wait on an mbarrier is bounded; one that runs out marks the CTA's parts
// with SV_ROW_TIMEOUT.
//
// 128 sequences with a prefix of 32600 slots, 64 query heads on 8 KV heads of 128: 110
// us for the prefix (1.24 PFLOP/s, 0.65; tensor pipe 53 % of the time: a pair of tiles is
// 2150 clocks of products and takes 3300, of which the softmax works 1700 on each and
// waits for the next scores, whose halves of 64 keys read Q twice from shared memory).
// With whole tiles in turn, the scores of the next behind the product of the last: 114;
// one S buffer: 367; two warps to a row of scores (16 of softmax): 142.  16 prefixes of
// 1500 to 9000 slots, 8 samples each, 32 heads on 8 of 64, weights in two parts: 57 us (3.9
// TB/s; a quarter of a query tile's rows are there, and a row's softmax takes as long for
// few).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>

#include "paged.cuh"
#include "tcgen05.cuh"

namespace sv {
namespace {

constexpr int kRows = 128;   // query rows of a tile = tensor-memory lanes
constexpr int kKeys = 128;   // rows of a tile of keys, of which a call uses a.keys
constexpr int kProducers = 64;
constexpr int kMmaWarp = kProducers / 32, kFirstSoftmax = kMmaWarp + 2;
// 12 warps: registers are given out to four warps at a time, and the softmax needs
// more than the 128 that 13 to 16 leave a thread
constexpr int kThreads = kProducers + 64 + 256;
constexpr uint32_t kBox = kKeys * 128;  // bytes of a box of 64 columns
constexpr float kLn2 = 0.693147180559945309f, kLog2e = 1.4426950408889634f;
// tensor-memory columns: two S (P, 16-bit pairs, in their first halves), two O
constexpr uint32_t kColS = 0, kColO = 256, kTmemCols = 512;

// A score moves the reference only when it is more than kSlack above it (log2
// units).  Weights go into the product as 16-bit numbers: in fp16 the reference
// lies 2^kBias below the maximum it was set by, so that they fill the type's range
// from the top (2^15 at most) and the small ones do not round to nothing.
// TWO: a weight is the sum of two 16-bit parts, so that it keeps twice the type's bits,
// as in the paged attention; one part alone (half a step, 2^-8 or 2^-11, of each weight,
// independent from key to key) adds a rounding as large as the output's own (bf16:
// 2.2e-3 from 64 bits, where rounding the output leaves 1.65e-3).  For one query tile,
// where the product is not the bound, it costs 4 to 10 % of the call (4 prefixes of 20000
// slots, 64 heads on 8 of 128: 4 sequences each 71 and 74 us, 16 each 87 and 90; one of
// them, from L2, 33 and 36; 16 of 5000, 32 on 8 of 64, fp16, pages of 20: 59 and 65).
// Beyond 128 rows the product is the bound, and the call 15 to 22 % longer with a second
// part (32 sequences each 103 and 118 us; 128 behind 32600 slots 131 and 159): one part.
template <typename T> constexpr float kSlack = 8.0f;
template <typename T> constexpr float kBias = 0.0f;
template <> constexpr float kSlack<__half> = 4.0f;
template <> constexpr float kBias<__half> = 11.0f;
template <typename T> constexpr uint32_t kAbType = 1;  // of the instruction descriptor: bf16
template <> constexpr uint32_t kAbType<__half> = 0;

template <typename T> __device__ __forceinline__ uint32_t pack2(float lo, float hi);
template <typename T> __device__ __forceinline__ unsigned long long unpack2(uint32_t v);
template <> __device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float lo, float hi) { return pack_bf16(lo, hi); }
template <> __device__ __forceinline__ unsigned long long unpack2<__nv_bfloat16>(uint32_t v) { return f2_pack(bf16_lo(v), bf16_hi(v)); }
template <> __device__ __forceinline__ unsigned long long unpack2<__half>(uint32_t v) {
  const float2 f = __half22float2(*(const __half2 *)&v);
  return f2_pack(f.x, f.y);
}
template <> __device__ __forceinline__ uint32_t pack2<__half>(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *(const uint32_t *)&v;
}

// A barrier tells one phase from the next by its parity alone, so whoever waits for a
// phase has to know that the one before is over.  K and V have places of their own,
// each filled by one producer, which has waited for every phase in turn; and the
// places are even in number, so that where the buffers take even and odd tiles a
// place is one buffer's, whose issuer has seen all of its phases.  (With K and V in
// one ring an issuer a tile and a half ahead of the other let K be loaded into a
// place that was still to be read: the launch failed.)
template <int D> struct Ring {
  static constexpr uint32_t kTileBytes = kKeys * D * 2;  // K or V rows of a key tile, or a query tile
  static constexpr int kK = D == 128 ? 2 : 4, kV = D == 128 ? 2 : 6;  // places
  static_assert(kK % 2 == 0 && kV % 2 == 0, "places of even and odd tiles");
  static constexpr uint32_t kOffV = kK * kTileBytes;
  static constexpr uint32_t kOffQ = kOffV + kV * kTileBytes;
  static constexpr uint32_t kOffBar = kOffQ + 2 * kTileBytes;
  static constexpr uint32_t kOffMisc = kOffBar + 40 * 8;
  static constexpr size_t kSmem = kOffMisc + 128 + 1024;  // + alignment
  // barriers: a place of K or V filled and free; by buffer: Q there; by half of a
  // buffer (2 s + half): S there, P there, its PV done
  static constexpr int kFullK = 0, kFreeK = kK, kFullV = 2 * kK, kFreeV = kFullV + kV, kQ = kFreeV + kV, kS = kQ + 2,
                       kP = kS + 4, kPV = kP + 4, kCount = kPV + 4;
  static_assert(kCount <= 40, "barriers");
};

template <int V> struct Int {
  static constexpr int value = V;
};

struct PrefixArgs {
  const void *q, *kv;
  int64_t kv_stride, page_stride;
  const int32_t *table, *len;  // [N][max_pages], [N]
  int B, N, W, Hq, Hkv, G, mtiles;  // query tiles of a KV head
  int page, page_shift, max_pages, num_pages, cap;
  int keys, box;  // keys of a tile; rows of a TMA box
  int shares2, shares1, rows;  // CTAs of a column of two tiles, and of one; rows of a part's buffer: min(128, W G)
  float scale_log2;
  // workspace: sums [parts][2][rows][D], references and sums of exponentials
  // [parts][2][rows], status bits [parts]
  float *w_o;
  float2 *w_ml;
  uint32_t *w_flag;
  uint32_t *status;  // [B], or null
};

__device__ __forceinline__ int tiles_of(const PrefixArgs &a, int len) {
  return len < 0 || len > a.cap ? 0 : (int)(((unsigned)len + (unsigned)a.keys - 1) / (unsigned)a.keys);
}
// tiles of all prefixes and of those before p, over the lanes of a warp
__device__ __forceinline__ longlong2 count_tiles(const PrefixArgs &a, int p) {
  longlong2 n = make_longlong2(0, 0);
  if (a.N == 1) {
    n.x = tiles_of(a, __ldcg(a.len));
    return n;
  }
  for (int i = threadIdx.x & 31; i < a.N; i += 32) {
    const int t = tiles_of(a, __ldcg(a.len + i));
    n.x += t;
    n.y += i < p ? t : 0;
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    n.x += __shfl_xor_sync(0xffffffffu, n.x, o);
    n.y += __shfl_xor_sync(0xffffffffu, n.y, o);
  }
  return n;
}

// Shares of a column that so many tiles are cut into: none without one.
__device__ __forceinline__ long long cut_into(long long shares, long long tiles) {
  return min(shares, max(tiles, 1LL));
}
// The share that tile t is in.
__device__ __forceinline__ int share_of(long long t, long long shares, long long tiles) {
  const unsigned long long x = (unsigned long long)(t + 1) * shares - 1;
  return x >> 32 || tiles >> 32 ? (int)(x / (unsigned long long)tiles) : (int)((uint32_t)x / (uint32_t)tiles);
}
// Part of a column's share r in segment sg: from part to part of a column one or
// the other grows.
__device__ __forceinline__ size_t part_at(const PrefixArgs &a, int column, long long r_sg) {
  return (size_t)column * (max(a.shares2, a.shares1) + (size_t)a.N * a.Hkv) + r_sg;
}

// A CTA's way through its share: the part of a segment it is at, tiles [t0, t1).
struct Walk {
  long long at, end, first;  // tiles of the column; the first of prefix p's segments
  int column, share, pair;   // pair: two query tiles, 2 column and 2 column + 1
  int p, head, t0, t1, len, base;
  __device__ __forceinline__ bool next(const PrefixArgs &a) {
    base += t1 - t0;
    while (at < end && p < a.N) {
      len = __ldcg(a.len + p);
      const int tiles = tiles_of(a, len);
      const long long block = (long long)tiles * a.Hkv;
      if (at < first + block) {
        head = (int)((at - first) / tiles);
        t0 = (int)((at - first) % tiles);
        t1 = (int)min((long long)tiles, t0 + (end - at));
        at += t1 - t0;
        return true;
      }
      first += block;
      ++p;
    }
    t0 = t1;
    return false;
  }
  __device__ __forceinline__ size_t part(const PrefixArgs &a) const {
    return part_at(a, column, (long long)share + (long long)p * a.Hkv + head);
  }
  // Tiles of buffer s: all of a pair's, or every other one, by the CTA's count of
  // tiles (`base` before this part); the first of them, and how many.
  __device__ __forceinline__ int first_for(int s) const { return pair ? t0 : t0 + ((s ^ base) & 1); }
  __device__ __forceinline__ int tiles_for(int s) const {
    return pair ? t1 - t0 : (t1 - first_for(s) + 1) >> 1;
  }
};

// 5-D tiled TMA load of one box into shared memory, completing on `bar`.
__device__ __forceinline__ void tma_load5(uint32_t dst, const CUtensorMap *map, int x, int h, int r, int page, int kv,
                                          uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(dst),
      "l"((uint64_t)map), "r"(x), "r"(h), "r"(r), "r"(page), "r"(kv), "r"(bar)
      : "memory");
}
// D = A B with both operands in shared memory
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
// 32 consecutive columns of this thread's tensor-memory lane; the values are there
// after tm_wait_ld
__device__ __forceinline__ void tm_ld32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
// (the registers pass through, so that nothing reads them before the wait)
__device__ __forceinline__ void tm_wait_ld(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]),
                 "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]),
                 "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]),
                 "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]),
                 "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}
__device__ __forceinline__ void tm_st16(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15,%16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
__device__ __forceinline__ void tm_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

template <typename T, int D, bool TMA, bool TWO>
__global__ void __launch_bounds__(kThreads, 1)
    prefix_attn_kernel(const __grid_constant__ CUtensorMap map, PrefixArgs a) {
  using R = Ring<D>;
  constexpr int kK = R::kK, kV = R::kV;
  constexpr uint32_t kTileBytes = R::kTileBytes;
  const unsigned FULL = 0xffffffffu;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *sm = (uint8_t *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint64_t *bars = (uint64_t *)(sm + R::kOffBar);
  uint32_t *tmem_slot = (uint32_t *)(sm + R::kOffMisc);
  volatile int *abort = (volatile int *)(sm + R::kOffMisc + 4);
  Walk *s_walk = (Walk *)(sm + R::kOffMisc + 8);
  volatile int *s_filled = (volatile int *)(sm + R::kOffMisc + 8 + sizeof(Walk));  // tiles, by producer warp
  static_assert(8 + sizeof(Walk) + 8 <= 128, "misc");
  const uint32_t bar0 = smem_addr(bars), sm0 = smem_addr(sm);
  auto bar = [&](int i) { return bar0 + 8u * (uint32_t)i; };

  if (threadIdx.x == 0) {
    // a place is free when both buffers' products are done with it, or that of the
    // one it is for
    const int users = blockIdx.x < a.mtiles / 2 * a.shares2 ? 2 : 1;
    for (int i = 0; i < kK; ++i) {
      mbar_init(bar(R::kFullK + i), TMA ? 1 : kProducers);
      mbar_init(bar(R::kFreeK + i), users);
    }
    for (int i = 0; i < kV; ++i) {
      mbar_init(bar(R::kFullV + i), TMA ? 1 : kProducers);
      mbar_init(bar(R::kFreeV + i), users);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar(R::kQ + s), 4);
      for (int half = 0; half < 2; ++half) {
        mbar_init(bar(R::kS + 2 * s + half), 1);
        mbar_init(bar(R::kP + 2 * s + half), 4);
        mbar_init(bar(R::kPV + 2 * s + half), 1);
      }
    }
    *abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(tmem_slot)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (TMA && a.keys < kKeys) {
    // rows of V that no box reaches: zeros, for weights of 0 to multiply
    const int rows = kKeys - a.keys, per = rows * 8;  // 16-byte pieces of a box
    for (int i = threadIdx.x; i < kV * (D / 64) * per; i += kThreads) {
      const int b = i / per, e = i % per;
      *(uint4 *)(sm + R::kOffV + b * kBox + a.keys * 128 + e * 16) = make_uint4(0, 0, 0, 0);
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  grid_dep_sync();
  if (a.status)  // for the join's bits
    for (int b = blockIdx.x * kThreads + threadIdx.x; b < a.B; b += gridDim.x * kThreads) a.status[b] = 0;
  if (warp == 0) {
    // this CTA's column and share, and the prefix it starts in
    Walk w;
    const int columns2 = a.mtiles / 2, cta = blockIdx.x;
    w.pair = cta < columns2 * a.shares2;
    w.column = w.pair ? cta % columns2 : columns2;
    w.share = w.pair ? cta / columns2 : cta - columns2 * a.shares2;
    const long long per = a.Hkv, all = per * count_tiles(a, 0).x, shares = cut_into(w.pair ? a.shares2 : a.shares1, all);
    w.at = min((long long)w.share, shares) * all / shares;
    w.end = min((long long)w.share + 1, shares) * all / shares;
    w.first = 0;
    w.p = w.base = w.t0 = w.t1 = 0;
    for (int p0 = 0; p0 < a.N && w.at < w.end; p0 += 32) {
      const int p = p0 + lane;
      const long long n = p < a.N ? per * tiles_of(a, __ldcg(a.len + p)) : 0;
      long long incl = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(FULL, incl, o);
        if (lane >= o) incl += x;
      }
      const unsigned past = __ballot_sync(FULL, w.first + incl > w.at);
      if (past) {
        const int l = __ffs(past) - 1;
        w.p = p0 + l;
        w.first += __shfl_sync(FULL, incl - n, l);
        break;
      }
      w.first += __shfl_sync(FULL, incl, 31);
    }
    if (lane == 0) *s_walk = w;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  Walk w = *s_walk;
  auto all = [&](bool x) { return __all_sync(FULL, x) != 0; };

  if (TMA && warp < kMmaWarp) {
    // ------------------------------------------------------------ producers
    // Warp 0 loads K, warp 1 V; a lane to each box of a tile.
    const int boxes = a.keys / a.box;
    const uint32_t bytes = (uint32_t)a.keys * D * 2;
    const int places = warp ? kV : kK, full = warp ? R::kFullV : R::kFullK, free = warp ? R::kFreeV : R::kFreeK;
    int t_all = 0, at = 0;  // tiles so far, and the next one's place
    uint32_t seen = 1;      // parity of the phase that frees it
    bool ok = true;
    while (w.next(a)) {
      bool bad = false;
      const int32_t *table = a.table + (size_t)w.p * a.max_pages;
      auto fetch = [&](int t) {
        const int slot = t * a.keys + lane * a.box;
        return lane < boxes && t < w.t1 && slot < w.len
                   ? __ldg(table + (a.page_shift >= 0 ? slot >> a.page_shift : slot / a.page))
                   : -1;
      };
      int id = fetch(w.t0);
      for (int t = w.t0; ok && t < w.t1; ++t, ++t_all) {
        const int slot = t * a.keys + lane * a.box, r = a.page_shift >= 0 ? slot & (a.page - 1) : slot % a.page;
        const bool there = (unsigned)id < (unsigned)a.num_pages;
        bad |= lane < boxes && slot < w.len && !there;
        const int page = there ? id : a.num_pages;  // out of bounds: zeros
        id = fetch(t + 1);
        ok = all(t_all < places || mbar_wait(bar(free + at), seen, abort));
        if (!ok) break;
        if (lane == 0) mbar_expect_tx(bar(full + at), bytes);
        __syncwarp();
        if (lane < boxes) {
          const uint32_t dst = sm0 + (warp ? R::kOffV : 0) + at * kTileBytes + lane * a.box * 128;
#pragma unroll
          for (int c = 0; c < D / 64; ++c)
            tma_load5(dst + c * kBox, &map, c * 64, w.head, r, page, warp, bar(full + at));
        }
        if (++at == places) {
          at = 0;
          seen ^= 1;
        }
      }
      if (warp == 0) {
        bad = __any_sync(FULL, bad);
        if (lane == 0) a.w_flag[w.part(a)] = bad ? SV_ROW_BAD_PAGE : 0u;
      }
    }
    if (lane == 0) s_filled[warp] = t_all;
  } else if (warp < kMmaWarp) {
    // ------------------------------------------------------------ producer
    // Warp w fills rows 64 w to 64 w + 63 of every tile: lane l looks rows l and l +
    // 32 of them up, one tile ahead; CPR lanes copy a row, 16 bytes each.  A place is
    // full when the copies of all producers into it have arrived.
    constexpr int CPR = D / 8, RPI = 32 / CPR;  // rows of one round of copies
    const int lr = lane / CPR, lc = lane % CPR;
    const int64_t row_elems = (int64_t)a.Hkv * D;
    int t_all = 0;  // tiles so far
    bool ok = true;
    while (w.next(a)) {
      bool bad = false;
      const T *kv = (const T *)a.kv + (int64_t)w.head * D + lc * 8;
      const int32_t *table = a.table + (size_t)w.p * a.max_pages;
      auto slot_of = [&](int t, int e) { return t * kKeys + warp * 64 + e * 32 + lane; };
      int id[2];
      auto fetch = [&](int t) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int slot = slot_of(t, e);
          id[e] = t < w.t1 && slot < w.len ? __ldg(table + (a.page_shift >= 0 ? slot >> a.page_shift : slot / a.page)) : -1;
        }
      };
      fetch(w.t0);
      for (int t = w.t0; ok && t < w.t1; ++t, ++t_all) {
        long long off[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int slot = slot_of(t, e);
          off[e] = -1;
          if (slot < w.len) {
            if ((unsigned)id[e] < (unsigned)a.num_pages) {
              const int in_page = a.page_shift >= 0 ? slot & (a.page - 1) : slot % a.page;
              off[e] = id[e] * (long long)a.page_stride + in_page * (long long)row_elems;
            } else {
              bad = true;
            }
          }
        }
        fetch(t + 1);
#pragma unroll
        for (int part = 0; part < 2; ++part) {  // K, V
          const int places = part ? kV : kK, at = t_all % places;
          ok = all(t_all < places ||
                   mbar_wait(bar((part ? R::kFreeV : R::kFreeK) + at), (t_all / places - 1) & 1, abort));
          if (!ok) break;
          const T *from = kv + part * a.kv_stride;
          const uint32_t dst = sm0 + (part ? R::kOffV : 0) + at * kTileBytes + (lc >> 3) * kBox + (warp * 64 + lr) * 128;
#pragma unroll 8
          for (int i = 0; i < 64 / RPI; ++i) {
            const long long o = __shfl_sync(FULL, i < 32 / RPI ? off[0] : off[1], (i * RPI + lr) & 31);
            const uint32_t d = dst + i * RPI * 128 + (((lc & 7) ^ ((i * RPI + lr) & 7)) << 4);
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(d), "l"(from + (o >= 0 ? o : 0)),
                         "r"(o >= 0 ? 16u : 0u)
                         : "memory");
          }
          asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar((part ? R::kFullV : R::kFullK) + at))
                       : "memory");
        }
      }
      // the part's status: a barrier of the producers with their votes, which they
      // all come to, whatever became of their waits
      uint32_t some;
      asm volatile(
          "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n bar.red.or.pred q, 1, %2, p;\n selp.u32 %0, 1, 0, q;\n}"
          : "=r"(some)
          : "r"((uint32_t)bad), "n"(kProducers)
          : "memory");
      if (threadIdx.x == 0) a.w_flag[w.part(a)] = some ? SV_ROW_BAD_PAGE : 0u;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else if (warp < kFirstSoftmax) {
    // ------------------------------------------------------------ MMA
    // A buffer's tiles in turn, 64 keys at a time: S of both halves of the first, then,
    // half by half, O += P V and the next tile's S into the place of P, while the
    // softmax is at the other half.  The warp runs converged and elect.sync picks the
    // issuing lane.
    const int s = warp - kMmaWarp;
    constexpr uint32_t kIdesc = (1u << 4) | (kAbType<T> << 7) | (kAbType<T> << 10) | ((uint32_t)(kRows >> 4) << 24);
    constexpr uint32_t kIdescS = kIdesc | ((uint32_t)(kKeys / 2 >> 3) << 17);
    constexpr uint32_t kIdescO = kIdesc | (1u << 16) | ((uint32_t)(D >> 3) << 17);  // V: head dim contiguous
    constexpr uint64_t kStep = kTileBytes >> 4;
    const uint64_t dK0 = sdesc(sm0, 16, 1024), dV0 = sdesc(sm0 + R::kOffV, kBox, 1024);
    const uint64_t dq = sdesc(sm0 + R::kOffQ + s * kTileBytes, 16, 1024);
    const uint32_t tS = tmem + kColS + s * 128, tO = tmem + kColO + s * D;
    // The places of the next tile's K and V, and the phases that fill them.  (Kept,
    // not divided out: this warp's own instructions stand between the products.)
    const int step = w.pair ? 1 : 2, first = w.pair ? 0 : s;
    int k_at = first, v_at = first;
    uint32_t k_phase = 0, v_phase = 0;
    uint32_t nq = 0, ns[2] = {0, 0}, done[2] = {0, 0};  // query tiles; S and PV products so far, by half
    bool ok = true;
    auto landed = [&](int full, uint32_t phase) {
      const bool r = all(mbar_wait(bar(full), phase, abort));
      if (!TMA) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the generic proxy's copies
      return r;
    };
    while (ok && w.next(a)) {
      const int n = w.tiles_for(s);
      auto issue_s = [&](auto which) {  // once its K has landed and the product that read P there is done
        constexpr int half = decltype(which)::value;
        ok = (half || landed(R::kFullK + k_at, k_phase)) &&
             all(done[half] == 0 || mbar_wait(bar(R::kPV + 2 * s + half), (done[half] - 1) & 1, abort));
        if (!ok) return;
        tc_fence_after();
        if (elect_one()) {
          const uint64_t dk = dK0 + k_at * kStep + (half ? 64 * 128 >> 4 : 0);
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks) {
            const uint64_t at = (uint64_t)(((ks >> 2) * kBox + (ks & 3) * 32) >> 4);
            mma_ss(tS + 64 * half, dq + at, dk + at, kIdescS, ks > 0);
          }
          mma_commit(bar(R::kS + 2 * s + half));
          if (half) mma_commit(bar(R::kFreeK + k_at));
        }
        __syncwarp();
        if (half && (k_at += step) >= kK) {
          k_at -= kK;
          k_phase ^= 1;
        }
        ++ns[half];
      };
      if (n > 0) {
        ok = all(mbar_wait(bar(R::kQ + s), nq++ & 1, abort));
        if (!ok) break;
        tc_fence_after();
        issue_s(Int<0>());
        if (ok) issue_s(Int<1>());
      }
      for (int i = 0; ok && i < n; ++i) {
        ok = landed(R::kFullV + v_at, v_phase);
        if (!ok) break;
        // The last tile's product takes the steps of 16 keys that hold one; a box
        // may bring rows behind the last key, which may hold anything: zeros there
        // (from both issuers), so that weights of 0 add 0.
        const int left = w.len - (w.first_for(s) + i * step) * a.keys;
        const int steps = (min(left, a.keys) + 15) >> 4;
        if (TMA && left < a.keys && (left & 15)) {
          const int at = left + (lane >> 1);
          if (at < 16 * steps) {
            uint8_t *v = sm + R::kOffV + v_at * kTileBytes + at * 128 + (lane & 1) * 64;
#pragma unroll
            for (int c = 0; c < D / 64; ++c)
#pragma unroll
              for (int e = 0; e < 4; ++e) *(uint4 *)(v + c * kBox + e * 16) = make_uint4(0, 0, 0, 0);
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
        }
        const uint64_t dv = dV0 + v_at * kStep;
        auto multiply = [&](auto which) {
          constexpr int half = decltype(which)::value;
          ok = all(mbar_wait(bar(R::kP + 2 * s + half), done[half] & 1, abort));
          if (!ok) return;
          tc_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int ks = 4 * half; ks < 4 * half + 4; ++ks)
              if (ks < steps) {
                const uint32_t p = tS + 64 * half + (ks - 4 * half) * 8;
                mma_ts(tO, p, dv + (uint64_t)(ks * 128), kIdescO, (i > 0 || ks > 0) ? 1u : 0u);
                if (TWO) mma_ts(tO, p + 32, dv + (uint64_t)(ks * 128), kIdescO, 1u);
              }
            mma_commit(bar(R::kPV + 2 * s + half));
            if (half) mma_commit(bar(R::kFreeV + v_at));
          }
          __syncwarp();
          ++done[half];
          if (i + 1 < n) issue_s(which);
        };
        multiply(Int<0>());
        if (ok) multiply(Int<1>());
        if (!ok) break;
        if ((v_at += step) >= kV) {
          v_at -= kV;
          v_phase ^= 1;
        }
      }
    }
    if (!ok) {
      // products in flight end before tensor memory is released: the newest phases
      // of the barriers that the last ones commit to
      volatile int no_abort = 0;
      for (int half = 0; half < 2; ++half) {
        if (ns[half]) mbar_wait(bar(R::kS + 2 * s + half), (ns[half] - 1) & 1, &no_abort);
        if (done[half]) mbar_wait(bar(R::kPV + 2 * s + half), (done[half] - 1) & 1, &no_abort);
      }
    }
  } else {
    // ------------------------------------------------------------ softmax
    // Four warps to a buffer; a thread has the query row of its tensor-memory lane.
    const int s = (warp - kFirstSoftmax) >> 2, quarter = warp & 3, row = quarter * 32 + lane;
    const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
    const uint32_t tS = tmem + lanes + kColS + s * 128, tO = tmem + lanes + kColO + s * D;
    int g = 0;  // tiles of this buffer so far
    bool ok = true;
    while (ok && w.next(a)) {
      const int mt = 2 * w.column + (w.pair ? s : 0), n = w.tiles_for(s);
      const int rows = min(kRows, a.W * a.G - mt * kRows);
      if (n > 0) {
        // This row of the query tile; rows behind the last are zeros.  (A buffer
        // without a tile takes no query: nothing would hold its warps back until
        // the last one had been seen.)
        const int at = mt * kRows + row;
        const uint4 *src = (const uint4 *)((const T *)a.q +
                                           (((size_t)w.p * a.W + at / a.G) * a.Hq + (size_t)w.head * a.G + at % a.G) * D);
        uint8_t *dst = sm + R::kOffQ + s * kTileBytes + row * 128;
#pragma unroll
        for (int c = 0; c < D / 8; ++c)
          *(uint4 *)(dst + (c >> 3) * kBox + (((c & 7) ^ (row & 7)) << 4)) =
              row < rows ? __ldg(src + c) : make_uint4(0, 0, 0, 0);
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(R::kQ + s));
      }
      float m_ref = -INFINITY;  // log2 units
      unsigned long long l2[2] = {0ull, 0ull};
      int behind = w.len - w.first_for(s) * a.keys;  // keys from this tile's first to the last
      const int stride = w.pair ? a.keys : 2 * a.keys;
      uint32_t x[4][32];
      auto ask = [&](auto which) {  // a half's scores
        constexpr int c = 2 * decltype(which)::value;
        tc_fence_after();
        tm_ld32(tS + 32 * c, x[c]);
        tm_ld32(tS + 32 * c + 32, x[c + 1]);
      };
      auto get = [&](auto which) {
        constexpr int c = 2 * decltype(which)::value;
        tm_wait_ld(x[c]);
        tm_wait_ld(x[c + 1]);
      };
      if (n > 0) {
        ok = all(mbar_wait(bar(R::kS + 2 * s), g & 1, abort));
        if (!ok) break;
        ask(Int<0>());
        get(Int<0>());
      }
      for (int i = 0; i < n; ++i, ++g, behind -= stride) {
        const int left = min(behind, a.keys);  // keys of this tile
        auto do_half = [&](auto which) -> bool {
          constexpr int half = decltype(which)::value;
          if (left < 64 * half + 64) {
#pragma unroll
            for (int c = 2 * half; c < 2 * half + 2; ++c)
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (32 * c + e >= left) x[c][e] = 0xff800000u;
          }
          float v[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int c = 2 * half; c < 2 * half + 2; ++c)
#pragma unroll
            for (int e = 0; e < 32; e += 2)
              v[e / 2 & 3] = max3(v[e / 2 & 3], __uint_as_float(x[c][e]), __uint_as_float(x[c][e + 1]));
          // scale > 0: the maximum commutes with it
          const float mx = fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3])) * a.scale_log2;
          const bool grow = mx > m_ref + (kSlack<T> + kBias<T>);
          const float m_new = grow ? mx - kBias<T> : m_ref;
          const float factor = grow && m_ref != -INFINITY ? ex2_approx(m_ref - m_new) : 1.0f;
          m_ref = m_new;
          if (__any_sync(FULL, factor != 1.0f)) {
            // O covers the keys before: the product of the half before is waited for (a
            // segment's first half finds no reference to move)
            if (!all(mbar_wait(bar(R::kPV + 2 * s + 1 - half), (half ? g : g - 1) & 1, abort))) return false;
            tc_fence_after();
            l2[0] = f2_mul(l2[0], f2_splat(factor));
            l2[1] = f2_mul(l2[1], f2_splat(factor));
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
              uint32_t o[32];
              tm_ld32(tO + c, o);
              tm_wait_ld(o);
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * factor);
              tm_st32u(tO + c, o);
            }
          }
          const unsigned long long sc2 = f2_splat(a.scale_log2), mn2 = f2_splat(m_ref == -INFINITY ? 0.0f : -m_ref);
#pragma unroll
          for (int c = 2 * half; c < 2 * half + 2; ++c) {
            uint32_t p[16], rest[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const unsigned long long y =
                  ex2_2(f2_fma(f2_pack(__uint_as_float(x[c][2 * e]), __uint_as_float(x[c][2 * e + 1])), sc2, mn2));
              l2[e & 1] = f2_add(l2[e & 1], y);
              float y0, y1;
              f2_unpack(y, y0, y1);
              p[e] = pack2<T>(y0, y1);
              if (TWO) {
                f2_unpack(f2_sub(y, unpack2<T>(p[e])), y0, y1);
                rest[e] = pack2<T>(y0, y1);
              }
            }
            tm_st16(tS + 64 * half + 16 * (c - 2 * half), p);  // in the place of keys that have been read
            if (TWO) tm_st16(tS + 64 * half + 32 + 16 * (c - 2 * half), rest);
          }
          auto done = [&]() {
            tm_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(R::kP + 2 * s + half));
          };
          // The next half's scores are on their way meanwhile, where they are there.
          // (Nothing but the wait stands between a load and its registers' use, a copy
          // of them at a join of two ways included.)
          const Int<1 - half> next;
          const uint32_t s_bar = bar(R::kS + 2 * s + 1 - half);
          const uint32_t s_phase = (half ? g + 1 : g) & 1;
          if (half && i + 1 == n) {
            done();
#pragma unroll
            for (int e = 0; e < 64; ++e) x[e >> 5][e & 31] = 0;  // (the old ones are not kept)
          } else if (all(mbar_test(s_bar, s_phase))) {
            ask(next);
            done();
            get(next);
          } else {
            done();
            if (!all(mbar_wait(s_bar, s_phase, abort))) return false;
            ask(next);
            get(next);
          }
          return true;
        };
        ok = do_half(Int<0>()) && do_half(Int<1>());
        if (!ok) break;
      }
      if (!ok) break;
      const size_t at = (w.part(a) * 2 + s) * a.rows + row;
      if (n > 0) {
        ok = all(mbar_wait(bar(R::kPV + 2 * s + 1), (g - 1) & 1, abort));
        if (!ok) break;
        tc_fence_after();
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          uint32_t o[32];
          tm_ld32(tO + c, o);
          tm_wait_ld(o);
          if (row < rows) {
            uint4 *dst = (uint4 *)(a.w_o + at * D + c);
#pragma unroll
            for (int e = 0; e < 8; ++e) dst[e] = make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
          }
        }
        tc_fence_before();
      }
      if (row < rows) {
        float l0, l1, l3, l4;
        f2_unpack(l2[0], l0, l1);
        f2_unpack(l2[1], l3, l4);
        a.w_ml[at] = make_float2(m_ref, (l0 + l1) + (l3 + l4));
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (*abort && threadIdx.x == 0) {
    // every copy has landed before the CTA exits: the newest into each place (all
    // have been waited for where no wait ran out)
    if (TMA) {
      volatile int no_abort = 0;
      for (int i = 0; i < kK + kV; ++i) {
        const bool k = i < kK;
        const int places = k ? kK : kV, at = k ? i : i - kK, filled = (s_filled[k ? 0 : 1] - 1 - at + places) / places;
        if (filled > 0) mbar_wait(bar((k ? R::kFullK : R::kFullV) + at), (filled - 1) & 1, &no_abort);
      }
    }
    Walk again = *s_walk;
    while (again.next(a)) a.w_flag[again.part(a)] = SV_ROW_TIMEOUT;
  }
  if (warp == kMmaWarp) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
  }
}

// The join: a warp to ROWS query rows of a segment, with their parts and the sums of
// the sequences' own slots.  Rows of one segment have the same parts, so that where the
// rows are many what it takes to find them is done once for four, and four rows' values
// are on their way together; where they are few, a warp has one, with more of its parts
// on their way (with 8 KV heads of 128 behind 20000 slots, 8192 rows take 127 us in all
// by fours and 130 one by one, 32768 rows 394 and 410, 2048 rows 51 and 48, 256 rows 35
// and 29).  32 / ROWS lanes to a row where references and sums are looked at, all of
// them for its values.
constexpr int kJoinRows = 4;
constexpr long long kFewRows = 2048;
constexpr int kJoinThreads = 256;
struct JoinArgs {
  const float *own_o;
  const float2 *own_ml;
  const uint32_t *own_flag;
  void *out;
  float *lse;
};
template <typename T, int D, int ROWS>
__global__ void __launch_bounds__(kJoinThreads) prefix_join_kernel(PrefixArgs a, JoinArgs j) {
  const unsigned FULL = 0xffffffffu;
  static_assert(kRows % ROWS == 0, "rows of one query tile");
  constexpr int kLanes = 32 / ROWS, E = D / 32, U = ROWS > 1 ? 4 : 8;  // U: places on their way together
  const int lane = threadIdx.x & 31, mine = lane / kLanes, sub = lane % kLanes;
  const int wg = a.W * a.G, fours = (wg + ROWS - 1) / ROWS;
  const int unit = blockIdx.x * (kJoinThreads / 32) + (threadIdx.x >> 5);  // below 2^27
  if (unit >= a.N * a.Hkv * fours) return;
  const int seg = unit / fours, at0 = (unit - seg * fours) * ROWS;
  const int p = seg / a.Hkv, head = seg - p * a.Hkv, count = min(ROWS, wg - at0);
  const int mt = at0 / kRows, column = mt / 2, pair = 2 * column + 1 < a.mtiles;
  // the row of the lane's eight; the last one's again behind it
  const int r = min(mine, count - 1), b = p * a.W + (at0 + r) / a.G, h = head * a.G + (at0 + r) % a.G;
  const int row = b * a.Hq + h;
  // lengths were there before the launches that this one waits for
  const longlong2 n = count_tiles(a, p);
  const int len = __ldcg(a.len + p), tiles = tiles_of(a, len);
  int c0 = 0, parts = 0;  // shares with a part
  if (tiles > 0) {
    const long long all = n.x * a.Hkv, first = n.y * a.Hkv + (long long)tiles * head;
    const long long shares = cut_into(pair ? a.shares2 : a.shares1, all);
    c0 = share_of(first, shares, all);
    parts = share_of(first + tiles - 1, shares, all) - c0 + 1;
  }
  // places in the parts: that of the rows' query tile in a pair, both otherwise
  const int two = pair ? 0 : 1, places = parts << two;
  const size_t part0 = part_at(a, column, (long long)p * a.Hkv + head + c0);
  const size_t place0 = (part0 * 2 + (pair ? mt & 1 : 0)) * a.rows + at0 % kRows, step = (size_t)a.rows << (1 - two);
  grid_dep_sync();
  auto load = [&](const float *src, float *x) {
    if constexpr (E == 4) {
      const float4 v = *(const float4 *)(src + lane * 4);
      x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
    } else {
      const float2 v = *(const float2 *)(src + lane * 2);
      x[0] = v.x, x[1] = v.y;
    }
  };
  // values first, whatever their references say: all loads are on their way at once
  float acc[ROWS][E], x[U][ROWS][E];
#pragma unroll
  for (int i = 0; i < ROWS; ++i) load(j.own_o + (size_t)__shfl_sync(FULL, row, i * kLanes) * D, acc[i]);
  auto fetch = [&](int at) {
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (at + u < places) {
#pragma unroll
        for (int i = 0; i < ROWS; ++i)
          load(a.w_o + (place0 + (at + u) * step + min(i, count - 1)) * D, x[u][i]);
      }
  };
  fetch(0);
  uint32_t flag = (len < 0 || len > a.cap ? SV_ROW_BAD_LEN : 0u) | j.own_flag[b];
  const float2 own = j.own_ml[row];
  float2 ml = make_float2(-INFINITY, 0.0f);  // of the lane's place of the eight in work
  float M = own.x;
  for (int i = sub; i < places; i += kLanes) {
    const float2 v = a.w_ml[place0 + i * step + r];
    if (i < kLanes) ml = v;
    M = fmaxf(M, v.x);
    flag |= a.w_flag[part0 + (i >> two)];
  }
#pragma unroll
  for (int o = kLanes / 2; o; o >>= 1) {
    M = fmaxf(M, __shfl_xor_sync(FULL, M, o));
    flag |= __shfl_xor_sync(FULL, flag, o);
  }
  // a sequence's status (0 from the first launch) is that of all its rows: a wait runs out
  // in one CTA, which has parts of some heads
  if (flag && a.status) atomicOr(a.status + b, flag);
  // A sum without a finite reference is 0, or NaN from the data: it stays, and so do
  // its values.  A buffer without a tile has no sums: it is passed over.
  auto factor = [&](float m) { return m == -INFINITY ? 1.0f : ex2_approx(m - M); };
  const float f0 = factor(own.x);
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    const float g = __shfl_sync(FULL, f0, i * kLanes);
#pragma unroll
    for (int e = 0; e < E; ++e) acc[i][e] *= g;
  }
  float sum = sub == 0 ? own.y * f0 : 0.0f, f = 0.0f;
  unsigned there = 0;
  for (int at = 0; at < places; at += U) {
    if (at % kLanes == 0) {
      const bool in = at + sub < places;
      if (at && in) ml = a.w_ml[place0 + (at + sub) * step + r];
      const bool some = in && (ml.x != -INFINITY || ml.y != 0.0f);
      f = some ? factor(ml.x) : 0.0f;
      if (some) sum += ml.y * f;
      there = __ballot_sync(FULL, some);
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < ROWS; ++i) {
        const int from = i * kLanes + (at + u) % kLanes;
        const float g = __shfl_sync(FULL, f, from);
        if (there >> from & 1) {
#pragma unroll
          for (int e = 0; e < E; ++e) acc[i][e] = fmaf(x[u][i][e], g, acc[i][e]);
        }
      }
    fetch(at + U);
  }
#pragma unroll
  for (int o = kLanes / 2; o; o >>= 1) sum += __shfl_xor_sync(FULL, sum, o);
  const float nan = __int_as_float(0x7fffffff), inv = flag ? nan : sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    const float g = __shfl_sync(FULL, inv, i * kLanes);
    const int to = __shfl_sync(FULL, row, i * kLanes);
    if (i >= count) break;
    uint32_t *out = (uint32_t *)((T *)j.out + (size_t)to * D) + lane * (E / 2);
    // (a row of nothing is zeros, whatever its values were)
    if constexpr (E == 4)
      *(uint2 *)out = g == 0.0f ? make_uint2(0u, 0u) : make_uint2(pack2<T>(acc[i][0] * g, acc[i][1] * g), pack2<T>(acc[i][2] * g, acc[i][3] * g));
    else
      *out = g == 0.0f ? 0u : pack2<T>(acc[i][0] * g, acc[i][1] * g);
  }
  if (sub == 0 && mine < count) {
    if (j.lse) j.lse[row] = flag ? nan : sum == 0.0f ? -INFINITY : (M + log2f(sum)) * kLn2;
  }
}

// ------------------------------------------------------------------ host side
constexpr int kSms = 152;
struct Sizes {
  int W, G, mtiles, rows, shares2, shares1, ctas;
  size_t o, ml, flag, own_o, own_ml, own_flag, own, own_bytes, total;
};
bool sizes_of(Sizes &z, int B, int N, int Hq, int Hkv, int D, int page, int max_pages) {
  z.W = B / N;
  z.G = Hq / Hkv;
  const long long wg = (long long)z.W * z.G, mtiles = (wg + kRows - 1) / kRows, columns = (mtiles + 1) / 2;
  const long long segments = (long long)Hkv * N;
  if (wg > (1 << 24) || segments > (1 << 24) || columns * segments > (1 << 24) || (long long)B * Hq > (1 << 26))
    return false;
  z.mtiles = (int)mtiles;
  z.rows = wg < kRows ? (int)wg : kRows;
  // the SMs of this part over the columns, by their tiles, and what they come to
  z.shares2 = mtiles >= 2 ? (int)(2 * kSms / mtiles > 1 ? 2 * kSms / mtiles : 1) : 0;
  z.shares1 = mtiles % 2 ? (int)(kSms / mtiles > 1 ? kSms / mtiles : 1) : 0;
  z.ctas = (int)(mtiles / 2 * z.shares2 + z.shares1);
  const size_t parts = (size_t)columns * ((size_t)(z.shares2 > z.shares1 ? z.shares2 : z.shares1) + (size_t)segments);
  size_t at = 0;
  auto take = [&](size_t n) {
    const size_t r = at;
    at = align_up(at + n, 256);
    return r;
  };
  z.o = take(parts * 2 * z.rows * D * 4);
  z.ml = take(parts * 2 * z.rows * 8);
  z.flag = take(parts * 4);
  z.own_o = take((size_t)B * Hq * D * 4);
  z.own_ml = take((size_t)B * Hq * 8);
  z.own_flag = take((size_t)B * 4);
  if (!paged_sums_workspace(&z.own_bytes, B, Hq, Hkv, D, page, max_pages)) return false;
  z.own = take(z.own_bytes);
  z.total = at;
  return true;
}
bool bad_shape(int B, int N, int Hq, int Hkv, int D, int page, int max_prefix_pages, int max_pages) {
  return B < 0 || N < 1 || B % N || Hq < 1 || Hkv < 1 || Hq % Hkv || D < 1 || page < 1 || max_prefix_pages < 1 ||
         max_pages < 1;
}

template <typename T, int D, bool TMA, bool TWO>
sv_status launch(const CUtensorMap &map, const PrefixArgs &a, const JoinArgs &j, const Sizes &z, const int32_t *block_table,
                 const int32_t *seq_len, int max_pages, float scale, sv_dtype dt, float *own_o, float2 *own_ml,
                 uint32_t *own_flag, void *own_ws, cudaStream_t st) {
  static thread_local int set_dev = -1;
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev != set_dev) {
    const cudaError_t e = cudaFuncSetAttribute(prefix_attn_kernel<T, D, TMA, TWO>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (int)Ring<D>::kSmem);
    if (e != cudaSuccess) return check_launch("prefix_attention", e);
    set_dev = dev;
  }
  sv_status s;
  {
    LaunchScope ls("prefix_attention", st);
    s = check_launch("prefix_attention",
                     launch_pdl(prefix_attn_kernel<T, D, TMA, TWO>, dim3((unsigned)z.ctas), dim3(kThreads), Ring<D>::kSmem, st, map, a));
    if (s != SV_OK) return s;
  }
  s = paged_sums(a.q, a.kv, a.kv_stride, a.page_stride, dt, block_table, seq_len, a.B, a.Hq, a.Hkv, D, a.page, max_pages,
                 a.num_pages, scale, own_o, own_ml, own_flag, own_ws, st);
  if (s != SV_OK) return s;
  const bool few = (long long)a.B * a.Hq <= kFewRows;
  const long long at_once = few ? 1 : kJoinRows, units = (long long)a.N * a.Hkv * (((long long)a.W * a.G + at_once - 1) / at_once);
  constexpr int kUnits = kJoinThreads / 32;
  LaunchScope ls("prefix_join", st);
  return check_launch("prefix_join", launch_pdl(few ? prefix_join_kernel<T, D, 1> : prefix_join_kernel<T, D, kJoinRows>,
                                                dim3((unsigned)((units + kUnits - 1) / kUnits)), dim3(kJoinThreads), 0, st, a, j));
}

}  // namespace
}  // namespace sv

using namespace sv;

extern "C" size_t sv_prefix_attention_workspace(int B, int N, int Hq, int Hkv, int D, int page,
                                                int max_prefix_pages, int max_pages) {
  Sizes z;
  if (bad_shape(B, N, Hq, Hkv, D, page, max_prefix_pages, max_pages) || B == 0 ||
      !sizes_of(z, B, N, Hq, Hkv, D, page, max_pages))
    return 0;
  return z.total;
}

extern "C" sv_status sv_prefix_attention(const void *q, const void *kv, int64_t kv_stride,
                                         int64_t page_stride, sv_dtype dt,
                                         const int32_t *prefix_table, const int32_t *prefix_len,
                                         const int32_t *block_table, const int32_t *seq_len, int B,
                                         int N, int Hq, int Hkv, int D, int page,
                                         int max_prefix_pages, int max_pages, int num_pages,
                                         float scale, void *out, float *out_lse,
                                         uint32_t *out_status, void *workspace,
                                         size_t workspace_bytes, void *stream) {
  if (bad_shape(B, N, Hq, Hkv, D, page, max_prefix_pages, max_pages) || num_pages < 1)
    return set_error(SV_ERR_INVALID_ARG,
                     "need B >= 0 a multiple of N >= 1, Hq a multiple of Hkv >= 1, page, max_prefix_pages, "
                     "max_pages and num_pages >= 1");
  if (dt != SV_BF16 && dt != SV_F16)
    return set_error(SV_ERR_INVALID_ARG, "the cache is SV_BF16 or SV_F16, not dtype %d", (int)dt);
  if (D != 64 && D != 128) return set_error(SV_ERR_UNSUPPORTED, "head dimension %d (64 or 128)", D);
  if (!(scale > 0.0f) || !isfinite(scale * kLog2e))
    return set_error(SV_ERR_INVALID_ARG, "scale must be > 0 and finite");
  if ((long long)page * max_prefix_pages > (1 << 30) || (long long)page * max_pages > (1 << 30))
    return set_error(SV_ERR_UNSUPPORTED, "more than 2^30 slots a sequence");
  const int64_t inner = (int64_t)page * Hkv * D;
  if (page_stride < inner || page_stride % 8 || kv_stride % 8 || kv_stride < 1 ||
      page_stride > INT64_MAX / 4 / num_pages || kv_stride > INT64_MAX / 4)
    return set_error(SV_ERR_INVALID_ARG,
                     "page_stride must cover a page (%lld elements), kv_stride be positive, and both "
                     "be multiples of 8",
                     (long long)inner);
  if (B == 0) return SV_OK;
  Sizes z;
  if (!sizes_of(z, B, N, Hq, Hkv, D, page, max_pages))
    return set_error(SV_ERR_UNSUPPORTED, "too many query rows or prefixes");
  if (!q || !kv || !prefix_table || !prefix_len || !block_table || !seq_len || !out)
    return set_error(SV_ERR_INVALID_ARG, "null pointer");
  if ((uintptr_t)q % 16 || (uintptr_t)kv % 16 || (uintptr_t)out % 16)
    return set_error(SV_ERR_INVALID_ARG, "q, kv and out need 16-byte alignment");
  if ((uintptr_t)prefix_table % 4 || (uintptr_t)prefix_len % 4 || (uintptr_t)block_table % 4 ||
      (uintptr_t)seq_len % 4 || (uintptr_t)out_lse % 4 || (uintptr_t)out_status % 4 || (uintptr_t)workspace % 256)
    return set_error(SV_ERR_INVALID_ARG, "misaligned pointer (the workspace needs 256 bytes)");
  if (workspace_bytes < z.total || !workspace)
    return set_error(SV_ERR_INVALID_ARG, "workspace of %zu bytes, need %zu", workspace_bytes, z.total);
  sv_status s;
  if ((s = map_arg(q, "q")) != SV_OK || (s = map_arg(kv, "kv")) != SV_OK ||
      (s = map_arg(prefix_table, "prefix_table")) != SV_OK ||
      (s = map_arg(prefix_len, "prefix_len")) != SV_OK ||
      (s = map_arg(block_table, "block_table")) != SV_OK ||
      (s = map_arg(seq_len, "seq_len")) != SV_OK || (s = map_arg(out, "out")) != SV_OK ||
      (s = map_arg(out_lse, "out_lse")) != SV_OK || (s = map_arg(out_status, "out_status")) != SV_OK ||
      (s = map_arg(workspace, "workspace")) != SV_OK)
    return s;
  char *w = (char *)workspace;
  PrefixArgs a;
  a.q = q;
  a.kv = kv;
  a.kv_stride = kv_stride;
  a.page_stride = page_stride;
  a.table = prefix_table;
  a.len = prefix_len;
  a.B = B;
  a.N = N;
  a.W = z.W;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.G = z.G;
  a.mtiles = z.mtiles;
  a.page = page;
  a.page_shift = -1;
  for (int i = 0; i < 31; ++i)
    if (page == 1 << i) a.page_shift = i;
  a.max_pages = max_prefix_pages;
  a.num_pages = num_pages;
  a.cap = page * max_prefix_pages;
  a.shares2 = z.shares2;
  a.shares1 = z.shares1;
  a.rows = z.rows;
  a.scale_log2 = scale * kLog2e;
  a.w_o = (float *)(w + z.o);
  a.w_ml = (float2 *)(w + z.ml);
  a.w_flag = (uint32_t *)(w + z.flag);
  a.status = out_status;
  float *own_o = (float *)(w + z.own_o);
  float2 *own_ml = (float2 *)(w + z.own_ml);
  uint32_t *own_flag = (uint32_t *)(w + z.own_flag);
  const JoinArgs j{own_o, own_ml, own_flag, out, out_lse};
  void *own_ws = z.own_bytes ? w + z.own : nullptr;
  cudaStream_t st = (cudaStream_t)stream;
  // Boxes of as many rows as a power of two divides the page by, where that is 16 and
  // more; of whole pages, with tiles of as many as 128 rows hold, for others of 8 to
  // 128 rows (16 prefixes of 1500 to 9000 slots, 8 KV heads of 64, pages of 20: tiles
  // of 120 keys by 6 boxes take 52 us where 32 boxes of 4 rows take 66); of 8 rows.
  // What is left goes by copies.
  a.box = kKeys;
  while (page % a.box) a.box /= 2;
  a.keys = kKeys;
  const int whole = page <= kKeys ? kKeys / page * page : 0;
  if (a.box < 16 && page >= 8 && whole >= 96) {
    a.box = page;
    a.keys = whole;
  }
  CUtensorMap map = {};
  bool tma = a.box >= 8 && is_device_memory(kv);
  if (tma) {
    EncodeTiledFn fn = encode_fn();
    const cuuint64_t dims[5] = {(cuuint64_t)D, (cuuint64_t)Hkv, (cuuint64_t)page, (cuuint64_t)num_pages, 2};
    const cuuint64_t strides[4] = {(cuuint64_t)D * 2, (cuuint64_t)Hkv * D * 2, (cuuint64_t)page_stride * 2,
                                   (cuuint64_t)kv_stride * 2};
    const cuuint32_t box[5] = {64, 1, (cuuint32_t)a.box, 1, 1}, es[5] = {1, 1, 1, 1, 1};
    tma = fn && page_stride < (1LL << 39) && kv_stride < (1LL << 39) &&
          fn(&map, dt == SV_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 5,
             const_cast<void *>(kv), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  }
  if (!tma) a.keys = kKeys;
  auto go = [&](auto kernel) {
    return kernel(map, a, j, z, block_table, seq_len, max_pages, scale, dt, own_o, own_ml, own_flag, own_ws, st);
  };
  auto by_head = [&](auto type, auto two) {
    typedef decltype(type) T;
    constexpr bool kTwo = decltype(two)::value != 0;
    if (D == 64) return tma ? go(launch<T, 64, true, kTwo>) : go(launch<T, 64, false, kTwo>);
    return tma ? go(launch<T, 128, true, kTwo>) : go(launch<T, 128, false, kTwo>);
  };
  const bool two = z.mtiles == 1;
  if (dt == SV_BF16) return two ? by_head(__nv_bfloat16(), Int<1>()) : by_head(__nv_bfloat16(), Int<0>());
  return two ? by_head(__half(), Int<1>()) : by_head(__half(), Int<0>());
}
