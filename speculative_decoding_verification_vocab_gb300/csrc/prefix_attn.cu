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
// Work: segments, one for each prefix, KV head and tile of 128 query rows (row r =
// sequence r / G, head r % G), lie one after the other as a row of 128-key tiles,
// and each CTA, one to an SM, takes an equal share of it, from one segment to the
// next: parts of a segment, whose sums go to the workspace.  Shares are cut from
// the lengths on the device, so a captured launch follows growing prefixes.
//   warps 0-1   producer: page table entries a tile ahead, K and V rows by
//               asynchronous copies of 16 bytes into a ring (rows of 128-byte
//               swizzled boxes of 64 columns; pages may end anywhere in a tile);
//               rows past the end are zeros;
//   warp 2      MMA issuer: S_j = Q K_j^T once S_{j-1} has been read out of tensor
//               memory, O += P_j V_j once P_j is there; A operands (Q, P) in
//               tensor memory;
//   warps 3-10  softmax: query rows to tensor memory, S_j to registers (a row over
//               a quad of threads), the running maximum with a lazy rescale of O,
//               P_j as 16-bit values to one of two buffers; at a segment's end O,
//               m and l to the workspace.
// Every wait on an mbarrier is bounded; one that runs out marks the CTA's parts
// with SV_ROW_TIMEOUT.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>

#include "paged.cuh"
#include "tcgen05.cuh"

namespace sv {
namespace {

constexpr int kRows = 128;   // query rows of a segment = tensor-memory lanes
constexpr int kKeys = 128;   // keys of a tile
constexpr int kProducers = 64;
constexpr int kSoftmaxWarps = 8;
constexpr int kMmaWarp = kProducers / 32, kFirstSoftmax = kMmaWarp + 1;
constexpr int kThreads = kProducers + 32 + 32 * kSoftmaxWarps;
constexpr uint32_t kBox = kKeys * 128;  // bytes of a box of 64 columns
constexpr float kLn2 = 0.693147180559945309f, kLog2e = 1.4426950408889634f;
// tensor-memory columns: S, O, Q and two buffers of P (16-bit pairs)
constexpr uint32_t kColS = 0, kColO = 128, kColQ = 256, kColP = 320, kTmemCols = 512;

// A score moves the reference only when it is more than kSlack above it (log2
// units).  Weights go into the product as 16-bit numbers: in fp16 the reference
// lies 2^kBias below the maximum it was set by, so that they fill the type's range
// from the top (2^15 at most) and the small ones do not round to nothing.  One
// 16-bit part (half a step, 2^-8 or 2^-11, of each weight, independent from key to
// key): a second one would double the product of a bound that is the product.
template <typename T> constexpr float kSlack = 8.0f;
template <typename T> constexpr float kBias = 0.0f;
template <> constexpr float kSlack<__half> = 4.0f;
template <> constexpr float kBias<__half> = 11.0f;
template <typename T> constexpr uint32_t kAbType = 1;  // of the instruction descriptor: bf16
template <> constexpr uint32_t kAbType<__half> = 0;

template <typename T> __device__ __forceinline__ uint32_t pack2(float lo, float hi);
template <> __device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float lo, float hi) { return pack_bf16(lo, hi); }
template <> __device__ __forceinline__ uint32_t pack2<__half>(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *(const uint32_t *)&v;
}

template <int D> struct Ring {
  static constexpr uint32_t kTileBytes = kKeys * D * 2;  // K or V rows of a tile
  static constexpr int kStages = D == 128 ? 3 : 6;
  static constexpr uint32_t kOffBar = kStages * 2 * kTileBytes;
  static constexpr uint32_t kOffRows = kOffBar + 32 * 8;         // two tiles' row offsets
  static constexpr uint32_t kOffMisc = kOffRows + 2 * kKeys * 8;
  static constexpr size_t kSmem = kOffMisc + 128 + 1024;  // + alignment
  // barriers: stage filled and free; Q there; S there and read out; P there and
  // its product done, by parity
  static constexpr int kFull = 0, kFree = kStages, kQ = 2 * kStages, kS = kQ + 1, kSF = kS + 1, kP = kSF + 1,
                       kPV = kP + 2, kCount = kPV + 2;
  static_assert(kCount <= 32, "barriers");
};

struct PrefixArgs {
  const void *q, *kv;
  int64_t kv_stride, page_stride;
  const int32_t *table, *len;  // [N][max_pages], [N]
  int B, N, W, Hq, Hkv, G, mtiles, HM;  // HM = Hkv mtiles segments to a prefix
  int page, page_shift, max_pages, num_pages, cap;
  int ctas, rows;  // rows of a part: min(128, W G)
  float scale_log2;
  // workspace: sums [parts][rows][D], references and sums of exponentials
  // [parts][rows], status bits [parts]
  float *w_o;
  float2 *w_ml;
  uint32_t *w_flag;
};

__device__ __forceinline__ int tiles_of(const PrefixArgs &a, int len) {
  return len < 0 || len > a.cap ? 0 : (len + kKeys - 1) / kKeys;
}
// tiles of all prefixes and of those before p, over the lanes of a warp
__device__ __forceinline__ longlong2 count_tiles(const PrefixArgs &a, int p) {
  longlong2 n = make_longlong2(0, 0);
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

// CTAs that share so many tiles: none without one
__device__ __forceinline__ long long sharing(const PrefixArgs &a, long long all) {
  return min((long long)a.ctas, max(all, 1LL));
}

// A CTA's way through its share: the part of a segment it is at.  Part index:
// CTA + segment, of which from part to part one or the other grows.
struct Walk {
  long long at, end, first;  // tiles in the row of all; the first of prefix p's segments
  int p, hm, t0, t1, len;
  __device__ __forceinline__ bool next(const PrefixArgs &a) {
    for (;;) {
      if (at >= end || p >= a.N) return false;
      len = __ldcg(a.len + p);
      const int tiles = tiles_of(a, len);
      const long long block = (long long)a.HM * tiles;
      if (at < first + block) {
        hm = (int)((at - first) / tiles);
        t0 = (int)((at - first) % tiles);
        t1 = (int)min((long long)tiles, t0 + (end - at));
        at += t1 - t0;
        return true;
      }
      first += block;
      ++p;
    }
  }
};

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 1) prefix_attn_kernel(PrefixArgs a) {
  using R = Ring<D>;
  constexpr int kStages = R::kStages;
  constexpr uint32_t kTileBytes = R::kTileBytes;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *sm = (uint8_t *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint64_t *bars = (uint64_t *)(sm + R::kOffBar);
  long long *s_row = (long long *)(sm + R::kOffRows);  // [2][kKeys]
  uint32_t *tmem_slot = (uint32_t *)(sm + R::kOffMisc);
  volatile int *abort = (volatile int *)(sm + R::kOffMisc + 4);
  Walk *s_walk = (Walk *)(sm + R::kOffMisc + 8);
  volatile uint8_t *s_bad = sm + R::kOffMisc + 8 + sizeof(Walk);  // [kStages][2], by producer warp
  static_assert(8 + sizeof(Walk) + kStages * 2 <= 128, "misc");
  const uint32_t bar0 = smem_addr(bars), sm0 = smem_addr(sm);
  auto bar = [&](int i) { return bar0 + 8u * (uint32_t)i; };

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(bar(R::kFull + s), kProducers / 32);
      mbar_init(bar(R::kFree + s), 1);
    }
    mbar_init(bar(R::kQ), kSoftmaxWarps);
    mbar_init(bar(R::kS), 1);
    mbar_init(bar(R::kSF), kSoftmaxWarps);
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar(R::kP + s), kSoftmaxWarps);
      mbar_init(bar(R::kPV + s), 1);
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
  grid_dep_sync();
  if (warp == 0) {
    // this CTA's share of all tiles, and the prefix it starts in
    const long long all = (long long)a.HM * count_tiles(a, 0).x;
    Walk w;
    const long long ctas = sharing(a, all);
    w.at = min((long long)blockIdx.x, ctas) * all / ctas;
    w.end = min((long long)blockIdx.x + 1, ctas) * all / ctas;
    w.first = 0;
    w.p = 0;
    for (int p0 = 0; p0 < a.N && w.at < w.end; p0 += 32) {
      const int p = p0 + lane;
      const long long n = p < a.N ? (long long)a.HM * tiles_of(a, __ldcg(a.len + p)) : 0;
      long long incl = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += x;
      }
      const unsigned past = __ballot_sync(0xffffffffu, w.first + incl > w.at);
      if (past) {
        const int l = __ffs(past) - 1;
        w.p = p0 + l;
        w.first += __shfl_sync(0xffffffffu, incl - n, l);
        break;
      }
      w.first += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane == 0) *s_walk = w;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  Walk w = *s_walk;

  if (warp < kMmaWarp) {
    // ------------------------------------------------------------ producer
    // Thread t finds rows t and t + 64 of a tile, one tile ahead; 16 bytes of a
    // row to a lane, CPR lanes to a row.
    constexpr int CPR = D / 8, RPI = kProducers / CPR;  // rows of one round of copies
    const int lr = threadIdx.x / CPR, lc = threadIdx.x % CPR;
    const int64_t row_elems = (int64_t)a.Hkv * D;
    int g = 0;  // tiles so far
    bool ok = true;
    // a barrier of the producer warps, with their votes: they go on or end together
    auto producers_all = [](bool x) {
      uint32_t r;
      asm volatile(
          "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n bar.red.and.pred q, 1, %2, p;\n selp.u32 %0, 1, 0, q;\n}"
          : "=r"(r)
          : "r"((uint32_t)x), "n"(kProducers)
          : "memory");
      return r != 0;
    };
    auto finish = [&](int t) {  // tile t is in shared memory: this warp's share of it
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(R::kFull + t % kStages));
    };
    while (ok && w.next(a)) {
      const T *kv = (const T *)a.kv + (int64_t)(w.hm / a.mtiles) * D + lc * 8;
      const int32_t *table = a.table + (size_t)w.p * a.max_pages;
      int id[2];
      auto fetch = [&](int t) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int slot = t * kKeys + (int)threadIdx.x + e * kProducers;
          id[e] = t < w.t1 && slot < w.len ? __ldg(table + (a.page_shift >= 0 ? slot >> a.page_shift : slot / a.page)) : -1;
        }
      };
      fetch(w.t0);
      for (int t = w.t0; t < w.t1; ++t, ++g) {
        const int st = g % kStages;
        long long *rows = s_row + (g & 1) * kKeys;
        bool bad = false;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = (int)threadIdx.x + e * kProducers, slot = t * kKeys + r;
          long long off = -1;
          if (slot < w.len) {
            if ((unsigned)id[e] < (unsigned)a.num_pages) {
              const int in_page = a.page_shift >= 0 ? slot & (a.page - 1) : slot % a.page;
              off = id[e] * (long long)a.page_stride + in_page * (long long)row_elems;
            } else {
              bad = true;
            }
          }
          rows[r] = off;
        }
        bad = __any_sync(0xffffffffu, bad);
        fetch(t + 1);
        // the stage's last tile has been multiplied; both warps' rows are there
        ok = g < kStages || mbar_wait(bar(R::kFree + st), (g / kStages - 1) & 1, abort);
        ok = producers_all(ok);
        if (!ok) break;
        if (lane == 0) s_bad[st * 2 + warp] = bad;
        const uint32_t dst = sm0 + st * 2 * kTileBytes + (lc >> 3) * kBox + lr * 128;
#pragma unroll
        for (int part = 0; part < 2; ++part) {  // K, V
#pragma unroll 4
          for (int r = 0; r < kKeys; r += RPI) {
            const long long off = rows[r + lr];
            const uint32_t n = off >= 0 ? 16u : 0u;
            const T *src = kv + (off >= 0 ? off : 0) + part * a.kv_stride;
            const uint32_t d = dst + part * kTileBytes + r * 128 + (((lc & 7) ^ ((r + lr) & 7)) << 4);
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(d), "l"(src), "r"(n) : "memory");
          }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        if (g > 0) {  // the tile before has arrived
          asm volatile("cp.async.wait_group 1;" ::: "memory");
          finish(g - 1);
        }
      }
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    if (ok && g > 0) finish(g - 1);
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------ MMA
    // The warp runs converged and elect.sync picks the issuing lane.  gS and gP
    // count the S and PV tiles of the CTA.
    constexpr uint32_t kIdesc = (1u << 4) | (kAbType<T> << 7) | (kAbType<T> << 10) | ((uint32_t)(kRows >> 4) << 24);
    constexpr uint32_t kIdescS = kIdesc | ((uint32_t)(kKeys >> 3) << 17);
    constexpr uint32_t kIdescO = kIdesc | (1u << 16) | ((uint32_t)(D >> 3) << 17);  // V: head dim contiguous
    int gS = 0, gP = 0, nq = 0;
    bool ok = true;
    const uint64_t dK0 = sdesc(sm0, 16, 1024), dV0 = sdesc(sm0 + kTileBytes, kBox, 1024);
    constexpr uint64_t kStageStep = 2 * kTileBytes >> 4;
    auto all = [&](bool x) { return __all_sync(0xffffffffu, x) != 0; };
    auto issue_s = [&]() {  // S_gS: its K has landed, S_{gS - 1} is read out
      ok = all((gS < 1 || mbar_wait(bar(R::kSF), (gS - 1) & 1, abort)) &&
               mbar_wait(bar(R::kFull + gS % kStages), (gS / kStages) & 1, abort));
      if (!ok) return;
      tc_fence_after();
      if (elect_one()) {
        const uint64_t dk = dK0 + (gS % kStages) * kStageStep;
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks)
          mma_ts(tmem + kColS, tmem + kColQ + ks * 8, dk + (uint64_t)(((ks >> 2) * kBox + (ks & 3) * 32) >> 4), kIdescS,
                 ks > 0);
        mma_commit(bar(R::kS));
      }
      __syncwarp();
      ++gS;
    };
    while (ok && w.next(a)) {
      ok = all(mbar_wait(bar(R::kQ), nq & 1, abort));
      ++nq;
      if (!ok) break;
      tc_fence_after();
      issue_s();
      const int n = w.t1 - w.t0;
      for (int i = 0; ok && i < n; ++i) {
        if (i + 1 < n) issue_s();
        if (!ok) break;
        ok = all(mbar_wait(bar(R::kP + (gP & 1)), (gP >> 1) & 1, abort));
        if (!ok) break;
        tc_fence_after();
        const int st = gP % kStages;
        if (elect_one()) {
          const uint64_t dv = dV0 + st * kStageStep;
          const uint32_t pa = tmem + kColP + (gP & 1) * 64;
#pragma unroll
          for (int ks = 0; ks < kKeys / 16; ++ks)
            mma_ts(tmem + kColO, pa + ks * 8, dv + (uint64_t)(ks * 128), kIdescO, (i > 0 || ks > 0) ? 1u : 0u);
          mma_commit(bar(R::kPV + (gP & 1)));
          mma_commit(bar(R::kFree + st));
        }
        __syncwarp();
        ++gP;
      }
    }
    if (!ok) {
      // products in flight end before tensor memory is released: the last S and
      // the last PV are the newest phases of their barriers
      volatile int no_abort = 0;
      if (gS > 0) mbar_wait(bar(R::kS), (gS - 1) & 1, &no_abort);
      if (gP > 0) mbar_wait(bar(R::kPV + ((gP - 1) & 1)), ((gP - 1) >> 1) & 1, &no_abort);
    }
  } else {
    // ------------------------------------------------------------ softmax
    // A warp reads the tensor-memory lanes of quarter warp % 4; the two warps of a
    // quarter take 16 lanes each.  Thread t holds rows t / 4 and t / 4 + 8 of them
    // and in every 8 columns the pair 2 (t % 4): row maxima and sums are two
    // shuffles, and P's pair column 4 c + t % 4 is the thread's own.
    const int quarter = warp & 3, half = (warp - kFirstSoftmax) >> 2, q4 = lane & 3;
    const uint32_t lane16 = (uint32_t)(quarter * 32 + half * 16) << 16;
    const int rowA = quarter * 32 + half * 16 + (lane >> 2);  // and rowA + 8
    int gT = 0;
    bool ok = true;
    auto all = [&](bool x) { return __all_sync(0xffffffffu, x) != 0; };
    auto wait_pv = [&](int i) { return all(mbar_wait(bar(R::kPV + (i & 1)), (i >> 1) & 1, abort)); };
    while (ok && w.next(a)) {
      const int mt = w.hm % a.mtiles, hkv = w.hm / a.mtiles, n = w.t1 - w.t0;
      const int rows = min(kRows, a.W * a.G - mt * kRows);
      {
        // this warp's columns (a half of the head for D = 128) of the quarter's 32
        // rows to tensor memory, a lane a row; rows behind the last are zeros
        const int r = quarter * 32 + lane;
        if (D == 128 || half == 0) {
          uint32_t qv[32];
          const int at = mt * kRows + r;
          const uint4 *src = (const uint4 *)((const T *)a.q + ((size_t)((size_t)w.p * a.W + at / a.G) * a.Hq +
                                                               (size_t)hkv * a.G + at % a.G) * D + half * 64);
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            const uint4 x = r < rows ? __ldg(src + c) : make_uint4(0, 0, 0, 0);
            qv[4 * c] = x.x;
            qv[4 * c + 1] = x.y;
            qv[4 * c + 2] = x.z;
            qv[4 * c + 3] = x.w;
          }
          tm_st32u(tmem + ((uint32_t)(quarter * 32) << 16) + kColQ + 32 * half, qv);
          asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(R::kQ));
      }
      float m_ref[2] = {-INFINITY, -INFINITY};  // log2 units
      float l[2] = {0.0f, 0.0f};                // of this thread's columns
      uint32_t bad = 0;
      for (int j = 0; j < n; ++j) {
        const int g = gT + j, pb = g & 1;
        ok = all(mbar_wait(bar(R::kS), g & 1, abort));
        if (!ok) break;
        tc_fence_after();
        // s[4 c + 0, 1]: row A, keys 8 c + 2 q4 + {0, 1}; s[4 c + 2, 3]: row B
        float s[64];
        tm_ld16x256_x8(tmem + lane16 + kColS, s);
        tm_ld16x256_x8(tmem + lane16 + kColS + 64, s + 32);
        asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(R::kSF));
        bad |= s_bad[g % kStages * 2] | s_bad[g % kStages * 2 + 1];
        const int left = w.len - (w.t0 + j) * kKeys;  // keys of this tile
        if (left < kKeys) {
#pragma unroll
          for (int c = 0; c < 16; ++c)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              if (8 * c + 2 * q4 + e >= left) s[4 * c + e] = s[4 * c + 2 + e] = -INFINITY;
        }
        float factor[2], mneg[2];
        bool any_grow = false;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float pm[4] = {s[2 * e], s[2 * e + 1], s[4 + 2 * e], s[4 + 2 * e + 1]};
#pragma unroll
          for (int c = 2; c < 16; c += 2) {
            pm[0] = fmaxf(pm[0], s[4 * c + 2 * e]);
            pm[1] = fmaxf(pm[1], s[4 * c + 2 * e + 1]);
            pm[2] = fmaxf(pm[2], s[4 * c + 4 + 2 * e]);
            pm[3] = fmaxf(pm[3], s[4 * c + 4 + 2 * e + 1]);
          }
          float mx = fmaxf(fmaxf(pm[0], pm[1]), fmaxf(pm[2], pm[3]));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
          mx *= a.scale_log2;  // > 0: the maximum commutes with it
          const bool grow = mx > m_ref[e] + (kSlack<T> + kBias<T>);
          const float m_new = grow ? mx - kBias<T> : m_ref[e];
          factor[e] = grow && m_ref[e] != -INFINITY ? ex2(m_ref[e] - m_new) : 1.0f;
          any_grow |= factor[e] != 1.0f;
          l[e] *= factor[e];
          m_ref[e] = m_new;
          mneg[e] = m_new == -INFINITY ? 0.0f : -m_new;
        }
        uint32_t pk[32];
        unsigned long long la2 = 0ull, lb2 = 0ull;
        const unsigned long long sc2 = f2_splat(a.scale_log2);
        const unsigned long long ma2 = f2_splat(mneg[0]), mb2 = f2_splat(mneg[1]);
#pragma unroll
        for (int c = 0; c < 16; ++c) {
          const unsigned long long pa = ex2_2(f2_fma(f2_pack(s[4 * c], s[4 * c + 1]), sc2, ma2));
          const unsigned long long pb2 = ex2_2(f2_fma(f2_pack(s[4 * c + 2], s[4 * c + 3]), sc2, mb2));
          la2 = f2_add(la2, pa);
          lb2 = f2_add(lb2, pb2);
          float p0, p1, p2, p3;
          f2_unpack(pa, p0, p1);
          f2_unpack(pb2, p2, p3);
          pk[2 * c] = pack2<T>(p0, p1);      // row A, pair column 4 c + q4
          pk[2 * c + 1] = pack2<T>(p2, p3);  // row B
        }
        {
          float u0, u1, v0, v1;
          f2_unpack(la2, u0, u1);
          f2_unpack(lb2, v0, v1);
          l[0] += u0 + u1;
          l[1] += v0 + v1;
        }
        if (g >= 2) {  // P buffer pb is free
          ok = wait_pv(g - 2);
          if (!ok) break;
        }
        if (__any_sync(0xffffffffu, any_grow)) {
          // bring these rows of O, once it covers the tiles before, to the new
          // reference (at j = 0 there is none: no factor differs from 1)
          ok = wait_pv(g - 1);
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int c = 0; c < D; c += 64) {
            float o[32];
            tm_ld16x256_x8(tmem + lane16 + kColO + c, o);
            asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
            for (int k = 0; k < 32; ++k) o[k] *= factor[(k >> 1) & 1];
            tm_st16x256_x8(tmem + lane16 + kColO + c, o);
          }
        }
        tm_st16x128_x16(tmem + lane16 + kColP + pb * 64, pk);
        asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(R::kP + pb));
      }
      if (!ok) break;
      ok = wait_pv(gT + n - 1);
      if (!ok) break;
      tc_fence_after();
      const size_t part = (size_t)blockIdx.x + (size_t)w.p * a.HM + w.hm;
#pragma unroll
      for (int c = 0; c < D; c += 64) {
        float o[32];
        tm_ld16x256_x8(tmem + lane16 + kColO + c, o);
        asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
        // o[4 k + 0, 1]: row A, columns c + 8 k + 2 q4 + {0, 1}; o[4 k + 2, 3]: row B
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          if (rowA + 8 * e >= rows) continue;
          float *dst = a.w_o + (part * a.rows + rowA + 8 * e) * D + c + 2 * q4;
#pragma unroll
          for (int k = 0; k < 8; ++k) *(float2 *)(dst + 8 * k) = make_float2(o[4 * k + 2 * e], o[4 * k + 2 * e + 1]);
        }
      }
      tc_fence_before();
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float v = l[e];
        v += __shfl_xor_sync(0xffffffffu, v, 1);
        v += __shfl_xor_sync(0xffffffffu, v, 2);
        if (q4 == 0 && rowA + 8 * e < rows) a.w_ml[part * a.rows + rowA + 8 * e] = make_float2(m_ref[e], v);
      }
      if (warp == kFirstSoftmax && lane == 0) a.w_flag[part] = bad ? SV_ROW_BAD_PAGE : 0u;
      gT += n;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (*abort && threadIdx.x == 0) {
    Walk again = *s_walk;
    while (again.next(a)) a.w_flag[(size_t)blockIdx.x + (size_t)again.p * a.HM + again.hm] = SV_ROW_TIMEOUT;
  }
  if (warp == kMmaWarp) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
  }
}

// The join: a warp to each (sequence, query head), with the parts of its segment
// and the sums of the sequence's own slots.
constexpr int kJoinThreads = 256;
struct JoinArgs {
  const float *own_o;
  const float2 *own_ml;
  const uint32_t *own_flag;
  void *out;
  float *lse;
  uint32_t *status;
};
template <typename T, int D>
__global__ void __launch_bounds__(kJoinThreads) prefix_join_kernel(PrefixArgs a, JoinArgs j) {
  const int lane = threadIdx.x & 31;
  const long long row = (long long)blockIdx.x * (kJoinThreads / 32) + (threadIdx.x >> 5);
  const bool live = row < (long long)a.B * a.Hq;
  const int b = live ? (int)(row / a.Hq) : 0, h = live ? (int)(row % a.Hq) : 0;
  const int p = b / a.W, at = b % a.W * a.G + h % a.G;
  const int hm = h / a.G * a.mtiles + at / kRows, r = at % kRows;
  // lengths were there before the launches that this one waits for
  const longlong2 n = count_tiles(a, p);
  const int len = __ldcg(a.len + p), tiles = tiles_of(a, len);
  grid_dep_sync();
  if (!live) return;
  uint32_t flag = (len < 0 || len > a.cap ? SV_ROW_BAD_LEN : 0u) | j.own_flag[b];
  const float2 own = j.own_ml[row];
  long long c0 = 0, c1 = -1;  // CTAs with a part
  if (tiles > 0) {
    const long long all = n.x * a.HM, first = n.y * a.HM + (long long)hm * tiles, ctas = sharing(a, all);
    c0 = ((first + 1) * ctas - 1) / all;
    c1 = ((first + tiles) * ctas - 1) / all;
  }
  const size_t part0 = (size_t)p * a.HM + hm;
  float M = own.x;
  for (long long c = c0 + lane; c <= c1; c += 32) {
    M = fmaxf(M, a.w_ml[(part0 + c) * a.rows + r].x);
    flag |= a.w_flag[part0 + c];
  }
  M = warp_max(M);
  flag = __reduce_or_sync(0xffffffffu, flag);
  // (a sum without a finite reference is 0, or NaN from the data: it stays)
  auto weight = [&](float m) { return m == -INFINITY ? (M == -INFINITY ? 1.0f : 0.0f) : ex2(m - M); };
  constexpr int E = D / 32;
  float acc[E], sum;
  auto take = [&](const float *o, float2 ml, bool add) {
    const float f = weight(ml.x);
    const float y = ml.x == -INFINITY ? ml.y : ml.y * f;
    sum = add ? sum + y : y;
#pragma unroll
    for (int e = 0; e < E; e += 2) {
      const float2 x = *(const float2 *)(o + e * 32 + lane * 2);
      acc[e] = add ? fmaf(x.x, f, acc[e]) : x.x * f;
      acc[e + 1] = add ? fmaf(x.y, f, acc[e + 1]) : x.y * f;
    }
  };
  take(j.own_o + row * D, own, false);
#pragma unroll 4
  for (long long c = c0; c <= c1; ++c) {
    const size_t u = (part0 + c) * a.rows + r;
    take(a.w_o + u * D, a.w_ml[u], true);
  }
  const float nan = __int_as_float(0x7fffffff), inv = 1.0f / sum;
  uint32_t *out = (uint32_t *)((T *)j.out + row * D);
#pragma unroll
  for (int e = 0; e < E; e += 2) {
    const float x = flag ? nan : sum == 0.0f ? 0.0f : acc[e] * inv, y = flag ? nan : sum == 0.0f ? 0.0f : acc[e + 1] * inv;
    out[e * 16 + lane] = pack2<T>(x, y);
  }
  if (lane == 0) {
    if (j.lse) j.lse[row] = flag ? nan : sum == 0.0f ? -INFINITY : (M + log2f(sum)) * kLn2;
    if (h == 0 && j.status) j.status[b] = flag;
  }
}

// ------------------------------------------------------------------ host side
struct Sizes {
  int W, G, mtiles, HM, rows, ctas;
  size_t o, ml, flag, own_o, own_ml, own_flag, own, own_bytes, total;
};
bool sizes_of(Sizes &z, int B, int N, int Hq, int Hkv, int D, int page, int max_pages) {
  z.W = B / N;
  z.G = Hq / Hkv;
  const long long wg = (long long)z.W * z.G, mtiles = (wg + kRows - 1) / kRows, HM = mtiles * Hkv;
  if (wg > (1 << 24) || HM > (1 << 24) || HM * N > (1 << 24) || (long long)B * Hq > (1 << 26)) return false;
  z.mtiles = (int)mtiles;
  z.HM = (int)HM;
  z.rows = wg < kRows ? (int)wg : kRows;
  z.ctas = 152;  // one to an SM of this part; the parts' places follow it
  const size_t parts = (size_t)z.ctas + (size_t)N * z.HM;
  size_t at = 0;
  auto take = [&](size_t n) {
    const size_t r = at;
    at = align_up(at + n, 256);
    return r;
  };
  z.o = take(parts * z.rows * D * 4);
  z.ml = take(parts * z.rows * 8);
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

template <typename T, int D>
sv_status launch(const PrefixArgs &a, const JoinArgs &j, const Sizes &z, const int32_t *block_table,
                 const int32_t *seq_len, int max_pages, float scale, sv_dtype dt, float *own_o, float2 *own_ml,
                 uint32_t *own_flag, void *own_ws, cudaStream_t st) {
  static thread_local int set_dev = -1;
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev != set_dev) {
    const cudaError_t e = cudaFuncSetAttribute(prefix_attn_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (int)Ring<D>::kSmem);
    if (e != cudaSuccess) return check_launch("prefix_attention", e);
    set_dev = dev;
  }
  sv_status s;
  {
    LaunchScope ls("prefix_attention", st);
    s = check_launch("prefix_attention",
                     launch_pdl(prefix_attn_kernel<T, D>, dim3((unsigned)z.ctas), dim3(kThreads), Ring<D>::kSmem, st, a));
    if (s != SV_OK) return s;
  }
  s = paged_sums(a.q, a.kv, a.kv_stride, a.page_stride, dt, block_table, seq_len, a.B, a.Hq, a.Hkv, D, a.page, max_pages,
                 a.num_pages, scale, own_o, own_ml, own_flag, own_ws, st);
  if (s != SV_OK) return s;
  const long long rows = (long long)a.B * a.Hq;
  LaunchScope ls("prefix_join", st);
  return check_launch("prefix_join",
                      launch_pdl(prefix_join_kernel<T, D>, dim3((unsigned)((rows + kJoinThreads / 32 - 1) / (kJoinThreads / 32))),
                                 dim3(kJoinThreads), 0, st, a, j));
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
  a.HM = z.HM;
  a.page = page;
  a.page_shift = -1;
  for (int i = 0; i < 31; ++i)
    if (page == 1 << i) a.page_shift = i;
  a.max_pages = max_prefix_pages;
  a.num_pages = num_pages;
  a.cap = page * max_prefix_pages;
  a.ctas = z.ctas;
  a.rows = z.rows;
  a.scale_log2 = scale * kLog2e;
  a.w_o = (float *)(w + z.o);
  a.w_ml = (float2 *)(w + z.ml);
  a.w_flag = (uint32_t *)(w + z.flag);
  float *own_o = (float *)(w + z.own_o);
  float2 *own_ml = (float2 *)(w + z.own_ml);
  uint32_t *own_flag = (uint32_t *)(w + z.own_flag);
  const JoinArgs j{own_o, own_ml, own_flag, out, out_lse, out_status};
  void *own_ws = z.own_bytes ? w + z.own : nullptr;
  cudaStream_t st = (cudaStream_t)stream;
  if (dt == SV_BF16)
    return D == 64 ? launch<__nv_bfloat16, 64>(a, j, z, block_table, seq_len, max_pages, scale, dt, own_o, own_ml, own_flag, own_ws, st)
                   : launch<__nv_bfloat16, 128>(a, j, z, block_table, seq_len, max_pages, scale, dt, own_o, own_ml, own_flag, own_ws, st);
  return D == 64 ? launch<__half, 64>(a, j, z, block_table, seq_len, max_pages, scale, dt, own_o, own_ml, own_flag, own_ws, st)
                 : launch<__half, 128>(a, j, z, block_table, seq_len, max_pages, scale, dt, own_o, own_ml, own_flag, own_ws, st);
}
