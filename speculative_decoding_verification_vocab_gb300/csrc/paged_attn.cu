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
// Bound: every visible K and V row is read once (4 D bytes a slot and KV
// head), 4 D G operations on it: memory, for any G a model has.  The matrix
// products therefore only have to keep up with HBM (45 GB/s per SM): m16n8k16
// tensor instructions on registers, with the 16 rows holding the query heads
// of one KV head, need no staging of S, P or O and no exchange between warps,
// and take a tenth of what the SM could do.
//
// Work: a unit is a run of 64-key tiles of one (sequence, KV head, 16 query
// heads); KV heads of the same tiles are neighbouring CTAs, so that the D-wide
// slices of one token's row are read at about the same time.  Each CTA finds
// its unit from the lengths alone (a sum and a scan over the batch), so the
// host never sees them and a captured graph follows them.  Within a unit each
// of the 4 warps owns 16 keys of every tile: it loads them (cp.async, one
// 16-byte piece per lane, rows found through the page table one tile ahead;
// slots past the end are zero-filled, never read), multiplies, and keeps its
// own m, l and O; nothing but the last merge crosses warps.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>

#include "common.cuh"

namespace sv {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = 4;
constexpr int kWarpKeys = 16;
constexpr int kTile = kWarps * kWarpKeys;  // keys of a CTA tile
constexpr int kRows = 16;                  // query heads of a unit
// Units aimed at, and the fewest tiles of one (below that a unit's fixed cost
// shows).  Batches of kWhole sequences and more are not split.
constexpr int kUnits = 1216;
constexpr int kMinTiles = 2;
constexpr int kWhole = 2048;
constexpr int kMaxSlots = 1 << 30;

struct PagedArgs {
  const void *q, *kv;
  int64_t kv_stride, page_stride;  // elements from K to V, and from page to page
  const int32_t *table, *seq_len;
  int B, Hq, Hkv, G, gt, NH;  // gt groups of 16 query heads per KV head, NH = Hkv gt
  int page, page_shift, max_pages, num_pages;
  int window, sinks, cap;
  float scale_log2;
  int rows;  // query heads of a unit: min(G, 16)
  int vis_max;
  float *weight_sum;
  int S;
  void *out;
  float *lse;
  uint32_t *status;
  // workspace
  float *w_o;        // [units][rows][D]
  float2 *w_ml;      // [units][rows]
  uint32_t *w_flag;  // [units]
  uint32_t *w_status;  // [B]
  float *w_lse;      // [B][Hq], log2 units
  float *w_score;    // [B][Hkv][vis_max][G], log2 units
};

// the visible slots of a sequence, in order: [0, first), then [lo, len)
struct Visible {
  int len, lo, first, n;
  bool bad;
};
__device__ __forceinline__ Visible visible(const PagedArgs &a, int len) {
  Visible v;
  v.bad = len < 0 || len > a.cap;
  v.len = v.bad ? 0 : len;
  v.lo = a.window > 0 ? max(0, v.len - a.window) : 0;
  v.first = min(a.sinks, v.lo);
  v.n = v.first + v.len - v.lo;
  return v;
}
__device__ __forceinline__ int tiles_of(const Visible &v) { return (v.n + kTile - 1) / kTile; }

struct Plan {
  int b, i, n;   // sequence, unit within it, units of it
  int first;     // group index of the sequence's first unit
};

// units of a sequence of t tiles when a unit may have `most`
__device__ __forceinline__ int units_of(const PagedArgs &a, int t, long long most) {
  if (a.B >= kWhole || t == 0) return 1;
  return (int)((t + most - 1) / most);
}

// The sequence and part that group g is (by_group), or the units of sequence g.
// Every thread of the CTA calls it; b = -1 when there is no such group.
__device__ Plan find_plan(const PagedArgs &a, int g, bool by_group) {
  __shared__ long long s_red[kWarps];
  __shared__ Plan s_plan;
  const unsigned FULL = 0xffffffffu;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  Plan p;
  if (a.B >= kWhole) {
    p.b = g < a.B ? g : -1;
    p.i = 0;
    p.n = 1;
    p.first = g;
    return p;
  }
  if (a.B == 1) {
    const int t = tiles_of(visible(a, a.seq_len[0]));
    const long long most = max((long long)kMinTiles, ((long long)t * a.NH + kUnits - 1) / kUnits);
    p.n = units_of(a, t, most);
    p.first = 0;
    p.b = by_group && g >= p.n ? -1 : 0;
    p.i = by_group ? g : 0;
    return p;
  }
  const int k = (a.B + kThreads - 1) / kThreads;
  const int b0 = min((int)threadIdx.x * k, a.B), b1 = min(b0 + k, a.B);
  long long tiles = 0;
  for (int b = b0; b < b1; ++b) tiles += tiles_of(visible(a, a.seq_len[b]));
#pragma unroll
  for (int o = 16; o; o >>= 1) tiles += __shfl_xor_sync(FULL, tiles, o);
  if (lane == 0) s_red[warp] = tiles;
  if (threadIdx.x == 0) s_plan.b = -1;
  __syncthreads();
  tiles = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) tiles += s_red[w];
  __syncthreads();
  const long long most = max((long long)kMinTiles, (tiles * a.NH + kUnits - 1) / kUnits);
  int mine = 0;
  for (int b = b0; b < b1; ++b) mine += units_of(a, tiles_of(visible(a, a.seq_len[b])), most);
  int incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(FULL, incl, o);
    if (lane >= o) incl += x;
  }
  if (lane == 31) s_red[warp] = incl;
  __syncthreads();
  int at = incl - mine;
  for (int w = 0; w < warp; ++w) at += (int)s_red[w];
  if (by_group ? g >= at && g < at + mine : g >= b0 && g < b1) {
    for (int b = b0; b < b1; ++b) {
      const int n = units_of(a, tiles_of(visible(a, a.seq_len[b])), most);
      if (by_group ? g < at + n : b == g) {
        s_plan.b = b;
        s_plan.i = by_group ? g - at : 0;
        s_plan.n = n;
        s_plan.first = at;
        break;
      }
      at += n;
    }
  }
  __syncthreads();
  return s_plan;
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
// 16 bytes to shared memory, zeros (nothing read) when `bytes` is 0
__device__ __forceinline__ void cp16(uint32_t dst, const void *src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <int D> struct Shape {
  static constexpr int kRowBytes = 2 * D;
  static constexpr int kPart = kWarpKeys * kRowBytes;     // a warp's K (or V) rows of a tile
  static constexpr int kStages = D == 64 ? 4 : 3;
  static constexpr int kWarpBytes = kStages * 2 * kPart;
  static constexpr bool kQRegs = D <= 128;                // the query tile stays in registers
  static constexpr int kQBytes = kQRegs ? 0 : kRows * kRowBytes;
  static constexpr size_t kSmem = (size_t)kWarps * kWarpBytes + kQBytes;
  static_assert((size_t)kWarps * kRows * D * 4 <= (size_t)kWarps * kWarpBytes, "merge buffer");
};

template <typename T, int D, bool WEIGHTS>
__global__ void __launch_bounds__(kThreads) paged_attn_kernel(PagedArgs a) {
  grid_dep_sync();
  using Sh = Shape<D>;
  extern __shared__ __align__(128) unsigned char smem[];
  const unsigned FULL = 0xffffffffu;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g4 = lane >> 2, t4 = lane & 3;
  const int unit = blockIdx.x;
  const int h = unit % a.NH;
  const Plan plan = find_plan(a, unit / a.NH, true);
  if (plan.b < 0) return;
  const int b = plan.b;
  const int hkv = h / a.gt, head0 = hkv * a.G + (h % a.gt) * kRows;
  const int rows = min(kRows, a.G - (h % a.gt) * kRows);
  const Visible vis = visible(a, a.seq_len[b]);
  const int tiles = tiles_of(vis);
  const int t0 = (int)((long long)tiles * plan.i / plan.n);
  const int t1 = (int)((long long)tiles * (plan.i + 1) / plan.n);
  const int v_end = min(t1 * kTile, vis.n);

  __shared__ float s_m[kWarps][kRows], s_l[kWarps][kRows];
  __shared__ uint32_t s_bad[kWarps];

  // ------------------------------------------------------------ query tile
  const T *q = (const T *)a.q + ((size_t)b * a.Hq + head0) * D;
  uint32_t qf[Sh::kQRegs ? D / 16 : 1][4];
  const uint32_t sm0 = (uint32_t)__cvta_generic_to_shared(smem);
  const uint32_t sm_q = sm0 + kWarps * Sh::kWarpBytes;
  if (Sh::kQRegs) {
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
      const uint32_t *r0 = (const uint32_t *)(q + (size_t)g4 * D + k * 16 + t4 * 2);
      const uint32_t *r1 = (const uint32_t *)(q + (size_t)(g4 + 8) * D + k * 16 + t4 * 2);
      qf[k][0] = g4 < rows ? r0[0] : 0;
      qf[k][1] = g4 + 8 < rows ? r1[0] : 0;
      qf[k][2] = g4 < rows ? r0[4] : 0;
      qf[k][3] = g4 + 8 < rows ? r1[4] : 0;
    }
  } else {
    for (int i = threadIdx.x; i < kRows * (D / 8); i += kThreads) {
      const int r = i / (D / 8), c = i % (D / 8);
      const uint4 v = r < rows ? *(const uint4 *)(q + (size_t)r * D + c * 8) : make_uint4(0, 0, 0, 0);
      *(uint4 *)(smem + kWarps * Sh::kWarpBytes + r * Sh::kRowBytes + ((c ^ (r & 7)) * 16)) = v;
    }
    __syncthreads();
  }

  // ------------------------------------------------------------ the loads
  const uint32_t sm_w = sm0 + warp * Sh::kWarpBytes;
  const int32_t *table = a.table + (size_t)b * a.max_pages;
  const T *kv = (const T *)a.kv;
  const int64_t head_off = (int64_t)hkv * D;
  const int64_t row_elems = (int64_t)a.Hkv * D;
  uint32_t bad = 0;
  // lane r (and r + 16) looks up row r of this warp's part of a tile
  int n_id = 0, n_slot = -1;
  auto look_up = [&](int t) {
    const int v = t * kTile + warp * kWarpKeys + (lane & 15);
    n_slot = -1;
    if (t < t1 && v < v_end) {
      const int key = v < vis.first ? v : v - vis.first + vis.lo;
      const int pg = a.page_shift >= 0 ? key >> a.page_shift : key / a.page;
      n_slot = key - pg * a.page;
      n_id = table[pg];
    }
  };
  constexpr int CPR = D / 8;         // 16-byte pieces of a row
  constexpr int RPI = 32 / CPR;      // rows of one round of the warp's copies
  auto load_tile = [&](int stage) {  // the rows looked up last
    int64_t off = -1;
    if (n_slot >= 0) {
      if ((unsigned)n_id < (unsigned)a.num_pages)
        off = (int64_t)n_id * a.page_stride + (int64_t)n_slot * row_elems + head_off;
      else
        bad = 1;
    }
    const uint32_t dst0 = sm_w + stage * 2 * Sh::kPart;
#pragma unroll
    for (int i = 0; i < kWarpKeys / RPI; ++i) {
      const int r = i * RPI + lane / CPR, c = lane % CPR;
      const int64_t o = __shfl_sync(FULL, off, r);
      const T *src = o >= 0 ? kv + o + c * 8 : kv;
      const uint32_t n = o >= 0 ? 16u : 0u;
      const uint32_t dst = dst0 + r * Sh::kRowBytes + ((c ^ (r & 7)) * 16);
      cp16(dst, src, n);
      cp16(dst + Sh::kPart, o >= 0 ? src + a.kv_stride : kv, n);
    }
  };

  float o[D / 8][4];
#pragma unroll
  for (int j = 0; j < D / 8; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.0f;
  float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.0f, l1 = 0.0f;

  look_up(t0);
#pragma unroll
  for (int s = 0; s < Sh::kStages - 1; ++s) {
    load_tile(s);
    cp_commit();
    look_up(t0 + s + 1);
  }
  int st_load = Sh::kStages - 1, st = 0;
  for (int t = t0; t < t1; ++t) {
    cp_wait<Sh::kStages - 2>();
    __syncwarp();
    load_tile(st_load);  // tile t + kStages - 1, into the stage read last round
    cp_commit();
    look_up(t + Sh::kStages);
    const uint32_t sm_k = sm_w + st * 2 * Sh::kPart, sm_v = sm_k + Sh::kPart;
    st = st + 1 == Sh::kStages ? 0 : st + 1;
    st_load = st_load + 1 == Sh::kStages ? 0 : st_load + 1;

    // S = Q K^T: 16 query rows x 16 keys
    float s[2][4] = {};
    {
      const int key = ((lane >> 4) << 3) + (lane & 7), half = (lane >> 3) & 1;
      const uint32_t base = sm_k + key * Sh::kRowBytes;
      const int qr = (lane & 7) + ((lane >> 3) & 1) * 8, qh = lane >> 4;
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        uint32_t bk[4];
        ldsm4(bk, base + (((2 * k + half) ^ (key & 7)) * 16));
        if (Sh::kQRegs) {
          Pair<T>::mma(s[0], qf[k], bk[0], bk[1]);
          Pair<T>::mma(s[1], qf[k], bk[2], bk[3]);
        } else {
          uint32_t aq[4];
          ldsm4(aq, sm_q + qr * Sh::kRowBytes + (((2 * k + qh) ^ (qr & 7)) * 16));
          Pair<T>::mma(s[0], aq, bk[0], bk[1]);
          Pair<T>::mma(s[1], aq, bk[2], bk[3]);
        }
      }
    }
    const int v0 = t * kTile + warp * kWarpKeys + 2 * t4;  // keys v0, v0+1, v0+8, v0+9
    float mx0 = -INFINITY, mx1 = -INFINITY;
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const bool in = v0 + 8 * n + e < v_end;
        s[n][e] = in ? s[n][e] * a.scale_log2 : -INFINITY;
        s[n][2 + e] = in ? s[n][2 + e] * a.scale_log2 : -INFINITY;
        if (WEIGHTS && in) {
          float *sc = a.w_score + (((size_t)b * a.Hkv + hkv) * a.vis_max + v0 + 8 * n + e) * a.G +
                      (h % a.gt) * kRows;
          if (g4 < rows) sc[g4] = s[n][e];
          if (g4 + 8 < rows) sc[g4 + 8] = s[n][2 + e];
        }
        mx0 = fmaxf(mx0, s[n][e]);
        mx1 = fmaxf(mx1, s[n][2 + e]);
      }
    mx0 = fmaxf(mx0, __shfl_xor_sync(FULL, mx0, 1));
    mx1 = fmaxf(mx1, __shfl_xor_sync(FULL, mx1, 1));
    mx0 = fmaxf(mx0, __shfl_xor_sync(FULL, mx0, 2));
    mx1 = fmaxf(mx1, __shfl_xor_sync(FULL, mx1, 2));
    if (__any_sync(FULL, mx0 > m0 || mx1 > m1)) {
      const float n0 = fmaxf(m0, mx0), n1 = fmaxf(m1, mx1);
      // a row without a finite score yet: nothing to rescale
      const float f0 = n0 == -INFINITY ? 1.0f : ex2_approx(m0 - n0);
      const float f1 = n1 == -INFINITY ? 1.0f : ex2_approx(m1 - n1);
      m0 = n0;
      m1 = n1;
      l0 *= f0;
      l1 *= f1;
#pragma unroll
      for (int j = 0; j < D / 8; ++j) {
        o[j][0] *= f0;
        o[j][1] *= f0;
        o[j][2] *= f1;
        o[j][3] *= f1;
      }
    }
    const float z0 = m0 == -INFINITY ? 0.0f : m0, z1 = m1 == -INFINITY ? 0.0f : m1;
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        s[n][e] = ex2_approx(s[n][e] - z0);
        s[n][2 + e] = ex2_approx(s[n][2 + e] - z1);
        l0 += s[n][e];
        l1 += s[n][2 + e];
      }
    // P as the sum of two 16-bit parts: the weights keep twice the type's bits
    // (one part alone would add a rounding as large as the output's own)
    uint32_t ph[4], pl[4];
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float x = s[n][2 * r], y = s[n][2 * r + 1];
        const uint32_t hi = Pair<T>::pack(x, y);
        const float2 back = Pair<T>::unpack(hi);
        ph[2 * n + r] = hi;
        pl[2 * n + r] = Pair<T>::pack(x - back.x, y - back.y);
      }
    // O += P V
    {
      const int key = (((lane >> 3) & 1) << 3) + (lane & 7), half = lane >> 4;
      const uint32_t base = sm_v + key * Sh::kRowBytes;
#pragma unroll
      for (int j = 0; j < D / 16; ++j) {
        uint32_t bv[4];
        ldsm4t(bv, base + (((2 * j + half) ^ (key & 7)) * 16));
        Pair<T>::mma(o[2 * j], ph, bv[0], bv[1]);
        Pair<T>::mma(o[2 * j + 1], ph, bv[2], bv[3]);
        Pair<T>::mma(o[2 * j], pl, bv[0], bv[1]);
        Pair<T>::mma(o[2 * j + 1], pl, bv[2], bv[3]);
      }
    }
    __syncwarp();  // every lane is done with this stage before it is filled again
  }
  cp_wait<0>();

  // ------------------------------------------------------------ merge the warps
  l0 += __shfl_xor_sync(FULL, l0, 1);
  l1 += __shfl_xor_sync(FULL, l1, 1);
  l0 += __shfl_xor_sync(FULL, l0, 2);
  l1 += __shfl_xor_sync(FULL, l1, 2);
  bad = __any_sync(FULL, bad);
  if (t4 == 0) {
    s_m[warp][g4] = m0;
    s_m[warp][g4 + 8] = m1;
    s_l[warp][g4] = l0;
    s_l[warp][g4 + 8] = l1;
  }
  if (lane == 0) s_bad[warp] = bad;
  __syncthreads();
  float M0 = -INFINITY, M1 = -INFINITY;
  uint32_t flag = vis.bad ? SV_ROW_BAD_LEN : 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    M0 = fmaxf(M0, s_m[w][g4]);
    M1 = fmaxf(M1, s_m[w][g4 + 8]);
    if (s_bad[w]) flag |= SV_ROW_BAD_PAGE;
  }
  const float f0 = m0 == -INFINITY ? 0.0f : ex2_approx(m0 - M0);
  const float f1 = m1 == -INFINITY ? 0.0f : ex2_approx(m1 - M1);
  float *mo = (float *)smem + (size_t)warp * kRows * D;
#pragma unroll
  for (int j = 0; j < D / 8; ++j) {
    *(float2 *)(mo + g4 * D + j * 8 + t4 * 2) = make_float2(o[j][0] * f0, o[j][1] * f0);
    *(float2 *)(mo + (g4 + 8) * D + j * 8 + t4 * 2) = make_float2(o[j][2] * f1, o[j][3] * f1);
  }
  __syncthreads();
  const float *mr = (const float *)smem;
  const bool whole = plan.n == 1;
  for (int i = threadIdx.x; i < rows * (D / 2); i += kThreads) {
    const int r = i / (D / 2), c = (i % (D / 2)) * 2;
    float x = 0.0f, y = 0.0f, l = 0.0f, M = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float2 p = *(const float2 *)(mr + ((size_t)w * kRows + r) * D + c);
      x += p.x;
      y += p.y;
      M = fmaxf(M, s_m[w][r]);
    }
#pragma unroll
    for (int w = 0; w < kWarps; ++w)
      l += s_m[w][r] == -INFINITY ? s_l[w][r] : s_l[w][r] * ex2_approx(s_m[w][r] - M);
    if (whole) {
      const float nan = __int_as_float(0x7fffffff);
      const float inv = 1.0f / l;
      x = flag ? nan : l == 0.0f ? 0.0f : x * inv;
      y = flag ? nan : l == 0.0f ? 0.0f : y * inv;
      *(uint32_t *)((T *)a.out + ((size_t)b * a.Hq + head0 + r) * D + c) = Pair<T>::pack(x, y);
      if (c == 0) {
        const float lse2 = flag ? nan : l == 0.0f ? -INFINITY : M + log2f(l);
        if (a.lse) a.lse[(size_t)b * a.Hq + head0 + r] = lse2 * 0.693147180559945309f;
        if (WEIGHTS) a.w_lse[(size_t)b * a.Hq + head0 + r] = lse2;
      }
    } else {
      *(float2 *)(a.w_o + ((size_t)unit * a.rows + r) * D + c) = make_float2(x, y);
      if (c == 0) a.w_ml[(size_t)unit * a.rows + r] = make_float2(M, l);
    }
  }
  if (threadIdx.x == 0) {
    if (whole) {
      if (h == 0) {
        if (a.status) a.status[b] = flag;
        if (WEIGHTS) a.w_status[b] = flag;
      }
    } else {
      a.w_flag[unit] = flag;
    }
  }
}

// ---------------------------------------------------------------------------
// The join: one CTA per (sequence, KV head group, query row) merges the units'
// m, l and O; a sequence that was one unit is written already.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) paged_join_kernel(PagedArgs a, int with_weights) {
  grid_dep_sync();
  const unsigned FULL = 0xffffffffu;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int h = blockIdx.x % a.NH, b = blockIdx.x / a.NH, r = blockIdx.y;
  const Plan plan = find_plan(a, b, false);
  if (plan.n == 1) return;
  const int hkv = h / a.gt, head0 = hkv * a.G + (h % a.gt) * kRows;
  if (r >= min(kRows, a.G - (h % a.gt) * kRows)) return;
  __shared__ float s_red[kWarps];
  __shared__ uint32_t s_flag[kWarps];
  __shared__ float s_l[kWarps];
  __shared__ float s_o[kWarps][D];
  float M = -INFINITY;
  uint32_t flag = 0;
  for (int i = threadIdx.x; i < plan.n; i += kThreads) {
    const size_t u = (size_t)(plan.first + i) * a.NH + h;
    M = fmaxf(M, a.w_ml[u * a.rows + r].x);
    flag |= a.w_flag[u];
  }
  M = warp_max(M);
  flag = __reduce_or_sync(FULL, flag);
  if (lane == 0) {
    s_red[warp] = M;
    s_flag[warp] = flag;
  }
  __syncthreads();
  M = fmaxf(fmaxf(s_red[0], s_red[1]), fmaxf(s_red[2], s_red[3]));
  flag = s_flag[0] | s_flag[1] | s_flag[2] | s_flag[3];
  constexpr int E = D / 32;
  float acc[E] = {}, l = 0.0f;
#pragma unroll 4
  for (int i = warp; i < plan.n; i += kWarps) {
    const size_t u = (size_t)(plan.first + i) * a.NH + h;
    const float2 ml = a.w_ml[u * a.rows + r];
    const float f = ml.x == -INFINITY ? 0.0f : ex2_approx(ml.x - M);
    // an l of NaN without a finite m comes from the data and stays
    l += ml.x == -INFINITY ? ml.y : ml.y * f;
    const float *src = a.w_o + (u * a.rows + r) * D;
#pragma unroll
    for (int e = 0; e < E; e += 2) {
      const float2 x = *(const float2 *)(src + (e / 2) * 64 + lane * 2);
      acc[e] += x.x * f;
      acc[e + 1] += x.y * f;
    }
  }
#pragma unroll
  for (int e = 0; e < E; e += 2)
    *(float2 *)&s_o[warp][(e / 2) * 64 + lane * 2] = make_float2(acc[e], acc[e + 1]);
  if (lane == 0) s_l[warp] = l;
  __syncthreads();
  l = s_l[0] + s_l[1] + s_l[2] + s_l[3];
  const float nan = __int_as_float(0x7fffffff);
  const float inv = 1.0f / l;
  const size_t row = (size_t)b * a.Hq + head0 + r;
  for (int c = threadIdx.x * 2; c < D; c += kThreads * 2) {
    float x = s_o[0][c] + s_o[1][c] + s_o[2][c] + s_o[3][c];
    float y = s_o[0][c + 1] + s_o[1][c + 1] + s_o[2][c + 1] + s_o[3][c + 1];
    x = flag ? nan : l == 0.0f ? 0.0f : x * inv;
    y = flag ? nan : l == 0.0f ? 0.0f : y * inv;
    *(uint32_t *)((T *)a.out + row * D + c) = Pair<T>::pack(x, y);
  }
  if (threadIdx.x == 0) {
    const float lse2 = flag ? nan : l == 0.0f ? -INFINITY : M + log2f(l);
    if (a.lse) a.lse[row] = lse2 * 0.693147180559945309f;
    if (with_weights) a.w_lse[row] = lse2;
    if (h == 0 && r == 0) {
      if (a.status) a.status[b] = flag;
      if (with_weights) a.w_status[b] = flag;
    }
  }
}

// ---------------------------------------------------------------------------
// weight_sum += sum over the G query heads of exp(s - lse), from the scores
// the attention left: one thread per visible slot, so no two add to one place.
constexpr int kSumKeys = 256;
__global__ void __launch_bounds__(kSumKeys) paged_weights_kernel(PagedArgs a) {
  grid_dep_sync();
  const int b = blockIdx.x / a.Hkv, hkv = blockIdx.x % a.Hkv;
  if (a.w_status[b]) return;
  const Visible vis = visible(a, a.seq_len[b]);
  const float *lse = a.w_lse + (size_t)b * a.Hq + (size_t)hkv * a.G;
  for (int v = blockIdx.y * kSumKeys + threadIdx.x; v < vis.n; v += gridDim.y * kSumKeys) {
    const float *sc = a.w_score + (((size_t)b * a.Hkv + hkv) * a.vis_max + v) * a.G;
    float w = 0.0f;
    for (int g = 0; g < a.G; ++g) {
      const float z = lse[g];
      w += z == -INFINITY ? 0.0f : ex2_approx(sc[g] - z);
    }
    const int key = v < vis.first ? v : v - vis.first + vis.lo;
    a.weight_sum[((size_t)b * a.Hkv + hkv) * a.S + key] += w;
  }
}

// ------------------------------------------------------------------ host side
struct Sizes {
  int G, gt, NH, rows, cap, vis_max;
  long long groups, units;
  size_t o, ml, flag, status, lse, score, total;
};

// 0 when the shape is beyond what the kernels index
bool sizes_of(Sizes &z, int B, int Hq, int Hkv, int D, int page, int max_pages, int window,
              int sinks, int weights) {
  z.G = Hq / Hkv;
  z.gt = (z.G + kRows - 1) / kRows;
  z.NH = Hkv * z.gt;
  z.rows = z.G < kRows ? z.G : kRows;
  const long long cap = (long long)page * max_pages;
  if (cap > kMaxSlots) return false;
  z.cap = (int)cap;
  z.vis_max = z.cap;
  if (window > 0 && (long long)window + sinks < cap) z.vis_max = window + sinks;
  const long long tiles = (z.vis_max + kTile - 1) / kTile;
  if (B >= kWhole) {
    z.groups = B;
  } else {
    const long long by_len = (long long)B * ((tiles + kMinTiles - 1) / kMinTiles);
    const long long by_units = (long long)B + kUnits / z.NH;
    z.groups = by_len < by_units ? by_len : by_units;
    if (z.groups < B) z.groups = B;
  }
  z.units = z.groups * z.NH;
  if (z.units > 0x7fffffffLL || (long long)B * z.NH > 0x7fffffffLL) return false;
  const bool split = z.groups > B;
  size_t at = 0;
  auto take = [&](size_t n) {
    const size_t r = at;
    at = align_up(at + n, 256);
    return r;
  };
  z.o = take(split ? (size_t)z.units * z.rows * D * 4 : 0);
  z.ml = take(split ? (size_t)z.units * z.rows * 8 : 0);
  z.flag = take(split ? (size_t)z.units * 4 : 0);
  z.status = take(weights ? (size_t)B * 4 : 0);
  z.lse = take(weights ? (size_t)B * Hq * 4 : 0);
  z.score = take(weights ? (size_t)B * Hq * z.vis_max * 4 : 0);
  z.total = at;
  return true;
}

template <typename T, int D, bool W>
cudaError_t allow_smem() {
  static thread_local int set_dev = -1;
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev == set_dev) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(
      paged_attn_kernel<T, D, W>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Shape<D>::kSmem);
  if (e == cudaSuccess) set_dev = dev;
  return e;
}

template <typename T, int D>
sv_status run(const PagedArgs &a, const Sizes &z, bool weights, cudaStream_t st) {
  sv_status s;
  cudaError_t e = weights ? allow_smem<T, D, true>() : allow_smem<T, D, false>();
  if (e != cudaSuccess) return check_launch("paged_attention", e);
  {
    LaunchScope ls("paged_attention", st);
    e = weights ? launch_pdl(paged_attn_kernel<T, D, true>, dim3((unsigned)z.units), dim3(kThreads),
                             Shape<D>::kSmem, st, a)
                : launch_pdl(paged_attn_kernel<T, D, false>, dim3((unsigned)z.units), dim3(kThreads),
                             Shape<D>::kSmem, st, a);
    if ((s = check_launch("paged_attention", e)) != SV_OK) return s;
  }
  if (z.groups > a.B) {
    LaunchScope ls("paged_join", st);
    e = launch_pdl(paged_join_kernel<T, D>, dim3((unsigned)(a.B * a.NH), (unsigned)a.rows),
                   dim3(kThreads), 0, st, a, weights ? 1 : 0);
    if ((s = check_launch("paged_join", e)) != SV_OK) return s;
  }
  if (weights) {
    const int want = (z.vis_max + kSumKeys - 1) / kSumKeys;
    LaunchScope ls("paged_weights", st);
    e = launch_pdl(paged_weights_kernel, dim3((unsigned)(a.B * a.Hkv), (unsigned)(want < 65535 ? want : 65535)),
                   dim3(kSumKeys), 0, st, a);
    if ((s = check_launch("paged_weights", e)) != SV_OK) return s;
  }
  return SV_OK;
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
  if (!(scale > 0.0f) || !isfinite(scale)) return set_error(SV_ERR_INVALID_ARG, "scale must be > 0");
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
  a.scale_log2 = scale * 1.4426950408889634f;
  a.rows = z.rows;
  a.vis_max = z.vis_max;
  a.weight_sum = weight_sum;
  a.S = S;
  a.out = out;
  a.lse = out_lse;
  a.status = out_status;
  char *w = (char *)workspace;
  a.w_o = (float *)(w + z.o);
  a.w_ml = (float2 *)(w + z.ml);
  a.w_flag = (uint32_t *)(w + z.flag);
  a.w_status = (uint32_t *)(w + z.status);
  a.w_lse = (float *)(w + z.lse);
  a.w_score = (float *)(w + z.score);
  cudaStream_t st = (cudaStream_t)stream;
  const bool wt = weight_sum != nullptr;
  if (dt == SV_BF16)
    return D == 64    ? run<__nv_bfloat16, 64>(a, z, wt, st)
           : D == 128 ? run<__nv_bfloat16, 128>(a, z, wt, st)
                      : run<__nv_bfloat16, 256>(a, z, wt, st);
  return D == 64    ? run<__half, 64>(a, z, wt, st)
         : D == 128 ? run<__half, 128>(a, z, wt, st)
                    : run<__half, 256>(a, z, wt, st);
}
