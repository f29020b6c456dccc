// vocab_rows.cuh -- one pass over a slice of a vocabulary row: 16-byte pieces
// on their way to shared memory by asynchronous copies, online softmax sums and
// the entropy's sum in registers (sm_103a).  Shared by the log probabilities of
// given tokens and the distillation loss.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "cluster.cuh"

namespace sv {

constexpr int kPieces = 4;  // of a thread in a group
// a group of a CTA: 16-byte pieces, and their bytes
template <int THREADS> constexpr int kGroupVecs = kPieces * THREADS;
template <int THREADS> constexpr int kGroupBytes = kGroupVecs<THREADS> * 16;
constexpr unsigned kMaxRowCluster = 8;
constexpr float kLog2eF = 1.4426950408889634f;
// The reference of the exponentials follows the maximum only when an element
// exceeds it by more than this (log2 units): past a row's first pieces hardly
// any does, and sums of 2^22 terms of 2^8 are far from the end of 32 bits.
constexpr float kRefSlack = 8.0f;

// ------------------------------------------------------------ element types
// most, most4: the largest element of a piece, of a group's pieces (NaN ones passed
// over)
template <typename T> struct RowElem;
template <> struct RowElem<float> {
  static constexpr int VEC = 4;
  static constexpr uint32_t kNegInf = 0xff800000u;
  static __device__ __forceinline__ float load(const float *p) { return *p; }
  static __device__ __forceinline__ void unpack(const uint4 &w, float (&x)[4]) {
    x[0] = __uint_as_float(w.x);
    x[1] = __uint_as_float(w.y);
    x[2] = __uint_as_float(w.z);
    x[3] = __uint_as_float(w.w);
  }
  static __device__ __forceinline__ float most(const uint4 &w) {
    return fmaxf(fmaxf(__uint_as_float(w.x), __uint_as_float(w.y)),
                 fmaxf(__uint_as_float(w.z), __uint_as_float(w.w)));
  }
  static __device__ __forceinline__ float most4(const uint4 (&w)[kPieces]) {
    float m = most(w[0]);
#pragma unroll
    for (int j = 1; j < kPieces; ++j) {
      m = max3(m, __uint_as_float(w[j].x), __uint_as_float(w[j].y));
      m = max3(m, __uint_as_float(w[j].z), __uint_as_float(w[j].w));
    }
    return m;
  }
  static __device__ __forceinline__ uint4 pack(const float (&x)[4]) {
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
  }
  static __device__ __forceinline__ float store(float x) { return x; }
};
template <> struct RowElem<__nv_bfloat16> {
  static constexpr int VEC = 8;
  static constexpr uint32_t kNegInf = 0xff80ff80u;
  static __device__ __forceinline__ float load(const __nv_bfloat16 *p) { return __bfloat162float(*p); }
  static __device__ __forceinline__ void unpack(const uint4 &w, float (&x)[8]) {
    const uint32_t q[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = bf16_lo(q[i]);
      x[2 * i + 1] = bf16_hi(q[i]);
    }
  }
  static __device__ __forceinline__ float most(const uint4 &w) {
    const uint32_t m = bf2_max(bf2_max(w.x, w.y), bf2_max(w.z, w.w));
    return fmaxf(bf16_lo(m), bf16_hi(m));
  }
  static __device__ __forceinline__ float most4(const uint4 (&w)[kPieces]) {
    uint32_t m[kPieces];
#pragma unroll
    for (int j = 0; j < kPieces; ++j) m[j] = bf2_max(bf2_max(w[j].x, w[j].y), bf2_max(w[j].z, w[j].w));
    const uint32_t a = bf2_max(bf2_max(m[0], m[1]), bf2_max(m[2], m[3]));
    return fmaxf(bf16_lo(a), bf16_hi(a));
  }
  static __device__ __forceinline__ uint32_t pair(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *(const uint32_t *)&v;
  }
  static __device__ __forceinline__ uint4 pack(const float (&x)[8]) {
    return make_uint4(pair(x[0], x[1]), pair(x[2], x[3]), pair(x[4], x[5]), pair(x[6], x[7]));
  }
  static __device__ __forceinline__ __nv_bfloat16 store(float x) { return __float2bfloat16_rn(x); }
};
template <> struct RowElem<__half> {
  static constexpr int VEC = 8;
  static constexpr uint32_t kNegInf = 0xfc00fc00u;
  static __device__ __forceinline__ float load(const __half *p) { return __half2float(*p); }
  static __device__ __forceinline__ void unpack(const uint4 &w, float (&x)[8]) {
    const uint32_t q[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(*(const __half2 *)&q[i]);
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
  static __device__ __forceinline__ float most(const uint4 &w) {
    const __half2 m = __hmax2(__hmax2(*(const __half2 *)&w.x, *(const __half2 *)&w.y),
                              __hmax2(*(const __half2 *)&w.z, *(const __half2 *)&w.w));
    const float2 f = __half22float2(m);
    return fmaxf(f.x, f.y);
  }
  static __device__ __forceinline__ float most4(const uint4 (&w)[kPieces]) {
    __half2 m[kPieces];
#pragma unroll
    for (int j = 0; j < kPieces; ++j)
      m[j] = __hmax2(__hmax2(*(const __half2 *)&w[j].x, *(const __half2 *)&w[j].y),
                     __hmax2(*(const __half2 *)&w[j].z, *(const __half2 *)&w[j].w));
    const float2 f = __half22float2(__hmax2(__hmax2(m[0], m[1]), __hmax2(m[2], m[3])));
    return fmaxf(f.x, f.y);
  }
  static __device__ __forceinline__ uint32_t pair(float lo, float hi) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *(const uint32_t *)&v;
  }
  static __device__ __forceinline__ uint4 pack(const float (&x)[8]) {
    return make_uint4(pair(x[0], x[1]), pair(x[2], x[3]), pair(x[4], x[5]), pair(x[6], x[7]));
  }
  static __device__ __forceinline__ __half store(float x) { return __float2half_rn(x); }
};

// A row of V elements lies as `head` elements up to the first 16-byte border,
// `vecs` whole pieces, and a tail.  CTA `rank` of C takes the pieces [v0, v1);
// the first CTA the single elements too, one to each of its first threads.
struct RowSlice {
  int head, vecs, v0, v1;
  int singles;  // of the head and the tail
};
template <typename T> __device__ __forceinline__ RowSlice row_slice(const T *row, int V, uint32_t rank, unsigned C) {
  constexpr int VEC = RowElem<T>::VEC;
  RowSlice s;
  const int off = (int)((uintptr_t)row % 16 / sizeof(T));
  s.head = min(off ? VEC - off : 0, V);
  s.vecs = (V - s.head) / VEC;
  s.singles = V - s.vecs * VEC;
  const int per = (s.vecs + (int)C - 1) / (int)C;
  s.v0 = min((int)rank * per, s.vecs);
  s.v1 = min(s.v0 + per, s.vecs);
  return s;
}
// element of the row that single i is
template <typename T> __device__ __forceinline__ int single_at(const RowSlice &s, int i) {
  return i < s.head ? i : i + s.vecs * RowElem<T>::VEC;
}
template <int THREADS> __device__ __forceinline__ int row_groups(const RowSlice &s) {
  return (s.v1 - s.v0 + kGroupVecs<THREADS> - 1) / kGroupVecs<THREADS>;
}

// Group g's pieces of this thread into its own places of slot `slot`; places
// without a piece hold -inf, which no sum and no list takes up.  What a thread
// reads there it has copied itself, so no barrier stands between.
template <int THREADS, typename T>
__device__ __forceinline__ void load_group(const T *row, const RowSlice &s, int g, int slot, unsigned char *ring) {
  const int v = s.v0 + g * kGroupVecs<THREADS> + (int)threadIdx.x;
  const uint4 *src = (const uint4 *)(row + s.head) + v;
  unsigned char *at = ring + (size_t)slot * kGroupBytes<THREADS> + threadIdx.x * 16;
  const uint32_t dst = (uint32_t)__cvta_generic_to_shared(at);
  if (s.v0 + (g + 1) * kGroupVecs<THREADS> <= s.v1) {  // all of them
#pragma unroll
    for (int j = 0; j < kPieces; ++j)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst + j * THREADS * 16), "l"(src + j * THREADS)
                   : "memory");
    return;
  }
#pragma unroll 1
  for (int j = 0; j < kPieces; ++j) {
    if (v + j * THREADS < s.v1)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst + j * THREADS * 16), "l"(src + j * THREADS)
                   : "memory");
    else
      *(uint4 *)(at + j * THREADS * 16) =
          make_uint4(RowElem<T>::kNegInf, RowElem<T>::kNegInf, RowElem<T>::kNegInf, RowElem<T>::kNegInf);
  }
}
__device__ __forceinline__ void group_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void group_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
template <int THREADS> __device__ __forceinline__ uint4 ring_piece(const unsigned char *ring, int slot, int j) {
  return *(const uint4 *)(ring + (size_t)slot * kGroupBytes<THREADS> + (j * THREADS + threadIdx.x) * 16);
}

// ------------------------------------------------------------ online sums
// l = sum 2^y and, if asked, s = sum 2^y y, y = (x - ref) k, k = log2(e) / T.
// Differences are taken before the product: a row masked with its type's lowest
// value then gives 2^-inf = 0 or, where nothing else is left, 2^0.  An element
// of -inf adds 0 to s too (y is held above -150, where 2^y is 0); a NaN or +inf
// makes l NaN.
struct RowSums {
  float top;                  // the reference, or -inf while nothing is above -inf
  float lim;                  // raise the reference above this
  unsigned long long nref;    // minus the reference (0 in place of -inf), twice
  unsigned long long l2, s2;  // packed pairs of partial sums
};
__device__ __forceinline__ RowSums row_sums() { return RowSums{-INFINITY, -INFINITY, 0ull, 0ull, 0ull}; }

template <bool ENT> __device__ __forceinline__ void raise(RowSums &r, float to, float k) {
  // y grows by d: 2^y y becomes 2^d (2^y y + d 2^y)
  const float d = r.top == -INFINITY ? 0.0f : (r.top - to) * k;
  const unsigned long long f = f2_splat(r.top == -INFINITY ? 0.0f : ex2_approx(d));
  if (ENT) r.s2 = f2_mul(f2_fma(f2_splat(fmaxf(d, -150.0f)), r.l2, r.s2), f);
  r.l2 = f2_mul(r.l2, f);
  r.top = to;
  r.nref = f2_splat(-to);
  r.lim = to + kRefSlack / k;
}
// k2: k, twice
template <bool ENT> __device__ __forceinline__ void add_pair(RowSums &r, float a, float b, unsigned long long k2) {
  const unsigned long long y = f2_mul(f2_add(f2_pack(a, b), r.nref), k2);
  float y0, y1;
  f2_unpack(y, y0, y1);
  const unsigned long long e = f2_pack(ex2_approx(y0), ex2_approx(y1));
  r.l2 = f2_add(r.l2, e);
  if (ENT) r.s2 = f2_fma(e, f2_pack(fmaxf(y0, -150.0f), fmaxf(y1, -150.0f)), r.s2);
}
template <typename T, bool ENT>
__device__ __forceinline__ void add_piece(RowSums &r, const uint4 &w, unsigned long long k2) {
  float x[RowElem<T>::VEC];
  RowElem<T>::unpack(w, x);
#pragma unroll
  for (int i = 0; i < RowElem<T>::VEC; i += 2) add_pair<ENT>(r, x[i], x[i + 1], k2);
}
template <bool ENT> __device__ __forceinline__ void add_single(RowSums &r, float x, float k) {
  if (x > r.lim) raise<ENT>(r, x, k);
  add_pair<ENT>(r, x, -INFINITY, f2_splat(k));
}

// The sums as three numbers that join: reference (-inf: none), l, s.
struct RowPart {
  float top, l, s;
};
// a part's sums against another reference, at least its own
__device__ __forceinline__ RowPart moved(const RowPart &p, float top, float k) {
  if (p.top == -INFINITY) return RowPart{top, p.l, p.s};  // 0, or NaN from the data
  const float d = (p.top - top) * k, f = ex2_approx(d);
  return RowPart{top, p.l * f, f * fmaf(fmaxf(d, -150.0f), p.l, p.s)};
}
__device__ __forceinline__ RowPart warp_join(RowPart p, float k) {
  p = moved(p, warp_max(p.top), k);
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    p.l += __shfl_xor_sync(0xffffffffu, p.l, o);
    p.s += __shfl_xor_sync(0xffffffffu, p.s, o);
  }
  return p;
}
__device__ __forceinline__ RowPart part_of(const RowSums &r) {
  float l0, l1, s0, s1;
  f2_unpack(r.l2, l0, l1);
  f2_unpack(r.s2, s0, s1);
  return RowPart{r.top, l0 + l1, s0 + s1};
}
__device__ __forceinline__ void cluster_arrive_relaxed() {
  asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }

// CTAs to a row: one for each 16 KB of it while there are no more than `most` in all.
// More of them have each its way to the first piece and back, and clusters wait for room
// together (120 rows of 128256 bf16 with 64 alternatives: 28 us by 4 CTAs each, 18 by 2;
// 300 rows: 29 by 2, 25 by 1; 80 rows with 5: 13 by 4, 14 by 2; 300 rows: 27 by 2, 21 by 1).
inline unsigned row_ctas(size_t row_bytes, long long rows, long long most) {
  unsigned c = 1;
  while (c < kMaxRowCluster && row_bytes > c * (size_t)16384 && rows * c * 2 <= most) c *= 2;
  return c;
}

}  // namespace sv
