// verify_probs.cu -- verification of a drafted chain from probabilities and
// given random numbers (sm_103a).
//
// [Lesson] "Decodificação Especulativa e EAGLE-3", "O invariante", Passo 1-3:
// accept d iff u < min(1, q(d) / p(d)), left to right; sample the first
// rejected position from (q - p)_+, or the bonus row on full acceptance.
//
// With probabilities given there is no row pass: the walk reads two numbers a
// position, and the draw needs one row (bonus) or one row pair (residual) per
// sequence, read once.  A cluster of C CTAs takes a sequence: every CTA walks
// (the same few loads) and sums the integer weights of its part of the row,
// warp by warp; each warp stores its sum to every CTA of the cluster, and after
// one cluster barrier every CTA finds the part that holds the threshold from
// its own shared memory.  The CTA whose part it is re-reads it (1 / (8 C) of
// the row, still in L2) and picks the token; the others are done.  No
// workspace, no counters, one launch.  (With the sums loaded from the other
// CTAs instead, which then have to stay until all have read, a CTA lived 19 us
// at V = 128256, 8 of them reading its rows.)
//
// Bound: one row pair per sequence, memory, where there are many sequences: 256
// at V = 128256 fp32, 43 us for 263 MB (0.90 of the copy rate; the rest is the
// first walk and the last pick, with idle memory).  Few: the chain of latencies
// (walk, row, barrier, pick), 6 us of GPU time for one sequence at V = 1000.
//
// The sum is exact: floor(w 2^62) of a w in [0, 2) is its 24-bit mantissa
// shifted into 63 bits, so the order of the additions cannot change the token.
#include "cluster.cuh"

namespace sv {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr unsigned kMaxCluster = 8;
constexpr int kDepth = 4;  // pieces of a lane in flight
constexpr uint32_t kTwo = 0x40000000u;  // bits of 2.0f: from here on, and below 0, an entry is bad

struct ProbArgs {
  const void *q, *p;  // p NULL: one-hot drafts
  int64_t q_seq, q_row, p_seq, p_row;  // elements between sequences and between rows
  const int32_t *draft, *n_draft;
  const float *ua, *us;
  int N, V;
  int per;  // elements of a warp's part, a multiple of 8
  int32_t *tokens, *alen;
  uint32_t *status;
};

// floor(w 2^62) for 0 <= w < 2: mantissa m of w = m 2^(e - 150), m 2^39 shifted
// right by 127 - e (other values give some number; they fault the sequence)
__device__ __forceinline__ unsigned long long weight(float w) {
  const uint32_t bits = __float_as_uint(w);
  const uint32_t m = (bits & 0x7fffffu) | 0x800000u;
  const uint32_t sh = min(127u - (bits >> 23), 63u);
  return ((unsigned long long)m << 39) >> sh;
}
// an entry's bits, -0 as +0: at least kTwo when it is negative, NaN or >= 2
__device__ __forceinline__ uint32_t entry_bits(float x) { return __float_as_uint(__fadd_rn(x, 0.0f)); }
__device__ __forceinline__ bool bad_entry(float x) { return entry_bits(x) >= kTwo; }
__device__ __forceinline__ bool bad_rand(float u) { return !(u >= 0.0f && u < 1.0f); }

// floor(u total) for 0 <= u < 1, total < 2^63
__device__ __forceinline__ unsigned long long threshold(float u, unsigned long long total) {
  const uint32_t bits = __float_as_uint(__fadd_rn(u, 0.0f));
  const uint32_t e = bits >> 23;
  const unsigned long long m = e ? ((bits & 0x7fffffu) | 0x800000u) : (bits & 0x7fffffu);
  const int sh = e ? 150 - (int)e : 149;  // u = m 2^-sh, sh >= 24
  const unsigned long long lo = m * total, hi = __umul64hi(m, total);
  if (sh >= 128) return 0;
  return sh >= 64 ? hi >> (sh - 64) : (hi << (64 - sh)) | (lo >> sh);
}

struct Sums {
  unsigned long long w;  // exact weights
  float f;               // the same in fp32, to see that 64 bits overflowed
  uint32_t top;          // largest entry_bits
};

template <bool PAIR>
__device__ __forceinline__ void add(Sums &s, float q, float p) {
  s.top = max(s.top, entry_bits(q));
  float w = q;
  if (PAIR) {
    s.top = max(s.top, entry_bits(p));
    w = fmaxf(__fsub_rn(q, p), 0.0f);
  }
  s.f += w;
  s.w += weight(w);
}

// one 16-byte vector of entries
template <bool PAIR>
__device__ __forceinline__ void add_vec(Sums &s, const uint4 &q, const uint4 &p, float) {
  add<PAIR>(s, __uint_as_float(q.x), __uint_as_float(p.x));
  add<PAIR>(s, __uint_as_float(q.y), __uint_as_float(p.y));
  add<PAIR>(s, __uint_as_float(q.z), __uint_as_float(p.z));
  add<PAIR>(s, __uint_as_float(q.w), __uint_as_float(p.w));
}
template <bool PAIR>
__device__ __forceinline__ void add_vec(Sums &s, const uint4 &q, const uint4 &p, uint16_t) {
  add<PAIR>(s, bf16_lo(q.x), bf16_lo(p.x));
  add<PAIR>(s, bf16_hi(q.x), bf16_hi(p.x));
  add<PAIR>(s, bf16_lo(q.y), bf16_lo(p.y));
  add<PAIR>(s, bf16_hi(q.y), bf16_hi(p.y));
  add<PAIR>(s, bf16_lo(q.z), bf16_lo(p.z));
  add<PAIR>(s, bf16_hi(q.z), bf16_hi(p.z));
  add<PAIR>(s, bf16_lo(q.w), bf16_lo(p.w));
  add<PAIR>(s, bf16_hi(q.w), bf16_hi(p.w));
}

__device__ __forceinline__ void cp16(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// This lane's share of the weights of [lo, hi) of a row (pair).  The lane's
// 16-byte pieces go through its own places in shared memory, kDepth of them in
// flight: registers enough for those would halve the CTAs on an SM, which are
// what hides the walk and the pick of one behind the rows of the others.
template <typename T, bool PAIR>
__device__ __forceinline__ Sums part_sums(const T *q, const T *p, int lo, int hi, int lane, uint4 *ring) {
  constexpr int VEC = 16 / sizeof(T);
  Sums s{0, 0.0f, 0};
  int i = lo;
  if (((uintptr_t)q | (PAIR ? (uintptr_t)p : 0)) % 16 == 0) {
    const int full = lo + (hi - lo) / VEC * VEC;  // lo is a multiple of 8
    const uint4 *mine = ring + threadIdx.x;
    const uint32_t at0 = (uint32_t)__cvta_generic_to_shared(mine);
    auto load = [&](int at, int slot) {
      if (at < full) {
        cp16(at0 + (2 * slot) * kThreads * 16, q + at);
        if (PAIR) cp16(at0 + (2 * slot + 1) * kThreads * 16, p + at);
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    int at = lo + lane * VEC;
#pragma unroll
    for (int j = 0; j < kDepth - 1; ++j) load(at + j * 32 * VEC, j);
    int slot = 0;
    for (; at < full; at += 32 * VEC) {
      load(at + (kDepth - 1) * 32 * VEC, slot == 0 ? kDepth - 1 : slot - 1);
      asm volatile("cp.async.wait_group %0;" ::"n"(kDepth - 1) : "memory");
      const uint4 qv = mine[(2 * slot) * kThreads];
      const uint4 pv = PAIR ? mine[(2 * slot + 1) * kThreads] : make_uint4(0, 0, 0, 0);
      add_vec<PAIR>(s, qv, pv, T());
      slot = slot + 1 == kDepth ? 0 : slot + 1;
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    i = full;
  }
  constexpr int U = 4;
  for (; i < hi; i += 32 * U) {
    float qv[U], pv[U];
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int at = i + j * 32 + lane;
      qv[j] = at < hi ? load_elem(q + at) : 0.0f;
      pv[j] = PAIR && at < hi ? load_elem(p + at) : 0.0f;
    }
#pragma unroll
    for (int j = 0; j < U; ++j) add<PAIR>(s, qv[j], pv[j]);
  }
  return s;
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 6) verify_probs_kernel(ProbArgs a, unsigned C) {
  grid_dep_sync();
  const unsigned FULL = 0xffffffffu;
  const int b = blockIdx.x / C;
  const uint32_t rank = C > 1 ? cluster_rank() : 0;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  __shared__ uint4 ring[2 * kDepth * kThreads];
  // all parts' sums, written by the cluster's warps: weights; fp32 sum (low
  // word) and largest entry (high).  A second round has places of its own.
  __shared__ unsigned long long s_w[2][kMaxCluster * kWarps], s_ft[2][kMaxCluster * kWarps];
  __shared__ int s_a, s_n;                     // accepted tokens; drafted tokens
  __shared__ uint32_t s_flags;                 // bits of the walk; kFault with them on a fault
  __shared__ unsigned long long s_left;        // the threshold within the part found
  __shared__ int s_part, s_again, s_token;
  __shared__ unsigned long long s_scan[kWarps];
  constexpr uint32_t kFault = 1u << 31;
  // every CTA has started before another stores to its shared memory: waited
  // for after the walk
  if (C > 1) asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory");
  const T *qrows = (const T *)a.q + b * a.q_seq;
  const T *prows = a.p ? (const T *)a.p + b * a.p_seq : nullptr;
  const float us = a.us[b];

  if (warp == 0) {  // the walk, 32 positions at a time
    int n = a.n_draft ? a.n_draft[b] : a.N;
    uint32_t flags = 0;
    if (n < 0 || n > a.N) {
      flags = kFault | SV_ROW_BAD_LEN;
      n = 0;
    }
    int acc = n;
    for (int i0 = 0; i0 < n && acc == n && !(flags & kFault); i0 += 32) {
      const int i = i0 + lane;
      uint32_t f = 0;
      bool stop = false;
      if (i < n) {
        const int d = a.draft[(size_t)b * a.N + i];
        const float u = a.ua[(size_t)b * a.N + i];
        if (d < 0 || d >= a.V) {
          f = kFault | SV_ROW_BAD_TOKEN;
        } else {
          const float qd = load_elem(qrows + i * a.q_row + d);
          const float pd = prows ? load_elem(prows + i * a.p_row + d) : 1.0f;
          if (bad_entry(qd) || bad_entry(pd)) f |= kFault | SV_ROW_NAN;
          if (pd == 0.0f) f |= SV_ROW_P_ZERO;
          // 24-bit mantissas: the product is exact in 64 bits
          stop = !((double)u * (double)pd < (double)qd) && pd != 0.0f;
        }
        if (bad_rand(u)) f |= kFault | SV_ROW_BAD_RAND;
      }
      const unsigned halt = __ballot_sync(FULL, stop || (f & kFault));
      const int first = halt ? __ffs(halt) - 1 : 32;
      // the bits of the positions walked, the one that ends the walk included
      flags |= __reduce_or_sync(FULL, lane <= first ? f : 0u);
      if (halt) acc = i0 + first;
    }
    if (bad_rand(us)) flags |= kFault | SV_ROW_BAD_RAND;
    if (lane == 0) {
      s_a = acc;
      s_n = n;
      s_flags = flags;
    }
  }
  __syncthreads();
  if (C > 1) asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
  const int n_acc = s_a;
  const bool rejected = n_acc < s_n;
  uint32_t flags = s_flags;
  const T *q = qrows + n_acc * a.q_row;
  const T *p = rejected && prows ? prows + n_acc * a.p_row : nullptr;
  // one-hot: the weight of the rejected token is what q has above 1
  int hot = rejected && !prows && !(flags & kFault) ? a.draft[(size_t)b * a.N + n_acc] : -1;
  const int parts = (int)C * kWarps;
  int token = -1;

  for (int round = 0; round < 2 && !(flags & kFault); ++round) {
    const int part = (int)rank * kWarps + warp;
    const long long lo64 = (long long)part * a.per;
    const int lo = (int)min(lo64, (long long)a.V), hi = (int)min(lo64 + a.per, (long long)a.V);
    Sums s = p ? part_sums<T, true>(q, p, lo, hi, lane, ring) : part_sums<T, false>(q, nullptr, lo, hi, lane, ring);
    if (hot >= lo && hot < hi && lane == 0) {
      const float x = load_elem(q + hot);
      const float over = fmaxf(__fsub_rn(x, 1.0f), 0.0f);
      s.w += weight(over) - weight(x);
      s.f += over - x;
    }
    const unsigned long long w = warp_sum_u64(s.w);
#pragma unroll
    for (int o = 16; o; o >>= 1) s.f += __shfl_xor_sync(FULL, s.f, o);
    const uint32_t top = __reduce_max_sync(FULL, s.top);
    const unsigned long long ft = (unsigned long long)top << 32 | __float_as_uint(s.f);
    if (C > 1) {
      if (lane < (int)C) {
        cluster_st_u64(&s_w[round][part], (uint32_t)lane, w);
        cluster_st_u64(&s_ft[round][part], (uint32_t)lane, ft);
      }
      cluster_sync();
    } else {
      if (lane == 0) {
        s_w[round][part] = w;
        s_ft[round][part] = ft;
      }
      __syncthreads();
    }
    if (warp == 0) {
      // lane l: the parts [l k, (l + 1) k)
      constexpr int K = (int)kMaxCluster * kWarps / 32;
      unsigned long long v[K], sum = 0;
      float f = 0.0f;
      uint32_t tp = 0;
      const int k = (parts + 31) / 32;
#pragma unroll
      for (int j = 0; j < K; ++j) {
        const int e = lane * k + j;
        v[j] = 0;
        if (j < k && e < parts) {
          v[j] = s_w[round][e];
          const unsigned long long ft = s_ft[round][e];
          f += __uint_as_float((uint32_t)ft);
          tp = max(tp, (uint32_t)(ft >> 32));
        }
        sum += v[j];
      }
      unsigned long long incl = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned long long x = __shfl_up_sync(FULL, incl, o);
        if (lane >= o) incl += x;
      }
      const unsigned long long total = __shfl_sync(FULL, incl, 31);
#pragma unroll
      for (int o = 16; o; o >>= 1) f += __shfl_xor_sync(FULL, f, o);
      tp = __reduce_max_sync(FULL, tp);
      // A sum of 2 or more is 2^63 or more in integers, exactly; from 4 on those
      // wrap around, which the fp32 sum, off by 2^-12 of itself at most (2048
      // additions a lane), tells from less than 2.
      const bool bad = tp >= kTwo || !(f < 3.0f) || total >> 63;
      const bool none = !bad && total == 0;
      if (lane == 0) {
        s_again = none && rejected && round == 0;
        s_part = -1;
        if (bad || (none && !s_again)) s_flags = flags | kFault | SV_ROW_NAN;
        if (s_again) s_flags = flags | SV_ROW_RESID_ZERO;
      }
      __syncwarp();
      if (!bad && total) {
        const unsigned long long t = threshold(us, total);
        unsigned long long before = incl - sum;
        if (t >= before && t < incl) {
#pragma unroll
          for (int j = 0; j < K; ++j) {
            if (t >= before && t < before + v[j]) {
              s_part = lane * k + j;
              s_left = t - before;
            }
            before += v[j];
          }
        }
      }
    }
    __syncthreads();
    flags = s_flags;
    const int found = s_part;
    const bool again = s_again;
    __syncthreads();  // read by all before another round writes them
    if (!again) {
      if (!(flags & kFault) && found / kWarps == (int)rank) {
        // this CTA's part `found`: thread t takes k elements in a row
        const int plo = found * a.per, phi = min(plo + a.per, a.V);
        const int k = (phi - plo + kThreads - 1) / kThreads;
        const int i0 = min(plo + (int)threadIdx.x * k, phi), i1 = min(i0 + k, phi);
        auto at = [&](int i) {
          const float x = load_elem(q + i);
          const float y = p ? load_elem(p + i) : i == hot ? 1.0f : 0.0f;
          return weight(fmaxf(__fsub_rn(x, y), 0.0f));
        };
        unsigned long long mine = 0;
        for (int i = i0; i < i1; ++i) mine += at(i);
        unsigned long long incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const unsigned long long x = __shfl_up_sync(FULL, incl, o);
          if (lane >= o) incl += x;
        }
        if (lane == 31) s_scan[warp] = incl;
        __syncthreads();
        for (int j = 0; j < warp; ++j) incl += s_scan[j];
        unsigned long long before = incl - mine;
        const unsigned long long t = s_left;
        if (t >= before && t < incl) {
          for (int i = i0; i < i1; ++i) {
            const unsigned long long x = at(i);
            if (t < before + x) {
              s_token = i;
              break;
            }
            before += x;
          }
        }
        __syncthreads();
        token = s_token;
      }
      break;
    }
    p = nullptr;  // no residual mass: draw from q itself
    hot = -1;
  }

  // the CTA that has the token writes the sequence's outputs (on a fault, the first)
  const bool fault = flags & kFault;
  if (fault ? rank == 0 : token >= 0) {
    int32_t *out = a.tokens + (size_t)b * (a.N + 1);
    for (int i = threadIdx.x; i <= a.N; i += kThreads)
      out[i] = fault || i > n_acc ? -1 : i < n_acc ? a.draft[(size_t)b * a.N + i] : token;
    if (threadIdx.x == 0) {
      a.alen[b] = fault ? 0 : n_acc;
      a.status[b] = flags & ~kFault;
    }
  }
}

template <typename T>
cudaError_t launch(const ProbArgs &a, int B, unsigned C, cudaStream_t st) {
  return launch_pdl_cluster(verify_probs_kernel<T>, dim3((unsigned)B * C), dim3(kThreads), C, 0, st,
                            a, C);
}

}  // namespace
}  // namespace sv

using namespace sv;

extern "C" sv_status sv_verify_chain_probs(const void *qprobs, int64_t q_seq, int64_t q_row,
                                           const void *pprobs, int64_t p_seq, int64_t p_row,
                                           sv_dtype dt, const int32_t *draft_tokens,
                                           const int32_t *n_draft, const float *u_accept,
                                           const float *u_sample, int B, int N, int V,
                                           int32_t *out_tokens, int32_t *out_accept_len,
                                           uint32_t *out_status, void *stream) {
  if (B < 0 || N < 0 || V < 1) return set_error(SV_ERR_INVALID_ARG, "need B >= 0, N >= 0, V >= 1");
  if (dt != SV_F32 && dt != SV_BF16)
    return set_error(SV_ERR_INVALID_ARG, "probabilities are SV_F32 or SV_BF16, not dtype %d", (int)dt);
  if (V > SV_MAX_VOCAB) return set_error(SV_ERR_UNSUPPORTED, "V > %d", SV_MAX_VOCAB);
  if (N > SV_MAX_POSITIONS) return set_error(SV_ERR_UNSUPPORTED, "N > %d", SV_MAX_POSITIONS);
  if (B > (1 << 24)) return set_error(SV_ERR_UNSUPPORTED, "B > %d", 1 << 24);
  const int64_t most = INT64_MAX / 16;  // of any offset, in elements
  auto bad_stride = [most](int64_t x, int64_t n) { return x < 0 || (n > 0 && x > most / n); };
  if (bad_stride(q_seq, B) || bad_stride(q_row, N) || (pprobs && (bad_stride(p_seq, B) || bad_stride(p_row, N))))
    return set_error(SV_ERR_INVALID_ARG, "negative or too large stride");
  if (B == 0) return SV_OK;
  if (!qprobs || !u_sample || !out_tokens || !out_accept_len || !out_status ||
      (N > 0 && (!draft_tokens || !u_accept)))
    return set_error(SV_ERR_INVALID_ARG, "null pointer");
  const size_t es = dt == SV_F32 ? 4 : 2;
  if ((uintptr_t)qprobs % es || (uintptr_t)pprobs % es || (uintptr_t)draft_tokens % 4 ||
      (uintptr_t)n_draft % 4 || (uintptr_t)u_accept % 4 || (uintptr_t)u_sample % 4 ||
      (uintptr_t)out_tokens % 4 || (uintptr_t)out_accept_len % 4 || (uintptr_t)out_status % 4)
    return set_error(SV_ERR_INVALID_ARG, "misaligned pointer");
  if (N == 0) pprobs = nullptr;
  sv_status s;
  if ((s = map_arg(qprobs, "qprobs")) != SV_OK || (s = map_arg(pprobs, "pprobs")) != SV_OK ||
      (s = map_arg(draft_tokens, "draft_tokens")) != SV_OK ||
      (s = map_arg(n_draft, "n_draft")) != SV_OK || (s = map_arg(u_accept, "u_accept")) != SV_OK ||
      (s = map_arg(u_sample, "u_sample")) != SV_OK ||
      (s = map_arg(out_tokens, "out_tokens")) != SV_OK ||
      (s = map_arg(out_accept_len, "out_accept_len")) != SV_OK ||
      (s = map_arg(out_status, "out_status")) != SV_OK)
    return s;
  // CTAs of a sequence: one per 32 KB of a row, up to 8 (4 at most: 49 us where
  // 8 take 44; twice as many for short rows: no change)
  unsigned C = 1;
  while (C < kMaxCluster && (size_t)V * es > C * (size_t)32768) C *= 2;
  ProbArgs a;
  a.q = qprobs;
  a.p = pprobs;
  a.q_seq = q_seq;
  a.q_row = q_row;
  a.p_seq = p_seq;
  a.p_row = p_row;
  a.draft = draft_tokens;
  a.n_draft = n_draft;
  a.ua = u_accept;
  a.us = u_sample;
  a.N = N;
  a.V = V;
  const int parts = (int)C * kWarps;
  a.per = ((V + parts - 1) / parts + 7) / 8 * 8;
  a.tokens = out_tokens;
  a.alen = out_accept_len;
  a.status = out_status;
  cudaStream_t st = (cudaStream_t)stream;
  LaunchScope ls("verify_probs", st);
  return check_launch("verify_probs", dt == SV_F32 ? launch<float>(a, B, C, st)
                                                   : launch<uint16_t>(a, B, C, st));
}
