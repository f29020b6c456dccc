// The prefix attention's join over a made-up workspace in which the wait of one
// CTA ran out: sequences whose rows it had parts of are told so, others not.
#include "prefix_attn.cu"

#include <cstdio>
#include <cstring>
#include <vector>

using namespace sv;

// The sequences' own slots have no part in this.
bool sv::paged_sums_workspace(size_t *bytes, int, int, int, int, int, int) {
  *bytes = 0;
  return true;
}
sv_status sv::paged_sums(const void *, const void *, int64_t, int64_t, sv_dtype, const int32_t *, const int32_t *, int, int, int, int,
                         int, int, int, float, float *, float2 *, uint32_t *, void *, cudaStream_t) {
  return SV_OK;
}

struct Part {
  size_t at;
  int column, p, head;
};

// Every part that the prefixes' launch writes, share by share.
static std::vector<Part> parts_of(const PrefixArgs &a, const std::vector<int> &len) {
  std::vector<Part> parts;
  long long all = 0;
  for (int n : len) all += (long long)a.Hkv * ((n + a.keys - 1) / a.keys);
  if (!all) return parts;
  for (int column = 0; column < (a.mtiles + 1) / 2; ++column) {
    const long long most = 2 * column + 1 < a.mtiles ? a.shares2 : a.shares1, shares = most < all ? most : all;
    long long t = 0;
    for (int p = 0; p < a.N; ++p)
      for (int head = 0; head < a.Hkv; ++head) {
        const long long end = t + (len[p] + a.keys - 1) / a.keys;
        for (long long s = 0; s < shares; ++s)
          if (s * all / shares < end && (s + 1) * all / shares > t)
            parts.push_back({(size_t)column * ((a.shares2 > a.shares1 ? a.shares2 : a.shares1) + (size_t)a.N * a.Hkv) + s +
                                 (size_t)p * a.Hkv + head, column, p, head});
        t = end;
      }
  }
  return parts;
}

template <typename V> static V *upload(const std::vector<V> &v) {
  V *d = nullptr;
  if (cudaMalloc(&d, v.size() * sizeof(V)) != cudaSuccess) return nullptr;
  cudaMemcpy(d, v.data(), v.size() * sizeof(V), cudaMemcpyHostToDevice);
  return d;
}

template <int ROWS> static int check(int N, int W, int Hkv, int G, const std::vector<int> &len) {
  constexpr int D = 64;
  const int B = N * W, Hq = Hkv * G, page = 16;
  int longest = 1;
  for (int n : len) longest = n > longest ? n : longest;
  Sizes z;
  if (!sizes_of(z, B, N, Hq, Hkv, D, page, 4)) return 1;
  PrefixArgs a = {};
  a.B = B, a.N = N, a.W = W, a.Hq = Hq, a.Hkv = Hkv, a.G = G, a.mtiles = z.mtiles;
  a.cap = (longest + page - 1) / page * page, a.keys = kKeys;
  a.shares2 = z.shares2, a.shares1 = z.shares1, a.rows = z.rows;
  const std::vector<Part> parts = parts_of(a, len);
  const size_t room = (size_t)((z.mtiles + 1) / 2) * ((z.shares2 > z.shares1 ? z.shares2 : z.shares1) + (size_t)N * Hkv);
  a.len = upload(len);
  a.w_o = upload(std::vector<float>(room * 2 * z.rows * D, 1.0f));
  a.w_ml = upload(std::vector<float2>(room * 2 * z.rows, make_float2(0.0f, 1.0f)));
  std::vector<uint32_t> clean(room, 0xffffffffu);  // nobody's: not to be looked at
  for (const Part &x : parts) clean[x.at] = 0;
  a.w_flag = upload(clean);
  JoinArgs j = {};
  j.own_o = upload(std::vector<float>((size_t)B * Hq * D, 1.0f));
  j.own_ml = upload(std::vector<float2>((size_t)B * Hq, make_float2(0.0f, 1.0f)));
  j.own_flag = upload(std::vector<uint32_t>(B, 0));
  j.out = upload(std::vector<uint16_t>((size_t)B * Hq * D, 0));
  j.lse = upload(std::vector<float>((size_t)B * Hq, 0.0f));
  a.status = upload(std::vector<uint32_t>(B, 0));
  const long long units = (long long)N * Hkv * (((long long)W * G + ROWS - 1) / ROWS);
  const unsigned ctas = (unsigned)((units + kJoinThreads / 32 - 1) / (kJoinThreads / 32));
  std::vector<uint32_t> status(B);
  std::vector<float> lse((size_t)B * Hq);
  int wrong = 0;
  for (size_t i = 0; i <= parts.size(); ++i) {  // the last time none
    std::vector<uint32_t> flags = clean;
    if (i < parts.size()) flags[parts[i].at] = SV_ROW_TIMEOUT;
    cudaMemcpy(a.w_flag, flags.data(), room * 4, cudaMemcpyHostToDevice);
    cudaMemset(a.status, 0, B * 4);  // as the prefixes' launch leaves it
    prefix_join_kernel<__nv_bfloat16, D, ROWS><<<ctas, kJoinThreads>>>(a, j);
    if (cudaMemcpy(status.data(), a.status, B * 4, cudaMemcpyDeviceToHost) != cudaSuccess) return 1;
    cudaMemcpy(lse.data(), j.lse, lse.size() * 4, cudaMemcpyDeviceToHost);
    for (int b = 0; b < B; ++b) {
      bool hit = false;  // some row of the sequence has the part
      for (int h = 0; h < Hq; ++h) {
        const bool of = i < parts.size() && parts[i].p == b / W && parts[i].head == h / G &&
                        parts[i].column == (b % W * G + h % G) / (2 * kRows);
        hit |= of;
        wrong += of != (lse[(size_t)b * Hq + h] != lse[(size_t)b * Hq + h]);
      }
      wrong += status[b] != (hit ? SV_ROW_TIMEOUT : 0u);
    }
  }
  printf("N %d W %d Hkv %d G %d rows %d: %zu parts, %d wrong\n", N, W, Hkv, G, ROWS, parts.size(), wrong);
  return wrong != 0;
}

template <int ROWS> static int checks() {
  return check<ROWS>(1, 4, 4, 2, {1000}) |                     // parts of four heads, many to each
         check<ROWS>(1, 3, 1, 5, {40000}) |                    // one head over the whole card
         check<ROWS>(2, 100, 3, 3, {700, 129}) |               // two columns, rows of a sequence in both
         check<ROWS>(40, 2, 8, 1, std::vector<int>(40, 300)) | // shares that hold several heads
         check<ROWS>(5, 2, 40, 1, {130, 0, 1, 500, 128}) |     // more heads than a warp's lanes, an empty prefix
         check<ROWS>(1, 2, 2, 300, {400}) |                    // a sequence's rows over three columns
         check<ROWS>(2, 3, 2, 2, {0, 0});
}

int main() { return checks<1>() | checks<kJoinRows>(); }
