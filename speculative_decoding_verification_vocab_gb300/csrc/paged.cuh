// paged.cuh -- the paged cache's attention as a part of another call: sums that
// are still to be joined.
#pragma once

#include "common.cuh"

namespace sv {

// sv_paged_attention without a window and weight sums, whose checks have been
// made: for every row (b, head) the unnormalised sums in fp32, o [B][Hq][D], the
// reference (log2 units) and the sum of its exponentials, ml [B][Hq], and the
// status bits of a sequence, flags [B].  False: a shape beyond what the kernels
// index.
bool paged_sums_workspace(size_t *bytes, int B, int Hq, int Hkv, int D, int page, int max_pages);
sv_status paged_sums(const void *q, const void *kv, int64_t kv_stride, int64_t page_stride, sv_dtype dt,
                     const int32_t *block_table, const int32_t *seq_len, int B, int Hq, int Hkv, int D, int page,
                     int max_pages, int num_pages, float scale, float *o, float2 *ml, uint32_t *flags, void *workspace,
                     cudaStream_t st);

}  // namespace sv
