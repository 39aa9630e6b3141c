// The paged 8-bit key / value cache (layout in qmv.h): what its kernels share.
#pragma once
#include "common.cuh"

namespace qmv {

constexpr int KV_HEADER = 16;     // bytes before the codes of a record
constexpr int KV_MAX_PAGES = 1 << 20;

__host__ __device__ constexpr int kv_page_bytes(int D, int P) { return KV_HEADER + 2 * P * D; }
__host__ __device__ constexpr int kv_bounds_bytes(int D) { return KV_HEADER + 2 * D; }

struct KvParams {
  uint8_t* pages;
  uint8_t* bounds;
  const int32_t* table;
  const int32_t* lens;
  const int32_t* starts;  // or nullptr: one token per sequence
  int H, P, log_p, n_pages, n_seq, max_pages, n_tok;
  unsigned* err;
#ifdef QMV_DEBUG
  long long pages_len, bounds_len, table_len;
#endif
};

// A sequence of the batch: tokens [t0, t0 + n) of the call, at positions
// len - n + i.
struct KvSeq {
  int t0, n, len;
};

// The sequence's fields, clamped to what the call's sizes allow (a
// contradiction sets QMV_DEVERR_BATCH): any content of lens and starts gives
// indexes inside the buffers.
__device__ __forceinline__ KvSeq kv_seq(const KvParams& p, int s) {
  KvSeq q;
  int a = s, b = s + 1;
  if (p.starts) {
    a = p.starts[s];
    b = p.starts[s + 1];
  }
  int len = p.lens[s];
  const long long cap = (long long)p.max_pages * p.P;
  if (a < 0 || b < a || b > p.n_tok || len < 0 || len > cap) {
    set_error(p.err, QMV_DEVERR_BATCH);
    a = min(max(a, 0), p.n_tok);
    b = min(max(b, a), p.n_tok);
    len = (int)min((long long)max(len, 0), cap);
  }
  q.t0 = a;
  q.n = b - a;
  q.len = len;
  return q;
}

// The last sequence whose at(s) is at most x (at does not fall with s, and the
// first is taken to be at most x): a 32-ary search by each warp of the caller,
// one or two loads deep, the same answer in all lanes.
template <class At>
__device__ __forceinline__ int last_seq_at_most(int n_seq, int x, At at) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = n_seq;  // the sequence is one of [lo, lo + n)
  while (n > 1) {
    const int step = (n + 31) / 32, s = lo + (lane + 1) * step;  // candidates after lo
    const bool at_or_after = (lane + 1) * step < n && at(s) <= x;
    const int k = __popc(__ballot_sync(0xffffffffu, at_or_after));
    lo += k * step;
    n = min(n - k * step, step);
  }
  return lo;
}

// The page of the cache that holds page `pg` of sequence s, or -1 if the
// table's entry is no page (QMV_DEVERR_PAGE).
__device__ __forceinline__ int kv_page(const KvParams& p, int s, int pg) {
  const long long at = (long long)s * p.max_pages + pg;
  if (!QMV_CHECK(in_range(at, 1, p.table_len, p.err))) return -1;
  const int id = p.table[at];
  if (id < 0 || id >= p.n_pages) {
    set_error(p.err, QMV_DEVERR_PAGE);
    return -1;
  }
  return id;
}

}  // namespace qmv
