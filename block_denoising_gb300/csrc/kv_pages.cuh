// Pages of the paged key/value cache (include/dinfer_kv.h): growing, forking,
// freeing and compacting sequences, and storing new rows.
//
// The book-keeping (who gets which page) is a few thousand integers and a
// chain of dependent decisions, so one CTA of 1024 threads does it with block
// scans; what moves bytes is a second kernel over the whole GPU that reads the
// list of (source page, destination page, tokens) the first one left.  Pages
// are always handed out lowest first, so a call's result does not depend on
// which thread ran when.
#pragma once
#include <cstdint>

#include "common.cuh"

namespace dinfer {

// status bits of the cache (DINFER_KV_* of dinfer_kv.h)
enum : uint32_t { KV_BAD_SEQ = 1, KV_NO_PAGES = 2, KV_BAD_PAGE = 4, KV_SHARED = 8, KV_FULL = 16 };

constexpr int kKvMaxEntries = 1024;  // sequences a call names: one thread each
constexpr int kKvPlanThreads = 1024;
constexpr int kKvScanItems = 16;     // pages a thread looks at per scan step
constexpr int kKvHead = 16;          // int32 header words of the state

// n / d for 0 <= n < 2^31 by multiplication (Granlund and Montgomery, "Division by
// invariant integers using multiplication", 1994): with 2^(shift-1) < d <= 2^shift
// and mul = floor(2^32 (2^shift - d) / d) + 1, n / d = (hi(mul n) + n) >> shift;
// hi(mul n) <= n, so the sum stays below 2^32.
struct FastDiv {
  uint32_t d, mul, shift;
  __host__ __device__ static FastDiv make(uint32_t d) {
    FastDiv f{d, 0, 0};
    while ((1ull << f.shift) < d) ++f.shift;
    f.mul = (uint32_t)((((1ull << f.shift) - d) << 32) / d + 1);
    return f;
  }
  __device__ __forceinline__ uint32_t div(uint32_t n) const { return (__umulhi(mul, n) + n) >> shift; }
};

// The cache as the kernels see it.  Strides in 16-byte vectors; the state is
//   [0] status  [1] pages below it are all in use  [2] pages to copy  [3] pages in use (compact)
//   owner [max_seqs] (zero between calls)  base [1024]  src, dst, tok [num_pages]
struct KvPages {
  uint4* k;
  uint4* v;
  int64_t layer_stride, page_stride, token_stride, head_stride;
  int32_t* table;
  int32_t* lens;
  int32_t* refs;
  int32_t* state;
  int n_layers, num_pages, page_size, kv_heads, head_vecs;  // head_vecs: 16-byte vectors of one head's row
  int max_seqs, max_pages;
  FastDiv page_div;

  __device__ int32_t* owner() const { return state + kKvHead; }
  __device__ int32_t* base() const { return owner() + max_seqs; }
  __device__ int32_t* src() const { return base() + kKvMaxEntries; }
  __device__ int32_t* dst() const { return src() + num_pages; }
  __device__ int32_t* tok() const { return dst() + num_pages; }
  __device__ void flag(uint32_t bit) const { atomicOr(reinterpret_cast<unsigned*>(state), bit); }
  __device__ int pages_of(int len) const { return len > 0 ? (int)page_div.div((uint32_t)len - 1u) + 1 : 0; }
  __device__ bool valid_len(int len) const { return len >= 0 && (int64_t)len <= (int64_t)max_pages * page_size; }
};

// Exclusive sum of v over the CTA's 1024 threads; *total receives the sum.
template <typename N>
__device__ __forceinline__ N kv_block_scan(N v, N* total) {
  __shared__ N warp_sums[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  N inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const N u = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += u;
  }
  if (lane == 31) warp_sums[warp] = inc;
  __syncthreads();
  if (warp == 0) {
    N w = warp_sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const N u = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += u;
    }
    warp_sums[lane] = w;
  }
  __syncthreads();
  const N before = warp ? warp_sums[warp - 1] : 0;
  *total = warp_sums[31];
  __syncthreads();  // the sums are read before the next scan writes them
  return before + inc - v;
}

// Lists the pages of [begin, end) with refs == 0 (used = false) or > 0, in
// order, until `want` are found; returns how many were listed (all threads).
template <bool kUsed>
__device__ int kv_list_pages(const KvPages& c, int begin, int end, int want, int32_t* out) {
  int found = 0;
  for (int at = begin; at < end && found < want; at += kKvPlanThreads * kKvScanItems) {
    const int i0 = at + threadIdx.x * kKvScanItems;
    uint32_t hit = 0;
#pragma unroll
    for (int k = 0; k < kKvScanItems; ++k)
      if (i0 + k < end) hit |= (uint32_t)((__ldcg(c.refs + i0 + k) > 0) == kUsed) << k;
    int total;
    int r = found + kv_block_scan<int>(__popc(hit), &total);
    while (hit && r < want) {
      out[r++] = i0 + __ffs(hit) - 1;
      hit &= hit - 1;
    }
    found = min(want, found + total);
  }
  __syncthreads();  // the list is visible to the whole CTA
  return found;
}

// True for the first of this call's entries that names sequence s (s in range
// or -1).  owner is zero before and after; called by all threads of the CTA.
__device__ __forceinline__ bool kv_first_mention(const KvPages& c, int s) {
  const int mark = kKvMaxEntries - (int)threadIdx.x;  // the earliest entry has the largest
  if (s >= 0) atomicMax(c.owner() + s, mark);
  __syncthreads();
  const bool first = s >= 0 && __ldcg(c.owner() + s) == mark;
  __syncthreads();
  if (first) c.owner()[s] = 0;
  return first;
}

// A call's running sums of wanted pages take 41 bits (1024 entries of up to 2^31 - 1
// pages).  Whether the `found` free pages reach the entry that wants `need` of them
// behind `before` others:
__host__ __device__ __forceinline__ bool kv_reaches(long long before, int need, int found) { return before + need <= found; }
// and a running sum as a place in the list of pages, which ends long before 2^31 - 1.
__host__ __device__ __forceinline__ int kv_place(long long before) { return (int)(before < 0x7fffffffll ? before : 0x7fffffffll); }

// Hands out need pages to every entry (thread i: entry i), entries in order,
// lowest free page first: the list of pages is left in c.dst().  Returns this
// entry's first index into the list, or -1 if the free pages do not reach it;
// *used receives how many pages were handed out.  prefix [1025] holds the
// exclusive sums of need afterwards, those behind the list's end cut off at 2^31 - 1.
__device__ __forceinline__ int kv_hand_out(const KvPages& c, int need, int* prefix, int* used) {
  __shared__ int served;
  long long want;
  const long long before = kv_block_scan<long long>(need, &want);
  const int at = kv_place(before);
  prefix[threadIdx.x] = at;
  if (threadIdx.x == 0) {
    prefix[kKvPlanThreads] = kv_place(want);
    served = 0;
  }
  const int hint = max(0, min(c.num_pages, __ldcg(c.state + 1)));
  const int found = kv_list_pages<false>(c, hint, c.num_pages, kv_place(want), c.dst());
  const bool ok = kv_reaches(before, need, found);
  if (need > 0 && ok) atomicMax(&served, at + need);  // sums grow with the entry: a prefix of the entries is served
  if (need > 0 && !ok) c.flag(KV_NO_PAGES);
  __syncthreads();
  *used = served;
  for (int r = threadIdx.x; r < served; r += kKvPlanThreads) c.refs[c.dst()[r]] = 1;
  if (threadIdx.x == 0 && served > 0) c.state[1] = c.dst()[served - 1] + 1;
  return (need == 0 || ok) ? at : -1;
}

// The entry that owns list index r: the last one whose prefix is <= r.
__device__ __forceinline__ int kv_entry_of(const int* prefix, int n, int r) {
  int lo = 0, hi = n;  // prefix[lo] <= r < prefix[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (prefix[mid] <= r) lo = mid; else hi = mid;
  }
  return lo;
}

// --------------------------------------------------------------------------
// set: another set of tables, one launch over the GPU (bound by the launch: three
// copies and the state's zeroing as calls of their own took 8 us more)
// --------------------------------------------------------------------------
__global__ void __launch_bounds__(256) kv_set_kernel(const KvPages c, const int32_t* table, const int32_t* lens,
                                                      const int32_t* refs) {
  pdl_wait();
  pdl_trigger();
  const int64_t tid = (int64_t)blockIdx.x * blockDim.x + threadIdx.x, step = (int64_t)gridDim.x * blockDim.x;
  const int64_t entries = (int64_t)c.max_seqs * c.max_pages;
  for (int64_t e = tid; e < entries; e += step) c.table[e] = table[e];
  for (int64_t e = tid; e < c.num_pages; e += step) c.refs[e] = refs[e];
  for (int64_t e = tid; e < c.max_seqs; e += step) {
    c.lens[e] = lens[e];
    c.owner()[e] = 0;
  }
  if (tid < kKvHead) c.state[tid] = 0;
}

// --------------------------------------------------------------------------
// extend: one CTA
// --------------------------------------------------------------------------
__global__ void __launch_bounds__(kKvPlanThreads) kv_extend_kernel(const KvPages c, const int32_t* seqs,
                                                                    const int32_t* add, int n) {
  __shared__ int prefix[kKvPlanThreads + 1];
  __shared__ int seq_of[kKvPlanThreads], held_of[kKvPlanThreads];
  pdl_wait();
  pdl_trigger();
  const int i = threadIdx.x;
  int s = -1;
  if (i < n) {
    s = seqs ? seqs[i] : i;
    if (s < 0 || s >= c.max_seqs) {
      c.flag(KV_BAD_SEQ);
      s = -1;
    }
  }
  const bool first = kv_first_mention(c, s);
  if (s >= 0 && !first) c.flag(KV_BAD_SEQ);
  int len = 0, grown = -1, need = 0;
  if (first) {
    len = __ldcg(c.lens + s);
    const int64_t want = (int64_t)len + (add ? add[i] : 1);
    if (!c.valid_len(len) || want < len) {
      c.flag(KV_BAD_SEQ);
    } else if (want > (int64_t)c.max_pages * c.page_size) {
      c.flag(KV_FULL);
    } else {
      grown = (int)want;
      need = c.pages_of(grown) - c.pages_of(len);
    }
  }
  seq_of[i] = s;
  held_of[i] = c.pages_of(len);
  int used;
  const int at = kv_hand_out(c, need, prefix, &used);
  for (int r = i; r < used; r += kKvPlanThreads) {
    const int e = kv_entry_of(prefix, kKvPlanThreads, r);
    c.table[(size_t)seq_of[e] * c.max_pages + held_of[e] + (r - prefix[e])] = c.dst()[r];
  }
  if (grown >= 0 && at >= 0) c.lens[s] = grown;
}

// --------------------------------------------------------------------------
// fork: the plan (one CTA), then kv_move_kernel<true>
// --------------------------------------------------------------------------
// Entry i leaves in base[i] its first index into the list of handed-out pages,
// or -1 if it is skipped; pair r of the list is (src()[r], dst()[r], tok()[r]).
__global__ void __launch_bounds__(kKvPlanThreads) kv_fork_plan_kernel(const KvPages c, const int32_t* src,
                                                                       const int32_t* dst, int n, int share) {
  __shared__ int prefix[kKvPlanThreads + 1];
  __shared__ int src_of[kKvPlanThreads], len_of[kKvPlanThreads];
  pdl_wait();
  pdl_trigger();
  const int i = threadIdx.x;
  int s = -1, d = -1;
  if (i < n) {
    s = src[i];
    d = dst[i];
    if (s < 0 || s >= c.max_seqs || d < 0 || d >= c.max_seqs) {
      c.flag(KV_BAD_SEQ);
      s = d = -1;
    }
  }
  const bool first = kv_first_mention(c, d);
  if (d >= 0 && !first) c.flag(KV_BAD_SEQ);
  int len = -1, need = 0;
  if (first) {
    len = __ldcg(c.lens + s);
    if (__ldcg(c.lens + d) != 0 || !c.valid_len(len)) {
      c.flag(KV_BAD_SEQ);
      len = -1;
    } else {
      need = c.pages_of(len) - (share ? (int)c.page_div.div((uint32_t)len) : 0);
    }
  }
  src_of[i] = s;
  len_of[i] = len;
  int used;
  const int at = kv_hand_out(c, need, prefix, &used);  // its barriers: every length is read before one is written
  for (int r = i; r < used; r += kKvPlanThreads) {
    const int e = kv_entry_of(prefix, kKvPlanThreads, r);
    const int kept = share ? (int)c.page_div.div((uint32_t)len_of[e]) : 0;
    const int j = kept + (r - prefix[e]);
    int page = c.table[(size_t)src_of[e] * c.max_pages + j];
    if (page < 0 || page >= c.num_pages) {
      c.flag(KV_BAD_PAGE);
      page = -1;
    }
    c.src()[r] = page;
    c.tok()[r] = min(c.page_size, len_of[e] - j * c.page_size);
  }
  const bool taken = len >= 0 && at >= 0;
  if (i < n) c.base()[i] = taken ? at : -1;
  if (taken) c.lens[d] = len;
  if (i == 0) c.state[2] = used;
}

// --------------------------------------------------------------------------
// compact: the plan (one CTA), then kv_move_kernel<false>
// --------------------------------------------------------------------------
__global__ void __launch_bounds__(kKvPlanThreads) kv_compact_plan_kernel(const KvPages c, int32_t* live_out) {
  pdl_wait();
  pdl_trigger();
  int live = 0;
  for (int at = threadIdx.x * 4; at < c.num_pages; at += kKvPlanThreads * 4)
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (at + k < c.num_pages) live += __ldcg(c.refs + at + k) > 0;
  int total;
  kv_block_scan<int>(live, &total);
  live = total;
  // as many free pages below `live` as used ones at or above it
  const int moves = kv_list_pages<false>(c, 0, live, live, c.dst());
  kv_list_pages<true>(c, live, c.num_pages, moves, c.src());
  for (int r = threadIdx.x; r < moves; r += kKvPlanThreads) {
    const int from = c.src()[r], to = c.dst()[r];
    c.refs[to] = __ldcg(c.refs + from);
    c.refs[from] = 0;
    c.tok()[from] = to;  // where the table entries that name `from` go
  }
  if (threadIdx.x == 0) {
    c.state[1] = live;
    c.state[2] = moves;
    c.state[3] = live;
    if (live_out) *live_out = live;
  }
}

// --------------------------------------------------------------------------
// what moves: pages in every layer, and the table rows that follow
// --------------------------------------------------------------------------
// A page is copied in parts of kKvPartVecs 16-byte vectors, one CTA a part at
// a time with all of a thread's loads issued before its stores.  Bound by HBM:
// every byte is read once and written once.  Vectors of a page are taken in
// the order of its memory: whole pages are one run if the slots or the heads
// are dense, so consecutive threads touch consecutive vectors.
constexpr int kKvMoveThreads = 256;
constexpr int kKvPartUnroll = 8;
constexpr int kKvPartVecs = kKvMoveThreads * kKvPartUnroll;

struct KvMove {
  const int32_t* src;  // fork: sequences
  const int32_t* dst;
  int n, share;
  int parts;                     // parts of a full page
  FastDiv heads;                 // kv_heads
  int vec_shift;                 // log2(head_vecs)
  int head_major;                // heads outside the slots in memory
};

// Vector v of `tokens` tokens of a page -> its offset in the page.
__device__ __forceinline__ int64_t kv_vec_offset(const KvPages& c, const KvMove& m, uint32_t v, const FastDiv& tokens) {
  const uint32_t row = v >> m.vec_shift, x = v & ((1u << m.vec_shift) - 1u);
  uint32_t t, h;
  if (m.head_major) {
    h = tokens.div(row);
    t = row - h * tokens.d;
  } else {
    t = m.heads.div(row);
    h = row - t * m.heads.d;
  }
  return (int64_t)t * c.token_stride + (int64_t)h * c.head_stride + x;
}

template <bool kFork>
__global__ void __launch_bounds__(kKvMoveThreads) kv_move_kernel(const KvPages c, const KvMove m) {
  pdl_wait();
  pdl_trigger();
  const int64_t tid = (int64_t)blockIdx.x * blockDim.x + threadIdx.x, step = (int64_t)gridDim.x * blockDim.x;
  if (kFork) {
    // table rows: pages held by both, then the new ones
    const int64_t entries = (int64_t)m.n * c.max_pages;
    for (int64_t e = tid; e < entries; e += step) {
      const int i = (int)(e / c.max_pages), j = (int)(e - (int64_t)i * c.max_pages);
      const int base = c.base()[i];
      if (base < 0) continue;
      const int s = m.src[i], d = m.dst[i];
      const int len = c.lens[d];
      if (j >= c.pages_of(len)) continue;
      const int kept = m.share ? (int)c.page_div.div((uint32_t)len) : 0;
      int page;
      if (j < kept) {
        page = c.table[(size_t)s * c.max_pages + j];
        if (page >= 0 && page < c.num_pages) atomicAdd(c.refs + page, 1);
        else c.flag(KV_BAD_PAGE);
      } else {
        page = c.dst()[base + j - kept];
      }
      c.table[(size_t)d * c.max_pages + j] = page;
    }
  } else {
    const int live = c.state[3];
    const int64_t entries = (int64_t)c.max_seqs * c.max_pages;
    for (int64_t e = tid; e < entries; e += step) {
      const int page = c.table[e];
      // a used page at or above `live` was moved
      if (page >= live && page < c.num_pages) c.table[e] = c.tok()[page];
    }
  }
  // jobs: (pair, layer, part), K and V of each
  const int pairs = c.state[2];
  const int64_t jobs = (int64_t)pairs * c.n_layers * m.parts;
  const FastDiv full = FastDiv{(uint32_t)c.page_size, c.page_div.mul, c.page_div.shift};
  for (int64_t job = blockIdx.x; job < jobs; job += gridDim.x) {
    const int64_t pl = job / m.parts;
    const int part = (int)(job - pl * m.parts);
    const int r = (int)(pl / c.n_layers), layer = (int)(pl - (int64_t)r * c.n_layers);
    const int from = c.src()[r], to = c.dst()[r];
    const int tokens = kFork ? c.tok()[r] : c.page_size;
    if (from < 0) continue;  // a table entry that was no page: flagged by the plan
    const uint32_t vecs = ((uint32_t)tokens * m.heads.d) << m.vec_shift;
    const uint32_t v0 = (uint32_t)part * kKvPartVecs;
    if (v0 >= vecs) continue;
    const FastDiv td = (!kFork || tokens == c.page_size || !m.head_major) ? full : FastDiv::make(tokens);
    const int64_t a = layer * c.layer_stride + from * c.page_stride, b = layer * c.layer_stride + to * c.page_stride;
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      uint4* p = kv ? c.v : c.k;
      uint4 x[kKvPartUnroll];
      int64_t off[kKvPartUnroll];
#pragma unroll
      for (int u = 0; u < kKvPartUnroll; ++u) {
        const uint32_t v = v0 + u * kKvMoveThreads + threadIdx.x;
        off[u] = -1;
        if (v < vecs) {
          off[u] = kv_vec_offset(c, m, v, td);
          x[u] = __ldcs(p + a + off[u]);
        }
      }
#pragma unroll
      for (int u = 0; u < kKvPartUnroll; ++u)
        if (off[u] >= 0) __stcs(p + b + off[u], x[u]);
    }
  }
}

// --------------------------------------------------------------------------
// free: one CTA per sequence
// --------------------------------------------------------------------------
__global__ void __launch_bounds__(128) kv_free_kernel(const KvPages c, const int32_t* seqs) {
  __shared__ int len_sh;
  pdl_wait();
  pdl_trigger();
  const int s = seqs[blockIdx.x];
  if (s < 0 || s >= c.max_seqs) {
    if (threadIdx.x == 0) c.flag(KV_BAD_SEQ);
    return;
  }
  // of two entries that name one sequence, one finds it in use
  if (threadIdx.x == 0) len_sh = atomicExch(c.lens + s, 0);
  __syncthreads();
  const int held = min(c.max_pages, c.pages_of(len_sh));
  int lowest = 0x7fffffff;
  for (int j = threadIdx.x; j < held; j += blockDim.x) {
    int32_t* e = c.table + (size_t)s * c.max_pages + j;
    const int page = *e;
    *e = -1;
    if (page < 0 || page >= c.num_pages) {
      c.flag(KV_BAD_PAGE);
      continue;
    }
    const int was = atomicSub(c.refs + page, 1);
    if (was == 1) lowest = min(lowest, page);
    if (was < 1) {  // it was free already: leave it so
      atomicAdd(c.refs + page, 1);
      c.flag(KV_BAD_PAGE);
    }
  }
  if (lowest != 0x7fffffff) atomicMin(c.state + 1, lowest);
}

// --------------------------------------------------------------------------
// append: a warp per row and tensor
// --------------------------------------------------------------------------
struct KvAppend {
  const int32_t* seqs;
  const int32_t* rows;
  const uint4* k;
  const uint4* v;
  int64_t k_stride, v_stride, layer_off;  // 16-byte vectors
  int n, total_rows;
  int vec_shift;
};

__global__ void __launch_bounds__(256) kv_append_kernel(const KvPages c, const KvAppend a) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int64_t warps = ((int64_t)gridDim.x * blockDim.x) >> 5;
  const int row_vecs = c.kv_heads << a.vec_shift;
  const int last = a.rows ? min(a.total_rows, a.rows[a.n]) : min(a.total_rows, a.n);
  for (int64_t w = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5; w < 2 * (int64_t)last; w += warps) {
    const int row = (int)(w >> 1);
    // the entry: the last one that begins at or before this row
    int i = row, begin = row, end = row + 1;
    if (a.rows) {
      int lo = 0, hi = a.n;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a.rows[mid] <= row) lo = mid; else hi = mid;
      }
      i = lo;
      begin = a.rows[lo];
      end = a.rows[lo + 1];
      if (row < begin || row >= end) continue;  // before the first entry, or rows out of order
    }
    const int s = a.seqs ? a.seqs[i] : i;
    if (s < 0 || s >= c.max_seqs) {
      if (lane == 0) c.flag(KV_BAD_SEQ);
      continue;
    }
    if (a.seqs) {  // two entries of one sequence would write the same slots: the first one does
      bool named = false;
      for (int e = lane; e < i; e += 32) named |= a.seqs[e] == s;
      if (__any_sync(0xffffffffu, named)) {
        if (lane == 0) c.flag(KV_BAD_SEQ);
        continue;
      }
    }
    const int64_t p = (int64_t)c.lens[s] - (end - row);
    if (p < 0 || p >= (int64_t)c.max_pages * c.page_size) {
      if (lane == 0) c.flag(KV_FULL);
      continue;
    }
    const int j = (int)c.page_div.div((uint32_t)p), slot = (int)p - j * c.page_size;
    const int page = c.table[(size_t)s * c.max_pages + j];
    if (page < 0 || page >= c.num_pages) {
      if (lane == 0) c.flag(KV_BAD_PAGE);
      continue;
    }
    if (c.refs[page] > 1) {
      if (lane == 0) c.flag(KV_SHARED);
      continue;
    }
    const uint4* from = (w & 1) ? a.v + row * a.v_stride : a.k + row * a.k_stride;
    uint4* to = ((w & 1) ? c.v : c.k) + a.layer_off + page * c.page_stride + slot * c.token_stride;
    for (int x0 = 0; x0 < row_vecs; x0 += 32 * 8) {
      uint4 x[8];
#pragma unroll
      for (int u = 0; u < 8; ++u)
        if (x0 + u * 32 + lane < row_vecs) x[u] = __ldcs(from + x0 + u * 32 + lane);
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int v = x0 + u * 32 + lane;
        if (v < row_vecs) to[(v >> a.vec_shift) * c.head_stride + (v & ((1 << a.vec_shift) - 1))] = x[u];
      }
    }
  }
  // what no row shows: bounds out of order, or more rows than there are
  if (a.rows && blockIdx.x == 0)
    for (int i = threadIdx.x; i < a.n; i += blockDim.x)
      if (a.rows[i] < 0 || a.rows[i + 1] < a.rows[i] || a.rows[i + 1] > a.total_rows) c.flag(KV_FULL);
}

}  // namespace dinfer
