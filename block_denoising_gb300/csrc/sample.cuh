// A token per row of logits by temperature, top-k, top-p and min-p from a given
// number, and its confidence (include/dinfer_ops.h, dinfer_op_sample).
//
// A row is read once: a cluster of up to 8 CTAs keeps it in shared memory, a slice
// each, and everything after the load is passes over those slices, joined
// through distributed shared memory.
//
// Weights are whole numbers, w = round(2^44 e^((l - max) / T)), so that sums are the
// same in any order and comparisons with u and top_p are exact.  Which token is
// drawn hangs on where u falls among up to 157000 sums of rounded weights: with
// fp32 exponentials one row in some ten thousand gets another token than the
// definition's, so the exponent is carried in two floats and the power of two
// comes from a table of 512 and a cubic, about 2^-32 of the weight in all.
//
// top-k and top-p cut the order (larger logit first, then lower index) at one
// place, found by histograms of 1024 bins: first over the exponent, then over the
// pair (logit, index) within the bin that holds the cut, until one element is left.
// Rows without them take one pass.
#pragma once
#include <cooperative_groups.h>

#include "common.cuh"

namespace dinfer {

constexpr int kSmThreads = 512;
constexpr int kSmWarps = kSmThreads / 32;
constexpr int kSmCluster = 8;     // CTAs of a row at most
constexpr int kSmBins = 1024;
constexpr int kSmIndexBits = 19;  // of a token's index
constexpr float kSmRange = 46.f;  // weights vanish below 2^-44

struct SmArgs {
  const void* x;
  int64_t stride;  // elements
  int rows, vocab, slice;  // slice: tokens of a CTA
  const float* temperature;
  const int32_t* top_k;
  const float* top_p;
  const float* min_p;
  const float* u;
  int32_t* tok;
  float* conf;
  uint64_t coarse[16], fine[32];  // 2^(j / 16), 2^(j / 512) in 2^-63rds
};

// Where the cut lies: elements [lo, hi] of the order hold it, `count` and `mass` lie before them.
struct SmRange {
  uint64_t lo, hi, mass;
  uint32_t count;
  int state;  // 0: go on, 1: found (hi is the last kept), 2: everything is kept
};

struct SmShared {
  uint32_t table[512];
  uint32_t count[kSmBins], all_count[kSmBins];  // all_: the row's, in the first CTA
  uint64_t mass[kSmBins], all_mass[kSmBins];
  uint64_t warp_sum[kSmWarps], cta_sum[kSmCluster];
  float warp_f[kSmWarps], max_of[kSmCluster], sum_of[kSmCluster];
  uint32_t warp_i[kSmWarps], first_of[kSmCluster];
  uint64_t lo_of[kSmCluster], hi_of[kSmCluster];
  SmRange range;
  int bin;
};

struct SmScale {
  float m, mh, ml, ch, cl;
};
// A logit as a multiple of 2^-10 and the rest: differences of the first parts are exact.
__device__ __forceinline__ float sm_high(float x) { return (x + 12288.f) - 12288.f; }

__device__ __forceinline__ uint64_t sm_weight(float l, const SmScale& k, const uint32_t* table) {
  const float lh = sm_high(l), dh = lh - k.mh, dl = (l - lh) - k.ml;
  const float p = __fmul_rn(dh, k.ch);  // not to be contracted with the sums below, which take its rounding off again
  float s = fmaf(dl, k.ch, fmaf(dh, k.cl, fmaf(dh, k.ch, -p)));
  constexpr float kMagic = 24576.f;  // 1.5 * 2^14: a float's last place is 1 / 512
  const float t = fmaf(dl, k.ch, p) + kMagic;
  s += p - (t - kMagic);
  const float q = s * fmaf(s, fmaf(s, 0.0555041086648f, 0.240226506959f), 0.693147180560f);  // 2^s - 1
  const int n = __float_as_int(t) - __float_as_int(kMagic);
  const uint32_t hi = table[n & 511];  // 2^30 and more
  const int64_t w = ((int64_t)hi << 14) + ((int64_t)__mulhi((int)hi, __float2int_rn(q * 0x1p41f)) << 5);
  // rounded, not cut off: half a unit of each of 10^5 small weights would be more than all other errors
  const uint64_t r = (((uint64_t)w << 1 >> min(63, -(n >> 9))) + 1) >> 1;
  return l == k.m ? 1ull << 44 : p >= -44.f ? r : 0;  // NaN: 0
}

// Larger logits first, then lower indexes.
__device__ __forceinline__ uint64_t sm_order(float l, int index) {
  const uint32_t b = __float_as_uint(l + 0.f);  // -0 is 0
  const uint32_t up = b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
  return ((uint64_t)~up << kSmIndexBits) | (uint32_t)index;
}

template <typename V, typename Op>
__device__ __forceinline__ V sm_reduce(V v, Op op) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = op(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// floor(a b 2^-64), and rounded up
__device__ __forceinline__ uint64_t sm_part(uint64_t a, uint64_t b) { return __umul64hi(a, b); }
__device__ __forceinline__ uint64_t sm_part_up(uint64_t a, uint64_t b) { return __umul64hi(a, b) + (a * b != 0); }
// a number below 1 in 2^-64ths (NaN, below 0: 0)
__device__ __forceinline__ uint64_t sm_fraction(float x) {
  return !(x > 0.f) ? 0ull : x >= 1.f ? ~0ull : (uint64_t)((double)x * 18446744073709551616.0);
}

template <typename T>
__global__ void __launch_bounds__(kSmThreads) sample_kernel(const __grid_constant__ SmArgs a) {
  namespace cg = cooperative_groups;
  extern __shared__ __align__(16) uint8_t sm_raw[];
  SmShared& sh = *reinterpret_cast<SmShared*>(sm_raw);
  cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = blockIdx.z, ctas = gridDim.z, row = blockIdx.x;
  if (tid < 512) sh.table[tid] = (uint32_t)(__umul64hi(a.coarse[tid >> 5], a.fine[tid & 31]) >> 32);
  cluster.barrier_arrive();  // waited for before the first access to another CTA's memory
  pdl_wait();
  pdl_trigger();

  // the slice, as it lies behind a boundary of 16 bytes
  const int begin = rank * a.slice, n = max(0, min(a.slice, a.vocab - begin));
  const T* from = reinterpret_cast<const T*>(a.x) + (int64_t)row * a.stride + begin;
  const int shift = (int)(reinterpret_cast<uintptr_t>(from) & 15);
  uint8_t* raw = sm_raw + (sizeof(SmShared) + 15) / 16 * 16;
  const T* x = reinterpret_cast<const T*>(raw + shift);
  {
    constexpr int kPer = 16 / (int)sizeof(T);
    const int head = min(n, shift ? (16 - shift) / (int)sizeof(T) : 0), vecs = (n - head) / kPer, tail = head + vecs * kPer;
    T* to = reinterpret_cast<T*>(raw + shift);
    for (int i = tid; i < vecs; i += kSmThreads) {
      const T* src = from + head + i * kPer;
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(to + head + i * kPer)), "l"(src) : "memory");
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    if (tid < head) to[tid] = from[tid];
    if (tail + tid < n) to[tail + tid] = from[tail + tid];  // fewer than kPer
    asm volatile("cp.async.wait_group 0;" ::: "memory");
  }
  __syncthreads();

  // each warp has a stretch of the slice, walked in order
  const int per = (n + kSmThreads - 1) / kSmThreads * 32, s0 = min(n, warp * per), s1 = min(n, s0 + per);
  auto each = [&](auto f) {
#pragma unroll 4
    for (int i = s0 + lane; i < s1; i += 32) f(begin + i, (float)x[i]);
  };

  float top = -INFINITY;
  each([&](int, float l) { top = fmaxf(top, l); });
  top = sm_reduce(top, [](float p, float q) { return fmaxf(p, q); });
  if (lane == 0) sh.warp_f[warp] = top;
  __syncthreads();
  cluster.barrier_wait();
  if (tid < ctas) {
    for (int w = 0; w < kSmWarps; ++w) top = fmaxf(w ? top : -INFINITY, sh.warp_f[w]);
    cluster.map_shared_rank(sh.max_of, tid)[rank] = top;
  }
  cluster.sync();
  top = sh.max_of[0];
  for (int r = 1; r < ctas; ++r) top = fmaxf(top, sh.max_of[r]);
  if (top == -INFINITY) {  // nothing to draw
    if (rank == 0 && tid == 0) {
      a.tok[row] = -1;
      if (a.conf) a.conf[row] = 0.f;
    }
    return;
  }

  // the softmax's sum at temperature 1
  if (a.conf) {
    float sum = 0.f;
    each([&](int, float l) { sum += l == top ? 1.f : l > -INFINITY ? exp2f((l - top) * 1.4426950408889634f) : 0.f; });
    sum = sm_reduce(sum, [](float p, float q) { return p + q; });
    __syncthreads();  // the maxima are read
    if (lane == 0) sh.warp_f[warp] = sum;
    __syncthreads();
    if (tid < ctas) {
      sum = 0.f;
      for (int w = 0; w < kSmWarps; ++w) sum += sh.warp_f[w];
      cluster.map_shared_rank(sh.sum_of, tid)[rank] = sum;
    }
  }
  // behind the next cluster barrier
  auto put = [&](int token, float l) {
    a.tok[row] = token;
    if (!a.conf) return;
    float sum = 0.f;
    for (int r = 0; r < ctas; ++r) sum += sh.sum_of[r];
    a.conf[row] = (l == top ? 1.f : (float)exp((double)l - (double)top)) / sum;
  };

  const float temperature = a.temperature ? a.temperature[row] : 1.f;
  const int top_k = a.top_k ? a.top_k[row] : 0;
  if (!(temperature > 0.f) || top_k == 1) {  // the first largest
    uint32_t first = 0xffffffffu;
    each([&](int i, float l) { if (l == top) first = min(first, (uint32_t)i); });
    first = __reduce_min_sync(0xffffffffu, first);
    if (lane == 0) sh.warp_i[warp] = first;
    __syncthreads();
    if (tid < ctas) {
      for (int w = 0; w < kSmWarps; ++w) first = min(w ? first : 0xffffffffu, sh.warp_i[w]);
      cluster.map_shared_rank(sh.first_of, tid)[rank] = first;
    }
    cluster.sync();
    if (rank == 0 && tid == 0) {
      first = sh.first_of[0];
      for (int r = 1; r < ctas; ++r) first = min(first, sh.first_of[r]);
      put((int)first, top);
    }
    return;
  }

  SmScale scale;
  {
    const double c = fmin(1.4426950408889634074 / (double)temperature, 0x1p100);
    scale.m = top;
    scale.mh = sm_high(top);
    scale.ml = top - scale.mh;
    scale.ch = (float)c;
    scale.cl = (float)(c - (double)scale.ch);
  }
  auto weight = [&](float l) { return sm_weight(l, scale, sh.table); };

  uint64_t cut = ~0ull;  // the last kept place of the order
  // The place where the elements kept so far reach `top_k` of them, or the part `top_p` of their weight.
  auto search = [&](auto by_mass, uint32_t want_count, uint64_t want_part) {
    constexpr bool kMass = decltype(by_mass)::value;
    uint64_t want = want_count;  // the first CTA's: what is to be reached
    SmRange at{0, 0, 0, 0, 0};
    for (int level = 0;; ++level) {
      for (int b = tid; b < kSmBins; b += kSmThreads) {
        sh.count[b] = 0;
        if (kMass) sh.mass[b] = 0;
        if (level == 0 && rank == 0) {
          sh.all_count[b] = 0;
          if (kMass) sh.all_mass[b] = 0;
        }
      }
      if (level == 0) cluster.sync(); else __syncthreads();
      const int bits = level ? max(0, 54 - __clzll((long long)(at.hi - at.lo))) : 0;  // (hi - lo) >> bits < 1024
      each([&](int i, float l) {
        if (!(l > -INFINITY)) return;
        int b;
        if (level == 0) {
          if (cut != ~0ull && sm_order(l, i) > cut) return;
          b = l == top ? 0 : (int)fminf((float)(kSmBins - 1), (top - l) * scale.ch * ((kSmBins - 1) / kSmRange));
        } else {
          const uint64_t c = sm_order(l, i);
          if (c < at.lo || c > at.hi) return;
          b = (int)((c - at.lo) >> bits);
        }
        atomicAdd(&sh.count[b], 1u);
        if (kMass) atomicAdd(reinterpret_cast<unsigned long long*>(&sh.mass[b]), (unsigned long long)weight(l));
      });
      __syncthreads();
      uint32_t* all_count = cluster.map_shared_rank(sh.all_count, 0);
      uint64_t* all_mass = cluster.map_shared_rank(sh.all_mass, 0);
      for (int b = tid; b < kSmBins; b += kSmThreads)
        if (sh.count[b]) {
          atomicAdd(all_count + b, sh.count[b]);
          if (kMass) atomicAdd(reinterpret_cast<unsigned long long*>(all_mass + b), (unsigned long long)sh.mass[b]);
        }
      cluster.sync();
      if (rank == 0) {  // the bin in which `want` is reached: two bins a thread
        constexpr int kPer = kSmBins / kSmThreads;
        uint64_t v[kPer], own = 0, before;
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
          v[e] = kMass ? sh.all_mass[tid * kPer + e] : sh.all_count[tid * kPer + e];
          own += v[e];
        }
        uint64_t inc = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint64_t y = __shfl_up_sync(0xffffffffu, inc, o);
          if (lane >= o) inc += y;
        }
        if (lane == 31) sh.warp_sum[warp] = inc;
        if (tid == 0) sh.bin = -1;
        __syncthreads();
        uint64_t total = 0;
        before = inc - own;
        for (int w = 0; w < kSmWarps; ++w) {
          if (w < warp) before += sh.warp_sum[w];
          total += sh.warp_sum[w];
        }
        if (kMass && level == 0) want = max((uint64_t)1, sm_part_up(want_part, total));
        const uint64_t base = level == 0 ? 0 : kMass ? at.mass : at.count;
        before += base;
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
          if (before < want && want <= before + v[e]) {
            const int b = tid * kPer + e;
            SmRange r;
            r.mass = kMass ? before : 0;
            r.count = kMass ? 0 : (uint32_t)before;
            r.lo = at.lo + ((uint64_t)b << bits);
            r.hi = min(at.hi, r.lo + (((uint64_t)1 << bits) - 1));
            r.state = level > 0 && (bits == 0 || sh.all_count[b] == 1) ? 1 : 0;
            if (level == 0 && b == kSmBins - 1) r.state = 2;  // only weights of 0 lie there
            sh.range = r;
            sh.bin = b;
          }
          before += v[e];
        }
        __syncthreads();
        if (tid == 0 && sh.bin < 0) sh.range.state = 2;
        for (int b = tid; b < kSmBins; b += kSmThreads) {
          sh.all_count[b] = 0;
          if (kMass) sh.all_mass[b] = 0;
        }
        __syncthreads();
        if (tid > 0 && tid < ctas) {
          *cluster.map_shared_rank(&sh.range, tid) = sh.range;
          *cluster.map_shared_rank(&sh.bin, tid) = sh.bin;
        }
      }
      cluster.sync();
      at = sh.range;
      if (at.state == 2) return;
      if (level == 0) {  // the first and last place of the bin's elements
        const int bin = sh.bin;
        uint64_t lo = ~0ull, hi = 0;
        each([&](int i, float l) {
          if (!(l > -INFINITY)) return;
          const int b = l == top ? 0 : (int)fminf((float)(kSmBins - 1), (top - l) * scale.ch * ((kSmBins - 1) / kSmRange));
          const uint64_t c = sm_order(l, i);
          if (b != bin || c > cut) return;
          lo = min(lo, c);
          hi = max(hi, c);
        });
        lo = sm_reduce(lo, [](uint64_t p, uint64_t q) { return min(p, q); });
        hi = sm_reduce(hi, [](uint64_t p, uint64_t q) { return max(p, q); });
        if (lane == 0) {
          sh.warp_sum[warp] = lo;
          sh.mass[warp] = hi;
        }
        __syncthreads();
        if (tid < ctas) {
          for (int w = 0; w < kSmWarps; ++w) {
            lo = min(lo, sh.warp_sum[w]);
            hi = max(hi, sh.mass[w]);
          }
          cluster.map_shared_rank(sh.lo_of, tid)[rank] = lo;
          cluster.map_shared_rank(sh.hi_of, tid)[rank] = hi;
        }
        cluster.sync();
        at.lo = sh.lo_of[0];
        at.hi = sh.hi_of[0];
        for (int r = 1; r < ctas; ++r) {
          at.lo = min(at.lo, sh.lo_of[r]);
          at.hi = max(at.hi, sh.hi_of[r]);
        }
        if (at.lo == at.hi) at.state = 1;
      }
      if (at.state == 1) {
        cut = at.hi;
        return;
      }
      __syncthreads();
    }
  };
  if (top_k > 0 && top_k < a.vocab) search(std::false_type{}, (uint32_t)top_k, 0);
  const float top_p = a.top_p ? a.top_p[row] : 1.f;
  if (top_p < 1.f) search(std::true_type{}, 0, sm_fraction(top_p));

  // the kept weights in index order
  const float min_p = a.min_p ? a.min_p[row] : 0.f;
  const uint64_t least = min_p > 0.f ? (uint64_t)ceil(fmin((double)min_p, 1.0) * 0x1p44) : 0;
  auto kept = [&](int i, float l) -> uint64_t {
    if (cut != ~0ull && (!(l > -INFINITY) || sm_order(l, i) > cut)) return 0;
    const uint64_t w = weight(l);
    return w >= least ? w : 0;
  };
  uint64_t sum = 0;
  each([&](int i, float l) { sum += kept(i, l); });
  sum = sm_reduce(sum, [](uint64_t p, uint64_t q) { return p + q; });
  __syncthreads();
  if (lane == 0) sh.warp_sum[warp] = sum;
  __syncthreads();
  if (tid < ctas) {
    sum = 0;
    for (int w = 0; w < kSmWarps; ++w) sum += sh.warp_sum[w];
    cluster.map_shared_rank(sh.cta_sum, tid)[rank] = sum;
  }
  cluster.sync();
  uint64_t total = 0, before = 0;
  for (int r = 0; r < ctas; ++r) {
    if (r == rank) before = total;
    total += sh.cta_sum[r];
  }
  const uint64_t target = sm_part(sm_fraction(a.u[row]), total);  // the first sum above it
  for (int w = 0; w < warp; ++w) before += sh.warp_sum[w];
  if (target < before || target >= before + sh.warp_sum[warp]) return;
  for (int i0 = s0;; i0 += 32) {  // this warp's
    const int i = i0 + lane;
    const float l = i < s1 ? (float)x[i] : -INFINITY;
    const uint64_t w = i < s1 ? kept(begin + i, l) : 0;
    uint64_t inc = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint64_t y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += y;
    }
    const uint32_t over = __ballot_sync(0xffffffffu, before + inc > target);
    if (over) {
      if (lane == __ffs(over) - 1) put(begin + i, l);
      return;
    }
    before += __shfl_sync(0xffffffffu, inc, 31);
    if (i0 + 32 >= s1) return;  // not reached: the stretch holds the sum
  }
}

}  // namespace dinfer
