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
// place.  A floor under it is found first: for top-k the k-th largest of the
// threads' own maxima, which k logits reach; for top-p from the weights of an eighth
// of the row, checked by the exact sums.  What lies above it (some hundred logits
// mostly) goes to the first CTA, which finds the place by histograms of 1024
// bins over (logit, index), each over the bin of the last one that holds it, until
// one element is left.  Where more than kSmList lie above it, all CTAs do the same on
// their slices.  (Histograms of the whole row, one atomic a logit: 512 rows of
// 126464, of which some 400 with top-k or top-p: 650 us.)  Rows without either take
// one pass.
#pragma once
#include <cooperative_groups.h>

#include "attention_tc.cuh"

namespace dinfer {

constexpr int kSmThreads = 512;
constexpr int kSmWarps = kSmThreads / 32;
constexpr int kSmCluster = 8;     // CTAs of a row at most
constexpr int kSmBins = 1024;
constexpr int kSmList = 1536;     // logits that the first CTA takes alone
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

// Where the cut lies: elements [lo, hi] of the order hold it, `before` (of their number or weight) lie before them.
struct SmRange {
  uint64_t lo, hi, before;
  int state;  // 0: go on, 1: found (hi is the last kept), 2: everything is kept
};

struct SmShared {
  uint32_t table[512];
  uint64_t all_mass[kSmBins];  // the row's, in the first CTA
  uint32_t all_count[kSmBins];
  union {
    struct {
      uint64_t mass[kSmBins];
      uint32_t count[kSmBins];
    };
    struct {  // in the first CTA, when all have told their counts
      float list[kSmList];  // the logits above the floor in index order,
      uint32_t index[kSmList];  // and their tokens
    };
  };
  uint64_t warp_sum[kSmWarps], warp_above[kSmWarps], cta_sum[kSmCluster], cta_above[kSmCluster];
  float warp_f[kSmWarps], max_of[kSmCluster], sum_of[kSmCluster];
  uint32_t warp_i[kSmWarps], cta_i[kSmCluster];
  SmRange range;
  float floor;
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

// A slice's logits in shared memory, 16 bytes at a time: pads and NaN read as -inf.
template <typename T>
struct SmVec;
template <>
struct SmVec<float> {
  static constexpr int kN = 4;
  static __device__ __forceinline__ void get(const uint4& d, float (&l)[4]) {
    l[0] = fmaxf(__uint_as_float(d.x), -INFINITY);
    l[1] = fmaxf(__uint_as_float(d.y), -INFINITY);
    l[2] = fmaxf(__uint_as_float(d.z), -INFINITY);
    l[3] = fmaxf(__uint_as_float(d.w), -INFINITY);
  }
};
template <>
struct SmVec<__nv_bfloat16> {
  static constexpr int kN = 8;
  static __device__ __forceinline__ void get(const uint4& d, float (&l)[8]) {
    const uint32_t w[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      l[2 * i] = fmaxf(__uint_as_float(w[i] << 16), -INFINITY);
      l[2 * i + 1] = fmaxf(__uint_as_float(w[i] & 0xffff0000u), -INFINITY);
    }
  }
};

template <typename T>
__global__ void __launch_bounds__(kSmThreads) sample_kernel(const __grid_constant__ SmArgs a) {
  namespace cg = cooperative_groups;
  constexpr int kN = SmVec<T>::kN;
  extern __shared__ __align__(16) uint8_t sm_raw[];
  SmShared& sh = *reinterpret_cast<SmShared*>(sm_raw);
  cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = blockIdx.z, ctas = gridDim.z, row = blockIdx.x;
  sh.table[tid] = (uint32_t)(__umul64hi(a.coarse[tid >> 5], a.fine[tid & 31]) >> 32);
  for (int b = tid; b < kSmBins; b += kSmThreads) {
    sh.count[b] = sh.all_count[b] = 0;
    sh.mass[b] = sh.all_mass[b] = 0;
  }
  cluster.barrier_arrive();  // waited for before the first access to another CTA's memory
  pdl_wait();
  pdl_trigger();

  // the slice, as it lies behind a boundary of 16 bytes, with -inf around it
  const int begin = rank * a.slice, n = max(0, min(a.slice, a.vocab - begin));
  const T* from = reinterpret_cast<const T*>(a.x) + (int64_t)row * a.stride + begin;
  const int off = (int)(reinterpret_cast<uintptr_t>(from) & 15) / (int)sizeof(T);
  uint8_t* raw = sm_raw + (sizeof(SmShared) + 15) / 16 * 16;
  T* x = reinterpret_cast<T*>(raw);  // token begin + i lies at x[off + i]
  const int vecs = (off + n + kN - 1) / kN;
  {
    for (int i = tid; i < vecs; i += kSmThreads)
      if (i * kN >= off && (i + 1) * kN <= off + n)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(x + i * kN)), "l"(from - off + i * kN) : "memory");
    asm volatile("cp.async.commit_group;" ::: "memory");
    if (tid < 2 * kN && vecs > 0) {  // the first and the last vector where they are not whole
      const int i = tid < kN ? tid : (vecs - 1) * kN + tid - kN, v = i / kN * kN;
      if (v < off || v + kN > off + n) x[i] = i >= off && i < off + n ? from[i - off] : (T)-INFINITY;
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
  }
  __syncthreads();

  // each warp has a stretch of the slice; each(f) hands over the logits and the first one's token, a vector at a time
  const int per = (vecs + kSmThreads - 1) / kSmThreads * 32, v0 = min(vecs, warp * per), v1 = min(vecs, v0 + per);
  auto each = [&](auto f) {
#pragma unroll 2
    for (int i = v0 + lane; i < v1; i += 32) {
      float l[kN];
      SmVec<T>::get(reinterpret_cast<const uint4*>(raw)[i], l);
      f(begin - off + i * kN, l);
    }
  };
  // v of every CTA to every CTA's to[rank]; behind the next cluster barrier
  auto tell = [&](auto* to, auto v) { *(cluster.map_shared_rank(to, tid) + rank) = v; };

  float mine = -INFINITY;  // the thread's largest
  each([&](int, const float (&l)[kN]) {
#pragma unroll
    for (int e = 0; e < kN; ++e) mine = fmaxf(mine, l[e]);
  });
  {
    const float m = sm_reduce(mine, [](float p, float q) { return fmaxf(p, q); });
    if (lane == 0) sh.warp_f[warp] = m;
  }
  __syncthreads();
  cluster.barrier_wait();
  if (tid < ctas) {
    float m = sh.warp_f[0];
    for (int w = 1; w < kSmWarps; ++w) m = fmaxf(m, sh.warp_f[w]);
    tell(sh.max_of, m);
  }
  cluster.sync();
  float top = sh.max_of[0];
  for (int r = 1; r < ctas; ++r) top = fmaxf(top, sh.max_of[r]);
  if (top == -INFINITY) {  // nothing to draw
    if (rank == 0 && tid == 0) {
      a.tok[row] = -1;
      if (a.conf) a.conf[row] = 0.f;
    }
    return;
  }

  const float temperature = a.temperature ? a.temperature[row] : 1.f, top_p = a.top_p ? a.top_p[row] : 1.f;
  const float min_p = a.min_p ? a.min_p[row] : 0.f;
  const int top_k = a.top_k ? a.top_k[row] : 0;
  const bool greedy = !(temperature > 0.f) || top_k == 1, by_k = !greedy && top_k > 0 && top_k < a.vocab, by_p = !greedy && top_p < 1.f;
  SmScale scale;
  {
    const double c = fmin(1.4426950408889634074 / (double)temperature, 0x1p100);
    scale.m = top;
    scale.mh = sm_high(top);
    scale.ml = top - scale.mh;
    scale.ch = (float)c;
    scale.cl = (float)(c - (double)scale.ch);
  }
  const float bin_scale = scale.ch * ((kSmBins - 1) / kSmRange);
  auto bin_of = [&](float l) { return l == top ? 0 : (int)fminf((float)(kSmBins - 1), (top - l) * bin_scale); };

  // The floor: a histogram over the exponent of the threads' maxima, or of weights: of the maxima, which hold what few
  // tokens have much of, and eight times those of every eighth vector.
  if (by_k) {
    if (mine > -INFINITY) atomicAdd(&sh.count[bin_of(mine)], 1u);
  } else if (by_p) {
    auto add = [&](float l, float scaled) {
      const float w = (l == top ? 1.f : ex2_approx((l - top) * scale.ch)) * scaled;
      if (w >= 1.f) atomicAdd(reinterpret_cast<unsigned long long*>(&sh.mass[bin_of(l)]), (unsigned long long)w);
    };
    add(mine, 0x1p32f);
    int k = 0;
    for (int i = v0 + lane; i < v1; i += 32, ++k) {
      if (k & 7) continue;
      float l[kN];
      SmVec<T>::get(reinterpret_cast<const uint4*>(raw)[i], l);
#pragma unroll
      for (int e = 0; e < kN; ++e)
        if (l[e] != mine) add(l[e], 0x1p35f);
    }
  }
  // the softmax's sum at temperature 1
  if (a.conf) {
    float sum = 0.f;
    each([&](int, const float (&l)[kN]) {
#pragma unroll
      for (int e = 0; e < kN; ++e) sum += top == INFINITY ? (l[e] == top ? 1.f : 0.f) : ex2_approx((l[e] - top) * 1.4426950408889634f);
    });
    sum = sm_reduce(sum, [](float p, float q) { return p + q; });
    __syncthreads();  // the maxima are read
    if (lane == 0) sh.warp_f[warp] = sum;
    __syncthreads();
    if (tid < ctas) {
      sum = 0.f;
      for (int w = 0; w < kSmWarps; ++w) sum += sh.warp_f[w];
      tell(sh.sum_of, sum);
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

  if (greedy) {  // the first largest
    uint32_t first = 0xffffffffu;
    each([&](int i, const float (&l)[kN]) {
#pragma unroll
      for (int e = 0; e < kN; ++e)
        if (l[e] == top) first = min(first, (uint32_t)(i + e));
    });
    first = __reduce_min_sync(0xffffffffu, first);
    if (lane == 0) sh.warp_i[warp] = first;
    __syncthreads();
    if (tid < ctas) {
      first = sh.warp_i[0];
      for (int w = 1; w < kSmWarps; ++w) first = min(first, sh.warp_i[w]);
      tell(sh.cta_i, first);
    }
    cluster.sync();
    if (rank == 0 && tid == 0) {
      first = sh.cta_i[0];
      for (int r = 1; r < ctas; ++r) first = min(first, sh.cta_i[r]);
      put((int)first, top);
    }
    return;
  }
  auto weight = [&](float l) { return sm_weight(l, scale, sh.table); };
  const uint64_t least = min_p > 0.f ? (uint64_t)ceil(fmin((double)min_p, 1.0) * 0x1p44) : 0;

  // The first CTA's threads: the bin at which the histogram's sum, on top of `before`, reaches `want`, into sh.bin (-1:
  // none), and its sum before the bin; two bins a thread.
  auto find_bin = [&](bool by_mass, uint64_t before, uint64_t want, uint64_t* at) {
    uint64_t v[2], own = 0;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      v[e] = by_mass ? sh.all_mass[tid * 2 + e] : sh.all_count[tid * 2 + e];
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
    uint64_t total = before;
    before += inc - own;
    for (int w = 0; w < kSmWarps; ++w) {
      if (w < warp) before += sh.warp_sum[w];
      total += sh.warp_sum[w];
    }
    if (want == 0) want = max((uint64_t)1, sm_part(at[0], total));  // a part of the whole
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      if (before < want && want <= before + v[e]) {
        sh.bin = tid * 2 + e;
        sh.range.before = before;
      }
      before += v[e];
    }
    __syncthreads();
  };

  // ------------------------------ rows without a cut ------------------------------
  float floor = -INFINITY;  // only logits from it on count
  uint64_t cut = ~0ull;     // the last kept place of the order
  int list = -1;            // the first CTA's: how many logits it has in its list
  uint64_t sum = 0;
  if (!by_k && !by_p) {
    if (least) floor = top + temperature * logf(fminf(min_p, 1.f)) * 1.0001f - 1e-6f * fabsf(top);
    if (!(floor <= top)) floor = -INFINITY;
  } else {
    // ------------------------------ the floor ------------------------------
    __syncthreads();
    for (int b = tid; b < kSmBins; b += kSmThreads) {
      if (by_k && sh.count[b]) atomicAdd(cluster.map_shared_rank(sh.all_count, 0) + b, sh.count[b]);
      if (!by_k && sh.mass[b]) atomicAdd(reinterpret_cast<unsigned long long*>(cluster.map_shared_rank(sh.all_mass, 0) + b), (unsigned long long)sh.mass[b]);
    }
    cluster.sync();
    if (rank == 0) {
      uint64_t part = sm_fraction(top_p + 0.25f * (1.f - top_p));
      find_bin(!by_k, 0, by_k ? (uint64_t)top_k : 0, &part);
      // no bin: fewer maxima than top_k; weights that are all below 2^-32
      const float depth = sh.bin >= 0 ? sh.bin + 1.1f : by_k ? INFINITY : 32.f * ((kSmBins - 1) / kSmRange);
      if (tid < ctas) *cluster.map_shared_rank(&sh.floor, tid) = sh.bin == kSmBins - 1 ? -INFINITY : top - depth / bin_scale;
      for (int b = tid; b < kSmBins; b += kSmThreads) {
        sh.all_count[b] = 0;
        sh.all_mass[b] = 0;
      }
    }
    cluster.sync();
    floor = sh.floor;
    if (!(floor > -INFINITY)) floor = -3.402823466e38f;  // every logit that is there
    // how many lie above it, and for top-p all weights and theirs
    uint32_t count = 0;
    uint64_t above = 0;
    each([&](int, const float (&l)[kN]) {
#pragma unroll
      for (int e = 0; e < kN; ++e) {
        count += l[e] >= floor;
        if (!by_k) {
          const uint64_t w = weight(l[e]);
          sum += w;
          above += l[e] >= floor ? w : 0;
        }
      }
    });
    count = __reduce_add_sync(0xffffffffu, count);
    sum = sm_reduce(sum, [](uint64_t p, uint64_t q) { return p + q; });
    above = sm_reduce(above, [](uint64_t p, uint64_t q) { return p + q; });
    if (lane == 0) {
      sh.warp_i[warp] = count;
      sh.warp_sum[warp] = sum;
      sh.warp_above[warp] = above;
    }
    __syncthreads();
    if (tid < ctas) {
      count = 0;
      sum = above = 0;
      for (int w = 0; w < kSmWarps; ++w) {
        count += sh.warp_i[w];
        sum += sh.warp_sum[w];
        above += sh.warp_above[w];
      }
      tell(sh.cta_i, count);
      tell(sh.cta_sum, sum);
      tell(sh.cta_above, above);
    }
    cluster.sync();
    uint32_t all = 0, before = 0;
    uint64_t total = 0;
    above = 0;
    for (int r = 0; r < ctas; ++r) {
      if (r == rank) before = all;
      all += sh.cta_i[r];
      total += sh.cta_sum[r];
      above += sh.cta_above[r];
    }
    uint64_t want = by_k ? (uint64_t)top_k : max((uint64_t)1, sm_part_up(sm_fraction(top_p), total));
    if (by_k ? all < (uint32_t)top_k : above < want) {  // the floor lies too high (no cut, or a logit's last place)
      floor = -3.402823466e38f;
      all = kSmList + 1;
    }
    if (all <= kSmList) {
      // ------------------------------ the list ------------------------------
      float* to = cluster.map_shared_rank(sh.list, 0);
      uint32_t* index = cluster.map_shared_rank(sh.index, 0);
      for (int w = 0; w < warp; ++w) before += sh.warp_i[w];
      for (int i0 = v0; i0 < v1; i0 += 32) {
        const int i = i0 + lane;
        float l[kN];
#pragma unroll
        for (int e = 0; e < kN; ++e) l[e] = -INFINITY;
        if (i < v1) SmVec<T>::get(reinterpret_cast<const uint4*>(raw)[i], l);
        uint32_t hit = 0;
#pragma unroll
        for (int e = 0; e < kN; ++e) hit |= (uint32_t)(l[e] >= floor) << e;
        if (!__any_sync(0xffffffffu, hit)) continue;
        uint32_t inc = __popc(hit);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint32_t y = __shfl_up_sync(0xffffffffu, inc, o);
          if (lane >= o) inc += y;
        }
        uint32_t at = before + inc - __popc(hit);
#pragma unroll
        for (int e = 0; e < kN; ++e)
          if ((hit >> e) & 1) {
            to[at] = l[e];
            index[at] = (uint32_t)(begin - off + i * kN + e);
            ++at;
          }
        before += __shfl_sync(0xffffffffu, inc, 31);
      }
      cluster.sync();
      if (rank) return;
      list = (int)all;
    }

    // ------------------------------ the cut ------------------------------
    // Of the list, by the first CTA alone, or of the slices.
    const bool alone = list >= 0;
    auto of_all = [&](auto f) {  // f(token, logit) of everything above the floor
      if (alone) {
        for (int i = tid; i < list; i += kSmThreads) f((int)sh.index[i], sh.list[i]);
      } else {
        each([&](int i, const float (&l)[kN]) {
#pragma unroll
          for (int e = 0; e < kN; ++e)
            if (l[e] >= floor) f(i + e, l[e]);
        });
      }
    };
    auto meet = [&]() {
      if (alone) __syncthreads(); else cluster.sync();
    };
    uint32_t* counts = alone ? sh.all_count : sh.count;
    uint64_t* masses = alone ? sh.all_mass : sh.mass;
    // The place where the elements kept so far reach `want` of their number or weight.
    auto search = [&](bool by_mass, uint64_t want) {
      SmRange at{sm_order(top, 0), min(cut, sm_order(floor, (1 << kSmIndexBits) - 1)), 0, 0};
      while (true) {
        if (!alone) {
          for (int b = tid; b < kSmBins; b += kSmThreads) {
            sh.count[b] = 0;
            sh.mass[b] = 0;
          }
          __syncthreads();
        }
        const int bits = max(0, 54 - __clzll((long long)(at.hi - at.lo)));  // (hi - lo) >> bits < 1024
        of_all([&](int i, float l) {
          const uint64_t c = sm_order(l, i);
          if (c < at.lo || c > at.hi) return;
          const int b = (int)((c - at.lo) >> bits);
          atomicAdd(counts + b, 1u);
          if (by_mass) atomicAdd(reinterpret_cast<unsigned long long*>(masses + b), (unsigned long long)weight(l));
        });
        __syncthreads();
        if (!alone) {
          uint32_t* all_count = cluster.map_shared_rank(sh.all_count, 0);
          uint64_t* all_mass = cluster.map_shared_rank(sh.all_mass, 0);
          for (int b = tid; b < kSmBins; b += kSmThreads)
            if (sh.count[b]) {
              atomicAdd(all_count + b, sh.count[b]);
              if (by_mass) atomicAdd(reinterpret_cast<unsigned long long*>(all_mass + b), (unsigned long long)sh.mass[b]);
            }
          cluster.sync();
        }
        if (rank == 0) {
          find_bin(by_mass, at.before, want, nullptr);
          const int b = sh.bin;
          if (tid == 0) {
            SmRange r = sh.range;
            r.lo = at.lo + ((uint64_t)max(b, 0) << bits);
            r.hi = min(at.hi, r.lo + (((uint64_t)1 << bits) - 1));
            r.state = b < 0 ? 2 : bits == 0 || sh.all_count[b] == 1 ? 1 : 0;
            for (int k = 0; k < (alone ? 1 : ctas); ++k) *cluster.map_shared_rank(&sh.range, k) = r;
          }
          __syncthreads();
          for (int i = tid; i < kSmBins; i += kSmThreads) {
            sh.all_count[i] = 0;
            sh.all_mass[i] = 0;
          }
        }
        meet();
        at = sh.range;
        if (at.state == 1) cut = at.hi;
        if (at.state) return;
        __syncthreads();
      }
    };
    if (by_k) search(false, (uint64_t)top_k);
    if (by_p) {
      if (by_k) {  // a part of what top-k left
        sum = 0;
        of_all([&](int i, float l) { sum += sm_order(l, i) <= cut ? weight(l) : 0; });
        sum = sm_reduce(sum, [](uint64_t p, uint64_t q) { return p + q; });
        __syncthreads();
        if (lane == 0) sh.warp_sum[warp] = sum;
        __syncthreads();
        total = 0;
        for (int w = 0; w < kSmWarps; ++w) total += sh.warp_sum[w];
        if (!alone) {
          if (tid < ctas) tell(sh.cta_sum, total);
          cluster.sync();
          total = 0;
          for (int r = 0; r < ctas; ++r) total += sh.cta_sum[r];
        }
        want = max((uint64_t)1, sm_part_up(sm_fraction(top_p), total));
        __syncthreads();
      }
      search(true, want);
    }
  }

  // ------------------------------ the token: kept weights in index order ------------------------------
  auto kept = [&](int i, float l) -> uint64_t {
    if (!(l >= floor) || (cut != ~0ull && sm_order(l, i) > cut)) return 0;
    const uint64_t w = weight(l);
    return w >= least ? w : 0;
  };
  // each warp has a stretch of the list or of the slice, a token a lane
  const int stretch = (list + kSmThreads - 1) / kSmThreads * 32;
  const int t0 = list >= 0 ? min(list, warp * stretch) : v0 * kN, t1 = list >= 0 ? min(list, t0 + stretch) : v1 * kN;
  auto read = [&](int i, int& token) -> float {
    token = list >= 0 ? (int)sh.index[min(i, t1 - 1)] : begin - off + i;
    return i >= t1 ? -INFINITY : list >= 0 ? sh.list[i] : fmaxf((float)x[i], -INFINITY);
  };
  sum = 0;
  if (list >= 0) {
    for (int i = t0 + lane; i < t1; i += 32) sum += kept((int)sh.index[i], sh.list[i]);
  } else {
    each([&](int i, const float (&l)[kN]) {
#pragma unroll
      for (int e = 0; e < kN; ++e) sum += kept(i + e, l[e]);
    });
  }
  sum = sm_reduce(sum, [](uint64_t p, uint64_t q) { return p + q; });
  __syncthreads();
  if (lane == 0) sh.warp_sum[warp] = sum;
  __syncthreads();
  uint64_t total = 0, before = 0;
  if (list >= 0) {
    for (int w = 0; w < kSmWarps; ++w) total += sh.warp_sum[w];
  } else {
    if (tid < ctas) {
      sum = 0;
      for (int w = 0; w < kSmWarps; ++w) sum += sh.warp_sum[w];
      tell(sh.cta_sum, sum);
    }
    cluster.sync();
    for (int r = 0; r < ctas; ++r) {
      if (r == rank) before = total;
      total += sh.cta_sum[r];
    }
  }
  const uint64_t target = sm_part(sm_fraction(a.u[row]), total);  // the first sum above it
  for (int w = 0; w < warp; ++w) before += sh.warp_sum[w];
  if (target < before || target >= before + sh.warp_sum[warp]) return;
  for (int i0 = t0; i0 < t1; i0 += 32) {
    int token;
    const float l = read(i0 + lane, token);
    uint64_t inc = l > -INFINITY ? kept(token, l) : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint64_t y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += y;
    }
    const uint32_t over = __ballot_sync(0xffffffffu, before + inc > target);
    if (over) {
      if (lane == __ffs(over) - 1) put(token, l);
      return;
    }
    before += __shfl_sync(0xffffffffu, inc, 31);
  }
}

}  // namespace dinfer
