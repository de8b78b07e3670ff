// A token per row of logits by temperature, top-k, top-p and min-p from a given
// number, and its confidence (include/dinfer_ops.h, dinfer_op_sample).
//
// A row is read once: a cluster of up to 16 CTAs keeps it in shared memory, a slice
// each, and everything after the load is passes over those slices, joined
// through distributed shared memory.
//
// Weights are whole numbers, w = round(2^44 e^((l - max) / T)), whose sums are the
// same in any order.  Which token is
// drawn hangs on where u falls among up to 157000 sums of rounded weights: with
// fp32 exponentials one row in some ten thousand gets another token than the
// definition's, so the exponent is carried in two floats and the power of two
// comes from a table of 512 and a cubic, about 2^-32 of the weight in all.  Passes
// over whole slices sum the same powers as pairs of floats, two tokens an instruction
// (some 28 instructions a token where whole numbers take 50), from a table of 32 in
// every lane's own banks and a quartic, to 2^-31 of a weight and 2^-38 of the largest; a
// thread's part of them is then rounded to a whole number, so that these sums do hang on how a
// row is dealt to threads, in their last 2^-31.
//
// top-k and top-p cut the order (larger logit first, then lower index) at one
// place.  A floor under it is found first: for top-k the k-th largest of the
// threads' own maxima, which k logits reach; for top-p from the weights of an eighth
// of the row, checked by the exact sums.  What lies above it (some hundred logits
// mostly) goes to the first CTA, which finds the place by histograms of 512
// bins over (logit, index), each over the bin of the last one that holds it, until
// one element is left.  Where more than kSmList lie above it, all CTAs do the same on
// their slices, until a bin holds few enough for the first one's list; for top-p only
// between the floor and a ceiling, which the eighth gives too.  Rows without either take
// one pass.
//
// 512 rows of 126464 in bf16 with settings of their own (130 MB) take 259 us in a graph, of
// which the memory needs 19; the first form, with histograms of whole rows, one atomic a logit,
// took 651.  64 rows of 157184 in fp32 at a temperature (40 MB) take 39 us: issue slots 44%
// busy, DRAM 11%.  One row of 126464: 5.5 us greedy, 9.0 at a temperature, 39 by top-p where
// it is flat.
#pragma once
#include <cooperative_groups.h>

#include "window_attention.cuh"

namespace dinfer {

constexpr int kSmThreads = 512;
constexpr int kSmWarps = kSmThreads / 32;
constexpr int kSmCluster = 16;    // CTAs of a row at most
constexpr int kSmBins = 512;      // a thread each
static_assert(kSmBins == kSmThreads, "sm_find");
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
  int cuts;  // top_k or top_p is given
  uint64_t coarse[16], fine[32];  // 2^(j / 16), 2^(j / 512) in 2^-63rds
};

// Where the cut lies: elements [lo, hi] of the order hold it, `before` (of their number or weight) lie before them.
struct SmRange {
  uint64_t lo, hi, before;
  uint32_t count;  // of [lo, hi]
  int state;  // 0: go on, 1: found (hi is the last kept), 2: everything is kept
};

struct alignas(16) SmShared {
  uint32_t table[512];   // 2^(j / 512) in 2^-30ths,
  float2 powers[32][32];  // [j][lane], so that no two lanes meet in a bank: 2^(j / 32) as a float, and what that leaves of it
  uint64_t warp_sum[kSmWarps], warp_above[kSmWarps], cta_sum[kSmCluster], cta_high[kSmCluster], cta_listed[kSmCluster];
  float warp_f[kSmWarps], max_of[kSmCluster], sum_of[kSmCluster];
  uint32_t warp_i[kSmWarps], warp_j[kSmWarps], cta_i[kSmCluster], cta_j[kSmCluster];
  SmRange range;
  float floor, ceiling;
  uint32_t listed;
  int bin;
};
// Behind it, for calls with top-k or top-p.
struct SmCut {
  // Histograms: how many (w), and their weight in 16 bits a word, 65536 of which do not overflow.
  // `all` is the row's, in the first CTA, whose words the others add
  // to with their carries done.
  uint4 hist[kSmBins], all[kSmBins];
  float list[kSmList];  // in the first CTA: the logits above the floor in index order,
  uint32_t index[kSmList];  // and their tokens
};

struct SmScale {
  float m, ch, cl;
  float least;  // logits below it weigh less than 2^-60
};

// In line at every use, large as its code is (512 rows of 126464 in bf16 with top-p 0.9: 554 us, with one copy out of line
// 581; one flat row 39.3 and 39.6).
__device__ __forceinline__ uint64_t sm_weight(float l, const SmScale& k, const uint32_t* table) {
  // half the difference, and what it is rounded by: the whole one may pass the largest float
  const float x = 0.5f * l, m = 0.5f * k.m, ch = 2.f * k.ch;
  const float d = x - m, back = d - x, dl = (x - (d - back)) - (m + back);
  const float p = __fmul_rn(d, ch);  // not to be contracted with the sums below, which take its rounding off again
  float s = fmaf(dl, ch, fmaf(d, 2.f * k.cl, fmaf(d, ch, -p)));
  constexpr float kMagic = 24576.f;  // 1.5 * 2^14: a float's last place is 1 / 512
  const float t = fmaf(dl, ch, p) + kMagic;
  s += p - (t - kMagic);
  const float q = s * fmaf(s, fmaf(s, 0.0555041086648f, 0.240226506959f), 0.693147180560f);  // 2^s - 1
  const int n = __float_as_int(t) - __float_as_int(kMagic);
  const uint32_t hi = table[n & 511];  // 2^30 and more
  const int64_t w = ((int64_t)hi << 14) + ((int64_t)__mulhi((int)hi, __float2int_rn(q * 0x1p41f)) << 5);
  // rounded, not cut off: half a unit of each of 10^5 small weights would be more than all other errors
  const uint64_t r = (((uint64_t)w << 1 >> min(63, -(n >> 9))) + 1) >> 1;
  return l == k.m ? 1ull << 44 : p >= -44.f ? r : 0;  // NaN: 0
}

__device__ __forceinline__ uint64_t both(float x) { return f32x2(__float_as_uint(x), __float_as_uint(x)); }

// Weights of two tokens as x + x rest.
struct SmPair {
  uint64_t x, rest;
  __device__ __forceinline__ SmPair(float l0, float l1, const SmScale& k, const float2 (*powers)[32]) {
    constexpr float kMagic = 393216.f;  // 1.5 * 2^18: a float's last place is 1 / 32
    const uint64_t one = both(-1.f);
    l0 = fmaxf(l0, k.least);
    l1 = fmaxf(l1, k.least);
    const uint64_t l = f32x2(__float_as_uint(l0), __float_as_uint(l1));
    const uint64_t d = add2(l, both(-k.m)), back = fma2(l, one, d);
    const uint64_t dl = fma2(add2(back, both(k.m)), one, fma2(fma2(back, one, d), one, l));
    const uint64_t p = mul2(d, both(k.ch)), ch = both(k.ch);
    const uint64_t t = add2(fma2(dl, ch, p), both(kMagic));
    uint64_t s = fma2(dl, ch, fma2(d, both(k.cl), fma2(d, ch, mul2(d, both(-k.ch)))));
    s = add2(s, fma2(add2(t, both(-kMagic)), one, p));
    const uint64_t q = mul2(s, fma2(s, fma2(s, fma2(s, both(0.00961812910763f), both(0.0555041086648f)), both(0.240226506959f)), both(0.693147180560f)));
    float t0, t1, p0, p1;
    f32x2_parts(t, t0, t1);
    f32x2_parts(p, p0, p1);
    const int n0 = __float_as_int(t0) - __float_as_int(kMagic), n1 = __float_as_int(t1) - __float_as_int(kMagic);
    const float2 w0 = powers[n0 & 31][threadIdx.x & 31], w1 = powers[n1 & 31][threadIdx.x & 31];
    // 0 where sm_weight gives 0: what counts in these sums counts in those of whole numbers
    x = f32x2(p0 >= -44.f ? __float_as_uint(w0.x) + ((n0 >> 5) << 23) : 0u, p1 >= -44.f ? __float_as_uint(w1.x) + ((n1 >> 5) << 23) : 0u);
    rest = add2(q, f32x2(__float_as_uint(w0.y), __float_as_uint(w1.y)));
  }
  __device__ __forceinline__ void keep(bool first, bool second) {
    float x0, x1;
    f32x2_parts(x, x0, x1);
    x = f32x2(first ? __float_as_uint(x0) : 0u, second ? __float_as_uint(x1) : 0u);
  }
};
// Their sums: x joins `high`, which is 64 at first and so never smaller, and what that loses of it `low`.
struct SmSum {
  uint64_t high = both(64.f), low = 0;
  __device__ __forceinline__ void add(const SmPair& w) {
    const uint64_t one = both(-1.f), h = add2(high, w.x);
    low = fma2(w.x, w.rest, add2(low, fma2(fma2(high, one, h), one, w.x)));
    high = h;
  }
  __device__ __forceinline__ uint64_t whole() const {
    float h0, h1, l0, l1;
    f32x2_parts(high, h0, h1);
    f32x2_parts(low, l0, l1);
    const long long w = __float2ll_rn((h0 - 64.f) * 0x1p44f) + __float2ll_rn((h1 - 64.f) * 0x1p44f) + __float2ll_rn(l0 * 0x1p44f) +
                        __float2ll_rn(l1 * 0x1p44f);
    return w > 0 ? (uint64_t)w : 0;
  }
};

// Larger logits first, then lower indexes.  kDrop: bits of a logit that are always zero (16 of a bf16's).
template <int kDrop>
__device__ __forceinline__ uint64_t sm_order(float l, int index) {
  const uint32_t b = __float_as_uint(l + 0.f);  // -0 is 0
  const uint32_t up = b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
  return ((uint64_t)(~up >> kDrop) << kSmIndexBits) | (uint32_t)index;
}
// The least logit at or before a place of the order.
template <int kDrop>
__device__ __forceinline__ float sm_logit(uint64_t place) {
  const uint32_t up = ~((uint32_t)(place >> kSmIndexBits) << kDrop);
  return __uint_as_float((up & 0x80000000u ? up ^ 0x80000000u : ~up) & ~((1u << kDrop) - 1u));
}

__device__ __forceinline__ void sm_count(uint4& bin) { atomicAdd(&bin.w, 1u); }
__device__ __forceinline__ void sm_weigh(uint4& bin, uint64_t w) {
  const uint32_t x = (uint32_t)w & 0xffffu, y = (uint32_t)w >> 16, z = (uint32_t)(w >> 32);
  if (x) atomicAdd(&bin.x, x);
  if (y) atomicAdd(&bin.y, y);
  if (z) atomicAdd(&bin.z, z);
}
__device__ __forceinline__ uint64_t sm_mass(const uint4& bin) { return bin.x + ((uint64_t)bin.y << 16) + ((uint64_t)bin.z << 32); }

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

// A slice's logits in shared memory, 16 bytes at a time: pads and NaN read as -inf.  What needs no fp32 stays packed
// (bf16: two of the type an instruction).
template <typename T>
struct SmVec;
template <>
struct SmVec<float> {
  static constexpr int kN = 4;
  using Max = float;
  static __device__ __forceinline__ Max lowest() { return -INFINITY; }
  static __device__ __forceinline__ void get(const uint4& d, float (&l)[4]) {
    l[0] = fmaxf(__uint_as_float(d.x), -INFINITY);
    l[1] = fmaxf(__uint_as_float(d.y), -INFINITY);
    l[2] = fmaxf(__uint_as_float(d.z), -INFINITY);
    l[3] = fmaxf(__uint_as_float(d.w), -INFINITY);
  }
  static __device__ __forceinline__ void max(const uint4& d, Max& m) {
    m = max3(m, __uint_as_float(d.x), __uint_as_float(d.y));
    m = max3(m, __uint_as_float(d.z), __uint_as_float(d.w));
  }
  static __device__ __forceinline__ float largest(Max m) { return m; }
  // bit e: logit e is `least` or more
  static __device__ __forceinline__ uint32_t reach(const uint4& d, float least) {
    return (uint32_t)(__uint_as_float(d.x) >= least) | (uint32_t)(__uint_as_float(d.y) >= least) << 1 |
           (uint32_t)(__uint_as_float(d.z) >= least) << 2 | (uint32_t)(__uint_as_float(d.w) >= least) << 3;
  }
};
template <>
struct SmVec<__nv_bfloat16> {
  static constexpr int kN = 8;
  using Max = __nv_bfloat162;
  static __device__ __forceinline__ __nv_bfloat162 two(uint32_t w) { return *reinterpret_cast<const __nv_bfloat162*>(&w); }
  static __device__ __forceinline__ Max lowest() { return two(0xff80ff80u); }
  static __device__ __forceinline__ void get(const uint4& d, float (&l)[8]) {
    const uint32_t w[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      l[2 * i] = fmaxf(__uint_as_float(w[i] << 16), -INFINITY);
      l[2 * i + 1] = fmaxf(__uint_as_float(w[i] & 0xffff0000u), -INFINITY);
    }
  }
  static __device__ __forceinline__ void max(const uint4& d, Max& m) {
    m = __hmax2(m, __hmax2(__hmax2(two(d.x), two(d.y)), __hmax2(two(d.z), two(d.w))));
  }
  static __device__ __forceinline__ float largest(Max m) { return fmaxf(__low2float(m), __high2float(m)); }
  static __device__ __forceinline__ uint32_t reach(const uint4& d, float least) {
    const uint32_t w[4] = {d.x, d.y, d.z, d.w};
    const __nv_bfloat162 f = __bfloat162bfloat162(__float2bfloat16_ru(least));  // no bf16 lies between
    uint32_t hit = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t m = __hge2_mask(two(w[i]), f);
      hit |= ((m & 1u) | (m >> 30 & 2u)) << (2 * i);
    }
    return hit;
  }
};

template <typename T, int kBlocks>
__global__ void __launch_bounds__(kSmThreads, kBlocks) sample_kernel(const __grid_constant__ SmArgs a) {
  namespace cg = cooperative_groups;
  constexpr int kN = SmVec<T>::kN, kDrop = 32 - 8 * (int)sizeof(T);
  extern __shared__ __align__(16) uint8_t sm_raw[];
  SmShared& sh = *reinterpret_cast<SmShared*>(sm_raw);
  SmCut& sc = *reinterpret_cast<SmCut*>(sm_raw + sizeof(SmShared));  // not where a.cuts is false
  cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = blockIdx.z, ctas = gridDim.z, row = blockIdx.x;
  sh.table[tid] = (uint32_t)(__umul64hi(a.coarse[tid >> 5], a.fine[tid & 31]) >> 32);
  for (int j = warp; j < 32; j += kSmWarps) {
    const uint64_t w = __umul64hi(a.coarse[j >> 1], a.fine[(j & 1) * 16]);  // 2^-62nds
    const float f = __ull2float_rn(w);
    sh.powers[j][lane] = make_float2(f * 0x1p-62f, __ll2float_rn((long long)(w - (uint64_t)f)) / f);
  }
  if (a.cuts) sc.hist[tid] = sc.all[tid] = make_uint4(0, 0, 0, 0);
  cluster.barrier_arrive();  // waited for before the first access to another CTA's memory
  pdl_wait();
  pdl_trigger();
  const float temperature = a.temperature ? a.temperature[row] : 1.f, top_p = a.top_p ? a.top_p[row] : 1.f;
  const float min_p = a.min_p ? a.min_p[row] : 0.f;
  const int top_k = a.top_k ? a.top_k[row] : 0;
  const uint64_t u = sm_fraction(a.u[row]);

  // the slice, as it lies behind a boundary of 16 bytes, with -inf around it
  const int begin = rank * a.slice, n = max(0, min(a.slice, a.vocab - begin));
  const T* from = reinterpret_cast<const T*>(a.x) + (int64_t)row * a.stride + begin;
  const int off = (int)(reinterpret_cast<uintptr_t>(from) & 15) / (int)sizeof(T);
  uint8_t* raw = sm_raw + sizeof(SmShared) + (a.cuts ? sizeof(SmCut) : 0);
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
#pragma unroll 1
    for (int i = v0 + lane; i < v1; i += 32) {
      float l[kN];
      SmVec<T>::get(reinterpret_cast<const uint4*>(raw)[i], l);
      f(begin - off + i * kN, l);
    }
  };
  // v of every CTA to every CTA's to[rank], to be read behind the next cluster barrier.  Told again only behind another one:
  // a CTA that is late would read the second value for the first, decide by it, and wait where the others do not.
  auto tell = [&](auto* to, auto v) { *(cluster.map_shared_rank(to, tid) + rank) = v; };

  auto each_raw = [&](auto f) {
#pragma unroll 1
    for (int i = v0 + lane; i < v1; i += 32) f(begin - off + i * kN, reinterpret_cast<const uint4*>(raw)[i]);
  };
  // f(token, logit) for the logits of a vector that `hit` names, one a turn: the lanes' turns are those of the one with
  // the most, where a turn for each place in the vector would be all of them
  auto each_hit = [&](int token, uint32_t hit, auto f) {
#pragma unroll 1
    for (; hit; hit &= hit - 1) {
      const int i = token + __ffs(hit) - 1;
      f(i, fmaxf((float)x[i - begin + off], -INFINITY));
    }
  };

  float mine;  // the thread's largest
  {
    typename SmVec<T>::Max most = SmVec<T>::lowest();
#pragma unroll 4
    for (int i = v0 + lane; i < v1; i += 32) SmVec<T>::max(reinterpret_cast<const uint4*>(raw)[i], most);
    mine = fmaxf(SmVec<T>::largest(most), -INFINITY);
  }
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

  const bool greedy = !(temperature > 0.f) || top_k == 1, by_k = !greedy && top_k > 0 && top_k < a.vocab, by_p = !greedy && top_p < 1.f;
  SmScale scale;
  {
    scale.m = top;
    // log2(e) / temperature in two floats
    constexpr float kLog2e = 1.44269502162933349609f, kLog2eRest = 1.92596299112661746887e-8f;
    scale.ch = fminf(__fdiv_rn(kLog2e, temperature), 0x1p100f);
    scale.cl = __fdiv_rn(fmaf(-scale.ch, temperature, kLog2e) + kLog2eRest, temperature);
    if (!(fabsf(scale.cl) <= 0x1p-20f * scale.ch)) scale.cl = 0.f;  // temperatures at the ends of a float's range
    scale.least = top - 60.f / scale.ch;
  }
  // else the sums are of whole numbers: temperatures whose span of weights is no float, or within the logits' last places
  const bool plain = fabsf(scale.least) < 1e30f && 60.f / scale.ch > 1e-5f * fabsf(top);
  constexpr int kLastBin = kSmBins - 1;  // of the exponent
  const float bin_scale = scale.ch * (kLastBin / kSmRange);
  auto bin_of = [&](float l) { return l == top ? 0 : (int)fminf((float)kLastBin, (top - l) * bin_scale); };

  // The floor: a histogram over the exponent of the threads' maxima, or of weights: of the maxima, which hold what few
  // tokens have much of, and eight times those of every eighth vector.
  if (by_k) {
    if (mine > -INFINITY) sm_count(sc.hist[bin_of(mine)]);
  } else if (by_p) {
    auto add = [&](float l, float scaled) {
      const float w = (l == top ? 1.f : ex2_approx((l - top) * scale.ch)) * scaled;
      if (w >= 1.f) sm_weigh(sc.hist[bin_of(l)], (uint64_t)w);
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
    if (top == INFINITY) {
      each([&](int, const float (&l)[kN]) {
#pragma unroll
        for (int e = 0; e < kN; ++e) sum += l[e] == top ? 1.f : 0.f;
      });
    } else {
      uint64_t sums = 0;
      each([&](int, const float (&l)[kN]) {
#pragma unroll
        for (int e = 0; e < kN; e += 2) {
          float p, q;
          f32x2_parts(mul2(add2(f32x2(__float_as_uint(l[e]), __float_as_uint(l[e + 1])), both(-top)), both(1.4426950408889634f)), p, q);
          sums = add2(sums, f32x2(__float_as_uint(ex2_approx(p)), __float_as_uint(ex2_approx(q))));
        }
      });
      float s1;
      f32x2_parts(sums, sum, s1);
      sum += s1;
    }
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
    const float d = l - top, back = d - l, rest = (l - (d - back)) - (top + back);  // what the difference is rounded by
    a.conf[row] = (l == top ? 1.f : expf(d) * (1.f + (fabsf(rest) < 1.f ? rest : 0.f))) / sum;
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

  // The first CTA's threads: the bin at which its histogram's sum (from 1), or the row's (2), on top of `before`, reaches
  // `want` (0: a part of the whole) into sh.bin (-1: none), its sum before the bin and its count.
  auto push_bins = [&]() {
    uint4 h = sc.hist[tid];
    h.y += h.x >> 16;
    h.z += h.y >> 16;
    uint4* to = cluster.map_shared_rank(sc.all, 0) + tid;
    if (h.x & 0xffffu) atomicAdd(&to->x, h.x & 0xffffu);
    if (h.y & 0xffffu) atomicAdd(&to->y, h.y & 0xffffu);
    if (h.z) atomicAdd(&to->z, h.z);
    if (h.w) atomicAdd(&to->w, h.w);
  };
  auto find_bin = [&](bool by_mass, int from, uint64_t before, uint64_t want, uint64_t part) {
    const uint4 h = from == 1 ? sc.hist[tid] : sc.all[tid];
    if (from > 1) sc.all[tid] = make_uint4(0, 0, 0, 0);
    const uint32_t count = h.w;
    const uint64_t v = by_mass ? sm_mass(h) : h.w;
    uint64_t inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint64_t y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += y;
    }
    if (lane == 31) sh.warp_sum[warp] = inc;
    if (tid == 0) sh.bin = -1;
    __syncthreads();
    uint64_t total = before;
    before += inc - v;
    for (int w = 0; w < kSmWarps; ++w) {
      if (w < warp) before += sh.warp_sum[w];
      total += sh.warp_sum[w];
    }
    if (want == 0) want = max((uint64_t)1, sm_part(part, total));
    if (before < want && want <= before + v) {
      sh.bin = tid;
      sh.range.before = before;
      sh.range.count = count;
    }
    __syncthreads();
  };

  // ------------------------------ rows without a cut ------------------------------
  constexpr float kLeast = -3.402823466e38f;  // every logit that is there reaches it
  float floor = -INFINITY, ceiling = INFINITY;  // only logits from the floor on count; all from the ceiling on are kept
  bool banded = false;
  uint64_t cut = ~0ull;     // the last kept place of the order
  int list = -1;            // the first CTA's: how many logits it has in its list
  uint64_t sum = 0;
  if (!by_k && !by_p) {
    if (least) floor = top + temperature * logf(fminf(min_p, 1.f)) * 1.0001f - 1e-6f * fabsf(top);
    if (!(floor <= top)) floor = -INFINITY;
  } else {
    // ------------------------------ the floor ------------------------------
    __syncthreads();
    push_bins();
    cluster.sync();
    if (rank == 0) {
      sc.hist[tid] = sc.all[tid];  // looked at twice
      sc.all[tid] = make_uint4(0, 0, 0, 0);
      // no bin: fewer maxima than top_k; weights that are all below 2^-32
#pragma unroll 1
      for (int side = 0; side < 2; ++side) {
        const float p = side ? top_p - fminf(0.25f * top_p, 0.03f) : top_p + fminf(0.25f * (1.f - top_p), 0.03f);
        find_bin(!by_k, 1, 0, by_k ? (uint64_t)top_k : 0, sm_fraction(p));
        const int b = sh.bin;
        if (tid < ctas) {
          if (side == 0)
            *cluster.map_shared_rank(&sh.floor, tid) = b == kLastBin ? -INFINITY : top - (b >= 0 ? b + 1.1f : by_k ? INFINITY : 32.f * (kLastBin / kSmRange)) / bin_scale;
          if (by_k || side) *cluster.map_shared_rank(&sh.ceiling, tid) = by_k || b <= 0 ? INFINITY : top - (b - 0.1f) / bin_scale;
        }
        if (by_k) break;
        __syncthreads();
      }
    }
    cluster.sync();
    floor = sh.floor;
    if (!(floor > -INFINITY)) floor = kLeast;
    // Top-p of a flat row keeps half of it: then only what lies between the floor and a ceiling, which all have that are
    // kept for certain, is looked at one by one.
    ceiling = sh.ceiling;
    // how many lie above them, and for top-p all weights and theirs
    uint32_t count = 0, high = 0;
    uint64_t certain = 0;
    auto over = [&](float l) {
      count += l >= floor;
      high += l >= ceiling;
    };
    if (by_k) {
      ceiling = INFINITY;
      each_raw([&](int, const uint4& d) { count += __popc(SmVec<T>::reach(d, floor)); });
    } else if (!plain) {
      ceiling = INFINITY;
      each([&](int, const float (&l)[kN]) {
#pragma unroll
        for (int e = 0; e < kN; ++e) {
          over(l[e]);
          sum += weight(l[e]);
        }
      });
    } else {
      SmSum all, some;
      each([&](int, const float (&l)[kN]) {
#pragma unroll
        for (int e = 0; e < kN; e += 2) {
          over(l[e]);
          over(l[e + 1]);
          SmPair w(l[e], l[e + 1], scale, sh.powers);
          all.add(w);
          w.keep(l[e] >= ceiling, l[e + 1] >= ceiling);
          some.add(w);
        }
      });
      sum = all.whole();
      certain = some.whole();
    }
    high = __reduce_add_sync(0xffffffffu, high);
    certain = sm_reduce(certain, [](uint64_t p, uint64_t q) { return p + q; });
    count = __reduce_add_sync(0xffffffffu, count);
    sum = sm_reduce(sum, [](uint64_t p, uint64_t q) { return p + q; });
    if (lane == 0) {
      sh.warp_i[warp] = count;
      sh.warp_j[warp] = high;
      sh.warp_sum[warp] = sum;
      sh.warp_above[warp] = certain;
    }
    __syncthreads();
    if (tid < ctas) {
      count = high = 0;
      sum = certain = 0;
      for (int w = 0; w < kSmWarps; ++w) {
        count += sh.warp_i[w];
        high += sh.warp_j[w];
        sum += sh.warp_sum[w];
        certain += sh.warp_above[w];
      }
      tell(sh.cta_i, count);
      tell(sh.cta_j, high);
      tell(sh.cta_sum, sum);
      tell(sh.cta_high, certain);
    }
    cluster.sync();
    uint32_t all = 0, all_high = 0, before = 0, before_high = 0;
    uint64_t total = 0;
    certain = 0;
    for (int r = 0; r < ctas; ++r) {
      if (r == rank) {
        before = all;
        before_high = all_high;
      }
      all += sh.cta_i[r];
      all_high += sh.cta_j[r];
      total += sh.cta_sum[r];
      certain += sh.cta_high[r];
    }
    uint64_t want = by_k ? (uint64_t)top_k : max((uint64_t)1, sm_part_up(sm_fraction(top_p), total));
    if (by_k && all < (uint32_t)top_k) {  // the floor lies too high (no cut, or a logit's last place)
      floor = kLeast;
      all = 0x7fffffff;
    }
    bool band = all > kSmList && ceiling < INFINITY && certain < want;
    if (!band) {
      ceiling = INFINITY;
      certain = 0;
    } else {
      all -= all_high;
      before -= before_high;
    }
    // Puts what lies between floor and ceiling, `all` logits, `before` of them before this warp's stretch, into the first
    // CTA's list; returns this thread's part of its weight, if that is asked for.
    auto gather = [&](bool weigh) -> uint64_t {
      uint64_t w = 0;
      float* to = cluster.map_shared_rank(sc.list, 0);
      uint32_t* index = cluster.map_shared_rank(sc.index, 0);
      for (int i0 = v0; i0 < v1; i0 += 32) {
        const int i = i0 + lane;
        uint32_t hit = 0;
        uint4 d{};
        if (i < v1) {
          d = reinterpret_cast<const uint4*>(raw)[i];
          hit = SmVec<T>::reach(d, floor);
          if (band) hit &= ~SmVec<T>::reach(d, ceiling);
        }
        if (!__any_sync(0xffffffffu, hit)) continue;
        uint32_t inc = __popc(hit);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint32_t y = __shfl_up_sync(0xffffffffu, inc, o);
          if (lane >= o) inc += y;
        }
        uint32_t at = before + inc - __popc(hit);
        each_hit(begin - off + i * kN, hit, [&](int token, float l) {
          to[at] = l;
          index[at] = (uint32_t)token;
          ++at;
          if (weigh) w += weight(l);
        });
        before += __shfl_sync(0xffffffffu, inc, 31);
      }
      return w;
    };
    // ------------------------------ the list ------------------------------
    bool listed = all <= kSmList;
    if (listed) {
      for (int w = 0; w < warp; ++w) before += sh.warp_i[w] - (band ? sh.warp_j[w] : 0);
      uint64_t w = sm_reduce(gather(!by_k), [](uint64_t p, uint64_t q) { return p + q; });
      if (!by_k) {  // does the floor lie low enough?
        __syncthreads();
        if (lane == 0) sh.warp_sum[warp] = w;
        __syncthreads();
        if (tid < ctas) {
          w = 0;
          for (int k = 0; k < kSmWarps; ++k) w += sh.warp_sum[k];
          tell(sh.cta_listed, w);
        }
      }
      cluster.sync();
      if (!by_k) {
        w = certain;
        for (int r = 0; r < ctas; ++r) w += sh.cta_listed[r];
        if (w < want) {
          listed = band = false;
          floor = kLeast;
          ceiling = INFINITY;
          certain = 0;
        }
      }
      if (listed && !band) {
        if (rank) return;
        list = (int)all;
      }
    }

    // ------------------------------ the cut ------------------------------
    // Of the list, by the first CTA alone, or of the slices.
    bool alone = listed;
    auto of_all = [&](auto f) {  // f(token, logit) of everything between the floor and the ceiling
      if (alone) {
        for (int i = tid; i < (int)all; i += kSmThreads) f((int)sc.index[i], sc.list[i]);
      } else {
        each_raw([&](int i, const uint4& d) {
          uint32_t hit = SmVec<T>::reach(d, floor);
          if (band) hit &= ~SmVec<T>::reach(d, ceiling);
          each_hit(i, hit, f);
        });
      }
    };
    auto meet = [&]() {
      if (alone) __syncthreads(); else cluster.sync();
    };
    // A level of the search: the bin of [lo, hi] at which what is kept so far reaches `want` in number or weight.
    auto level = [&](bool by_mass, uint64_t want, const SmRange& at) -> SmRange {
      sc.hist[tid] = make_uint4(0, 0, 0, 0);
      __syncthreads();
      const int bits = max(0, 55 - __clzll((long long)(at.hi - at.lo)));  // (hi - lo) >> bits < 512
      of_all([&](int i, float l) {
        const uint64_t c = sm_order<kDrop>(l, i);
        if (c < at.lo || c > at.hi) return;
        uint4& bin = sc.hist[(int)((c - at.lo) >> bits)];
        sm_count(bin);
        if (by_mass) sm_weigh(bin, weight(l));
      });
      __syncthreads();
      if (!alone) {
        push_bins();
        cluster.sync();
      }
      if (rank == 0) {
        find_bin(by_mass, alone ? 1 : 2, at.before, want, 0);
        if (tid == 0) {
          SmRange r = sh.range;
          const int b = sh.bin;
          r.lo = at.lo + ((uint64_t)max(b, 0) << bits);
          r.hi = min(at.hi, r.lo + (((uint64_t)1 << bits) - 1));
          r.state = b < 0 ? 2 : bits == 0 || r.count == 1 ? 1 : 0;
          for (int k = 0; k < (alone ? 1 : ctas); ++k) *cluster.map_shared_rank(&sh.range, k) = r;
          sh.listed = 0;
        }
      }
      meet();
      const SmRange r = sh.range;
      __syncthreads();  // it is written again
      return r;
    };
    // By number, then by weight, and that again where the floor of an eighth of the row lay too high.  One place calls
    // level(): its code is large.
    enum { kByNumber, kByWeight, kAgain, kDone };
    int phase = by_k ? kByNumber : kByWeight;
    if (listed && rank) phase = kDone;
    bool fresh = true, solo = false, idle = false;  // solo: the first CTA takes what is left; idle: the others meanwhile
    SmRange at{};
    uint32_t was = all;
    while (phase != kDone) {
      if (fresh) {
        if (phase == kByWeight && by_k) {  // a part of what top-k left
          sum = 0;
          of_all([&](int i, float l) { sum += sm_order<kDrop>(l, i) <= cut ? weight(l) : 0; });
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
        if (phase == kAgain) {
          band = false;
          floor = kLeast;
          ceiling = INFINITY;
          certain = 0;
        }
        at = SmRange{sm_order<kDrop>(fminf(top, ceiling), 0), min(cut, sm_order<kDrop>(floor, (1 << kSmIndexBits) - 1)), certain, 0, 0};
        fresh = false;
      }
      if (!idle) at = level(phase != kByNumber, want, at);
      if (at.state == 0 && !alone && at.count <= kSmList) {  // the bin's logits to the list, in any order
        of_all([&](int i, float l) {
          const uint64_t c = sm_order<kDrop>(l, i);
          if (c < at.lo || c > at.hi) return;
          const uint32_t k = atomicAdd(cluster.map_shared_rank(&sh.listed, 0), 1u);
          cluster.map_shared_rank(sc.list, 0)[k] = l;
          cluster.map_shared_rank(sc.index, 0)[k] = (uint32_t)i;
        });
        cluster.sync();
        if (rank == 0) {
          solo = alone = true;
          all = at.count;
          continue;
        }
        idle = true;
      }
      if (solo && at.state) {
        solo = alone = false;
        all = was;
        if (tid < ctas) *cluster.map_shared_rank(&sh.range, tid) = at;
        idle = true;
      }
      if (idle) {
        cluster.sync();
        at = sh.range;
        __syncthreads();
        idle = false;
      }
      if (at.state == 0) continue;
      if (at.state == 1) cut = at.hi;
      fresh = true;
      phase = phase == kByNumber ? (by_p ? kByWeight : kDone) : at.state == 2 && phase == kByWeight && !alone ? kAgain : kDone;
    }
    if (listed && band) {
      if (rank == 0 && tid < ctas) cluster.map_shared_rank(&sh.range, tid)->hi = cut;
      cluster.sync();
      cut = sh.range.hi;
    }
    banded = band;
  }

  // ------------------------------ the token: kept weights in index order ------------------------------
  // the cut as a logit and, among its equals, a token
  const float cut_l = cut == ~0ull ? -INFINITY : sm_logit<kDrop>(cut);
  const int cut_i = cut == ~0ull ? 0x7fffffff : (int)(cut & ((1 << kSmIndexBits) - 1));
  if (floor < cut_l) floor = cut_l;
  auto is_kept = [&](int i, float l) { return l > cut_l || (l == cut_l && i <= cut_i); };
  auto kept = [&](int i, float l) -> uint64_t {
    if (!(l >= floor) || !is_kept(i, l)) return 0;
    const uint64_t w = weight(l);
    return w >= least ? w : 0;
  };
  // each warp has a stretch of the list or of the slice
  const int stretch = (list + kSmThreads - 1) / kSmThreads * 32;
  sum = 0;
  if (list >= 0) {
    for (int i = warp * stretch + lane; i < min(list, (warp + 1) * stretch); i += 32) sum += kept((int)sc.index[i], sc.list[i]);
  } else if (plain && least == 0 && cut == ~0ull) {
    SmSum pairs;
    each([&](int, const float (&l)[kN]) {
#pragma unroll
      for (int e = 0; e < kN; e += 2) pairs.add(SmPair(l[e], l[e + 1], scale, sh.powers));
    });
    sum = pairs.whole();
  } else if (banded && least == 0) {  // what lies above the ceiling is summed already
    if (lane == 0) sum = sh.warp_above[warp];
    each_raw([&](int i, const uint4& d) {
      const uint32_t hit = SmVec<T>::reach(d, floor) & ~SmVec<T>::reach(d, ceiling);
      each_hit(i, hit, [&](int token, float l) { sum += kept(token, l); });
    });
  } else if (plain && least == 0) {
    SmSum pairs;
    each([&](int i, const float (&l)[kN]) {
#pragma unroll
      for (int e = 0; e < kN; e += 2) {
        SmPair w(l[e], l[e + 1], scale, sh.powers);
        w.keep(is_kept(i + e, l[e]), is_kept(i + e + 1, l[e + 1]));
        pairs.add(w);
      }
    });
    sum = pairs.whole();
  } else {
    each_raw([&](int i, const uint4& d) {
      const uint32_t hit = SmVec<T>::reach(d, floor);
      each_hit(i, hit, [&](int token, float l) { sum += kept(token, l); });
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
  const uint64_t target = sm_part(u, total);  // the first sum above it
  // the warp whose stretch it lies in, then all warps on that stretch, then the one whose part it lies in
  int owner = -1;
  for (int w = 0; w < kSmWarps; ++w) {
    if (target < before) break;
    if (target < before + sh.warp_sum[w]) {
      owner = w;
      break;
    }
    before += sh.warp_sum[w];
  }
  if (owner < 0) return;  // another CTA's: all its warps
  const int o0 = list >= 0 ? min(list, owner * stretch) : min(vecs, owner * per) * kN;
  const int o1 = list >= 0 ? min(list, o0 + stretch) : min(vecs, min(vecs, owner * per) + per) * kN;
  const int part = (o1 - o0 + kSmThreads - 1) / kSmThreads * 32, t0 = min(o1, o0 + warp * part), t1 = min(o1, t0 + part);
  auto read = [&](int i, int& token) -> float {
    token = list >= 0 ? (int)sc.index[min(i, t1 - 1)] : begin - off + i;
    return i >= t1 ? -INFINITY : list >= 0 ? sc.list[i] : fmaxf((float)x[i], -INFINITY);
  };
  sum = 0;
  for (int i0 = t0; i0 < t1; i0 += 32) {
    int token;
    const float l = read(i0 + lane, token);
    sum += l > -INFINITY ? kept(token, l) : 0;
  }
  sum = sm_reduce(sum, [](uint64_t p, uint64_t q) { return p + q; });
  __syncthreads();  // the warps' sums are read
  if (lane == 0) sh.warp_sum[warp] = sum;
  __syncthreads();
  // The last part that holds any weight.  There is one: the stretch's sum is above 0, in floats too only where a token counts,
  // and one that counts weighs 1 at least in whole numbers.
  int last_part = -1;
  for (int w = 0; w < kSmWarps; ++w)
    if (sh.warp_sum[w]) last_part = w;
  for (int w = 0; w < warp; ++w) before += sh.warp_sum[w];
  const bool here = before <= target && target < before + sh.warp_sum[warp];
  if (!here && !(warp == last_part && target >= before + sh.warp_sum[warp])) return;
  // Where the stretch's sum in floats is a few units above that in whole numbers: its last token that counts.
  int last = -1;
  float last_l = 0.f;
  for (int i0 = t0; i0 < t1; i0 += 32) {
    int token;
    const float l = read(i0 + lane, token);
    const uint64_t w = l > -INFINITY ? kept(token, l) : 0;
    uint64_t inc = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint64_t y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += y;
    }
    const uint32_t over = __ballot_sync(0xffffffffu, before + inc > target), some = __ballot_sync(0xffffffffu, w > 0);
    if (over) {
      if (lane == __ffs(over) - 1) put(token, l);
      return;
    }
    if (some) {
      last = __shfl_sync(0xffffffffu, token, 31 - __clz(some));
      last_l = __shfl_sync(0xffffffffu, l, 31 - __clz(some));
    }
    before += __shfl_sync(0xffffffffu, inc, 31);
  }
  if (lane == 0) put(last, last_l);
}

}  // namespace dinfer
