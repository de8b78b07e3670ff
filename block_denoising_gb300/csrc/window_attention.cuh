// Attention of many rows with a sliding window and sinks over ragged
// sequences (include/dinfer_kv.h, dinfer_op_window_attention): what its
// kernels share, and the fp32 kernel.
//
// Row i of a sequence with nq rows and nk keys stands at p = nk - nq + i and
// sees key j if j <= p + right and (j >= p - left or j < sinks): one interval
// [lo, hi] and the sinks in front of it.
#pragma once
#include "attention_tc.cuh"
#include "kv_attention.cuh"

namespace dinfer {

// Two fp32 operations an instruction, on register pairs.
__device__ __forceinline__ uint64_t f32x2(uint32_t lo, uint32_t hi) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(lo), "r"(hi));
  return d;
}
__device__ __forceinline__ void f32x2_parts(uint64_t d, float& lo, float& hi) {
  uint32_t a, b;
  asm("mov.b64 {%0, %1}, %2;" : "=r"(a), "=r"(b) : "l"(d));
  lo = __uint_as_float(a);
  hi = __uint_as_float(b);
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

struct WaArgs {
  const void* q;
  const void* k;
  const void* v;
  void* o;
  const int32_t* cu_q;  // both NULL: one sequence of all rows
  const int32_t* cu_k;
  int64_t q_stride, k_stride, v_stride, o_stride;  // elements
  int batch, total_q, total_k, heads, kv_heads, group;
  int left, right, sinks;
  float scale_log2;
  int last_first;  // fp32: CTAs take the tiles from the last to the first
  DevState* status;
  float* partial;  // the keys of a tile dealt to up to `splits` CTAs
  int* tickets;
  int splits;
};

// One sequence's rows and keys; out-of-order or out-of-range cu entries give an empty one.
struct WaSeq {
  int q0, nq, k0, nk;
};
__device__ __forceinline__ int wa_rows_of(const WaArgs& a, int b, int* begin) {
  const int x0 = a.cu_q ? a.cu_q[b] : 0, x1 = a.cu_q ? a.cu_q[b + 1] : a.total_q;
  *begin = x0;
  return (x0 < 0 || x1 > a.total_q) ? 0 : max(0, x1 - x0);
}
__device__ __forceinline__ WaSeq wa_seq(const WaArgs& a, int b) {
  WaSeq s;
  s.nq = wa_rows_of(a, b, &s.q0);
  s.k0 = a.cu_k ? a.cu_k[b] : 0;
  const int x1 = a.cu_k ? a.cu_k[b + 1] : a.total_k;
  s.nk = (s.k0 < 0 || x1 > a.total_k) ? 0 : max(0, x1 - s.k0);
  if (s.nk == 0) s.k0 = 0;
  return s;
}

// Which sequence and which of its tiles of `tile_rows` rows is tile number x:
// whole warps, 32 sequences a step.  Returns false behind the last tile.
__device__ __forceinline__ bool wa_find_tile(const WaArgs& a, int x, int tile_rows, int* b, int* tile) {
  const int lane = threadIdx.x & 31;
  for (int b0 = 0; b0 < a.batch; b0 += 32) {
    int begin, tiles = 0;
    if (b0 + lane < a.batch) tiles = (wa_rows_of(a, b0 + lane, &begin) + tile_rows - 1) / tile_rows;
    int inc = tiles;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += u;
    }
    const uint32_t past = __ballot_sync(0xffffffffu, inc > x);
    if (past) {
      const int l = __ffs(past) - 1;
      *b = b0 + l;
      *tile = x - __shfl_sync(0xffffffffu, inc - tiles, l);
      return true;
    }
    x -= __shfl_sync(0xffffffffu, inc, 31);
  }
  return false;
}

// The keys row i sees: [lo, hi] and the first min(sinks, lo, hi + 1) ones.
struct WaRange {
  int lo, hi;
};
__device__ __forceinline__ WaRange wa_range(const WaArgs& a, const WaSeq& s, int i) {
  const int64_t p = (int64_t)s.nk - s.nq + i;
  WaRange r;
  r.lo = a.left < 0 ? 0 : (int)max((int64_t)0, min((int64_t)s.nk, p - a.left));
  r.hi = a.right < 0 ? s.nk - 1 : (int)max((int64_t)-1, min((int64_t)s.nk - 1, p + a.right));
  return r;
}
__device__ __forceinline__ bool wa_sees(const WaRange& r, int sinks, int j) {
  return j <= r.hi && (j >= r.lo || j < sinks);
}

// Key tile at which part `part` of `parts` of w key tiles begins, floor(part w / parts):
// the product itself would pass 2^31 from 2.3e8 keys on (7.1 million tiles of 32 keys in 304 parts).
__host__ __device__ __forceinline__ int wa_part_begin(int w, int part, int parts) {
  return part * (w / parts) + part * (w % parts) / parts;
}

// One row by the definition (ka_row_exact): only keys that the row sees are read,
// so nothing a masked key holds can reach the result.  The tile kernels multiply
// masked keys' values by a weight of 0, which is NaN for an infinite or NaN value,
// and their sums of weights up to 2^8 overflow where the mean does not; a row that
// comes out not finite is done again here, and then holds what its own keys give.
// (Masked scores are left out before anything is summed, so a sum of weights that is
// NaN or 0 is the row's own: such rows are NaN or zeros at once.)  One warp, eight
// keys at a time: some 160 us a thousand keys, paid only by such rows.
template <typename T, int HD>
__device__ __noinline__ void wa_row_exact(const WaArgs& a, const WaSeq s, int i, int head) {
  constexpr int kE = HD / 32;
  const WaRange r = wa_range(a, s, i);
  const T* k0 = reinterpret_cast<const T*>(a.k) + (int64_t)s.k0 * a.k_stride + (head / a.group) * HD;
  const T* v0 = reinterpret_cast<const T*>(a.v) + (int64_t)s.k0 * a.v_stride + (head / a.group) * HD;
  const int front = min(a.sinks, min(r.lo, r.hi + 1));
  float o[kE];
  ka_row_exact<T, HD, false>(reinterpret_cast<const T*>(a.q) + (int64_t)(s.q0 + i) * a.q_stride + head * HD,
                      front + max(0, r.hi - r.lo + 1), a.scale_log2,
                      [&](int x, const T*& k, const T*& v) {
                        const int j = x < front ? x : x - front + r.lo;
                        k = k0 + (int64_t)j * a.k_stride;
                        v = v0 + (int64_t)j * a.v_stride;
                      },
                      o);
  T* out = reinterpret_cast<T*>(a.o) + (int64_t)(s.q0 + i) * a.o_stride + head * HD + (threadIdx.x & 31) * kE;
#pragma unroll
  for (int e = 0; e < kE; ++e) {
    if constexpr (sizeof(T) == 2) out[e] = __float2bfloat16(o[e]); else out[e] = o[e];
  }
}

// ---------------------------------------------------------------------------
// fp32
// ---------------------------------------------------------------------------
// One CTA = 4 kTy rows of one head, 16 kTy threads; K and V in tiles of 32 keys,
// two of them in shared memory, the next one copied in while the current one is
// worked on.  Thread (ty, tx) of kTy x 16 computes the scores of rows 4 ty .. + 3
// and keys tx, tx + 16, and owns 4 rows x HD / 16 columns of the output; two FMAs
// an instruction.  Bound by the fp32 FMA rate (there is no fp32 tensor product
// that keeps 24 bits) and the shared-memory reads that feed it, which is why a
// thread has four rows in the short tiles too.
//
// kTy = 16 (64 rows): 41 TFLOP/s (16 heads of 128, 4096 causal rows; peak 80).
// kTy = 4 (16 rows) for short calls, two or more CTAs an SM: 62 rows in five
// sequences behind 975 keys each, 32 heads of 64: 52 us; 16 x 16 threads with a
// row each read every key tile eight times: 86 us.  Where these leave SMs idle
// the keys of a tile go to several CTAs too (one row over 4001 keys, 32 heads of
// 64: 30 us, 188 without).
constexpr int kWfKeys = 32;
constexpr int kWfE = 4;  // rows of a thread
// key tiles of a part at least (4 heads of 64, one row over 600 keys, and over 4001:
// with 3 11.3 and 19.2 us, 2 10.9 and 21.9, 4 12.1 and 18.0, 8 19.2 and 20.2)
constexpr int kWfPartTiles = 3;
template <int HD, int kTy>
struct WfCfg {
  static constexpr int kThreads = 16 * kTy;
  static constexpr int kRows = kWfE * kTy;
  static constexpr int kPad = HD + 4;              // rows of Q and K start 4 banks apart
  static constexpr int kPitchP = kWfKeys + 4;
  static constexpr int kStage = kWfKeys * (kPad + HD);  // floats: K, then V
  static constexpr int kOffKv = kRows * kPad;
  static constexpr int kOffP = kOffKv + 2 * kStage;
  static constexpr int kSmem = (kOffP + kRows * kPitchP) * 4;
  static constexpr int kSlotFloats = kRows * (2 + HD);  // a part's rows in the workspace: (m, l), then O
};

// kSplit: the keys of a tile dealt to up to a.splits CTAs.
template <int HD, int kTy, bool kSplit>
__global__ void __launch_bounds__(16 * kTy, kTy == 16 ? 2 : 4) window_f32_kernel(const __grid_constant__ WaArgs a) {
  using Cfg = WfCfg<HD, kTy>;
  constexpr int kRows = Cfg::kRows, kVecs = HD / 4, kE = kWfE, kThreads = Cfg::kThreads;
  extern __shared__ __align__(16) float wf_sm[];
  float* qs = wf_sm;
  float* ps = wf_sm + Cfg::kOffP;
  pdl_wait();
  pdl_trigger();
  int b, tile;
  const int unit = kSplit ? blockIdx.x / a.splits : a.last_first ? gridDim.x - 1 - blockIdx.x : blockIdx.x;
  if (!wa_find_tile(a, unit / a.heads, kRows, &b, &tile)) return;
  const WaSeq s = wa_seq(a, b);
  const int head = unit % a.heads, i0 = tile * kRows, rows = min(kRows, s.nq - i0);
  const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
  const float* q = reinterpret_cast<const float*>(a.q) + (int64_t)(s.q0 + i0) * a.q_stride + head * HD;
  const float* k = reinterpret_cast<const float*>(a.k) + (int64_t)s.k0 * a.k_stride + (head / a.group) * HD;
  const float* v = reinterpret_cast<const float*>(a.v) + (int64_t)s.k0 * a.v_stride + (head / a.group) * HD;
  for (int x = tid; x < kRows * kVecs; x += kThreads) {
    const int r = x / kVecs, d = x % kVecs * 4;
    cp_async16(smem_u32(qs + r * Cfg::kPad + d), q + (int64_t)min(r, rows - 1) * a.q_stride + d, r < rows ? 16 : 0);
  }
  // keys some row of the tile sees: the sinks, then from the first row's lo to the last row's hi
  const WaRange top = wa_range(a, s, i0), bottom = wa_range(a, s, i0 + rows - 1);
  int front = min(a.sinks, min(top.lo, bottom.hi + 1)), end = bottom.hi + 1;
  int begin = max((front + kWfKeys - 1) / kWfKeys, top.lo / kWfKeys) * kWfKeys;  // the window's tiles
  int parts = 1, part = 0;
  if constexpr (kSplit) {  // the sinks go to the first part
    const int w = max(0, (end - begin + kWfKeys - 1) / kWfKeys);
    parts = max(1, min(a.splits, w / kWfPartTiles));
    part = blockIdx.x % a.splits;
    if (part >= parts) {
      cp_async_wait<0>();
      return;
    }
    if (part > 0) front = 0;
    end = min(end, begin + wa_part_begin(w, part + 1, parts) * kWfKeys);
    begin += wa_part_begin(w, part, parts) * kWfKeys;
  }
  auto load = [&](int j0, int buf) {  // keys behind the sequence's end: zeros
    float* ks = wf_sm + Cfg::kOffKv + buf * Cfg::kStage;
#pragma unroll
    for (int x = tid; x < kWfKeys * kVecs; x += kThreads) {
      const int r = x / kVecs, d = x % kVecs * 4, j = min(j0 + r, s.nk - 1), bytes = j0 + r < s.nk ? 16 : 0;
      cp_async16(smem_u32(ks + r * Cfg::kPad + d), k + (int64_t)j * a.k_stride + d, bytes);
      cp_async16(smem_u32(ks + kWfKeys * Cfg::kPad + r * HD + d), v + (int64_t)j * a.v_stride + d, bytes);
    }
  };
  auto behind = [&](int j0) {  // the tile after j0's: behind the sinks, on to the window
    const int j = j0 + kWfKeys;
    return j >= front ? max(j, begin) : j;
  };
  constexpr int kC = HD / 16;  // output columns of a thread: tx * 4 + 64 * (c / 4) + c % 4, as pairs
  uint64_t o[kE][kC / 2] = {};
  float m[kE], l[kE] = {};
  WaRange rr[kE];
#pragma unroll
  for (int e = 0; e < kE; ++e) {
    m[e] = -INFINITY;
    rr[e] = wa_range(a, s, i0 + min(ty * kE + e, rows - 1));
  }
  int j0 = front > 0 ? 0 : begin;
  if (j0 < end) load(j0, 0);
  cp_async_commit();
  for (int buf = 0; j0 < end; buf ^= 1) {
    const int jn = behind(j0);
    __syncthreads();  // the other buffer has been read
    if (jn < end) load(jn, buf ^ 1);
    cp_async_commit();
    cp_async_wait<1>();
    __syncthreads();
    const float* ks = wf_sm + Cfg::kOffKv + buf * Cfg::kStage;
    const float* vs = ks + kWfKeys * Cfg::kPad;
    uint64_t sc2[kE][2] = {};  // sums over the even and the odd dimensions
#pragma unroll 4
    for (int d = 0; d < HD; d += 4) {
      ulonglong2 kk[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) kk[u] = *reinterpret_cast<const ulonglong2*>(ks + (tx + 16 * u) * Cfg::kPad + d);
#pragma unroll
      for (int e = 0; e < kE; ++e) {
        const ulonglong2 qq = *reinterpret_cast<const ulonglong2*>(qs + (ty * kE + e) * Cfg::kPad + d);
#pragma unroll
        for (int u = 0; u < 2; ++u) sc2[e][u] = fma2(qq.x, kk[u].x, fma2(qq.y, kk[u].y, sc2[e][u]));
      }
    }
#pragma unroll
    for (int e = 0; e < kE; ++e) {
      float mx = -INFINITY, sc[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        float even, odd;
        f32x2_parts(sc2[e][u], even, odd);
        sc[u] = wa_sees(rr[e], a.sinks, j0 + tx + 16 * u) ? (even + odd) * a.scale_log2 : -INFINITY;
        mx = fmaxf(mx, sc[u]);
      }
#pragma unroll
      for (int d = 8; d > 0; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
      const float mn = fmaxf(m[e], mx);
      const float nm = mn == -INFINITY ? 0.f : mn;
      const float alpha = m[e] == -INFINITY ? 0.f : ex2_approx(m[e] - nm);
      m[e] = mn;
      l[e] *= alpha;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const float p = ex2_approx(sc[u] - nm);
        l[e] += p;
        ps[(ty * kE + e) * Cfg::kPitchP + tx + 16 * u] = p;
      }
      const uint64_t alpha2 = f32x2(__float_as_uint(alpha), __float_as_uint(alpha));
#pragma unroll
      for (int c = 0; c < kC / 2; ++c) o[e][c] = mul2(o[e][c], alpha2);
    }
    __syncwarp();  // a row's 16 threads are half a warp
#pragma unroll 2
    for (int j = 0; j < kWfKeys; j += 4) {
      float pj[kE][4];
#pragma unroll
      for (int e = 0; e < kE; ++e)
        *reinterpret_cast<float4*>(pj[e]) = *reinterpret_cast<const float4*>(ps + (ty * kE + e) * Cfg::kPitchP + j);
#pragma unroll
      for (int jj = 0; jj < 4; ++jj) {
        uint64_t vv[kC / 2];
#pragma unroll
        for (int c = 0; c < kC / 2; c += 2)
          *reinterpret_cast<ulonglong2*>(vv + c) = *reinterpret_cast<const ulonglong2*>(vs + (j + jj) * HD + tx * 4 + 32 * c);
#pragma unroll
        for (int e = 0; e < kE; ++e) {
          const uint64_t p2 = f32x2(__float_as_uint(pj[e][jj]), __float_as_uint(pj[e][jj]));
#pragma unroll
          for (int c = 0; c < kC / 2; ++c) o[e][c] = fma2(p2, vv[c], o[e][c]);
        }
      }
    }
    j0 = jn;
  }
  cp_async_wait<0>();
  if constexpr (kSplit) {
    if (parts > 1) {
      // (m, l) and O of this part to the workspace; the last part's CTA to get here
      // joins them, in the order of the parts, and goes on with the sums
      __shared__ int join_sh;
      float* unit0 = a.partial + (int64_t)unit * a.splits * Cfg::kSlotFloats;
      float* slot = unit0 + (int64_t)part * Cfg::kSlotFloats;
#pragma unroll
      for (int e = 0; e < kE; ++e) {
        const int r = ty * kE + e;
#pragma unroll
        for (int d = 8; d > 0; d >>= 1) l[e] += __shfl_xor_sync(0xffffffffu, l[e], d);
        if (tx == 0) __stcg(reinterpret_cast<float2*>(slot) + r, make_float2(m[e], l[e]));
#pragma unroll
        for (int c = 0; c < kC / 2; c += 2)
          __stcg(reinterpret_cast<ulonglong2*>(slot + 2 * kRows + r * HD + tx * 4 + 32 * c), make_ulonglong2(o[e][c], o[e][c + 1]));
      }
      __threadfence();
      __syncthreads();
      if (tid == 0) join_sh = ticket_acq_rel(a.tickets + unit) == parts - 1;
      __syncthreads();
      if (!join_sh) return;
      if (tid == 0) a.tickets[unit] = 0;
#pragma unroll
      for (int e = 0; e < kE; ++e) {
        const int r = ty * kE + e;
        float mm = -INFINITY, ll = 0.f, acc[kC] = {};
        for (int k0 = 0; k0 < parts; k0 += 4) {
          float2 w[4];
          float4 v[4][kC / 4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            w[k] = make_float2(-INFINITY, 0.f);
#pragma unroll
            for (int c = 0; c < kC / 4; ++c) v[k][c] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (k0 + k < parts) {
              const float* from = unit0 + (int64_t)(k0 + k) * Cfg::kSlotFloats;
              w[k] = __ldcg(reinterpret_cast<const float2*>(from) + r);
#pragma unroll
              for (int c = 0; c < kC / 4; ++c)
                v[k][c] = __ldcg(reinterpret_cast<const float4*>(from + 2 * kRows + r * HD + tx * 4 + 64 * c));
            }
          }
          const float mn = fmaxf(fmaxf(mm, fmaxf(w[0].x, w[1].x)), fmaxf(w[2].x, w[3].x));
          const float f0 = mm == -INFINITY ? 0.f : ex2_approx(mm - mn);
          mm = mn;
          ll *= f0;
#pragma unroll
          for (int c = 0; c < kC; ++c) acc[c] *= f0;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float f = w[k].x == -INFINITY ? 0.f : ex2_approx(w[k].x - mn);
            ll = fmaf(f, w[k].y, ll);
#pragma unroll
            for (int c = 0; c < kC / 4; ++c) {
              acc[4 * c] = fmaf(f, v[k][c].x, acc[4 * c]);
              acc[4 * c + 1] = fmaf(f, v[k][c].y, acc[4 * c + 1]);
              acc[4 * c + 2] = fmaf(f, v[k][c].z, acc[4 * c + 2]);
              acc[4 * c + 3] = fmaf(f, v[k][c].w, acc[4 * c + 3]);
            }
          }
        }
        l[e] = tx == 0 ? ll : 0.f;
#pragma unroll
        for (int c = 0; c < kC; c += 2) o[e][c / 2] = f32x2(__float_as_uint(acc[c]), __float_as_uint(acc[c + 1]));
      }
    }
  }
  // sums over the 16 threads of a row, and whether all of it is finite
  uint32_t redo = 0;
#pragma unroll
  for (int e = 0; e < kE; ++e) {
    float sum = l[e], worst = 0.f, out[kC];
#pragma unroll
    for (int c = 0; c < kC; ++c) {
      if (c % 2 == 0) f32x2_parts(o[e][c / 2], out[c], out[c + 1]);
      worst = fmaxf(worst, fabsf(out[c]) <= 3.0e38f ? 0.f : 1.f);
    }
#pragma unroll
    for (int d = 8; d > 0; d >>= 1) {
      sum += __shfl_xor_sync(0xffffffffu, sum, d);
      worst = fmaxf(worst, __shfl_xor_sync(0xffffffffu, worst, d));
    }
    const int r = ty * kE + e;
    const bool bad = worst != 0.f && sum > 0.f;
    const uint32_t bads = __ballot_sync(0xffffffffu, bad && r < rows);
    redo |= ((bads & 0xffffu) ? 1u << e : 0u) | ((bads >> 16) ? 16u << e : 0u);
    if (r < rows) {
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
      float* to = reinterpret_cast<float*>(a.o) + (int64_t)(s.q0 + i0 + r) * a.o_stride + head * HD;
#pragma unroll
      for (int c = 0; c < kC; c += 4)
        ka_store4(to + tx * 4 + 16 * c, ka_scaled(make_float4(out[c], out[c + 1], out[c + 2], out[c + 3]), inv));
    }
  }
  __syncwarp();
  while (redo) {  // warp-uniform: bits 0-3 the rows of its lower half, 4-7 of its upper half
    const int e = __ffs(redo) - 1;
    redo &= redo - 1;
    wa_row_exact<float, HD>(a, s, i0 + ((tid >> 5) * 2 + (e >> 2)) * kE + (e & 3), head);
  }
}

}  // namespace dinfer
