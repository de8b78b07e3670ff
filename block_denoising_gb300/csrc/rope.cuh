// Rotary positions (include/dinfer_ops.h, dinfer_op_rope), and rows of a prompt
// or a token step rotated on their way to the paged cache (include/dinfer_kv.h,
// dinfer_kv_append_rope).
//
// A pair (a, b) of a head at position p becomes (a cos - b sin, a sin + b cos)
// of the angle p f: some 6 FLOP for 8 bytes of bf16, so bound by HBM, or for a
// token step by the launch.
//
// The angle.  f is kept in turns, as 64 bits behind the point: p f modulo one
// turn is then the low half of an integer product, off by p 2^-53 f at most,
// whatever p (an fp32 product at position 10^6 is off by 0.06 radians).  The
// turn's top two bits are the quadrant; the rest, within an eighth of a turn of
// its middle, goes to sincospif as a float, so the angle is rounded by 2^-25 of
// at most pi / 4.
//
// The cosines of a row are the same for all its heads: a block computes those of
// its rows into shared memory, one pair a thread, and then streams the heads.  They
// lie there in the order in which the threads of a head read them: those of the first
// pair of every work item, then of the second (pair by pair, 64 bytes apart, four
// threads met in a bank: 8704 rows of 32 heads of 128 31 us).  Those rows, 143 MB, take
// 25.0 us (5.7 TB/s); appended with their queries, 214 MB, 41.2 us (5.2 TB/s).
#pragma once
#include "attention_tc.cuh"
#include "kv_pages.cuh"

namespace dinfer {

constexpr int kRopeThreads = 256;
constexpr int kRopePairs = 128;   // of a head of at most 256
constexpr int kRopeRows = 4;      // rows of a block at a time, at most: a warp each looks its place up

struct RopeTurns {
  uint64_t f[kRopePairs];  // turns per position, 2^-64ths
  float magnitude;
  int pairs;  // rot_dim / 2
};

// One operand whose heads are rotated (q, k) or copied (v).
struct RopeRows {
  const void* from;
  void* to;
  int64_t from_stride, to_stride;  // elements
  int heads;
};

struct RopeArgs {
  RopeRows x[3];       // op_rope: x alone; append: q (heads 0: none), k, v
  const int32_t* positions;  // NULL: first + row, or the token's place
  int first, rows, head_dim;
  int chunk, parts;          // rows of a block at a time; blocks that share them
  FastDiv head_items, copies;  // work items of a rotated head, of a copied one: two of its 16-byte vectors
  FastDiv row_items;         // of a row, all operands
  int rot_items;             // of head_items, those that are rotated
  bool in_place;             // x[0].to is x[0].from: what is not rotated stays
  // append
  KvPages c;
  const int32_t* seqs;
  const int32_t* bounds;
  int n;
};

// cos and sin of p * f turns
__device__ __forceinline__ float2 rope_turn(int p, uint64_t f, float magnitude) {
  const uint32_t turn = (uint32_t)(((uint64_t)(int64_t)p * f) >> 32);
  const uint32_t quadrant = (turn + 0x20000000u) >> 30;
  float s, c;
  sincospif((float)(int32_t)(turn - (quadrant << 30)) * 0x1p-31f, &s, &c);
  s *= magnitude;
  c *= magnitude;
  if (quadrant & 1) {
    const float t = c;
    c = -s;
    s = t;
  }
  return (quadrant & 2) ? make_float2(-c, -s) : make_float2(c, s);
}

// V elements as floats, and back: 16 bytes, or one element
template <typename T, int V>
struct RopeVec;
template <>
struct RopeVec<float, 4> {
  uint4 d;
  __device__ __forceinline__ float get(int e) const { return __uint_as_float((&d.x)[e]); }
  __device__ __forceinline__ void set2(int e, float a, float b) {
    (&d.x)[e] = __float_as_uint(a);
    (&d.x)[e + 1] = __float_as_uint(b);
  }
};
template <>
struct RopeVec<__nv_bfloat16, 8> {
  uint4 d;
  __device__ __forceinline__ float get(int e) const {
    const uint32_t w = (&d.x)[e >> 1];
    return __uint_as_float((e & 1) ? w & 0xffff0000u : w << 16);
  }
  __device__ __forceinline__ void set2(int e, float a, float b) { (&d.x)[e >> 1] = pack_bf16x2(a, b); }
};
template <typename Vec>
__device__ __forceinline__ Vec rope_load(const void* p) {
  Vec v;
  if constexpr (sizeof(Vec) == 16) v.d = __ldcs(reinterpret_cast<const uint4*>(p)); else v = *reinterpret_cast<const Vec*>(p);
  return v;
}
template <typename T>
struct RopeVec<T, 1> {
  T d;
  __device__ __forceinline__ float get(int) const { return (float)d; }
  __device__ __forceinline__ void set(float a) { d = (T)a; }
};

// kPairs: (2 i, 2 i + 1), else (i, i + pairs).  V: elements of a work item's vector, 16
// bytes, or 1 where the rotated part is not made of such vectors.  An item has a
// second vector, its pairs' other halves, unless neighbours are paired within one.
template <typename T, bool kPairs, int V, bool kPlace>
__global__ void __launch_bounds__(kRopeThreads, 4) rope_kernel(const __grid_constant__ RopeArgs a, const __grid_constant__ RopeTurns turns) {
  using Vec = RopeVec<T, V>;
  constexpr int kFull = 16 / (int)sizeof(T), kU = V > 1 && !kPlace ? 4 : 2;
  constexpr bool kTwo = !kPairs || V == 1;
  constexpr int kEach = V == 1 ? 1 : kPairs ? V / 2 : V;  // pairs of an item
  __shared__ float2 cs[kRopeRows * kRopePairs];
  __shared__ int64_t place[kRopeRows];  // append: where the row lies in the cache, or -1
  __shared__ int where[kRopeRows];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_wait();
  pdl_trigger();
  const int last = kPlace && a.bounds ? min(a.rows, a.bounds[a.n]) : a.rows;
  const int units = (last + a.chunk - 1) / a.chunk * a.parts;
  for (int unit = blockIdx.x; unit < units; unit += gridDim.x) {
    const int row0 = unit / a.parts * a.chunk, part = unit % a.parts, rows = min(a.chunk, last - row0);
    if (kPlace) {
      if (warp < rows) {
        int p = 0;
        const int64_t at = kv_row_place(a.c, a.seqs, a.bounds, a.n, row0 + warp, &p);
        if (lane == 0) {
          place[warp] = at;
          where[warp] = a.positions ? a.positions[row0 + warp] : p;
        }
      }
    } else if (tid < rows) {
      where[tid] = a.positions ? a.positions[row0 + tid] : a.first + row0 + tid;
    }
    __syncthreads();
    for (int i = tid; i < rows * turns.pairs; i += kRopeThreads) {
      const int r = i / turns.pairs;
      const int p = i - r * turns.pairs;
      cs[r * turns.pairs + p % kEach * a.rot_items + p / kEach] = rope_turn(where[r], turns.f[p], turns.magnitude);
    }
    __syncthreads();
    const int all = rows * (int)a.row_items.d;
    for (int i0 = part * kRopeThreads + tid; i0 < all; i0 += a.parts * kRopeThreads * kU) {
      Vec lo[kU], hi[kU];
      uint4 copy[kU][2];
      T* to[kU];
      int kind[kU], pair[kU];  // 0: nothing, 1: rotated, 2: one vector as it is, 3: two vectors of 16 bytes as they are
#pragma unroll
      for (int u = 0; u < kU; ++u) {  // all loads before the first store
        const int i = i0 + u * a.parts * kRopeThreads;
        kind[u] = 0;
        if (i >= all) continue;
        const int r = (int)a.row_items.div((uint32_t)i), row = row0 + r;
        if (kPlace && place[r] < 0) continue;
        int x = i - r * (int)a.row_items.d, op = 0;
        const int nq = a.x[0].heads * (int)a.head_items.d;
        if (kPlace && x >= nq) {
          x -= nq;
          op = 1;
          if (x >= a.x[1].heads * (int)a.head_items.d) {
            x -= a.x[1].heads * (int)a.head_items.d;
            op = 2;
          }
        }
        const RopeRows& o = a.x[op];
        const T* from = reinterpret_cast<const T*>(o.from) + row * o.from_stride;
        T* dst = kPlace && op ? reinterpret_cast<T*>(reinterpret_cast<uint4*>(o.to) + place[r]) : reinterpret_cast<T*>(o.to) + row * o.to_stride;
        const int64_t step = kPlace && op ? a.c.head_stride * kFull : a.head_dim;
        if (kPlace && op == 2) {
          const int h = (int)a.copies.div((uint32_t)x), v = x - h * (int)a.copies.d;
          const uint4* row_v = reinterpret_cast<const uint4*>(from + h * a.head_dim) + v;
          copy[u][0] = __ldcs(row_v);
          copy[u][1] = __ldcs(row_v + a.copies.d);
          to[u] = dst + h * step + v * kFull;
          kind[u] = 3;
          continue;
        }
        const int h = (int)a.head_items.div((uint32_t)x), v = x - h * (int)a.head_items.d;
        from += h * a.head_dim;
        dst += h * step;
        if (v < a.rot_items) {
          const int e = kPairs && V == 1 ? 2 * v : v * V;
          pair[u] = r * turns.pairs + v;
          lo[u] = rope_load<Vec>(from + e);
          if constexpr (kTwo) hi[u] = rope_load<Vec>(from + e + (kPairs ? 1 : turns.pairs));
          to[u] = dst + e;
          kind[u] = 1;
        } else if (op || !a.in_place) {
          const int e = 2 * turns.pairs + (v - a.rot_items) * V;
          lo[u] = rope_load<Vec>(from + e);
          to[u] = dst + e;
          kind[u] = 2;
        }
      }
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        if (kind[u] == 1) {
          if constexpr (V == 1) {
            const float2 t = cs[pair[u]];
            const float x = lo[u].get(0), y = hi[u].get(0);
            lo[u].set(fmaf(x, t.x, -y * t.y));
            hi[u].set(fmaf(x, t.y, y * t.x));
          } else if constexpr (kPairs) {
#pragma unroll
            for (int e = 0; e < V; e += 2) {
              const float2 t = cs[pair[u] + e / 2 * a.rot_items];
              const float x = lo[u].get(e), y = lo[u].get(e + 1);
              lo[u].set2(e, fmaf(x, t.x, -y * t.y), fmaf(x, t.y, y * t.x));
            }
          } else {
#pragma unroll
            for (int e = 0; e < V; e += 2) {
              const float2 t0 = cs[pair[u] + e * a.rot_items], t1 = cs[pair[u] + (e + 1) * a.rot_items];
              const float x0 = lo[u].get(e), y0 = hi[u].get(e), x1 = lo[u].get(e + 1), y1 = hi[u].get(e + 1);
              lo[u].set2(e, fmaf(x0, t0.x, -y0 * t0.y), fmaf(x1, t1.x, -y1 * t1.y));
              hi[u].set2(e, fmaf(x0, t0.y, y0 * t0.x), fmaf(x1, t1.y, y1 * t1.x));
            }
          }
          *reinterpret_cast<Vec*>(to[u]) = lo[u];
          if constexpr (kTwo) *reinterpret_cast<Vec*>(to[u] + (kPairs ? 1 : turns.pairs)) = hi[u];
        } else if (kind[u] == 2) {
          *reinterpret_cast<Vec*>(to[u]) = lo[u];
        } else if (kPlace && kind[u] == 3) {
          *reinterpret_cast<uint4*>(to[u]) = copy[u][0];
          reinterpret_cast<uint4*>(to[u])[a.copies.d] = copy[u][1];
        }
      }
    }
    __syncthreads();  // cs is written again
  }
  if (kPlace && a.bounds && blockIdx.x == 0) kv_check_bounds(a.c, a.bounds, a.n, a.rows);
}

}  // namespace dinfer
