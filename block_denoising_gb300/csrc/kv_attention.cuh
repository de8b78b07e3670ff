// Attention of one new token per sequence over the paged key/value cache
// (include/dinfer_kv.h, dinfer_kv_attention).
//
// For one sequence and one key/value head, `group` query heads read the same
// keys and values, all of them under the same mask (there is one position), so
// the work is a stream of visible key rows that each want 2 * group dot
// products: bound by HBM, 4 * group FLOP a byte.  The kernel is built around
// that stream:
//
//   - the visible keys of a sequence (the sinks, then the window) are numbered
//     0 .. seen - 1 and cut into units of 64; the units of all (sequence, key
//     head) pairs, end to end, are split evenly over the CTAs, whatever the
//     sequences' lengths.  A pair that several CTAs share is joined by the last
//     of them to finish, in CTA order, from fp32 partials in the workspace: one
//     launch, and the same bits every time;
//   - each of the 4 warps of a CTA takes 16 keys of a unit and streams its own
//     rows through a private ring of cp.async stages, so no barrier stands
//     between the loads and the products.  The ring runs ahead across pair
//     boundaries.  Page numbers are looked up per key (any page size, any
//     stride), one unit ahead of the copies that need them;
//   - each warp keeps an online softmax of its own (running maximum, sum and
//     output); the four meet in shared memory at the end of a pair.
//
// bf16: S = Q K^T and O += P V on mma.sync m16n8k16 with the query heads of
// the group as the 16 rows (one token has too few rows for a tcgen05 tile of
// 128, and the products are far from the bound either way).  P is rounded to
// bf16 for its product, l sums the rounded values, so O / l weights the keys
// exactly in proportion; everything else is fp32.  fp32: plain FMAs.
#pragma once
#include "attention_tc.cuh"
#include "kv_pages.cuh"

namespace dinfer {

constexpr int kKaWarps = 4;
constexpr int kKaThreads = kKaWarps * 32;
constexpr int kKaWarpKeys = 16;
constexpr int kKaUnit = kKaWarps * kKaWarpKeys;  // keys of a unit
constexpr int kKaMergeRows = 4;                  // rows merged per round

template <typename T, int HD>
struct KaCfg {
  static constexpr int kRows = sizeof(T) == 2 ? 16 : 8;       // query heads a CTA takes at once
  static constexpr int kRowBytes = HD * (int)sizeof(T);
  static constexpr int kVecs = kRowBytes / 16;                // 16-byte vectors of a head's row
  static constexpr int kStageBytes = 2 * kKaWarpKeys * kRowBytes;  // K and V rows of one warp
  static constexpr int kStages = kStageBytes >= 16384 ? 2 : (kStageBytes >= 8192 ? 3 : 6);
  static constexpr int kRing = kKaWarps * kStages * kStageBytes;
  static constexpr int kMerge = kKaWarps * kKaMergeRows * HD * 4;  // fp32 output rows of the 4 warps
  static constexpr int kOffMerge = kRing;
  static constexpr int kOffMl = kOffMerge + kMerge;            // [4 warps][rows][m, l]
  static constexpr int kOffQ = kOffMl + kKaWarps * kRows * 8;  // fp32 only: the query rows
  static constexpr int kOffCum = kOffQ + (sizeof(T) == 4 ? kRows * HD * 4 : 0);
  static constexpr int kOffMask = kOffCum + (kKvMaxEntries + 4) * 4;  // [warp][stage]: keys present
  static constexpr int kSmem = kOffMask + kKaWarps * kStages * 4;
  static constexpr int kSlotFloats = kRows * (HD + 2);         // a partial: m, l [rows], O [rows][HD]
};

struct KaArgs {
  KvPages c;
  const int32_t* seqs;
  const void* q;
  void* o;
  int64_t q_stride, o_stride, layer_off;  // elements; layer_off in 16-byte vectors
  int n, group, subgroups;                // query heads per key head; pieces of at most kRows of them
  int window, sinks, min_units;
  float scale_log2;
  float* partial;  // [CTA][2][kSlotFloats]
  int* tickets;    // [CTA], zero between calls
};

// Visible keys of a sequence of `len` tokens: the first `sink` ones, then
// those from `first` on.
struct KaSeen {
  int sink, first, seen;
};
__device__ __forceinline__ KaSeen ka_seen(int len, int window, int sinks) {
  KaSeen r;
  r.first = window < 0 ? 0 : max(0, len - 1 - window);
  r.sink = min(sinks, r.first);
  r.seen = max(0, len - r.first + r.sink);
  return r;
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldmatrix_x4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// D (16 x 8 fp32) += A (16 x 16 bf16) B (16 x 8 bf16)
__device__ __forceinline__ void mma_m16n8k16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The units of the call, walked in order: entry (sequence of the call), head
// piece, unit of that pair.
struct KaWalk {
  int entry, piece, unit, units;  // units: of this entry
  __device__ void start(int u, const int* cum, int n, int pieces) {
    int lo = 0, hi = n;  // cum[lo] * pieces <= u < cum[hi] * pieces
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (cum[mid] * pieces <= u) lo = mid; else hi = mid;
    }
    entry = lo;
    units = cum[lo + 1] - cum[lo];
    const int r = u - cum[lo] * pieces;
    piece = r / units;
    unit = r - piece * units;
  }
  __device__ void next(const int* cum, int n, int pieces) {
    if (++unit < units) return;
    unit = 0;
    if (++piece < pieces) return;
    piece = 0;
    do {
      ++entry;
      if (entry >= n) return;
      units = cum[entry + 1] - cum[entry];
    } while (units == 0);
  }
};

// ---------------------------------------------------------------------------
// a warp's running state over its keys of one (sequence, head piece)
// ---------------------------------------------------------------------------
// Both forms offer reset(), a step over one ring stage, and store(row0, ...)
// of kKaMergeRows output rows and of (m, l).

// bf16.  Fragments of mma.m16n8k16: lane = 4 g + t holds rows g and g + 8.
template <int HD>
struct KaStateBf16 {
  static constexpr int kKs = HD / 16, kNt = HD / 8;
  uint32_t q[kKs][4];
  float o[kNt][4];
  float m[2], l[2];

  __device__ void reset(const __nv_bfloat16* qrow, int rows, int lane, float*) {
    // A fragment: a0 (g, 2t), a1 (g + 8, 2t), a2 (g, 2t + 8), a3 (g + 8, 2t + 8); absent heads are zeros
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int ks = 0; ks < kKs; ++ks)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int row = g + (e & 1) * 8, col = ks * 16 + 2 * t + (e >> 1) * 8;
        q[ks][e] = row < rows ? *reinterpret_cast<const uint32_t*>(qrow + row * HD + col) : 0u;
      }
#pragma unroll
    for (int i = 0; i < kNt; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
    m[0] = m[1] = -INFINITY;
    l[0] = l[1] = 0.f;
  }

  // stage: K rows [16][HD], V rows [16][HD], 16-byte vector x of row r at x ^ (r & 7); mask: bit r = key r is there
  __device__ void step(uint32_t stage, uint32_t mask, float sc, int lane, const float*) {
    constexpr int kRowBytes = HD * 2;
    const int mi = lane >> 3, r8 = lane & 7;
    float s[2][4] = {};
    {
      const int row = (mi >> 1) * 8 + r8;
      const uint32_t base = stage + row * kRowBytes;
#pragma unroll
      for (int ks = 0; ks < kKs; ++ks) {
        uint32_t b[4];
        ldmatrix_x4(base + (((ks * 2 + (mi & 1)) ^ r8) << 4), b);
        mma_m16n8k16(s[0], q[ks], b[0], b[1]);
        mma_m16n8k16(s[1], q[ks], b[2], b[3]);
      }
    }
    const int t2 = (lane & 3) * 2;
#pragma unroll
    for (int nt = 0; nt < 2; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        s[nt][e] = (mask >> (nt * 8 + t2 + (e & 1))) & 1u ? s[nt][e] * sc : -INFINITY;
    uint32_t p[4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {  // rows g, g + 8
      float mx = fmaxf(fmaxf(s[0][2 * h], s[0][2 * h + 1]), fmaxf(s[1][2 * h], s[1][2 * h + 1]));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      const float mn = fmaxf(m[h], mx);
      const float nm = mn == -INFINITY ? 0.f : mn;  // nothing seen yet: every weight is 2^-inf = 0
      const float alpha = m[h] == -INFINITY ? 0.f : ex2_approx(m[h] - nm);
      m[h] = mn;
      const uint32_t p0 = pack_bf16x2(ex2_approx(s[0][2 * h] - nm), ex2_approx(s[0][2 * h + 1] - nm));
      const uint32_t p1 = pack_bf16x2(ex2_approx(s[1][2 * h] - nm), ex2_approx(s[1][2 * h + 1] - nm));
      p[h] = p0;      // a0 / a1: keys 2t, 2t + 1
      p[2 + h] = p1;  // a2 / a3: keys 2t + 8, 2t + 9
      // this lane's four keys; the lanes of a row are summed at the end
      l[h] = l[h] * alpha + (__uint_as_float(p0 << 16) + __uint_as_float(p0 & 0xffff0000u)) +
             (__uint_as_float(p1 << 16) + __uint_as_float(p1 & 0xffff0000u));
#pragma unroll
      for (int i = 0; i < kNt; ++i) {
        o[i][2 * h] *= alpha;
        o[i][2 * h + 1] *= alpha;
      }
    }
    const uint32_t vbase = stage + kKaWarpKeys * kRowBytes + ((mi & 1) * 8 + r8) * kRowBytes;
#pragma unroll
    for (int i = 0; i < kNt; i += 2) {
      uint32_t b[4];
      ldmatrix_x4_trans(vbase + (((i + (mi >> 1)) ^ r8) << 4), b);
      mma_m16n8k16(o[i], p, b[0], b[1]);
      mma_m16n8k16(o[i + 1], p, b[2], b[3]);
    }
  }

  __device__ void store_ml(float* ml, int lane) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float s = l[h];
      s += __shfl_xor_sync(0xffffffffu, s, 1);
      s += __shfl_xor_sync(0xffffffffu, s, 2);
      if ((lane & 3) == 0) {
        ml[((lane >> 2) + 8 * h) * 2] = m[h];
        ml[((lane >> 2) + 8 * h) * 2 + 1] = s;
      }
    }
  }
  __device__ void store_rows(float* buf, int row0, int lane) {
    const int g = lane >> 2, t2 = (lane & 3) * 2;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int row = g + 8 * h - row0;
      if (row >= 0 && row < kKaMergeRows)
#pragma unroll
        for (int i = 0; i < kNt; ++i)
          *reinterpret_cast<float2*>(buf + row * HD + i * 8 + t2) = make_float2(o[i][2 * h], o[i][2 * h + 1]);
    }
  }
};

// fp32.  For the scores lane = 16 half + key takes half of the head's
// dimensions of one key; for the output a lane owns HD / 32 dimensions.
template <int HD>
struct KaStateF32 {
  static constexpr int kRows = 8, kOut = HD / 32;
  float o[kRows][kOut];
  float m[kRows], l[kRows];

  __device__ void reset(const float* qrow, int rows, int lane, float* qs) {
    // every warp writes the same values: no barrier between the warps is needed for its own reads
    for (int x = lane; x < kRows * HD; x += 32) qs[x] = x < rows * HD ? qrow[x] : 0.f;
    __syncwarp();
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      m[r] = -INFINITY;
      l[r] = 0.f;
#pragma unroll
      for (int e = 0; e < kOut; ++e) o[r][e] = 0.f;
    }
  }

  __device__ void step(const uint8_t* stage, uint32_t mask, float sc, int lane, const float* qs) {
    constexpr int kRowBytes = HD * 4;
    const int key = lane & 15, half = lane >> 4;
    float s[kRows] = {};
    const uint8_t* krow = stage + key * kRowBytes;
#pragma unroll 4
    for (int x = 0; x < HD / 8; ++x) {
      const int vec = half * (HD / 8) + x;
      const float4 kk = *reinterpret_cast<const float4*>(krow + ((vec ^ (key & 7)) << 4));
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        const float4 qq = *reinterpret_cast<const float4*>(qs + r * HD + vec * 4);
        s[r] = fmaf(qq.x, kk.x, fmaf(qq.y, kk.y, fmaf(qq.z, kk.z, fmaf(qq.w, kk.w, s[r]))));
      }
    }
    const bool there = (mask >> key) & 1u;
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      float v = (s[r] + __shfl_xor_sync(0xffffffffu, s[r], 16)) * sc;
      if (!there) v = -INFINITY;
      float mx = v;
#pragma unroll
      for (int d = 8; d > 0; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
      const float mn = fmaxf(m[r], mx);
      const float nm = mn == -INFINITY ? 0.f : mn;
      const float alpha = m[r] == -INFINITY ? 0.f : ex2_approx(m[r] - nm);
      m[r] = mn;
      s[r] = ex2_approx(v - nm);
      l[r] = l[r] * alpha + (half ? 0.f : s[r]);
#pragma unroll
      for (int e = 0; e < kOut; ++e) o[r][e] *= alpha;
    }
    const uint8_t* vrows = stage + kKaWarpKeys * kRowBytes;
#pragma unroll 4
    for (int k = 0; k < kKaWarpKeys; ++k) {
      const int byte = lane * kOut * 4, vec = byte >> 4;
      const float* vp = reinterpret_cast<const float*>(vrows + k * kRowBytes + ((vec ^ (k & 7)) << 4) + (byte & 15));
      float vv[kOut];
#pragma unroll
      for (int e = 0; e < kOut; ++e) vv[e] = vp[e];
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        const float p = __shfl_sync(0xffffffffu, s[r], k);
#pragma unroll
        for (int e = 0; e < kOut; ++e) o[r][e] = fmaf(p, vv[e], o[r][e]);
      }
    }
  }

  __device__ void store_ml(float* ml, int lane) {
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      const float s = warp_sum(l[r]);
      if (lane == 0) {
        ml[r * 2] = m[r];
        ml[r * 2 + 1] = s;
      }
    }
  }
  __device__ void store_rows(float* buf, int row0, int lane) {
#pragma unroll
    for (int r = 0; r < kRows; ++r)
      if (r >= row0 && r < row0 + kKaMergeRows)
#pragma unroll
        for (int e = 0; e < kOut; ++e) buf[(r - row0) * HD + lane * kOut + e] = o[r][e];
  }
};

template <typename T, int HD>
struct KaState;
template <int HD>
struct KaState<__nv_bfloat16, HD> : KaStateBf16<HD> {};
template <int HD>
struct KaState<float, HD> : KaStateF32<HD> {};

__device__ __forceinline__ void ka_store4(__nv_bfloat16* p, float4 v) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
}
__device__ __forceinline__ void ka_store4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }

template <typename T, int HD>
__global__ void __launch_bounds__(kKaThreads) kv_attention_kernel(const KaArgs a) {
  using Cfg = KaCfg<T, HD>;
  constexpr int kRows = Cfg::kRows, kStages = Cfg::kStages;
  extern __shared__ __align__(128) uint8_t sm[];
  int* cum = reinterpret_cast<int*>(sm + Cfg::kOffCum);  // units before each entry, for one head piece
  float* merge = reinterpret_cast<float*>(sm + Cfg::kOffMerge);
  float* ml = reinterpret_cast<float*>(sm + Cfg::kOffMl);
  float* qs = reinterpret_cast<float*>(sm + Cfg::kOffQ);
  __shared__ int warp_units[kKaWarps], join_sh;
  const KvPages& c = a.c;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int pieces = c.kv_heads * a.subgroups;
  pdl_wait();

  auto seq_of = [&](int e) { return a.seqs ? a.seqs[e] : e; };
  auto len_of = [&](int e) {
    const int s = seq_of(e);
    if (s < 0 || s >= c.max_seqs) return 0;
    const int len = c.lens[s];
    return c.valid_len(len) ? len : 0;
  };
  // units before each entry: thread i sums the entries of its own stretch
  {
    const int per = (a.n + kKaThreads - 1) / kKaThreads;
    const int e0 = min(a.n, tid * per), e1 = min(a.n, e0 + per);
    int sum = 0;
    for (int e = e0; e < e1; ++e) {
      const int u = (ka_seen(len_of(e), a.window, a.sinks).seen + kKaUnit - 1) / kKaUnit;
      cum[e + 1] = u;
      sum += u;
      if (blockIdx.x == 0) {
        const int s = seq_of(e);
        if (s < 0 || s >= c.max_seqs || !c.valid_len(c.lens[s])) c.flag(KV_BAD_SEQ);
      }
    }
    int inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += u;
    }
    if (lane == 31) warp_units[warp] = inc;
    __syncthreads();
    int run = inc - sum;
    for (int w = 0; w < warp; ++w) run += warp_units[w];
    if (tid == 0) cum[0] = 0;
    for (int e = e0; e < e1; ++e) {
      run += cum[e + 1];
      cum[e + 1] = run;
    }
    __syncthreads();
  }
  // entries without a key: zeros, the entries dealt round the CTAs
  for (int e = blockIdx.x; e < a.n; e += gridDim.x) {
    if (cum[e + 1] != cum[e]) continue;
    T* orow = reinterpret_cast<T*>(a.o) + e * a.o_stride;
    const int vecs = c.kv_heads * a.group * Cfg::kVecs;
    for (int x = tid; x < vecs; x += kKaThreads) reinterpret_cast<uint4*>(orow)[x] = make_uint4(0, 0, 0, 0);
  }
  // units of the call (the host bounds them below 2^31) and the CTAs that
  // take them: at least min_units each, so that none is without
  const int64_t total = (int64_t)cum[a.n] * pieces;
  const int64_t G = min((int64_t)gridDim.x, max((int64_t)1, total / a.min_units));
  if (total == 0 || blockIdx.x >= G) return;
  const int64_t u0 = total * blockIdx.x / G, u1 = total * (blockIdx.x + 1) / G;
  const int count = (int)(u1 - u0);

  uint8_t* ring = sm + warp * (kStages * Cfg::kStageBytes);
  const uint32_t ring_u32 = smem_u32(ring);
  uint32_t* masks = reinterpret_cast<uint32_t*>(sm + Cfg::kOffMask) + warp * kStages;
  KaWalk load, use;
  load.start((int)u0, cum, a.n, pieces);
  use = load;
  int load_entry = -1, load_seq = 0;
  KaSeen seen{};
  // the address of key `lane & 15` of the unit at `load`, in 16-byte vectors of
  // the layer, or -1 (no such key); kept one unit ahead of its copies
  auto look_up = [&]() -> int64_t {
    if (load.entry != load_entry) {
      load_entry = load.entry;
      load_seq = seq_of(load_entry);
      seen = ka_seen(c.lens[load_seq], a.window, a.sinks);
    }
    const int x = load.unit * kKaUnit + warp * kKaWarpKeys + (lane & 15);
    if (x >= seen.seen) return -1;
    const int key = x < seen.sink ? x : x - seen.sink + seen.first;
    const int j = (int)c.page_div.div((uint32_t)key);
    const int page = c.table[(size_t)load_seq * c.max_pages + j];
    if (page < 0 || page >= c.num_pages) {
      c.flag(KV_BAD_PAGE);
      return -1;
    }
    return a.layer_off + page * c.page_stride + (key - j * c.page_size) * c.token_stride +
           (load.piece / a.subgroups) * c.head_stride;
  };
  int64_t at = look_up();
  int issued = 0;
  auto issue = [&](int stage) {
    if (issued < count) {
      const uint32_t mask = __ballot_sync(0xffffffffu, at >= 0) & 0xffffu;
      if (lane == 0) masks[stage] = mask;
      constexpr int kPer = 32 / Cfg::kVecs > 0 ? 32 / Cfg::kVecs : 1;  // rows an instruction covers
      const int x = lane % Cfg::kVecs;
#pragma unroll
      for (int r0 = 0; r0 < kKaWarpKeys; r0 += kPer) {
        const int r = r0 + lane / Cfg::kVecs;
        const int64_t off = __shfl_sync(0xffffffffu, at, r);
        const int bytes = off >= 0 ? 16 : 0;  // an absent key's row is zeros
        const int64_t v = off >= 0 ? off + x : 0;
        const uint32_t d = ring_u32 + stage * Cfg::kStageBytes + r * Cfg::kRowBytes + ((x ^ (r & 7)) << 4);
        cp_async16(d, c.k + v, bytes);
        cp_async16(d + kKaWarpKeys * Cfg::kRowBytes, c.v + v, bytes);
      }
      ++issued;
      if (issued < count) {
        load.next(cum, a.n, pieces);
        at = look_up();
      }
    }
    cp_async_commit();
  };
  for (int s = 0; s < kStages - 1; ++s) issue(s);

  KaState<T, HD> state;
  int done = 0, stage = 0, seg_unit = use.unit;  // the pair's first unit in this CTA
  while (done < count) {
    if (done == 0 || use.unit == 0) {
      const int sub = use.piece % a.subgroups, rows = min(kRows, a.group - sub * kRows);
      const int head = (use.piece / a.subgroups) * a.group + sub * kRows;
      state.reset(reinterpret_cast<const T*>(a.q) + use.entry * a.q_stride + head * HD, rows, lane, qs);
      seg_unit = use.unit;
    }
    issue(stage == 0 ? kStages - 1 : stage - 1);
    cp_async_wait<kStages - 1>();
    __syncwarp();
    if constexpr (sizeof(T) == 2)
      state.step(ring_u32 + stage * Cfg::kStageBytes, masks[stage], a.scale_log2, lane, qs);
    else
      state.step(ring + stage * Cfg::kStageBytes, masks[stage], a.scale_log2, lane, qs);
    __syncwarp();  // the stage is refilled next turn
    stage = stage + 1 == kStages ? 0 : stage + 1;
    ++done;
    const int seg_end = use.unit + 1;
    const bool last_unit = seg_end == use.units;
    if (last_unit || done == count) {
      // the pair's keys of this CTA are done: merge the four warps
      const int sub = use.piece % a.subgroups, rows = min(kRows, a.group - sub * kRows);
      const int head = (use.piece / a.subgroups) * a.group + sub * kRows;
      const bool whole = last_unit && seg_unit == 0;
      const int slot = seg_unit == 0 ? 1 : 0;  // 0: the pair began in an earlier CTA
      float* part = a.partial + ((int64_t)blockIdx.x * 2 + slot) * Cfg::kSlotFloats;
      state.store_ml(ml + warp * kRows * 2, lane);
      T* orow = reinterpret_cast<T*>(a.o) + use.entry * a.o_stride + head * HD;
      for (int r0 = 0; r0 < rows; r0 += kKaMergeRows) {
        state.store_rows(merge + warp * (kKaMergeRows * HD), r0, lane);
        __syncthreads();
        for (int x = tid; x < kKaMergeRows * HD / 4; x += kKaThreads) {
          const int row = r0 + x / (HD / 4), c4 = (x % (HD / 4)) * 4;
          if (row < rows) {
            float mm = -INFINITY;
#pragma unroll
            for (int w = 0; w < kKaWarps; ++w) mm = fmaxf(mm, ml[(w * kRows + row) * 2]);
            float ll = 0.f;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kKaWarps; ++w) {
              const float mw = ml[(w * kRows + row) * 2];
              const float f = mw == -INFINITY ? 0.f : ex2_approx(mw - mm);
              const float4 v =
                  *reinterpret_cast<const float4*>(merge + w * (kKaMergeRows * HD) + (row - r0) * HD + c4);
              ll = fmaf(f, ml[(w * kRows + row) * 2 + 1], ll);
              acc.x = fmaf(f, v.x, acc.x);
              acc.y = fmaf(f, v.y, acc.y);
              acc.z = fmaf(f, v.z, acc.z);
              acc.w = fmaf(f, v.w, acc.w);
            }
            if (whole) {
              const float inv = ll == 0.f ? 0.f : 1.f / ll;
              ka_store4(orow + row * HD + c4, make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv));
            } else {
              __stcg(reinterpret_cast<float4*>(part + kRows * 2 + row * HD + c4), acc);
              if (c4 == 0) __stcg(reinterpret_cast<float2*>(part + row * 2), make_float2(mm, ll));
            }
          }
        }
        __syncthreads();
      }
      if (!whole) {
        // units of the pair, and the CTAs that share it
        const int64_t pair0 = (int64_t)cum[use.entry] * pieces + (int64_t)use.piece * use.units;
        const int64_t pair1 = pair0 + use.units;
        const int c_first = (int)(((pair0 + 1) * G - 1) / total), c_last = (int)((pair1 * G - 1) / total);
        __threadfence();
        __syncthreads();
        if (tid == 0) join_sh = atomicAdd(a.tickets + c_first, 1) == c_last - c_first;
        __syncthreads();
        if (join_sh) {
          __threadfence();
          const int nc = c_last - c_first + 1;
          auto slot_of = [&](int k) {
            return a.partial + ((int64_t)(c_first + k) * 2 + (k == 0 ? 1 : 0)) * Cfg::kSlotFloats;
          };
          for (int x = tid; x < rows * HD / 4; x += kKaThreads) {
            const int row = x / (HD / 4), c4 = (x % (HD / 4)) * 4;
            float mm = -INFINITY;
#pragma unroll 4
            for (int k = 0; k < nc; ++k) mm = fmaxf(mm, __ldcg(slot_of(k) + row * 2));
            float ll = 0.f;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
            for (int k = 0; k < nc; ++k) {
              const float* p = slot_of(k);
              const float2 w = __ldcg(reinterpret_cast<const float2*>(p + row * 2));
              const float4 v = __ldcg(reinterpret_cast<const float4*>(p + kRows * 2 + row * HD + c4));
              const float f = w.x == -INFINITY ? 0.f : ex2_approx(w.x - mm);
              ll = fmaf(f, w.y, ll);
              acc.x = fmaf(f, v.x, acc.x);
              acc.y = fmaf(f, v.y, acc.y);
              acc.z = fmaf(f, v.z, acc.z);
              acc.w = fmaf(f, v.w, acc.w);
            }
            const float inv = ll == 0.f ? 0.f : 1.f / ll;
            ka_store4(orow + row * HD + c4, make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv));
          }
          if (tid == 0) a.tickets[c_first] = 0;
        }
      }
    }
    use.next(cum, a.n, pieces);
  }
  cp_async_wait<0>();
}

}  // namespace dinfer
