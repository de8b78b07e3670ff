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
//     0 .. seen - 1 and cut into steps of kKeys keys; the steps of all (sequence,
//     key head) pairs, end to end, are split evenly over the CTAs,
//     whatever the sequences' lengths.  A pair that several CTAs share is joined
//     by the last of them to finish, in CTA order, from fp32 partials in the
//     workspace: one launch, and the same bits every time.  The split counts a
//     pair as kPairCost steps more than its keys, about what its beginning and
//     its merge take: without it the CTAs that got many short sequences ran
//     twice as long as the others (64 sequences of 1 .. 8192 tokens);
//   - each warp streams its own keys' rows through a private ring of cp.async
//     stages, so no barrier stands between the loads and the products.  The ring
//     runs ahead across pair boundaries.  Page numbers are looked up per key (any
//     page size, any stride), two rounds ahead of the copies that need them;
//   - each warp keeps an online softmax of its own (running maximum, sum and
//     output); they meet in shared memory at the end of a pair;
//   - groups of more than 16 heads (fp32: 8) are cut into pieces, each of which
//     reads the keys again (64 sequences of 2048 tokens, 256 heads on 8 of 128: 196 us,
//     32 heads on 8 99 us).
//
// bf16: S = Q K^T and O += P V on mma.sync m16n8k16 with the query heads of
// the group as the 16 rows (one token has too few rows for a tcgen05 tile of
// 128, and the products are far from the bound either way).  P goes through its
// product as two bf16 (the number below it cut off, and the rounded rest, 16 bits together):
// the products have the room, and the output's own rounding is then all that is
// left.  Everything else is fp32.  fp32: plain FMAs.
#pragma once
#include "attention_tc.cuh"
#include "kv_pages.cuh"

namespace dinfer {

constexpr int kKaJoin = 16;      // partials read at once by a join
constexpr int kKaPairCost = 3;   // a pair's beginning and merge, in steps

template <typename T, int HD, int R>  // R: query heads a CTA takes at once
struct KaCfg {
  static constexpr int kKeys = sizeof(T) == 2 ? 32 : 16;      // keys of a warp's step
  // a step of 16 KB hides its own latencies; steps of 8 KB want a second warp a scheduler (16 sequences that see
  // 4100 tokens, 64 heads of 64 on 8: 29 us with 8 warps, 36 with 4)
  static constexpr int kWarps = HD == 64 ? 8 : 4;
  static constexpr int kThreads = kWarps * 32;
  static constexpr int kRows = R;
  static constexpr int kRowBytes = HD * (int)sizeof(T);
  static constexpr int kVecs = kRowBytes / 16;                // 16-byte vectors of a head's row
  static constexpr int kStageBytes = 2 * kKeys * kRowBytes;   // K and V rows of one step: 8 or 16 KB
  static constexpr int kStages = 3;
  static constexpr int kRing = kWarps * kStages * kStageBytes;   // 192 KB: one CTA an SM
  static constexpr int kMergeRows = R < 4 ? R : 4;             // rows merged per round
  static constexpr int kMerge = kWarps * kMergeRows * HD * 4;  // fp32 output rows of the warps
  static constexpr int kOffMerge = kRing;
  static constexpr int kOffMl = kOffMerge + kMerge;            // [warps][rows][m, l]
  static constexpr int kOffQ = kOffMl + kWarps * kRows * 8;  // fp32 only: the query rows
  static constexpr int kOffCum = kOffQ + (sizeof(T) == 4 ? kRows * HD * 4 : 0);
  static constexpr int kOffLen = kOffCum + (kKvMaxEntries + 4) * 4;
  static constexpr int kOffMask = kOffLen + kKvMaxEntries * 4;  // [warp][stage]: keys present
  static constexpr int kSmem = kOffMask + kWarps * kStages * 4;
  // a partial in the workspace: (m, l) [rows], padded so that O [rows][HD] begins at 16 bytes
  static constexpr int kSlotO = (2 * R + 3) / 4 * 4;
  static constexpr int kSlotFloats = kSlotO + R * HD;
  static_assert(kSlotO % 4 == 0 && kSlotFloats % 4 == 0, "16-byte accesses to the partials");
  static_assert(kOffMerge % 16 == 0 && kOffMl % 16 == 0 && kOffQ % 16 == 0 && kOffCum % 4 == 0, "shared-memory alignment");
  static_assert(kStageBytes == 8192 || kStageBytes == 16384, "stage size");
};
static_assert(KaCfg<float, 128, 8>::kSmem <= 232448, "attention shared memory above 227 KB");

struct KaArgs {
  KvPages c;
  const int32_t* seqs;
  const void* q;
  void* o;
  int64_t q_stride, o_stride, layer_off;  // elements; layer_off in 16-byte vectors
  int n, group, subgroups;                // query heads per key head; pieces of at most kRows of them
  int window, sinks;
  int min_steps;  // the least a CTA is given
  int in_place;   // o is q
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

// Rounds of `round` keys that `seen` > 0 keys take (up to 2^31 - 1 of them: no sum passes that).
__host__ __device__ __forceinline__ int ka_rounds(int seen, int round) { return (seen - 1) / round + 1; }

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

__device__ __forceinline__ int ticket_acq_rel(int* p) {
  int old;
  asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], 1;" : "=r"(old) : "l"(p) : "memory");
  return old;
}

// How the places [0, total) are dealt to CTAs 0 .. ctas - 1: as evenly as whole
// places go, the longer ranges first.
struct KaSplit {
  int ctas, each, longer;  // CTAs 0 .. longer - 1 have each + 1 places
  __device__ __forceinline__ void make(int total, int n) {
    ctas = n;
    each = (int)((unsigned)total / (unsigned)n);
    longer = total - each * n;
  }
  __device__ __forceinline__ int begin(int cta) const { return cta * each + min(cta, longer); }
  __device__ __forceinline__ int owner(int place) const {
    const int head = longer * (each + 1);
    return place < head ? (int)((unsigned)place / (unsigned)(each + 1)) : longer + (int)((unsigned)(place - head) / (unsigned)each);
  }
};

// The part of the call's work that a CTA has, walked in order: entry (sequence
// of the call), head piece, and a round of kWarps steps of that pair (a step
// is kKeys keys, a warp's).  A pair of `steps` steps takes kKaPairCost + steps
// places from `base` on; this CTA has those at [x0, x1): steps from .. to - 1.
struct KaWalk {
  int entry, piece, step;  // step: the round's first
  int steps, base, to;     // of this pair
  __device__ __forceinline__ void set_entry(int e, const int* cum, int pieces) {
    entry = e;
    steps = (int)((unsigned)(cum[e + 1] - cum[e]) / (unsigned)pieces) - kKaPairCost;
  }
  // entry == n: nothing is left
  __device__ __forceinline__ void start(int x0, int x1, const int* cum, int n, int pieces) {
    int lo = 0, hi = n;  // cum[lo] <= x0 < cum[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (cum[mid] <= x0) lo = mid; else hi = mid;
    }
    set_entry(lo, cum, pieces);
    const unsigned size = steps + kKaPairCost;
    piece = (int)((unsigned)(x0 - cum[lo]) / size);
    base = cum[lo] + piece * (int)size;
    step = max(0, x0 - base - kKaPairCost);
    to = min(steps, x1 - base - kKaPairCost);
    if (to <= 0) entry = n;  // the range ends in the pair's cost
  }
  template <int kWarps>
  __device__ __forceinline__ void next(int x1, const int* cum, int n, int pieces) {
    step += kWarps;
    if (step < to) return;
    step = 0;
    base += steps + kKaPairCost;
    if (++piece == pieces) {
      piece = 0;
      int e = entry + 1;
      while (e < n && cum[e + 1] == cum[e]) ++e;  // entries without a key
      entry = e;
      if (e < n) set_entry(e, cum, pieces);
    }
    to = min(steps, x1 - base - kKaPairCost);
    if (to <= 0) entry = n;
  }
};

template <bool kL2, typename V>
__device__ __forceinline__ V ka_read(const V* p) {
  if constexpr (kL2) return __ldcg(p); else return *p;
}

// ---------------------------------------------------------------------------
// a warp's running state over its keys of one (sequence, head piece)
// ---------------------------------------------------------------------------
// Both forms offer load_q() (the query rows of a pair, into registers, ahead of
// its beginning), begin(), step() over one ring stage, and store_ml() and
// store_rows() of kMergeRows output rows.

// bf16.  Fragments of mma.m16n8k16: lane = 4 g + t holds rows g and g + 8.
// R = 8: rows g + 8 are zeros in Q and left out of the softmax; in P they hold the
// second parts of rows g, so that one product takes both parts and O is the sum
// of rows g and g + 8 (64 sequences of 1 .. 8192 tokens, 32 heads on 8: 54.8 us,
// with a product of their own 58).
template <int HD, int R>
struct KaStateBf16 {
  static constexpr int kKs = HD / 16, kNt = HD / 8, kKeys = 32, kHalves = R / 8, kMergeRows = 4;
  uint32_t q[kKs][4], qn[kKs][2 * kHalves];
  float o[kNt][4];
  float m[kHalves], l[kHalves];

  // qrow(r): the row of query r; kL2: read past L1 (see kv_own_kernel)
  template <bool kL2 = false, typename Row>
  __device__ __forceinline__ void load_q(const Row& qrow, int rows, int lane) {
    // A fragment: a0 (g, 2t), a1 (g + 8, 2t), a2 (g, 2t + 8), a3 (g + 8, 2t + 8); absent heads are zeros
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int ks = 0; ks < kKs; ++ks)
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int h = 0; h < kHalves; ++h) {
          const int row = g + h * 8, col = ks * 16 + 2 * t + e * 8;
          qn[ks][e * kHalves + h] = row < rows ? ka_read<kL2>(reinterpret_cast<const uint32_t*>(qrow(row) + col)) : 0u;
        }
  }
  __device__ __forceinline__ void begin(int, float*) {
#pragma unroll
    for (int ks = 0; ks < kKs; ++ks)
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int h = 0; h < 2; ++h) q[ks][2 * e + h] = h < kHalves ? qn[ks][e * kHalves + (h < kHalves ? h : 0)] : 0u;
#pragma unroll
    for (int i = 0; i < kNt; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
#pragma unroll
    for (int h = 0; h < kHalves; ++h) {
      m[h] = -INFINITY;
      l[h] = 0.f;
    }
  }

  // stage: K rows [32][HD], V rows [32][HD], 16-byte vector x of row r at x ^ (r & 7); mask: bit r = key r is there
  __device__ __forceinline__ void step(const uint8_t*, uint32_t stage, uint32_t mask, float sc, int lane, const float*) {
    constexpr int kRowBytes = HD * 2;
    const int mi = lane >> 3, r8 = lane & 7;
    float s[4][4] = {};
    {
      const uint32_t base = stage + ((mi >> 1) * 8 + r8) * kRowBytes;
#pragma unroll
      for (int ks = 0; ks < kKs; ++ks)
#pragma unroll
        for (int kp = 0; kp < 2; ++kp) {  // 16 keys
          uint32_t b[4];
          ldmatrix_x4(base + kp * 16 * kRowBytes + (((ks * 2 + (mi & 1)) ^ r8) << 4), b);
          mma_m16n8k16(s[2 * kp], q[ks], b[0], b[1]);
          mma_m16n8k16(s[2 * kp + 1], q[ks], b[2], b[3]);
        }
    }
    const int t2 = (lane & 3) * 2;
    uint32_t p[2][4], pl[2][4];  // R = 8: pl is part of p
#pragma unroll
    for (int h = 0; h < kHalves; ++h) {  // rows g, g + 8
      float x[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = s[e >> 1][2 * h + (e & 1)] * sc;
      if (mask != 0xffffffffu)
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (!((mask >> ((e >> 1) * 8 + t2 + (e & 1))) & 1u)) x[e] = -INFINITY;
      float mx = fmaxf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])), fmaxf(fmaxf(x[4], x[5]), fmaxf(x[6], x[7])));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      // the maximum is raised only when it grows by more than 8 in log2 (P stays <= 2^8):
      // O / l is exact whatever maximum was used
      const bool grow = mx > m[h] + kAtcLazy;
      if (__any_sync(0xffffffffu, grow)) {
        const float alpha = !grow ? 1.f : m[h] == -INFINITY ? 0.f : ex2_approx(m[h] - mx);
        if (grow) m[h] = mx;
        l[h] *= alpha;
#pragma unroll
        for (int i = 0; i < kNt; ++i)
#pragma unroll
          for (int e = 2 * h; e < (R == 8 ? 4 : 2 * h + 2); ++e) o[i][e] *= alpha;
      }
      const float nm = m[h] == -INFINITY ? 0.f : m[h];  // nothing seen yet: every weight is 2^-inf = 0
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        const float p0 = ex2_approx(x[e] - nm), p1 = ex2_approx(x[e + 1] - nm);
        // the upper half of the bits of the number just below p, and the rest, which is thus more than 0 wherever p is:
        // an infinite value does not meet 0 there, and a weight of 0 (0 and 0) adds nothing
        const uint32_t u0 = max(__float_as_uint(p0), 1u) - 1u, u1 = max(__float_as_uint(p1), 1u) - 1u;
        const int at = ((e >> 1) & 1) * 2 + h;  // a0 / a1: keys 2t, 2t + 1; a2 / a3: keys 2t + 8, 2t + 9
        p[e >> 2][at] = __byte_perm(u0, u1, 0x7632);
        const uint32_t rest = pack_bf16x2(p0 - __uint_as_float(u0 & 0xffff0000u), p1 - __uint_as_float(u1 & 0xffff0000u));
        if constexpr (R == 8) p[e >> 2][at + 1] = rest; else pl[e >> 2][at] = rest;
        l[h] += p0 + p1;  // this lane's keys; the lanes of a row are summed at the end
      }
    }
    const uint32_t vbase = stage + kKeys * kRowBytes + ((mi & 1) * 8 + r8) * kRowBytes;
#pragma unroll
    for (int kp = 0; kp < 2; ++kp)
#pragma unroll
      for (int i = 0; i < kNt; i += 2) {
        uint32_t b[4];
        ldmatrix_x4_trans(vbase + kp * 16 * kRowBytes + (((i + (mi >> 1)) ^ r8) << 4), b);
        mma_m16n8k16(o[i], p[kp], b[0], b[1]);
        mma_m16n8k16(o[i + 1], p[kp], b[2], b[3]);
        if constexpr (R == 16) {
          mma_m16n8k16(o[i], pl[kp], b[0], b[1]);
          mma_m16n8k16(o[i + 1], pl[kp], b[2], b[3]);
        }
      }
  }

  __device__ __forceinline__ void store_ml(float* ml, int lane) {
#pragma unroll
    for (int h = 0; h < kHalves; ++h) {
      float s = l[h];
      s += __shfl_xor_sync(0xffffffffu, s, 1);
      s += __shfl_xor_sync(0xffffffffu, s, 2);
      if ((lane & 3) == 0) *reinterpret_cast<float2*>(ml + ((lane >> 2) + 8 * h) * 2) = make_float2(m[h], s);
    }
  }
  __device__ __forceinline__ void store_rows(float* buf, int row0, int lane) {
    const int g = lane >> 2, t2 = (lane & 3) * 2;
#pragma unroll
    for (int h = 0; h < kHalves; ++h) {
      const int row = g + 8 * h - row0;
      if (row >= 0 && row < kMergeRows)
#pragma unroll
        for (int i = 0; i < kNt; ++i)
          *reinterpret_cast<float2*>(buf + row * HD + i * 8 + t2) =
              R == 8 ? make_float2(o[i][0] + o[i][2], o[i][1] + o[i][3]) : make_float2(o[i][2 * h], o[i][2 * h + 1]);
    }
  }
};

// fp32.  For the scores lane = 16 half + key takes half of the head's
// dimensions of one key; for the output a lane owns HD / 32 dimensions.
template <int HD, int R>
struct KaStateF32 {
  static constexpr int kRows = R, kOut = HD / 32, kKeys = 16, kQ = kRows * HD / 32, kMergeRows = R < 4 ? R : 4;
  float o[kRows][kOut], qn[kQ];
  float m[kRows], l[kRows];

  template <bool kL2 = false, typename Row>
  __device__ __forceinline__ void load_q(const Row& qrow, int rows, int lane) {
#pragma unroll
    for (int x = 0; x < kQ; ++x) qn[x] = x * 32 < rows * HD ? ka_read<kL2>(qrow(x / (HD / 32)) + x % (HD / 32) * 32 + lane) : 0.f;
  }
  __device__ __forceinline__ void begin(int lane, float* qs) {
    // every warp writes the same values: no barrier between the warps is needed for its own reads
#pragma unroll
    for (int x = 0; x < kQ; ++x) qs[x * 32 + lane] = qn[x];
    __syncwarp();
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      m[r] = -INFINITY;
      l[r] = 0.f;
#pragma unroll
      for (int e = 0; e < kOut; ++e) o[r][e] = 0.f;
    }
  }

  __device__ __forceinline__ void step(const uint8_t* stage, uint32_t, uint32_t mask, float sc, int lane, const float* qs) {
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
    const uint8_t* vrows = stage + kKeys * kRowBytes;
#pragma unroll 4
    for (int k = 0; k < kKeys; ++k) {
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

  __device__ __forceinline__ void store_ml(float* ml, int lane) {
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      const float s = warp_sum(l[r]);
      if (lane == 0) {
        ml[r * 2] = m[r];
        ml[r * 2 + 1] = s;
      }
    }
  }
  __device__ __forceinline__ void store_rows(float* buf, int row0, int lane) {
#pragma unroll
    for (int r = 0; r < kRows; ++r)
      if (r >= row0 && r < row0 + kMergeRows)
#pragma unroll
        for (int e = 0; e < kOut; ++e) buf[(r - row0) * HD + lane * kOut + e] = o[r][e];
  }
};

template <typename T, int HD, int R>
struct KaState;
template <int HD, int R>
struct KaState<__nv_bfloat16, HD, R> : KaStateBf16<HD, R> {};
template <int HD, int R>
struct KaState<float, HD, R> : KaStateF32<HD, R> {};

__device__ __forceinline__ void ka_store4(__nv_bfloat16* p, float4 v) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
}
__device__ __forceinline__ void ka_store4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }

// O / l; zeros where no weight was seen (whatever the values of weight 0 were)
__device__ __forceinline__ float4 ka_scaled(float4 o, float inv) {
  return inv == 0.f ? make_float4(0.f, 0.f, 0.f, 0.f) : make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
}

template <typename T>
__device__ __forceinline__ float ka_f32(T x) {
  if constexpr (sizeof(T) == 2) return __bfloat162float(x); else return x;
}

// w x, where an infinite x stays what it is under a weight too small for fp32
__device__ __forceinline__ float ka_weigh(float w, float x) { return w == 0.f && isinf(x) ? x : w * x; }

// One row by the definition, by a warp, eight keys at a time; a lane owns HD / 32
// dimensions of q and o.  keys(x, k, v) gives the rows of the x-th of `seen` keys;
// with kGaps it returns whether the key is there (the rows are readable anyway).
// The running output is a mean, each step's weights summing to at most 1, so it stays
// within the values' range whatever their size; an infinite value makes its column
// infinite however small its weight.  Scores of -inf alone give zeros.
template <typename T, int HD, bool kGaps, typename Keys>
__device__ __forceinline__ void ka_row_exact(const T* q, int seen, float scale_log2, const Keys& keys, float (&o)[HD / 32]) {
  constexpr int kE = HD / 32, kU = 8;
  const int at = (threadIdx.x & 31) * kE;
  float qq[kE], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int e = 0; e < kE; ++e) {
    qq[e] = ka_f32(q[at + e]);
    o[e] = 0.f;
  }
  // unsigned: the last step may pass 2^31
  for (uint32_t x0 = 0; x0 < (uint32_t)seen; x0 += kU) {  // kU keys' loads and sums at once
    float d[kU], vv[kU][kE];
    uint32_t there = 0xffffffffu;
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const T *k, *v;
      if constexpr (kGaps) there ^= (uint32_t)!keys((int)min(x0 + u, (uint32_t)seen - 1u), k, v) << u;
      else keys((int)min(x0 + u, (uint32_t)seen - 1u), k, v);
      d[u] = 0.f;
#pragma unroll
      for (int e = 0; e < kE; ++e) {
        d[u] = fmaf(qq[e], ka_f32(k[at + e]), d[u]);
        vv[u][e] = ka_f32(v[at + e]);
      }
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1)
#pragma unroll
      for (int u = 0; u < kU; ++u) d[u] += __shfl_xor_sync(0xffffffffu, d[u], off);
    float mn = m;
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      d[u] = x0 + u < (uint32_t)seen ? d[u] * scale_log2 : -INFINITY;  // the last key again: without weight
      if constexpr (kGaps) {
        d[u] = (there >> u) & 1u ? d[u] : -INFINITY;
#pragma unroll
        for (int e = 0; e < kE; ++e) vv[u][e] = (there >> u) & 1u ? vv[u][e] : 0.f;
      }
      mn = fmaxf(mn, d[u]);
    }
    const float nm = mn == -INFINITY ? 0.f : mn, before = m == -INFINITY ? 0.f : l * exp2f(m - nm);
    m = mn;
    l = before;
#pragma unroll
    for (int u = 0; u < kU; ++u) l += exp2f(d[u] - nm);
    const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
    for (int e = 0; e < kE; ++e) o[e] = ka_weigh(before * inv, o[e]);
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const float p = exp2f(d[u] - nm) * inv;
#pragma unroll
      for (int e = 0; e < kE; ++e) o[e] += ka_weigh(p, vv[u][e]);
    }
  }
#pragma unroll
  for (int e = 0; e < kE; ++e) o[e] = l == 0.f ? 0.f : o[e];
}

// Query head `head` (key head kvh) of an entry, a sequence of `len` tokens, done again
// key by key: its sums of weights up to 2^8 overflowed where the mean does not, or it
// sees an infinite or NaN value.  One warp, and paid only by such rows: one over 8704
// keys takes 1.4 ms.
template <typename T, int HD>
__device__ __noinline__ void ka_redo(const KaArgs& a, int entry, int len, int head, int kvh) {
  constexpr int kE = HD / 32;
  const KvPages& c = a.c;
  const int32_t* row = c.table + (size_t)(a.seqs ? a.seqs[entry] : entry) * c.max_pages;
  const KaSeen s = ka_seen(len, a.window, a.sinks);
  float o[kE];
  ka_row_exact<T, HD, true>(
      reinterpret_cast<const T*>(a.q) + entry * a.q_stride + head * HD, s.seen, a.scale_log2,
      [&](int x, const T*& k, const T*& v) {
        const int key = x < s.sink ? x : x - s.sink + s.first, j = (int)c.page_div.div((uint32_t)key), page = row[j];
        const bool ok = page >= 0 && page < c.num_pages;
        const int64_t off = a.layer_off + (ok ? page : 0) * c.page_stride + (key - j * c.page_size) * c.token_stride +
                            kvh * c.head_stride;
        k = reinterpret_cast<const T*>(c.k + off);
        v = reinterpret_cast<const T*>(c.v + off);
        return ok;
      },
      o);
  T* out = reinterpret_cast<T*>(a.o) + entry * a.o_stride + head * HD + (threadIdx.x & 31) * kE;
#pragma unroll
  for (int e = 0; e < kE; ++e) {
    if constexpr (sizeof(T) == 2) out[e] = __float2bfloat16(o[e]); else out[e] = o[e];
  }
}

template <typename T, int HD, int R>
__global__ void __launch_bounds__(KaCfg<T, HD, R>::kThreads, 1) kv_attention_kernel(const __grid_constant__ KaArgs a) {
  using Cfg = KaCfg<T, HD, R>;
  constexpr int kRows = R, kMergeRows = Cfg::kMergeRows, kStages = Cfg::kStages, kKeys = Cfg::kKeys, kWarps = Cfg::kWarps, kThreads = Cfg::kThreads;
  extern __shared__ __align__(128) uint8_t sm[];
  int* cum = reinterpret_cast<int*>(sm + Cfg::kOffCum);  // places before each entry
  int* lens = reinterpret_cast<int*>(sm + Cfg::kOffLen);  // tokens of each entry
  float* merge = reinterpret_cast<float*>(sm + Cfg::kOffMerge);
  float* ml = reinterpret_cast<float*>(sm + Cfg::kOffMl);
  float* qs = reinterpret_cast<float*>(sm + Cfg::kOffQ);
  __shared__ int warp_places[kWarps], join_sh;
  const KvPages& c = a.c;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int pieces = c.kv_heads * a.subgroups;
  pdl_wait();
  pdl_trigger();

  auto seq_of = [&](int e) { return a.seqs ? a.seqs[e] : e; };
  // places before each entry: thread i sums the entries of its own stretch
  {
    const int per = (a.n + kThreads - 1) / kThreads;
    const int e0 = min(a.n, tid * per), e1 = min(a.n, e0 + per);
    int sum = 0;
    for (int e = e0; e < e1; ++e) {
      const int s = seq_of(e);
      int len = s >= 0 && s < c.max_seqs ? c.lens[s] : -1;
      if (!c.valid_len(len)) {
        if (blockIdx.x == 0) c.flag(KV_BAD_SEQ);
        len = 0;
      }
      lens[e] = len;
      const int seen = ka_seen(len, a.window, a.sinks).seen;
      const int x = seen ? (ka_rounds(seen, kKeys * kWarps) * kWarps + kKaPairCost) * pieces : 0;
      cum[e + 1] = x;
      sum += x;
    }
    int inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += u;
    }
    if (lane == 31) warp_places[warp] = inc;
    __syncthreads();
    int run = inc - sum;
    for (int w = 0; w < warp; ++w) run += warp_places[w];
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
    for (int x = tid; x < vecs; x += kThreads) reinterpret_cast<uint4*>(orow)[x] = make_uint4(0, 0, 0, 0);
  }
  // the host bounds the places of the call below 2^31
  const int total = cum[a.n];
  KaSplit split;
  split.make(total, max(1, min((int)gridDim.x, total / a.min_steps)));
  if (total == 0 || blockIdx.x >= split.ctas) return;
  const int x0 = split.begin(blockIdx.x), x1 = split.begin(blockIdx.x + 1);
  KaWalk load;
  load.start(x0, x1, cum, a.n, pieces);
  if (load.entry >= a.n) return;

  uint8_t* ring = sm + warp * (kStages * Cfg::kStageBytes);
  const uint32_t ring_u32 = smem_u32(ring);
  uint32_t* masks = reinterpret_cast<uint32_t*>(sm + Cfg::kOffMask) + warp * kStages;
  KaWalk use = load;
  // Where key `lane` of this warp's step of a round lies: its page's number as
  // the table has it (not looked at until the copies are issued, two rounds
  // later, so that the load's latency is hidden) and the rest of its address in
  // 16-byte vectors; -1: no such key.
  struct Where {
    int page;
    int64_t off;
  };
  int load_entry = -1;
  const int32_t* load_row = nullptr;
  KaSeen seen{};
  auto look_up = [&]() -> Where {
    if (load.entry != load_entry) {
      load_entry = load.entry;
      load_row = c.table + (size_t)seq_of(load_entry) * c.max_pages;
      seen = ka_seen(lens[load_entry], a.window, a.sinks);
    }
    const uint32_t at = (uint32_t)(load.step + warp) * kKeys + lane % kKeys;  // unsigned: the last round may pass 2^31
    if (load.step + warp >= load.to || at >= (uint32_t)seen.seen) return {0, -1};
    const int x = (int)at, key = x < seen.sink ? x : x - seen.sink + seen.first;
    const int j = (int)c.page_div.div((uint32_t)key);
    return {load_row[j], a.layer_off + (key - j * c.page_size) * c.token_stride + (load.piece / a.subgroups) * c.head_stride};
  };
  Where at = look_up(), at_next{0, -1};
  int ahead_rounds = 1;  // looked up and not issued yet: at, at_next
  auto advance = [&]() {
    load.template next<kWarps>(x1, cum, a.n, pieces);
    if (load.entry < a.n) {
      if (load.step == 0 && warp == 0) {  // a new pair: its query rows into L2 by the time they are wanted
        const int sub = load.piece % a.subgroups, rows = min(kRows, a.group - sub * kRows);
        const char* qp = reinterpret_cast<const char*>(reinterpret_cast<const T*>(a.q) + load.entry * a.q_stride +
                                                       ((load.piece / a.subgroups) * a.group + sub * kRows) * HD);
        for (int x = lane * 128; x < rows * Cfg::kRowBytes; x += 32 * 128)
          asm volatile("prefetch.global.L2 [%0];" ::"l"(qp + x));
      }
      at_next = look_up();
      ++ahead_rounds;
    }
  };
  advance();
  // Copies of one step: eight lanes take 128 bytes of a row at a time, so that
  // each line is asked for once; an absent key's row is zeros.
  auto issue = [&](int stage) {
    if (ahead_rounds > 0) {
      int64_t place = -1;
      if (at.off >= 0) {
        if (at.page >= 0 && at.page < c.num_pages) place = at.off + at.page * c.page_stride;
        else c.flag(KV_BAD_PAGE);
      }
      const uint32_t mask = __ballot_sync(0xffffffffu, place >= 0) & (kKeys == 32 ? 0xffffffffu : 0xffffu);
      if (lane == 0) masks[stage] = mask;
      if (mask) {
#pragma unroll
        for (int j = 0; j < kKeys / 4; ++j) {
          const int r = j * 4 + (lane >> 3);
          const int64_t off = __shfl_sync(0xffffffffu, place, r);
          const int bytes = off >= 0 ? 16 : 0;
          const uint4* ks = c.k + (off >= 0 ? off : 0) + (lane & 7);
          const uint4* vs = c.v + (off >= 0 ? off : 0) + (lane & 7);
          const uint32_t d = ring_u32 + stage * Cfg::kStageBytes + r * Cfg::kRowBytes + (((lane & 7) ^ (r & 7)) << 4);
#pragma unroll
          for (int i = 0; i < Cfg::kVecs / 8; ++i) {
            cp_async16(d + 128 * i, ks + 8 * i, bytes);
            cp_async16(d + 128 * i + kKeys * Cfg::kRowBytes, vs + 8 * i, bytes);
          }
        }
      }
      --ahead_rounds;
      at = at_next;
      if (ahead_rounds > 0) advance();
    }
    cp_async_commit();
  };
  KaState<T, HD, R> state;
  auto load_q = [&](const KaWalk& w) {
    const int sub = w.piece % a.subgroups, head = (w.piece / a.subgroups) * a.group + sub * kRows;
    const T* qrow = reinterpret_cast<const T*>(a.q) + w.entry * a.q_stride + head * HD;
    state.load_q([&](int r) { return qrow + r * HD; }, min(kRows, a.group - sub * kRows), lane);
  };
  load_q(use);
  for (int s = 0; s < kStages - 1; ++s) issue(s);
  state.begin(lane, qs);

  int stage = 0, seg_step = use.step;  // the pair's first step in this CTA
  while (true) {
    issue(stage == 0 ? kStages - 1 : stage - 1);
    cp_async_wait<kStages - 1>();
    __syncwarp();
    const uint32_t mask = masks[stage];
    if (mask)
      state.step(ring + stage * Cfg::kStageBytes, ring_u32 + stage * Cfg::kStageBytes, mask, a.scale_log2, lane, qs);
    __syncwarp();  // the stage is refilled next turn
    stage = stage + 1 == kStages ? 0 : stage + 1;
    KaWalk ahead = use;
    ahead.template next<kWarps>(x1, cum, a.n, pieces);
    const bool go = ahead.entry < a.n;
    if (!go || ahead.base != use.base) {
      // the pair's keys of this CTA are done: merge the warps
      if (go) load_q(ahead);
      const int sub = use.piece % a.subgroups, rows = min(kRows, a.group - sub * kRows);
      const int head = (use.piece / a.subgroups) * a.group + sub * kRows;
      const bool whole = use.to == use.steps && seg_step == 0;
      const int slot = seg_step == 0 ? 1 : 0;  // 0: the pair began in an earlier CTA
      float* part = a.partial + ((int64_t)blockIdx.x * 2 + slot) * Cfg::kSlotFloats;
      state.store_ml(ml + warp * kRows * 2, lane);
      T* orow = reinterpret_cast<T*>(a.o) + use.entry * a.o_stride + head * HD;
      // Four columns of a row, or nothing (!on); the lanes of a row are one warp's, or half of them.  Rows that are not
      // finite are done again at the pair's end, by one call for all its rows (a call at each store: 56.4 us for 64
      // sequences of 1 .. 8192 tokens, 32 heads on 8, this 55.4, without either 55.3).  Where o is q such a row is not
      // stored at all, as its query is wanted still.
      uint32_t redo = 0;
      auto put = [&](bool on, int row, int c4, float4 acc, float ll) {
        // a row whose weights' sum is NaN or 0 is NaN or zeros: nothing else could come out
        const bool bad = on && ll > 0.f && !(fabsf(acc.x) + fabsf(acc.y) + fabsf(acc.z) + fabsf(acc.w) <= 1.0e38f);
        if (bad) redo |= 1u << row;
        bool store = on;
        if (a.in_place) {
          const uint32_t bads = __ballot_sync(0xffffffffu, bad);  // of all lanes, those that are not on too
          store = on && !(bads & (HD == 128 ? 0xffffffffu : 0xffffu << (lane & 16)));
        }
        if (store) ka_store4(orow + row * HD + c4, ka_scaled(acc, ll == 0.f ? 0.f : 1.f / ll));
      };
      static_assert(kMergeRows * HD / 4 <= kThreads, "a round of rows is at most four columns a thread");
      for (int r0 = 0; r0 < rows; r0 += kMergeRows) {
        state.store_rows(merge + warp * (kMergeRows * HD), r0, lane);
        __syncthreads();
        const int row = r0 + tid / (HD / 4), c4 = (tid % (HD / 4)) * 4;
        const bool on = tid < kMergeRows * HD / 4 && row < rows;
        float mm = -INFINITY, ll = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        if (on) {
#pragma unroll
          for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, ml[(w * kRows + row) * 2]);
#pragma unroll
          for (int w = 0; w < kWarps; ++w) {
            const float mw = ml[(w * kRows + row) * 2];
            const float f = mw == -INFINITY ? 0.f : ex2_approx(mw - mm);
            const float4 v = *reinterpret_cast<const float4*>(merge + w * (kMergeRows * HD) + (row - r0) * HD + c4);
            ll = fmaf(f, ml[(w * kRows + row) * 2 + 1], ll);
            acc.x = fmaf(f, v.x, acc.x);
            acc.y = fmaf(f, v.y, acc.y);
            acc.z = fmaf(f, v.z, acc.z);
            acc.w = fmaf(f, v.w, acc.w);
          }
        }
        if (whole) {
          put(on, row, c4, acc, ll);
        } else if (on) {
          __stcg(reinterpret_cast<float4*>(part + Cfg::kSlotO + row * HD + c4), acc);
          if (c4 == 0) __stcg(reinterpret_cast<float2*>(part + row * 2), make_float2(mm, ll));
        }
        __syncthreads();
      }
      if (!whole) {
        const int c_first = split.owner(use.base + kKaPairCost), c_last = split.owner(use.base + kKaPairCost + use.steps - 1);
        // the barrier orders the CTA's partials before the ticket, which is taken with
        // release and acquire: the last CTA sees the partials of all before it
        __syncthreads();
        if (tid == 0) join_sh = ticket_acq_rel(a.tickets + c_first) == c_last - c_first;
        __syncthreads();
        if (join_sh) {
          const int nc = c_last - c_first + 1;
          for (int x0 = 0; x0 < rows * HD / 4; x0 += kThreads) {
            const int x = x0 + tid, row = x / (HD / 4), c4 = (x % (HD / 4)) * 4;
            const bool on = row < rows;
            float mm = -INFINITY, ll = 0.f;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int k0 = 0; k0 < nc && on; k0 += kKaJoin) {  // all loads of a round before the first use
              float2 w[kKaJoin];
              float4 v[kKaJoin];
#pragma unroll
              for (int k = 0; k < kKaJoin; ++k) {
                w[k] = make_float2(-INFINITY, 0.f);
                v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (k0 + k < nc) {
                  const float* p = a.partial + ((int64_t)(c_first + k0 + k) * 2 + (k0 + k == 0 ? 1 : 0)) * Cfg::kSlotFloats;
                  w[k] = __ldcg(reinterpret_cast<const float2*>(p + row * 2));
                  v[k] = __ldcg(reinterpret_cast<const float4*>(p + Cfg::kSlotO + row * HD + c4));
                }
              }
              float mn = mm;
#pragma unroll
              for (int k = 0; k < kKaJoin; ++k) mn = fmaxf(mn, w[k].x);
              const float f0 = mm == -INFINITY ? 0.f : ex2_approx(mm - mn);
              mm = mn;
              ll *= f0;
              acc.x *= f0;
              acc.y *= f0;
              acc.z *= f0;
              acc.w *= f0;
#pragma unroll
              for (int k = 0; k < kKaJoin; ++k) {
                const float f = w[k].x == -INFINITY ? 0.f : ex2_approx(w[k].x - mm);
                ll = fmaf(f, w[k].y, ll);
                acc.x = fmaf(f, v[k].x, acc.x);
                acc.y = fmaf(f, v[k].y, acc.y);
                acc.z = fmaf(f, v[k].z, acc.z);
                acc.w = fmaf(f, v[k].w, acc.w);
              }
            }
            put(on, row, c4, acc, ll);
          }
          if (tid == 0) a.tickets[c_first] = 0;
        }
      }
      for (redo = __reduce_or_sync(0xffffffffu, redo); redo; redo &= redo - 1) {
        __syncwarp();  // behind the row's first stores
        ka_redo<T, HD>(a, use.entry, lens[use.entry], head + __ffs(redo) - 1, use.piece / a.subgroups);
      }
      if (!go) break;
      state.begin(lane, qs);
      seg_step = 0;
    }
    use = ahead;
  }
  cp_async_wait<0>();
}

}  // namespace dinfer
