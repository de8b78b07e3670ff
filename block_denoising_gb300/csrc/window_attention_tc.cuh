// Attention of many bf16 rows with a sliding window and sinks on the tcgen05
// tensor cores (include/dinfer_kv.h, dinfer_op_window_attention).
//
// One CTA = two tiles A and B of 128 query rows over the same key head: two
// query heads of a group at the same rows where the group is even (both tiles
// then want the same keys), else 256 consecutive rows of one head.  The key
// tiles (128 keys) that some row sees -- the sinks' tiles, then the window's --
// pass once through a ring of shared-memory slots and serve both.  320 threads:
//   warp 0     TMA: Q of both tiles, then K_0 V_0 K_1 V_1 ... (128-byte swizzle)
//   warp 1     tensor memory and the single-thread MMA issue, per key tile
//              P_A V, S_A = Q_A K', P_B V, S_B = Q_B K' (K' the next tile's keys)
//   warps 2-5  softmax of tile A, a thread per row; warps 6-9 tile B
// While one tile's softmax runs, the tensor cores work for the other.
//
// Tensor memory (512 columns): S_A | S_B | O_A | O_B.  P = bf16(2^(s - m))
// overwrites the first half of its own S (the row's thread has S in registers
// by then) and is the A operand of P V from there, so the products read shared
// memory for Q, K and V alone: Q K^T already takes the whole 128 bytes a cycle
// of shared memory.  The next S of a tile is issued once its P V has completed.
//
// A running maximum is raised only when a tile's maximum exceeds it by more than
// 8 in log2 (P stays <= 2^8); O and l are rescaled then.  O / l is exact
// whatever maximum was used.  l sums the rounded P, so O / l weights the keys
// exactly in proportion.  Tiles that every row sees whole skip the masks.
#pragma once
#include "window_attention.cuh"

namespace dinfer {

struct WtMaps {
  CUtensorMap q;  // [rows][heads][hd], boxes of 128 rows x 1 head x 64 elements
  CUtensorMap k;
  CUtensorMap v;
};

constexpr int kWtThreads = 320;
constexpr int kWtRows = 128;  // rows of a tile
constexpr int kWtKeys = 128;  // keys of a tile
constexpr uint32_t kDiagWindow = 4;

template <int HD>
struct WtCfg {
  static constexpr int kSlab = 128 * 128;                 // 128 rows x 64 bf16
  static constexpr int kTile = 128 * HD * 2;              // 128 rows or keys of one head
  static constexpr int kSlots = HD == 128 ? 5 : 8;        // K and V tiles in flight
  static constexpr int kOffRing = 2 * kTile;
  static constexpr int kOffBar = kOffRing + kSlots * kTile;
  static constexpr int kSmem = 1024 + kOffBar + 256;
  static constexpr int kColO = 256;                       // O of tile x at kColO + x HD
};
static_assert(WtCfg<128>::kSmem <= 232448, "window attention shared memory above 227 KB");

// The key tiles of a CTA: `front` sink tiles 0 .. front - 1, then first .. ; n in all.
struct WtTiles {
  int front, first, n;
  __device__ __forceinline__ int at(int j) const { return j < front ? j : j - front + first; }
};

// What a tile of rows sees as a whole: any row sees keys only in [0, hi], from
// lo on or below sinks; every row sees [all_lo, all_hi] and the sinks up to all_hi.
struct WtBand {
  int rows;  // valid rows (<= 0: none)
  int lo, hi, all_lo, all_hi;
  __device__ __forceinline__ bool touches(int key0, int sinks) const {
    return rows > 0 && key0 <= hi && (key0 + kWtKeys > lo || key0 < sinks);
  }
  __device__ __forceinline__ bool whole(int key0, int sinks) const {
    return key0 + kWtKeys - 1 <= all_hi && (key0 >= all_lo || key0 + kWtKeys <= sinks);
  }
};
__device__ __forceinline__ WtBand wt_band(const WaArgs& a, const WaSeq& s, int i0) {
  WtBand b;
  b.rows = min(kWtRows, s.nq - i0);
  if (b.rows <= 0) {
    b.lo = b.all_lo = 0;
    b.hi = b.all_hi = -1;
    return b;
  }
  const WaRange t = wa_range(a, s, i0), u = wa_range(a, s, i0 + b.rows - 1);
  b.lo = t.lo;
  b.all_hi = t.hi;
  b.all_lo = u.lo;
  b.hi = u.hi;
  return b;
}

// D[tmem] (+)= A[tmem] B[smem]
__device__ __forceinline__ void tc_mma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                               uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

#define WT_O4(x, b) "=r"(x[(b)]), "=r"(x[(b) + 1]), "=r"(x[(b) + 2]), "=r"(x[(b) + 3])
#define WT_O32(x, b)                                                                               \
  WT_O4(x, b), WT_O4(x, (b) + 4), WT_O4(x, (b) + 8), WT_O4(x, (b) + 12), WT_O4(x, (b) + 16),       \
      WT_O4(x, (b) + 20), WT_O4(x, (b) + 24), WT_O4(x, (b) + 28)
#define WT_I4(x, b) "+r"(x[(b)]), "+r"(x[(b) + 1]), "+r"(x[(b) + 2]), "+r"(x[(b) + 3])
#define WT_I32(x, b)                                                                               \
  WT_I4(x, b), WT_I4(x, (b) + 4), WT_I4(x, (b) + 8), WT_I4(x, (b) + 12), WT_I4(x, (b) + 16),       \
      WT_I4(x, (b) + 20), WT_I4(x, (b) + 24), WT_I4(x, (b) + 28)
#define WT_R4(x, b) "r"(x[(b)]), "r"(x[(b) + 1]), "r"(x[(b) + 2]), "r"(x[(b) + 3])

// 128 consecutive columns of this warp's 32 lanes, one wait for the four
// loads; the empty statements carry the registers past the wait.
__device__ __forceinline__ void tmem_ld128(uint32_t t, uint32_t (&x)[128]) {
#define WT_LD(b)                                                                                             \
  asm volatile(                                                                                              \
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"   \
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"                                 \
      : WT_O32(x, b)                                                                                         \
      : "r"(t + b))
  WT_LD(0);
  WT_LD(32);
  WT_LD(64);
  WT_LD(96);
#undef WT_LD
  asm volatile("tcgen05.wait::ld.sync.aligned;" : WT_I32(x, 0)::"memory");
  asm volatile("" : WT_I32(x, 32));
  asm volatile("" : WT_I32(x, 64));
  asm volatile("" : WT_I32(x, 96));
}
__device__ __forceinline__ void tmem_ld32(uint32_t t, uint32_t (&x)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : WT_O32(x, 0)
      : "r"(t));
  asm volatile("tcgen05.wait::ld.sync.aligned;" : WT_I32(x, 0)::"memory");
}
// 16 columns, no wait
__device__ __forceinline__ void tmem_st16_nowait(uint32_t t, const uint32_t* x) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(t),
      WT_R4(x, 0), WT_R4(x, 4), WT_R4(x, 8), WT_R4(x, 12)
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

template <int HD>
__global__ void __launch_bounds__(kWtThreads, 1)
    window_tc_kernel(const __grid_constant__ WtMaps maps, const __grid_constant__ WaArgs a, const int pair_heads, const int row_blocks) {
  using Cfg = WtCfg<HD>;
  constexpr int kSlots = Cfg::kSlots;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + Cfg::kOffBar);
  uint64_t* q_full = bars;
  uint64_t* full = bars + 1;            // [kSlots]
  uint64_t* empty = full + kSlots;      // [kSlots]
  uint64_t* s_full = empty + kSlots;    // [2]
  uint64_t* p_full = s_full + 2;        // [2]
  uint64_t* pv_done = p_full + 2;       // [2]
  uint64_t* drain = pv_done + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  // head pieces fastest, so that CTAs which run together share keys; the last
  // rows (under a causal mask those with the most keys) first
  const int pieces = pair_heads ? a.heads / 2 : a.heads;
  const int piece = blockIdx.x % pieces;
  const int block_rows = pair_heads ? kWtRows : 2 * kWtRows;
  int b, block;
  if (!wa_find_tile(a, row_blocks - 1 - (int)(blockIdx.x / pieces), block_rows, &b, &block)) return;
  const WaSeq s = wa_seq(a, b);
  const int i0 = block * block_rows;
  const int head0 = pair_heads ? 2 * piece : piece;  // tile x: head head0 + x, or rows i0 + 128 x
  const int kvh = head0 / a.group;
  const WtBand ba = wt_band(a, s, i0);
  const WtBand bb = pair_heads ? ba : wt_band(a, s, i0 + kWtRows);
  WtTiles kt;
  {
    // tile A holds the first row, the last row is B's or, without B, A's
    const int hi = bb.rows > 0 ? bb.hi : ba.hi;
    kt.front = (max(0, min(a.sinks, min(ba.lo, hi + 1))) + kWtKeys - 1) / kWtKeys;
    kt.first = max(kt.front, ba.lo / kWtKeys);
    kt.n = kt.front + (hi < 0 ? 0 : max(0, hi / kWtKeys - kt.first + 1));
  }

  if (threadIdx.x == 0) {
    mbar_init(q_full, 1);
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(&s_full[x], 1);
      mbar_init(&p_full[x], kWtRows);
      mbar_init(&pv_done[x], 1);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&maps.q);
    prefetch_tmap(&maps.k);
    prefetch_tmap(&maps.v);
  }
  if (warp == 1) tmem_alloc(tmem_slot, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 0) {
    // ------------------------------ TMA ------------------------------
    if (elect_one_sync() && kt.n > 0) {
      mbar_arrive_expect_tx(q_full, 2 * Cfg::kTile);
      for (int x = 0; x < 2; ++x)
        for (int h = 0; h < HD / 64; ++h)
          tma_load_3d(sm + x * Cfg::kTile + h * Cfg::kSlab, &maps.q, q_full, h * 64, pair_heads ? head0 + x : head0,
                      s.q0 + i0 + (pair_heads ? 0 : x * kWtRows));
      int issued = 0;
      for (int i = 0; i < 2 * kt.n; ++i) {  // K_0, V_0, K_1, V_1, ...
        const int slot = i % kSlots;
        if (!mbar_wait_diag(&empty[slot], ((i / kSlots) & 1) ^ 1, abort_flag, a.status, kDiagWindow, 1, i)) break;
        issued = i + 1;
        mbar_arrive_expect_tx(&full[slot], Cfg::kTile);
        uint8_t* dst = sm + Cfg::kOffRing + slot * Cfg::kTile;
        const CUtensorMap* map = (i & 1) ? &maps.v : &maps.k;
        const int key = s.k0 + kt.at(i >> 1) * kWtKeys;
        for (int h = 0; h < HD / 64; ++h) tma_load_3d(dst + h * Cfg::kSlab, map, &full[slot], h * 64, kvh, key);
      }
      if (*abort_flag) {  // let the copies in flight land before the CTA exits
        mbar_wait_drain(q_full, 0);
        for (int i = max(0, issued - kSlots); i < issued; ++i) mbar_wait_drain(&full[i % kSlots], (i / kSlots) & 1);
      }
    }
  } else if (warp == 1) {
    // ------------------------------ MMA ------------------------------
    if (elect_one_sync() && kt.n > 0) {
      constexpr uint32_t idesc_s = make_idesc_bf16(128, 128);
      constexpr uint32_t idesc_pv = make_idesc_bf16(128, HD) | (1u << 16);  // B (V) MN-major
      int ns[2] = {0, 0}, np[2] = {0, 0};  // S and P V products issued per tile
      auto wait_full = [&](int i, int site) -> bool {
        return mbar_wait_diag(&full[i % kSlots], (i / kSlots) & 1, abort_flag, a.status, kDiagWindow, site, i);
      };
      auto touches = [&](int x, int j) -> bool {
        return (x ? bb : ba).touches(kt.at(j) * kWtKeys, a.sinks);
      };
      // S_x = Q_x K_j^T over the P that P V has read
      auto issue_s = [&](int x, int j) -> bool {
        if (ns[x] > 0 && !mbar_wait_diag(&pv_done[x], (ns[x] - 1) & 1, abort_flag, a.status, kDiagWindow, 3, j))
          return false;
        tc_fence_after();
        const uint32_t q_addr = smem_u32(sm + x * Cfg::kTile);
        const uint32_t k_addr = smem_u32(sm + Cfg::kOffRing + ((2 * j) % kSlots) * Cfg::kTile);
#pragma unroll
        for (int kk = 0; kk < HD / 16; ++kk)
          tc_mma_bf16(tmem + x * 128, make_sw128_desc(q_addr + (kk >> 2) * Cfg::kSlab + (kk & 3) * 32),
                      make_sw128_desc(k_addr + (kk >> 2) * Cfg::kSlab + (kk & 3) * 32), idesc_s, kk > 0 ? 1u : 0u);
        tc_commit(&s_full[x]);
        ++ns[x];
        return true;
      };
      // O_x += P_x V_j
      auto issue_pv = [&](int x, int j) -> bool {
        if (!mbar_wait_diag(&p_full[x], np[x] & 1, abort_flag, a.status, kDiagWindow, 4, j)) return false;
        tc_fence_after();
        const uint32_t v_addr = smem_u32(sm + Cfg::kOffRing + ((2 * j + 1) % kSlots) * Cfg::kTile);
#pragma unroll
        for (int kk = 0; kk < kWtKeys / 16; ++kk)  // 16 keys: 8 columns of P, 16 rows of V
          tc_mma_bf16_ts(tmem + Cfg::kColO + x * HD, tmem + x * 128 + kk * 8,
                         make_sw128_desc_mn(v_addr + kk * 2048, Cfg::kSlab), idesc_pv, (np[x] > 0 || kk > 0) ? 1u : 0u);
        tc_commit(&pv_done[x]);
        ++np[x];
        return true;
      };
      bool ok = mbar_wait_diag(q_full, 0, abort_flag, a.status, kDiagWindow, 2, 0) && wait_full(0, 5);
      for (int x = 0; x < 2 && ok; ++x)
        if (touches(x, 0)) ok = issue_s(x, 0);
      if (ok) tc_commit(&empty[0]);
      for (int j = 0; j < kt.n && ok; ++j) {
        ok = wait_full(2 * j + 1, 6);
        for (int x = 0; x < 2 && ok; ++x) {
          if (touches(x, j)) ok = issue_pv(x, j);
          if (x == 1 && ok) tc_commit(&empty[(2 * j + 1) % kSlots]);
          if (j + 1 < kt.n && ok) {
            if (x == 0) ok = wait_full(2 * j + 2, 7);
            if (ok && touches(x, j + 1)) ok = issue_s(x, j + 1);
            if (x == 1 && ok) tc_commit(&empty[(2 * j + 2) % kSlots]);
          }
        }
      }
      tc_commit(drain);
      mbar_wait_drain(drain, 0);
    }
  } else {
    // ------------------------------ softmax, output ------------------------------
    const int x = (warp - 2) >> 2;                 // tile
    const int r = (warp & 3) * 32 + lane;          // row of the tile = lane of tensor memory
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const WtBand band = x ? bb : ba;
    const int i_tile = i0 + ((!pair_heads && x) ? kWtRows : 0);
    const int head = pair_heads ? head0 + x : head0;
    const bool live = (warp & 3) * 32 < band.rows;  // warp-uniform
    const WaRange rr = wa_range(a, s, i_tile + max(0, min(r, band.rows - 1)));
    const uint32_t t_s = tmem + x * 128 + lanes, t_o = tmem + Cfg::kColO + x * HD + lanes;
    const float sc = a.scale_log2;
    float m_used = -INFINITY, l = 0.f;
    bool ok = true;
    int c = 0;  // tiles of keys done
    for (int j = 0; j < kt.n; ++j) {
      const int key0 = kt.at(j) * kWtKeys;
      if (!band.touches(key0, a.sinks)) continue;
      const uint32_t parity = c & 1;
      ++c;
      if (ok && !__all_sync(0xffffffffu, mbar_wait_diag(&s_full[x], parity, abort_flag, a.status, kDiagWindow, 8, j)))
        ok = false;
      if (!live || !ok) {  // rows past the sequence: keep the counts only
        mbar_arrive(&p_full[x]);
        continue;
      }
      uint32_t sv[128];
      tc_fence_after();
      tmem_ld128(t_s, sv);
      if (!band.whole(key0, a.sinks)) {
        const int hi = rr.hi - key0, lo = rr.lo - key0, sk = a.sinks - key0;
#pragma unroll
        for (int e = 0; e < 128; ++e)
          if (e > hi || (e < lo && e >= sk)) sv[e] = 0xff800000u;  // -inf
      }
      float mx[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) mx[e] = __uint_as_float(sv[e]);
#pragma unroll
      for (int e = 4; e < 128; ++e) mx[e & 3] = fmaxf(mx[e & 3], __uint_as_float(sv[e]));
      const float mj = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * sc;  // -inf: no key seen
      if (m_used == -INFINITY) m_used = mj;  // nothing accumulated yet
      const bool grow = mj > m_used + kAtcLazy;
      if (__any_sync(0xffffffffu, grow)) {
        // S of this tile was issued after the last P V completed: O is whole
        const float alpha = grow ? ex2_approx(m_used - mj) : 1.f;
        if (c > 1) {
#pragma unroll 1
          for (int k = 0; k < HD / 16; ++k) {
            float o16[16];
            tmem_ld16(t_o + k * 16, o16);
#pragma unroll
            for (int e = 0; e < 16; ++e) o16[e] *= alpha;
            tmem_st16(t_o + k * 16, o16);
          }
        }
        l *= alpha;
        if (grow) m_used = mj;
      }
      const float nm = m_used == -INFINITY ? 0.f : -m_used;
      uint32_t pk[64];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const float p0 = ex2_approx(fmaf(__uint_as_float(sv[k * 32 + 2 * e]), sc, nm));
          const float p1 = ex2_approx(fmaf(__uint_as_float(sv[k * 32 + 2 * e + 1]), sc, nm));
          pk[k * 16 + e] = pack_bf16x2(p0, p1);
        }
        tmem_st16_nowait(t_s + k * 16, pk + k * 16);
      }
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(&p_full[x]);
      // the sum of what the tensor cores multiply, while they do
      float rs[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int e = 0; e < 64; ++e)
        rs[e & 3] += __uint_as_float(pk[e] << 16) + __uint_as_float(pk[e] & 0xffff0000u);
      l += (rs[0] + rs[1]) + (rs[2] + rs[3]);
    }
    if (live) {
      if (c > 0 && ok &&
          !__all_sync(0xffffffffu, mbar_wait_diag(&pv_done[x], (c - 1) & 1, abort_flag, a.status, kDiagWindow, 9, c)))
        ok = false;
      const bool some = ok && c > 0 && l != 0.f;  // l NaN: the row is done again below
      const float inv = some ? 1.f / l : 0.f;
      bool fine = ok && l <= 3.0e38f;
      __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(a.o) + (int64_t)(s.q0 + i_tile + r) * a.o_stride + head * HD;
#pragma unroll 1
      for (int k = 0; k < HD / 32; ++k) {
        uint32_t o[32];
        if (ok && c > 0) {
          tc_fence_after();
          tmem_ld32(t_o + k * 32, o);
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = 0;
        }
        uint4 w[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          float f[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float v = __uint_as_float(o[u * 8 + e]);
            fine = fine && fabsf(v) <= 3.0e38f;
            f[e] = some ? v * inv : 0.f;
          }
          w[u] = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
        }
        if (r < band.rows)
#pragma unroll
          for (int u = 0; u < 4; ++u) reinterpret_cast<uint4*>(out + k * 32)[u] = w[u];
      }
      tc_fence_before();
      uint32_t redo = __ballot_sync(0xffffffffu, ok && !fine && r < band.rows);
      __syncwarp();
      while (redo) {
        const int e = __ffs(redo) - 1;
        redo &= redo - 1;
        wa_row_exact<__nv_bfloat16, HD>(a, s, i_tile + (warp & 3) * 32 + e, head);
      }
    }
  }

  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

#undef WT_O4
#undef WT_O32
#undef WT_I4
#undef WT_I32
#undef WT_R4

}  // namespace dinfer
