// Attention of many bf16 rows with a sliding window and sinks on the tcgen05
// tensor cores (include/dinfer_kv.h, dinfer_op_window_attention).
//
// A piece of work is two tiles A and B of 128 query rows over the same key head:
// two query heads of a group at the same rows where the group is even (both tiles
// then want the same keys), else 256 consecutive rows of one head.  Short calls
// give every tile an SM of its own (A alone), and where SMs are left over several,
// each with a part of the keys: the parts are joined in fp32 through the workspace,
// by the last of their CTAs.  (One row over 4001 keys, 32 heads of 128 on 4: two
// heads a CTA 50 us, one 41, in four parts 17; 64 rows over
// 8704 keys, 32 heads of 128: 79 and 36.)  The key tiles
// (128 keys) that some row sees -- the sinks' tiles, then the window's -- pass
// once through a ring of shared-memory slots and serve both.  One CTA an SM takes
// its pieces in turn, so that a piece's output is written, and the next one's
// queries and keys arrive, while the other tile is still at work.  352 threads:
//   warp 0     TMA: Q of both tiles, then K_0 V_0 K_1 V_1 ... (128-byte swizzle);
//              a slot is free once both tiles' products over it have completed
//   warp 1     tensor memory and the single-thread MMA issue, tiles in turn:
//              S_A, S_B, S_A', P_A V, S_B', P_B V, ...  (A alone: S, S', P V, S'', P' V, ...)
//   warps 2-5  softmax and output of tile A, a thread per row; warps 6-9 tile B
//   warp 10    looks the pieces up, one ahead
//
// Bound by the chain of a tile's turn and by the issuing thread, as clocks in the
// kernel show.  The links cost more than their work: a product of 128 x 128 x 128
// (512 cycles) is seen by the next link some 840 cycles after its issue, S comes
// out of tensor memory in 220 to 350, 64 exponentials a row take 430.  (Times:
// 8704 causal rows, 16 heads of 128, window 4096, in bursts of calls of some
// milliseconds at 2070 MHz.  A second of them meets the power cap: 171 us where a
// burst has 159.)
//   - With S and P of a tile in the same columns the next S waits until P V is
//     seen to be done (199 us).  So P has columns of its own and, at head_dim 128,
//     S_A and S_B take turns in one buffer: S is free again as soon as its rows are
//     in registers, the next S of a tile runs under its softmax, and the tiles stay
//     half a turn apart.  P is handed over in halves of 64 keys.
//   - Every cycle of the issuing thread between two products is one of the whole.
//     It has one instance of each product's code and no indexed array: its code is
//     evicted by the softmax warps that share its instruction cache, and local
//     memory is L2 here, as is any spill of the softmax (203 us with both, 167 us
//     without).  For the same reason the softmax's instructions are few: packed
//     pairs for the scaling and the sums, maxima of three (159 us, 1.40 PFLOP/s;
//     without a window 202 us, 1.54 PFLOP/s).
//   - Measured and not kept: an issuing thread for each tile, or one for S and one
//     for P V (183 to 201 us), a second commit per product in place of the TMA
//     thread's own waits (258 us), four threads a row (241 us), a lock that keeps
//     the two softmaxes apart (187 us), registers moved by setmaxnreg (192 us).
//
// Tensor memory (512 columns): head_dim 128: S | P_A | P_B | O_A | O_B, head_dim
// 64: S_A | S_B | P_A | P_B | O_A | O_B.  P = bf16(2^(s - m)) is the A operand of
// P V, so the products read shared memory for Q, K and V alone (Q K^T takes all
// of its 128 bytes a cycle).
//
// A running maximum is raised only when a tile's maximum exceeds it by more than
// 8 in log2 (P stays <= 2^8); O and l are rescaled then.  O / l is exact
// whatever maximum was used.  P is rounded to 8 bits, as the A operand has V's
// type; a second part for what is lost would be another product per tile.  l sums the
// rounded P, so O / l weights the keys exactly in proportion (8704 causal rows: off by
// 2.0e-3 of the output's size; with 32-bit weights the output's own rounding leaves
// 1.5e-3).  Tiles that every row sees whole skip the masks; the others test a bit per
// key (compared bounds instead: 66 us where this took 60, ragged prompts with a window
// of 256 on both sides).
#pragma once
#include "window_attention.cuh"

namespace dinfer {

struct WtMaps {
  CUtensorMap q;  // [rows][heads][hd], boxes of 128 rows x 1 head x 64 elements
  CUtensorMap k;
  CUtensorMap v;
};

constexpr int kWtThreads = 352;
constexpr int kWtRows = 128;  // rows of a tile
constexpr int kWtKeys = 128;  // keys of a tile
// the tiles of a piece: two heads' rows, 256 rows of a head, one tile alone
enum WtForm { kWtPairHeads, kWtPairRows, kWtSingle };
constexpr int kWtPartTiles = 2;  // key tiles of a part at least

template <int HD>
struct WtCfg {
  static constexpr int kSlab = 128 * 128;                 // 128 rows x 64 bf16
  static constexpr int kTile = 128 * HD * 2;              // 128 rows or keys of one head
  static constexpr int kSlots = HD == 128 ? 5 : 8;        // K and V tiles in flight
  static constexpr int kOffRing = 2 * kTile;
  static constexpr int kOffBar = kOffRing + kSlots * kTile;
  static constexpr int kSmem = 1024 + kOffBar + 336;
  // a part's rows in the workspace: (m, l) of 128, then O
  static constexpr int kSlotFloats = 2 * 128 + 128 * HD;
  // tensor memory: S buffers, then P (64 columns) and O (HD) of each tile
  static constexpr int kBufs = HD == 128 ? 1 : 2;
  static constexpr int kColP = kBufs * 128;
  static constexpr int kColO = kColP + 128;
  static_assert(kColO + 2 * HD <= 512, "tensor memory");
};
static_assert(WtCfg<128>::kSmem + 512 <= 232448, "window attention shared memory above 227 KB");

// What a tile of rows sees as a whole: any row sees keys only in [0, hi], from
// lo on or below sinks; every row sees [all_lo, all_hi] and the sinks up to all_hi.
struct WtBand {
  int rows;  // valid rows (<= 0: none)
  int lo, hi, all_lo, all_hi;
  __device__ __forceinline__ bool touches(int key0, int sinks) const volatile {
    return rows > 0 && key0 <= hi && (key0 + kWtKeys > lo || key0 < sinks);
  }
  __device__ __forceinline__ bool whole(int key0, int sinks) const volatile {
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

// A place in the ring of slots and the parity of its phase.
struct WtSlot {
  int slot;
  uint32_t parity;
  template <int kSlots>
  __device__ __forceinline__ void next() {
    if (++slot == kSlots) {
      slot = 0;
      parity ^= 1;
    }
  }
};

// A piece of work, in shared memory.  The softmax threads have 128 registers of
// S and none to spare -- a spill goes to L2, as nothing of the SM's memory is left
// to be a cache, and made the ragged case 1.6 times as slow -- so they read what
// they want of it where they want it.
struct WtPiece {
  WaSeq s;
  int i0, head0, kvh;   // first row, first query head, key head
  int front, first, n;  // key tiles: the sinks' 0 .. front - 1, then first ..; n in all (-1: no piece is left)
  int unit, part, parts;  // kSplit: which tile, which part of its keys, of how many
  int joins;              // kSplit: pieces with several parts that this CTA had before
  WtBand band[2];
  __device__ __forceinline__ void put(const WtPiece& p) volatile {
    s.q0 = p.s.q0;
    s.nq = p.s.nq;
    s.k0 = p.s.k0;
    s.nk = p.s.nk;
    i0 = p.i0;
    head0 = p.head0;
    kvh = p.kvh;
    front = p.front;
    first = p.first;
    n = p.n;
    unit = p.unit;
    part = p.part;
    parts = p.parts;
    joins = p.joins;
    for (int x = 0; x < 2; ++x) {
      band[x].rows = p.band[x].rows;
      band[x].lo = p.band[x].lo;
      band[x].hi = p.band[x].hi;
      band[x].all_lo = p.band[x].all_lo;
      band[x].all_hi = p.band[x].all_hi;
    }
  }
  __device__ __forceinline__ WtBand copy_band(int x) const volatile {
    return {band[x].rows, band[x].lo, band[x].hi, band[x].all_lo, band[x].all_hi};
  }
  __device__ __forceinline__ int key0(int j) const volatile { return (j < front ? j : j - front + first) * kWtKeys; }
};

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
#define WT_O16(x, b) WT_O4(x, b), WT_O4(x, (b) + 4), WT_O4(x, (b) + 8), WT_O4(x, (b) + 12)
// early-clobber: written before the last address is read
#define WT_E4(x, b) "=&r"(x[(b)]), "=&r"(x[(b) + 1]), "=&r"(x[(b) + 2]), "=&r"(x[(b) + 3])
#define WT_E16(x, b) WT_E4(x, b), WT_E4(x, (b) + 4), WT_E4(x, (b) + 8), WT_E4(x, (b) + 12)
#define WT_E64(x, b) WT_E16(x, b), WT_E16(x, (b) + 16), WT_E16(x, (b) + 32), WT_E16(x, (b) + 48)
#define WT_R4(x, b) "r"(x[(b)]), "r"(x[(b) + 1]), "r"(x[(b) + 2]), "r"(x[(b) + 3])

// Consecutive columns of this warp's 32 lanes, a row a thread.  Load and wait
// are one statement: a register that a load still fills is never moved.
__device__ __forceinline__ void tmem_ld128(uint32_t t, uint32_t (&x)[128]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {"
      "%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31"
      "}, [%128];\n"
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {"
      "%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,"
      "%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63"
      "}, [%129];\n"
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {"
      "%64,%65,%66,%67,%68,%69,%70,%71,%72,%73,%74,%75,%76,%77,%78,%79,"
      "%80,%81,%82,%83,%84,%85,%86,%87,%88,%89,%90,%91,%92,%93,%94,%95"
      "}, [%130];\n"
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {"
      "%96,%97,%98,%99,%100,%101,%102,%103,%104,%105,%106,%107,%108,%109,%110,%111,"
      "%112,%113,%114,%115,%116,%117,%118,%119,%120,%121,%122,%123,%124,%125,%126,%127"
      "}, [%131];\n"
      " tcgen05.wait::ld.sync.aligned;"
      : WT_E64(x, 0), WT_E64(x, 64)
      : "r"(t), "r"(t + 32), "r"(t + 64), "r"(t + 96)
      : "memory");
}
__device__ __forceinline__ void tmem_ld32(uint32_t t, uint32_t (&x)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {"
      "%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31"
      "}, [%32];\n tcgen05.wait::ld.sync.aligned;"
      : WT_O16(x, 0), WT_O16(x, 16)
      : "r"(t)
      : "memory");
}
// 16 columns, no wait
__device__ __forceinline__ void tmem_st16_nowait(uint32_t t, const uint32_t* x) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {"
      "%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16"
      "};" ::"r"(t),
      WT_R4(x, 0), WT_R4(x, 4), WT_R4(x, 8), WT_R4(x, 12)
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// Bits 0 .. n - 1.
__device__ __forceinline__ uint32_t bits_below(int n) {
  uint32_t d;
  asm("bmsk.clamp.b32 %0, 0, %1;" : "=r"(d) : "r"(max(n, 0)));
  return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// Cluster launch control: asks for a CTA of this grid that has not begun; the
// answer (16 bytes) completes the barrier.  clc_taken reads it: the CTA's x
// index, which is now this CTA's to do, or -1: all have begun (not to be asked
// again).
__device__ __forceinline__ void clc_ask(uint4* answer, uint64_t* bar) {
  mbar_arrive_expect_tx(bar, 16);
  asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
                   smem_u32(answer)),
               "r"(smem_u32(bar))
               : "memory");
}
__device__ __forceinline__ int clc_taken(const uint4* answer) {
  uint32_t ok, x;
  asm volatile(
      "{\n .reg .b128 r;\n .reg .pred p;\n .reg .b64 lo, hi;\n .reg .b32 y, z;\n"
      " ld.shared.v2.b64 {lo, hi}, [%2];\n mov.b128 r, {lo, hi};\n"
      " clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n"
      " selp.u32 %0, 1, 0, p;\n mov.u32 %1, 0;\n"
      " @p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {%1, y, z, _}, r;\n}"
      : "=r"(ok), "=r"(x)
      : "r"(smem_u32(answer))
      : "memory");
  return ok ? (int)x : -1;
}

// kSplit: A alone, its keys dealt to up to a.splits CTAs.  A kernel of its own: with
// the join among its code the other forms ran 3 to 5 % longer.
template <int HD, bool kSplit>
__global__ void __launch_bounds__(kWtThreads, 1)
    window_tc_kernel(const __grid_constant__ WtMaps maps, const __grid_constant__ WaArgs a, const int form,
                     const int row_blocks) {
  const bool pair_heads = !kSplit && form == kWtPairHeads, single = kSplit || form == kWtSingle;
  const int splits = kSplit ? a.splits : 1;
  using Cfg = WtCfg<HD>;
  constexpr int kSlots = Cfg::kSlots;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + Cfg::kOffBar);
  uint64_t* q_full = bars;
  uint64_t* full = bars + 1;             // [kSlots]
  // A tile's n-th product completes phase n / 4 of barrier n % 4.  The TMA thread
  // waits for the products that read a slot before it fills it again, and may be
  // late: but K and V of a tile's product n + 4 need the slots (at most 8) of those
  // of product n, so a barrier is never two phases on when it is looked at.
  uint64_t* s_full = full + kSlots;      // [2 tiles][4]
  uint64_t* pv_done = s_full + 8;        // [2 tiles][4]
  uint64_t* p_full = pv_done + 8;        // [2 tiles][2 halves of 64 keys]
  uint64_t* s_free = p_full + 4;         // [kBufs]: the rows of S are in registers
  uint64_t* piece_full = s_free + 2;     // [2]
  uint64_t* piece_empty = piece_full + 2;  // [2]
  uint64_t* drain = piece_empty + 2;
  uint64_t* clc_bar = drain + 1;
  uint64_t* loaded = clc_bar + 1;        // a piece's last copies are issued
  uint64_t* part_out = loaded + 1;       // a part's rows are in the workspace
  uint64_t* part_told = part_out + 1;    // whether this CTA joins the parts
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(part_told + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  static_assert((1 + kSlots + 8 + 8 + 4 + 2 + 2 + 2 + 2 + 3 + 1) * 8 <= 336, "barriers");
  __shared__ volatile WtPiece pieces[2];
  __shared__ uint4 clc_answer[2];
  __shared__ volatile int redoing;  // warps that do rows again
  __shared__ volatile int join_here;
  // of each slot's tile, for the TMA thread: which tiles' products read it (bits
  // 0, 1) and whether it is V (bit 2); the products' numbers (the long waits look at slot 0's)
  __shared__ int slot_use[kSlots][3];

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    mbar_init(q_full, 1);
    for (int i = 0; i < kSlots; ++i) mbar_init(&full[i], 1);
    for (int i = 0; i < 8; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&pv_done[i], 1);
    }
    for (int i = 0; i < 4; ++i) mbar_init(&p_full[i], 4);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_free[i], 4);
      mbar_init(&piece_full[i], 1);
      mbar_init(&piece_empty[i], kSplit ? 6 : 10);  // the TMA and the MMA thread, the softmax warps
    }
    mbar_init(drain, 1);
    mbar_init(clc_bar, 1);
    mbar_init(loaded, 1);
    if (kSplit) {
      mbar_init(part_out, 4);
      mbar_init(part_told, 1);
    }
    *abort_flag = 0;
    redoing = 0;
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
  pdl_wait();
  pdl_trigger();

  // Bounded; a wait that ran out sets the status at the kernel's end (the code of a
  // record at every wait would crowd the instruction caches).  While rows are done
  // again key by key, which may take long, the others' waits do not run out.
  auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
    if (mbar_try_wait(bar, parity)) return true;
    long long t0 = clock64();
    while (!mbar_try_wait(bar, parity)) {
      if (*abort_flag) return false;
      if (clock64() - t0 > kWaitCycles) {
        if (redoing == 0) *abort_flag = 1;
        t0 = clock64();
      }
    }
    return true;
  };
  // A wait that may last as long as a piece (warp 10's for its last copies, and that of
  // warps without a part in it for the next one: the limit's second is reached at some
  // 1e8 keys): it runs out when slot 0 got no tile since it last looked.
  auto wait_long = [&](uint64_t* bar, uint32_t parity) -> bool {
    if (mbar_try_wait(bar, parity)) return true;
    long long t0 = clock64();
    int before = -1;
    while (!mbar_try_wait(bar, parity)) {
      if (*abort_flag) return false;
      if (clock64() - t0 > kWaitCycles) {
        const int now = *(volatile int*)&slot_use[0][1] + *(volatile int*)&slot_use[0][2];
        if (now == before && redoing == 0) *abort_flag = 1;
        before = now;
        t0 = clock64();
      }
    }
    return true;
  };
  // piece number it of this CTA lies in pieces[it & 1] (named as an array, so that
  // its fields are loads from shared memory and not through a generic address)
  auto have_piece = [&](int it) -> bool { return wait_long(&piece_full[it & 1], (it >> 1) & 1); };

  if (warp == 10) {
    // ------------------------------ pieces ------------------------------
    // heads fastest, so that CTAs which run together share keys; the last rows
    // (under a causal mask those with the most keys) first
    const int per_block = pair_heads ? a.heads / 2 : a.heads * splits, block_rows = form == kWtPairRows ? 2 * kWtRows : kWtRows;
    int asked = 0, joins = 0;
    int at = blockIdx.x;  // of the grid's pieces: this CTA's own, then one that no CTA has begun
    bool left = true, own = true;
    for (int it = 0; left; ++it) {
      // asked for once the last piece's copies are issued, some three key tiles
      // before its end: no CTA holds pieces that another could have begun
      if (it > 0 && !__all_sync(0xffffffffu, wait_long(loaded, (it - 1) & 1))) break;
      int b = 0, block = 0, piece = 0;
      left = false;
      while (!left) {
        if (!own) {
          if (lane == 0) clc_ask(&clc_answer[asked & 1], clc_bar);
          if (!__all_sync(0xffffffffu, wait(clc_bar, asked & 1))) break;
          at = clc_taken(&clc_answer[asked & 1]);
          fence_async_shared();  // read before another answer is written over it
          __syncwarp();
          ++asked;
        }
        own = false;
        if (at < 0) break;
        piece = at % per_block;
        left = wa_find_tile(a, row_blocks - 1 - at / per_block, block_rows, &b, &block);
      }
      if (it >= 2 && !__all_sync(0xffffffffu, wait(&piece_empty[it & 1], ((it >> 1) - 1) & 1))) break;
      if (lane == 0) {
        WtPiece p;
        p.n = -1;
        p.unit = p.part = 0;
        p.parts = 1;
        p.joins = joins;
        if (left) {
          p.s = wa_seq(a, b);
          p.i0 = block * block_rows;
          p.head0 = pair_heads ? 2 * piece : piece / splits;  // tile x: head head0 + x, or rows i0 + 128 x
          p.kvh = p.head0 / a.group;
          p.band[0] = wt_band(a, p.s, p.i0);
          p.band[1] = pair_heads ? p.band[0] : wt_band(a, p.s, single ? p.s.nq : p.i0 + kWtRows);
          // tile A holds the first row, the last row is B's or, without B, A's
          const int lo = p.band[0].lo, hi = p.band[1].rows > 0 ? p.band[1].hi : p.band[0].hi;
          p.front = (max(0, min(a.sinks, min(lo, hi + 1))) + kWtKeys - 1) / kWtKeys;
          p.first = max(p.front, lo / kWtKeys);
          p.n = p.front + (hi < 0 ? 0 : max(0, hi / kWtKeys - p.first + 1));
          if constexpr (kSplit) {
            // a part has at least two key tiles, and one more for every 32 rows to be
            // joined (128 rows over 3000 keys, 8 heads of 128: 25.8 us; one more for every
            // 16 rows 30.2, none 31.8; 64 rows over 1500 keys: 16.7, 18.2, 20.6); the sinks
            // go to the first part
            const int w = p.n - p.front, parts = max(1, min(splits, w / (kWtPartTiles + p.band[0].rows / 32)));
            p.unit = at / splits;
            p.part = at % splits;
            if (p.part >= parts) {  // too few keys for another part
              p.n = 0;
              p.band[0].rows = 0;
            } else {
              const int w0 = wa_part_begin(w, p.part, parts), w1 = wa_part_begin(w, p.part + 1, parts);
              if (p.part > 0) p.front = 0;
              p.first += w0;
              p.n = p.front + w1 - w0;
              p.parts = parts;
              joins += parts > 1;
            }
          }
        }
        pieces[it & 1].put(p);
        mbar_arrive(&piece_full[it & 1]);
      }
      __syncwarp();
    }
  } else if (warp == 0) {
    // ------------------------------ TMA ------------------------------
    if (elect_one_sync()) {
      int i = 0;              // K and V tiles loaded
      int n[2] = {0, 0};      // products of each tile over the key tiles loaded
      int loads_q = 0;
      bool ok = true;
      for (int it = 0; ok; ++it) {
        if (!have_piece(it)) break;
        volatile WtPiece& p = pieces[it & 1];
        if (p.n < 0) break;
        const int kn = p.n;
        if (kn > 0) {
          // the last piece's S have all read its Q
#pragma unroll
          for (int x = 0; x < 2; ++x)
            if (ok && n[x] > 0) ok = wait(&s_full[4 * x + ((n[x] - 1) & 3)], ((n[x] - 1) >> 2) & 1);
          if (!ok) break;
          const int tiles = single ? 1 : 2;
          mbar_arrive_expect_tx(q_full, tiles * Cfg::kTile);
          ++loads_q;
          for (int x = 0; x < tiles; ++x)
            for (int h = 0; h < HD / 64; ++h)
              tma_load_3d(sm + x * Cfg::kTile + h * Cfg::kSlab, &maps.q, q_full, h * 64, pair_heads ? p.head0 + x : p.head0,
                          p.s.q0 + p.i0 + (pair_heads ? 0 : x * kWtRows));
          const int kvh = p.kvh, k0 = p.s.k0;
          for (int j = 0; j < 2 * kn && ok; ++j, ++i) {  // K_0, V_0, K_1, V_1, ...
            const int slot = i % kSlots;
            if (i >= kSlots) {
              // the slot's last tile: K was read by S, V by P V, of each tile that touches it
              const int use = slot_use[slot][0];
#pragma unroll
              for (int x = 0; x < 2; ++x)
                if (ok && ((use >> x) & 1)) {
                  const int was = slot_use[slot][1 + x];
                  ok = wait(((use & 4) ? pv_done : s_full) + 4 * x + (was & 3), (was >> 2) & 1);
                }
              if (!ok) break;
            }
            const int key0 = p.key0(j >> 1);
            int use = (j & 1) << 2;
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const bool t = p.band[x].touches(key0, a.sinks);
              use |= t << x;
              slot_use[slot][1 + x] = n[x];
              n[x] += t && (j & 1);
            }
            slot_use[slot][0] = use;
            mbar_arrive_expect_tx(&full[slot], Cfg::kTile);
            uint8_t* dst = sm + Cfg::kOffRing + slot * Cfg::kTile;
            const CUtensorMap* map = (j & 1) ? &maps.v : &maps.k;
            for (int h = 0; h < HD / 64; ++h) tma_load_3d(dst + h * Cfg::kSlab, map, &full[slot], h * 64, kvh, k0 + key0);
          }
        }
        mbar_arrive(loaded);
        mbar_arrive(&piece_empty[it & 1]);
      }
      if (*abort_flag) {  // let the copies in flight land before the CTA exits
        if (loads_q > 0) mbar_wait_drain(q_full, (loads_q - 1) & 1);
        for (int j = max(0, i - kSlots); j < i; ++j) mbar_wait_drain(&full[j % kSlots], (j / kSlots) & 1);
      }
    }
  } else if (warp == 1) {
    // ------------------------------ MMA ------------------------------
    if (elect_one_sync()) {
      constexpr uint32_t idesc_s = make_idesc_bf16(128, 128);
      constexpr uint32_t idesc_pv = make_idesc_bf16(128, HD) | (1u << 16);  // B (V) MN-major
      const uint64_t qd = make_sw128_desc(smem_u32(sm));
      const uint64_t kd = make_sw128_desc(smem_u32(sm + Cfg::kOffRing));
      const uint64_t vd = make_sw128_desc_mn(smem_u32(sm + Cfg::kOffRing), Cfg::kSlab);
      // One instance of each product's code, the tile a number: this thread shares
      // an instruction cache with softmax warps that stream some 11 KB a turn, and
      // its time between products is time of the whole (two instances: 188 against
      // 179 us).  Counts modulo 8, 8 bits for each tile, so that no array is indexed
      // (local memory is L2 here).
      int q_loads = 0;
      uint32_t ns = 0, np = 0;  // S and P V products issued
      uint32_t fresh = 3;       // bit x: no P V of this piece yet
      uint32_t used = 0;        // S buffers in use: kBufs bits
      int turns = 0;            // S of both tiles
      WtSlot ring{0, 0};        // K of the key tile at hand
      bool ok = true;
      for (int it = 0; ok; ++it) {
        if (!have_piece(it)) break;
        volatile WtPiece& p = pieces[it & 1];
        if (p.n < 0) break;
        // in registers: a load from shared memory behind a commit waits for it
        const int kn = p.n, front = p.front, first = p.first;
        const WtBand b0 = p.copy_band(0), b1 = p.copy_band(1);
        if (kn > 0) {
          ok = wait(q_full, q_loads & 1);
          ++q_loads;
          fresh = 3;
          // S of a turn, then P V of the turn before the last: of the same tile where
          // both are at work, so that its next S runs under its softmax.  A product
          // due is key tile << 8 | slot of V << 2 | parity << 1 | tile, or -1.
          int j = 0, x = 0, due0 = -1, due1 = -1;
          auto seek = [&]() {  // on to the next turn
            while (j < kn) {
              const int key0 = (j < front ? j : j - front + first) * kWtKeys;
              if (x == 0 && b0.touches(key0, a.sinks)) return;
              if (x == 1 && b1.touches(key0, a.sinks)) return;
              if (++x == 2) {
                x = 0;
                ++j;
                ring.template next<kSlots>();
                ring.template next<kSlots>();
              }
            }
          };
          seek();
          while (ok && (j < kn || due0 >= 0 || due1 >= 0)) {
            int mine = -1;
            // K of key tile j takes the slot of V of the one three before (5 slots)
            if (j < kn && (due0 < 0 || (due0 >> 8) >= j - 2)) {
              // S = Q K^T once the buffer's last S is in registers.  Descriptor
              // addresses count 16 bytes: + 2 the next 16 elements of a 128-byte row
              const int buf = Cfg::kBufs == 1 ? 0 : x;
              const uint32_t n = (ns >> (8 * x)) & 7, last = Cfg::kBufs == 1 ? (uint32_t)turns - 1 : n - 1;
              ok = wait(full + ring.slot, ring.parity) && (!((used >> buf) & 1) || wait(s_free + buf, last & 1));
              if (!ok) break;
              tc_fence_after();
              const uint64_t qb = qd + (uint32_t)(x * (Cfg::kTile >> 4)), kb = kd + (uint32_t)(ring.slot * (Cfg::kTile >> 4));
#pragma unroll
              for (int kk = 0; kk < HD / 16; ++kk) {
                const uint32_t off = (kk >> 2) * (Cfg::kSlab >> 4) + (kk & 3) * 2;
                tc_mma_bf16(tmem + buf * 128, qb + off, kb + off, idesc_s, kk > 0 ? 1u : 0u);
              }
              tc_commit(s_full + 4 * x + (n & 3));
              ns = (ns & ~(0xffu << (8 * x))) | (((n + 1) & 7) << (8 * x));
              used |= 1u << buf;
              ++turns;
              WtSlot v = ring;
              v.template next<kSlots>();
              mine = j << 8 | v.slot << 2 | (int)v.parity << 1 | x;
              if (++x == 2) {
                x = 0;
                ++j;
                ring.template next<kSlots>();
                ring.template next<kSlots>();
              }
              seek();
            }
            if (single) {  // P V of the turn before
              due0 = due1;
              due1 = -1;
            }
            if (due0 >= 0) {
              // O += P V, a half of the keys as soon as its P is there: 16 keys are 8
              // columns of P and 16 rows (2048 bytes) of V
              const int y = due0 & 1, slot = (due0 >> 2) & 63;
              const uint32_t n = (np >> (8 * y)) & 7;
              ok = wait(full + slot, (due0 >> 1) & 1);
              const uint64_t vb = vd + (uint32_t)(slot * (Cfg::kTile >> 4));
              const uint32_t po = tmem + Cfg::kColO + y * HD, pp = tmem + Cfg::kColP + y * 64;
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                ok = ok && wait(p_full + 2 * y + h, n & 1);
                if (!ok) break;
                tc_fence_after();
#pragma unroll
                for (int kk = h * 4; kk < h * 4 + 4; ++kk)
                  tc_mma_bf16_ts(po, pp + kk * 8, vb + kk * (2048 >> 4), idesc_pv, kk > 0 ? 1u : (((fresh >> y) & 1) ^ 1));
              }
              if (!ok) break;
              fresh &= ~(1u << y);
              tc_commit(pv_done + 4 * y + (n & 3));
              np = (np & ~(0xffu << (8 * y))) | (((n + 1) & 7) << (8 * y));
            }
            due0 = due1;
            due1 = mine;
          }
        }
        mbar_arrive(&piece_empty[it & 1]);
      }
      tc_commit(drain);
      mbar_wait_drain(drain, 0);
    }
  } else if (!kSplit || warp < 6) {
    // ------------------------------ softmax, output ------------------------------
    // Every wait's outcome is made warp-uniform: the accesses to tensor memory are
    // warp-collective.
    const int x = kSplit ? 0 : (warp - 2) >> 2;    // tile
    const int r = (warp & 3) * 32 + lane;          // row of the tile = lane of tensor memory
    const uint32_t t_lane = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const float sc = a.scale_log2;
    bool ok = true;
    int c = 0;  // key tiles begun, over all pieces
    auto all_wait = [&](uint64_t* bar, uint32_t parity) -> bool {
      return __all_sync(0xffffffffu, wait(bar, parity));
    };
    // P V of the key tile before the c-th has completed
    auto last_pv_done = [&](int c) -> bool { return c < 2 || all_wait(&pv_done[4 * x + ((c - 2) & 3)], ((c - 2) >> 2) & 1); };
    auto hand_over = [&](int half) {
      if (lane == 0) mbar_arrive(&p_full[2 * x + half]);
    };
    for (int it = 0; ok; ++it) {
      if (!__all_sync(0xffffffffu, have_piece(it))) break;
      volatile WtPiece& p = pieces[it & 1];
      if (p.n < 0) break;
      const bool live = (warp & 3) * 32 < p.band[x].rows;  // warp-uniform
      float m_used = -INFINITY, l = 0.f;
      const int c_before = c;
      for (int j = 0; j < p.n; ++j) {
        const int key0 = p.key0(j);
        if (!p.band[x].touches(key0, a.sinks)) continue;
        const int bar = 4 * x + (c & 3), parity = (c >> 2) & 1;
        ++c;
        if (ok && !all_wait(&s_full[bar], parity)) ok = false;
        if (!live || !ok) {
          // rows past the sequence: keep the counts only, and no earlier than the
          // others could (S runs a turn ahead: a warp that handed over at S alone
          // would complete the phase of a P that its neighbours still write)
          if (lane == 0) mbar_arrive(&s_free[Cfg::kBufs == 1 ? 0 : x]);
          if (ok && !last_pv_done(c)) ok = false;
          hand_over(0);
          hand_over(1);
          continue;
        }
        uint32_t sv[128];
        tc_fence_after();
        tmem_ld128(t_lane + (Cfg::kBufs == 1 ? 0 : x * 128), sv);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s_free[Cfg::kBufs == 1 ? 0 : x]);
        if (!p.band[x].whole(key0, a.sinks)) {
          const WaSeq s{p.s.q0, p.s.nq, p.s.k0, p.s.nk};
          const WaRange rr = wa_range(a, s, p.i0 + ((!pair_heads && x) ? kWtRows : 0) + min(r, p.band[x].rows - 1));
          const int hi = rr.hi - key0, lo = rr.lo - key0, sk = a.sinks - key0;
#pragma unroll
          for (int g = 0; g < 128; g += 32) {  // a bit per key
            const uint32_t seen = bits_below(hi + 1 - g) & (~bits_below(lo - g) | bits_below(sk - g));
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (!((seen >> e) & 1u)) sv[g + e] = 0xff800000u;  // -inf
          }
        }
        float mx[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          mx[e] = max3(__uint_as_float(sv[e]), __uint_as_float(sv[4 + e]), __uint_as_float(sv[8 + e]));
#pragma unroll
        for (int e = 12; e < 124; e += 8)
#pragma unroll
          for (int u = 0; u < 4; ++u) mx[u] = max3(mx[u], __uint_as_float(sv[e + u]), __uint_as_float(sv[e + 4 + u]));
#pragma unroll
        for (int u = 0; u < 4; ++u) mx[u] = fmaxf(mx[u], __uint_as_float(sv[124 + u]));
        const float mj = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * sc;  // -inf: no key seen
        if (m_used == -INFINITY) m_used = mj;  // nothing accumulated yet
        const bool grow = mj > m_used + kAtcLazy;
        if (__any_sync(0xffffffffu, grow)) {
          const float alpha = grow ? ex2_approx(m_used - mj) : 1.f;
          l *= alpha;
          if (grow) m_used = mj;
          if (last_pv_done(c)) {
            tc_fence_after();
#pragma unroll 1
            for (int k = 0; k < HD / 16; ++k) {
              float o16[16];
              tmem_ld16(t_lane + Cfg::kColO + x * HD + k * 16, o16);
#pragma unroll
              for (int e = 0; e < 16; ++e) o16[e] *= alpha;
              tmem_st16(t_lane + Cfg::kColO + x * HD + k * 16, o16);
            }
          }
        }
        const float nm = m_used == -INFINITY ? 0.f : -m_used;
        const uint64_t sc2 = f32x2(__float_as_uint(sc), __float_as_uint(sc)), nm2 = f32x2(__float_as_uint(nm), __float_as_uint(nm));
        uint32_t pk[64];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            float p0, p1;
            f32x2_parts(fma2(f32x2(sv[k * 32 + 2 * e], sv[k * 32 + 2 * e + 1]), sc2, nm2), p0, p1);
            pk[k * 16 + e] = pack_bf16x2(ex2_approx(p0), ex2_approx(p1));
          }
          if (k == 0) {
            // P is free once the last P V has completed: looked at after the first
            // exponentials, by when it mostly has
            if (!last_pv_done(c)) ok = false;
            tc_fence_after();
          }
          tmem_st16_nowait(t_lane + Cfg::kColP + x * 64 + k * 16, pk + k * 16);
          if (k & 1) {
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            hand_over(k >> 1);
          }
        }
        // the sum of what the tensor cores multiply, while they do
        uint64_t rs[2] = {0, 0};
#pragma unroll
        for (int e = 0; e < 64; ++e) rs[e & 1] = add2(rs[e & 1], f32x2(pk[e] << 16, pk[e] & 0xffff0000u));
        float s0, s1;
        f32x2_parts(add2(rs[0], rs[1]), s0, s1);
        l += s0 + s1;
      }
      if (kSplit && p.parts > 1) {
        // A part of the keys: (m, l) and O go to the workspace; the last part's CTA to
        // get there joins them, in the order of the parts.
        const int rows = p.band[0].rows, parts = p.parts, parity = p.joins & 1;
        float* unit0 = a.partial + (int64_t)p.unit * splits * Cfg::kSlotFloats;
        float* slot = unit0 + (int64_t)p.part * Cfg::kSlotFloats;
        if (ok && !last_pv_done(c + 1)) ok = false;
        if (live && ok) {
          tc_fence_after();
          if (r < rows) __stcg(reinterpret_cast<float2*>(slot) + r, make_float2(m_used, l));
#pragma unroll 1
          for (int k = 0; k < HD / 32; ++k) {
            uint32_t o[32];
            tmem_ld32(t_lane + Cfg::kColO + k * 32, o);
            if (r < rows)
#pragma unroll
              for (int u = 0; u < 8; ++u)
                __stcg(reinterpret_cast<uint4*>(slot + 256 + r * HD + k * 32) + u,
                       make_uint4(o[4 * u], o[4 * u + 1], o[4 * u + 2], o[4 * u + 3]));
          }
          tc_fence_before();
        }
        __threadfence();
        __syncwarp();
        if (lane == 0) mbar_arrive(part_out);
        if (warp == 2) {
          if (!all_wait(part_out, parity)) ok = false;
          if (lane == 0) {
            join_here = ticket_acq_rel(a.tickets + p.unit) == parts - 1;
            mbar_arrive(part_told);
          }
        }
        if (!all_wait(part_told, parity)) ok = false;
        if (ok && join_here) {
          if (warp == 2 && lane == 0) a.tickets[p.unit] = 0;
          constexpr int kE = HD / 32;  // a row a warp, kE columns a lane; four rows and four parts at once
          const WaSeq s{p.s.q0, p.s.nq, p.s.k0, p.s.nk};
#pragma unroll 1
          for (int r0 = (warp & 3) * 4; r0 < rows; r0 += 16) {
            float mm[4], ll[4] = {}, acc[4][kE] = {};
#pragma unroll
            for (int u = 0; u < 4; ++u) mm[u] = -INFINITY;
#pragma unroll 1
            for (int k0 = 0; k0 < parts; k0 += 4) {
              float2 w[4][4];
              float v[4][4][kE];
#pragma unroll
              for (int k = 0; k < 4; ++k)
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                  w[k][u] = make_float2(-INFINITY, 0.f);
#pragma unroll
                  for (int e = 0; e < kE; ++e) v[k][u][e] = 0.f;
                  if (k0 + k < parts && r0 + u < rows) {
                    const float* from = unit0 + (int64_t)(k0 + k) * Cfg::kSlotFloats;
                    w[k][u] = __ldcg(reinterpret_cast<const float2*>(from) + r0 + u);
                    from += 256 + (r0 + u) * HD + lane * kE;
                    if constexpr (kE == 4)
                      *reinterpret_cast<float4*>(v[k][u]) = __ldcg(reinterpret_cast<const float4*>(from));
                    else
                      *reinterpret_cast<float2*>(v[k][u]) = __ldcg(reinterpret_cast<const float2*>(from));
                  }
                }
#pragma unroll
              for (int u = 0; u < 4; ++u) {
                const float mn = fmaxf(fmaxf(mm[u], fmaxf(w[0][u].x, w[1][u].x)), fmaxf(w[2][u].x, w[3][u].x));
                const float f0 = mm[u] == -INFINITY ? 0.f : ex2_approx(mm[u] - mn);
                mm[u] = mn;
                ll[u] *= f0;
#pragma unroll
                for (int e = 0; e < kE; ++e) acc[u][e] *= f0;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  const float f = w[k][u].x == -INFINITY ? 0.f : ex2_approx(w[k][u].x - mn);
                  ll[u] = fmaf(f, w[k][u].y, ll[u]);
#pragma unroll
                  for (int e = 0; e < kE; ++e) acc[u][e] = fmaf(f, v[k][u][e], acc[u][e]);
                }
              }
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              if (r0 + u >= rows) break;
              bool fine = true;
              const float inv = ll[u] == 0.f ? 0.f : 1.f / ll[u];
              uint32_t h[kE / 2];
#pragma unroll
              for (int e = 0; e < kE; e += 2) {
                fine = fine && fabsf(acc[u][e]) <= 3.0e38f && fabsf(acc[u][e + 1]) <= 3.0e38f;
                h[e / 2] = inv == 0.f ? 0u : pack_bf16x2(acc[u][e] * inv, acc[u][e + 1] * inv);
              }
              const int i = p.i0 + r0 + u;
              uint32_t* out = reinterpret_cast<uint32_t*>(reinterpret_cast<__nv_bfloat16*>(a.o) +
                                                          (int64_t)(s.q0 + i) * a.o_stride + p.head0 * HD + lane * kE);
              if constexpr (kE == 4) *reinterpret_cast<uint2*>(out) = make_uint2(h[0], h[1]); else *out = h[0];
              if (__any_sync(0xffffffffu, !fine && ll[u] > 0.f)) {
                if (lane == 0) atomicAdd(const_cast<int*>(&redoing), 1);
                wa_row_exact<__nv_bfloat16, HD>(a, s, i, p.head0);
                __syncwarp();
                if (lane == 0) atomicSub(const_cast<int*>(&redoing), 1);
              }
            }
          }
        }
      } else if (live) {
        const int rows = p.band[x].rows, i_tile = p.i0 + ((!pair_heads && x) ? kWtRows : 0);
        const int head = p.head0 + (pair_heads ? x : 0);
        const WaSeq s{p.s.q0, p.s.nq, p.s.k0, p.s.nk};
        if (c > c_before && ok && !last_pv_done(c + 1)) ok = false;
        const bool some = ok && c > c_before && l != 0.f;  // l NaN: so is the row
        const float inv = some ? 1.f / l : 0.f;
        bool fine = true;
        // whole sectors a store where rows begin at 32 bytes (ragged prompts: 56 us, with 16-byte stores 60)
        const bool wide = ((reinterpret_cast<uintptr_t>(a.o) | (uintptr_t)(a.o_stride * 2)) & 31) == 0;
        __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(a.o) + (int64_t)(s.q0 + i_tile + r) * a.o_stride + head * HD;
#pragma unroll 1
        for (int k = 0; k < HD / 32; ++k) {
          uint32_t o[32];
          if (ok && c > c_before) {
            tc_fence_after();
            tmem_ld32(t_lane + Cfg::kColO + x * HD + k * 32, o);
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = 0;
          }
          uint32_t h[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float v0 = __uint_as_float(o[2 * e]), v1 = __uint_as_float(o[2 * e + 1]);
            fine = fine && fabsf(v0) <= 3.0e38f && fabsf(v1) <= 3.0e38f;
            h[e] = some ? pack_bf16x2(v0 * inv, v1 * inv) : 0u;
          }
          if (r < rows) {
            if (wide) {
#pragma unroll
              for (int u = 0; u < 2; ++u)
                asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(out + k * 32 + u * 16), WT_R4(h, u * 8),
                             WT_R4(h, u * 8 + 4)
                             : "memory");
            } else {
#pragma unroll
              for (int u = 0; u < 4; ++u)
                reinterpret_cast<uint4*>(out + k * 32)[u] = make_uint4(h[4 * u], h[4 * u + 1], h[4 * u + 2], h[4 * u + 3]);
            }
          }
        }
        tc_fence_before();  // before the hand-over of the next piece's first P, which lets its P V write O
        uint32_t redo = __ballot_sync(0xffffffffu, ok && !fine && l > 0.f && r < rows);
        __syncwarp();
        if (redo) {
          if (lane == 0) atomicAdd(const_cast<int*>(&redoing), 1);
          while (redo) {
            const int e = __ffs(redo) - 1;
            redo &= redo - 1;
            wa_row_exact<__nv_bfloat16, HD>(a, s, i_tile + (warp & 3) * 32 + e, head);
          }
          __syncwarp();
          if (lane == 0) atomicSub(const_cast<int*>(&redoing), 1);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&piece_empty[it & 1]);
    }
  }

  __syncthreads();
  if (threadIdx.x == 0 && *abort_flag) set_status(a.status, ST_WAIT_TIMEOUT);
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

#undef WT_O4
#undef WT_O16
#undef WT_E4
#undef WT_E16
#undef WT_E64
#undef WT_R4

}  // namespace dinfer
