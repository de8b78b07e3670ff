// The shared keys of dinfer_kv_prefix_attention in bf16 on the tcgen05 tensor cores.
//
// A unit of work is a key head of a group and up to 256 of the rows that read it
// (members * heads / kv_heads queries), two tiles of 128; its keys come in tiles of 128.
// The tiles of all units, end to end, are split evenly over the CTAs, one an SM; a
// unit's part in a CTA is a segment, whose sums (m, l, O) go to the workspace and are
// joined with the others and the entry's own keys' by kv_join_kernel.
//
// By its floor HBM-bound up to some 230 rows: a key tile of K and V, 64 KB at head_dim 128, takes
// 2800 cycles of an SM's share of the bandwidth, its products for 256 rows some 3100
// cycles of the tensor cores.  What stands between is the chain S, softmax, P V of a
// tile, which takes longer, so two of them run at a time (streams): the two tiles of rows
// on the same keys, or, of a unit of at most 128 rows, one tile of rows on every other
// key tile each, with sums of their own.  Measured 2.7 us for 128 keys of 256 rows at head_dim 128 and 1.7 us
// at 64, 1.8 and 1.2 us of 64 rows; tensor cores 42% and issue slots 41% busy with 96 sequences in three
// groups, 64 heads of 64 on 8.  352 threads:
//   warp 0      the key tiles: page numbers, a tile ahead, and a TMA box per page and 64
//               columns, a page a lane; a page that is not there is asked for behind the
//               last one, which reads as zeros, and its keys are missing from the tile's
//               mask.  Pages that do not divide a tile, or it them, go by 16-byte
//               cp.async from warps 0 and 1
//   warp 2      tensor memory and the products, S_0 S_1 S_2 P_0 V S_3 P_1 V ..., whichever of S
//               and P V can go
//   warps 3-6   queries, softmax and sums of stream 0, a thread per row; warps 7-10 stream 1
// A weight goes through P V as two bf16, cut off and the rest, as in kv_attention_kernel:
// 2^-16 of it is lost (with one bf16, 2^-9: 2.1 and 1.6 us for 256 rows).  P so fills the
// 128 columns of the S that it is made of, which has been read when it is written.  There are
// two such places, at head_dim 64 three, which the turns of both streams take in order (with
// two at 64 the call above 102 us, with three 86).  P's two halves and the lazily raised
// maximum are as in window_attention_tc.cuh.
#pragma once
#include "kv_prefix.cuh"
#include "window_attention_tc.cuh"

namespace dinfer {

constexpr int kPtThreads = 352;
constexpr int kPtLoaders = 64;
constexpr int kPtAhead = 3;  // key or value tiles in flight behind the one being asked for

template <int HD>
struct PtCfg {
  static constexpr int kSlab = 128 * 128;           // 128 rows x 64 bf16
  static constexpr int kTile = 128 * HD * 2;
  static constexpr int kSlots = HD == 128 ? 5 : 8;  // K and V tiles
  static constexpr int kOffRing = 2 * kTile;        // behind Q
  static constexpr int kOffBar = kOffRing + kSlots * kTile;
  static constexpr int kSmem = 1024 + kOffBar + 512;
  static constexpr int kBufs = HD == 128 ? 2 : 3;   // places of S and P
  static constexpr int kColO = kBufs * 128;
};
static_assert(PtCfg<128>::kSmem + 512 <= 232448, "prefix attention shared memory above 227 KB");

struct PtMaps {
  CUtensorMap k, v;  // of one layer: [pages][heads][slots][hd], boxes of a page's slots (at most 128) x 64 elements
};
struct PtArgs {
  KpArgs p;
  DevState* status;
  int tile_pages;  // pages of a tile (1: a page is whole tiles)
};

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, uint64_t* bar, int x, int y, int z, int w) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_u32(bar))
      : "memory");
}

// The segments of a CTA's places [x0, x1), in order.
struct PtWalk {
  KpEntry gr;
  int g, u;              // group, unit of it
  int from, to, base;    // key tiles of the segment; the unit's first place
  int x1;
  __device__ __forceinline__ bool set(int x0) {
    from = max(0, x0 - base - kPtCost);
    to = min(gr.tiles(), x1 - base - kPtCost);
    return to > from;
  }
  __device__ __forceinline__ bool start(const KpArgs& p, int x0, int end) {
    x1 = end;
    int lo = 0, hi = p.groups;  // unit0[lo] <= x0 < unit0[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (__ldcg(&p.plan[mid].unit0) <= x0) lo = mid; else hi = mid;
    }
    g = lo;
    gr = kp_entry(p, g);
    u = (int)((unsigned)(x0 - gr.unit0) / (unsigned)gr.size());
    base = gr.unit0 + u * gr.size();
    return set(x0);
  }
  __device__ __forceinline__ bool next(const KpArgs& p) {
    base += gr.size();
    if (base >= x1) return false;
    if (++u == p.a.c.kv_heads * gr.pairs()) {
      u = 0;
      do gr = kp_entry(p, ++g);
      while (gr.shared == 0);  // there is one more: base is below the end
    }
    return set(base);
  }
  __device__ __forceinline__ int kvh() const { return u / gr.pairs(); }
  __device__ __forceinline__ int row0() const { return u % gr.pairs() * 256; }  // of the group's
  __device__ __forceinline__ int rows() const { return min(256, gr.rows - row0()); }
};

template <int HD, bool kTma>
__global__ void __launch_bounds__(kPtThreads, 1)
    kv_prefix_tc_kernel(const __grid_constant__ PtMaps maps, const __grid_constant__ PtArgs pa) {
  using Cfg = PtCfg<HD>;
  constexpr int kSlots = Cfg::kSlots;
  const KpArgs& p = pa.p;
  const KaArgs& a = p.a;
  const KvPages& c = a.c;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + Cfg::kOffBar);  // [kSlots]
  // A stream's n-th product completes phase n / 4 of barrier n % 4 (see window_tc_kernel).
  uint64_t* s_full = full + kSlots;   // [2 streams][4]
  uint64_t* pv_done = s_full + 8;     // [2 streams][4]
  uint64_t* p_full = pv_done + 8;     // [2 streams][2 halves of 64 keys]
  uint64_t* q_full = p_full + 4;      // a segment's queries
  uint64_t* drain = q_full + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  uint32_t* masks = tmem_slot + 2;    // [8 key tiles][4]: keys that are there
  static_assert((kSlots + 8 + 8 + 4 + 2) * 8 + 8 + 128 <= 512, "barriers");
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < kSlots; ++i) mbar_init(&full[i], kTma ? 1 : kPtLoaders);
    for (int i = 0; i < 8; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&pv_done[i], 1);
    }
    for (int i = 0; i < 4; ++i) mbar_init(&p_full[i], 4);
    mbar_init(q_full, 8);
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
    if (kTma) {
      prefetch_tmap(&maps.k);
      prefetch_tmap(&maps.v);
    }
  }
  if (warp == 2) tmem_alloc(tmem_slot, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();
  pdl_trigger();  // the own kernel may begin: what it reads is there
  const int4 head = __ldcg(p.head);
  KaSplit split;
  kp_split(p, head, split);
  PtWalk w;
  bool any = head.y > 0 && blockIdx.x < split.ctas;
  if (any) any = w.start(p, split.begin(blockIdx.x), split.begin(blockIdx.x + 1));

  // Bounded; a wait that ran out sets the status at the kernel's end.
  auto wait = [&](uint64_t* bar, uint32_t parity) -> bool { return mbar_wait(bar, parity, abort_flag); };

  if (!any) {
  } else if (warp < 2) {
    // ------------------------------ keys ------------------------------
    int hist[kSlots];  // what read the last kSlots tiles, oldest first: V << 2 | streams, then their products' numbers
#pragma unroll
    for (int i = 0; i < kSlots; ++i) hist[i] = 0;
    int n[2] = {0, 0};   // products of each stream over the tiles loaded
    WtSlot at{0, 0}, told{0, 0};
    int key_tiles = 0, loads = 0;
    bool ok = true;
    auto took = [&](int kv, int streams) {
      at.template next<kSlots>();
      ++loads;
#pragma unroll
      for (int i = 0; i + 1 < kSlots; ++i) hist[i] = hist[i + 1];
      hist[kSlots - 1] = (kv << 2) | streams | (n[0] & 7) << 3 | (n[1] & 7) << 6;
    };
    // The slot's last tile has been read by the products of both streams; before(): in front of a wait that may last
    auto wait_free = [&](auto before) {
      const int use = hist[0];
#pragma unroll
      for (int x = 0; x < 2; ++x)
        if ((use >> x) & 1) {
          const int m = (use >> (3 + 3 * x)) & 7;
          uint64_t* bar = ((use & 4) ? pv_done : s_full) + 4 * x + (m & 3);
          if (!mbar_try_wait(bar, (m >> 2) & 1)) {
            before();
            ok = ok && wait(bar, (m >> 2) & 1);
          }
        }
      ok = __all_sync(0xffffffffu, ok);  // warp-uniform, also where a wait ran out
    };
    if constexpr (kTma) {
      if (warp == 0) {
        const int pages = pa.tile_pages, slots = 128 / pages;  // of a tile; keys of a box
        do {
          const bool pair = w.rows() > 128;
          const int kvh = w.kvh();
          const int32_t* table = c.table + (size_t)w.gr.leader * c.max_pages;
          // a lane's page of a tile, and where in it the tile begins; page -1: no such key
          auto look_up = [&](int tile, int& page, int& slot) {
            const int key = tile * 128 + lane * slots;
            page = -1;
            slot = 0;
            if (lane < pages && tile < w.to && key < w.gr.shared) {
              const int j = (int)c.page_div.div((uint32_t)key);
              page = table[j];
              slot = key - j * c.page_size;
              if (page < 0 || page >= c.num_pages) {
                c.flag(KV_BAD_PAGE);
                page = -1;
              }
            }
          };
          int page, slot, page_next, slot_next;
          look_up(w.from, page, slot);
          for (int j = w.from; j < w.to && ok; ++j, ++key_tiles) {
            const uint32_t there = __ballot_sync(0xffffffffu, page >= 0);
            const int from = page >= 0 ? page : c.num_pages, slot0 = slot;
            look_up(j + 1, page_next, slot_next);
            const int streams = pair ? 3 : 1 << ((j - w.from) & 1);
#pragma unroll
            for (int kv = 0; kv < 2; ++kv) {
              wait_free([] {});
              if (!ok) break;
              uint64_t* bar = full + at.slot;
              if (kv == 0 && lane < 4) {
                uint32_t mask = 0;
#pragma unroll
                for (int b = 0; b < 4; ++b) mask |= (there >> ((lane * 32 + b * 8) / slots)) & 1u ? 0xffu << (8 * b) : 0u;
                masks[(key_tiles & 7) * 4 + lane] = mask;
              }
              __syncwarp();
              if (lane == 0) mbar_arrive_expect_tx(bar, Cfg::kTile);
              __syncwarp();
              if (lane < pages) {
                const uint32_t dst = smem_u32(sm) + Cfg::kOffRing + at.slot * Cfg::kTile + lane * slots * 128;
#pragma unroll
                for (int h = 0; h < HD / 64; ++h)
                  tma_load_4d(dst + h * Cfg::kSlab, kv ? &maps.v : &maps.k, bar, h * 64, slot0, kvh, from);
              }
              took(kv, streams);
            }
            n[0] += streams & 1;
            n[1] += streams >> 1;
            page = page_next;
            slot = slot_next;
          }
        } while (ok && w.next(p));
        if (*abort_flag)  // let the copies in flight land before the CTA exits
          for (int j = max(0, loads - kSlots); j < loads; ++j) mbar_wait_drain(&full[j % kSlots], (j / kSlots) & 1);
      }
    } else {
      int pending = 0;  // tiles asked for and not announced
      auto announce = [&]() {
        fence_async_shared();
        mbar_arrive(&full[told.slot]);
        told.template next<kSlots>();
        --pending;
      };
      auto flush = [&]() {
        cp_async_wait<0>();
        while (pending > 0) announce();
      };
      do {
        const bool pair = w.rows() > 128;
        const int kvh = w.kvh();
        const int32_t* table = c.table + (size_t)w.gr.leader * c.max_pages;
        // keys warp * 64 + lane and + 32 of a tile
        auto look_up = [&](int tile, int64_t (&off)[2], int (&page)[2]) {
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const int key = tile * 128 + warp * 64 + u * 32 + lane;
            off[u] = -1;
            page[u] = 0;
            if (tile < w.to && key < w.gr.shared) {
              const int j = (int)c.page_div.div((uint32_t)key);
              page[u] = table[j];
              off[u] = a.layer_off + (key - j * c.page_size) * c.token_stride + kvh * c.head_stride;
            }
          }
        };
        int64_t off[2], off_next[2];
        int page[2], page_next[2];
        look_up(w.from, off, page);
        for (int j = w.from; j < w.to && ok; ++j, ++key_tiles) {
          int64_t place[2];
          uint32_t there[2];
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            place[u] = -1;
            if (off[u] >= 0) {
              if (page[u] >= 0 && page[u] < c.num_pages) place[u] = off[u] + page[u] * c.page_stride;
              else c.flag(KV_BAD_PAGE);
            }
            there[u] = __ballot_sync(0xffffffffu, place[u] >= 0);
          }
          look_up(j + 1, off_next, page_next);
          const int streams = pair ? 3 : 1 << ((j - w.from) & 1);
#pragma unroll
          for (int kv = 0; kv < 2; ++kv) {
            // what is in flight is announced before a wait: the products that free the slot may need it
            wait_free(flush);
            if (!ok) break;
            if (kv == 0 && lane < 2) masks[(key_tiles & 7) * 4 + warp * 2 + lane] = lane ? there[1] : there[0];
            const uint4* from = kv ? c.v : c.k;
            const uint32_t dst0 = smem_u32(sm) + Cfg::kOffRing + at.slot * Cfg::kTile;
#pragma unroll 8
            for (int k = 0; k < 16; ++k) {
              const int r = k * 4 + (lane >> 3);  // of this warp's 64 keys
              const int64_t at_key = __shfl_sync(0xffffffffu, k < 8 ? place[0] : place[1], r & 31);
              const int row = warp * 64 + r;
              const uint4* src = from + (at_key >= 0 ? at_key : 0) + (lane & 7);
              const uint32_t dst = dst0 + row * 128 + (((lane & 7) ^ (row & 7)) << 4);
#pragma unroll
              for (int h = 0; h < HD / 64; ++h) cp_async16(dst + h * Cfg::kSlab, src + h * 8, at_key >= 0 ? 16 : 0);
            }
            cp_async_commit();
            ++pending;
            took(kv, streams);
            if (pending > kPtAhead) {
              cp_async_wait<kPtAhead>();
              announce();
            }
          }
          n[0] += streams & 1;
          n[1] += streams >> 1;
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            off[u] = off_next[u];
            page[u] = page_next[u];
          }
        }
      } while (ok && w.next(p));
      flush();
    }
  } else if (warp == 2) {
    // ------------------------------ products ------------------------------
    if (elect_one_sync()) {
      constexpr uint32_t idesc_s = make_idesc_bf16(128, 128);
      constexpr uint32_t idesc_pv = make_idesc_bf16(128, HD) | (1u << 16);  // B (V) MN-major
      const uint64_t qd = make_sw128_desc(smem_u32(sm));
      const uint64_t kd = make_sw128_desc(smem_u32(sm + Cfg::kOffRing));
      const uint64_t vd = make_sw128_desc_mn(smem_u32(sm + Cfg::kOffRing), Cfg::kSlab);
      uint32_t ns = 0, np = 0;  // products issued, 8 bits for each stream (see window_tc_kernel)
      int held[Cfg::kBufs];     // the last turns, oldest first: 4 n + x, the n-th of stream x; -1: none yet
#pragma unroll
      for (int i = 0; i < Cfg::kBufs; ++i) held[i] = -1;
      int buf = 0;              // place of the next S
      WtSlot ring{0, 0};        // K of the key tile at hand
      bool ok = true;
      for (int seg = 0;; ++seg) {
        const bool pair = w.rows() > 128;
        ok = wait(q_full, seg & 1);
        const int last = pair ? 2 * (w.to - w.from) : w.to - w.from;
        uint32_t fresh = 3;  // bit x: no P V of this segment yet
        // The turns whose P V is due, oldest first.  S of the next turn goes first where its keys and a place are there, up to
        // two turns ahead of P V; else P V, whose V makes room for other keys.  (In the order S_t, P_t-2 V without a look: a
        // unit of 32 rows over 8192 keys took 1.75 us a key tile, the latency of its loads.)
        int due[3] = {-1, -1, -1}, waiting = 0;
        for (int t = 0; ok && (t < last || waiting > 0);) {
          const int x = t & 1;
          const uint32_t n_s = (ns >> (8 * x)) & 7;
          const int prev = held[0];  // its P V makes room
          uint64_t* prev_done = pv_done + 4 * (prev & 1) + ((prev >> 2) & 3);
          bool go = t < last && waiting == 0;
          if (go) {
            ok = wait(full + ring.slot, ring.parity) && (prev < 0 || wait(prev_done, (prev >> 4) & 1));
          } else if (t < last && waiting < 3) {  // whichever can go first
            const int y = due[0] & 1;
            const long long t0 = clock64();
            while (true) {
              go = mbar_test(full + ring.slot, ring.parity) && (prev < 0 || mbar_test(prev_done, (prev >> 4) & 1));
              if (go || mbar_test(p_full + 2 * y, (np >> (8 * y)) & 1)) break;
              if (*abort_flag || clock64() - t0 > kWaitCycles) break;  // the wait below sees to it
            }
          }
          if (go) {
            if (!ok) break;
            tc_fence_after();
            const uint64_t qb = qd + (pair && x ? (uint32_t)(Cfg::kTile >> 4) : 0u), kb = kd + (uint32_t)(ring.slot * (Cfg::kTile >> 4));
#pragma unroll
            for (int kk = 0; kk < HD / 16; ++kk) {
              const uint32_t off = (kk >> 2) * (Cfg::kSlab >> 4) + (kk & 3) * 2;
              tc_mma_bf16(tmem + buf * 128, qb + off, kb + off, idesc_s, kk > 0 ? 1u : 0u);
            }
            tc_commit(s_full + 4 * x + (n_s & 3));
            ns = (ns & ~(0xffu << (8 * x))) | (((n_s + 1) & 7) << (8 * x));
#pragma unroll
            for (int i = 0; i + 1 < Cfg::kBufs; ++i) held[i] = held[i + 1];
            held[Cfg::kBufs - 1] = (int)n_s << 2 | x;
            ++t;
            WtSlot v = ring;
            v.template next<kSlots>();
            const int mine = v.slot << 4 | buf << 2 | (int)v.parity << 1 | x;
            buf = buf + 1 == Cfg::kBufs ? 0 : buf + 1;
            if (waiting == 0) due[0] = mine; else if (waiting == 1) due[1] = mine; else due[2] = mine;
            ++waiting;
            if (!pair || x) {
              ring.template next<kSlots>();
              ring.template next<kSlots>();
            }
          }
          if (ok && (waiting == 3 || (waiting > 0 && !go))) {
            const int y = due[0] & 1, slot = due[0] >> 4;
            const uint32_t n = (np >> (8 * y)) & 7;
            ok = wait(full + slot, (due[0] >> 1) & 1);
            const uint64_t vb = vd + (uint32_t)(slot * (Cfg::kTile >> 4));
            const uint32_t po = tmem + Cfg::kColO + y * HD, pp = tmem + ((due[0] >> 2) & 3) * 128;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              ok = ok && wait(p_full + 2 * y + h, n & 1);
              if (!ok) break;
              tc_fence_after();
#pragma unroll
              for (int kk = h * 4; kk < h * 4 + 4; ++kk)
#pragma unroll
                for (int part = 0; part < 2; ++part)  // cut off, the rest
                  tc_mma_bf16_ts(po, pp + (h + part) * 32 + kk * 8, vb + kk * (2048 >> 4), idesc_pv,
                                 kk + part > 0 ? 1u : (((fresh >> y) & 1) ^ 1));
            }
            if (!ok) break;
            fresh &= ~(1u << y);
            tc_commit(pv_done + 4 * y + (n & 3));
            np = (np & ~(0xffu << (8 * y))) | (((n + 1) & 7) << (8 * y));
            due[0] = due[1];
            due[1] = due[2];
            --waiting;
          }
        }
        if (!ok || !w.next(p)) break;
      }
      tc_commit(drain);
      mbar_wait_drain(drain, 0);
    }
  } else {
    // ------------------------------ softmax, sums ------------------------------
    // Every wait's outcome is made warp-uniform: the accesses to tensor memory are warp-collective.
    const int x = (warp - 3) >> 2;         // stream
    const int r = (warp & 3) * 32 + lane;  // row of the tile = lane of tensor memory
    const uint32_t t_lane = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const float sc = a.scale_log2;
    bool ok = true;
    int cnt = 0, other = 0, turns = 0, key_tiles = 0;  // turns of this stream, of the other one, of both, key tiles, over all segments
    auto all_wait = [&](uint64_t* bar, uint32_t parity) -> bool { return __all_sync(0xffffffffu, wait(bar, parity)); };
    // P V of the turn before the cnt-th has completed
    auto last_pv_done = [&](int cnt) -> bool { return cnt < 2 || all_wait(&pv_done[4 * x + ((cnt - 2) & 3)], ((cnt - 2) >> 2) & 1); };
    // behind the last turn's P V: a warp ahead of another one would arrive twice in a phase
    auto hand_over = [&](int half) {
      if (lane == 0) mbar_arrive(&p_full[2 * x + half]);
    };
    do {
      const bool pair = w.rows() > 128;
      const int tiles = w.to - w.from, rows = pair ? (x ? w.rows() - 128 : 128) : w.rows();
      const bool live = (warp & 3) * 32 < rows;  // warp-uniform
      {
        // The queries, eight lanes on 128 bytes of a row; rows that are not there are zeros.  Where both streams read one
        // tile, stream 0 fills it.  The last segment's S have all read what is written over.
        if (ok && other > 0 && !all_wait(&s_full[4 * (x ^ 1) + ((other - 1) & 3)], ((other - 1) >> 2) & 1)) ok = false;
        if (ok && (pair || x == 0)) {
          const int row0 = w.row0() + x * 128, kvh = w.kvh();
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int tile_row = (warp & 3) * 32 + i * 4 + (lane >> 3), row = row0 + min(tile_row, rows - 1);
            const int e = (int)p.group_div.div((uint32_t)row);
            const __nv_bfloat16* q = reinterpret_cast<const __nv_bfloat16*>(a.q) + (w.gr.e0 + e) * a.q_stride +
                                     (kvh * a.group + row - e * a.group) * HD + (lane & 7) * 8;
            const uint32_t dst = smem_u32(sm) + x * Cfg::kTile + tile_row * 128 + (((lane & 7) ^ (tile_row & 7)) << 4);
#pragma unroll
            for (int h = 0; h < HD / 64; ++h) cp_async16(dst + h * Cfg::kSlab, q + h * 64, tile_row < rows ? 16 : 0);
          }
          cp_async_commit();
          cp_async_wait<0>();
          fence_async_shared();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(q_full);
        other += pair ? tiles : (tiles + x) / 2;
      }
      float m_used = -INFINITY, l = 0.f;
      const int cnt_before = cnt;
      for (int j = pair ? 0 : x; j < tiles; j += pair ? 1 : 2) {
        const int bar = 4 * x + (cnt & 3), parity = (cnt >> 2) & 1;
        ++cnt;
        if (ok && !all_wait(&s_full[bar], parity)) ok = false;
        if (!live || !ok) {  // keep the counts only
          if (ok && !last_pv_done(cnt)) ok = false;
          hand_over(0);
          hand_over(1);
          continue;
        }
        uint32_t sv[128];
        tc_fence_after();
        const uint32_t t_sp = t_lane + (turns + (pair ? 2 * j + x : j)) % Cfg::kBufs * 128;
        tmem_ld128(t_sp, sv);
        const volatile uint32_t* mask = masks + ((key_tiles + j) & 7) * 4;
        const uint32_t m0 = mask[0], m1 = mask[1], m2 = mask[2], m3 = mask[3];
        if ((m0 & m1 & m2 & m3) != 0xffffffffu) {
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            const uint32_t there = g == 0 ? m0 : g == 1 ? m1 : g == 2 ? m2 : m3;
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (!((there >> e) & 1u)) sv[g * 32 + e] = 0xff800000u;  // -inf
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
        const float mj = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * sc;
        if (m_used == -INFINITY) m_used = mj;  // nothing accumulated yet
        const bool grow = mj > m_used + kAtcLazy;
        if (__any_sync(0xffffffffu, grow)) {
          const float alpha = grow ? ex2_approx(m_used - mj) : 1.f;
          l *= alpha;
          if (grow) m_used = mj;
          if (last_pv_done(cnt)) {
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
        const uint64_t minus = f32x2(__float_as_uint(-1.f), __float_as_uint(-1.f));
        uint64_t rs[2] = {0, 0};  // of the weights as they are
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint32_t pk[32];  // cut off, the rest
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            float p0, p1, r0, r1;
            f32x2_parts(fma2(f32x2(sv[k * 32 + 2 * e], sv[k * 32 + 2 * e + 1]), sc2, nm2), p0, p1);
            const uint32_t u0 = __float_as_uint(ex2_approx(p0)), u1 = __float_as_uint(ex2_approx(p1));
            const uint64_t w2 = f32x2(u0, u1);
            rs[e & 1] = add2(rs[e & 1], w2);
            pk[e] = __byte_perm(u0, u1, 0x7632);
            f32x2_parts(fma2(f32x2(u0 & 0xffff0000u, u1 & 0xffff0000u), minus, w2), r0, r1);
            pk[16 + e] = pack_bf16x2(r0, r1);
          }
          const uint32_t at = t_sp + (k >> 1) * 64 + (k & 1) * 16;
          tmem_st16_nowait(at, pk);
          tmem_st16_nowait(at + 32, pk + 16);
          if (k & 1) {
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (k == 1 && !last_pv_done(cnt)) ok = false;
            hand_over(k >> 1);
          }
        }
        float s0, s1;
        f32x2_parts(add2(rs[0], rs[1]), s0, s1);
        l += s0 + s1;
      }
      key_tiles += tiles;
      turns += pair ? 2 * tiles : tiles;
      // (m, l) and O of the segment; before the hand-over of the next one's first P, which lets its P V write O
      const int64_t row = (int64_t)kp_row(w.gr, w.kvh(), w.row0()) + 256 * blockIdx.x + (x ? (pair ? 128 : w.rows()) : 0) + r;
      if (cnt > cnt_before && ok && !last_pv_done(cnt + 1)) ok = false;
      if (live && ok) {
        tc_fence_after();
        if (r < rows) __stcg(p.seg_ml + row, make_float2(m_used, l));
        if (cnt > cnt_before) {
#pragma unroll 1
          for (int k = 0; k < HD / 32; ++k) {
            uint32_t o[32];
            tmem_ld32(t_lane + Cfg::kColO + x * HD + k * 32, o);
            if (r < rows)
#pragma unroll
              for (int u = 0; u < 4; ++u)  // whole sectors
                asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p.seg_o + row * HD + k * 32 + u * 8),
                             "r"(o[8 * u]), "r"(o[8 * u + 1]), "r"(o[8 * u + 2]), "r"(o[8 * u + 3]), "r"(o[8 * u + 4]),
                             "r"(o[8 * u + 5]), "r"(o[8 * u + 6]), "r"(o[8 * u + 7])
                             : "memory");
          }
        }
        tc_fence_before();
      }
      __syncwarp();
    } while (ok && w.next(p));
  }

  __syncthreads();
  if (tid == 0 && *abort_flag) set_status(pa.status, ST_WAIT_TIMEOUT);
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace dinfer
