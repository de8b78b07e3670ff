// Attention of one new token per sequence where groups of sequences share the pages
// of their first tokens (include/dinfer_kv.h, dinfer_kv_prefix_attention).
//
// softmax(scale q K^T) V over the shared keys and over a sequence's own ones are sums
// with a maximum each, (m, l, O), which join exactly, whatever the keys are cut into:
//   m = max m_i, l = sum 2^(m_i - m) l_i, O = sum 2^(m_i - m) O_i, o = O / l.
// So the shared keys are read once for all the rows of their group (members * heads /
// kv_heads queries per key head), the rest once per sequence.  Up to four kernels:
//   plan    one CTA: what each group shares, and how the work is dealt out
//   own     every sequence's own keys on mma.sync (fp32: FMAs), a warp for itself:
//           the steps of 32 (16) keys of all (entry, key head) pairs, end to end,
//           are split evenly over the warps, and a warp's part of a pair goes to
//           the workspace as it is.  (A pair to a CTA, its warps merged in shared
//           memory as in kv_attention_kernel, took 2 to 3 us a pair for 1 us of keys:
//           64 sequences of some 150 tokens of their own, 32 heads on 8: 30 us.)
//           In fp32, and where 16 rows hold all queries of a key head, the shared keys
//           are pairs of their own here, a piece of up to 16 (8) rows at a time
//   prefix  in bf16 the shared keys on the tensor cores (kv_prefix_tc.cuh), at the same
//           time: the plan deals the SMs to the two by what their work takes
//   join    a warp per row of the output
// All of it in a graph: 64 sequences behind 8192 tokens, 32 heads on 8 (66 MB) 34.8 us; 32 behind
// 8192 with 512 of their own, 16 heads on 16 (202 MB) 48.9 us, 4.1 TB/s.
#pragma once
#include "kv_attention.cuh"

namespace dinfer {

constexpr int kKjThreads = 256;
constexpr int kKpCost = 2;  // own: a pair's beginning and end, in steps
constexpr int kPtCost = 2;  // prefix: the same of a unit, in tiles of 128 keys

// What the plan says of an entry v: first the groups, then the call's entries, then the end.
struct alignas(16) KpEntry {
  int place0;       // own: steps (and costs) before it
  int first, keys;  // own: its keys
  int seq;          // the sequence whose table holds them
  // of its group (an entry of none: shared 0)
  int shared;       // tokens that it shares: whole pages
  int e0, rows;     // first entry; queries per key head
  int unit0;        // prefix: places before its units; or own: before its pairs
  int row0;         // prefix: rows of sums before its
  int leader;       // the sequence whose table is read
  int pad[2];
  __device__ __forceinline__ int tiles() const { return (shared + 127) / 128; }
  __device__ __forceinline__ int size() const { return tiles() + kPtCost; }  // places of a unit
  __device__ __forceinline__ int pairs() const { return (rows + 255) / 256; }  // units per key head
  // rows of sums per key head and CTA: a unit of at most 128 rows has two for each
  __device__ __forceinline__ int sums() const {
    const int last = rows - (pairs() - 1) * 256;
    return (pairs() - 1) * 256 + (last <= 128 ? 2 * last : last);
  }
};
static_assert(sizeof(KpEntry) == 48, "read as three int4");

struct KpArgs {
  KaArgs a;  // window -1
  const int32_t* bounds;  // [groups + 1] first entries; NULL: one group of all
  const int32_t* prefix;  // [groups]
  int groups;
  int with_prefix;        // the shared keys are pairs of the own kernel
  int sms, warps, keys, rows;  // of the own kernel: warps of a CTA, keys of a step, rows of a piece
  int step_ns, pair_ns, single_ns;  // what an SM takes for a step of the own kernel, a key tile of the prefix kernel
  FastDiv group_div;
  int4* head;     // steps of the own kernel, places of the prefix kernel, SMs of the own kernel
  KpEntry* plan;  // [groups + entries + 1]
  // sums: own, of the shared keys at row (entry * heads + head) of a group's piece order, of an entry's own ones
  // entries * heads on, and `rows` further for each warp
  float* own_o;
  float2* own_ml;
  float* seg_o;  // prefix: KpEntry::row0 and 256 further for each CTA
  float2* seg_ml;
};

__device__ __forceinline__ KpEntry kp_entry(const KpArgs& p, int v) {
  KpEntry r;
  const int4* from = reinterpret_cast<const int4*>(p.plan + v);
#pragma unroll
  for (int i = 0; i < 3; ++i) reinterpret_cast<int4*>(&r)[i] = __ldcg(from + i);
  return r;
}

// How the places of all units are dealt to the prefix kernel's CTAs.
__device__ __forceinline__ void kp_split(const KpArgs& p, const int4& head, KaSplit& split) {
  split.make(head.y, max(1, min(p.sms - head.z, head.y / (2 * kPtCost))));
}
// Where the sums of a unit's rows begin, for CTA 0 (each CTA's are 256 rows on: a unit has at most 256, and two CTAs
// share at most one).
__device__ __forceinline__ int kp_row(const KpEntry& g, int kvh, int row) { return g.row0 + kvh * g.sums() + row; }

// --------------------------------------------------------------------------
// plan
// --------------------------------------------------------------------------
// Exclusive sums of v's parts over the CTA's threads, whole warps; returns the totals.
__device__ __forceinline__ int4 kp_scan(int4& v) {
  __shared__ int4 warp_sums[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int4 own = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, v.x, o), y = __shfl_up_sync(0xffffffffu, v.y, o);
    const int z = __shfl_up_sync(0xffffffffu, v.z, o), w = __shfl_up_sync(0xffffffffu, v.w, o);
    if (lane >= o) v = make_int4(v.x + x, v.y + y, v.z + z, v.w + w);
  }
  if (lane == 31) warp_sums[warp] = v;
  __syncthreads();
  int4 all{};
  v = make_int4(v.x - own.x, v.y - own.y, v.z - own.z, v.w - own.w);
  for (int i = 0; i < warps; ++i) {
    const int4 s = warp_sums[i];
    if (i < warp) v = make_int4(v.x + s.x, v.y + s.y, v.z + s.z, v.w + s.w);
    all = make_int4(all.x + s.x, all.y + s.y, all.z + s.z, all.w + s.w);
  }
  return all;
}

__global__ void __launch_bounds__(kKvPlanThreads) kv_prefix_plan_kernel(const __grid_constant__ KpArgs p) {
  const KaArgs& a = p.a;
  const KvPages& c = a.c;
  __shared__ int bounds[kKvMaxEntries + 1], seqs[kKvMaxEntries];
  __shared__ int least[kKvMaxEntries], leader[kKvMaxEntries], live[kKvMaxEntries], unit0[kKvMaxEntries], row0[kKvMaxEntries];
  const int t = threadIdx.x, groups = p.groups, e = t - groups;
  const bool is_group = t < groups, is_entry = !is_group && e < a.n;
  pdl_wait();
  pdl_trigger();
  KpEntry r{};
  int len = 0, wanted = 0, s = 0;
  if (is_group) {
    bounds[t] = p.bounds ? p.bounds[t] : 0;
    if (t == groups - 1) bounds[groups] = p.bounds ? p.bounds[groups] : a.n;
    wanted = p.prefix[t];
    least[t] = leader[t] = 0x7fffffff;
    live[t] = 0;
  } else if (is_entry) {
    s = a.seqs ? a.seqs[e] : e;
    len = s >= 0 && s < c.max_seqs ? c.lens[s] : -1;
    if (!c.valid_len(len)) {
      c.flag(KV_BAD_SEQ);
      len = 0;
    }
    seqs[e] = s;
  }
  __syncthreads();
  const bool order = __syncthreads_and(!is_group || (bounds[t] >= 0 && bounds[t] <= bounds[t + 1] && bounds[t + 1] <= a.n));
  if (!order && t == 0) c.flag(KV_FULL);
  int g = -1;
  if (is_entry && order) {
    int lo = 0, hi = groups;  // the last group that begins at or before e
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (bounds[mid] <= e) lo = mid; else hi = mid;
    }
    if (e >= bounds[lo] && e < bounds[lo + 1] && len > 0) {
      g = lo;
      atomicMin(&least[g], len);
      atomicMin(&leader[g], e);
      atomicAdd(&live[g], 1);
    }
  }
  __syncthreads();
  int places = 0, units = 0, rows = 0, weight = 0;
  if (is_group && live[t] > 1) {
    r.shared = (int)c.page_div.div((uint32_t)max(0, min(wanted, least[t] - 1))) * c.page_size;
    r.e0 = bounds[t];
    r.rows = (bounds[t + 1] - bounds[t]) * a.group;
    r.seq = seqs[leader[t]];
    if (r.shared && p.with_prefix) {
      r.keys = r.shared;
      places = ((r.keys - 1) / p.keys + 1 + kKpCost) * a.c.kv_heads * ((r.rows + p.rows - 1) / p.rows);
    } else if (r.shared) {
      units = a.c.kv_heads * r.pairs() * r.size();
      rows = a.c.kv_heads * r.sums();
      // a unit of two tiles of rows, and of one: its chain, or its keys
      const float unit_ns = (float)(r.pairs() - 1) * p.pair_ns + ((r.rows - 1) % 256 >= 128 ? p.pair_ns : p.single_ns);
      weight = (int)((float)a.c.kv_heads * r.size() * unit_ns * 0x1p-12f) + 1;  // at most 2^31 places of less than 1 each
    }
  }
  if (is_group) least[t] = r.shared;
  __syncthreads();
  if (is_entry && len > 0) {
    r.first = g >= 0 ? least[g] : 0;
    r.keys = len - r.first;
    r.seq = s;
    places = ((r.keys - 1) / p.keys + 1 + kKpCost) * a.c.kv_heads * a.subgroups;
  }
  int4 sum{places, units, rows, weight};
  const int4 all = kp_scan(sum);
  r.place0 = sum.x;
  r.unit0 = sum.y;
  r.row0 = sum.z;
  if (is_group) {
    if (p.with_prefix) r.unit0 = r.place0;
    unit0[t] = r.unit0;
    row0[t] = r.row0;
    live[t] = r.rows;
    r.leader = r.seq;
    leader[t] = r.seq;
  }
  __syncthreads();
  if (is_entry && g >= 0 && r.first > 0) {
    r.shared = r.first;
    r.e0 = bounds[g];
    r.rows = live[g];
    r.unit0 = unit0[g];
    r.row0 = row0[g];
    r.leader = leader[g];
  }
  if (is_group || is_entry) p.plan[t] = r;
  if (t == 0) {
    KpEntry end{};
    end.place0 = all.x;
    end.unit0 = all.y;
    p.plan[groups + a.n] = end;
    // the SMs by the time that each kernel's work takes one
    const float own = (float)all.x * p.step_ns, shared = (float)all.w * 4096.f;
    const int sms = all.y == 0 ? p.sms : all.x == 0 ? 0 : max(1, min(p.sms - 1, (int)(p.sms * (own / (own + shared)) + 0.5f)));
    *p.head = make_int4(all.x, all.y, sms, 0);
  }
}

// --------------------------------------------------------------------------
// own
// --------------------------------------------------------------------------
template <typename T, int HD, int R>
struct KoCfg : KaCfg<T, HD, R> {
  using Base = KaCfg<T, HD, R>;
  static constexpr int kOffQ = Base::kRing;  // fp32 only: the query rows, each warp's
  static constexpr int kOffPlaces = kOffQ + (sizeof(T) == 4 ? Base::kWarps * R * HD * 4 : 0);
  static constexpr int kOffSubs = kOffPlaces + (kKvMaxEntries + 4) * 4;
  static constexpr int kOffMask = kOffSubs + kKvMaxEntries * 4;
  static constexpr int kSmem = kOffMask + Base::kWarps * Base::kStages * 4;
};
static_assert(KoCfg<float, 128, 8>::kSmem <= 232448 && KoCfg<float, 64, 8>::kSmem <= 232448, "shared memory above 227 KB");

__device__ __forceinline__ void ko_split(const int4& head, int warps, KaSplit& split) {
  split.make(head.x, max(1, min(head.z * warps, head.x / (2 * kKpCost))));
}

// A warp's part of the steps, walked in order (as KaWalk).
struct KoWalk {
  int entry, piece, step;
  int steps, base, to, pieces;
  __device__ __forceinline__ bool set(int e, int x0, int x1, const int* places, const int* subs, int kv_heads) {
    entry = e;
    pieces = kv_heads * subs[e];
    const int size = (int)((unsigned)(places[e + 1] - places[e]) / (unsigned)pieces);
    steps = size - kKpCost;
    piece = (int)((unsigned)(x0 - places[e]) / (unsigned)size);
    base = places[e] + piece * size;
    step = max(0, x0 - base - kKpCost);
    to = min(steps, x1 - base - kKpCost);
    return to > step;
  }
  __device__ __forceinline__ bool start(int x0, int x1, const int* places, const int* subs, int n, int kv_heads) {
    int lo = 0, hi = n;  // places[lo] <= x0 < places[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (places[mid] <= x0) lo = mid; else hi = mid;
    }
    return set(lo, x0, x1, places, subs, kv_heads);
  }
  // false: nothing is left
  __device__ __forceinline__ bool next(int x1, const int* places, const int* subs, int kv_heads) {
    if (++step < to) return true;
    base += steps + kKpCost;
    if (base >= x1) return false;
    if (++piece < pieces) {
      step = 0;
      to = min(steps, x1 - base - kKpCost);
      return to > 0;
    }
    int e = entry + 1;
    while (places[e + 1] == places[e]) ++e;  // there is one more: base is below the end
    return set(e, base, x1, places, subs, kv_heads);
  }
};

// A warp's sums of a pair's rows into the workspace.
template <int HD, int R>
__device__ __forceinline__ void ko_store(const KaStateBf16<HD, R>& st, float* o, float2* ml, int rows, int lane) {
  const int g = lane >> 2, t2 = (lane & 3) * 2;
#pragma unroll
  for (int h = 0; h < R / 8; ++h) {
    float s = st.l[h];
    s += __shfl_xor_sync(0xffffffffu, s, 1);
    s += __shfl_xor_sync(0xffffffffu, s, 2);
    const int row = g + 8 * h;
    if (row >= rows) continue;
    if ((lane & 3) == 0) __stcg(ml + row, make_float2(st.m[h], s));
#pragma unroll
    for (int i = 0; i < HD / 8; ++i)
      __stcg(reinterpret_cast<float2*>(o + row * HD + i * 8 + t2),
             R == 8 ? make_float2(st.o[i][0] + st.o[i][2], st.o[i][1] + st.o[i][3]) : make_float2(st.o[i][2 * h], st.o[i][2 * h + 1]));
  }
}
template <int HD, int R>
__device__ __forceinline__ void ko_store(const KaStateF32<HD, R>& st, float* o, float2* ml, int rows, int lane) {
#pragma unroll
  for (int r = 0; r < R; ++r) {
    if (r >= rows) continue;
    const float s = warp_sum(st.l[r]);
    if (lane == 0) __stcg(ml + r, make_float2(st.m[r], s));
    if constexpr (HD == 128)
      __stcg(reinterpret_cast<float4*>(o + r * HD) + lane, make_float4(st.o[r][0], st.o[r][1], st.o[r][2], st.o[r][3]));
    else
      __stcg(reinterpret_cast<float2*>(o + r * HD) + lane, make_float2(st.o[r][0], st.o[r][1]));
  }
}

template <typename T, int HD, int R>
__global__ void __launch_bounds__(KoCfg<T, HD, R>::kThreads, 1) kv_own_kernel(const __grid_constant__ KpArgs p) {
  using Cfg = KoCfg<T, HD, R>;
  constexpr int kStages = Cfg::kStages, kKeys = Cfg::kKeys, kWarps = Cfg::kWarps, kThreads = Cfg::kThreads;
  extern __shared__ __align__(128) uint8_t sm[];
  const KaArgs& a = p.a;
  const KvPages& c = a.c;
  int* places = reinterpret_cast<int*>(sm + Cfg::kOffPlaces);
  int* subs = reinterpret_cast<int*>(sm + Cfg::kOffSubs);  // pieces of an entry's key head
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, groups = p.groups, entries = groups + a.n;
  // Beside the prefix kernel, which began behind the plan, there is nothing to wait for but its end, in front of this
  // one's: the join waits for this kernel alone.  Without a wait in front nothing orders what an L1 still holds, so the
  // queries, the table and the plan are read from L2, as the keys are.
  if (p.with_prefix) pdl_wait();
  pdl_trigger();
  struct Behind {
    bool on;
    __device__ __forceinline__ ~Behind() {
      if (on) pdl_wait();
    }
  } behind{!p.with_prefix};
  const int4 head = __ldcg(p.head);
  for (int v = tid; v <= entries; v += kThreads) {
    places[v] = __ldcg(&p.plan[v].place0);
    if (v < entries) subs[v] = v < groups ? (__ldcg(&p.plan[v].rows) + R - 1) / R : a.subgroups;
  }
  __syncthreads();
  KaSplit split;
  ko_split(head, kWarps, split);
  const int self = blockIdx.x * kWarps + warp;
  if ((int)blockIdx.x >= head.z || head.x == 0 || self >= split.ctas) return;
  const int x0 = split.begin(self), x1 = split.begin(self + 1);
  KoWalk load;
  if (!load.start(x0, x1, places, subs, entries, c.kv_heads)) return;
  bool more = true;  // `load` is a step

  const uint8_t* ring = sm + warp * (kStages * Cfg::kStageBytes);
  const uint32_t ring_u32 = smem_u32(ring);
  uint32_t* masks = reinterpret_cast<uint32_t*>(sm + Cfg::kOffMask) + warp * kStages;
  float* qs = reinterpret_cast<float*>(sm + Cfg::kOffQ) + (sizeof(T) == 4 ? warp * R * HD : 0);
  KoWalk use = load;
  // Where key `lane` of a step lies: its page's number as the table has it, looked up two steps ahead of the copies, and
  // the rest of its address in 16-byte vectors; -1: no such key.
  struct Where {
    int page;
    int64_t off;
  };
  int load_entry = -1, first = 0, keys = 0;
  const int32_t* row = nullptr;
  auto look_up = [&]() -> Where {
    if (load.entry != load_entry) {
      load_entry = load.entry;
      const int4 r = __ldcg(reinterpret_cast<const int4*>(p.plan + load_entry));  // place0, first, keys, seq
      first = r.y;
      keys = r.z;
      row = c.table + (size_t)r.w * c.max_pages;
    }
    const uint32_t at = (uint32_t)load.step * kKeys + lane % kKeys;
    if (at >= (uint32_t)keys) return {0, -1};
    const int key = first + (int)at, j = (int)c.page_div.div((uint32_t)key);
    return {__ldcg(row + j), a.layer_off + (key - j * c.page_size) * c.token_stride + (load.piece / subs[load_entry]) * c.head_stride};
  };
  Where at = look_up(), at_next{0, -1};
  int ahead_steps = 1;  // looked up and not issued yet: at, at_next
  auto advance = [&]() {
    more = more && load.next(x1, places, subs, c.kv_heads);
    if (more) {
      at_next = look_up();
      ++ahead_steps;
    }
  };
  advance();
  // copies of one step, as in kv_attention_kernel
  auto issue = [&](int stage) {
    if (ahead_steps > 0) {
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
      --ahead_steps;
      at = at_next;
      if (ahead_steps > 0) advance();
    }
    cp_async_commit();
  };
  KaState<T, HD, R> state;
  int pair_rows = 0, pair_row = 0;  // of the pair at hand: rows, where its sums go for warp 0
  int next_rows = 0, next_row = 0;
  auto load_q = [&](const KoWalk& w) {
    const int pieces = subs[w.entry], sub = w.piece % pieces, kvh = w.piece / pieces;
    const T* q = reinterpret_cast<const T*>(a.q);
    const int heads = c.kv_heads * a.group;
    if (w.entry >= groups) {
      const int e = w.entry - groups, head0 = kvh * a.group + sub * R;
      next_rows = min(R, a.group - sub * R);
      next_row = (a.n + e) * heads + head0;
      const T* qrow = q + e * a.q_stride + head0 * HD;
      state.template load_q<true>([&](int r) { return qrow + r * HD; }, next_rows, lane);
    } else {  // a prefix: the queries of its group's entries in turn
      const int4 r1 = __ldcg(reinterpret_cast<const int4*>(p.plan + w.entry) + 1);  // shared, e0, rows, unit0
      next_rows = min(R, r1.z - sub * R);
      next_row = r1.y * heads + kvh * r1.z + sub * R;
      state.template load_q<true>([&](int r) {
        const int x = sub * R + r, e = (int)p.group_div.div((uint32_t)x);
        return q + (r1.y + e) * a.q_stride + (kvh * a.group + x - e * a.group) * HD;
      }, next_rows, lane);
    }
  };
  load_q(use);
  for (int s = 0; s < kStages - 1; ++s) issue(s);
  state.begin(lane, qs);
  pair_rows = next_rows;
  pair_row = next_row;

  int stage = 0;
  while (true) {
    issue(stage == 0 ? kStages - 1 : stage - 1);
    cp_async_wait<kStages - 1>();
    __syncwarp();
    const uint32_t mask = masks[stage];
    if (mask) state.step(ring + stage * Cfg::kStageBytes, ring_u32 + stage * Cfg::kStageBytes, mask, a.scale_log2, lane, qs);
    __syncwarp();  // the stage is refilled next turn
    stage = stage + 1 == kStages ? 0 : stage + 1;
    KoWalk ahead = use;
    const bool go = ahead.next(x1, places, subs, c.kv_heads);
    if (!go || ahead.base != use.base) {  // this warp's part of the pair is done
      if (go) load_q(ahead);
      const int64_t at = (int64_t)pair_row + R * self;
      ko_store(state, p.own_o + at * HD, p.own_ml + at, pair_rows, lane);
      if (!go) break;
      __syncwarp();
      state.begin(lane, qs);
      pair_rows = next_rows;
      pair_row = next_row;
    }
    use = ahead;
  }
  cp_async_wait<0>();
}

// --------------------------------------------------------------------------
// join: a warp per (entry, head), a lane HD / 32 columns
// --------------------------------------------------------------------------
template <typename T, int HD>
__global__ void __launch_bounds__(kKjThreads) kv_join_kernel(const __grid_constant__ KpArgs p) {
  constexpr int kE = HD / 32;
  const KaArgs& a = p.a;
  const KvPages& c = a.c;
  const int lane = threadIdx.x & 31, heads = c.kv_heads * a.group;
  const int64_t row = ((int64_t)blockIdx.x * kKjThreads + threadIdx.x) >> 5, rows = (int64_t)a.n * heads;
  pdl_wait();
  pdl_trigger();
  if (row >= rows) return;
  const int e = (int)(row / heads), head = (int)(row - (int64_t)e * heads), kvh = (int)p.group_div.div((uint32_t)head);
  const int4 all = __ldcg(p.head);
  const KpEntry r = kp_entry(p, p.groups + e);
  float m = -INFINITY, l = 0.f, acc[kE] = {};
  // n sums, the k-th at row at(k): all loads of a round before the first use
  auto add = [&](const float* o, const float2* ml, int n, auto at) {
    constexpr int kN = 8;
    for (int k0 = 0; k0 < n; k0 += kN) {
      float2 w[kN];
      float v[kN][kE];
#pragma unroll
      for (int k = 0; k < kN; ++k) {
        w[k] = make_float2(-INFINITY, 0.f);
#pragma unroll
        for (int i = 0; i < kE; ++i) v[k][i] = 0.f;
        if (k0 + k >= n) continue;
        const int64_t x = at(k0 + k);
        w[k] = __ldcg(ml + x);
        const float* from = o + x * HD + lane * kE;
        if constexpr (kE == 4)
          *reinterpret_cast<float4*>(v[k]) = __ldcg(reinterpret_cast<const float4*>(from));
        else
          *reinterpret_cast<float2*>(v[k]) = __ldcg(reinterpret_cast<const float2*>(from));
      }
      float mn = m;
#pragma unroll
      for (int k = 0; k < kN; ++k) mn = fmaxf(mn, w[k].x);
      const float f0 = m == -INFINITY ? 0.f : ex2_approx(m - mn);
      m = mn;
      l *= f0;
#pragma unroll
      for (int i = 0; i < kE; ++i) acc[i] *= f0;
#pragma unroll
      for (int k = 0; k < kN; ++k) {
        const float f = w[k].x == -INFINITY ? 0.f : ex2_approx(w[k].x - m);
        l = fmaf(f, w[k].y, l);  // NaN where a score was
#pragma unroll
        for (int i = 0; i < kE; ++i) acc[i] = w[k].x == -INFINITY ? acc[i] : fmaf(f, v[k][i], acc[i]);  // no sum: O may not be written
      }
    }
  };
  if (r.keys > 0) {
    KaSplit split;
    ko_split(all, p.warps, split);
    // a pair's sums: one of each warp that has some of its steps
    auto add_own = [&](int place, int keys, int64_t at) {
      const int steps = (keys - 1) / p.keys + 1, w0 = split.owner(place + kKpCost), w1 = split.owner(place + kKpCost + steps - 1);
      add(p.own_o, p.own_ml, w1 - w0 + 1, [&](int k) { return at + (int64_t)p.rows * (w0 + k); });
    };
    const int x = (e - r.e0) * a.group + head - kvh * a.group;  // its row of the group's
    if (r.shared > 0 && p.with_prefix) {
      const int pieces = (r.rows + p.rows - 1) / p.rows, size = (r.shared - 1) / p.keys + 1 + kKpCost;
      add_own(r.unit0 + (kvh * pieces + x / p.rows) * size, r.shared, (int64_t)r.e0 * heads + kvh * r.rows + x);
    } else if (r.shared > 0) {  // the segments of the row's unit, CTA by CTA, stream by stream
      KaSplit units;
      kp_split(p, all, units);
      const int row0 = x & ~255, unit_rows = min(256, r.rows - row0), base = r.unit0 + (kvh * r.pairs() + row0 / 256) * r.size() + kPtCost;
      const int c0 = units.owner(base), c1 = units.owner(base + r.tiles() - 1);
      const int64_t at = (int64_t)kp_row(r, kvh, row0) + 256 * c0 + (x - row0);
      if (unit_rows > 128)
        add(p.seg_o, p.seg_ml, c1 - c0 + 1, [&](int k) { return at + 256 * k; });
      else
        add(p.seg_o, p.seg_ml, 2 * (c1 - c0 + 1), [&](int k) { return at + 256 * (k >> 1) + (k & 1) * unit_rows; });
    }
    const int sub = (head - kvh * a.group) / p.rows, size = (r.keys - 1) / p.keys + 1 + kKpCost;
    add_own(r.place0 + (kvh * a.subgroups + sub) * size, r.keys, rows + row);
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  bool fine = true;
#pragma unroll
  for (int i = 0; i < kE; ++i) fine = fine && fabsf(acc[i]) <= 1.0e38f;
  if (__any_sync(0xffffffffu, !fine && l > 0.f)) {
    ka_redo<T, HD>(a, e, c.lens[r.seq], head, kvh);
  } else {
    T* out = reinterpret_cast<T*>(a.o) + e * a.o_stride + head * HD + lane * kE;
    float o[kE];
#pragma unroll
    for (int i = 0; i < kE; ++i) o[i] = inv == 0.f ? 0.f : acc[i] * inv;
    if constexpr (kE == 4) {
      ka_store4(out, make_float4(o[0], o[1], o[2], o[3]));
    } else if constexpr (sizeof(T) == 2) {
      *reinterpret_cast<uint32_t*>(out) = pack_bf16x2(o[0], o[1]);
    } else {
      *reinterpret_cast<float2*>(out) = make_float2(o[0], o[1]);
    }
  }
  // a sequence that does not hold the pages its group shares: the heads' warps look at 32 of them each
  if (r.shared > 0) {
    const int pages = c.pages_of(r.shared);
    const int32_t* mine = c.table + (size_t)r.seq * c.max_pages;
    const int32_t* first = c.table + (size_t)r.leader * c.max_pages;
    bool same = true;
    for (int64_t j = (int64_t)head * 32 + lane; j < pages; j += (int64_t)heads * 32) same = same && mine[j] == first[j];
    if (!same) c.flag(KV_BAD_SEQ);
  }
}

}  // namespace dinfer
