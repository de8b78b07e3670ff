// Attention of one new token per sequence where groups of sequences share the pages
// of their first tokens (include/dinfer_kv.h, dinfer_kv_prefix_attention).
//
// softmax(scale q K^T) V over the shared keys and over a sequence's own ones are two
// sums with a maximum each, (m, l, O), which join exactly:
//   m = max(m_0, m_1), l = sum 2^(m_i - m) l_i, O = sum 2^(m_i - m) O_i, o = O / l.
// So the shared keys are read once for all the rows of their group, members * heads /
// kv_heads queries per key head, and the rest once per sequence.
#pragma once
#include "kv_attention.cuh"

namespace dinfer {

constexpr int kKjThreads = 256;

// Joins a row's sums: a warp per (entry, head), a lane HD / 32 columns.
template <typename T, int HD>
__global__ void __launch_bounds__(kKjThreads) kv_join_kernel(const __grid_constant__ KaArgs a) {
  constexpr int kE = HD / 32;
  const KvPages& c = a.c;
  const int lane = threadIdx.x & 31, heads = c.kv_heads * a.group;
  const int64_t row = ((int64_t)blockIdx.x * kKjThreads + threadIdx.x) >> 5, rows = (int64_t)a.n * heads;
  pdl_wait();
  pdl_trigger();
  if (row >= rows) return;
  const int e = (int)(row / heads), head = (int)(row - (int64_t)e * heads);
  const int4 info = __ldcg(a.p.info + e);
  float m = -INFINITY, l = 0.f, acc[kE] = {};
  // kN sums more: all loads before the first use
  constexpr int kN = 8;
  auto add = [&](int n, auto ml_of, auto o_of) {
    float2 w[kN];
    float v[kN][kE];
#pragma unroll
    for (int k = 0; k < kN; ++k) {
      w[k] = make_float2(-INFINITY, 0.f);
#pragma unroll
      for (int i = 0; i < kE; ++i) v[k][i] = 0.f;
      if (k >= n) continue;
      w[k] = __ldcg(ml_of(k));
      const float* from = o_of(k) + lane * kE;
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
      for (int i = 0; i < kE; ++i) acc[i] = w[k].x == -INFINITY ? acc[i] : fmaf(f, v[k][i], acc[i]);  // no sum: O is not written
    }
  };
  if (a.p.with_prefix) {
    add(2, [&](int k) { return a.p.ml_part + k * rows + row; }, [&](int k) { return a.p.o_part + (k * rows + row) * HD; });
  } else {
    if (info.x > 0) {  // the segments of the row's unit, CTA by CTA, stream by stream
      const KpGroup g = kp_group(a, info.z);
      KaSplit split;
      kp_split(a, split);
      const int kvh = head / a.group, x = (e - g.e0) * a.group + head - kvh * a.group, row0 = x & ~255, unit_rows = min(256, g.rows - row0);
      const int base = g.place0 + (kvh * g.pairs() + row0 / 256) * g.size() + kPtCost;
      const int c0 = split.owner(base), c1 = split.owner(base + g.tiles() - 1), streams = unit_rows <= 128 ? 2 : 1;
      const int64_t at = (int64_t)kp_row(a, g, kvh, row0) + 256 * c0 + (x - row0);
      const int parts = (c1 - c0 + 1) * streams;
      for (int k0 = 0; k0 < parts; k0 += kN) {
        auto at_of = [&](int k) { return streams == 1 ? at + 256 * (k0 + k) : at + 256 * ((k0 + k) >> 1) + ((k0 + k) & 1) * unit_rows; };
        add(parts - k0, [&](int k) { return a.p.seg_ml + at_of(k); }, [&](int k) { return a.p.seg_o + at_of(k) * HD; });
      }
    }
    add(1, [&](int) { return a.p.ml_part + rows + row; }, [&](int) { return a.p.o_part + (rows + row) * HD; });
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  bool fine = true;
#pragma unroll
  for (int i = 0; i < kE; ++i) fine = fine && fabsf(acc[i]) <= 1.0e38f;
  if (__any_sync(0xffffffffu, !fine && l > 0.f)) {  // see ka_redo
    const int s = a.seqs ? a.seqs[e] : e;
    ka_redo<T, HD>(a, e, c.lens[s], head, head / a.group);
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
  const int pages = c.pages_of(info.x);
  if (pages > 0) {
    const int32_t* mine = c.table + (size_t)(a.seqs ? a.seqs[e] : e) * c.max_pages;
    const int32_t* first = c.table + (size_t)(a.seqs ? a.seqs[info.y] : info.y) * c.max_pages;
    bool same = true;
    for (int64_t j = (int64_t)head * 32 + lane; j < pages; j += (int64_t)heads * 32) same = same && mine[j] == first[j];
    if (!same) c.flag(KV_BAD_SEQ);
  }
}

}  // namespace dinfer
