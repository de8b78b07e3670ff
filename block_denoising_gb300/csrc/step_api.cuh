// Host side of a serving loop's other steps (include/dinfer_ops.h: rotary
// positions; include/dinfer_kv.h: rotated appends): argument checks and launches.
// Included behind kv_api.cuh, whose helpers it uses.
#pragma once
#include "kv_prefix_tc.cuh"
#include "rope.cuh"
#include "sample.cuh"

namespace {

constexpr uint64_t kRopeReady = 0x726f7065cf0157a1;  // dinfer_rope::ready of a filled one

// Why the rotation is unusable, or NULL.
const char* rope_bad(const dinfer_rope* r) {
  if (!r) return "rope is NULL";
  if (r->rot_dim < 2 || r->rot_dim % 2 || r->rot_dim > 2 * kRopePairs) return "rope: rot_dim must be even, 2 .. head_dim";
  if (r->layout != DINFER_ROPE_HALF && r->layout != DINFER_ROPE_PAIRS) return "rope: unknown layout";
  if (r->scaling < DINFER_ROPE_NONE || r->scaling > DINFER_ROPE_BANDS) return "rope: unknown scaling";
  if (!(r->theta > 0) || !std::isfinite(r->theta) || !(r->magnitude > 0) || !(r->magnitude < 3e38))
    return "rope: theta and magnitude must be positive";
  if (r->scaling != DINFER_ROPE_NONE && (!(r->factor > 0) || !std::isfinite(r->factor)))
    return "rope: factor must be positive";
  if (r->scaling == DINFER_ROPE_BANDS &&
      (r->trained < 1 || !(r->slow >= 0) || !(r->fast > r->slow) || !std::isfinite(r->fast)))
    return "rope: bands need trained >= 1 and 0 <= slow < fast";
  return nullptr;
}

// The same for a call on heads of head_dim; else the kernel's table.
const char* rope_turns(const dinfer_rope* r, int head_dim, RopeTurns& t) {
  if (const char* why = rope_bad(r)) return why;
  if (r->ready != kRopeReady) return "rope: dinfer_rope_init has not filled it";
  if (r->rot_dim > head_dim) return "rope: rot_dim must be even, 2 .. head_dim";
  t.pairs = r->rot_dim / 2;
  t.magnitude = (float)r->magnitude;
  std::copy(r->turns, r->turns + t.pairs, t.f);
  return nullptr;
}

template <typename T, bool kPlace>
cudaError_t launch_rope(RopeArgs& a, const RopeTurns& t, bool pairs, cudaStream_t s) {
  constexpr int kVec = 16 / (int)sizeof(T);
  // whole vectors where the pairs, and what is not rotated, begin at them
  const bool vec = (pairs ? 2 * t.pairs : t.pairs) % kVec == 0;
  const int per = vec ? kVec : 1;
  a.rot_items = pairs && vec ? 2 * t.pairs / per : t.pairs / per;
  a.head_items = FastDiv::make((uint32_t)(a.rot_items + (a.head_dim - 2 * t.pairs) / per));
  a.vecs = FastDiv::make((uint32_t)(a.head_dim / kVec));
  const int items = (a.x[0].heads + a.x[1].heads) * (int)a.head_items.d + a.x[2].heads * (int)a.vecs.d;
  a.row_items = FastDiv::make((uint32_t)items);
  // Four rows a block share its barriers and its cosines' threads where every SM has work all the same; else a row's
  // items are dealt to as many blocks as there are SMs to take them.
  const int sms = num_sms();
  a.chunk = a.rows >= 16 * sms ? kRopeRows : 1;
  const int chunks = (a.rows + a.chunk - 1) / a.chunk, most = (a.chunk * items + kRopeThreads - 1) / kRopeThreads;
  a.parts = std::max(1, std::min(most, 4 * sms / chunks));
  const int grid = (int)std::min<int64_t>((int64_t)chunks * a.parts, 8 * sms);
  auto go = [&](auto* kernel) { return launchk(kernel, dim3(grid), dim3(kRopeThreads), 0, s, 1, a, t); };
  if (pairs) return vec ? go(rope_kernel<T, true, kVec, kPlace>) : go(rope_kernel<T, true, 1, kPlace>);
  return vec ? go(rope_kernel<T, false, kVec, kPlace>) : go(rope_kernel<T, false, 1, kPlace>);
}

// Bytes of the workspace in front of the sums of dinfer_kv_prefix_attention: the token kernel's partials of each CTA
// (at most 18 KB twice), the plan, the entries' records.
constexpr size_t kPrefixHead = 8u << 20;
static_assert((sizeof(KpGroup) + sizeof(int4)) * (kKvMaxEntries + 1) <= 64 * 1024, "plan and records");

bool g_step_setup[kMaxDevices] = {};
constexpr int kSmMostBytes = 232448 - 2048;

// Shared-memory limits of this file's kernels, set once per device.
bool step_setup() {
  const int dev = current_device();
  std::lock_guard<std::mutex> lk(g_setup_mutex);
  if (!g_step_setup[dev]) {
    g_step_setup[dev] = max_smem(sample_kernel<__nv_bfloat16>, kSmMostBytes) && max_smem(sample_kernel<float>, kSmMostBytes) &&
                        max_smem(kv_prefix_tc_kernel<64>, PtCfg<64>::kSmem) && max_smem(kv_prefix_tc_kernel<128>, PtCfg<128>::kSmem);
    if (!g_step_setup[dev]) cudaGetLastError();
  }
  return g_step_setup[dev];
}

}  // namespace

extern "C" {

dinfer_status dinfer_rope_init(dinfer_rope* r) {
  dinfer_ctx* c = nullptr;
  if (const char* why = rope_bad(r)) return fail(c, DINFER_EINVAL, "%s", why);
  const double two_pi = 6.283185307179586476925286766559;
  r->ready = 0;
  std::fill(r->turns, r->turns + kRopePairs, 0);
  for (int i = 0; i < r->rot_dim / 2; ++i) {
    double f = std::pow(r->theta, -2.0 * i / r->rot_dim);
    if (r->scaling == DINFER_ROPE_LINEAR) f /= r->factor;
    if (r->scaling == DINFER_ROPE_BASE && i > 0) f *= std::pow(r->factor, -2.0 * i / (r->rot_dim - 2));
    if (r->scaling == DINFER_ROPE_BANDS) {
      const double g = std::min(1.0, std::max(0.0, (r->trained * f / two_pi - r->slow) / (r->fast - r->slow)));
      f = g * f + (1 - g) * f / r->factor;
    }
    if (!(f <= 65536.0)) return fail(c, DINFER_EINVAL, "rope: a frequency above 2^16");
    const double turns = f / two_pi;
    r->turns[i] = (uint64_t)std::ldexp(turns - std::floor(turns), 64);
  }
  r->ready = kRopeReady;
  return DINFER_OK;
}

dinfer_status dinfer_op_rope(const void* x, void* y, int32_t dtype, const dinfer_rope* rope, const int32_t* positions,
                             int32_t first, int32_t rows, int32_t heads, int32_t head_dim, int64_t x_stride,
                             int64_t y_stride, void* stream) {
  dinfer_ctx* c = nullptr;
  if (!x || !y) return fail(c, DINFER_EINVAL, "NULL operand");
  if (dtype != DINFER_BF16 && dtype != DINFER_FP32) return fail(c, DINFER_EINVAL, "unknown dtype");
  const int64_t per = dtype == DINFER_BF16 ? 8 : 4;
  if (head_dim < 1 || head_dim > 2 * kRopePairs || head_dim % per)
    return fail(c, DINFER_EINVAL, "head_dim must be whole vectors of 16 bytes, at most %d", 2 * kRopePairs);
  if (rows < 1 || rows > (1 << 30) || heads < 1 || heads > 65536) return fail(c, DINFER_EINVAL, "unsupported number of rows or heads");
  if (!positions && (int64_t)first + rows > (1ll << 31)) return fail(c, DINFER_EINVAL, "positions beyond 2^31");
  RopeTurns t;
  if (const char* why = rope_turns(rope, head_dim, t)) return fail(c, DINFER_EINVAL, "%s", why);
  const int64_t row = (int64_t)heads * head_dim;
  if (!rows_ok(x, x_stride, rows, row, per) || !rows_ok(y, y_stride, rows, row, per))
    return fail(c, DINFER_EINVAL, "x, y: 16-byte aligned rows at least a row apart are needed");
  if (x == y && rows > 1 && x_stride != y_stride) return fail(c, DINFER_EINVAL, "y is x with another stride");
  if (!ints_ok(positions)) return fail(c, DINFER_EINVAL, "misaligned positions");
  RopeArgs a{};
  a.x[0] = {x, y, x_stride, y_stride, heads};
  a.positions = positions;
  a.first = first;
  a.rows = rows;
  a.head_dim = head_dim;
  a.in_place = x == y;
  const bool pairs = rope->layout == DINFER_ROPE_PAIRS;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  CK((dtype == DINFER_BF16 ? launch_rope<__nv_bfloat16, false>(a, t, pairs, s) : launch_rope<float, false>(a, t, pairs, s)));
  return DINFER_OK;
}

dinfer_status dinfer_kv_append_rope(const dinfer_kv_cache* kc, int32_t layer, const dinfer_rope* rope,
                                    const int32_t* positions, const int32_t* seqs, const int32_t* rows, int32_t n,
                                    const void* q, void* q_out, int32_t heads, int64_t q_stride, int64_t q_out_stride,
                                    const void* k, const void* v, int64_t k_stride, int64_t v_stride,
                                    int32_t total_rows, void* stream) {
  dinfer_ctx* c = nullptr;
  if (const char* why = kv_bad(kc)) return fail(c, DINFER_EINVAL, "%s", why);
  if (!k || !v || !q != !q_out) return fail(c, DINFER_EINVAL, "NULL operand");
  if (layer < 0 || layer >= kc->n_layers) return fail(c, DINFER_EINVAL, "no layer %d", layer);
  if (n < 1 || total_rows < 1 || total_rows > (1 << 30) || (!rows && total_rows != n))
    return fail(c, DINFER_EINVAL, "bad number of rows or entries");
  if (n > (seqs ? kKvMaxEntries : kc->max_seqs)) return fail(c, DINFER_EINVAL, "more entries than sequences, or than %d", kKvMaxEntries);
  if (q && (heads < 1 || heads > 65536)) return fail(c, DINFER_EINVAL, "unsupported number of heads");
  RopeTurns t;
  if (const char* why = rope_turns(rope, kc->head_dim, t)) return fail(c, DINFER_EINVAL, "%s", why);
  const int64_t per = kc->dtype == DINFER_BF16 ? 8 : 4, row = (int64_t)kc->kv_heads * kc->head_dim, qr = (int64_t)heads * kc->head_dim;
  if (!rows_ok(k, k_stride, total_rows, row, per) || !rows_ok(v, v_stride, total_rows, row, per) ||
      (q && (!rows_ok(q, q_stride, total_rows, qr, per) || !rows_ok(q_out, q_out_stride, total_rows, qr, per))))
    return fail(c, DINFER_EINVAL, "q, k, v: 16-byte aligned rows at least a row apart are needed");
  if (q && q == q_out && total_rows > 1 && q_stride != q_out_stride) return fail(c, DINFER_EINVAL, "q_out is q with another stride");
  if (q && (q_out == k || q_out == v)) return fail(c, DINFER_EINVAL, "q_out must not overlap k or v");
  if (!ints_ok(seqs, rows) || !ints_ok(positions)) return fail(c, DINFER_EINVAL, "misaligned seqs, rows or positions");
  RopeArgs a{};
  a.c = kv_pages(*kc);
  const int64_t layer_off = layer * a.c.layer_stride;
  a.x[0] = {q, q_out, q_stride, q_out_stride, q ? heads : 0};
  a.x[1] = {k, a.c.k + layer_off, k_stride, 0, kc->kv_heads};
  a.x[2] = {v, a.c.v + layer_off, v_stride, 0, kc->kv_heads};
  a.positions = positions;
  a.rows = total_rows;
  a.head_dim = kc->head_dim;
  a.in_place = q == q_out;
  a.seqs = seqs;
  a.bounds = rows;
  a.n = n;
  const bool pairs = rope->layout == DINFER_ROPE_PAIRS;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  CK((kc->dtype == DINFER_BF16 ? launch_rope<__nv_bfloat16, true>(a, t, pairs, s) : launch_rope<float, true>(a, t, pairs, s)));
  return DINFER_OK;
}

dinfer_status dinfer_kv_prefix_attention(const dinfer_kv_cache* kc, int32_t layer, const int32_t* seqs, int32_t n,
                                         const int32_t* groups, const int32_t* prefix, int32_t n_groups, const void* q,
                                         void* o, int64_t q_stride, int64_t o_stride, int32_t heads, float scale,
                                         void* workspace, size_t workspace_bytes, void* stream) {
  dinfer_ctx* c = nullptr;
  if (const char* why = kv_bad(kc)) return fail(c, DINFER_EINVAL, "%s", why);
  if (!q || !o || !prefix) return fail(c, DINFER_EINVAL, "NULL operand");
  if (layer < 0 || layer >= kc->n_layers) return fail(c, DINFER_EINVAL, "no layer %d", layer);
  if (n < 1 || n_groups < 1 || n > kKvMaxEntries || n_groups > kKvMaxEntries || n + n_groups > kKvMaxEntries || (!groups && n_groups != 1))
    return fail(c, DINFER_EINVAL, "n and n_groups must be 1 or more, together at most %d, with groups unless there is one", kKvMaxEntries);
  if (heads < 1 || heads > 65536 || heads % kc->kv_heads) return fail(c, DINFER_EINVAL, "heads must be a multiple of kv_heads");
  if (!(scale > 0.f) || !std::isfinite(scale * 1.4426950408889634f)) return fail(c, DINFER_EINVAL, "bad scale");
  const int64_t per = kc->dtype == DINFER_BF16 ? 8 : 4, row = (int64_t)heads * kc->head_dim;
  if (!rows_ok(q, q_stride, n, row, per) || !rows_ok(o, o_stride, n, row, per))
    return fail(c, DINFER_EINVAL, "q, o: 16-byte aligned rows at least a row apart are needed");
  if (!ints_ok(seqs, groups) || !ints_ok(prefix)) return fail(c, DINFER_EINVAL, "misaligned seqs, groups or prefix");
  OpWs w;
  if (!op_ws(workspace, workspace_bytes, w)) return fail(c, DINFER_EINVAL, "workspace too small");
  if (reinterpret_cast<uintptr_t>(workspace) & 15) return fail(c, DINFER_EINVAL, "workspace must be 16-byte aligned");
  if ((kc->max_pages * (int64_t)kc->page_size / 16 + 11) * (2 * n + n_groups) >= ((1ll << 31) + heads - 1) / heads)
    return fail(c, DINFER_EINVAL, "more than 2^31 steps of keys in one call");
  // of the workspace: the kernels' own partials, the plan, the sums of all rows, those of the segments
  const int64_t sums = (int64_t)n * heads, seg_rows = 2 * sums + 256 * num_sms();
  const int64_t row_bytes = 4 * kc->head_dim + 8;
  if ((int64_t)kPrefixHead + (2 * sums + seg_rows) * row_bytes > (int64_t)w.data_bytes) return fail(c, DINFER_EINVAL, "workspace too small");
  if (!kv_setup() || !step_setup()) return fail(c, DINFER_ECUDA, "kernel set-up failed");
  KaArgs a{};
  a.c = kv_pages(*kc);
  a.seqs = seqs;
  a.q = q;
  a.o = o;
  a.q_stride = q_stride;
  a.o_stride = o_stride;
  a.layer_off = layer * a.c.layer_stride;
  a.n = n;
  a.group = heads / kc->kv_heads;
  a.window = -1;
  a.min_steps = 8;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.partial = reinterpret_cast<float*>(w.data);
  a.tickets = w.tickets;
  const bool bf16 = kc->dtype == DINFER_BF16;
  // the prefixes' rows: in bf16 on the tensor cores, unless one piece of 16 rows holds all that a group can have
  const bool tc = bf16 && (int64_t)n * a.group > 16;
  const int rows = kv_rows(bf16, (int)std::min<int64_t>(tc ? a.group : (int64_t)a.group * n, 16));
  a.subgroups = (a.group + rows - 1) / rows;
  uint8_t* at = w.data + kPrefixHead;
  a.p.info = reinterpret_cast<int4*>(at - 64 * 1024);
  a.p.plan = tc ? reinterpret_cast<KpGroup*>(at - 128 * 1024) : nullptr;
  a.p.o_part = reinterpret_cast<float*>(at);
  a.p.seg_o = a.p.o_part + 2 * sums * kc->head_dim;
  a.p.ml_part = reinterpret_cast<float2*>(a.p.seg_o + seg_rows * kc->head_dim);
  a.p.seg_ml = a.p.ml_part + 2 * sums;
  a.p.seg_ctas = num_sms();
  a.p.bounds = groups;
  a.p.prefix = prefix;
  a.p.groups = n_groups;
  a.p.with_prefix = !tc;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  CK((kc->head_dim == 128 ? launch_kv_attention<128>(a, bf16, rows, s) : launch_kv_attention<64>(a, bf16, rows, s)));
  if (tc) {
    const PtArgs pa{a, w.st};
    CK((kc->head_dim == 128 ? launchk(kv_prefix_tc_kernel<128>, dim3(num_sms()), dim3(kPtThreads), PtCfg<128>::kSmem, s, 1, pa)
                            : launchk(kv_prefix_tc_kernel<64>, dim3(num_sms()), dim3(kPtThreads), PtCfg<64>::kSmem, s, 1, pa)));
  }
  const dim3 grid((unsigned)((sums + kKjThreads / 32 - 1) / (kKjThreads / 32)));
  auto join = [&](auto* kernel) { return launchk(kernel, grid, dim3(kKjThreads), 0, s, 1, a); };
  CK((kc->head_dim == 128 ? (bf16 ? join(kv_join_kernel<__nv_bfloat16, 128>) : join(kv_join_kernel<float, 128>))
                          : (bf16 ? join(kv_join_kernel<__nv_bfloat16, 64>) : join(kv_join_kernel<float, 64>))));
  return DINFER_OK;
}

dinfer_status dinfer_op_sample(const void* logits, int32_t dtype, int32_t rows, int32_t vocab, int64_t stride,
                               const float* temperature, const int32_t* top_k, const float* top_p, const float* min_p,
                               const float* u, int32_t* tok, float* conf, void* stream) {
  dinfer_ctx* c = nullptr;
  if (!logits || !u || !tok) return fail(c, DINFER_EINVAL, "NULL operand");
  if (dtype != DINFER_BF16 && dtype != DINFER_FP32) return fail(c, DINFER_EINVAL, "unknown dtype");
  if (rows < 1 || rows > (1 << 20) || vocab < 1 || vocab > (1 << kSmIndexBits)) return fail(c, DINFER_EINVAL, "unsupported number of rows or tokens");
  if (rows > 1 && (stride < vocab || stride > (1ll << 40))) return fail(c, DINFER_EINVAL, "rows at least a row apart are needed");
  const int size = dtype == DINFER_BF16 ? 2 : 4;
  if (reinterpret_cast<uintptr_t>(logits) % size) return fail(c, DINFER_EINVAL, "misaligned logits");
  if (!ints_ok(temperature, top_k) || !ints_ok(top_p, min_p) || !ints_ok(u, tok) || !ints_ok(conf))
    return fail(c, DINFER_EINVAL, "misaligned operand");
  if (!step_setup()) return fail(c, DINFER_ECUDA, "kernel set-up failed");
  SmArgs a{};
  a.x = logits;
  a.stride = rows > 1 ? stride : vocab;
  a.rows = rows;
  a.vocab = vocab;
  a.temperature = temperature;
  a.top_k = top_k;
  a.top_p = top_p;
  a.min_p = min_p;
  a.u = u;
  a.tok = tok;
  a.conf = conf;
  for (int j = 0; j < 16; ++j) a.coarse[j] = (uint64_t)std::ldexp(std::exp2(j / 16.0), 63);
  for (int j = 0; j < 32; ++j) a.fine[j] = (uint64_t)std::ldexp(std::exp2(j / 512.0), 63);
  // a CTA for every 2048 tokens, up to a cluster
  int ctas = 1;
  while (ctas < kSmCluster && (int64_t)ctas * 2048 < vocab) ctas *= 2;
  a.slice = (vocab + ctas - 1) / ctas;
  const size_t smem = (sizeof(SmShared) + 15) / 16 * 16 + (size_t)a.slice * size + 16;
  if (smem > kSmMostBytes) return fail(c, DINFER_EINVAL, "too many tokens");
  const dim3 grid(rows, 1, ctas);
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  CK((dtype == DINFER_BF16 ? launchk(sample_kernel<__nv_bfloat16>, grid, dim3(kSmThreads), smem, s, ctas, a)
                           : launchk(sample_kernel<float>, grid, dim3(kSmThreads), smem, s, ctas, a)));
  return DINFER_OK;
}

}  // extern "C"
