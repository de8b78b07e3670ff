// Host side of a serving loop's other steps (include/dinfer_ops.h: rotary
// positions, sampling; include/dinfer_kv.h: rotated appends, attention over shared
// prefixes): argument checks and launches.
// Included behind kv_api.cuh, whose helpers it uses.
#pragma once
#include "kv_prefix_tc.cuh"
#include "rope.cuh"
#include "sample.cuh"

namespace {

// dinfer_rope::ready of one that is filled for the fields it has: all of them, mixed.
uint64_t rope_mark(const dinfer_rope& r) {
  static_assert(offsetof(dinfer_rope, turns) == 56, "fields without gaps");
  uint64_t fields[7], mark = 0x726f7065cf0157a1;
  std::memcpy(fields, &r, sizeof(fields));
  for (uint64_t f : fields) mark = (mark ^ f) * 0x9e3779b97f4a7c15, mark ^= mark >> 29;
  return mark;
}

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
  if (r->ready != rope_mark(*r)) return "rope: dinfer_rope_init has not filled it, or not since a field changed";
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
  a.copies = FastDiv::make((uint32_t)std::max(1, a.head_dim / kVec / 2));  // appended heads are 64 or 128
  const int items = (a.x[0].heads + a.x[1].heads) * (int)a.head_items.d + a.x[2].heads * (int)a.copies.d;
  a.row_items = FastDiv::make((uint32_t)items);
  // Several rows a block share its barriers and its cosines' threads where every SM has work all the same; else a row's
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

// Bytes of the workspace in front of the sums of dinfer_kv_prefix_attention: its plan.
constexpr size_t kPrefixHead = 64 * 1024;
static_assert(sizeof(int4) + sizeof(KpEntry) * (kKvMaxEntries + 1) <= kPrefixHead - 16, "plan");
// Where the sums begin: the prefix kernel stores theirs 32 bytes at a time, and the workspace may begin at 16.
float* prefix_sums(uint8_t* data) { return reinterpret_cast<float*>(reinterpret_cast<uintptr_t>(data + kPrefixHead) & ~uintptr_t(31)); }

// One layer of a bf16 cache as [pages][heads][slots][hd]: boxes of a page's slots, at most 128, x 64 elements with the
// 128-byte swizzle; pages behind the last read as zeros.
bool make_map_pages(CUtensorMap* m, const dinfer_kv_cache& kc, const void* base, int layer) {
  EncodeTiledFn enc = get_encode_fn();
  if (!enc) return false;
  const int64_t row = kc.head_dim;
  auto stride = [&](int64_t s, int64_t size) { return (cuuint64_t)(size > 1 ? s : row) * 2; };  // of one entry: never stepped over
  cuuint64_t dims[4] = {(cuuint64_t)kc.head_dim, (cuuint64_t)kc.page_size, (cuuint64_t)kc.kv_heads, (cuuint64_t)kc.num_pages};
  cuuint64_t strides[3] = {stride(kc.token_stride, kc.page_size), stride(kc.head_stride, kc.kv_heads), stride(kc.page_stride, kc.num_pages)};
  for (cuuint64_t s : strides)
    if (s >= (1ull << 40)) return false;
  cuuint32_t box[4] = {64, (cuuint32_t)std::min(kc.page_size, 128), 1, 1};
  cuuint32_t es[4] = {1, 1, 1, 1};
  const uint16_t* from = reinterpret_cast<const uint16_t*>(base) + (kc.n_layers > 1 ? layer * kc.layer_stride : 0);
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<uint16_t*>(from), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, int HD, int R>
cudaError_t launch_kv_own_r(const KpArgs& p, cudaStream_t s) {
  using Cfg = KoCfg<T, HD, R>;
  return launchk(kv_own_kernel<T, HD, R>, dim3(p.sms), dim3(Cfg::kThreads), Cfg::kSmem, s, 1, p);
}
template <int HD>
cudaError_t launch_kv_own(const KpArgs& p, bool bf16, cudaStream_t s) {
  if (bf16) return p.rows == 8 ? launch_kv_own_r<__nv_bfloat16, HD, 8>(p, s) : launch_kv_own_r<__nv_bfloat16, HD, 16>(p, s);
  switch (p.rows) {
    case 1: return launch_kv_own_r<float, HD, 1>(p, s);
    case 2: return launch_kv_own_r<float, HD, 2>(p, s);
    case 4: return launch_kv_own_r<float, HD, 4>(p, s);
    default: return launch_kv_own_r<float, HD, 8>(p, s);
  }
}
template <typename T, int HD, int R>
bool step_setup_own() {
  return max_smem(kv_own_kernel<T, HD, R>, KoCfg<T, HD, R>::kSmem);
}
template <int HD>
bool step_setup_hd() {
  return step_setup_own<__nv_bfloat16, HD, 8>() && step_setup_own<__nv_bfloat16, HD, 16>() && step_setup_own<float, HD, 1>() &&
         step_setup_own<float, HD, 2>() && step_setup_own<float, HD, 4>() && step_setup_own<float, HD, 8>() &&
         max_smem(kv_prefix_tc_kernel<HD, true>, PtCfg<HD>::kSmem) && max_smem(kv_prefix_tc_kernel<HD, false>, PtCfg<HD>::kSmem);
}

bool g_step_setup[kMaxDevices] = {};
constexpr int kSmMostBytes = 232448 - 2048;

template <typename T, int kBlocks>
bool step_setup_sample_one() {
  return max_smem(sample_kernel<T, kBlocks>, kSmMostBytes) &&
         cudaFuncSetAttribute(sample_kernel<T, kBlocks>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess;
}
template <typename T>
bool step_setup_sample() {
  return step_setup_sample_one<T, 1>() && step_setup_sample_one<T, 2>() && step_setup_sample_one<T, 3>();
}
template <typename T>
cudaError_t launch_sample(const SmArgs& a, dim3 grid, size_t smem, cudaStream_t s) {
  // registers for as many CTAs an SM as there are, or as its shared memory takes
  const int blocks = (int64_t)grid.x * grid.z <= num_sms() ? 1 : (int)std::min<int64_t>(3, 232448 / (smem + 1024));
  auto go = [&](auto* kernel) { return launchk(kernel, grid, dim3(kSmThreads), smem, s, (int)grid.z, a); };
  return blocks <= 1 ? go(sample_kernel<T, 1>) : blocks == 2 ? go(sample_kernel<T, 2>) : go(sample_kernel<T, 3>);
}

// Shared-memory limits of this file's kernels, set once per device.
bool step_setup() {
  const int dev = current_device();
  std::lock_guard<std::mutex> lk(g_setup_mutex);
  if (!g_step_setup[dev]) {
    g_step_setup[dev] = step_setup_sample<__nv_bfloat16>() && step_setup_sample<float>() &&
                        step_setup_hd<64>() && step_setup_hd<128>();
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
  r->ready = rope_mark(*r);
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
  // of the workspace: the plan, then sums of the own keys' warps (at most 8 an SM, 16 rows) and of the prefixes' segments
  const int64_t sums = (int64_t)n * heads, own_rows = 2 * sums + 128 * num_sms(), seg_rows = 2 * sums + 256 * num_sms();
  if ((int64_t)kPrefixHead + (own_rows + seg_rows) * (4 * kc->head_dim + 8) > (int64_t)w.data_bytes)
    return fail(c, DINFER_EINVAL, "workspace too small");
  if (!kv_setup() || !step_setup()) return fail(c, DINFER_ECUDA, "kernel set-up failed");
  KpArgs p{};
  KaArgs& a = p.a;
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
  a.scale_log2 = scale * 1.4426950408889634f;
  const bool bf16 = kc->dtype == DINFER_BF16, hd128 = kc->head_dim == 128;
  // the prefixes' rows: in bf16 on the tensor cores, unless one piece of 16 rows holds all that a group can have
  const bool tc = bf16 && (int64_t)n * a.group > 16;
  const int rows = kv_rows(bf16, (int)std::min<int64_t>(tc ? a.group : (int64_t)a.group * n, 16));
  a.subgroups = (a.group + rows - 1) / rows;
  p.bounds = groups;
  p.prefix = prefix;
  p.groups = n_groups;
  p.with_prefix = !tc;
  p.sms = num_sms();
  p.warps = hd128 ? KaCfg<float, 128, 8>::kWarps : KaCfg<float, 64, 8>::kWarps;
  p.keys = bf16 ? KaCfg<__nv_bfloat16, 128, 8>::kKeys : KaCfg<float, 128, 8>::kKeys;
  p.rows = rows;
  // what an SM takes for a step of own keys and for a tile of shared ones, in the company of the others, keys from HBM (head_dim
  // 128: 64 sequences behind 8192 tokens, 32 heads on 8, 35.6 us, with 0.7 of the tiles' 38.1, with 1.3 38.4; 32 behind 8192,
  // 16 heads on 16, 48.4, 55.7 and with 1.4 52.3; head_dim 64: three groups, 96 sequences, 64 heads on 8, 86.3, 91.9 and 101.6)
  p.step_ns = hd128 ? 360 : 165;
  p.pair_ns = hd128 ? 3200 : 1860;
  p.single_ns = hd128 ? 1440 : 1320;
  p.group_div = FastDiv::make((uint32_t)a.group);
  p.head = reinterpret_cast<int4*>(w.data);
  p.plan = reinterpret_cast<KpEntry*>(p.head + 1);
  p.own_o = prefix_sums(w.data);
  p.seg_o = p.own_o + own_rows * kc->head_dim;
  p.own_ml = reinterpret_cast<float2*>(p.seg_o + seg_rows * kc->head_dim);
  p.seg_ml = p.own_ml + own_rows;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  PtMaps maps{};
  // TMA boxes of whole pages or whole tiles
  const int64_t page = kc->page_size;
  const bool boxes = tc && ((page >= 8 && 128 % page == 0) || page % 128 == 0) && make_map_pages(&maps.k, *kc, kc->k, layer) &&
                     make_map_pages(&maps.v, *kc, kc->v, layer);
  CK(launchk(kv_prefix_plan_kernel, dim3(1), dim3((n + n_groups + 31) / 32 * 32), 0, s, 1, p));
  if (tc) {
    const PtArgs pa{p, w.st, (int)std::max<int64_t>(1, 128 / page)};
    auto go = [&](auto* kernel, int smem) { return launchk(kernel, dim3(p.sms), dim3(kPtThreads), smem, s, 1, maps, pa); };
    CK((hd128 ? go(boxes ? kv_prefix_tc_kernel<128, true> : kv_prefix_tc_kernel<128, false>, PtCfg<128>::kSmem)
              : go(boxes ? kv_prefix_tc_kernel<64, true> : kv_prefix_tc_kernel<64, false>, PtCfg<64>::kSmem)));
  }
  CK((hd128 ? launch_kv_own<128>(p, bf16, s) : launch_kv_own<64>(p, bf16, s)));
  const dim3 grid((unsigned)((sums + kKjThreads / 32 - 1) / (kKjThreads / 32)));
  auto join = [&](auto* kernel) { return launchk(kernel, grid, dim3(kKjThreads), 0, s, 1, p); };
  CK((hd128 ? (bf16 ? join(kv_join_kernel<__nv_bfloat16, 128>) : join(kv_join_kernel<float, 128>))
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
  a.cuts = top_k || top_p;
  for (int j = 0; j < 16; ++j) a.coarse[j] = (uint64_t)std::ldexp(std::exp2(j / 16.0), 63);
  for (int j = 0; j < 32; ++j) a.fine[j] = (uint64_t)std::ldexp(std::exp2(j / 512.0), 63);
  // As few CTAs a row as two or three an SM can hold it with, which saves their meetings (512 rows of 126464 in bf16 at a
  // temperature: 4 CTAs 149 us, 2 174, 8 202).  With a cut, whose meetings are more, no more than four where they hold it, one
  // an SM (300 rows of 157184 in fp32 with top-k 20, with top-p 0.9: 4 CTAs 159 and 642 us, 8 253 and 1002, 16 315 and 1170),
  // and no fewer, whose threads' maxima give too low a floor (512 rows of 126464 in bf16 with top-k 1000: 4 CTAs 203 us, 2 366).
  // More while there are SMs to spare and 2048 tokens for each (one row of 126464 at a temperature: 16 CTAs 9.2 us, 8 11.2, 4 15.5).
  int ctas = 1;
  while (ctas < kSmCluster && ((int64_t)vocab * size > (int64_t)ctas * (!a.cuts ? 80 : ctas < 4 ? 64 : 160) * 1024 ||
                               ((int64_t)rows * ctas * 2 <= num_sms() && (int64_t)ctas * 2048 < vocab)))
    ctas *= 2;
  a.slice = (vocab + ctas - 1) / ctas;
  const size_t smem = sizeof(SmShared) + (a.cuts ? sizeof(SmCut) : 0) + (size_t)a.slice * size + 48;  // pads before and behind
  if (smem > kSmMostBytes) return fail(c, DINFER_EINVAL, "too many tokens");
  const dim3 grid(rows, 1, ctas);
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  CK((dtype == DINFER_BF16 ? launch_sample<__nv_bfloat16>(a, grid, smem, s) : launch_sample<float>(a, grid, smem, s)));
  return DINFER_OK;
}

}  // extern "C"
