// Host side of include/dinfer_kv.h: argument checks and launches.  Included at
// the end of dinfer_api.cu, whose launch, error and workspace helpers it uses.
#pragma once
#include "kv_attention.cuh"
#include "kv_pages.cuh"
#include "window_attention.cuh"
#include "window_attention_tc.cuh"

namespace {

// Why the cache description is unusable, or NULL.
const char* kv_bad(const dinfer_kv_cache* kc) {
  if (!kc) return "cache is NULL";
  if (!kc->k || !kc->v || !kc->table || !kc->lens || !kc->refs || !kc->state) return "cache: NULL buffer";
  if (kc->dtype != DINFER_BF16 && kc->dtype != DINFER_FP32) return "cache: unknown dtype";
  if (kc->head_dim != 64 && kc->head_dim != 128) return "cache: head_dim must be 64 or 128";
  if (kc->n_layers < 1 || kc->num_pages < 1 || kc->kv_heads < 1 || kc->kv_heads > 1024 || kc->page_size < 1 ||
      kc->page_size > 65536 || kc->max_seqs < 1 || kc->max_pages < 1)
    return "cache: size out of range";
  if ((int64_t)kc->max_pages * kc->page_size >= (1ll << 31)) return "cache: max_pages * page_size must be below 2^31";
  if ((int64_t)kc->page_size * kc->kv_heads * kc->head_dim >= (1ll << 31)) return "cache: page too large";
  if ((reinterpret_cast<uintptr_t>(kc->k) | reinterpret_cast<uintptr_t>(kc->v)) & 15)
    return "cache: k and v must be 16-byte aligned";
  if ((reinterpret_cast<uintptr_t>(kc->table) | reinterpret_cast<uintptr_t>(kc->lens) |
       reinterpret_cast<uintptr_t>(kc->refs) | reinterpret_cast<uintptr_t>(kc->state)) & 3)
    return "cache: misaligned table, lens, refs or state";
  // no two elements share a place: smallest stride first, each steps over all that the ones before it reach
  int64_t size[4] = {kc->n_layers, kc->num_pages, kc->page_size, kc->kv_heads};
  int64_t stride[4] = {kc->layer_stride, kc->page_stride, kc->token_stride, kc->head_stride};
  const int64_t per = kc->dtype == DINFER_BF16 ? 8 : 4;  // elements of 16 bytes
  for (int i = 0; i < 4; ++i)
    for (int j = i + 1; j < 4; ++j)
      if (stride[j] < stride[i]) {
        std::swap(stride[i], stride[j]);
        std::swap(size[i], size[j]);
      }
  int64_t reach = kc->head_dim;
  for (int i = 0; i < 4; ++i) {
    if (size[i] == 1) continue;
    if (stride[i] % per) return "cache: strides must be multiples of 16 bytes";
    if (stride[i] < reach || stride[i] > (1ll << 56) / size[i]) return "cache: strides overlap or are out of range";
    reach += (size[i] - 1) * stride[i];
  }
  return nullptr;
}

KvPages kv_pages(const dinfer_kv_cache& kc) {
  const int64_t per = kc.dtype == DINFER_BF16 ? 8 : 4;
  KvPages c{};
  c.k = (uint4*)kc.k;
  c.v = (uint4*)kc.v;
  // the stride of a dimension of one entry is never multiplied by more than 0
  c.layer_stride = kc.layer_stride / per;
  c.page_stride = kc.page_stride / per;
  c.token_stride = kc.token_stride / per;
  c.head_stride = kc.head_stride / per;
  c.table = kc.table;
  c.lens = kc.lens;
  c.refs = kc.refs;
  c.state = kc.state;
  c.n_layers = kc.n_layers;
  c.num_pages = kc.num_pages;
  c.page_size = kc.page_size;
  c.kv_heads = kc.kv_heads;
  c.head_vecs = (int)(kc.head_dim / per);
  c.max_seqs = kc.max_seqs;
  c.max_pages = kc.max_pages;
  c.page_div = FastDiv::make((uint32_t)kc.page_size);
  return c;
}

int log2_of(int x) {
  int s = 0;
  while ((1 << s) < x) ++s;
  return s;
}

// Shared-memory limits of this file's kernels, set once per device.
bool g_kv_setup[kMaxDevices] = {};

template <typename K>
bool max_smem(K* kernel, int bytes) {
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) == cudaSuccess;
}

template <typename T, int HD, int R>
bool kv_setup_attention() {
  return max_smem(kv_attention_kernel<T, HD, R>, KaCfg<T, HD, R>::kSmem);
}

template <int HD>
bool kv_setup_hd() {
  return kv_setup_attention<__nv_bfloat16, HD, 8>() && kv_setup_attention<__nv_bfloat16, HD, 16>() &&
         kv_setup_attention<float, HD, 1>() && kv_setup_attention<float, HD, 2>() && kv_setup_attention<float, HD, 4>() &&
         kv_setup_attention<float, HD, 8>() && max_smem(window_f32_kernel<HD, 4, false>, WfCfg<HD, 4>::kSmem) &&
         max_smem(window_f32_kernel<HD, 4, true>, WfCfg<HD, 4>::kSmem) &&
         max_smem(window_f32_kernel<HD, 16, false>, WfCfg<HD, 16>::kSmem) &&
         max_smem(window_tc_kernel<HD, false>, WtCfg<HD>::kSmem) &&
         max_smem(window_tc_kernel<HD, true>, WtCfg<HD>::kSmem);
}

bool kv_setup() {
  const int dev = current_device();
  std::lock_guard<std::mutex> lk(g_setup_mutex);
  if (!g_kv_setup[dev]) {
    g_kv_setup[dev] = kv_setup_hd<64>() && kv_setup_hd<128>();
    if (!g_kv_setup[dev]) cudaGetLastError();
  }
  return g_kv_setup[dev];
}

template <typename T, int HD, int R>
cudaError_t launch_kv_attention_r(const KaArgs& a, cudaStream_t s) {
  using Cfg = KaCfg<T, HD, R>;
  return launchk(kv_attention_kernel<T, HD, R>, dim3(num_sms()), dim3(Cfg::kThreads), Cfg::kSmem, s, 1, a);
}
template <int HD, int kTy, bool kSplit>
cudaError_t launch_window_f32(const WaArgs& a, dim3 grid, cudaStream_t s) {
  using Cfg = WfCfg<HD, kTy>;
  return launchk(window_f32_kernel<HD, kTy, kSplit>, grid, dim3(Cfg::kThreads), Cfg::kSmem, s, 1, a);
}
template <int HD, bool kSplit>
cudaError_t launch_window_tc(const WtMaps& maps, const WaArgs& a, int form, int blocks, dim3 grid, cudaStream_t s) {
  return launchk(window_tc_kernel<HD, kSplit>, grid, dim3(kWtThreads), WtCfg<HD>::kSmem, s, 1, maps, a, form, blocks);
}
// rows: the query heads a CTA takes at once (kv_rows)
template <int HD>
cudaError_t launch_kv_attention(const KaArgs& a, bool bf16, int rows, cudaStream_t s) {
  if (bf16) return rows == 8 ? launch_kv_attention_r<__nv_bfloat16, HD, 8>(a, s) : launch_kv_attention_r<__nv_bfloat16, HD, 16>(a, s);
  switch (rows) {
    case 1: return launch_kv_attention_r<float, HD, 1>(a, s);
    case 2: return launch_kv_attention_r<float, HD, 2>(a, s);
    case 4: return launch_kv_attention_r<float, HD, 4>(a, s);
    default: return launch_kv_attention_r<float, HD, 8>(a, s);
  }
}
// bf16: 8 or 16 rows of the tensor product; fp32: the smallest power of two, up to 8, that takes the group
int kv_rows(bool bf16, int group) {
  if (bf16) return group <= 8 ? 8 : 16;
  return group <= 1 ? 1 : group <= 2 ? 2 : group <= 4 ? 4 : 8;
}

KvMove kv_move(const dinfer_kv_cache& kc, const KvPages& c) {
  KvMove m{};
  m.vec_shift = log2_of(c.head_vecs);
  const int64_t vecs = (int64_t)c.page_size * c.kv_heads * c.head_vecs;
  m.parts = (int)((vecs + kKvPartVecs - 1) / kKvPartVecs);
  m.heads = FastDiv::make((uint32_t)c.kv_heads);
  m.head_major = kc.kv_heads > 1 && kc.head_stride > kc.token_stride;
  return m;
}

// A packed-head-rows operand: aligned, its row stride a multiple of 16 bytes
// and, where there is more than one row, no shorter than a row.
bool rows_ok(const void* p, int64_t stride, int64_t rows, int64_t row, int64_t per) {
  if (reinterpret_cast<uintptr_t>(p) & 15) return false;
  return rows <= 1 || (stride % per == 0 && stride >= row && stride < (1ll << 36));
}

// int32 operands (NULL where that is allowed): aligned
bool ints_ok(const void* a, const void* b = nullptr) {
  return ((reinterpret_cast<uintptr_t>(a) | reinterpret_cast<uintptr_t>(b)) & 3) == 0;
}

// bf16 rows [rows][heads][hd], `stride` elements apart: boxes of 128 rows x one
// head x 64 elements with the 128-byte swizzle; rows behind the last read as zeros.
bool make_map_rows(CUtensorMap* m, const void* base, int64_t rows, int64_t heads, int64_t hd, int64_t stride) {
  EncodeTiledFn enc = get_encode_fn();
  if (!enc) return false;
  cuuint64_t dims[3] = {(cuuint64_t)hd, (cuuint64_t)heads, (cuuint64_t)rows};
  cuuint64_t strides[2] = {(cuuint64_t)hd * 2, (cuuint64_t)(rows > 1 ? stride : heads * hd) * 2};
  cuuint32_t box[3] = {64, 1, kWtRows};
  cuuint32_t es[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

extern "C" {

size_t dinfer_kv_state_ints(int32_t num_pages, int32_t max_seqs) {
  if (num_pages < 1 || max_seqs < 1) return 0;
  return (size_t)kKvHead + max_seqs + kKvMaxEntries + 3 * (size_t)num_pages;
}

dinfer_status dinfer_kv_status(const dinfer_kv_cache* kc, uint32_t* bits, void* stream) {
  dinfer_ctx* c = nullptr;
  if (const char* why = kv_bad(kc)) return fail(c, DINFER_EINVAL, "%s", why);
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  uint32_t word = 0;
  CK(cudaMemcpyAsync(&word, kc->state, 4, cudaMemcpyDeviceToHost, s));
  CK(cudaStreamSynchronize(s));
  if (bits) *bits = word;
  if (!word) return DINFER_OK;
  CK(cudaMemsetAsync(kc->state, 0, 4, s));
  return fail(c, DINFER_EDEVICE, "paged cache: status 0x%x:%s%s%s%s%s", word,
              word & KV_BAD_SEQ ? " bad sequence number" : "", word & KV_NO_PAGES ? " out of pages" : "",
              word & KV_BAD_PAGE ? " bad page number in a table" : "",
              word & KV_SHARED ? " rows for a shared page" : "", word & KV_FULL ? " sequence too long" : "");
}

dinfer_status dinfer_kv_set(const dinfer_kv_cache* kc, const int32_t* table, const int32_t* lens, const int32_t* refs,
                            void* stream) {
  dinfer_ctx* c = nullptr;
  if (const char* why = kv_bad(kc)) return fail(c, DINFER_EINVAL, "%s", why);
  if (!table || !lens || !refs) return fail(c, DINFER_EINVAL, "NULL operand");
  if (!ints_ok(table, lens) || !ints_ok(refs))
    return fail(c, DINFER_EINVAL, "misaligned table, lens or refs");
  const int64_t most = std::max<int64_t>((int64_t)kc->max_seqs * kc->max_pages, kc->num_pages);
  const int grid = (int)std::min<int64_t>((most + 255) / 256, (int64_t)num_sms() * 8);
  CK(launchk(kv_set_kernel, dim3(grid), dim3(256), 0, reinterpret_cast<cudaStream_t>(stream), 1, kv_pages(*kc), table,
             lens, refs));
  return DINFER_OK;
}

dinfer_status dinfer_kv_extend(const dinfer_kv_cache* kc, const int32_t* seqs, const int32_t* add, int32_t n,
                               void* stream) {
  dinfer_ctx* c = nullptr;
  if (const char* why = kv_bad(kc)) return fail(c, DINFER_EINVAL, "%s", why);
  if (n < 1 || n > kKvMaxEntries) return fail(c, DINFER_EINVAL, "n must be 1 .. %d", kKvMaxEntries);
  if (!ints_ok(seqs, add)) return fail(c, DINFER_EINVAL, "misaligned seqs or add");
  CK(launchk(kv_extend_kernel, dim3(1), dim3(kKvPlanThreads), 0, reinterpret_cast<cudaStream_t>(stream), 1,
             kv_pages(*kc), seqs, add, (int)n));
  return DINFER_OK;
}

dinfer_status dinfer_kv_append(const dinfer_kv_cache* kc, int32_t layer, const int32_t* seqs, const int32_t* rows,
                               int32_t n, const void* k, const void* v, int64_t k_stride, int64_t v_stride,
                               int32_t total_rows, void* stream) {
  dinfer_ctx* c = nullptr;
  if (const char* why = kv_bad(kc)) return fail(c, DINFER_EINVAL, "%s", why);
  if (!k || !v) return fail(c, DINFER_EINVAL, "NULL operand");
  if (layer < 0 || layer >= kc->n_layers) return fail(c, DINFER_EINVAL, "no layer %d", layer);
  if (n < 1 || total_rows < 1 || (!rows && total_rows != n)) return fail(c, DINFER_EINVAL, "bad number of rows or entries");
  if (n > (seqs ? kKvMaxEntries : kc->max_seqs)) return fail(c, DINFER_EINVAL, "more entries than sequences, or than %d", kKvMaxEntries);
  const int64_t per = kc->dtype == DINFER_BF16 ? 8 : 4, row = (int64_t)kc->kv_heads * kc->head_dim;
  if (!rows_ok(k, k_stride, total_rows, row, per) || !rows_ok(v, v_stride, total_rows, row, per))
    return fail(c, DINFER_EINVAL, "k, v: 16-byte aligned rows at least a row apart are needed");
  if (!ints_ok(seqs, rows)) return fail(c, DINFER_EINVAL, "misaligned seqs or rows");
  const KvPages p = kv_pages(*kc);
  KvAppend a{};
  a.seqs = seqs;
  a.rows = rows;
  a.k = (const uint4*)k;
  a.v = (const uint4*)v;
  a.k_stride = k_stride / per;
  a.v_stride = v_stride / per;
  a.layer_off = layer * p.layer_stride;
  a.n = n;
  a.total_rows = total_rows;
  a.vec_shift = log2_of(p.head_vecs);
  const int64_t warps = 2 * (int64_t)total_rows;
  const int grid = (int)std::min<int64_t>((warps + 7) / 8, (int64_t)num_sms() * 8);
  CK(launchk(kv_append_kernel, dim3(grid), dim3(256), 0, reinterpret_cast<cudaStream_t>(stream), 1, p, a));
  return DINFER_OK;
}

dinfer_status dinfer_kv_fork(const dinfer_kv_cache* kc, const int32_t* src, const int32_t* dst, int32_t n,
                             int32_t share, void* stream) {
  dinfer_ctx* c = nullptr;
  if (const char* why = kv_bad(kc)) return fail(c, DINFER_EINVAL, "%s", why);
  if (!src || !dst) return fail(c, DINFER_EINVAL, "NULL operand");
  if (!ints_ok(src, dst)) return fail(c, DINFER_EINVAL, "misaligned src or dst");
  if (n < 1 || n > kKvMaxEntries) return fail(c, DINFER_EINVAL, "n must be 1 .. %d", kKvMaxEntries);
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const KvPages p = kv_pages(*kc);
  KvMove m = kv_move(*kc, p);
  m.src = src;
  m.dst = dst;
  m.n = n;
  m.share = share != 0;
  CK(launchk(kv_fork_plan_kernel, dim3(1), dim3(kKvPlanThreads), 0, s, 1, p, src, dst, (int)n, m.share));
  CK(launchk(kv_move_kernel<true>, dim3(num_sms() * 8), dim3(kKvMoveThreads), 0, s, 1, p, m));
  return DINFER_OK;
}

dinfer_status dinfer_kv_free(const dinfer_kv_cache* kc, const int32_t* seqs, int32_t n, void* stream) {
  dinfer_ctx* c = nullptr;
  if (const char* why = kv_bad(kc)) return fail(c, DINFER_EINVAL, "%s", why);
  if (!seqs) return fail(c, DINFER_EINVAL, "NULL operand");
  if (!ints_ok(seqs)) return fail(c, DINFER_EINVAL, "misaligned seqs");
  if (n < 1) return fail(c, DINFER_EINVAL, "n must be positive");
  CK(launchk(kv_free_kernel, dim3(n), dim3(128), 0, reinterpret_cast<cudaStream_t>(stream), 1, kv_pages(*kc), seqs));
  return DINFER_OK;
}

dinfer_status dinfer_kv_compact(const dinfer_kv_cache* kc, int32_t* live, void* stream) {
  dinfer_ctx* c = nullptr;
  if (const char* why = kv_bad(kc)) return fail(c, DINFER_EINVAL, "%s", why);
  if (!ints_ok(live)) return fail(c, DINFER_EINVAL, "misaligned live");
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const KvPages p = kv_pages(*kc);
  CK(launchk(kv_compact_plan_kernel, dim3(1), dim3(kKvPlanThreads), 0, s, 1, p, live));
  CK(launchk(kv_move_kernel<false>, dim3(num_sms() * 8), dim3(kKvMoveThreads), 0, s, 1, p, kv_move(*kc, p)));
  return DINFER_OK;
}

dinfer_status dinfer_kv_attention(const dinfer_kv_cache* kc, int32_t layer, const int32_t* seqs, int32_t n,
                                  const void* q, void* o, int64_t q_stride, int64_t o_stride, int32_t heads,
                                  int32_t window, int32_t sinks, float scale, void* workspace, size_t workspace_bytes,
                                  void* stream) {
  dinfer_ctx* c = nullptr;
  if (const char* why = kv_bad(kc)) return fail(c, DINFER_EINVAL, "%s", why);
  if (!q || !o) return fail(c, DINFER_EINVAL, "NULL operand");
  if (layer < 0 || layer >= kc->n_layers) return fail(c, DINFER_EINVAL, "no layer %d", layer);
  if (n < 1 || n > kKvMaxEntries) return fail(c, DINFER_EINVAL, "n must be 1 .. %d", kKvMaxEntries);
  if (heads < 1 || heads > 65536 || heads % kc->kv_heads) return fail(c, DINFER_EINVAL, "heads must be a multiple of kv_heads");
  if (sinks < 0 || !(scale > 0.f) || !std::isfinite(scale * 1.4426950408889634f)) return fail(c, DINFER_EINVAL, "bad sinks or scale");
  const int64_t per = kc->dtype == DINFER_BF16 ? 8 : 4, row = (int64_t)heads * kc->head_dim;
  if (!rows_ok(q, q_stride, n, row, per) || !rows_ok(o, o_stride, n, row, per))
    return fail(c, DINFER_EINVAL, "q, o: 16-byte aligned rows at least a row apart are needed");
  if (!ints_ok(seqs)) return fail(c, DINFER_EINVAL, "misaligned seqs");
  OpWs w;
  if (!op_ws(workspace, workspace_bytes, w)) return fail(c, DINFER_EINVAL, "workspace too small");
  if (reinterpret_cast<uintptr_t>(workspace) & 15) return fail(c, DINFER_EINVAL, "workspace must be 16-byte aligned");
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
  a.window = window < 0 ? -1 : window;
  a.sinks = sinks;
  a.min_steps = 8;
  a.in_place = o == q;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.partial = reinterpret_cast<float*>(w.data);
  a.tickets = w.tickets;
  const bool bf16 = kc->dtype == DINFER_BF16;
  const int rows = kv_rows(bf16, a.group);
  a.subgroups = (a.group + rows - 1) / rows;
  const int64_t most = std::min<int64_t>((int64_t)kc->max_pages * kc->page_size,
                                         window < 0 ? INT64_MAX : (int64_t)window + 1 + sinks);
  const int keys = bf16 ? KaCfg<__nv_bfloat16, 128, 8>::kKeys : KaCfg<float, 128, 8>::kKeys;
  if ((most / keys + 8 + kKaPairCost) * n * kc->kv_heads * a.subgroups >= (1ll << 31))
    return fail(c, DINFER_EINVAL, "more than 2^31 steps of keys in one call");
  const size_t slot = (2 * rows + 3) / 4 * 4 + rows * kc->head_dim;  // KaCfg::kSlotFloats
  if ((size_t)num_sms() * 2 * slot * 4 > w.data_bytes) return fail(c, DINFER_EINVAL, "workspace too small");
  if (!kv_setup()) return fail(c, DINFER_ECUDA, "kernel set-up failed");
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  CK(kc->head_dim == 128 ? launch_kv_attention<128>(a, bf16, rows, s) : launch_kv_attention<64>(a, bf16, rows, s));
  return DINFER_OK;
}

dinfer_status dinfer_op_window_attention(const void* q, const void* k, const void* v, void* o, int32_t dtype,
                                         int32_t batch, const int32_t* cu_q, const int32_t* cu_k, int32_t total_q,
                                         int32_t total_k, int32_t heads, int32_t kv_heads, int32_t head_dim,
                                         int64_t q_stride, int64_t k_stride, int64_t v_stride, int64_t o_stride,
                                         int32_t left, int32_t right, int32_t sinks, float scale, void* workspace,
                                         size_t workspace_bytes, void* stream) {
  dinfer_ctx* c = nullptr;
  if (!q || !k || !v || !o) return fail(c, DINFER_EINVAL, "NULL operand");
  if (dtype != DINFER_BF16 && dtype != DINFER_FP32) return fail(c, DINFER_EINVAL, "unknown dtype");
  if (head_dim != 64 && head_dim != 128) return fail(c, DINFER_EINVAL, "head_dim must be 64 or 128");
  if (batch < 1 || batch > 1024 || !cu_q != !cu_k || (!cu_q && batch != 1))
    return fail(c, DINFER_EINVAL, "batch must be 1 .. 1024, with cu_q and cu_k both given unless it is 1");
  if (total_q < 1 || total_k < 1 || total_q > (1 << 30) || total_k > (1 << 30)) return fail(c, DINFER_EINVAL, "unsupported number of rows");
  if (heads < 1 || heads > 65536 || kv_heads < 1 || heads % kv_heads) return fail(c, DINFER_EINVAL, "heads must be a multiple of kv_heads");
  if (sinks < 0 || !(scale > 0.f) || !std::isfinite(scale * 1.4426950408889634f)) return fail(c, DINFER_EINVAL, "bad sinks or scale");
  const int64_t per = dtype == DINFER_BF16 ? 8 : 4, qr = (int64_t)heads * head_dim, kr = (int64_t)kv_heads * head_dim;
  if (!rows_ok(q, q_stride, total_q, qr, per) || !rows_ok(o, o_stride, total_q, qr, per) ||
      !rows_ok(k, k_stride, total_k, kr, per) || !rows_ok(v, v_stride, total_k, kr, per))
    return fail(c, DINFER_EINVAL, "16-byte aligned rows at least a row apart are needed");
  if (!ints_ok(cu_q, cu_k)) return fail(c, DINFER_EINVAL, "misaligned cu_q or cu_k");
  OpWs w{};
  if (workspace && !op_ws(workspace, workspace_bytes, w)) return fail(c, DINFER_EINVAL, "workspace too small");
  if (reinterpret_cast<uintptr_t>(workspace) & 15) return fail(c, DINFER_EINVAL, "workspace must be 16-byte aligned");
  if (o == q || o == k || o == v) return fail(c, DINFER_EINVAL, "o must not overlap q, k or v");
  if (!kv_setup()) return fail(c, DINFER_ECUDA, "kernel set-up failed");
  WaArgs a{};
  a.q = q;
  a.k = k;
  a.v = v;
  a.o = o;
  a.cu_q = cu_q;
  a.cu_k = cu_k;
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.o_stride = o_stride;
  a.batch = batch;
  a.total_q = total_q;
  a.total_k = total_k;
  a.heads = heads;
  a.kv_heads = kv_heads;
  a.group = heads / kv_heads;
  a.left = left < 0 ? -1 : left;
  a.right = right < 0 ? -1 : right;
  a.sinks = sinks;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.status = w.st;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  // fp32: tiles of 64 rows once there are more full ones of them than run at once (two an SM), else of 16 (causal, heads
  // of 128: 1024 rows, 4 heads, 68 tiles of 64: 124 us, 85 with 16 rows; 4096 rows, 4 heads, 260 tiles: 745 and 638 us;
  // 4096 rows, 16 heads, 1040 tiles: 1.69 and 2.37 ms).  By the rows alone: the partly filled tiles that a batch adds
  // hold few rows, and are the cheaper the fewer rows a tile has.
  const bool small = dtype == DINFER_FP32 && (int64_t)(total_q / 64 + 1) * heads <= 2 * num_sms();
  // bf16: two tiles a CTA, or one while there is an SM for each (1024 causal rows, 16 heads of 128, 144 tiles: 15.2 us
  // alone, 18.3 in pairs; 18 heads, 162 tiles: pairs 19.1)
  const int form = (int64_t)(total_q / kWtRows + batch) * heads <= num_sms() ? kWtSingle
                   : a.group % 2 == 0                                        ? kWtPairHeads
                                                                             : kWtPairRows;
  const int block_rows = dtype == DINFER_FP32 ? (small ? 16 : 64) : form == kWtPairRows ? 2 * kWtRows : kWtRows;
  const int blocks = total_q / block_rows + batch;  // every sequence adds at most one partly filled tile
  int64_t ctas = (int64_t)blocks * (dtype == DINFER_BF16 && form == kWtPairHeads ? heads / 2 : heads);
  a.splits = 1;
  if (workspace && (dtype == DINFER_FP32 ? small : form == kWtSingle)) {
    // SMs to spare: a tile's keys go to several of them (fp32: two CTAs an SM)
    const bool f32 = dtype == DINFER_FP32;
    const int64_t slot = 4ll * (f32 ? (head_dim == 128 ? WfCfg<128, 4>::kSlotFloats : WfCfg<64, 4>::kSlotFloats)
                                    : (head_dim == 128 ? WtCfg<128>::kSlotFloats : WtCfg<64>::kSlotFloats));
    const int most = f32 ? total_k / kWfKeys / kWfPartTiles : total_k / kWtKeys / kWtPartTiles;
    const int splits = (int)std::min<int64_t>((f32 ? 2 : 1) * num_sms() / ctas, most);
    if (splits > 1 && ctas * splits * slot <= (int64_t)w.data_bytes) {
      a.splits = splits;
      a.partial = reinterpret_cast<float*>(w.data);
      a.tickets = w.tickets;
      ctas *= splits;
    }
  }
  if (ctas >= (1ll << 31)) return fail(c, DINFER_EINVAL, "too many rows");
  const dim3 grid((unsigned)ctas);
  if (dtype == DINFER_FP32) {
    // Causal rows see the more keys the later they come: where the CTAs do not all start at once, the last ones go
    // first (16 heads of 64, 4096 rows: 940 us, else 1077).
    a.last_first = ctas > 2 * num_sms();
    const bool split = a.splits > 1;
    CK(head_dim == 128 ? (split   ? launch_window_f32<128, 4, true>(a, grid, s)
                          : small ? launch_window_f32<128, 4, false>(a, grid, s)
                                  : launch_window_f32<128, 16, false>(a, grid, s))
                       : (split   ? launch_window_f32<64, 4, true>(a, grid, s)
                          : small ? launch_window_f32<64, 4, false>(a, grid, s)
                                  : launch_window_f32<64, 16, false>(a, grid, s)));
    return DINFER_OK;
  }
  WtMaps maps;
  if (!make_map_rows(&maps.q, q, total_q, heads, head_dim, q_stride) ||
      !make_map_rows(&maps.k, k, total_k, kv_heads, head_dim, k_stride) ||
      !make_map_rows(&maps.v, v, total_k, kv_heads, head_dim, v_stride))
    return fail(c, DINFER_EINVAL, "tensor map encoding failed");
  const bool split = a.splits > 1;
  CK(head_dim == 128 ? (split ? launch_window_tc<128, true>(maps, a, form, blocks, grid, s)
                              : launch_window_tc<128, false>(maps, a, form, blocks, grid, s))
                     : (split ? launch_window_tc<64, true>(maps, a, form, blocks, grid, s)
                              : launch_window_tc<64, false>(maps, a, form, blocks, grid, s)));
  return DINFER_OK;
}

}  // extern "C"
