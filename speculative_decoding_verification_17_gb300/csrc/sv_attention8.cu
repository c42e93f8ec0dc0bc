// sv_attention8.cu — attention of a verify step's new positions over a paged cache in 8 bits: host
// side. The kernel is in sv_kv_tiles.cuh and sv_kv8_tiles.cuh.
#include <atomic>
#include <cstdint>

#include "specverify_kv8.h"
#include "sv_kv8.h"
#include "sv_kv8_tiles.cuh"

namespace sv {
namespace {

// Query rows per pass: as many whole positions as 64 columns hold (32 where D is 256, whose
// accumulators take twice the tensor memory), evenly over the passes.
void row_blocks8(const sv_kv_shape* s, int* pos_block, int* blocks, int* columns) {
  const int G = s->Hq / s->Hkv, most = (s->D == 256 ? 32 : 64) / G;
  *blocks = (s->P + most - 1) / most;
  *pos_block = (s->P + *blocks - 1) / *blocks;
  const int rows = G * *pos_block;
  *columns = rows <= 8 ? 8 : rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 48 ? 48 : 64;
}

sv_status check_shape8(const sv_kv_shape* s) {
  const sv_status ok = check_kv_shape(s, true);
  if (ok != SV_OK) return ok;
  return s->D == 256 && s->Hq / s->Hkv > 32 ? SV_ERR_UNSUPPORTED : SV_OK;
}

// Workspace: what each CTA leaves to join, then two pieces per CTA.
constexpr int kMaxCtasPerSm = 2;  // of every shape
struct Layout8 {
  size_t part, total;
};
Layout8 layout8(const sv_kv_shape* s) {
  int pos_block, blocks, columns;
  row_blocks8(s, &pos_block, &blocks, &columns);
  const size_t ctas = kMaxCtasPerSm * (size_t)device_sm_count();
  Layout8 L{};
  L.part = round_up(ctas * sizeof(JoinItem), 256);
  L.total = round_up(L.part + 2 * ctas * columns * (s->D + 2) * sizeof(float), 256);
  return L;
}

sv_status encode_pool8(CUtensorMap* map, const sv_kv_shape* s, const sv_kv_pool* pool) {
  const uint32_t box = s->page_size < kTileKeys ? s->page_size : kTileKeys;
  return encode_tiles(map, pool->data, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1,
                      s->D == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
                      CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                      {(uint64_t)s->D, (uint64_t)s->page_size, (uint64_t)s->Hkv,
                       (uint64_t)(s->num_pages > 0 ? s->num_pages : 1)},
                      {pool->token_stride, pool->head_stride, pool->page_stride},
                      {s->D == 64 ? 64u : 128u, box, 1u, 1u});
}

template <int D, int N, bool kBf16>
sv_status launch8(const TileArgs& A, const CUtensorMap& mk, const CUtensorMap& mv,
                  const ValuePool& v, cudaStream_t st) {
  using S = TileShape8<D, N, kBf16>;
  static_assert(S::CtasPerSm <= kMaxCtasPerSm, "the workspace holds two slots for each CTA");
  auto kernel = tile_kernel<S>;
  static std::atomic<uint64_t> ready{0};  // devices whose shared-memory limit is raised
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e);
  const uint64_t bit = 1ull << (dev & 63);
  if (dev > 63 || !(ready.load() & bit)) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::Smem);
    if (e != cudaSuccess) return cuda_fail(e);
    ready.fetch_or(bit);
  }
  const unsigned ctas = S::CtasPerSm * (unsigned)device_sm_count();
  kernel<<<ctas, S::Threads, S::Smem, st>>>(mk, mk, mv, A, v);  // (queries come without a map)
  const sv_status s = launch_status();
  if (s != SV_OK) return s;
  // the join takes its place while the tiles are still walked, and waits for their end
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(ctas, kJoinShares<D, N>);
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, join_kernel<D, N, kBf16>, (const JoinItem*)A.joins,
                         (const float*)A.part, A.G, A.Hq, A.out, A.out_lse);
  return e == cudaSuccess ? launch_status() : cuda_fail(e);
}

template <int D, bool kBf16>
sv_status launch_columns8(int columns, const TileArgs& A, const CUtensorMap& mk,
                          const CUtensorMap& mv, const ValuePool& v, cudaStream_t st) {
  switch (columns) {
    case 8: return launch8<D, 8, kBf16>(A, mk, mv, v, st);
    case 16: return launch8<D, 16, kBf16>(A, mk, mv, v, st);
    case 32: return launch8<D, 32, kBf16>(A, mk, mv, v, st);
    case 48: return launch8<D, D == 256 ? 32 : 48, kBf16>(A, mk, mv, v, st);
  }
  return launch8<D, D == 256 ? 32 : 64, kBf16>(A, mk, mv, v, st);
}

template <bool kBf16>
sv_status launch_width8(int D, int columns, const TileArgs& A, const CUtensorMap& mk,
                        const CUtensorMap& mv, const ValuePool& v, cudaStream_t st) {
  switch (D) {
    case 64: return launch_columns8<64, kBf16>(columns, A, mk, mv, v, st);
    case 128: return launch_columns8<128, kBf16>(columns, A, mk, mv, v, st);
  }
  return launch_columns8<256, kBf16>(columns, A, mk, mv, v, st);
}

sv_status attend8(const sv_kv_shape* shape, const sv_score_rule* rule, const void* q,
                  int64_t q_req, int64_t q_row, int64_t q_head, const sv_kv_pool* k,
                  const sv_kv_pool* v, const float* k_scale, const float* v_scale, int block,
                  const int32_t* page_table, const int32_t* seq_len, const int32_t* num_draft,
                  void* out, float* out_lse, void* workspace, size_t workspace_bytes,
                  uint64_t wait_ns, sv_stream_t stream) {
  sv_status s = check_shape8(shape);
  if (s != SV_OK) return s;
  s = check_rule(rule);
  if (s != SV_OK) return s;
  s = check_block(shape, block);
  if (s != SV_OK) return s;
  if (shape->B == 0) return SV_OK;
  if (check_pool8(k) != SV_OK || check_pool8(v) != SV_OK) return SV_ERR_INVALID_ARG;
  if (!q || !page_table || !seq_len || !k_scale || !v_scale || !out || !aligned_to(q, 16) ||
      !aligned_to(page_table, 4) || !aligned_to(seq_len, 4) || !aligned_to(num_draft, 4) ||
      !aligned_to(k_scale, 4) || !aligned_to(v_scale, 4) || !aligned_to(out, 16) ||
      !aligned_to(out_lse, 4))
    return SV_ERR_INVALID_ARG;
  for (int64_t st : {q_req, q_row, q_head})
    if (st < 0 || st % 8 != 0 || st >= (1ll << 39)) return SV_ERR_INVALID_ARG;
  if ((shape->B > 1 && q_req == 0) || (shape->P > 1 && q_row == 0) ||
      (shape->Hq > 1 && q_head == 0))
    return SV_ERR_INVALID_ARG;
  TileArgs A{};
  int columns;
  row_blocks8(shape, &A.pos_block, &A.blocks, &columns);
  if (!ranges_fit(shape, A.blocks)) return SV_ERR_UNSUPPORTED;
  const Layout8 L = layout8(shape);
  if (!workspace || !aligned_to(workspace, 256) || workspace_bytes < L.total)
    return SV_ERR_WORKSPACE;
  CUtensorMap mk, mv;
  s = encode_pool8(&mk, shape, k);
  if (s == SV_OK) s = encode_pool8(&mv, shape, v);
  if (s != SV_OK) return s;
  A.table = page_table;
  A.seq_len = seq_len;
  A.num_draft = num_draft;
  A.B = shape->B;
  A.P = shape->P;
  A.Hq = shape->Hq;
  A.Hkv = shape->Hkv;
  A.G = shape->Hq / shape->Hkv;
  A.log_page = log2_of(shape->page_size);
  A.log_block = log2_of(block);
  A.scale_page = (uint32_t)(shape->page_size / block) * (uint32_t)shape->Hkv;
  A.num_pages = shape->num_pages;
  A.max_pages = shape->max_pages;
  A.box = shape->page_size < kTileKeys ? shape->page_size : kTileKeys;
  A.bf16 = shape->dtype == SV_KV_BF16;
  A.rule = score_rule(rule);
  A.wait_ns = wait_ns;
  A.k_scale = k_scale;
  A.v_scale = v_scale;
  A.q = q;
  A.q_req = q_req;
  A.q_row = q_row;
  A.q_head = q_head;
  char* ws = static_cast<char*>(workspace);
  A.joins = reinterpret_cast<JoinItem*>(ws);
  A.part = reinterpret_cast<float*>(ws + L.part);
  A.out = out;
  A.out_lse = out_lse;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const ValuePool vp{v->data, v->page_stride, v->token_stride, v->head_stride};
  return A.bf16 ? launch_width8<true>(shape->D, columns, A, mk, mv, vp, st)
                : launch_width8<false>(shape->D, columns, A, mk, mv, vp, st);
}

}  // namespace
}  // namespace sv

using namespace sv;

extern "C" size_t paged_attention_q8_workspace(const sv_kv_shape* shape) {
  return check_shape8(shape) == SV_OK ? layout8(shape).total : 0;
}

extern "C" sv_status paged_attention_q8(
    const sv_kv_shape* shape, const sv_score_rule* rule, const void* q, int64_t q_req,
    int64_t q_row, int64_t q_head, const sv_kv_pool* k, const sv_kv_pool* v, const float* k_scale,
    const float* v_scale, int block, const int32_t* page_table, const int32_t* seq_len,
    const int32_t* num_draft, void* out, float* out_lse, void* workspace, size_t workspace_bytes,
    sv_stream_t stream) {
  return attend8(shape, rule, q, q_req, q_row, q_head, k, v, k_scale, v_scale, block, page_table,
                 seq_len, num_draft, out, out_lse, workspace, workspace_bytes, kTileWaitNs, stream);
}

extern "C" sv_status paged_attention_q8_wait_selftest(
    const sv_kv_shape* shape, const sv_score_rule* rule, const void* q, int64_t q_req,
    int64_t q_row, int64_t q_head, const sv_kv_pool* k, const sv_kv_pool* v, const float* k_scale,
    const float* v_scale, int block, const int32_t* page_table, const int32_t* seq_len,
    const int32_t* num_draft, void* out, float* out_lse, void* workspace, size_t workspace_bytes,
    unsigned int wait_us, sv_stream_t stream) {
  if (wait_us < 1 || wait_us > 100000) return SV_ERR_INVALID_ARG;
  return attend8(shape, rule, q, q_req, q_row, q_head, k, v, k_scale, v_scale, block, page_table,
                 seq_len, num_draft, out, out_lse, workspace, workspace_bytes,
                 (uint64_t)wait_us * 1000ull, stream);
}
