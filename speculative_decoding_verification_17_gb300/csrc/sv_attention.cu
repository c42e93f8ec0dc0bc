// sv_attention.cu — attention of a verify step's new positions over a paged cache: host side.
// The kernel is in sv_kv_tiles.cuh; sv_keyweight.cu holds the key weights' host side.
#include <atomic>
#include <cstdint>

#include "specverify_kv.h"
#include "sv_kv_tiles.cuh"

namespace sv {

namespace {

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                              const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                              const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The driver's encoder, looked up once (the library does not link against the driver).
EncodeFn encoder() {
  static std::atomic<EncodeFn> cached{nullptr};
  EncodeFn f = cached.load();
  if (f) return f;
  void* p = nullptr;
  cudaDriverEntryPointQueryResult found;
  if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                       &found) != cudaSuccess ||
      found != cudaDriverEntryPointSuccess)
    return nullptr;
  f = reinterpret_cast<EncodeFn>(p);
  cached.store(f);
  return f;
}

}  // namespace

sv_status encode_tiles(CUtensorMap* map, const void* data, CUtensorMapDataType type, int size,
                       CUtensorMapSwizzle swizzle, CUtensorMapL2promotion promotion,
                       const uint64_t (&dims)[4],
                       const int64_t (&strides)[3], const uint32_t (&box)[4]) {
  const EncodeFn f = encoder();
  if (!f) return cuda_fail(cudaErrorSymbolNotFound);
  cuuint64_t d[4], s[3];
  cuuint32_t b[4];
  const cuuint32_t ones[4] = {1, 1, 1, 1};
  for (int i = 0; i < 4; ++i) {
    d[i] = dims[i];
    b[i] = box[i];
  }
  // a dimension of one element is never stepped along: any stride will do
  for (int i = 0; i < 3; ++i) s[i] = dims[i + 1] == 1 ? 16 : (cuuint64_t)strides[i] * size;
  const CUresult r = f(map, type, 4, const_cast<void*>(data), d, s, b, ones,
                       CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, promotion,
                       CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? SV_OK : cuda_fail(cudaErrorInvalidValue);
}

sv_status encode_map(CUtensorMap* map, const void* data, bool bf16, const uint64_t (&dims)[4],
                     const int64_t (&strides)[3], const uint32_t (&box)[4]) {
  return encode_tiles(map, data,
                      bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2,
                      CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, dims, strides,
                      box);
}

sv_status encode_pool(CUtensorMap* map, const sv_kv_shape* s, const sv_kv_pool* pool) {
  const uint32_t box = s->page_size < kTileKeys ? s->page_size : kTileKeys;
  return encode_map(map, pool->data, s->dtype == SV_KV_BF16,
                    {(uint64_t)s->D, (uint64_t)s->page_size, (uint64_t)s->Hkv,
                     (uint64_t)(s->num_pages > 0 ? s->num_pages : 1)},
                    {pool->token_stride, pool->head_stride, pool->page_stride},
                    {64u, box, 1u, 1u});
}

sv_status check_tile_call(const sv_kv_shape* s, const sv_score_rule* rule, const void* q,
                          int64_t q_req, int64_t q_row, int64_t q_head, const sv_kv_pool* k,
                          const int32_t* page_table, const int32_t* seq_len,
                          const int32_t* num_draft) {
  const sv_status ok = check_kv_shape(s, true);
  if (ok != SV_OK) return ok;
  const sv_status okr = check_rule(rule);
  if (okr != SV_OK) return okr;
  if (s->B == 0) return SV_OK;
  const sv_status okp = check_pool(k);
  if (okp != SV_OK) return okp;
  if (!q || !page_table || !seq_len || !aligned_to(q, 16) || !aligned_to(page_table, 4) ||
      !aligned_to(seq_len, 4) || !aligned_to(num_draft, 4))
    return SV_ERR_INVALID_ARG;
  for (int64_t st : {q_req, q_row, q_head})
    if (st < 0 || st % 8 != 0 || st >= (1ll << 39)) return SV_ERR_INVALID_ARG;
  if ((s->B > 1 && q_req == 0) || (s->P > 1 && q_row == 0) || (s->Hq > 1 && q_head == 0))
    return SV_ERR_INVALID_ARG;
  return SV_OK;
}

sv_status fill_tile_args(TileArgs& A, CUtensorMap* mq, CUtensorMap* mk, const sv_kv_shape* s,
                         const sv_score_rule* rule, const void* q, int64_t q_req, int64_t q_row,
                         int64_t q_head, const sv_kv_pool* k, const int32_t* page_table,
                         const int32_t* seq_len, const int32_t* num_draft, bool weigh) {
  A = TileArgs{};
  A.table = page_table;
  A.seq_len = seq_len;
  A.num_draft = num_draft;
  A.B = s->B;
  A.P = s->P;
  A.Hq = s->Hq;
  A.Hkv = s->Hkv;
  A.G = s->Hq / s->Hkv;
  A.log_page = log2_of(s->page_size);
  A.num_pages = s->num_pages;
  A.max_pages = s->max_pages;
  int columns;
  row_blocks(s, weigh, &A.pos_block, &A.blocks, &columns);
  if (!ranges_fit(s, A.blocks)) return SV_ERR_UNSUPPORTED;
  A.box = s->page_size < kTileKeys ? s->page_size : kTileKeys;
  A.bf16 = s->dtype == SV_KV_BF16;
  A.rule = score_rule(rule);
  A.wait_ns = kTileWaitNs;
  const sv_status ok = encode_map(
      mq, q, A.bf16, {(uint64_t)s->D, (uint64_t)s->Hq, (uint64_t)s->P, (uint64_t)s->B},
      {q_head, q_row, q_req}, {64u, (uint32_t)A.G, (uint32_t)A.pos_block, 1u});
  return ok != SV_OK ? ok : encode_pool(mk, s, k);
}

namespace {

// Workspace: what each CTA leaves to join, then two pieces per CTA.
struct AttnLayout {
  size_t part, total;
};
AttnLayout attn_layout(const sv_kv_shape* s) {
  int pos_block, blocks, columns;
  row_blocks(s, false, &pos_block, &blocks, &columns);
  const size_t ctas = (size_t)device_sm_count();
  AttnLayout L{};
  L.part = round_up(ctas * sizeof(JoinItem), 256);
  L.total = round_up(L.part + 2 * ctas * columns * (s->D + 2) * sizeof(float), 256);
  return L;
}

template <int D, int N, bool kBf16>
sv_status launch_attention(const TileArgs& A, const CUtensorMap& mq, const CUtensorMap& mk,
                           const CUtensorMap& mv, const ValuePool& v, cudaStream_t st) {
  using S = TileShape<D, N, false, kBf16>;
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
  const unsigned ctas = (unsigned)device_sm_count();
  kernel<<<ctas, S::Threads, S::Smem, st>>>(mq, mk, mv, A, v);
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
sv_status launch_columns(int columns, const TileArgs& A, const CUtensorMap& mq,
                         const CUtensorMap& mk, const CUtensorMap& mv, const ValuePool& v,
                         cudaStream_t st) {
  switch (columns) {
    case 16: return launch_attention<D, 16, kBf16>(A, mq, mk, mv, v, st);
    case 32: return launch_attention<D, 32, kBf16>(A, mq, mk, mv, v, st);
    case 64: return launch_attention<D, 64, kBf16>(A, mq, mk, mv, v, st);
  }
  return launch_attention<D, D == 256 ? 64 : 128, kBf16>(A, mq, mk, mv, v, st);
}

template <bool kBf16>
sv_status launch_width(int D, int columns, const TileArgs& A, const CUtensorMap& mq,
                       const CUtensorMap& mk, const CUtensorMap& mv, const ValuePool& v,
                       cudaStream_t st) {
  switch (D) {
    case 64: return launch_columns<64, kBf16>(columns, A, mq, mk, mv, v, st);
    case 128: return launch_columns<128, kBf16>(columns, A, mq, mk, mv, v, st);
  }
  return launch_columns<256, kBf16>(columns, A, mq, mk, mv, v, st);
}

sv_status attend(const sv_kv_shape* shape, const sv_score_rule* rule, const void* q,
                 int64_t q_req, int64_t q_row, int64_t q_head, const sv_kv_pool* k,
                 const sv_kv_pool* v, const int32_t* page_table, const int32_t* seq_len,
                 const int32_t* num_draft, void* out, float* out_lse, void* workspace,
                 size_t workspace_bytes, uint64_t wait_ns, sv_stream_t stream) {
  const sv_status ok = check_tile_call(shape, rule, q, q_req, q_row, q_head, k, page_table,
                                       seq_len, num_draft);
  if (ok != SV_OK) return ok;
  if (shape->B == 0) return SV_OK;
  const sv_status okv = check_pool(v);
  if (okv != SV_OK) return okv;
  if (!out || !aligned_to(out, 16) || !aligned_to(out_lse, 4)) return SV_ERR_INVALID_ARG;
  const AttnLayout L = attn_layout(shape);
  if (!workspace || !aligned_to(workspace, 256) || workspace_bytes < L.total)
    return SV_ERR_WORKSPACE;
  TileArgs A;
  CUtensorMap mq, mk, mv;
  sv_status s = fill_tile_args(A, &mq, &mk, shape, rule, q, q_req, q_row, q_head, k, page_table,
                               seq_len, num_draft, false);
  if (s == SV_OK) s = encode_pool(&mv, shape, v);
  if (s != SV_OK) return s;
  A.wait_ns = wait_ns;
  char* ws = static_cast<char*>(workspace);
  A.joins = reinterpret_cast<JoinItem*>(ws);
  A.part = reinterpret_cast<float*>(ws + L.part);
  A.out = out;
  A.out_lse = out_lse;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const ValuePool vp{v->data, v->page_stride, v->token_stride, v->head_stride};
  int pos_block, blocks, columns;
  row_blocks(shape, false, &pos_block, &blocks, &columns);
  return A.bf16 ? launch_width<true>(shape->D, columns, A, mq, mk, mv, vp, st)
                : launch_width<false>(shape->D, columns, A, mq, mk, mv, vp, st);
}

}  // namespace
}  // namespace sv

using namespace sv;

extern "C" size_t paged_attention_workspace(const sv_kv_shape* shape) {
  return check_kv_shape(shape, true) == SV_OK ? attn_layout(shape).total : 0;
}

extern "C" sv_status paged_attention(const sv_kv_shape* shape, const sv_score_rule* rule,
                                     const void* q, int64_t q_req, int64_t q_row,
                                     int64_t q_head, const sv_kv_pool* k, const sv_kv_pool* v,
                                     const int32_t* page_table, const int32_t* seq_len,
                                     const int32_t* num_draft, void* out, float* out_lse,
                                     void* workspace, size_t workspace_bytes,
                                     sv_stream_t stream) {
  return attend(shape, rule, q, q_req, q_row, q_head, k, v, page_table, seq_len, num_draft, out,
                out_lse, workspace, workspace_bytes, kTileWaitNs, stream);
}

extern "C" sv_status paged_attention_wait_selftest(
    const sv_kv_shape* shape, const sv_score_rule* rule, const void* q, int64_t q_req,
    int64_t q_row, int64_t q_head, const sv_kv_pool* k, const sv_kv_pool* v,
    const int32_t* page_table, const int32_t* seq_len, const int32_t* num_draft, void* out,
    float* out_lse, void* workspace, size_t workspace_bytes, unsigned int wait_us,
    sv_stream_t stream) {
  if (wait_us < 1 || wait_us > 100000) return SV_ERR_INVALID_ARG;
  return attend(shape, rule, q, q_req, q_row, q_head, k, v, page_table, seq_len, num_draft, out,
                out_lse, workspace, workspace_bytes, (uint64_t)wait_us * 1000ull, stream);
}
