// sv_keyweight.cu — the softmax weight each cached key received: host side. The kernel is in
// sv_kv_tiles.cuh: the scores' half of the attention, with the rows' known log-sum-exp in
// place of the running maximum and a sum over the columns in place of the product with V.
#include <atomic>
#include <cstdint>

#include "specverify_kv.h"
#include "sv_kv_tiles.cuh"

namespace sv {
namespace {

template <int D, int N>
sv_status launch_weights(const TileArgs& A, const CUtensorMap& mq, const CUtensorMap& mk,
                         cudaStream_t st) {
  using S = TileShape<D, N, true>;
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
  kernel<<<(unsigned)device_sm_count(), S::Threads, S::Smem, st>>>(mq, mk, mk, A, ValuePool{});
  return launch_status();
}

template <int D>
sv_status launch_columns(int columns, const TileArgs& A, const CUtensorMap& mq,
                         const CUtensorMap& mk, cudaStream_t st) {
  switch (columns) {
    case 16: return launch_weights<D, 16>(A, mq, mk, st);
    case 32: return launch_weights<D, 32>(A, mq, mk, st);
    case 64: return launch_weights<D, 64>(A, mq, mk, st);
    default: return launch_weights<D, 128>(A, mq, mk, st);
  }
}

sv_status weigh(const sv_kv_shape* shape, const sv_score_rule* rule, const void* q, int64_t q_req,
                int64_t q_row, int64_t q_head, const sv_kv_pool* k, const int32_t* page_table,
                const int32_t* seq_len, const int32_t* num_draft, const float* lse,
                int64_t lse_req, int64_t lse_row, int64_t lse_head, const int32_t* accept_len,
                const float* prior, float* out, int64_t stride, uint64_t wait_ns,
                sv_stream_t stream) {
  const sv_status ok = check_tile_call(shape, rule, q, q_req, q_row, q_head, k, page_table,
                                       seq_len, num_draft);
  if (ok != SV_OK) return ok;
  if (stride < 1 || lse_req < 0 || lse_row < 0 || lse_head < 0) return SV_ERR_INVALID_ARG;
  if (shape->B == 0) return SV_OK;
  if (!lse || !out || !aligned_to(lse, 4) || !aligned_to(out, 4) || !aligned_to(prior, 4) ||
      !aligned_to(accept_len, 4))
    return SV_ERR_INVALID_ARG;
  TileArgs A;
  CUtensorMap mq, mk;
  const sv_status s = fill_tile_args(A, &mq, &mk, shape, rule, q, q_req, q_row, q_head, k,
                                     page_table, seq_len, num_draft, true);
  if (s != SV_OK) return s;
  A.accept_len = accept_len;
  A.lse = lse;
  A.lse_req = lse_req;
  A.lse_row = lse_row;
  A.lse_head = lse_head;
  A.prior = prior;
  A.weights = out;
  A.stride = stride;
  A.wait_ns = wait_ns;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  int pos_block, blocks, columns;
  row_blocks(shape, true, &pos_block, &blocks, &columns);
  switch (shape->D) {
    case 64: return launch_columns<64>(columns, A, mq, mk, st);
    case 128: return launch_columns<128>(columns, A, mq, mk, st);
    default: return launch_columns<256>(columns, A, mq, mk, st);
  }
}

}  // namespace
}  // namespace sv

using namespace sv;

extern "C" sv_status attention_weight_sum(const sv_kv_shape* shape, const sv_score_rule* rule,
                                          const void* q, int64_t q_req, int64_t q_row,
                                          int64_t q_head, const sv_kv_pool* k,
                                          const int32_t* page_table, const int32_t* seq_len,
                                          const int32_t* num_draft, const float* lse,
                                          int64_t lse_req, int64_t lse_row, int64_t lse_head,
                                          const int32_t* accept_len, const float* prior,
                                          float* out, int64_t stride, sv_stream_t stream) {
  return weigh(shape, rule, q, q_req, q_row, q_head, k, page_table, seq_len, num_draft, lse,
               lse_req, lse_row, lse_head, accept_len, prior, out, stride, kTileWaitNs, stream);
}

extern "C" sv_status attention_weight_sum_wait_selftest(
    const sv_kv_shape* shape, const sv_score_rule* rule, const void* q, int64_t q_req,
    int64_t q_row, int64_t q_head, const sv_kv_pool* k, const int32_t* page_table,
    const int32_t* seq_len, const int32_t* num_draft, const float* lse, int64_t lse_req,
    int64_t lse_row, int64_t lse_head, const int32_t* accept_len, const float* prior, float* out,
    int64_t stride, unsigned int wait_us, sv_stream_t stream) {
  if (wait_us < 1 || wait_us > 100000) return SV_ERR_INVALID_ARG;
  return weigh(shape, rule, q, q_req, q_row, q_head, k, page_table, seq_len, num_draft, lse,
               lse_req, lse_row, lse_head, accept_len, prior, out, stride,
               (uint64_t)wait_us * 1000ull, stream);
}
