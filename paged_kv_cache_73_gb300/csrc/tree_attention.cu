// Attention of drafted tokens over a paged fp16 cache, for sm_103a: each sequence's new tokens, a
// chain or a tree, see its context and those of each other that their mask rows name; groups of
// query heads share a cached head.
//
//   o_i = sum_t softmax_t(scale q_i . k_t) v_t   over t < ctx - n and t = ctx - n + j, bit j of row i set
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "launch.cuh"
#include "pkv_internal.h"

namespace {

__device__ int g_dev_error_tree_attention = 0;
__device__ __forceinline__ void record_error(int code) { atomicCAS(&g_dev_error_tree_attention, 0, code); }

struct TreeParams {
  const __half* q;
  const __half* k;
  const __half* v;
  const int32_t* tables;
  const int32_t* lens;
  const int32_t* qstart;
  const uint32_t* mask;
  __half* out;
  int64_t q_stride;
  int mask_words, num_seqs, total_q, max_query_len;
  int num_heads, num_kv_heads, group, num_blocks, max_blocks, log2_block;
  float scale_log2;
};

// grid (heads, max_query_len, sequences), a warp each
template <int D>
__global__ void __launch_bounds__(32) tree_attention_kernel(const TreeParams p) {
  constexpr int V = D / 32;
  pkv::pdl_trigger();
  pkv::pdl_wait();
  const int h = blockIdx.x, i = blockIdx.y, s = blockIdx.z, lane = threadIdx.x, B = 1 << p.log2_block;
  const int q0 = p.qstart[s], n = p.qstart[s + 1] - q0, ctx = p.lens[s];
  if (n == 0 || i >= max(n, 1)) return;
  if (ctx < 0 || ctx > p.max_blocks * B) {
    if (lane == 0) record_error(PKV_DEV_BAD_CONTEXT_LEN);
    return;
  }
  if (n < 0 || n > ctx || n > p.max_query_len || q0 < 0 || q0 > p.total_q - n) {
    if (lane == 0) record_error(PKV_DEV_BAD_QUERY_RANGE);
    return;
  }
  float q[V], o[V], m = -INFINITY, l = 0.f;
  for (int c = 0; c < V; ++c) {
    q[c] = __half2float(p.q[(q0 + i) * p.q_stride + h * D + lane * V + c]);
    o[c] = 0.f;
  }
  for (int t = 0; t < ctx; ++t) {
    const int j = t - (ctx - n);
    if (j >= 0) {
      if (p.mask == nullptr ? j > i : (p.mask[static_cast<int64_t>(q0 + i) * p.mask_words + j / 32] >> (j % 32) & 1) == 0) continue;
    }
    const int phys = p.tables[static_cast<int64_t>(s) * p.max_blocks + (t >> p.log2_block)];
    if (phys < 0 || phys >= p.num_blocks) {
      if (lane == 0) record_error(PKV_DEV_BAD_BLOCK_ID);
      continue;
    }
    const int64_t at = (((static_cast<int64_t>(phys) * p.num_kv_heads + h / p.group) << p.log2_block) + (t & (B - 1))) * D + lane * V;
    float dot = 0.f;
    for (int c = 0; c < V; ++c) dot = fmaf(q[c], __half2float(p.k[at + c]), dot);
    for (int d = 16; d > 0; d /= 2) dot += __shfl_xor_sync(0xffffffffu, dot, d);
    const float x = dot * p.scale_log2, top = fmaxf(m, x), f = exp2f(m - top), w = exp2f(x - top);
    m = top;
    l = fmaf(l, f, w);
    for (int c = 0; c < V; ++c) o[c] = fmaf(o[c], f, w * __half2float(p.v[at + c]));
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  for (int c = 0; c < V; ++c)
    p.out[(static_cast<int64_t>(q0 + i) * p.num_heads + h) * D + lane * V + c] = __float2half_rn(o[c] * inv);
}

bool aligned16(const void* ptr) { return (reinterpret_cast<uintptr_t>(ptr) & 15u) == 0; }

}  // namespace

namespace pkv {
int device_error_word_tree_attention(void** word) {
  return static_cast<int>(cudaGetSymbolAddress(word, g_dev_error_tree_attention));
}
}  // namespace pkv

extern "C" {

size_t pkv_paged_attention_tree_workspace_size(int num_seqs, int total_q, int max_query_len, int num_heads,
                                               int num_kv_heads, int head_dim, int max_blocks_per_seq,
                                               int block_size) {
  (void)num_seqs, (void)total_q, (void)max_query_len, (void)num_heads, (void)num_kv_heads, (void)head_dim;
  (void)max_blocks_per_seq, (void)block_size;
  return 0;
}

int pkv_paged_attention_tree(const uint16_t* q, int64_t q_stride, const uint16_t* k_cache, const uint16_t* v_cache,
                             const int32_t* block_tables, const int32_t* context_lens, const int32_t* query_start,
                             const int32_t* tree_mask, int mask_words, int num_seqs, int total_q, int max_query_len,
                             int num_heads, int num_kv_heads, int head_dim, int num_blocks, int max_blocks_per_seq,
                             float scale, int block_size, uint16_t* out, void* workspace, size_t workspace_bytes,
                             void* stream) {
  const char* fn = "pkv_paged_attention_tree";
  if (num_seqs < 0 || total_q < 0 || max_query_len < 0 || num_heads <= 0 || num_kv_heads <= 0 || num_blocks <= 0 ||
      max_blocks_per_seq <= 0)
    return pkv::fail(PKV_ERR_INVALID_ARG,
                     "%s: num_seqs=%d total_q=%d max_query_len=%d num_heads=%d num_kv_heads=%d num_blocks=%d "
                     "max_blocks_per_seq=%d",
                     fn, num_seqs, total_q, max_query_len, num_heads, num_kv_heads, num_blocks, max_blocks_per_seq);
  if (num_heads % num_kv_heads)
    return pkv::fail(PKV_ERR_INVALID_ARG, "%s: num_heads=%d is not a multiple of num_kv_heads=%d", fn, num_heads,
                     num_kv_heads);
  if (head_dim != 64 && head_dim != 128)
    return pkv::fail(PKV_ERR_UNSUPPORTED, "%s: head_dim %d not in {64, 128}", fn, head_dim);
  if (block_size != 4 && block_size != 8 && block_size != 16 && block_size != 32)
    return pkv::fail(PKV_ERR_UNSUPPORTED, "%s: block_size %d not in {4, 8, 16, 32}", fn, block_size);
  if (tree_mask && (mask_words <= 0 || static_cast<long long>(mask_words) * 32 < max_query_len))
    return pkv::fail(PKV_ERR_INVALID_ARG, "%s: %d mask words a row for max_query_len=%d", fn, mask_words, max_query_len);
  if (num_seqs == 0 || total_q == 0 || max_query_len == 0) {
    pkv::clear_error();
    return PKV_OK;
  }
  if (num_seqs > 65535 || num_heads > 65535 || max_query_len > 65535)
    return pkv::fail(PKV_ERR_UNSUPPORTED, "%s: num_seqs/num_heads/max_query_len above 65535", fn);
  if (static_cast<long long>(max_blocks_per_seq) * block_size > (1LL << 30))
    return pkv::fail(PKV_ERR_UNSUPPORTED, "%s: context capacity above 2^30 tokens", fn);
  if (!q || !k_cache || !v_cache || !block_tables || !context_lens || !query_start || !out)
    return pkv::fail(PKV_ERR_INVALID_ARG, "%s: null pointer", fn);
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out) || !aligned16(workspace))
    return pkv::fail(PKV_ERR_INVALID_ARG, "%s: q, caches, out, workspace must be 16-byte aligned", fn);
  if (q_stride < static_cast<int64_t>(num_heads) * head_dim || q_stride % 8)
    return pkv::fail(PKV_ERR_INVALID_ARG, "%s: q_stride must be a multiple of 8 and at least a token's length", fn);
  if (!std::isfinite(scale) || !(scale > 0.f))
    return pkv::fail(PKV_ERR_INVALID_ARG, "%s: scale must be finite and positive", fn);
  (void)workspace_bytes;
  TreeParams p{};
  p.q = reinterpret_cast<const __half*>(q);
  p.k = reinterpret_cast<const __half*>(k_cache);
  p.v = reinterpret_cast<const __half*>(v_cache);
  p.tables = block_tables;
  p.lens = context_lens;
  p.qstart = query_start;
  p.mask = reinterpret_cast<const uint32_t*>(tree_mask);
  p.out = reinterpret_cast<__half*>(out);
  p.q_stride = q_stride;
  p.mask_words = mask_words;
  p.num_seqs = num_seqs;
  p.total_q = total_q;
  p.max_query_len = max_query_len;
  p.num_heads = num_heads;
  p.num_kv_heads = num_kv_heads;
  p.group = num_heads / num_kv_heads;
  p.num_blocks = num_blocks;
  p.max_blocks = max_blocks_per_seq;
  while ((1 << p.log2_block) < block_size) ++p.log2_block;
  p.scale_log2 = scale * 1.4426950408889634f;
  const dim3 grid(num_heads, max_query_len, num_seqs);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = head_dim == 128 ? pkv::launch_pdl(tree_attention_kernel<128>, grid, dim3(32), 0, st, p)
                                  : pkv::launch_pdl(tree_attention_kernel<64>, grid, dim3(32), 0, st, p);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) return pkv::fail(PKV_ERR_CUDA, "%s launch: %s", fn, cudaGetErrorString(e));
  pkv::clear_error();
  return PKV_OK;
}

}  // extern "C"
