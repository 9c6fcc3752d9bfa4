// kvq_fp4_host.h -- argument checks that the 4-bit cache's entry points share.
#pragma once

#include "../../include/kvq_fp4.h"
#include "kvq_host.h"

namespace kvq {
namespace fp4 {

inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

inline int check_scales(const float* k_scale, int k_len, const float* v_scale, int v_len, int gran,
                        int num_kv_heads) {
  if (gran != KVQ_SCALE_PER_TENSOR && gran != KVQ_SCALE_PER_HEAD) return KVQ_ERR_ARG;
  if (!k_scale || !v_scale) return KVQ_ERR_NULL;
  const int want = gran == KVQ_SCALE_PER_HEAD ? num_kv_heads : 1;
  if (k_len != want || v_len != want) return KVQ_ERR_SHAPE;
  return aligned4(k_scale) && aligned4(v_scale) ? KVQ_OK : KVQ_ERR_ALIGN;
}

// The caches' sizes: their byte offsets fit 63 bits.
inline int check_caches(int64_t num_blocks, int block_size, int num_kv_heads, int head_dim) {
  if (head_dim != 64 && head_dim != 128) return KVQ_ERR_UNSUPPORTED;
  if (block_size != 16) return KVQ_ERR_UNSUPPORTED;
  if (num_kv_heads > 65535) return KVQ_ERR_UNSUPPORTED;
  if (num_blocks > (INT64_MAX / 16) / (static_cast<int64_t>(num_kv_heads) * head_dim))
    return KVQ_ERR_SHAPE;
  return KVQ_OK;
}

// What the two attentions check alike.  Without rows q and out may be NULL, as empty tensors' are.
inline int check_attn(bool rows, const void* q, const void* k_cache, const void* v_cache,
                      const int32_t* block_tables, int max_blocks, const int32_t* seq_lens,
                      int num_seqs, int hq, int hkv, int dh, int64_t num_blocks, int block_size,
                      const float* k_scale, int k_len, const float* v_scale, int v_len, int gran,
                      int window, int sinks, const void* workspace, const void* out) {
  if (num_seqs <= 0 || hq <= 0 || hkv <= 0 || num_blocks <= 0 || max_blocks <= 0 || window < 0 ||
      sinks < 0)
    return KVQ_ERR_ARG;
  int st = check_scales(k_scale, k_len, v_scale, v_len, gran, hkv);
  if (st != KVQ_OK) return st;
  if (!k_cache || !v_cache || !block_tables || !seq_lens || !workspace || (rows && (!q || !out)))
    return KVQ_ERR_NULL;
  st = check_caches(num_blocks, block_size, hkv, dh);
  if (st != KVQ_OK) return st;
  if (hq % hkv) return KVQ_ERR_SHAPE;
  if (hq / hkv > 8 || hkv > 256) return KVQ_ERR_UNSUPPORTED;
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out) ||
      (reinterpret_cast<uintptr_t>(workspace) & 255u) || !aligned4(block_tables) ||
      !aligned4(seq_lens))
    return KVQ_ERR_ALIGN;
  return KVQ_OK;
}

}  // namespace fp4
}  // namespace kvq
