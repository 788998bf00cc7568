// Shared by the kernels of the attention over the 4-bit cache: the split kernel for
// few query rows (lq_attn_q4.cu) and the one for many (lq_attn_q4_tiles.cu).  Internal
// to the library.
#pragma once

#include "lq_attn_paged.cuh"
#include "lq_q4.cuh"

namespace lq {
namespace q4 {

// attn::Args, without its cache, and the 4-bit one.
struct CacheArgs {
  attn::Args a;
  const uint8_t* kc;
  const uint8_t* vc;
  const uint32_t* ks;        // (scale, base) pairs
  const uint32_t* vs;
  int log2_group;
};

// Untiled copy of `bytes` (a multiple of 16) to shared memory, completing on `bar`.
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
               ::"r"(smem_addr(dst)), "l"(src), "r"(bytes), "r"(smem_addr(bar)) : "memory");
}

// The kernel for many query rows (lq_attn_q4_tiles.cu); most_tokens: positions that any
// request can have.
lq_status launch_tiles(const CacheArgs& ca, int head_dim, int64_t most_tokens, int sms, void* workspace, void* stream);
// Its workspace: what the CTAs that share a row leave of it, and where.
size_t tiles_workspace(int batch, int64_t total_q, int q_heads, int kv_heads, int head_dim, int sms);

}  // namespace q4
}  // namespace lq
