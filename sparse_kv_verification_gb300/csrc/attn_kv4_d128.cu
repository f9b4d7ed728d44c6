// Attention over a 4-bit cache, head dim 128 (attn_kv4.cuh).
#define DUSTIN_KV4_KERNEL
#include "attn_kv4.cuh"

namespace dustin {

cudaError_t launch_attn_kv4_d128(const Kv4KArgs& k, bool gather, cudaStream_t st) {
  return launch_kv4_rows<128>(k, gather, st);
}

cudaError_t take_attn_kv4_d128_flags(unsigned* flags) { return take_kv4_kernel_flags(flags); }

}  // namespace dustin
