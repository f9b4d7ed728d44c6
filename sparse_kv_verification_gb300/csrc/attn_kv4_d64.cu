// Attention over a 4-bit cache, head dim 64 (attn_kv4.cuh).
#define DUSTIN_KV4_KERNEL
#include "attn_kv4.cuh"

namespace dustin {

cudaError_t launch_attn_kv4_d64(const Kv4KArgs& k, bool gather, cudaStream_t st) {
  return launch_kv4_rows<64>(k, gather, st);
}

cudaError_t take_attn_kv4_d64_flags(unsigned* flags) { return take_kv4_kernel_flags(flags); }

}  // namespace dustin
