// attention_blocks.cu -- decode attention over listed packed blocks and the
// window (see block_attention.cuh).
#include "block_attention.cuh"

namespace kivi {

cudaError_t launch_attention_list(const CacheView& cv, const AttnArgs& a, const SeqLens& lens, cudaStream_t st) {
  // bf16 outputs round by up to 2^-8 of themselves, one fp16 weight a token by up to
  // 2^-11: 1.69e-3 off 64 bits for 1.66e-3 with pairs (64 sequences of up to 24
  // listed blocks, seven heads a KV head: 21.5 us, 26.2 as pairs).  The attention
  // with block weights keeps pairs for every type: it sums the weights before
  // they are rounded, and its products stay those of f16 and f32 lists.
  if (a.q_dtype == kBF16) return launch_block_attention<kAttnListOne>(cv, a, lens, st);
  return launch_block_attention<kAttnList>(cv, a, lens, st);
}

}  // namespace kivi
