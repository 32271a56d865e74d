// Latent attention in its expanded form: the chunk attention over packed keys, f16 and bf16.
#include "paged.cuh"

namespace sdpa {

cudaError_t launch_paged_packed(bool bf16, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                                const CUtensorMap& tr, const PagedParams& p, cudaStream_t st) {
  if (p.one)
    return bf16 ? launch_paged_one<true, false, 192, 128, true, true>(tq, tk, tv, tr, p, st)
                : launch_paged_one<false, false, 192, 128, true, true>(tq, tk, tv, tr, p, st);
  return bf16 ? launch_paged_one<true, false, 192, 128, false, true>(tq, tk, tv, tr, p, st)
              : launch_paged_one<false, false, 192, 128, false, true>(tq, tk, tv, tr, p, st);
}

}  // namespace sdpa
