// Chunk attention over quantised pages (e4m3 codes, a scale per row), fp16 and bf16 queries.
#include "paged.cuh"

namespace sdpa {

namespace {
template <bool BF16>
cudaError_t launch(int D, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const PagedParams& p,
                   cudaStream_t st) {
  if (D == 64) return launch_paged_instance<BF16, true, 64, 64>(tq, tk, tv, p, st);
  if (D == 128) return launch_paged_instance<BF16, true, 128, 128>(tq, tk, tv, p, st);
  return launch_paged_instance<BF16, true, 192, 128>(tq, tk, tv, p, st);
}
}  // namespace

cudaError_t launch_paged_fp8(bool bf16, int D, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                             const PagedParams& p, cudaStream_t st) {
  return bf16 ? launch<true>(D, tq, tk, tv, p, st) : launch<false>(D, tq, tk, tv, p, st);
}

}  // namespace sdpa
