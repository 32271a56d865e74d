// Chunk attention over 16-bit pages, bf16.
#include "paged.cuh"

namespace sdpa {

cudaError_t launch_paged_bf16(int D, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                             const PagedParams& p, cudaStream_t st) {
  if (D == 64) return launch_paged_instance<true, false, 64, 64>(tq, tk, tv, p, st);
  if (D == 128) return launch_paged_instance<true, false, 128, 128>(tq, tk, tv, p, st);
  return launch_paged_instance<true, false, 192, 128>(tq, tk, tv, p, st);
}

}  // namespace sdpa
