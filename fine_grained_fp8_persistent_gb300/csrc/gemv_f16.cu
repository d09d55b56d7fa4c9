// gemv_f16.cu -- launcher of the gated block with 16-bit weights for a few tokens (gemv.cuh).
#include "gemv.cuh"

namespace fgf8 {
namespace {

template <bool BF16>
int by_rows(const GemvKArgs& k, cudaStream_t stream) {
  return k.M <= 8 ? launch_gemv<WType::W16, BF16, 2, 1>(k, stream) : launch_gemv<WType::W16, BF16, 2, 2>(k, stream);
}

}  // namespace

int launch_gated_gemv_f16(const GatedArgs& a, const void* X, const void* Wg, const void* Wu, void* H, void* G, void* U,
                          cudaStream_t stream) {
  GemvKArgs k;
  std::memset(&k, 0, sizeof(k));
  k.X = X;
  k.W[0] = Wg;
  k.W[1] = Wu;
  k.out = H;
  k.keep[0] = G;
  k.keep[1] = U;
  k.M = a.M;
  k.N = a.N;
  k.K = a.K;
  k.act = a.act;
  return a.bf16 ? by_rows<true>(k, stream) : by_rows<false>(k, stream);
}

}  // namespace fgf8
