// gemv_fp4.cu -- launcher of the products of a few rows of X with 4-bit weights, plain
// or gated (gemv.cuh).
#include "gemv.cuh"

namespace fgf8 {
namespace {

// eight tokens per N = 8 instruction
template <WType WT, bool BF16, int MATS>
int by_rows(const GemvKArgs& k, cudaStream_t stream) {
  return k.M <= 8 ? launch_gemv<WT, BF16, MATS, 1>(k, stream) : launch_gemv<WT, BF16, MATS, 2>(k, stream);
}

template <WType WT>
int by_type(const GemvArgs& a, const GemvKArgs& k, cudaStream_t stream) {
  if (a.act >= 0) return a.bf16 ? by_rows<WT, true, 2>(k, stream) : by_rows<WT, false, 2>(k, stream);
  return a.bf16 ? by_rows<WT, true, 1>(k, stream) : by_rows<WT, false, 1>(k, stream);
}

}  // namespace

int launch_gemv_fp4(const GemvArgs& a, cudaStream_t stream) {
  GemvKArgs k;
  std::memset(&k, 0, sizeof(k));
  k.X = a.X;
  for (int j = 0; j < 2; ++j) {
    k.W[j] = a.W[j];
    k.SF[j] = a.SF[j];
  }
  k.out = a.out;
  k.M = a.M;
  k.N = a.N;
  k.K = a.K;
  k.act = a.act;
  return a.fmt == 0 ? by_type<WType::MX>(a, k, stream) : by_type<WType::NV>(a, k, stream);
}

}  // namespace fgf8
