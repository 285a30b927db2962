// The failures that kernels recorded on a device, gathered over the translation units
// (include/moe_failures.h).
#include "../../include/moe_failures.h"
#include "../../include/moe.h"
#include "common.cuh"

namespace moe {

namespace {
constexpr int kMaxWords = 32;                        // translation units of the library
const void* g_symbols[kMaxWords];                    // (zero before any constructor runs)
int g_words;
}  // namespace

FailureWord::FailureWord(const void* symbol) {
  if (g_words < kMaxWords) g_symbols[g_words++] = symbol;
}

}  // namespace moe

using namespace moe;

extern "C" int moe_device_failure(int32_t clear, int32_t out[3], void* stream) {
  if (!out) return MOE_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  void* word[kMaxWords];
  int32_t got[kMaxWords][4];
  for (int i = 0; i < g_words; ++i)
    if (cudaGetSymbolAddress(&word[i], g_symbols[i]) != cudaSuccess ||
        cudaMemcpyAsync(got[i], word[i], sizeof(got[i]), cudaMemcpyDeviceToHost, s) != cudaSuccess)
      return MOE_ERR_CUDA;
  if (cudaStreamSynchronize(s) != cudaSuccess) return MOE_ERR_CUDA;
  out[0] = out[1] = out[2] = 0;
  for (int i = 0; i < g_words; ++i) {
    if (got[i][0] == 0) continue;
    if (out[0] == 0)
      for (int j = 0; j < 3; ++j) out[j] = got[i][j];
    if (clear && cudaMemsetAsync(word[i], 0, sizeof(got[i]), s) != cudaSuccess) return MOE_ERR_CUDA;
  }
  return MOE_OK;
}
