// Attention of a step's prompts on the matrix cores: f16 rows of up to 128 elements.
#include "prompt.hpp"

namespace fk {

template <> hipError_t launch_prompt_narrow<FK_F16>(const PromptArgs& a, void* ws, hipStream_t s) {
  return a.cache.dim <= 32   ? run_mfma<FK_F16, 32>(a, ws, s)
         : a.cache.dim <= 64 ? run_mfma<FK_F16, 64>(a, ws, s)
         : a.cache.dim <= 96 ? run_mfma<FK_F16, 96>(a, ws, s)
                             : run_mfma<FK_F16, 128>(a, ws, s);
}

}  // namespace fk
