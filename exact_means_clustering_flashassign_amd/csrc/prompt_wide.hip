// Attention of a step's prompts on the matrix cores: rows of 129 to 256 elements.
#include "prompt.hpp"

namespace fk {
namespace {

template <int DT> hipError_t run(const PromptArgs& a, void* ws, hipStream_t s) {
  return a.cache.dim <= 192 ? run_mfma<DT, 192>(a, ws, s) : run_mfma<DT, 256>(a, ws, s);
}

}  // namespace

hipError_t launch_prompt_wide(const PromptArgs& a, int dt, void* ws, hipStream_t s) {
  return dt == FK_F32 ? run<FK_F32>(a, ws, s) : dt == FK_F16 ? run<FK_F16>(a, ws, s) : run<FK_BF16>(a, ws, s);
}

}  // namespace fk
