// Stub launchers of the step's entry points for the host-only sanitizer
// build of qmat_step_api.cpp: each records that it was reached and succeeds.
#include <hip/hip_runtime.h>

#include "lora_plan.hpp"
#include "qmat_launch.hpp"

extern int g_launches;

namespace qmat {
hipError_t launch_embed(int, int, const void*, const int32_t*, void*, int64_t, int64_t, int64_t,
                        int64_t, hipStream_t) {
  ++g_launches;
  return hipSuccess;
}
hipError_t launch_norm(const qmat_norm_args&, hipStream_t) {
  ++g_launches;
  return hipSuccess;
}
hipError_t launch_rope(const qmat_rope_args&, hipStream_t) {
  ++g_launches;
  return hipSuccess;
}
int64_t page_workspace_bytes(const qmat_page_args& a) { return a.max_tokens > 1000 ? 4096 : 0; }
hipError_t launch_page_step(const qmat_page_args&, void*, hipStream_t) {
  ++g_launches;
  return hipSuccess;
}
int64_t lora_workspace_bytes(const qmat_lora_args& a) { return lora_plan(a).bytes(a); }
hipError_t launch_lora(const qmat_lora_args&, void*, hipStream_t) {
  ++g_launches;
  return hipSuccess;
}
}  // namespace qmat
