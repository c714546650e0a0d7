// Device-side entry points of the library for the host-only sanitizer
// build (build.build_host_sanitized): the packer, the layout arithmetic and
// the C ABI's validation are compiled with AddressSanitizer and
// UndefinedBehaviorSanitizer, and every enqueue is replaced by a refusal, so
// the host tests exercise all host code paths without a GPU or GPU code.
#include <hip/hip_runtime.h>

#include "block_launch.h"
#include "moe_host.h"
#include "moe_launch.h"

namespace moe {

hipError_t launch_route(int, int, const RouteArgs&, hipStream_t, hipEvent_t*) { return hipErrorNoDevice; }
hipError_t launch_decode(int, int, const DecodeArgs&, hipStream_t, hipEvent_t*) { return hipErrorNoDevice; }
hipError_t launch_grouped(int, int, const GroupedArgs&, hipStream_t, hipEvent_t*) { return hipErrorNoDevice; }
hipError_t launch_grp_sort(const GroupedArgs&, hipStream_t, hipEvent_t*) { return hipErrorNoDevice; }
hipError_t launch_route_exact(int, int, const RouteArgs&, hipStream_t, hipEvent_t*) { return hipErrorNoDevice; }
hipError_t launch_exact_experts(int, int, const DecodeArgs&, hipStream_t, hipEvent_t*) { return hipErrorNoDevice; }

hipError_t launch_dense(int, int, int, int, const DenseArgs&, hipStream_t) { return hipErrorNoDevice; }
bool dense_decode_quantises(int, int, int, int) { return true; }
hipError_t launch_dense_decode(int, int, int, const DenseDecodeArgs&, hipStream_t) { return hipErrorNoDevice; }
hipError_t launch_dense_pad(int, const DensePad&, hipStream_t) { return hipErrorNoDevice; }
hipError_t launch_quant_rows(int, const void*, int64_t, int, int, int8_t*, int64_t, float*, const DensePad*,
                             hipStream_t) {
  return hipErrorNoDevice;
}
hipError_t launch_glu_grad(int, bool, int, const void*, int64_t, const float*, int, int, int, void*, const DensePad&,
                           const DensePairs&, float*, hipStream_t) {
  return hipErrorNoDevice;
}

hipError_t launch_norm(int, const NormArgs&, hipStream_t) { return hipErrorNoDevice; }
int64_t norm_grad_words(int rows, int hidden) { return (rows < 512 ? rows : 512) * (int64_t)hidden; }
hipError_t launch_norm_grad(int, const NormGradArgs&, hipStream_t) { return hipErrorNoDevice; }
int64_t balance_part_words(int rows, int experts) { return (rows < 256 ? rows : 256) * (2 * (int64_t)experts + 4); }
hipError_t launch_balance(int, const BalanceArgs&, hipStream_t) { return hipErrorNoDevice; }
hipError_t launch_balance_grad(int, const BalanceArgs&, hipStream_t) { return hipErrorNoDevice; }
bool lora_by_row(int rows, int, int, int) { return rows <= 16; }
hipError_t launch_lora_sort(const LoraSort&, hipStream_t) { return hipErrorNoDevice; }
int lora_splits(int, int k, int) { return k > 256 ? 2 : 1; }
hipError_t launch_lora_shrink(int, bool, const LoraShrink&, hipStream_t) { return hipErrorNoDevice; }
int lora_chunk(int, int) { return 64; }
hipError_t launch_lora_expand(int, bool, const LoraExpand&, hipStream_t) { return hipErrorNoDevice; }
hipError_t launch_lora_grad(int, const LoraGrad&, hipStream_t) { return hipErrorNoDevice; }
hipError_t launch_lora_row(int, const LoraRow&, hipStream_t) { return hipErrorNoDevice; }

}  // namespace moe

extern "C" int moe_forward_windows_noalloc(const moe_layer*, const void*, int, const float*, int32_t*, float*,
                                           float*, float*, void*) {
  moe::set_error("moe_forward_windows_noalloc: not in the host-only sanitizer build");
  return MOE_EHIP;
}
