#include "attention_span.cuh"

namespace spec {
namespace span {
bool tc_takes(const spec_attn_params*) { return false; }
int tc_row_tile(const spec_attn_params*) { return 128; }
spec_status_t launch_span_tc(const spec_attn_params*, Dev, cudaStream_t) { return SPEC_ERR_UNSUPPORTED; }
}  // namespace span
}  // namespace spec
