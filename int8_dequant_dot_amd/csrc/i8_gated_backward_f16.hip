// i8_gated_backward_f16.hip -- the gated projection's gradients for float16 (one file a type: they compile side by
// side).
#include "i8_gated_backward.hpp"

namespace loom {

hipError_t launch_i8_gated_backward_f16(const loom_launch_config &cfg, const I8Product &p, const void *d_out,
                                         int64_t d_stride, void *d_x, float *d_gate, float *d_up, void *workspace,
                                         hipStream_t stream) {
    return run_backward<i8_limbs(LOOM_F16)>(cfg, p, d_out, LOOM_F16, d_stride, d_x, d_gate, d_up,
                                                  workspace, stream);
}

}  // namespace loom
