// The gated delta rule on given q, k and v over a paged state pool.
#include "ssu_delta_impl.h"

namespace ssu {

hipError_t launch_delta_rows_f32(const DeltaParams &p, hipStream_t stream);
hipError_t launch_delta_rows_f16(const DeltaParams &p, hipStream_t stream);
hipError_t launch_delta_rows_bf16(const DeltaParams &p, hipStream_t stream);

int64_t delta_workspace_bytes(int64_t, int64_t, int64_t, int64_t, int64_t, int32_t) { return 0; }

hipError_t launch_delta(const DeltaParams &p, hipStream_t stream)
{
    (void)hipGetLastError();  // report only this launch's status
    switch (p.io_dtype) {
    case kF32: return launch_delta_rows_f32(p, stream);
    case kF16: return launch_delta_rows_f16(p, stream);
    default: return launch_delta_rows_bf16(p, stream);
    }
}

}  // namespace ssu
