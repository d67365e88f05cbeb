// The gated delta rule token by token with fp32 q, k, v and out (see ssu_delta_rows.h).
#include "ssu_delta_rows.h"

namespace ssu {

hipError_t launch_delta_rows_f32(const DeltaParams &p, hipStream_t stream)
{
    return launch_delta_rows_io<float>(p, stream);
}

}  // namespace ssu
