// The gated delta rule token by token with fp16 q, k, v and out (see ssu_delta_rows.h).
#include "ssu_delta_rows.h"

namespace ssu {

hipError_t launch_delta_rows_f16(const DeltaParams &p, hipStream_t stream)
{
    return launch_delta_rows_io<_Float16>(p, stream);
}

}  // namespace ssu
