// The gated delta rule in chunks with fp16 q, k, v and out (see ssu_delta_chunks.h).
#include "ssu_delta_chunks.h"

namespace ssu {

hipError_t launch_delta_chunks_f16(const DeltaParams &p, const DeltaPlan &plan, hipStream_t stream)
{
    return launch_delta_chunks_io<_Float16>(p, plan, stream);
}

}  // namespace ssu
