// The gated delta rule in chunks with fp32 q, k, v and out (see ssu_delta_chunks.h).
#include "ssu_delta_chunks.h"

namespace ssu {

hipError_t launch_delta_chunks_f32(const DeltaParams &p, const DeltaPlan &plan, hipStream_t stream)
{
    return launch_delta_chunks_io<float>(p, plan, stream);
}

}  // namespace ssu
