// Scan of prompts with fp32 x, z and out (see ssu_scan_prompt.h).
#include "ssu_scan_prompt.h"

namespace ssu {

hipError_t launch_scan_prompt_f32(const ScanParams &p, const ScanPlan &q, hipStream_t stream)
{
    return launch_prompt_dt<float>(p, q, stream);
}

}  // namespace ssu
