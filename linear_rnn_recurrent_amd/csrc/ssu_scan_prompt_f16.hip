// Scan of prompts with fp16 x, z and out (see ssu_scan_prompt.h).
#include "ssu_scan_prompt.h"

namespace ssu {

hipError_t launch_scan_prompt_f16(const ScanParams &p, const ScanPlan &q, hipStream_t stream)
{
    return launch_prompt_dt<_Float16>(p, q, stream);
}

}  // namespace ssu
