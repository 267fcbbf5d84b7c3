// fa_paged_f16.cu -- paged attention of fp16 queries over fp16 pages.
#include "fa_paged_launch.cuh"

namespace fa {

fa_status paged_f16(DeviceInfo& di, const PagedCall& c) { return paged_call<Elem::kF16, false>(di, c); }

}  // namespace fa
