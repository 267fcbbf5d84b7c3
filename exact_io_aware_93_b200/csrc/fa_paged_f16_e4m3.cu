// fa_paged_f16_e4m3.cu -- paged attention of fp16 queries over e4m3 pages.
#include "fa_paged_launch.cuh"

namespace fa {

fa_status paged_f16_e4m3(DeviceInfo& di, const PagedCall& c) { return paged_call<Elem::kF16, true>(di, c); }

}  // namespace fa
