// fa_paged_bf16_e4m3.cu -- paged attention of bf16 queries over e4m3 pages.
#include "fa_paged_launch.cuh"

namespace fa {

fa_status paged_bf16_e4m3(DeviceInfo& di, const PagedCall& c) { return paged_call<Elem::kBf16, true>(di, c); }

}  // namespace fa
