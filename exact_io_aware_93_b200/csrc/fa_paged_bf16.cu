// fa_paged_bf16.cu -- paged attention of bf16 queries over bf16 pages.
#include "fa_paged_launch.cuh"

namespace fa {

fa_status paged_bf16(DeviceInfo& di, const PagedCall& c) { return paged_call<Elem::kBf16, false>(di, c); }

}  // namespace fa
