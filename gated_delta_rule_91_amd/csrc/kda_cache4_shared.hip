// kda_cache4_shared.hip -- attention over shared prefixes (kda_cache4_shared.hpp)
// in bf16, and what the host asks of either type.
#include "kda_cache4_shared.hpp"

namespace kda {

bool cache4_shared_fits(bool bf16, int d, const Cache4SharedArgs& s) {
    const Plan prefix = plan_of(bf16, d, prefix_args(s), PREFIX), own = plan_of(bf16, d, s.a, OWN);
    return (workgroups(prefix) + workgroups(own)) * s.a.c.heads <= UINT32_MAX / (kWaves * 64) && part_places(s.a, prefix) <= INT32_MAX &&
           part_places(s.a, own) <= INT32_MAX;
}

size_t cache4_shared_workspace_bytes(bool bf16, int d, const Cache4SharedArgs& s) { return lay_out(bf16, d, s, nullptr).bytes; }

hipError_t launch_cache4_shared(bool bf16, int d, const Cache4SharedArgs& s, char* ws, hipStream_t stream) {
    if (!bf16) return launch_cache4_shared_f32(d, s, ws, stream);
    return d == 128 ? launch_shared<__bf16, 128>(s, ws, stream) : launch_shared<__bf16, 64>(s, ws, stream);
}

}  // namespace kda
