// kda_cache4_shared_f32.hip -- attention over shared prefixes
// (kda_cache4_shared.hpp) in fp32.
#include "kda_cache4_shared.hpp"

namespace kda {

hipError_t launch_cache4_shared_f32(int d, const Cache4SharedArgs& s, char* ws, hipStream_t stream) {
    return d == 128 ? launch_shared<float, 128>(s, ws, stream) : launch_shared<float, 64>(s, ws, stream);
}

}  // namespace kda
