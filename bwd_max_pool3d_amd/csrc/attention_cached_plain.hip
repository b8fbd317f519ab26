// attention_cached_plain.hip -- attention over plain caches.
#include "attention_cached.hpp"

namespace mp3d {

template <>
hipError_t launch_cached<F32, kPlain>(const CachedArgs &c, hipStream_t s)
{
    return run_cached_width<F32, kPlain>(c, s);
}
template <>
hipError_t launch_cached<F16, kPlain>(const CachedArgs &c, hipStream_t s)
{
    return run_cached_width<F16, kPlain>(c, s);
}
template <>
hipError_t launch_cached<BF16, kPlain>(const CachedArgs &c, hipStream_t s)
{
    return run_cached_width<BF16, kPlain>(c, s);
}

}  // namespace mp3d
