// attention_cached_plain.hip -- attention over caches: the kernels of one format.
#include "attention_cached.hpp"

namespace mp3d {

template <typename T>
hipError_t launch_cached_plain(const CachedArgs &c, hipStream_t s)
{
    return run_cached_width<T, kPlain>(c, s);
}

template hipError_t launch_cached_plain<F32>(const CachedArgs &, hipStream_t);
template hipError_t launch_cached_plain<F16>(const CachedArgs &, hipStream_t);
template hipError_t launch_cached_plain<BF16>(const CachedArgs &, hipStream_t);

}  // namespace mp3d
