// attention_cached_e4m3.hip -- attention over caches: the kernels of one format.
#include "attention_cached.hpp"

namespace mp3d {

template <typename T>
hipError_t launch_cached_e4m3(const CachedArgs &c, hipStream_t s)
{
    return run_cached_width<T, kE4M3>(c, s);
}

template hipError_t launch_cached_e4m3<F32>(const CachedArgs &, hipStream_t);
template hipError_t launch_cached_e4m3<F16>(const CachedArgs &, hipStream_t);
template hipError_t launch_cached_e4m3<BF16>(const CachedArgs &, hipStream_t);

}  // namespace mp3d
