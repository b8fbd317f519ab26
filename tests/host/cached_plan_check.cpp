// Host-side check of how attention over caches cuts its work: over long
// caches in use whole, a call has as many workgroups as run at once, which is
// what the kernels that it takes are declared for.  Linked with the library;
// launches nothing.
#include <cstdio>

#include "../../bwd_max_pool3d_amd/csrc/tokens.hpp"

using namespace mp3d;

int main()
{
    constexpr int kCus = 256, kStep = 128;
    int fails = 0, seen = 0;
    for (int format : {0, 1, 2})           // plain, e4m3, e2m1
        for (int f32 : {0, 1})
            for (int any : {0, 1})
                for (float cap : {0.f, 30.f})
                    for (int D : {32, 64, 65, 80, 96, 100, 128})
                        for (int rows : {1, 4, 16, 200}) {
                            CachedArgs c = {};
                            AttnArgs &a = c.a;
                            a.B = 1;
                            a.Tq = 1;
                            a.Hk = 1;
                            a.Hq = a.G = rows;
                            a.D = D;
                            a.scale = 1.f;
                            a.cap = cap;
                            c.format = format;
                            c.f32 = f32;
                            c.any = any;
                            c.part[0].seqs = c.part[1].seqs = 1;
                            c.part[1].caches = 1;
                            c.part[1].T = 1 << 24;
                            plan_attn_cached(&c, kCus);
                            // three: 16 rows over codes of 16-byte rows, without a cap, whose
                            // tiles leave room; one for plain float32 over 64 channels, but two
                            // are planned (measured beside the rule)
                            const bool three = format != 0 && c.part[1].mb == 16 && !any && cap == 0.f &&
                                               !(f32 && D > 64);
                            const long at_once = kCus * (three ? 3L : 2L), units = c.part[1].units;
                            // (blocks of 16 rows share the workgroups; a chunk is whole steps)
                            const long all = units * c.part[1].nrb;
                            ++seen;
                            if (all > at_once + c.part[1].nrb || all < at_once - at_once / 8) {
                                if (fails++ < 20)
                                    std::printf("FAIL format %d f32 %d any %d cap %g D %d rows %d: %ld "
                                                "workgroups, %ld at once\n", format, f32, any, cap, D,
                                                rows, all, at_once);
                            }
                            if ((long)c.part[1].chunk * c.part[1].nsplit < c.part[1].T || c.part[1].chunk % kStep)
                                ++fails;
                        }
    if (fails) return 1;
    std::printf("cached plans: ok (%d)\n", seen);
    return 0;
}
