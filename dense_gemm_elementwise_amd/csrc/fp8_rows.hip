// fp8_rows.hip -- launches of the 8-bit products of few rows.
#include "fp8_launch.hpp"
#include "fp8_rows.hpp"
#include "ops_host.hpp"

namespace gemm_epi {

template <bool BF, int FX, bool X8, int XL, int WAVES>
static hipError_t launch_rows3(const FewRows8 &p, hipStream_t s)
{
    return launch(fp8_few_rows_kernel<BF, FX, X8, XL, WAVES>, dim3((unsigned)ceil_div(p.N, 16)), dim3(64 * WAVES), s, p);
}
template <bool BF, int FX>
static hipError_t launch_rows2(const FewRows8 &p, hipStream_t s)
{
    // One row of 16 bits with 16 waves a workgroup and with 4, us: N x K = 256 x 4096
    // 3.6 and 4.4, 1024 x 8192 5.3 and 6.9, 2048 x 4096 4.3 and 4.8, 4096 x 4096
    // 6.0 and 6.1, 6144 x 4096 9.4 and 8.3.  In 8 bits 4 were as good or better (1024 x 8192
    // 5.2 and 5.2, 6144 x 4096 8.3 and 7.4): what the waves share is the work of quantising.
    if (!p.XS)
        return p.N < 16 * kCUs ? launch_rows3<BF, FX, false, 1, 16>(p, s) : launch_rows3<BF, FX, false, 1, 4>(p, s);
    return p.M <= 8 ? launch_rows3<BF, FX, true, 1, 4>(p, s) : launch_rows3<BF, FX, true, 2, 4>(p, s);
}
hipError_t fp8_launch_rows(bool bf, bool e5m2, const FewRows8 &p, hipStream_t s)
{
    if (e5m2) return bf ? launch_rows2<true, 1>(p, s) : launch_rows2<false, 1>(p, s);
    return bf ? launch_rows2<true, 0>(p, s) : launch_rows2<false, 0>(p, s);
}

}  // namespace gemm_epi
