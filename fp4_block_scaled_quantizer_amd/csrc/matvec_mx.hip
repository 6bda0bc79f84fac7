// matvec_mx.hip -- products of few rows with MXFP4 weights (matvec.h).
#include "matvec.h"

namespace fp4q {

int launch_matvec_mx(const MatvecArgs &g, hipStream_t st)
{
    const int units = device_cu_count();
    if (units <= 0) return 1;
    const Matvec a = matvec_of(g);
    if (g.x_scales)
        pick_matvec<kMx, true>(a, !g.tiled, (uint32_t)units, st);
    else
        pick_matvec<kMx, false>(a, !g.tiled, (uint32_t)units, st);
    return hipGetLastError() == hipSuccess ? 0 : 1;
}

}  // namespace fp4q
