// norm_grad_pack8.hip -- the gradient of the norms (norm_grad.h) with the
// normed rows read from 8-bit rows: the values that fp4_unpack8 gives, through
// the same binary32 steps, so that the results are those of the rows unpacked.
#include "norm_grad.h"

namespace fp4q {

int norm_grad_rows_pack8(const NormGradArgs &a, float *dgamma, float *dbeta, hipStream_t st)
{
    return norm_grad_rows<true>(a, dgamma, dbeta, st);
}

}  // namespace fp4q
