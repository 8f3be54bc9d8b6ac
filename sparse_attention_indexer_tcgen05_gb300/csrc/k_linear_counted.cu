// k_linear_counted.cu -- products whose rows, or whose k axis, the device counts: the gradients of a vocabulary's loss, of the rows
// that have a target.  The kernel is the projections' (k_linear_tc.cu) with its arguments corrected from the count by every CTA.
#include "k_linear_tc.cuh"

namespace csa {

cudaError_t linear_counted_read_clear_error(int *flag)
{
    *flag = 0;
    cudaError_t e = cudaMemcpyFromSymbol(flag, g_lin_error, sizeof(int));
    if (e == cudaSuccess && *flag != 0) {
        const int zero = 0;
        e = cudaMemcpyToSymbol(g_lin_error, &zero, sizeof(int));
    }
    return e;
}

namespace linear {

cudaError_t launch_product_counted(const Product &p, int sms, cudaStream_t st)
{
    // dz or its transpose with rows that lie along n; a k axis cut in pieces would leave some of them empty
    if (p.b.k_major || p.a.k_major == p.along_k || p.passes != 1 || (p.along_k && p.plan.splits != 1)) return cudaErrorInvalidValue;
    if (p.plan.shape != (p.planes == 3 ? PAIR_128 : PAIR_256)) return cudaErrorInvalidValue;
    Args a = {};
    Maps m = {};
    const cudaError_t e = describe(p, sms, a, m);
    if (e != cudaSuccess) return e;
    a.counted = p.counted;
    a.first = p.first;
    a.along_k = p.along_k;
    a.many = 0;
    if (p.planes == 3) {
        if (p.along_k) return launch<2, 128, 3, 8, true, false, false, false, true>(m, a, sms, st);
        return launch<2, 128, 3, 8, true, true, false, false, true>(m, a, sms, st);
    }
    if (p.along_k) return launch<2, 256, 1, 8, false, false, false, false, true>(m, a, sms, st);
    return launch<2, 256, 1, 8, false, true, false, false, true>(m, a, sms, st);
}

}  // namespace linear
}  // namespace csa
