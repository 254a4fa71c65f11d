// Products with 4-bit codes in float16.
#include "lscd_quant_product.h"

namespace lscd {
hipError_t launch_quant_f16(const QuantArgs& a, int kind, const QuantPlan& p, hipStream_t s) {
    return run_product<F16>(a, kind, p, s);
}
}  // namespace lscd
