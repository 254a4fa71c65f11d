// Products with 4-bit codes in bfloat16.
#include "lscd_quant_product.h"

namespace lscd {
hipError_t launch_quant_bf16(const QuantArgs& a, int kind, const QuantPlan& p, hipStream_t s) {
    return run_product<BF16>(a, kind, p, s);
}
}  // namespace lscd
