// gqa_decode_sinks.cu -- instantiates the split-KV kernels for a sliding window
// whose first tokens stay visible (kernels in gqa_decode_kernels.cuh).
#include "gqa_decode_kernels.cuh"

namespace gqa {
namespace dec {

bool pick_sinks(int dtype, int kind, int d, int nw, Variant& v) {
    return pick_variant<true, true>(dtype, kind, d, nw, v);
}

}  // namespace dec
}  // namespace gqa
