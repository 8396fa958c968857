// gqa_decode_tail.cu -- instantiates the split-KV kernels for what lies behind a
// shared prefix (kernels in gqa_decode_kernels.cuh).
#include "gqa_decode_kernels.cuh"

namespace gqa {
namespace dec {

bool pick_tail(int dtype, int kind, int d, int nw, Variant& v) {
    return pick_variant<true, false, true>(dtype, kind, d, nw, v);
}

}  // namespace dec
}  // namespace gqa
