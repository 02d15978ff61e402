// xs_span_serve_d96.cu -- the span attention kernel's instances for head dimension 96
// over packed prompts and for drafted trees. The kernel is in xs_span_kernel.cuh.
#include "xs_span_kernel.cuh"

namespace xs {

XS_DEFINE_SPAN_SERVE_ENTRY(96)

}  // namespace xs
