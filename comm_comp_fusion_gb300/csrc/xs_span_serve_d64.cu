// xs_span_serve_d64.cu -- the span attention kernel's instances for head dimension 64
// over packed prompts and for drafted trees. The kernel is in xs_span_kernel.cuh.
#include "xs_span_kernel.cuh"

namespace xs {

XS_DEFINE_SPAN_SERVE_ENTRY(64)

}  // namespace xs
