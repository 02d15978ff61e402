// xs_span_d96.cu -- the span attention kernel's instances for head dimension 96
// (whole sequences and paged cache). The kernel is in xs_span_kernel.cuh.
#include "xs_span_kernel.cuh"

namespace xs {

XS_DEFINE_SPAN_ENTRY(96)

}  // namespace xs
