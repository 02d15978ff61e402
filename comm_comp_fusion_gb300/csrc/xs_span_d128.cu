// xs_span_d128.cu -- the span attention kernel's instances for head dimension 128
// (whole sequences and paged cache). The kernel is in xs_span_kernel.cuh.
#include "xs_span_kernel.cuh"

namespace xs {

XS_DEFINE_SPAN_ENTRY(128)

}  // namespace xs
