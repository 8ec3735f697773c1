// The gated linear recurrence's kernels for bf16 activations.
#include "ssd_glr.hpp"

namespace ssd {
SSD_GLR_INSTANTIATE(bf16)
}  // namespace ssd
