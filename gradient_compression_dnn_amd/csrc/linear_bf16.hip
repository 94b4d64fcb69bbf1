// The layer products of bf16 activations.
#include "linear_kernels.hpp"

namespace gc {

template gc_status linear_launch<BF16>(const char *, Kind, const Product &, const Cut &, hipStream_t);

}  // namespace gc
