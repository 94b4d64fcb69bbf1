// The layer products of fp32 activations.
#include "linear_kernels.hpp"

namespace gc {

template gc_status linear_launch<F32>(const char *, Kind, const Product &, const Cut &, hipStream_t);

}  // namespace gc
