// layers_linear_bf16.hip -- linear attention's kernels, bf16.
#include "layers_linear_instances.hpp"

template struct lic::Linear<lic::bf16>;
