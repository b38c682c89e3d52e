// layers_linear_f16.hip -- linear attention's kernels, f16.
#include "layers_linear_instances.hpp"

template struct lic::Linear<lic::f16>;
