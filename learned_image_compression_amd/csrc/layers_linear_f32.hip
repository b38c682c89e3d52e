// layers_linear_f32.hip -- linear attention's kernels, f32.
#include "layers_linear_instances.hpp"

template struct lic::Linear<float>;
