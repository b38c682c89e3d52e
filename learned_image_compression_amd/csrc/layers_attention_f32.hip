// layers_attention_f32.hip -- attention's kernels for this element type.
#include "layers_attention_instances.hpp"

template struct lic::Attention<float>;
