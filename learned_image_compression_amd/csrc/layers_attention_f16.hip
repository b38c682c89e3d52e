// layers_attention_f16.hip -- attention's kernels for this element type.
#include "layers_attention_instances.hpp"

template struct lic::Attention<lic::f16>;
