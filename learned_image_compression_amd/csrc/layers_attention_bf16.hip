// layers_attention_bf16.hip -- attention's kernels for this element type.
#include "layers_attention_instances.hpp"

template struct lic::Attention<lic::bf16>;
