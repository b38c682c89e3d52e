"""MI355X (gfx950) indexed rANS64 entropy coder for learned image compression.

The coder is the hand-written HIP library ``librans_hip.so`` behind the C ABI
declared in ``include/rans_hip.h``; ``learned_image_compression_amd.binding``
marshals torch tensors into it.  The network operators that stand before it (group and RMS
norms, rotary positions, attention, linear attention, clipping) are ``learned_image_compression_amd.layers``
(``liblic_layers.so``, ``include/lic_layers.h``).  Importing this package does not load the
libraries; the first call does, and fails loudly if they were not built.
"""
