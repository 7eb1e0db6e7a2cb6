"""MI355X-native GSPN 2D line-scan linear propagation.

`gspn` is the binding of libgspn (include/gspn.h): the C ABI's calls under
the same names, and `gspn4`, the four-direction propagation as a
differentiable op.  `sequence` binds its operators over token rows
(include/gspn_sequence.h): the short causal convolution, the selective scan
and the join of a block to the residual stream.  `attention` binds those of
layers that look at every token (include/gspn_attention.h): the norm and
rotation of heads, softmax attention with its caches.  `build` compiles libgspn.so
in-tree for gfx950; `workloads` draws the seeded synthetic inputs.
"""
