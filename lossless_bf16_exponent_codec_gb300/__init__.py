"""libexpzip: lossless BF16 exponent codecs (ZipCCL 3-bit exponent code and
CIERA cross-iteration exponent reuse) as hand-written CUDA kernels for sm_103a
behind a C ABI (include/expzip.h).

``binding`` is the ctypes marshalling of that ABI, ``codec.Codec`` allocates
the caller-owned buffers of one plan with torch, ``build`` compiles the
library in-tree, ``breakeven`` is the host-side break-even model and ``bsc``
the benefit-driven choice of the shards to send with exponent reuse.  ``mx``
holds the microscaled (4- and 8-bit) forms of what was gathered, their products,
the gated unit with its 8-bit checkpoint and the norm in front of them, ``mlp`` a
gated MLP made of them, ``moe`` the sorting of tokens by expert, the experts'
products and a layer of gated experts.
"""
from . import binding, breakeven, bsc  # noqa: F401

__all__ = ["binding", "breakeven", "bsc", "codec", "build", "mx", "mlp", "moe"]
