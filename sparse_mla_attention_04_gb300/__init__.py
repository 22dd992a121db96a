"""GB300-native (sm_103a) sparse MLA attention forward, and the operators of a
serving step around it: block tables, rotary positions, a block-scaled 8-bit
cache and attention over it, and those of steps that draft and branch: norms
with the rotation, tree masks and tree attention, kept tokens, forked block
tables and block copies.

The compute path is the CUDA library ``libsparse_mla.so`` (built from
``csrc/``) behind a C ABI declared in ``include/sparse_mla.h``. This package
holds its thin ctypes binding (``binding``) and the seeded synthetic input
recipes (``inputs``). Importing the package loads nothing; the binding loads
the library on first use and raises if it is missing.
"""
