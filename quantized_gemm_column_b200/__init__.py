"""Averis mean-residual split NVFP4 linear layer on B200 (sm_100a).

The compute lives in ``libaveris.so`` (hand-written CUDA for sm_100a behind
a C ABI, declared in ``include/averis.h``); ``api`` is a thin ctypes binding
with the same entry-point names: the split and vanilla NVFP4 linears, the
8-bit linear layer with blocks of 128, and the routing of a mixture of
experts (router, sort, dispatch, combine).  The library is loaded on first use and a
missing or unloadable library raises: there is no CPU fallback.
"""
