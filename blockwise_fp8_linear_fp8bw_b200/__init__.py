"""Blockwise-FP8 (E4M3) training linear layer for B200 (sm_100a), and the
operators around it.

The computation lives in the CUDA library libfp8bw.so (C ABI in
include/fp8bw.h and include/fp8bw_layer.h); `ops` is its thin Python binding.
Importing `ops` loads the library and raises if it is missing. On top of it:
`linear`, `mlp` (training layers), `muon` (optimiser), `data_parallel`.
"""
__all__ = ["ops", "build"]
