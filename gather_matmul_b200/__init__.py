"""B200 (sm_100a) multi-LoRA shrink / expand: BGMV (per-token adapters, for
decode) and SGMV (segment-grouped, for prefill) behind the C ABI of
include/lora.h (liblora_b200.so), with a thin torch binding in ops.py; and the
8-bit base product, rotation and head norms of the projection that carries the
adapters, and the paged 8-bit key/value cache and attention behind it (ops.py,
layers.py).

Importing the package does not load the CUDA library; the first call in
ops.py does, and raises if it has not been built.
"""
__all__ = ["ops", "layers", "workloads", "build"]
