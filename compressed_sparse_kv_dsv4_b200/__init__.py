"""B200 (sm_100a) library for the DeepSeek-V4 hybrid-attention decode step.

The compute lives in libdsv4.so (CUDA kernels behind the C ABI of include/dsv4.h);
this package is its thin Python binding over torch CUDA tensors.
"""

from .binding import (DeviceCache, DeviceKv4Cache, DeviceLayer, DeviceRing, DeviceState, DeviceStep,  # noqa: F401
                      compress, compress_project,
                      hybrid_decode, indexer_args, indexer_scores, indexer_topk, indexer_topk_noalloc,
                      kv4_append, kv4_attention, kv4_attention_args, kv4_attention_plan, kv4_attention_workspace,
                      kv4_attention_workspace_size, layer_state_bytes, mqa_args,
                      mqa_workspace_size, qk_norm_rope, sparse_mqa_decode, swa_insert,
                      to_device_codes, to_numpy_codes)
from ._abi import Dsv4Error, load  # noqa: F401
