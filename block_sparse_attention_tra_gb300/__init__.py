"""GB300-native fused causal attention forwards.

Two forwards that never materialise the T x T score matrix, each one CUDA
kernel for sm_103a behind a C ABI (``include/bsa.h``, ``libbsa.so``):

* ``tra_forward``        -- threshold rectified attention,
  ``out = ReLU(Q K^T - tau(i))^p V`` with ``tau(i) = beta sqrt(2 ln(i+1)/D)``,
  causal and unnormalised (page "triton_threshold_attention.py").
* ``nsa_select_forward`` -- NSA selection-branch attention over gathered key
  blocks, GQA, causal, scaled softmax (page "nsa_selection_kernel.py").
* ``nsa_select_forward_fsa`` -- the same result in the page's block-outer
  split-K form: each selected block's K/V read once, per-pair softmax
  partials, a log-sum-exp combine.
* ``nsa_select_backward`` and ``nsa_select_attention`` -- the gradients of
  ``nsa_select_forward``, and the forward as a ``torch.autograd.Function``
  whose backward runs them.
* ``nsa_cache_append`` and ``nsa_select_decode`` -- the selection attention in
  serving: new tokens' keys (rotated by position) and values into a paged
  cache of e4m3 codes with a scale for each page and head, and one query token
  per sequence over that cache, its selected blocks or all of them.
* ``qk_norm_rope`` -- what stands before the attention: the RMS norm of every
  query and key head and its rotation by position, in one pass, with its
  gradients (``qk_norm_rope_forward``, ``qk_norm_rope_backward``;
  ``rope_frequencies`` makes the frequencies).
* ``nsa_cache4_append``, ``nsa_cache4_read`` and ``nsa_cache4_decode`` -- a
  paged cache of 4-bit codes with a scale for every 16 elements: filled (keys
  normalised and rotated on the way), read back, attended to.
* ``tra_forward_host`` -- ``tra_forward`` on host tensors, streamed through
  the GPU in chunks of heads with overlapped copies.
* ``tra_backward`` and ``tra_attention`` -- the gradients of ``tra_forward``,
  and the forward as a ``torch.autograd.Function`` whose backward runs them
  (the page's ThresholdRelaFunction); ``tra_diff_forward``,
  ``tra_diff_backward`` and ``tra_diff_attention`` -- the page's differential
  form, its gradients and the two as an autograd function.

The binding in ``bsa`` only marshals arguments; every step runs in the CUDA
library, which is loaded on first use and must be built (``build.build()``).
"""

from .bsa import (  # noqa: F401
    BsaError,
    device_error,
    library_path,
    load_library,
    nsa_cache4_append,
    nsa_cache4_append_raw,
    nsa_cache4_decode,
    nsa_cache4_decode_raw,
    nsa_cache4_decode_workspace_size,
    nsa_cache4_read,
    nsa_cache4_read_raw,
    nsa_cache_append,
    nsa_cache_append_raw,
    nsa_select_attention,
    nsa_select_backward,
    nsa_select_backward_raw,
    nsa_select_backward_workspace_size,
    nsa_select_decode,
    nsa_select_decode_raw,
    nsa_select_decode_workspace_size,
    nsa_select_forward,
    nsa_select_forward_fsa,
    nsa_select_forward_fsa_raw,
    nsa_select_forward_raw,
    nsa_select_fsa_workspace_size,
    qk_norm_rope,
    qk_norm_rope_backward,
    qk_norm_rope_backward_raw,
    qk_norm_rope_backward_workspace_size,
    qk_norm_rope_forward,
    qk_norm_rope_forward_raw,
    rope_frequencies,
    status_string,
    tra_attention,
    tra_backward,
    tra_backward_raw,
    tra_diff_attention,
    tra_diff_backward,
    tra_diff_backward_raw,
    tra_diff_forward,
    tra_diff_forward_raw,
    tra_forward,
    tra_forward_ex_raw,
    tra_forward_host,
    tra_forward_host_raw,
    tra_forward_host_workspace_size,
    tra_forward_raw,
)

__all__ = [
    "BsaError",
    "device_error",
    "library_path",
    "load_library",
    "tra_forward",
    "tra_forward_raw",
    "tra_forward_ex_raw",
    "tra_forward_host",
    "tra_forward_host_raw",
    "tra_forward_host_workspace_size",
    "tra_attention",
    "tra_backward",
    "tra_backward_raw",
    "tra_diff_attention",
    "tra_diff_backward",
    "tra_diff_backward_raw",
    "tra_diff_forward",
    "tra_diff_forward_raw",
    "nsa_select_forward",
    "nsa_select_forward_raw",
    "nsa_select_forward_fsa",
    "nsa_select_forward_fsa_raw",
    "nsa_select_fsa_workspace_size",
    "nsa_select_attention",
    "nsa_select_backward",
    "nsa_select_backward_raw",
    "nsa_select_backward_workspace_size",
    "nsa_cache_append",
    "nsa_cache_append_raw",
    "nsa_select_decode",
    "nsa_select_decode_raw",
    "nsa_select_decode_workspace_size",
    "nsa_cache4_append",
    "nsa_cache4_append_raw",
    "nsa_cache4_decode",
    "nsa_cache4_decode_raw",
    "nsa_cache4_decode_workspace_size",
    "nsa_cache4_read",
    "nsa_cache4_read_raw",
    "qk_norm_rope",
    "qk_norm_rope_backward",
    "qk_norm_rope_backward_raw",
    "qk_norm_rope_backward_workspace_size",
    "qk_norm_rope_forward",
    "qk_norm_rope_forward_raw",
    "rope_frequencies",
    "status_string",
]
