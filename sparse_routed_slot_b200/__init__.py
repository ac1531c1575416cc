"""librsm: a B200 (sm_100a) implementation of Raven's routing-state-model (RSM) mixer.

The product is the C ABI in include/rsm.h (librsm.so, built in-tree from csrc/). This package adds
a thin ctypes binding with the same calls:

    route(logits, K)                          -> TopK slot indices and sigmoid scores
    forward(q, k, v, logits, f, K, H0=None)   -> chunked prefill: o and the final state H_T
    decode_step(q, k, v, logits, f, K, state) -> one generation token, state updated in place
    backward(q, k, v, logits, f, K, dO, dHT)  -> gradients of the prefill (RSMFunction: autograd)

and the other operators of a hybrid stack, whose attention layers alternate with mixer layers:

    window_forward(q, k, v, window, sinks)    -> sliding-window attention with visible first tokens
    window_backward(...)                      -> its gradients (WindowFunction: autograd)
    paged_append(k, v, caches, ...)           -> new tokens' keys and values into a paged cache
    paged_forward(q, caches, ...)             -> their attention over it (chunks and single tokens)
    block_norm_forward(y, gate, residual, ..) -> norms around a block with its gate and residual
    block_norm_backward(...)                  -> their gradients (BlockNormFunction: autograd)
"""
from .api import RSMFunction, backward, decode_step, device_status, forward, route  # noqa: F401
from .hybrid import (BlockNormFunction, WindowFunction, block_norm_backward, block_norm_forward,  # noqa: F401
                     paged_append, paged_forward, window_backward, window_forward)
from ._lib import RSMError  # noqa: F401

__all__ = ["route", "forward", "backward", "decode_step", "device_status", "RSMFunction", "RSMError",
           "window_forward", "window_backward", "WindowFunction", "paged_append", "paged_forward",
           "block_norm_forward", "block_norm_backward", "BlockNormFunction"]
