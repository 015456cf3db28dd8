"""Symmetric-window collectives on one GB300: AllReduce(sum), AllGather and
chunked put+signal over R rank windows carved from one GPU's HBM; and the training
step's operators around that AllReduce (linear layer, policy loss, AdamW).

The compute path is libsymar.so (hand-written CUDA for sm_103a behind the C ABI
in include/symar.h); this package is its thin ctypes binding.
"""
from ._binding import (  # noqa: F401
    ALGOS, DTYPES, NO_ID, OPS, SYM_ERR_INVALID_ARG, SYM_ERR_TIMEOUT, SYM_ERR_UNSUPPORTED, SYM_OK,
    SymError, Window, header_symbols, load, sym_abi_version, sym_allgather,
    sym_allgather_put_signal, sym_allreduce, sym_alltoall, sym_barrier, sym_scale_allreduce, sym_allreduce_algo, sym_counter_read,
    sym_counter_reset, sym_counter_wait, sym_get, sym_last_error, sym_launch_count, sym_put_signal,
    sym_allreduce_noalloc, sym_signal, sym_signal_read, sym_signal_reset, sym_signal_wait,
    sym_status_string,
    sym_stream_status,
    ACTS, SYM_ACT_GELU, SYM_ACT_NONE, SYM_ACT_RELU, SYM_ACT_SILU,
    SYM_WINDOW_CUDA_MALLOC, SYM_WINDOW_REGISTERED, SYM_WINDOW_VMM, SYM_WINDOW_VMM_EXPORTABLE,
)
from ._binding import LIB_PATH  # noqa: F401

# the training operators need torch; they are imported when first asked for
_TRAINING = ("AdamW", "sym_adamw_step", "sym_grad_norm", "sym_linear", "sym_linear_backward",
             "sym_policy_loss", "sym_policy_loss_backward")


def __getattr__(name):
    if name in _TRAINING:
        from . import _training

        for n in _TRAINING:
            globals()[n] = getattr(_training, n)
        return globals()[name]
    raise AttributeError(f"module {__name__!r} has no attribute {name!r}")


def __dir__():
    return sorted(set(globals()) | set(_TRAINING))
