"""GB300-native (sm_103a) Kimi Delta Attention forward pass.

The computation lives in libkda.so (CUDA sources in csrc/, C ABI in include/kda.h);
this package builds and loads it and marshals arguments.  There is no CPU path.
"""
from ._native import KDAError, build, load  # noqa: F401
from .api import device_status, kda_fwd, kda_fwd_host, kda_fwd_recurrent, workspace_size  # noqa: F401
from .step import (beam_select_workspace_size, kda_beam_select, kda_kv_append, kda_state_reorder,  # noqa: F401
                   kda_window_attn, window_attn_workspace_size)

__all__ = ["kda_fwd", "kda_fwd_recurrent", "workspace_size", "device_status", "kda_fwd_host", "KDAError", "build", "load",
           "kda_kv_append", "kda_window_attn", "kda_beam_select", "kda_state_reorder", "window_attn_workspace_size",
           "beam_select_workspace_size"]
