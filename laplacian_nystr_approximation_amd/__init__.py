"""MI355X-native forward (and backward) pass of LaplacianFormer's Laplacian-kernel Nystrom attention.

The computation lives in the HIP library ``liblapnys.so`` (C ABI in
``include/lapnys.h``); ``laplacian_nystr_approximation_amd.lapnys`` is its
ctypes binding, whose names are re-exported here, and so are those of
``laplacian_nystr_approximation_amd.lapmix``, the binding of the operators beside
the attention (``include/lapmix.h``).  The library is loaded on
first use of any of them, and that use raises ImportError if it has not been
built (``python -m laplacian_nystr_approximation_amd.build``).
"""

import importlib

_BINDING_NAMES = {
    "HipEvents", "LapnysError", "lapnys_debug", "lapnys_params", "lapnys_forward", "lapnys_forward_ws",
    "lapnys_forward_debug", "lapnys_forward_profiled", "lapnys_landmark_count", "lapnys_workspace_size",
    "lapnys_release", "lapnys_status_string", "make_params", "params_for", "library", "LIB_PATH",
    "DEBUG_FIELDS", "STAGE_NAMES", "LAPNYS_NUM_STAGES", "lapnys_backward_ws", "lapnys_backward_workspace_size",
    "lapnys_forward_noalloc",
}

_MIX_NAMES = {
    "lapmix_scan_params", "lapmix_norm_params", "make_scan_params", "make_norm_params",
    "lapmix_scan_workspace_size", "lapmix_scan_states_size", "lapmix_scan_forward_ws", "lapmix_scan_backward_ws",
    "lapmix_scan_step", "lapmix_norm_forward", "lapmix_norm_workspace_size", "lapmix_norm_backward_ws",
    "LAPMIX_SCAN_TILE",
}


def __getattr__(name):
    module = ".lapnys" if name in _BINDING_NAMES else ".lapmix" if name in _MIX_NAMES else None
    if module is None:
        raise AttributeError(name)
    # Kept in the module's namespace: later uses find it without coming here.
    value = globals()[name] = getattr(importlib.import_module(module, __name__), name)
    return value
