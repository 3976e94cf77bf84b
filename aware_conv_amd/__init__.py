"""Fused WTConv (multi-level 2-D Haar wavelet depthwise convolution) for AMD
Instinct MI355X.

The layer runs in hand-written HIP kernels behind the C ABI of
``include/wtconv.h`` (``libwtconv.so``); :mod:`aware_conv_amd._lib` binds it
with ctypes.  :class:`WTConv2d` is a drop-in replacement for a depthwise
``nn.Conv2d`` that saves only its input for the backward.

Beside the layer: a gated linear recurrence over whole planes or token
sequences (``include/gscan.h``, :mod:`aware_conv_amd.gscan`,
:class:`GatedScan2d`) and the AdamW step over many tensors
(``include/adamw.h``, :mod:`aware_conv_amd.adamw`, :class:`AdamW`).

Nothing is imported eagerly, so ``import aware_conv_amd.build`` works before
the library exists.
"""

__all__ = ["WTConv2d", "WTConvFunction", "wtconv_fwd", "wtconv_bwd_input",
           "wtconv_bwd_weight", "wtconv_workspace_size",
           "gscan_fwd", "gscan_bwd", "gscan_step", "gated_scan", "GatedScan2d",
           "adamw_grad_norm", "adamw_step", "AdamW"]


_HOMES = {"_lib": ("wtconv_fwd", "wtconv_bwd_input", "wtconv_bwd_weight",
                   "wtconv_workspace_size", "wtconv_strerror", "make_shape"),
          "module": ("WTConv2d", "WTConvFunction", "GatedScan2d"),
          "gscan": ("gscan_fwd", "gscan_bwd", "gscan_step", "gated_scan", "GatedScanFunction"),
          "adamw": ("adamw_grad_norm", "adamw_step", "AdamW")}


def __getattr__(name):
    for home, names in _HOMES.items():
        if name in names:
            import importlib
            value = getattr(importlib.import_module("." + home, __name__), name)
            globals()[name] = value  # found directly from now on
            return value
    raise AttributeError(name)
