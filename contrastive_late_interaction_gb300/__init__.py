"""In-batch contrastive scoring on one GB300: the fused SigLIP sigmoid pair loss and hard MaxSim.

The compute path is the CUDA library built from `csrc/` (C ABI in `include/cli.h`);
`_binding` and, for what stands between a tower's blocks, `_norms` only marshal
arguments to it and raise if the library is missing.  `synth` draws the seeded
inputs.  The binding's names are re-exported lazily, so `synth` imports without
a built library.
"""

import importlib
import sys
import types

_BINDING_NAMES = {
    "CliError", "DeviceError", "InternalError", "InvalidArgumentError", "MalformedError", "ShapeMismatchError",
    "UnsupportedError", "check_device_status", "device_edges", "maxsim_backward", "maxsim_backward_workspace_bytes",
    "maxsim_scores", "maxsim_workspace_bytes", "pair_loss_sigmoid_fwd_bwd", "pair_loss_sigmoid_scores_fwd_bwd",
    "pair_loss_sigmoid_scores_workspace_bytes", "pair_loss_sigmoid_workspace_bytes", "status_name", "LIB_PATH",
    "raise_for", "pair_loss_scores_fwd_bwd", "pair_loss_scores_workspace_bytes",
    "pair_loss_sigmoid_matryoshka_fwd_bwd", "pair_loss_sigmoid_matryoshka_workspace_bytes",
    "pair_loss_sigmoid_groups_fwd_bwd", "maxsim_scores_named", "maxsim_named_workspace_bytes",
    "maxsim_backward_named", "selftest_bounded_wait", "rotary_table", "rotary_heads", "rotary_heads_backward",
    "norm_rotary_heads", "norm_rotary_heads_backward", "cross_attention", "cross_attention_backward",
    "cross_attention_workspace_bytes", "cross_attention_backward_workspace_bytes",
    "norm_rotary_heads_backward_workspace_bytes",
}

_NORM_NAMES = {
    "layer_norm", "layer_norm_backward", "layer_norm_backward_workspace_bytes", "dropout", "dropout_backward",
    "dropout_layer_norm", "dropout_layer_norm_backward",
}


class _Name:
    """A name of the binding, looked up there each time: cheaper than a module's __getattr__, and a name that is set on the
    package itself still comes first."""

    def __init__(self, name, module):
        self.name, self.module = name, module

    def __get__(self, package, kind=None):
        binding = _loaded.get(self.module)
        if binding is None:
            binding = _loaded[self.module] = importlib.import_module(self.module, __name__)
        return getattr(binding, self.name)


_loaded = {}
_Package = type("_Package", (types.ModuleType,), {name: _Name(name, module) for names, module in (
    (_BINDING_NAMES, "._binding"), (_NORM_NAMES, "._norms")) for name in names})
sys.modules[__name__].__class__ = _Package
