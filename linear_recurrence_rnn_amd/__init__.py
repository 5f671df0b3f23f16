"""MI355X (gfx950) per-channel linear recurrences: RWKV-4 WKV forward/backward and
real/complex diagonal scans with their adjoints, the gated delta rule (a matrix of state per head)
and the per-token group norm that follows it, and the parts of a selective state space layer (its scan,
the short causal convolution, the root-mean-square norm), as hand-written HIP kernels behind a C ABI
(``include/linrec.h``).  The Python functions here marshal torch tensors to that ABI.

The binding is imported lazily so that ``linear_recurrence_rnn_amd.workloads`` (the seeded
input generators) can be used without loading the GPU library.
"""

__all__ = ["wkv4_forward", "wkv4_forward_noalloc", "wkv4_forward_ex", "wkv4_decode_step", "token_shift", "token_shift_backward", "wkv4_backward", "wkv4_backward_gated", "wkv4_backward_ex",
           "wkv4_forward_ckpt", "wkv4_backward_ckpt", "wkv4_forward_ckpt_ex", "wkv4_backward_ckpt_ex", "wkv4_checkpoint_size", "scan_real", "scan_complex", "scan_real_backward",
           "scan_complex_backward", "scan_mingru", "scan_minlstm", "scan_real_decay",
           "scan_complex_normalized", "scan_mingru_backward", "scan_minlstm_backward",
           "scan_real_decay_backward", "scan_complex_normalized_backward", "workspace_size", "LinrecError",
           "gated_delta_forward", "gated_delta_forward_ckpt", "gated_delta_backward", "gated_delta_checkpoint_size",
           "gated_delta_decode_step", "gated_delta_workspace_size",
           "group_norm_act", "group_norm_act_backward", "group_norm_act_workspace_size",
           "scan_selective", "scan_selective_ckpt", "scan_selective_backward", "scan_selective_decode_step",
           "scan_selective_workspace_size", "scan_selective_checkpoint_size",
           "short_conv_act", "short_conv_act_backward", "short_conv_decode_step", "short_conv_act_workspace_size",
           "rms_norm_add", "rms_norm_add_backward", "rms_norm_add_workspace_size"]


def __getattr__(name):
    if name in __all__:
        from . import binding
        value = globals()[name] = getattr(binding, name)
        return value
    raise AttributeError(name)
