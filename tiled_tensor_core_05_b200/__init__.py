"""fp16 GEMM with a fused ReLU (or bias + GELU) epilogue for NVIDIA B200 (sm_100a).

The compute lives in ``libttc05.so`` (hand-written CUDA, C ABI declared in
``include/gemm_f16.h``).  The Python layer in ``ops.py`` only marshals
pointers, sizes and the current CUDA stream into that library; it never
computes anything itself and raises if the library is missing.

    from tiled_tensor_core_05_b200 import gemm_relu_f16, gemm_bias_act_f16
    c = gemm_relu_f16(a, b)                        # ReLU(a @ b), a (M, K), b (K, N) fp16
    y = gemm_bias_act_f16(x, w, bias, "gelu")      # GELU(x @ w + bias)
    z = gemm_general(x, w_nk, bias, "relu", trans_b=True)  # w stored N x K
    c_host = gemm_host(a_cpu, b_cpu)               # CPU tensors in and out, copies pipelined

Microscaled (8- and 4-bit) operands live beside them in ``libttcmx.so``
(``include/gemm_mx.h``, bound by ``mx.py``):

    w_q = mx_quantize(w_nk, "mxfp4")               # blocks of 32 with a power-of-two scale
    x_q, h = rms_norm(x, g, residual=r, format="mxfp4")
    y = gemm_mx(x_q, w_q, bias, "gelu")            # GELU(norm(x + r) @ w_nk.T + bias)

The feed-forward part of a model, with its backward pass and with 4-bit weights in
groups, in ``libttcff.so`` (``include/gemm_ff.h``, bound by ``ff.py``):

    h, gate, up = gemm_gated(x, w_gate, w_up, "silu", save=True)  # silu(x @ w_gate.T) * (x @ w_up.T)
    dx, dw_gate, dw_up = gemm_gated_backward(dh, x, w_gate, w_up, gate, up, "silu")
    y = gemm_w4(x, w4_pack(codes, scales, zeros), bias, "gelu")   # few rows, 4 bits a weight

``tune`` is the offline configuration sweep (``python -m
tiled_tensor_core_05_b200.tune``), ``shard`` the column-sharded product across
ranks, ``build`` compiles the library in-tree.

Importing this package does not load the library (so that ``workloads`` can be
used on machines without a GPU); the first call does.
"""
from __future__ import annotations

__all__ = ["gemm_relu_f16", "gemm_f16", "gemm_f16_ex", "gemm_bias_act_f16", "gemm_general",
           "gemm_config_run", "GemmConfig", "auto_config", "config_list", "config_smem_bytes",
           "activation_f32", "read_probe", "select_path", "device_status", "status_string",
           "gemm_host", "host_plan", "host_release", "lib",
           "MxTensor", "mx_quantize", "mx_dequantize", "rms_norm", "gemm_mx", "mx_empty",
           "mx_row_bytes", "mx_scale_bytes", "mx_tile_scales", "mx_untile_scales",
           "mx_device_status", "mx_lib",
           "gemm_gated", "gemm_gated_backward", "W4Tensor", "w4_pack", "w4_unpack", "gemm_w4",
           "gemm_gated_w4", "ff_device_status", "ff_lib"]

_FF = __all__[__all__.index("gemm_gated"):]
_MX = __all__[__all__.index("MxTensor"):__all__.index("gemm_gated")]


def __getattr__(name):
    if name in __all__:
        from . import ff, mx, ops
        value = getattr(mx if name in _MX else ff if name in _FF else ops, name)
        globals()[name] = value  # looked up once
        return value
    raise AttributeError(name)
