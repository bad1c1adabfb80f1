"""GB300-native hot path of the FLUX.2 MMDiT denoiser: the joint attention and the
products and norms around it in a block.

The compute runs in the CUDA library built from ``csrc/`` (C-ABI declared in
``include/flux_attn.h``); ``binding`` marshals torch device tensors into it:

- ``rope_tables`` / ``rope_tables_packed``: cos/sin tables from 4-axis ids;
- ``joint_rope_attention`` (and ``joint_rope_attention_tabled``): RoPE fused
  into the Q/K tile loads, softmax(QK^T / sqrt(128)) V over [txt ; img],
  optionally with the QK RMS normalisation before RoPE (``qk_norm=``);
- ``attention_extract`` / ``attention_cached``: the reference-image KV modes;
- ``qkv_mlp_proj``: the single-stream block's fused Q/K/V + SwiGLU-MLP input
  projection, writing Q, K, V in the attention's [B, S, H, 128] layout;
- ``linear``: a block's other products, with bias, activation, gate and
  residual in the epilogue;
- ``modulated_norm``: the modulated norm with the gated residual in front;
- ``quantize_fp8`` and ``linear_fp8``: ``linear`` over 8-bit operands with a scale
  per 128 channels, and what makes them;
- ``cross_attention``: attention to another sequence (an encoder's states).

Importing this package does not load the library; the first call does, and
fails loudly when it is missing (there is no CPU path).
"""
from . import workloads  # noqa: F401

__all__ = ["workloads"]
