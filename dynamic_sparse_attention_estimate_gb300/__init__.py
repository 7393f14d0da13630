"""GB300-native (sm_103a) dynamic sparse 3D attention for video DiT training (DSV), and the operators around it in a DiT
block: fused AdaLN (LayerNorm + modulation), rotary positions and the qk norm, the gated feed-forward, the gated residual with
its norms, and products of a few vectors with 4-bit weights (the modulation's projection).

The compute path is a C-ABI CUDA library (``libdsv.so``, entry points declared in
``include/dsv.h``); :mod:`.binding` is a thin ctypes layer over it that passes
device pointers, sizes and the current CUDA stream.  Importing this package does not
load the library; the first call does, and fails loudly if it has not been built.
"""
from .binding import (  # noqa: F401
    DSVError,
    RopeTable,
    W4Weight,
    dsv_adaln_bwd,
    dsv_adaln_bwd_workspace,
    dsv_adaln_fwd,
    dsv_estimate_mass_k,
    dsv_estimate_topk,
    dsv_estimate_topk_csr,
    dsv_estimate_topk_workspace,
    dsv_ffn_gated_bwd,
    dsv_ffn_gated_bwd_workspace,
    dsv_ffn_gated_fwd,
    dsv_ffn_gated_fwd_workspace,
    dsv_qk_norm_rope_bwd,
    dsv_qk_norm_rope_bwd_workspace,
    dsv_qk_norm_rope_fwd,
    dsv_residual_norm_bwd,
    dsv_residual_norm_bwd_workspace,
    dsv_residual_norm_fwd,
    dsv_rope3d_bwd,
    dsv_rope3d_fwd,
    dsv_rope3d_table,
    dsv_sparse_attn_bwd,
    dsv_sparse_attn_bwd_csr,
    dsv_sparse_attn_bwd_prepare,
    dsv_sparse_attn_bwd_prepared,
    dsv_sparse_attn_bwd_workspace,
    dsv_sparse_attn_fwd,
    dsv_sparse_attn_fwd_csr,
    dsv_w4_linear_bwd,
    dsv_w4_linear_bwd_workspace,
    dsv_w4_linear_fwd,
    dsv_w4_quantize,
    library_path,
    load_library,
)
