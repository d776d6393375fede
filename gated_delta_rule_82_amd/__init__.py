"""MI355X-native KDA decode: the HIP library libkda and its thin binding.

    from gated_delta_rule_82_amd import kda      # binding (needs torch)
    kda.decode(out, q, k, v, raw_gate, beta_logits, a_log, dt_bias,
               cu_seqlens, state_pool, state_indices, gate_mode="softplus")

``kda.gdr_decode`` and ``kda.gdr_prefill`` run the gated delta rule with one decay
per head, ``kda.decode_window`` a window of drafted tokens and ``kda.verify``
decides which of them stand.  ``kda.ssm_decode`` and ``kda.ssm_prefill`` run the
selective state space scan with its convolution, ``kda.norm_residual`` and
``kda.norm_gate`` the norms before and after a block.

``workloads`` draws the seeded synthetic inputs; ``build`` compiles the
library for gfx950.
"""
__all__ = ["kda", "workloads", "build"]
