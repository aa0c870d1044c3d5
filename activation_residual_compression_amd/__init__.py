"""librescomp: residual compression with error feedback for parallel diffusion
inference, as hand-written HIP kernels for gfx950 behind a small C ABI.

Submodules:
  librescomp -- ctypes binding of the C ABI (loads the HIP library; fails loudly
                when it is not built).
  session    -- warm-up, schedule of schemes over the steps, ablation modes.
  peer_attention -- exchange of keys and values as residuals, 8-bit cache, attention.
  synth      -- seeded synthetic activation sequences (inputs only).
  build      -- compiles the HIP library for gfx950.
"""
