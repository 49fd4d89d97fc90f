"""Chunked Kimi Delta Attention (KDA) forward for NVIDIA GB300 (sm_103a).

The compute path is the C-ABI library ``libkda.so`` built from ``csrc/``
(hand-written CUDA kernels).  ``kda_fwd`` (Python, in ``binding.py``) only
marshals torch tensors into that C call; importing it loads the library and
fails loudly when it is missing.  ``inputs`` (synthetic workloads) is
importable without the library.  ``latent`` has the latent attention, its
paged cache and its tables, for the full-attention layers beside KDA layers,
``pages`` what shares, frees and moves the cache's pages, ``drafts`` the
verification of drafted tokens.
"""

__all__ = ["fwd", "kda_fwd", "load_library", "latent", "pages", "drafts"]


def __getattr__(name):
    if name in ("fwd", "kda_fwd", "load_library", "workspace_bytes", "KdaError"):
        from . import binding
        return getattr(binding, name)
    if name in ("latent", "pages", "drafts"):
        import importlib
        return importlib.import_module("." + name, __name__)
    raise AttributeError(name)
