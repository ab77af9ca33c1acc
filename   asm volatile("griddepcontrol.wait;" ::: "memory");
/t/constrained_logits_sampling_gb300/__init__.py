"""GB300-native batched constrained logits sampler, and the operators of a speculative step
around it (``speculative``; ``tree`` where drafted tokens form a tree, ``pages`` for the cache's pages).

The compute path is the CUDA library ``libclsample.so`` (built from ``csrc/``); the
Python side only marshals arguments.  Importing the package does not load the
library: ``sampler.Sampler`` and the operators' classes do, and they raise if the library is missing.
"""

__all__ = ["workloads", "sampler", "speculative", "tree", "pages"]
