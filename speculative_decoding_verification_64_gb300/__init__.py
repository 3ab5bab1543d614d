"""GB300-native target-side verify step of speculative decoding.

The compute path is the C-ABI library ``libspecdec.so`` (hand-written CUDA for
sm_103a, built from ``csrc/`` by ``build.py``); ``binding`` is its thin ctypes
binding and ``workloads`` holds the seeded synthetic input generators.
"""
from .binding import (AppendOut, AttendOut, DistillOut, KVCache, LinearOut, SampleOut, SpecdecError,
                      TopOut, TreeOut, alloc_attend_workspace, alloc_workspace, attend,
                      attend_workspace_size, distill, distill_loss, filter_logits, kv_append,
                      linear_finalize, load_library, rope, rope_frequencies, row_stats, sample,
                      status_string, top_logits, top_logits_workspace_size, tree_finalize,
                      verify_linear, verify_tree, workspace_size)

__all__ = ["AppendOut", "AttendOut", "DistillOut", "KVCache", "LinearOut", "SampleOut", "TopOut",
           "TreeOut", "SpecdecError", "alloc_attend_workspace", "alloc_workspace", "attend",
           "attend_workspace_size", "distill", "distill_loss", "filter_logits", "kv_append",
           "linear_finalize", "load_library", "rope", "rope_frequencies", "row_stats", "sample",
           "status_string", "top_logits", "top_logits_workspace_size", "tree_finalize",
           "verify_linear", "verify_tree", "workspace_size"]
