"""The stages for a profiler make the operators' own arrays."""
import sys

import pytest

import workloads as wl
from tree_verify_b200 import profile_case

pytestmark = pytest.mark.gpu


def test_paged_attention_stage_passes_nodes_before_heads(cuda_lib, monkeypatch):
    seen = []
    call = cuda_lib.tree_attention_paged

    def record(shape, pages, q, k_pages, v_pages, table, lens, shared, k_tree, v_tree, parents, out, *rest):
        seen.append((q, k_tree, v_tree, out))
        call(shape, pages, q, k_pages, v_pages, table, lens, shared, k_tree, v_tree, parents, out, *rest)

    monkeypatch.setattr(cuda_lib, "tree_attention_paged", record)
    monkeypatch.setattr(sys, "argv", ["profile_case", "--workload", "llama3_8b", "--stage", "paged_attention",
                                      "--launches", "1"])
    profile_case.main()
    w = wl.WORKLOADS["llama3_8b"]
    (q, k_tree, v_tree, out), = seen
    rows = (w.batch, w.num_nodes)
    assert q.shape == out.shape == (*rows, w.num_q_heads, w.head_dim)
    assert k_tree.shape == v_tree.shape == (*rows, w.num_kv_heads, w.head_dim)
