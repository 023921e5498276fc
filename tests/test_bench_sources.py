"""Which sources the benchmark's stored counter readings depend on (runs without
a GPU): those of its own workloads, and none of the separate operators'."""
from __future__ import annotations

import os
import shutil

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join("activation_sparse_gated_amd", "csrc")
OPERATORS = {"k_linear.hip", "k_linear_skinny.hip", "k_rmsnorm.hip", "k_quant.hip", "lin_util.cuh", "linear.cuh", "linear_api.hip",
             "k_router.hip", "k_rows.hip", "experts.cuh", "experts_api.hip", "k_adapter.hip", "adapter.cuh", "adapter_api.hip"}


@pytest.mark.parametrize("name", sorted(os.listdir(os.path.join(ROOT, CSRC))))
def test_source_hash(name, tmp_path, monkeypatch):
    import bench
    shutil.copytree(os.path.join(ROOT, CSRC), tmp_path / CSRC)
    monkeypatch.setattr(bench, "ROOT", str(tmp_path))
    before = bench.src_hash()
    with open(tmp_path / CSRC / name, "a") as fh:
        fh.write("\n")
    assert (bench.src_hash() == before) == (name in OPERATORS)


def test_operators_are_there():
    assert OPERATORS <= set(os.listdir(os.path.join(ROOT, CSRC)))
