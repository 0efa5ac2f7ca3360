"""Recorded DRAM traffic stands for the sources it was measured on: a change to anything that takes part
in the recorded launches, their host planning among it, changes the digest."""
import os
import shutil

import pytest

import bench

CSRC = os.path.join("fp4_sparse_attention_gb300", "csrc")
FILES = sorted(os.listdir(os.path.join(bench.ROOT, CSRC)))
OTHERS = {"api_attention.cu", "attention.cu", "attention.h", "attn_ptx.cuh", "build_tables.cu", "store_rows.cu"}


@pytest.mark.parametrize("name", FILES + ["new_kernel.cu"])
def test_digest_follows_every_unit_but_the_attention_ones(name, tmp_path, monkeypatch):
    shutil.copytree(os.path.join(bench.ROOT, CSRC), tmp_path / CSRC)
    monkeypatch.setattr(bench, "ROOT", str(tmp_path))
    before = bench.source_sha()
    with open(tmp_path / CSRC / name, "a") as f:
        f.write("// changed\n")
    assert (bench.source_sha() == before) == (name in OTHERS)
