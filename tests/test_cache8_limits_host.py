"""What the native binding of the tables, writes and 8-bit calls refuses and reports, without a GPU."""
import os
import subprocess

import pytest
import torch

import block_sparse_kv_pred_gb300 as bs
from block_sparse_kv_pred_gb300 import build as B
from _parity import ensure_built

D = 128


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def test_writes_without_rows_check_everything_else():
    rows = torch.zeros((0, 2, D), dtype=torch.bfloat16)
    pool, plain = torch.zeros((3, 32, D), dtype=torch.float8_e5m2), torch.zeros((3, 32, D), dtype=torch.bfloat16)
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    good = {"page_table": i(1, 2, 4), "seq_len": i(1), "K_scale": torch.zeros(3), "V_scale": torch.zeros(3),
            "prev_len": i(1), "status": i(1)}

    def write8(**kw):
        v = {**good, **kw}
        bs.append_kv8(rows, rows, v["page_table"], v["seq_len"], 1, 2, 32, pool, pool, v["K_scale"], v["V_scale"],
                      prev_len=v["prev_len"], status=v["status"])

    for name in good:
        with pytest.raises(bs.ScoutError, match=f"^{name} must be a contiguous"):
            write8(**{name: good[name].double()})
    with pytest.raises(bs.ScoutError, match="K_pool must be a CUDA tensor on"):  # everything else fits
        write8()
    for name, kw in (("slot_map", {"slot_map": i(0, 2)}), ("status", {"status": i(2)}), ("K_pool", {})):
        with pytest.raises(bs.ScoutError, match=f"^{name} must be a"):
            bs.append_kv(rows, rows, **{"slot_map": torch.zeros((0, 2), dtype=torch.int64), "Hkv": 2, "P": 32,
                                        "K_pool": plain, "V_pool": plain, **kw})


@pytest.mark.parametrize("missing", ["libscout.so", "libscoutgen.so", "_binding.so", None])
def test_a_tree_without_one_of_the_built_files_is_built(missing, monkeypatch, tmp_path):
    for n in ("libscout.so", "libscoutgen.so", "_binding.so"):
        if n != missing:
            (tmp_path / n).touch()
    built = []
    monkeypatch.setattr(bs, "lib_path", lambda: os.path.join(tmp_path, "libscout.so"))
    monkeypatch.setattr(B, "build", lambda: built.append(True))
    ensure_built()
    assert bool(built) == (missing is not None)


def test_the_libraries_are_built_where_the_binding_cannot_be(monkeypatch, tmp_path):
    # a compiler and a linker that only touch their output, and PyTorch headers that are not there
    def run(cmd, **kw):
        src = cmd[cmd.index("-c") + 1] if "-c" in cmd else ""
        if src == B.BINDING:
            return subprocess.CompletedProcess(cmd, 1, "", "torch/extension.h: No such file or directory")
        open(cmd[cmd.index("-o") + 1], "w").close()
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(B, "PKG", str(tmp_path))
    monkeypatch.setattr(B, "BUILD", str(tmp_path / "o"))
    monkeypatch.setattr(B.subprocess, "run", run)
    with pytest.raises(RuntimeError, match="binding.cpp"):
        B.build()
    assert {n for n in os.listdir(tmp_path) if n.endswith(".so")} == {"libscout.so", "libscoutgen.so"}


def test_a_binding_built_with_another_pytorch_is_refused(monkeypatch):
    assert torch.__version__.startswith(bs._native().torch_version)
    monkeypatch.setattr(bs, "_NATIVE", None)
    monkeypatch.setattr(torch, "__version__", "1.2.3+cpu")
    with pytest.raises(bs.ScoutError, match=r"built with PyTorch \d+\.\d+\.\d+, this is 1\.2\.3"):
        bs.build_tables(None, None, 1, 1, 1, 16, None, None)


def test_the_bytes_of_a_workspace_that_start_as_zero():
    n = bs._native().attn8_zero_bytes
    assert n == 4096 * 8 * 4  # a counter for each head of the most units
    assert bs.lib().scout_sparse_attn8_workspace_bytes(1, 8, 1, 128, 32) > n
    w = bs.sparse_attn8_workspace(1, 8, 1, 32, device="cpu")
    assert w.numel() == bs.lib().scout_sparse_attn8_workspace_bytes(1, 8, 1, 128, 32) and not w[:n].any()
