"""The smoke run needs no solver library on the GPU (one may be missing where the rest of PyTorch is present)."""
import pytest
import torch

import __graft_entry__ as entry

pytestmark = pytest.mark.gpu


def test_smoke_without_gpu_solvers(monkeypatch, capsys):
    def missing(*args, **kwargs):
        raise RuntimeError("no GPU solver library")

    for name in ("svd", "svdvals", "qr", "eigh", "eigvalsh", "eig", "inv", "solve", "cholesky", "lstsq", "pinv", "matrix_rank"):
        monkeypatch.setattr(torch.linalg, name, missing)
    for name in ("svd", "qr", "inverse", "cholesky"):
        monkeypatch.setattr(torch, name, missing)
    entry.smoke()
    assert "smoke ok" in capsys.readouterr().out
