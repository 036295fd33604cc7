"""swiglu_describe_backward names what the launches plan (needs a device: its compute units)."""
from __future__ import annotations

import pytest
import torch

from gated_mlp_gemm_amd import swiglu as sw

pytestmark = pytest.mark.gpu
F32 = torch.float32


@pytest.fixture(autouse=True)
def _default_dispatch(monkeypatch):
    monkeypatch.delenv("SWIGLU_I_TILE", raising=False)
    monkeypatch.delenv("SWIGLU_TAIL", raising=False)


def test_few_rows_split_alike_whatever_the_epilogue():
    """Up to 128 rows the gradient by an activation is planned by its product alone: dGU's
    tiles (whose epilogue moves more) split as dH's do."""
    size = sw.swiglu_workspace_size(64, 1024, 1024, "ablation")
    texts = set()
    for M in (1, 64, 128):
        for N in (8, 520, 1032, 2056, 4104, 5440, 8192, 12296, 16384, 18944):
            for K in (64, 264, 520, 896, 1536, 1800, 1984, 2112, 3584, 5120, 8192):
                block = sw.swiglu_describe_backward(M, N, K, "gated_mlp", F32, False, size)
                down = sw.swiglu_describe_backward(M, N, K, "down_proj", F32, False, size)
                dgu = block.split(", then ")[0].replace("GateGradEpilogue", "StorePairs")
                assert dgu == down, (M, N, K)
                texts.add(dgu)
    assert any("split" in t for t in texts) and any("(1 tiles" in t for t in texts)


@pytest.mark.parametrize("call,parts", [("down_proj", 1), ("fused_gemm", 2), ("gated_mlp", 2)])
def test_stages(call, parts):
    text = sw.swiglu_describe_backward(300, 520, 264, call, F32)
    assert len(text.split(", then ")) == parts and "gemm_pair_kernel" not in text
    assert text.startswith("gate_grad_kernel") == (call == "fused_gemm")
    none = sw.swiglu_describe_backward(0, 520, 264, call, F32)      # only zeros are stored
    assert none.count("WeightGradEpilogue") == (2 if call == "gated_mlp" else 1)
    assert "StorePairs" not in none and "GateGrad" not in none and "gate_grad" not in none
