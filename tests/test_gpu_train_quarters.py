"""Quarter-size tails of the training calls (needs an MI355X): forced, with contractions that
end inside a K step and quarters wholly past the output's edge; bounds as in
test_gpu_train.py."""
from __future__ import annotations

import pytest
import torch

import test_gpu_train as train
from gated_mlp_gemm_amd import swiglu as sw

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a ROCm device"
    sw.load_library()
    return torch.device("cuda:0")


# (the last one: whole rounds of tiles, then quarters)
@pytest.mark.parametrize("M,K,N", [(129, 8, 8), (130, 72, 136), (300, 264, 520), (385, 200, 264),
                                   (513, 328, 136), (640, 1000, 72), (2100, 136, 4360)])
def test_quarters(dev, monkeypatch, M, K, N):
    monkeypatch.setenv("SWIGLU_I_TILE", "256")
    monkeypatch.setenv("SWIGLU_TAIL", "quarter")
    text = sw.swiglu_describe_backward(M, N, K, "gated_mlp", train.F32, True)
    assert "run as" in text.split(", then ")[0], text
    train.check_forward(dev, M, K, N, None, M)
    train.check_backward(dev, M, K, N, None, M, train.F32, add=True)
    train.check_backward(dev, M, K, N, None, M, train.BF, add=True, in_place=True)
