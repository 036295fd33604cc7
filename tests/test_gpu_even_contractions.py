"""Contractions of whole K steps (needs an MI355X): widths that are multiples of 64, as those
of real models are, take the unrolled walk round the LDS rings, one compiled step for each
stage.  The training calls and the calls on 4-bit weights, in every tile and tail, with every
number of steps that a walk can leave over; against 64-bit products (bounds as in
test_gpu_train.py and test_gpu_mx4.py)."""
from __future__ import annotations

import pytest
import torch

import test_gpu_mx4 as mx4
import test_gpu_train as train
from gated_mlp_gemm_amd import swiglu as sw

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def _default_dispatch(monkeypatch):
    monkeypatch.delenv("SWIGLU_I_TILE", raising=False)
    monkeypatch.delenv("SWIGLU_TAIL", raising=False)


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a ROCm device"
    sw.load_library()
    return torch.device("cuda:0")


SCHEDULES = [("256", "whole"), ("256", "split"), ("256", "quarter"), ("128", "whole"),
             ("128", "split")]


def force(monkeypatch, schedule):
    monkeypatch.setenv("SWIGLU_I_TILE", schedule[0])
    monkeypatch.setenv("SWIGLU_TAIL", schedule[1])


# 1 to 3 steps, and 9 to 14: the rings' walks are of 2, 4 and 6 steps
STEPS = [1, 2, 3, 9, 10, 11, 12, 13, 14]


@pytest.mark.parametrize("schedule", SCHEDULES)
def test_training_forward(dev, monkeypatch, schedule):
    force(monkeypatch, schedule)
    for steps in STEPS:
        K, N = 64 * steps, 64 * (steps % 5 + 4)
        train.check_forward(dev, 300, K, N, train.workspace_of(dev, 300, N, K), steps)


@pytest.mark.parametrize("schedule", SCHEDULES)
def test_training_backward(dev, monkeypatch, schedule):
    force(monkeypatch, schedule)
    for steps in STEPS:
        K, N = 64 * steps, 64 * (14 - steps % 7)
        train.check_backward(dev, 64 * (steps % 4 + 4), K, N, train.workspace_of(dev, 512, N, K),
                             steps, F32 if steps % 2 else BF, add=steps % 3 == 0)


@pytest.mark.parametrize("M", [1, 64, 100, 128, 129, 512, 1536])
def test_training_as_chosen(dev, M):
    """More tiles than compute units among them: whole rounds, then a tail."""
    K, N = 896, 2816
    for ws in (None, train.workspace_of(dev, M, N, K)):
        train.check_forward(dev, M, K, N, ws, M)
        train.check_backward(dev, M, K, N, ws, M, F32, add=ws is not None)


@pytest.mark.parametrize("schedule", [s for s in SCHEDULES if s[1] != "quarter"])
def test_4_bit_tiles(dev, monkeypatch, schedule):
    force(monkeypatch, schedule)
    for steps in STEPS:
        K, N = 64 * steps, 64 * (14 - steps % 7)
        mx4.check_block(dev, 300, K, N, mx4.workspace_of(dev, 300, N, K), steps)


@pytest.mark.parametrize("M", [1, 24, 64, 65, 100, 128, 129, 257, 512, 1536])
def test_4_bit_as_chosen(dev, M):
    K, N = 896, 2816
    for ws in (None, mx4.workspace_of(dev, M, N, K)):
        mx4.check_block(dev, M, K, N, ws, M)
    for steps in STEPS:
        mx4.check_block(dev, M, 64 * steps, 64 * (15 - steps), mx4.workspace_of(dev, M, 960, 896), steps)
