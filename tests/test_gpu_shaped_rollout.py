"""The rollout and training step of examples/shaped_rollout.py: adapters, shaping,
shaped log-probs and their gradient in the order in which a program uses them."""
import importlib.util
import os

import pytest
import torch

from gpu_helpers import gpu_lib  # noqa: F401

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _example():
    spec = importlib.util.spec_from_file_location("shaped_rollout", os.path.join(ROOT, "examples", "shaped_rollout.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_rollout_then_training_step(gpu_lib):
    m = _example()
    tokens, old, logp, seam, dlogits, settings = m.main(requests=8, prompt=9, new_tokens=20, V=3001)
    # 8 rows a step and 160 rows at once take other tiles, column ranges and chains: the same bits, so a ratio of 1
    assert torch.equal(logp.view(torch.int32), old.view(torch.int32))
    assert torch.all(seam["seg_ratio"] == 1.0)
    assert torch.all(torch.isfinite(old)) and torch.all(old < 0)
    new = tokens[:, 9:]
    banned = settings["bias_set"] == 0
    assert not torch.any(new[banned] == 1)                       # biased to -inf
    assert torch.all(new[settings["allow_row"] == 0] < 128)      # the grammar
    # each row's gradient sums to 0 over z' (softmax minus one-hot), so over z it is 0 where no slope differs: check
    # that it is finite and vanishes at barred tokens
    d = dlogits.float().view(8, 20, -1)
    assert torch.all(torch.isfinite(d)) and torch.all(d[settings["allow_row"] == 0][:, :, 128:] == 0)
    assert d.abs().sum() > 0
