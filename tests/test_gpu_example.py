"""The post-training example: its phases learn, and its weights are the owners' masters in fp16."""
import importlib.util
import math
import os

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_post_training_example_learns():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    spec = importlib.util.spec_from_file_location("post_training", os.path.join(ROOT, "examples", "post_training.py"))
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    t = ex.Trainer()
    rewards = ex.policy_phase(t, 60)
    assert rewards[-1] > 5 * rewards[0] and rewards[-1] > 0.2  # chance is 1 in 96
    seen = ex.preference_phase(t, 30)
    assert abs(seen[0][0] - math.log(2)) < 1e-3  # the reference is the model itself
    assert seen[-1][0] < 0.5 * seen[0][0] and seen[-1][1] == 1.0
    assert t.step == 90
    for own in t.owners:
        dense = torch.zeros(own.dense_total, device="cuda")
        own.to_dense(own.master, dense)
        for (o, n), d in zip(t.slots, own.dense_offsets):
            lo, hi = max(o, own.begin), min(o + n, own.end)
            if lo < hi:
                d = int(d)
                assert torch.equal(t.flat[lo:hi], dense[d + lo - o:d + hi - o].half())
