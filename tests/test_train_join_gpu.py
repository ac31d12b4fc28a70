"""The example's decoder with its joins in one pass: it runs, and its gradients
are those of torch's norms and additions."""
import os
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import train_muon
    finally:
        sys.path.pop(0)
    return train_muon


def test_gradients_without_dropout_are_those_of_torch(example):
    """Two blocks in fp16.  Each number passes some sixty roundings of 2^-11 forward
    and back, independent of one another in the two programs where they differ:
    sqrt(2 * 60) 2^-11 = 5e-3 of a gradient's norm in the mean, tested at 2.5e-2."""
    import torch
    import zero_sharded_mixed_05_gb300 as z  # noqa: F401
    from zero_sharded_mixed_05_gb300.qk import rotation_tables
    dev = torch.device("cuda", torch.cuda.current_device())
    tokens = example.batch_of(torch.Generator(device=dev).manual_seed(3), 4, 48, dev)
    cos, sin = rotation_tables(128, example.HEAD, device=dev)
    grads = []
    for dropout in (None, 0.0):
        model = example.Decoder(128, 2, dev, dropout)
        flats = [example.Flat(model.matrices()), example.Flat(model.others())]
        loss = model.loss(tokens, cos, sin)
        (loss * 1024.0).backward()
        grads.append([p.grad.clone() for f in flats for p in f.params])
        assert 3.0 < float(loss.detach()) < 6.0
        model.close()
    for a, b in zip(*grads):
        assert a.isfinite().all() and b.isfinite().all()
        assert (a.double() - b.double()).norm() <= 2.5e-2 * a.double().norm()


def test_training_with_dropout_runs(example):
    losses = example.train(steps=4, width=128, layers=2, quiet=True, dropout=0.1)
    assert len(losses) == 4 and all(v == v and v < 20 for v in losses)
