"""The example's decoder with a dropout: which numbers its joins drop."""
import pytest

from test_train_join_gpu import example  # noqa: F401

pytestmark = pytest.mark.gpu
LAYERS, WIDTH = 2, 128


@pytest.fixture
def logged(example, monkeypatch):  # noqa: F811
    """Calls of the example's joins: (x, y, x', call, step, seed)."""
    log = []

    class Logged(example.BlockJoin):
        def __call__(self, x, y, *args, **kw):
            out = super().__call__(x, y, *args, **kw)
            log.append((x.detach(), y.detach(), out[0].detach(), kw["call"], kw["step"], kw["seed"]))
            return out
    monkeypatch.setattr(example, "BlockJoin", Logged)
    return log


def losses_of(example, dropout, steps):  # noqa: F811
    import torch
    from zero_sharded_mixed_05_gb300.qk import rotation_tables
    dev = torch.device("cuda", torch.cuda.current_device())
    tokens = example.batch_of(torch.Generator(device=dev).manual_seed(5), 4, 48, dev)
    cos, sin = rotation_tables(128, example.HEAD, device=dev)
    model = example.Decoder(WIDTH, LAYERS, dev, dropout)
    flats = [example.Flat(model.matrices()), example.Flat(model.others())]
    with torch.no_grad():
        out = [float(model.loss(tokens, cos, sin, step)) for step in steps]
    model.close()
    del flats
    return out


def test_the_loss_goes_by_dropout_and_step(example):  # noqa: F811
    """The same weights and data: a step's loss is the same bits again, another
    step's and that of no dropout are others."""
    a, b, again = losses_of(example, 0.1, (0, 1, 0))
    (none,) = losses_of(example, 0.0, (0,))
    assert a == again and len({a, b, none}) == 3


def test_every_join_drops_numbers_of_its_own(example, logged):  # noqa: F811
    """Of the numbers whose branch would change the stream (|y| above 2^-9 |x|; fp16's
    half step is 2^-11) a tenth stay what they were, by five standard deviations, and
    which ones is another choice in every join and step."""
    losses_of(example, 0.1, (0, 1))
    assert [(c, s) for *_, c, s, _ in logged] == [(c, s) for s in (0, 1) for c in range(2 * LAYERS)]
    gone = [(xo == x) & (y.abs() > 2.0 ** -9 * x.abs()) for x, y, xo, *_ in logged]
    there = [y.abs() > 2.0 ** -9 * x.abs() for x, y, *_ in logged]
    for g, t in zip(gone, there):
        n = t.sum().item()
        assert n > 10000 and abs(g.sum().item() - 0.1 * n) <= 5 * (0.09 * n) ** 0.5 + n / 65536
    for i in range(len(gone)):
        for j in range(i):
            both = there[i] & there[j]
            n, k = both.sum().item(), (gone[i] & gone[j] & both).sum().item()
            assert abs(k - 0.01 * n) <= 5 * (0.0099 * n) ** 0.5 + n / 32768


def test_training_passes_the_step_on(example, logged):  # noqa: F811
    example.train(steps=3, width=WIDTH, layers=LAYERS, quiet=True, dropout=0.1)
    assert [(c, s) for *_, c, s, _ in logged] == [(c, s) for s in range(3) for c in range(2 * LAYERS)]
    assert len({seed for *_, seed in logged}) == 1
