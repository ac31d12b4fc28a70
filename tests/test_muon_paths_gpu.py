"""The orthogonalised update's kernels path by path: what decides between them
is in csrc/muon.cu (choose_resident, products_cost, splits_of), and the sizes
here are chosen by it.  Definitions and tolerances are those of test_muon_gpu.py."""
import pytest

from test_muon_gpu import close, ortho64, spectrum, z  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("m,n,b", [(128, 400, 60), (900, 100, 36), (128, 2048, 18)])
def test_a_clusters_ctas_agree_call_after_call(z, m, n, b):  # noqa: F811
    """Clusters of two, four and eight CTAs, which send one another their parts
    of A while they go on to B: the same matrix in every place of the batch
    gives the same bits, in every call."""
    import torch
    g = spectrum("signal", 1, m, n, torch.Generator(device="cuda").manual_seed(n)).repeat(b, 1, 1)
    h = z.zero_muon_create(z.make_muon_config(), [(m, n, b)])
    try:
        first = torch.empty_like(g)
        z.zero_muon_orthogonalize(h, [g], [first])
        close(first, ortho64(g), "fp32")
        differ = torch.zeros((), device="cuda", dtype=torch.int64)
        out = torch.empty_like(g)
        for _ in range(60):
            z.zero_muon_orthogonalize(h, [g], [out])
            differ += (out != first[:1]).sum()
        assert int(differ) == 0
        assert z.zero_muon_last_step(h).fault == 0
    finally:
        z.zero_muon_destroy(h)


@pytest.mark.parametrize("shape", [(200, 60, 3), (90, 128, 400), (128, 400, 90), (1500, 100, 30), (40, 2000, 1)], ids=str)
def test_a_wait_that_runs_out_on_the_chip(z, shape):  # noqa: F811
    """One CTA a matrix with 256 columns and two CTAs an SM; clusters of two and
    eight, more than run at once: the call leaves its steps at the first wait
    that runs out (two seconds, not two a product), writes nothing, says so, and
    TMEM, barriers and clusters are as the next calls need them."""
    import time

    import torch
    m, n, b = shape
    g = torch.randn(b, m, n, device="cuda", generator=torch.Generator(device="cuda").manual_seed(8))
    h = z.zero_muon_create(z.make_muon_config(), [shape])
    try:
        want, out = torch.empty_like(g), torch.full_like(g, 7.0)
        z.zero_muon_orthogonalize(h, [g], [want])
        close(want, ortho64(g), "fp32")
        z.zero_muon_inject_wait_fault(h)
        t0 = time.time()
        z.zero_muon_orthogonalize(h, [g], [out])
        assert z.zero_muon_last_step(h).fault == 1 and (out == 7).all()
        assert time.time() - t0 < 5.0
        for _ in range(3):
            z.zero_muon_orthogonalize(h, [g], [out])
            assert z.zero_muon_last_step(h).fault == 0 and torch.equal(out, want)
    finally:
        z.zero_muon_destroy(h)


@pytest.mark.parametrize("shapes", [[(100, 100, 400)], [(128, 1000, 40)], [(60, 60, 300), (90, 700, 50)]], ids=str)
def test_a_call_after_a_faulted_one_is_whole(z, shapes):  # noqa: F811
    """Queued behind it, with more CTAs than run at once and in several launches:
    it starts without the fault, gives what it always gives, and reports none;
    the faulted call reports its own, whichever of its launches ends last."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(4)
    g = [torch.randn(b, m, n, device="cuda", generator=gen) for m, n, b in shapes]
    h = z.zero_muon_create(z.make_muon_config(), shapes)
    try:
        want, out = ([torch.empty_like(t) for t in g] for _ in range(2))
        z.zero_muon_orthogonalize(h, g, want)
        for w, t in zip(want, g):
            close(w, ortho64(t), "fp32")
        for _ in range(2):
            z.zero_muon_inject_wait_fault(h)
            z.zero_muon_orthogonalize(h, g, out)
            assert z.zero_muon_last_step(h).fault == 1
            z.zero_muon_inject_wait_fault(h)
            z.zero_muon_orthogonalize(h, g, out)
            z.zero_muon_orthogonalize(h, g, out)
            assert z.zero_muon_last_step(h).fault == 0
            for w, t in zip(want, out):
                assert torch.equal(w, t)
    finally:
        z.zero_muon_destroy(h)


@pytest.mark.parametrize("shapes", [[(64, 64, 2)], [(60, 60, 300), (90, 700, 50)], [(257, 300, 1)]], ids=str)
def test_a_fault_that_nobody_asked_about_is_counted(z, shapes):  # noqa: F811
    """Once a faulted call, on the chip (one launch and several) and through the
    workspace, whatever calls come after it."""
    import torch
    g = [torch.randn(b, m, n, device="cuda") for m, n, b in shapes]
    out = [torch.empty_like(t) for t in g]
    h = z.zero_muon_create(z.make_muon_config(), shapes)
    try:
        for count in range(3):
            assert z.zero_muon_fault_count(h) == count
            z.zero_muon_orthogonalize(h, g, out)
            assert z.zero_muon_fault_count(h) == count and z.zero_muon_last_step(h).fault == 0
            z.zero_muon_inject_wait_fault(h)
            z.zero_muon_orthogonalize(h, g, out)
            if count == 1:
                assert z.zero_muon_fault_count(h) == 2 and z.zero_muon_last_step(h).fault == 1
            z.zero_muon_orthogonalize(h, g, out)
            z.zero_muon_orthogonalize(h, g, out)
    finally:
        z.zero_muon_destroy(h)


def test_step_refuses_tensors_that_are_not_the_handles(z):  # noqa: F811
    """Another order, type, size, shape or device than the handle's: an error on
    the host, before any launch; and the list is checked against every handle
    that it is given to."""
    import torch
    shapes = [(8, 16, 1), (16, 8, 1), (4, 4, 3)]

    def items(types=(torch.float16, torch.float32, torch.float32, torch.bfloat16)):
        return [{name: torch.zeros(b, m, n, device="cuda", dtype=t)
                 for name, t in zip(("grad", "momentum", "master", "param16"), types)} for m, n, b in shapes]
    cfg = z.make_muon_config(grad_dtype=z.FP16, param_dtype=z.BF16)
    h = z.zero_muon_create(cfg, shapes)
    try:
        good = items()
        good[0] = {k: t[0] for k, t in good[0].items()}            # one matrix without its batch
        good[1] = {k: t.flatten() for k, t in good[1].items()}     # a slice of a flat buffer
        lst = z.make_muon_list(good)
        z.zero_muon_step(h, lst)
        launches = z.zero_muon_launch_count(h)
        x = items()
        bad = [x[::-1], [x[1], x[0], x[2]], x[:2], x + x[:1]]
        for i, name, t in [(0, "grad", x[0]["grad"].bfloat16()), (1, "param16", x[1]["grad"]),
                           (0, "momentum", x[0]["momentum"].half()), (2, "master", x[2]["param16"]),
                           (2, "grad", x[2]["grad"][:2]), (0, "master", x[1]["master"]),
                           (1, "momentum", x[1]["momentum"].cpu()), (2, "grad", x[2]["grad"].view(12, 4)),
                           (0, "grad", x[0]["grad"].flatten()[:64])]:
            bad.append([m | ({name: t} if j == i else {}) for j, m in enumerate(x)])
        for b in bad:
            with pytest.raises(ValueError):
                z.zero_muon_step(h, z.make_muon_list(b))
        other = z.zero_muon_create(z.make_muon_config(grad_dtype=z.BF16), shapes)
        with pytest.raises(ValueError):
            z.zero_muon_step(other, lst)
        z.zero_muon_destroy(other)
        with pytest.raises(ValueError):
            z.zero_muon_step(other, lst)                           # a handle that is gone
        assert z.zero_muon_launch_count(h) == launches
        z.zero_muon_step(h, lst)
    finally:
        z.zero_muon_destroy(h)
