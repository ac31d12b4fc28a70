"""The orthogonalised update's kernels path by path: what decides between them
is in csrc/muon.cu (choose_resident, products_cost, splits_of), and the sizes
here are chosen by it.  Definitions and tolerances are those of test_muon_gpu.py."""
import pytest

from test_muon_gpu import U, close, dt, expected, matrices, ortho64, spectrum, z  # noqa: F401

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
        good[2] = {k: t.view(12, 4) for k, t in good[2].items()}   # all matrices' rows
        lst = z.make_muon_list(good)
        z.zero_muon_step(h, lst)
        launches = z.zero_muon_launch_count(h)
        x = items()
        bad = [x[::-1], [x[1], x[0], x[2]], x[:2], x + x[:1]]
        for i, name, t in [(0, "grad", x[0]["grad"].bfloat16()), (1, "param16", x[1]["grad"]),
                           (0, "momentum", x[0]["momentum"].half()), (2, "master", x[2]["param16"]),
                           (2, "grad", x[2]["grad"][:2]), (0, "master", x[1]["master"]),
                           (1, "momentum", x[1]["momentum"].cpu()), (2, "grad", x[2]["grad"].view(6, 8)),
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


def expect(z, shapes, kind, src, dst, seed):  # noqa: F811
    """O of a list against the definition, with equal bits in a second call."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(seed)
    ins = [spectrum(kind, b, m, n, gen).to(dt(src)) for m, n, b in shapes]
    outs = [torch.full(x.shape, float("nan"), device="cuda", dtype=dt(dst)) for x in ins]
    h = z.zero_muon_create(z.make_muon_config(), shapes)
    try:
        z.zero_muon_orthogonalize(h, ins, outs)
        for x, o, s in zip(ins, outs, shapes):
            close(o, ortho64(x), dst, s)
        again = [torch.empty_like(o) for o in outs]
        z.zero_muon_orthogonalize(h, ins, again)
        for o, a in zip(outs, again):
            assert torch.equal(o, a)
        assert z.zero_muon_fault_count(h) == 0
    finally:
        z.zero_muon_destroy(h)


# 256 x 256 tiles of CTA pairs: square, wide and tall, sides that end inside a
# tile, X X^T whole and cut along its depth, X that stays in L2 and that does not.
PAIRS = [[(1500, 3001, 3)], [(3001, 1500, 3)], [(1000, 8000, 2)], [(8001, 1000, 2)], [(768, 8100, 4)],
         [(8100, 768, 4)], [(700, 1500, 20)], [(1500, 700, 20)],
         [(1536, 1536, 2), (1000, 1700, 2), (1700, 1000, 2), (600, 600, 4)]]


@pytest.mark.parametrize("shapes", PAIRS, ids=str)
@pytest.mark.parametrize("kind,src,dst", [("signal", "bf16", "fp32"), ("gauss", "fp32", "bf16")])
def test_pairs(z, shapes, kind, src, dst):  # noqa: F811
    expect(z, shapes, kind, src, dst, 41)


@pytest.mark.parametrize("shapes", [[(520, 4200, 8)], [(4200, 520, 8)], [(11840, 80, 24)], [(72, 9000, 30)],
                                    [(400, 12000, 2)], [(1000, 4000, 2)], [(8000, 500, 6)]], ids=str)
def test_single_ctas_with_x_beyond_l2_and_cut_depths(z, shapes):  # noqa: F811
    expect(z, shapes, "signal", "bf16", "fp32", 42)


LISTS = [[(60 + 8 * i, 40 + 9 * i, 1 + i % 3) for i in range(8)] + [(128, 128, 2), (1, 77, 3)],      # on the chip
         [(60 + i, 100 + 150 * i, 2) for i in range(12)],                                            # with clusters
         [(200 + 8 * i, 300 + 9 * i, 1) for i in range(6)] + [(500 - 31 * i, 260 - 17 * i, 1 + i % 2) for i in range(8)],
         [(1536, 1536, 1), (1000, 1700, 1), (1700, 1000, 1)] * 3 + [(600, 900, 4), (33, 700, 2)]]    # pairs


@pytest.mark.parametrize("shapes", LISTS, ids=["chip", "clusters", "singles", "pairs"])
def test_lists_of_more_than_eight_shapes(z, shapes):  # noqa: F811
    """More than a small launch argument and the first eight tensor maps hold."""
    assert len(shapes) > 8
    expect(z, shapes, "signal", "fp32", "fp32", 43)


@pytest.mark.parametrize("shapes", LISTS + PAIRS[-1:] + [PAIRS[0], PAIRS[3]],
                         ids=["chip", "clusters", "singles", "pairs", "list", "wide", "tall"])
@pytest.mark.parametrize("master", [True, False])
def test_steps_of_lists(z, shapes, master):  # noqa: F811
    """The step by path, with binary32 and with 16-bit masters."""
    import torch
    mats = matrices(shapes, "bf16", 44)
    for m in mats:
        m["master"] = m["master"] if master else None
    want = [expected(z, m, 1.0, 1e-2, 0.9, 0.1, True, 1) for m in mats]
    h = z.zero_muon_create(z.make_muon_config(grad_dtype=z.BF16, lr=1e-2, momentum=0.9, weight_decay=0.1,
                                              scale_rule=1), shapes)
    try:
        z.zero_muon_step(h, z.make_muon_list(mats))
        for m, (mom, tol_m, w, tol_w) in zip(mats, want):
            assert ((m["momentum"].double() - mom).abs() <= tol_m).all()
            got = m["master"] if master else m["param16"]
            tol = tol_w if master else tol_w + U["bf16"] * w.flatten(-2).norm(dim=-1)
            assert ((got.double() - w).flatten(-2).norm(dim=-1) <= tol).all()
            if master:
                assert torch.equal(m["param16"], m["master"].to(torch.bfloat16))
        assert z.zero_muon_fault_count(h) == 0
    finally:
        z.zero_muon_destroy(h)


@pytest.mark.parametrize("shapes", [[(300, 280, 1), (257, 130, 2)], PAIRS[-1]], ids=["singles", "pairs"])
def test_the_decision_through_the_workspace(z, shapes):  # noqa: F811
    """Unscale, clip and skip by the other parameters' decision in all three
    kernels: an overflow moves nothing, and the step after it is whole."""
    import torch
    lr, mu, n = 1e-2, 0.95, 1000
    opt = z.zero_opt_create(z.make_config(numel=n, grad_dtype=z.FP16, max_grad_norm=0.5, init_scale=1024.0,
                                          lr=1e-3))
    h = z.zero_muon_create(z.make_muon_config(lr=lr), shapes)
    try:
        p, m, v = (torch.zeros(n, device="cuda") for _ in range(3))
        p16 = torch.zeros(n, device="cuda", dtype=torch.float16)
        grad = torch.full((n,), 64.0, device="cuda", dtype=torch.float16)
        bufs = z.make_buffers(p, m, v, p16, [grad], grads_shard_local=True)
        mats = matrices(shapes, "fp16", 14, 1024.0)
        lst = z.make_muon_list(mats)
        where = z.zero_opt_decision(opt)
        for step in range(3):
            over = step == 1
            grad[5] = float("inf") if over else 64.0
            held = mats[0]["grad"][0, 0, 0].clone()
            if over:
                mats[0]["grad"][0, 0, 0] = float("inf")
            before = [{k: t.clone() for k, t in x.items()} for x in mats]
            z.zero_opt_step(opt, 0, bufs)
            info = z.zero_opt_last_step(opt)
            assert info.skipped == over
            want = None if over else [expected(z, x, info.coef, lr, mu, 0.0, True, 0) for x in mats]
            z.zero_muon_step(h, lst, decision=where)
            assert z.zero_muon_last_step(h).skipped == over
            if over:
                for x, y in zip(mats, before):
                    for k in x:
                        assert torch.equal(x[k], y[k])
                mats[0]["grad"][0, 0, 0] = held
                continue
            for x, (mom, tol_m, w, tol_w) in zip(mats, want):
                assert ((x["momentum"].double() - mom).abs() <= tol_m).all()
                assert ((x["master"].double() - w).flatten(-2).norm(dim=-1) <= tol_w).all()
    finally:
        z.zero_muon_destroy(h)
        z.zero_opt_destroy(opt)


@pytest.mark.parametrize("shape", [(300, 200, 4), (200, 300, 4), (1500, 1600, 4)], ids=str)
def test_zero_and_bad_matrices_through_the_workspace(z, shape):  # noqa: F811
    """A zero matrix gives zeros, one with a NaN or an infinity NaN, the others
    their result; and the workspace holds nothing of them over."""
    import torch
    m, n, b = shape
    g = torch.randn(b, m, n, device="cuda", generator=torch.Generator(device="cuda").manual_seed(6))
    good = g.clone()
    g[0] = 0
    g[1, 3, 4] = float("nan")
    g[2, m - 1, n - 1] = float("inf")
    h = z.zero_muon_create(z.make_muon_config(), [shape])
    try:
        out = torch.empty_like(g)
        z.zero_muon_orthogonalize(h, [g], [out])
        assert (out[0] == 0).all() and out[1].isnan().all() and out[2].isnan().all()
        close(out[3:], ortho64(g[3:]), "fp32")
        z.zero_muon_orthogonalize(h, [good], [out])
        close(out, ortho64(good), "fp32")
    finally:
        z.zero_muon_destroy(h)


@pytest.mark.parametrize("scale", [1e-6, 1e-3, 1e4])
@pytest.mark.parametrize("eps", [1e-7, 0.0])
def test_scale_of_the_input_through_the_workspace(z, scale, eps):  # noqa: F811
    import torch
    g = spectrum("gauss", 1, 260, 400, torch.Generator(device="cuda").manual_seed(1))[0] * scale
    h = z.zero_muon_create(z.make_muon_config(eps=eps), [(260, 400)])
    out = torch.empty_like(g)
    z.zero_muon_orthogonalize(h, [g], [out])
    close(out, ortho64(g, eps), "fp32")
    z.zero_muon_destroy(h)


def test_odd_addresses_through_the_workspace(z):  # noqa: F811
    """Arrays at addresses that are multiples of their element only."""
    import torch
    m, n = 265, 200
    want, got = matrices([(m, n, 1)], "fp16", 13)[0], matrices([(m, n, 1)], "fp16", 13)[0]
    for name in got:
        flat = torch.full((m * n + 2,), 5.0, device="cuda", dtype=got[name].dtype)
        flat[1:-1] = got[name].flatten()
        got[name] = flat[1:-1].view(1, m, n)
    h = z.zero_muon_create(z.make_muon_config(lr=1e-2), [(m, n)])
    try:
        for x in (want, got):
            z.zero_muon_step(h, z.make_muon_list([x]))
        for name in got:
            assert torch.equal(got[name], want[name]), name
            assert got[name]._base[0] == 5 and got[name]._base[-1] == 5
    finally:
        z.zero_muon_destroy(h)


@pytest.mark.parametrize("m,n", [(100, 60), (70, 900), (300, 200)])
def test_strides_past_32_bits(z, m, n):  # noqa: F811
    """Rows and matrices that lie more than 2^32 bytes and 2^31 numbers apart,
    one CTA, a cluster and the workspace."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(9)
    g = torch.randn(2, m, n, device="cuda", generator=gen).bfloat16()
    want = torch.empty_like(g)
    store = torch.empty(5_000_000_000, device="cuda", dtype=torch.bfloat16)
    h = z.zero_muon_create(z.make_muon_config(), [(m, n, 2)])
    try:
        z.zero_muon_orthogonalize(h, [g], [want])
        close(want, ortho64(g), "bf16")
        row = 4_700_000_000 // m
        for strides in ((2_400_000_000, n, 1), (n, row, 1)):     # matrices, then rows far apart
            far = store.as_strided((2, m, n), strides, 8)
            far.copy_(g)
            z.zero_muon_orthogonalize(h, [far], [far])
            close(far, ortho64(g), "bf16")
    finally:
        z.zero_muon_destroy(h)
        del store, far
        torch.cuda.empty_cache()


@pytest.mark.parametrize("kind", ["gauss", "signal", "rank1", "decay"])
@pytest.mark.parametrize("k,l", [(1, 3), (2, 2), (3, 12), (5, 6), (8, 8), (13, 40), (16, 17), (31, 31), (32, 40),
                                 (64, 64), (128, 130), (2, 3000), (130, 160)])
def test_accuracy_by_size(z, k, l, kind):  # noqa: F811
    """What zero_muon.h states.  With a shorter side of 32 or more the bound that
    test_muon_gpu.py derives from roundings that average out, for each matrix.
    Below, of few numbers, each of the fifteen roundings (2^-12 at most) may go
    the same way, times the same |b| + 2 |c|: 15 * 2^-12 * 8.84 = 3.2e-2; over
    many matrices they average out again, and the mean square has the first bound."""
    import torch
    b = max(4, min(500, 2_000_000 // (k * l)))
    g = spectrum(kind, b, k, l, torch.Generator(device="cuda").manual_seed(7 * k + l))
    h = z.zero_muon_create(z.make_muon_config(), [(k, l, b)])
    try:
        out = torch.empty_like(g)
        z.zero_muon_orthogonalize(h, [g], [out])
        ref = ortho64(g)
        off = (out.double() - ref).flatten(-2).norm(dim=-1) / ref.flatten(-2).norm(dim=-1)
        assert off.max() <= (4.8e-3 if k >= 32 else 3.2e-2), off.max()
        assert off.square().mean().sqrt() <= 4.8e-3
    finally:
        z.zero_muon_destroy(h)
