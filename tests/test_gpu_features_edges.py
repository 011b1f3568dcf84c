"""Feature-field operators where rows share an offset, temperatures are
extreme, rows are constant, sites outnumber the pairs by far, and a field's
lists or graphs change between calls.

u = 2^-24 is the most a float32 operation is off by, relative to its result; a
16-bit result is rounded once more, by half a step.
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

U = 2.0 ** -24
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def feat():
    from soft_voronoi_render_b200 import features
    return features


def rng(seed):
    return torch.Generator("cuda").manual_seed(seed)


def randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def teacher(g, T, V, M):
    """M distinct classes a row and their logits, one of them empty."""
    tid = (torch.randint(0, V, (T, 1), generator=g, device="cuda") + torch.arange(M, device="cuda") * (V // M)) % V
    tid = tid.int().contiguous()
    if M > 2:
        tid[:, 1] = -1
    return tid, randn(g, T, M).mul_(2.0)


@pytest.mark.parametrize("dt,step,offset", [("f32", 2.0 ** -8, 1000.0), ("f32", 2.0 ** -8, -30000.0),
                                            ("f16", 0.25, 500.0), ("bf16", 0.5, -100.0)])
@pytest.mark.parametrize("T,V,M", [(300, 19, 4), (65, 150, 8), (9, 1001, 16), (7, 5000, 8), (3, 40001, 32),
                                   (1, 300001, 64)])
def test_distill_of_rows_that_share_an_offset(T, V, M, dt, step, offset):
    """A softmax does not see what all logits of a row have in common: logits
    on a grid that holds both z and z + offset give the same bits, the
    teacher's too."""
    f, t = feat(), TYPES[dt]
    g = rng(V)
    z = (randn(g, T, V).mul_(2.0 / step).round() * step).clamp(-8.0, 8.0)
    tid, tl = teacher(g, T, V, M)
    tl = (tl * 256.0).round() / 256.0
    for tau in (1.0, 0.3):
        loss, dz = f.distill(z.to(t), tid, tl, tau)
        loss2, dz2 = f.distill((z + offset).to(t), tid, tl, tau)
        loss3, dz3 = f.distill(z.to(t), tid, tl + 1000.0, tau)
        assert torch.equal(loss, loss2) and torch.equal(dz, dz2)
        assert torch.equal(loss, loss3) and torch.equal(dz, dz3)
        assert bool(torch.isfinite(loss).all()) and bool(torch.isfinite(dz).all())


@pytest.mark.parametrize("offset", [0.0, 1000.0, -20000.0])
@pytest.mark.parametrize("T,V,M", [(300, 19, 4), (65, 150, 8), (9, 1001, 16), (7, 5000, 8), (3, 40001, 32),
                                   (1, 300001, 64)])
def test_distill_error_goes_by_the_distance_from_the_maximum(T, V, M, offset):
    """Against 64 bits, with a tolerance in which the logits' size has no part.

    An argument (z - max) k takes a subtraction and a product, and k (log2(e)
    rounded, divided by tau) is off by 2 u: 4 u of its size, d in natural
    units; the exponential adds 2 ulp, 4 u.  A sum of V exponentials adds its
    depth, and a running maximum rescales it: by (4 span + 4) u for each
    change, whose distances add up to the row's span; V / 8192 + 4 at most.
    """
    f = feat()
    g = rng(V + 1)
    z = randn(g, T, V).mul_(2.0) + offset
    tid, tl = teacher(g, T, V, M)
    tl = tl + offset / 4
    rw = torch.rand(T, generator=g, device="cuda") + 0.5
    for tau in (1.0, 0.3):
        loss, dz = f.distill(z, tid, tl, tau, rw)
        zd, td, w = z.double() / tau, tl.double() / tau, rw.double()
        ok = tid >= 0
        at = tid.clamp(min=0).long()
        td = torch.where(ok, td, -torch.inf)
        lq, lp = torch.log_softmax(td, 1), torch.log_softmax(zd, 1)
        q, p = lq.exp(), lp.exp()
        terms = torch.where(ok, q * (lq - lp.gather(1, at)), 0.0)
        mass = torch.zeros_like(p).scatter_add_(1, at, torch.where(ok, q, 0.0))
        rl, rz = w * tau * tau * terms.sum(1), (w * tau)[:, None] * (p - mass)
        d = zd.max(1, keepdim=True).values - zd
        span = d.max(1, keepdim=True).values
        tspan = torch.where(ok, td.max(1, keepdim=True).values - td, 0.0).max(1, keepdim=True).values
        e_sum = (8 * span + 4 * (V / 8192 + 4) + 4 + min(V + 1, V / 32 + 24)) * U
        e_q = (8 * tspan + 8 + M) * U
        size = span + tspan + float(np.log(V) + np.log(M))
        slack = (w * tau * tau)[:, None] * (e_sum + e_q + size * ((M + 16) * U + e_q))
        assert bool(((loss.double() - rl).abs() <= slack[:, 0]).all())
        slack = (w * tau)[:, None] * (p * ((4 * d + 8) * U + e_sum) + mass * (e_q + (M + 4) * U)) + 3 * U * rz.abs()
        assert bool(((dz.double() - rz).abs() <= slack + 1e-37).all())


@pytest.mark.parametrize("V", [20, 150, 1001, 40001, 300001])
@pytest.mark.parametrize("tau", [1e-30, 1e-12, 1e-6, 1e-3])
def test_distill_at_sharp_temperatures(V, tau):
    """Logits at least 1 apart and a small tau: both softmaxes are one class,
    the loss is tau (max - z of the teacher's class), up to the roundings of
    its five factors and of k."""
    f = feat()
    g = rng(V)
    T, M = 3, 5
    z = torch.rand((T, V), generator=g, device="cuda").mul_(50.0)
    best = torch.randint(0, V - 1, (T,), generator=g, device="cuda")
    z[torch.arange(T), best] = 60.3
    tid = ((best[:, None] + 1 + torch.arange(M, device="cuda")) % V).int()
    tl = torch.tensor([7.7, 3.0, -2.0, 5.1, 0.0], device="cuda").repeat(T, 1)
    loss, dz = f.distill(z, tid, tl, tau)
    ref = tau * (z.double().max(1).values - z.gather(1, tid[:, :1].long())[:, 0].double())
    # (z - max) k, log2 and LN2, tau twice: 16 u covers them
    assert bool(((loss.double() - ref).abs() <= 16 * U * ref).all()), (loss, ref)
    want = torch.zeros((T, V), dtype=torch.float64, device="cuda")
    want[torch.arange(T), best] = tau
    want[torch.arange(T), tid[:, 0].long()] = -tau
    assert bool(((dz.double() - want).abs() <= 8 * U * want.abs()).all())


def test_distill_at_flat_temperatures():
    """tau^2 beyond float32: a divergence of 0 stays 0, and the gradient is
    tau (p - q) as ever."""
    f = feat()
    one = torch.zeros((2, 1), device="cuda")
    loss, dz = f.distill(one, one.int(), one, 1e30)
    assert loss.tolist() == [0.0, 0.0] and dz.tolist() == [[0.0], [0.0]]
    z = randn(rng(3), 4, 64)
    tid, tl = teacher(rng(4), 4, 64, 8)
    tid[:, 1] = 0
    _, dz = f.distill(z, tid, tl, 1e20)
    mass = torch.zeros((4, 64), dtype=torch.float64, device="cuda").scatter_add_(1, tid.long(), torch.full((4, 8), 0.125, device="cuda").double())
    ref = 1e20 * (1.0 / 64 - mass)
    # exponentials of 2 ulp, their sum, its reciprocal, the products
    assert bool(((dz.double() - ref).abs() <= 1e20 * (1.0 / 64 + mass) * 90 * U).all())


@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("T,V,M", [(6, 19, 4), (6, 150, 8), (6, 1001, 16), (6, 5000, 8), (6, 40001, 32)])
@pytest.mark.parametrize("tau", [0.5, 1.0, 2.0])
def test_distill_of_logits_masked_by_the_lowest_value(T, V, M, dt, tau):
    """A mask of the type's lowest finite value in place of -infinity: on all
    of a row, on the teacher's classes too, on all but one class.  The loss
    then is rw tau q (max - lowest), finite; tolerances as above."""
    f, t = feat(), TYPES[dt]
    low = torch.finfo(t).min
    g = rng(V + M)
    z = randn(g, T, V).mul_(2.0).to(t)
    tid = torch.arange(M, device="cuda").int().repeat(T, 1)
    tl = randn(g, T, M)
    z[0] = low
    z[1, :V // 2] = low       # some of the teacher's classes, or all
    z[2, 1:] = low
    z[3, M:] = low            # none of them
    z[4, M - 1] = low
    rw = torch.tensor([1.0, 0.5, 0.25, 1.0, 0.25, 2.0], device="cuda")
    loss, dz = f.distill(z, tid, tl, tau, rw)
    zd, td, w = z.double() / tau, tl.double() / tau, rw.double()
    lq, lp = torch.log_softmax(td, 1), torch.log_softmax(zd, 1)
    q, p = lq.exp(), lp.exp()
    rl = w * tau * tau * (q * (lq - lp.gather(1, tid.long()))).sum(1)
    mass = torch.zeros_like(p).scatter_add_(1, tid.long(), q)
    rz = (w * tau)[:, None] * (p - mass)
    d = zd.max(1, keepdim=True).values - zd
    span = torch.where(p > 0, d, 0.0).max(1, keepdim=True).values  # beyond it exponentials are 0 on both sides
    tspan = (td.max(1, keepdim=True).values - td).max(1, keepdim=True).values
    e_sum = (8 * span + 4 * (V / 8192 + 4) + 4 + min(V + 1, V / 32 + 24)) * U
    e_q = (8 * tspan + 8 + M) * U
    far = d.gather(1, tid.long()).max(1, keepdim=True).values
    size = span + far + tspan + float(np.log(V) + np.log(M))
    slack = (w * tau * tau)[:, None] * (e_sum + e_q + size * ((M + 16) * U + e_q))
    # Row 1 with few classes has only masked teacher's classes: at rw tau = 1
    # (tau 2) its loss is max - lowest, the largest float, and a q above 1 by
    # its rounding gives infinity: rl + slack > max, so that lies within the
    # tolerance.  Every other loss has to be finite.
    fits = rl + slack[:, 0] < torch.finfo(torch.float32).max
    assert bool(torch.isfinite(loss[fits]).all()) and int((~fits).sum()) <= (tau == 2.0), (loss, rl)
    assert bool(((loss.double() - rl).abs() <= slack[:, 0])[fits].all())
    assert bool((loss.double() >= rl - slack[:, 0]).all())
    half = torch.finfo(t).eps / 2 if t != torch.float32 else 0.0
    slack = (w * tau)[:, None] * (p * ((4 * torch.where(p > 0, d, 0.0) + 8) * U + e_sum) + mass * (e_q + (M + 4) * U)) \
        + 3 * U * rz.abs()
    slack = slack + half * (rz.abs() + slack) + (2.0 ** -25 if t == torch.float16 else 0.0) + 1e-37
    assert bool(((dz.double() - rz).abs() <= slack).all())


def small_field(D=6, seed=2):
    import synth
    from soft_voronoi_render_b200 import Sad
    H, W, N = 24, 40, 60
    s = Sad(H, W, N, seed=3)
    s.set_sites(synth.uniform_sites(H, W, N, 4))
    s.refresh(2)
    field = feat().FeatureField(s, D, seed=seed)
    field.features.mul_(100.0)
    g = rng(9)
    tid = torch.rand((H * W, D), generator=g, device="cuda").topk(3, 1).indices.int().contiguous()
    return s, field, tid, randn(g, H * W, 3)


def test_gradients_after_lists_were_taken_without_a_route():
    """update_lists(route=False) leaves the routing to the next gradient,
    which is that of the lists as they are."""
    import synth
    s, field, tid, tl = small_field()
    field.update_lists(route=False)
    field.loss_and_grads(tid, tl)
    first = field.grad_features.clone()
    field.update_lists()
    field.loss_and_grads(tid, tl)
    assert torch.equal(field.grad_features, first) and bool(first.any())
    s.set_sites(synth.uniform_sites(24, 40, 60, 11))  # other places, other lists
    s.refresh(2)
    field.update_lists(route=False)
    field.loss_and_grads(tid, tl)
    got = field.grad_features.clone()
    field.update_lists()
    field.loss_and_grads(tid, tl)
    assert torch.equal(got, field.grad_features) and not torch.equal(got, first)
    # a capture routes too, as often as it is replayed, and says nothing of
    # what has run
    s.set_sites(synth.uniform_sites(24, 40, 60, 12))
    s.refresh(2)
    field.update_lists(route=False)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        field.loss_and_grads(tid, tl)
    field.loss_and_grads(tid, tl)
    eager = field.grad_features.clone()
    field.grad_features.zero_()
    graph.replay()
    assert torch.equal(eager, field.grad_features) and not torch.equal(eager, got)
    # lists that a graph takes: each of its replays is seen
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        field.update_lists(route=False)
    for seed in (13, 14):
        s.set_sites(synth.uniform_sites(24, 40, 60, seed))
        s.refresh(2)
        graph.replay()
        field.loss_and_grads(tid, tl)
        got = field.grad_features.clone()
        field.update_lists()
        field.loss_and_grads(tid, tl)
        assert torch.equal(got, field.grad_features) and not torch.equal(got, eager)
    s.close()


@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("D", [3, 19, 33, 64, 250, 516, 1000, 2500, 5000, 5001, 12000, 16384])
def test_layer_norm_of_constant_rows(D, dt):
    """Rows of equal elements have that mean, and give beta, whatever bits the
    element has."""
    f, t = feat(), TYPES[dt]
    g = rng(D)
    c = torch.cat([torch.tensor([0.1, 1000.3, -3.7e-4, 65000.0], device="cuda"), randn(g, 60) * 100.0]).to(t)
    beta = randn(g, D).to(t).float()
    for x in (c[:, None].repeat(1, D), torch.cat([c] * 12)[:, None].repeat(1, D)):
        y, mean, rstd = f.layer_norm(x, None, beta, 1e-5)
        assert torch.equal(mean, x[:, 0].float())
        assert torch.equal(y, beta.to(t).expand_as(y))
        # eps as given, and rsqrtf within 2 ulp
        assert bool(((rstd.double() * 1e-5 ** 0.5 - 1.0).abs() <= 5 * U).all())


@pytest.mark.parametrize("D", [19, 64, 250, 1000, 4096, 5001, 16384])
def test_layer_norm_mean_goes_by_the_spread(D):
    """Rows at 1000 +- 0.1.  The mean is corrected by the mean of the
    deviations from its first value m1: it is off by its own rounding, u |m|,
    and by the correction's error, depth + 4 roundings of the deviations."""
    f = feat()
    x = 1000.0 + 0.1 * randn(rng(D), 700, D)
    y, mean, rstd = f.layer_norm(x, None, None, 1e-6)
    xd = x.double()
    m = xd.mean(1)
    depth = D + 1 if D < 1024 else D // 32 + 16
    spread = (xd - m[:, None]).abs().mean(1)
    first = (depth + 2) * U * xd.abs().mean(1)
    em = 1.01 * U * m.abs() + (depth + 4) * U * (spread + first)
    assert bool(((mean.double() - m).abs() <= em).all())
    var = ((xd - m[:, None]) ** 2).mean(1) + 1e-6
    rs = var.rsqrt()
    # the variance about m1, less the square of the correction: depth + 6
    # roundings of a sum of at most var + first^2
    ev = (depth + 6) * U * (var + 2 * first ** 2) / (2 * var) + 4 * U
    assert bool(((rstd.double() / rs - 1.0).abs() <= ev).all())
    h = (xd - m[:, None]) * rs[:, None]
    assert bool(((y.double() - h).abs() <= (em * rs)[:, None] + h.abs() * (ev[:, None] + 4 * U)).all())


@pytest.mark.parametrize("T,E,D,dt", [(1, 1 << 21, 1, "f32"), (32, 131072, 32, "bf16"), (1000, 131072, 200, "f32"),
                                      (5, 1 << 20, 77, "f16")])
def test_blend_backward_of_few_rows_over_many_sites(T, E, D, dt):
    """Sites without pairs cost no more than their zeros and a search: the
    sums of few rows are right, and their time goes by the pairs."""
    f, t = feat(), TYPES[dt]
    g = rng(T)
    ids = torch.randint(0, E, (T, 8), generator=g, device="cuda").int()
    ids[0, 0], ids[0, 7] = 0, E - 1
    w = torch.rand((T, 8), generator=g, device="cuda")
    F, dout = torch.zeros((E, D), dtype=t, device="cuda"), randn(g, T, D).to(t)
    r = f.Route(T, 8, E).build(ids)
    dF, _ = f.blend_backward(dout, F, ids, w, r)
    flat = ids.reshape(-1).long()
    s = (dout.double()[:, None] * w.double()[..., None]).reshape(-1, D)
    at, where = flat.unique(return_inverse=True)
    ref = torch.zeros((at.numel(), D), dtype=torch.float64, device="cuda").index_add_(0, where, s)
    big = torch.zeros_like(ref).index_add_(0, where, s.abs())
    count = torch.zeros(at.numel(), device="cuda").index_add_(0, where, torch.ones(T * 8, device="cuda"))
    assert bool(((dF[at].double() - ref).abs() <= ((count + 1)[:, None] * U) * big).all())
    dF[at] = 0.0
    assert not bool(dF.any())
    times = []
    for _ in range(5):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        f.blend_backward(dout, F, ids, w, r, dF=dF)
        b.record()
        torch.cuda.synchronize()
        times.append(a.elapsed_time(b))
    # a site's turn one by one is a round trip to the L2, 0.3 us or more: 600
    # ms for 2^21 of them, 20 for 131,072 split over two chunks.  Clearing dF
    # takes up to 0.06 ms.
    assert min(times) < 2.0, times


def test_gradients_of_a_field_are_one_set_of_buffers():
    """Captured steps and eager ones fill the same three buffers: after a
    replay all of them are the replayed step's."""
    s, field, tid, tl = small_field()
    assert field.grad_gamma.shape == field.grad_beta.shape == (field.D,)
    field.update_lists()
    other = -tl
    grads = lambda: [v.clone() for v in (field.grad_features, field.grad_gamma, field.grad_beta)]
    field.loss_and_grads(tid, tl)
    want = grads()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        field.loss_and_grads(tid, tl)
    field.loss_and_grads(tid, other)
    assert not torch.equal(field.grad_gamma, want[1])
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(grads(), want))
    s.close()


def test_layer_norm_backward_into_given_sums():
    f = feat()
    from soft_voronoi_render_b200 import SadError
    for T, D in ((1, 64), (500, 19), (300, 4096), (0, 8)):
        g = rng(D)
        x, dy, gamma = randn(g, T, D), randn(g, T, D), randn(g, D)
        _, mean, rstd = f.layer_norm(x, gamma)
        _, dg, db = f.layer_norm_backward(dy, x, gamma, mean, rstd)
        a, b = torch.full((D,), 7.0, device="cuda"), torch.full((D,), 7.0, device="cuda")
        _, dg2, db2 = f.layer_norm_backward(dy, x, gamma, mean, rstd, dgamma=a, dbeta=b)
        assert dg2 is a and db2 is b and torch.equal(a, dg) and torch.equal(b, db)
    for kw in (dict(dgamma=a), dict(dgamma=a, dbeta=b, want_affine=False), dict(dgamma=a[:4], dbeta=b[:4]),
               dict(dgamma=a.half(), dbeta=b)):
        with pytest.raises(SadError):
            f.layer_norm_backward(dy, x, gamma, mean, rstd, **kw)
