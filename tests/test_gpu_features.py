"""Feature-field operators (route, dispatch, combine, blend, layer norm,
distill) against their definitions in 64 bits.

Tolerances.  u = 2^-24 is the most a float32 operation is off by, relative to
its result.  A float32 sum of n products taken in any order is off by at most
(n + 1) u times the sum of the terms' absolute values; sums that the kernels
split over lanes are held to their depth, n / 32 + 16, where that is smaller
(at least 32 lanes share such a sum, and joining takes at most 16 more
additions).  A result kept in a 16-bit type is rounded once: half a step,
finfo(t).eps / 2 relative, and in binary16 half of its smallest step, 2^-25,
below the normal range.
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


def randn(g, *shape, dtype=torch.float32):
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def close(got, ref, slack):
    """got within slack (float32 errors, a tensor or a number) of ref, plus
    the rounding to got's type."""
    t = got.dtype
    half = torch.finfo(t).eps / 2 if t != torch.float32 else 0.0
    tol = slack + half * (ref.abs() + slack) + (2.0 ** -25 if t == torch.float16 else 0.0) + 1e-37
    err = (got.double() - ref).abs()
    assert bool(torch.isfinite(got).all())
    assert bool((err <= tol).all()), float((err - tol).max())


def strided(x, pad, shift):
    """The same rows with `pad` more elements between them, starting `shift`
    elements into the buffer (shift 1: no 16-byte alignment)."""
    T, D = x.shape
    buf = torch.full((T * (D + pad) + shift + 8,), float("nan"), dtype=x.dtype, device=x.device)
    v = buf[shift:shift + T * (D + pad)].view(T, D + pad)[:, :D]
    v.copy_(x)
    return v


def make_ids(g, T, K, E, drop=0.1):
    ids = torch.randint(0, E, (T, K), generator=g, device="cuda")
    u = torch.rand((T, K), generator=g, device="cuda")
    wild = torch.tensor([-1, -2 ** 31, E, 2 ** 31 - 1], device="cuda")[
        torch.randint(0, 4, (T, K), generator=g, device="cuda")]
    return torch.where(u < drop, wild, ids).int().contiguous()


def ref_route(ids, E):
    flat = ids.cpu().numpy().reshape(-1).astype(np.int64)
    key = np.where((flat >= 0) & (flat < E), flat, E)
    perm = np.argsort(key, kind="stable")
    m = int((key < E).sum())
    order = np.full(flat.size, -1, dtype=np.int32)
    order[:m] = perm[:m]
    place = np.full(flat.size, -1, dtype=np.int32)
    place[perm[:m]] = np.arange(m)
    offsets = np.searchsorted(key[perm], np.arange(E + 1), side="left").astype(np.int32)
    return offsets, order, place.reshape(tuple(ids.shape))


ROUTES = [(1, 1, 1), (1, 8, 64), (1, 8, 100000), (3, 5, 2), (33, 1, 7), (128, 8, 1024), (129, 8, 255), (1000, 2, 3),
          (1024, 8, 1023), (4097, 3, 1024), (777, 8, 5000), (20000, 8, 4), (30011, 7, 131072), (65536, 8, 1 << 20),
          (300, 8, (1 << 30) - 1 >> 9), (200001, 8, 50000), (5000, 8, 1 << 21)]


@pytest.mark.parametrize("T,K,E", ROUTES)
@pytest.mark.parametrize("drop", [0.0, 0.3, 1.0])
def test_route(T, K, E, drop):
    g = rng(T + K + E)
    ids = make_ids(g, T, K, E, drop)
    r = feat().Route(T, K, E)
    for _ in range(2):  # a second build sees nothing of the first
        r.build(ids)
        for got, want in zip((r.offsets, r.order, r.place), ref_route(ids, E)):
            assert np.array_equal(got.cpu().numpy(), want)
        ids = make_ids(g, T, K, E, drop)


def test_route_one_expert_takes_all_and_sorted_input():
    T, K, E = 50000, 8, 4096
    for ids in (torch.full((T, K), 77, dtype=torch.int32, device="cuda"),
                (torch.arange(T * K, device="cuda") // 100).int().view(T, K).clamp(max=E - 1),
                (E - 1 - torch.arange(T * K, device="cuda") // 100 % E).int().view(T, K)):
        ids = ids.contiguous()
        r = feat().Route(T, K, E).build(ids)
        for got, want in zip((r.offsets, r.order, r.place), ref_route(ids, E)):
            assert np.array_equal(got.cpu().numpy(), want)


# T, K, D, E, pad, shift
ROWS = [(1, 1, 1, 1, 0, 0), (1, 8, 1024, 64, 0, 0), (5, 3, 7, 4, 2, 1), (37, 8, 64, 16, 0, 0), (64, 2, 203, 5, 0, 0),
        (33, 4, 40, 9, 8, 0), (17, 8, 129, 300, 3, 0), (9, 5, 8, 6, 0, 1), (130, 8, 16, 40, 0, 0),
        (70, 7, 4, 11, 4, 0), (12, 6, 2056, 8, 0, 0), (2, 8, 5001, 3, 0, 0), (40, 8, 520, 12, 0, 8)]


@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("T,K,D,E,pad,shift", ROWS)
@pytest.mark.parametrize("weighted", [True, False])
def test_exchange(T, K, D, E, pad, shift, dt, weighted):
    f, t = feat(), TYPES[dt]
    g = rng(T * D + K)
    ids = make_ids(g, T, K, E, 0.2 if T > 1 else 0.0)
    w = torch.rand((T, K), generator=g, device="cuda") if weighted else None
    if weighted:
        bad = (ids < 0) | (ids >= E)
        w[bad] = float("nan")  # not read
    r = f.Route(T, K, E).build(ids)
    n, m = T * K, int(r.offsets[-1])
    x = strided(randn(g, T, D, dtype=t), pad, shift)
    y = strided(randn(g, n, D, dtype=t), pad, shift)
    y[m:] = float("nan")  # no pair's rows: not read
    valid = r.place >= 0
    at = r.place.clamp(min=0).long()
    wd = torch.where(valid, w.double() if weighted else 1.0, 0.0)
    yd = torch.where(valid[..., None], y[at].double(), 0.0)                   # T K D
    xd = x.double()
    sums = D + 1 if D < 1024 else D // 32 + 16

    # dispatch: one product, one rounding; rows behind the last pair stay
    out = strided(torch.full((n, D), 7.0, device="cuda", dtype=t), pad, shift)
    assert r.dispatch(x, w, out=out) is out
    want = torch.full((n, D), 7.0, dtype=torch.float64, device="cuda")
    want[at[valid]] = (xd[:, None] * wd[..., None])[valid]
    close(out, want, 2 * U * want.abs())
    assert bool((out[m:] == 7.0).all())

    # combine
    ref = (yd * wd[..., None]).sum(1)
    c = r.combine(y, w)
    close(c, ref, (K + 1) * U * (yd * wd[..., None]).abs().sum(1))
    assert bool((c[~valid.any(1)] == 0).all())

    # gradients of both
    dref = (yd * xd[:, None]).sum(2) * valid
    dslack = sums * U * (yd * xd[:, None]).abs().sum(2)
    dx, dw = r.dispatch_backward(y, x, w)
    assert torch.equal(dx, c)
    close(dw, dref, dslack)
    assert bool((dw[~valid] == 0).all())
    dy = torch.full((n, D), 7.0, device="cuda", dtype=t)
    dy2, dw2 = r.combine_backward(x, y, w, dy=dy)
    assert dy2 is dy and torch.equal(dy, out)
    close(dw2, dref, dslack)
    # without the weights' gradient
    assert r.dispatch_backward(y, None, w)[1] is None
    assert torch.equal(r.dispatch_backward(y, None, w)[0], c)
    dy.fill_(7.0)
    assert torch.equal(r.combine_backward(x, None, w, dy=dy)[0], out)


BLENDS = ROWS + [(3000, 8, 24, 1, 0, 0), (2000, 8, 32, 700, 0, 0), (5000, 8, 3, 37, 0, 0), (1500, 4, 96, 2, 0, 0),
                 (40000, 8, 16, 3, 0, 0), (40, 8, 64, 100000, 0, 0), (6001, 8, 64, 5, 0, 0), (7, 8, 12, 33, 0, 0)]


@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("T,K,D,E,pad,shift", BLENDS)
def test_blend(T, K, D, E, pad, shift, dt):
    f, t = feat(), TYPES[dt]
    g = rng(T + D + K)
    ids = make_ids(g, T, K, E, 0.2 if T > 1 else 0.0)
    valid = (ids >= 0) & (ids < E)
    w = torch.rand((T, K), generator=g, device="cuda")
    w[~valid] = float("nan")
    F = strided(randn(g, E, D, dtype=t), pad, shift)
    dout = strided(randn(g, T, D, dtype=t), pad, shift)
    at = torch.where(valid, ids, 0).long()
    wd = torch.where(valid, w.double(), 0.0)
    Fd = F.double()
    out = f.blend(F, ids, w)
    ref, big = torch.zeros((T, D), dtype=torch.float64, device="cuda"), torch.zeros((T, D), device="cuda").double()
    dref = torch.empty((T, K), dtype=torch.float64, device="cuda")
    dbig = torch.empty_like(dref)
    sref, sbig = torch.zeros((E, D), device="cuda").double(), torch.zeros((E, D), device="cuda").double()
    for k in range(K):
        v = Fd[at[:, k]] * wd[:, k, None]
        ref, big = ref + v, big + v.abs()
        p = Fd[at[:, k]] * dout.double() * valid[:, k, None]
        dref[:, k], dbig[:, k] = p.sum(1), p.abs().sum(1)
        s = dout.double() * wd[:, k, None]
        sref.index_add_(0, at[:, k], s)
        sbig.index_add_(0, at[:, k], s.abs())
    close(out, ref, (K + 1) * U * big)
    assert bool((out[~valid.any(1)] == 0).all())
    r = f.Route(T, K, E).build(ids)
    dF, dw = f.blend_backward(dout, F, ids, w, r)
    close(dw, dref, (D + 1 if D < 1024 else D // 32 + 16) * U * dbig)
    assert bool((dw[~valid] == 0).all())
    count = (r.offsets[1:] - r.offsets[:-1])[:, None].double()
    close(dF, sref, (count + 1) * U * sbig)
    assert bool((dF[count[:, 0] == 0] == 0).all())
    # the same bits again; without a route only the weights' gradient
    dF2, dw2 = f.blend_backward(dout, F, ids, w, r)
    assert torch.equal(dF, dF2) and torch.equal(dw, dw2)
    none, dw3 = f.blend_backward(dout, F, ids, w)
    assert none is None and torch.equal(dw, dw3)


NORMS = [(1, 1, 0, 0), (1, 2, 0, 0), (3, 7, 2, 1), (5, 64, 0, 0), (1000, 64, 0, 0), (37, 100, 4, 0), (129, 33, 0, 0),
         (64, 256, 8, 8), (300, 1000, 0, 0), (2, 1024, 0, 0), (17, 4096, 0, 0), (9, 5000, 0, 1), (3, 16384, 0, 0),
         (2, 16381, 0, 0), (5003, 16, 0, 0), (20011, 8, 0, 0), (700, 2048, 0, 0), (33, 516, 0, 0), (40, 8200, 0, 0)]


@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("T,D,pad,shift", NORMS)
@pytest.mark.parametrize("affine", [True, False])
def test_layer_norm(T, D, pad, shift, dt, affine):
    f, t = feat(), TYPES[dt]
    g = rng(T + D)
    x = strided((randn(g, T, D) * 1.5 + 0.5 * randn(g, T, 1)).to(t), pad, shift)
    gamma = 1.0 + 0.2 * randn(g, D) if affine else None
    beta = 0.2 * randn(g, D) if affine else None
    y, mean, rstd = f.layer_norm(x, gamma, beta, 1e-3)
    xd = x.double()
    gd = gamma.double() if affine else torch.ones(D, device="cuda").double()
    bd = beta.double() if affine else torch.zeros(D, device="cuda").double()
    m = xd.mean(1, keepdim=True)
    var = ((xd - m) ** 2).mean(1, keepdim=True)
    rs = 1.0 / torch.sqrt(var + 1e-3)
    h = (xd - m) * rs
    depth = D + 1 if D < 1024 else D // 32 + 16
    # the mean's error em; each deviation then is off by em + u |x - m| and
    # their squares' mean by em^2 (the deviations cancel in the cross term up
    # to their own rounding) + (depth + 3) u var; 1 / sqrt adds 3 u
    em = (depth + 2) * U * xd.abs().mean(1, keepdim=True)
    erel = (em ** 2 + 2 * em * U * depth * (xd - m).abs().mean(1, keepdim=True) + (depth + 4) * U * var) \
        / (2 * (var + 1e-3)) + 4 * U
    close(mean, m[:, 0], em[:, 0])
    close(rstd, rs[:, 0], (erel * rs)[:, 0])
    eh = em * rs + h.abs() * (erel + 2 * U)
    close(y, h * gd + bd, eh * gd.abs() + 3 * U * ((h * gd).abs() + bd.abs()))
    # in place: the same bits (rows laid out alike: sums may be shared out
    # over the lanes by the rows' alignment)
    x2 = strided(x, pad, shift)
    y2, _, _ = f.layer_norm(x2, gamma, beta, 1e-3, out=x2)
    assert y2 is x2 and torch.equal(y2, y)

    dy = strided(randn(g, T, D, dtype=t), pad, shift)
    dx, dg, db = f.layer_norm_backward(dy, x, gamma, mean, rstd)
    # from the saved statistics, as given: their own errors are the forward's
    m, rs = mean.double()[:, None], rstd.double()[:, None]
    h = (xd - m) * rs
    a = dy.double() * gd
    ma, mb = a.mean(1, keepdim=True), (a * h).mean(1, keepdim=True)
    ref = rs * (a - ma - h * mb)
    eh = 3 * U * (xd.abs() + m.abs()) * rs
    ema = (depth + 2) * U * a.abs().mean(1, keepdim=True)
    emb = (depth + 4) * U * (a * h).abs().mean(1, keepdim=True) + (a.abs() * eh).mean(1, keepdim=True)
    slack = rs * (ema + h.abs() * emb + eh * mb.abs() + 5 * U * (a.abs() + ma.abs() + (h * mb).abs()))
    close(dx, ref, slack)
    dyd = dy.double()
    close(dg, (dyd * h).sum(0), (T + 4) * U * (dyd * h).abs().sum(0) + (dyd.abs() * eh).sum(0))
    close(db, dyd.sum(0), (T + 1) * U * dyd.abs().sum(0))
    # dx in the place of dy, sums not wanted, the same bits
    dy2 = strided(dy, pad, shift)
    dx2, n1, n2 = f.layer_norm_backward(dy2, x, gamma, mean, rstd, want_affine=False, dx=dy2)
    assert dx2 is dy2 and n1 is None and n2 is None and torch.equal(dx2, dx)
    dy2 = strided(dy, pad, shift)
    dx3, dg3, db3 = f.layer_norm_backward(dy2, x, gamma, mean, rstd, dx=dy2)
    assert torch.equal(dx3, dx) and torch.equal(dg3, dg) and torch.equal(db3, db)


def test_layer_norm_far_from_zero_and_constant_rows():
    """The variance is taken about the mean: rows at 1000 +- 0.1 keep it, and
    a constant row gives beta."""
    f = feat()
    g = rng(3)
    for D in (64, 1000, 4096):
        x = 1000.0 + 0.1 * randn(g, 50, D)
        x[7] = -3.25
        beta = randn(g, D)
        y, mean, rstd = f.layer_norm(x, None, beta, 1e-6)
        xd = x.double()
        m = xd.mean(1, keepdim=True)
        rs = 1.0 / torch.sqrt(((xd - m) ** 2).mean(1, keepdim=True) + 1e-6)
        # the mean is off by at most (D / 32 + 18) u 1000, the deviations by as much
        e = (D / 32 + 18) * U * 1000.0
        live = torch.arange(50, device="cuda") != 7
        close(rstd[live], rs[live, 0], rs[live, 0] * ((e * rs[live, 0]) ** 2 + (D / 32 + 20) * U))
        close(y[live], ((xd - m) * rs + beta.double())[live],
              (e * rs + ((xd - m) * rs).abs() * ((e * rs) ** 2 + (D / 32 + 24) * U) + 3 * U * 8)[live])
        assert torch.equal(y[7], beta)


DISTILLS = [(1, 1, 1, 0, 0), (1, 2, 2, 0, 0), (3, 5, 3, 2, 1), (200, 19, 4, 0, 0), (65, 150, 8, 0, 0),
            (33, 152, 8, 0, 0), (130, 64, 64, 0, 0), (40, 1000, 32, 24, 8), (37, 1023, 16, 0, 0), (5, 8192, 128, 0, 0),
            (3, 10007, 64, 0, 1), (2, 50001, 32, 0, 0), (1, 128000, 32, 0, 0), (1, 300001, 128, 0, 0),
            (300, 5000, 8, 0, 0), (9, 2050, 5, 6, 2), (1, 1300000, 7, 0, 0), (16, 70000, 3, 0, 0)]


def ref_distill(z, tid, tl, tau, rw):
    """(loss, dz, sum of the terms' absolute values) in 64 bits."""
    T, V = z.shape
    zd, tld, rwd = z.double() / tau, tl.double() / tau, rw.double()
    ok = (tid >= 0) & (tid < V) & (tl != -torch.inf)
    at = torch.where(ok, tid, 0).long()
    tld = torch.where(ok, tld, -torch.inf)
    q = torch.where(ok, torch.exp(tld - torch.logsumexp(tld, 1, keepdim=True)), 0.0)
    big = zd.max(1, keepdim=True).values
    live = ok.any(1) & (rwd != 0) & (big[:, 0] > -torch.inf)
    logp = zd - torch.logsumexp(zd, 1, keepdim=True)
    lq = torch.where(ok, tld - torch.logsumexp(tld, 1, keepdim=True), 0.0)
    terms = torch.where(q > 0, q * (lq - logp.gather(1, at)), 0.0)
    loss = torch.where(live, rwd * tau * tau * terms.sum(1), 0.0)
    p = logp.exp()
    dz = p.scatter_add(1, at, torch.where(ok, -q, 0.0))
    dz = torch.where(live[:, None], (rwd * tau)[:, None] * dz, 0.0)
    return loss, dz, p, live, ok, at, q


def check_distill(z, tid, tl, tau, rw, M, V, loss, dz):
    rl, rz, p, live, ok, at, q = ref_distill(z, tid, tl, tau, rw)
    zd = torch.where(z == -torch.inf, 0.0, z.double()) / tau
    span = (zd.abs().max(1).values * 2 + (torch.where(ok, tl.double(), 0.0) / tau).abs().max(1).values * 2)[:, None]
    # an exponential of an argument of size `span` is off by (span + 4) u
    # (its argument by two operations, the function by 2 ulp); the sum of V
    # of them adds its depth, the logarithms 2 ulp of at most ln V + span
    e = (3 * span + 8 + min(V + 1, V / 32 + 24)) * U
    es = e * (1 + 0 * rl[:, None])
    size = (np.log(V) + np.log(M) + span[:, 0] * 2 + 2)
    close(loss[live], rl[live], (rw.double().abs() * tau * tau * (es[:, 0] * 4 + (M + 8) * U * size))[live])
    assert bool((loss[~live] == 0).all())
    if dz is not None:
        mass = torch.zeros_like(p).scatter_add_(1, at, torch.where(ok, q, 0.0))
        slack = (rw.double().abs() * tau)[:, None] * ((p + mass) * (2 * es + (M + 6) * U)) + U * 2.0 ** -20
        close(dz[live], rz[live], slack[live])
        assert bool((dz[~live] == 0).all())


@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("T,V,M,pad,shift", DISTILLS)
@pytest.mark.parametrize("tau", [1.0, 2.5])
def test_distill(T, V, M, pad, shift, dt, tau):
    f, t = feat(), TYPES[dt]
    g = rng(V + M)
    z = strided(randn(g, T, V).mul_(2.0).to(t), pad, shift)
    tid = torch.randint(0, V, (T, M), generator=g, device="cuda")  # repeats among them
    u = torch.rand((T, M), generator=g, device="cuda")
    tid = torch.where(u < 0.1, -1, torch.where(u < 0.15, V, tid)).int().contiguous()
    tl = randn(g, T, M).mul_(2.0)
    tl[(tid < 0) | (tid >= V)] = float("nan")  # not read
    if M > 2:
        tl[:, 2] = -torch.inf
    rw = torch.rand(T, generator=g, device="cuda") + 0.5
    if T > 2:
        rw[1] = 0.0
        z[1] = float("nan")  # a row of no weight may hold anything
        tid[2] = -1          # no teacher
    if T > 4:
        z[3] = -torch.inf    # no student
        z[4, V // 2:] = -torch.inf  # a masked vocabulary
        tid[4] = torch.where(tid[4] < V // 2, tid[4], 0)
        tid[4] = torch.where(tid[4] < 0, 0, tid[4])
        tl[4] = torch.where(torch.isfinite(tl[4]), tl[4], -1.0)
    loss, dz = f.distill(z, tid, tl, tau, rw)
    zz = z.clone()
    if T > 2:
        zz[1] = 0.0
    check_distill(zz, tid, tl, tau, rw, M, V, loss, dz)
    # loss alone, and the gradient in the logits' place: the same bits
    alone, none = f.distill(z, tid, tl, tau, rw, want_grad=False)
    assert none is None and torch.equal(alone, loss)
    z2 = strided(z, pad, shift)
    _, same = f.distill(z2, tid, tl, tau, rw, dlogits=z2)
    assert same is z2 and torch.equal(same, dz)
    ones, dz1 = f.distill(z, tid, tl, tau)
    keep = rw == rw if T <= 2 else torch.arange(T, device="cuda") != 1
    check_distill(zz[keep], tid[keep], tl[keep], tau, torch.ones_like(rw[keep]), M, V, ones[keep], dz1[keep])


@pytest.mark.parametrize("V", [50, 3001, 40000, 400000])
def test_distill_infinities_and_nan(V):
    f = feat()
    z = randn(rng(1), 6, V)
    tid = torch.tensor([[0, 3]], dtype=torch.int32, device="cuda").repeat(6, 1).contiguous()
    tl = torch.tensor([[1.0, 2.0]], device="cuda").repeat(6, 1).contiguous()
    z[0, 3] = -torch.inf          # the teacher wants a masked class: loss infinite, gradient finite
    z[1, V - 1] = float("nan")    # shows
    z[2] = float("nan")           # a row of NaN is no empty row
    tl[3] = -torch.inf            # no teacher
    z[4, :] = -torch.inf
    z[4, V - 2] = 3.0             # one class left
    loss, dz = f.distill(z, tid, tl)
    assert float(loss[0]) == np.inf and bool(torch.isfinite(dz[0]).all())
    assert bool(torch.isnan(loss[1])) and bool(torch.isnan(loss[2])) and bool(torch.isnan(dz[2]).all())
    assert float(loss[3]) == 0.0 and bool((dz[3] == 0).all())
    assert float(loss[4]) == np.inf and abs(float(dz[4, V - 2]) - 1.0) <= 4 * U
    assert bool(torch.isfinite(loss[5]))


def test_no_rows():
    f = feat()
    z = torch.empty((0, 8), device="cuda")
    i, w = torch.empty((0, 2), dtype=torch.int32, device="cuda"), torch.empty((0, 2), device="cuda")
    r = f.Route(0, 2, 5)
    r.offsets.fill_(9)
    r.build(i)
    assert r.offsets.tolist() == [0] * 6
    assert r.dispatch(z).shape == (0, 8) and r.combine(z, w).shape == (0, 8)
    assert r.combine_backward(z, z, w)[1].shape == (0, 2) and r.dispatch_backward(z, z, w)[0].shape == (0, 8)
    F = torch.ones((5, 8), device="cuda")
    assert f.blend(F, i, w).shape == (0, 8)
    dF, dw = f.blend_backward(z, F, i, w, r)
    assert bool((dF == 0).all()) and dw.shape == (0, 2)
    y, mean, rstd = f.layer_norm(z)
    assert y.shape == (0, 8)
    dx, dg, db = f.layer_norm_backward(z, z, None, mean, rstd)
    assert bool((dg == 0).all()) and bool((db == 0).all())
    loss, dz = f.distill(z, i, w)
    assert loss.shape == (0,) and dz.shape == (0, 8)


def _chain(f, route, F, ids, w, gamma, beta, tid, tl):
    """A feature field's step: blend, norm, distill and back."""
    out = f.blend(F, ids, w)
    y, mean, rstd = f.layer_norm(out, gamma, beta)
    loss, dz = f.distill(y, tid, tl, 2.0)
    dx, dg, db = f.layer_norm_backward(dz, out, gamma, mean, rstd)
    route.build(ids)
    dF, dw = f.blend_backward(dx, F, ids, w, route)
    return loss, dF, dw, dg, db


def _chain_inputs(g, T=500, E=40, D=21):
    ids = make_ids(g, T, 8, E)
    w = torch.rand((T, 8), generator=g, device="cuda")
    F, gamma, beta = randn(g, E, D), 1.0 + 0.1 * randn(g, D), 0.1 * randn(g, D)
    tid = torch.rand((T, D), generator=g, device="cuda").topk(5, 1).indices.int().contiguous()
    return F, ids, w, gamma, beta, tid, randn(g, T, 5)


def _chain_loss64(F, ids, w, gamma, beta, tid, tl, tau=2.0, eps=1e-5):
    E = F.shape[0]
    ok = (ids >= 0) & (ids < E)
    rows = F[torch.where(ok, ids, 0).long()] * torch.where(ok, w, torch.zeros_like(w))[..., None]
    x = rows.sum(1)
    xc = x - x.mean(1, keepdim=True)
    y = xc / torch.sqrt((xc * xc).mean(1, keepdim=True) + eps) * gamma + beta
    lq, lp = torch.log_softmax(tl / tau, 1), torch.log_softmax(y / tau, 1)
    return tau * tau * (lq.exp() * (lq - lp.gather(1, tid.long()))).sum()


def test_chain_gradients():
    """The operators together: gradients against 64-bit automatic
    differentiation of the formula, and against differences of the 64-bit
    loss along random directions."""
    f = feat()
    g = rng(11)
    F, ids, w, gamma, beta, tid, tl = _chain_inputs(g)
    route = f.Route(ids.shape[0], 8, F.shape[0])
    loss, dF, dw, dg, db = _chain(f, route, F, ids, w, gamma, beta, tid, tl)
    p = [v.double().requires_grad_() for v in (F, w, gamma, beta)]
    L = _chain_loss64(p[0], ids, p[1], p[2], p[3], tid, tl.double())
    L.backward()
    assert abs(float(loss.double().sum()) - float(L.detach())) <= 1e-5 * abs(float(L.detach()))
    got = (dF, dw, dg, db)
    for a, b in zip(got, p):
        # a chain of four float32 stages whose sums have at most 600 terms:
        # 1e-5 of the gradient's size, the parity tests' tolerance for gradients
        assert float((a.double() - b.grad).norm()) <= 1e-5 * float(b.grad.norm())
    base = [v.detach() for v in p]
    for k in range(4):
        d = torch.randn(base[k].shape, generator=g, device="cuda").double()
        h = 1e-5
        up = [v + h * d if q == k else v for q, v in enumerate(base)]
        dn = [v - h * d if q == k else v for q, v in enumerate(base)]
        num = float(_chain_loss64(up[0], ids, up[1], up[2], up[3], tid, tl.double())
                    - _chain_loss64(dn[0], ids, dn[1], dn[2], dn[3], tid, tl.double())) / (2 * h)
        ana = float((got[k].double() * d).sum())
        # the central difference is off by about h^2 times a third derivative
        # of the loss's size; 1e-5 as above
        assert abs(num - ana) <= 1e-5 * (abs(num) + float((got[k].double() * d).abs().sum())), k


def test_side_stream_and_two_graphs():
    """On a stream of their own, and as two captured graphs with a route each
    that replay side by side with new inputs: the eager results' bits."""
    f = feat()
    g = rng(5)
    ins = [_chain_inputs(g, T=700 + 40 * q) for q in range(2)]
    new = [_chain_inputs(g, T=700 + 40 * q) for q in range(2)]
    routes = [f.Route(i[1].shape[0], 8, i[0].shape[0]) for i in ins]
    want = [[v.clone() for v in _chain(f, r, *i)] for r, i in zip(routes, new)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = _chain(f, routes[0], *new[0])
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want[0]))
    graphs, outs = [], []
    for r, i in zip(routes, ins):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(_chain(f, r, *i))
        graphs.append(gr)
    for i, j in zip(ins, new):
        for a, b in zip(i, j):
            a.copy_(b)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(3):
        for s, gr in zip(streams, graphs):
            with torch.cuda.stream(s):
                gr.replay()
    torch.cuda.synchronize()
    for o, wv in zip(outs, want):
        assert all(torch.equal(a, b) for a, b in zip(o, wv))


def test_blend_weights_are_the_renders():
    """Sum w c is the rendered image, the ids are the list's, and empty or
    stray slots take no part; also on a coarser candidate grid."""
    import synth
    from soft_voronoi_render_b200 import Sad
    H, W, N = 37, 70, 300
    prm = synth.uniform_sites(H, W, N, 5)
    prm[0, ::17] = -1.0  # unused slots
    s = Sad(H, W, N + 4, seed=2)
    s.set_sites(prm)
    for cell in (1, 3):
        s.set_candidate_grid(cell)
        s.refresh(2)
        table = s.get_table()
        table[::13, 3] = N + 50
        table[::7, 5] = 17  # inactive
        table[5] = 0xFFFFFFFF
        s.set_table(table)
        img = s.render().cpu().numpy().astype(np.float64)
        ids, w = (v.cpu().numpy() for v in s.blend_weights())
        jj, ii = np.divmod(np.arange(H * W), W)
        lists = table[(jj // cell) * ((W + cell - 1) // cell) + ii // cell].astype(np.int64)
        live = ids >= 0
        assert np.array_equal(ids[live], lists[live]) and np.all(w[~live] == 0)
        act = (lists < N + 4) & (np.pad(prm[0], (0, 4), constant_values=-1.0)[np.minimum(lists, N + 3)] >= 0)
        assert np.array_equal(live, act)
        some = live.any(1)
        # eight float32 weights, each off by at most 6 u of the sum
        assert np.all(np.abs(w.sum(1, dtype=np.float64)[some] - 1.0) <= 16 * U)
        c = prm[4:7].T.astype(np.float64)[np.where(live, ids, 0)]
        ref = (c * w[..., None]).sum(1).T.reshape(3, H, W)
        assert np.abs(ref - img).max() <= 32 * U
    s.close()


def test_python_refusals_on_device_tensors():
    f = feat()
    from soft_voronoi_render_b200 import SadError
    x = torch.zeros((4, 8), device="cuda")
    i, w = torch.zeros((4, 2), dtype=torch.int32, device="cuda"), torch.zeros((4, 2), device="cuda")
    r = f.Route(4, 2, 5).build(i)
    F = torch.zeros((5, 8), device="cuda")
    bad = [lambda: r.build(i.long()), lambda: r.build(i[:2]), lambda: r.build(i.cpu()), lambda: r.dispatch(x[:3]),
           lambda: r.dispatch(x, w.double()), lambda: r.dispatch(x, out=x), lambda: r.combine(x),
           lambda: r.dispatch(x.t()[:4]), lambda: r.dispatch(x[:, :0]), lambda: r.dispatch(x[:1].expand(4, 8)),
           lambda: r.dispatch(x, out=torch.zeros((8, 8), dtype=torch.float16, device="cuda")),
           lambda: r.combine_backward(x, x), lambda: r.dispatch_backward(x), lambda: f.blend(F, i.t(), w),
           lambda: f.blend(F, i, w[:, :1]), lambda: f.blend(F, i, w.t().contiguous().t()),
           lambda: f.blend_backward(x, F.half(), i, w), lambda: f.blend_backward(x, F, i, w, f.Route(4, 2, 6)),
           lambda: f.blend_backward(x, F, i, w, None, dF=F), lambda: f.blend_backward(x[:, :4], F, i, w),
           lambda: f.layer_norm(x, torch.zeros(7, device="cuda")), lambda: f.layer_norm(x, None, None, -1.0),
           lambda: f.layer_norm_backward(x, x, None, w[:, 0], w[:, 0]),
           lambda: f.distill(x, i[:3], w), lambda: f.distill(x, i, w.half()), lambda: f.distill(x, i, w, 0.0),
           lambda: f.distill(x, i, w, 1.0, torch.zeros(5, device="cuda"))]
    for q, call in enumerate(bad):
        with pytest.raises(SadError):
            call()
            pytest.fail(str(q))
    torch.cuda.synchronize()


def test_feature_field_fit():
    """The framework's own path: the lists of a small diagram, a teacher of
    five classes, gradients against 64-bit automatic differentiation, and a
    few iterations of the fit."""
    import synth
    from soft_voronoi_render_b200 import Sad, fit
    H, W, N, D = 24, 40, 60, 5
    s = Sad(H, W, N, seed=3)
    s.set_sites(synth.uniform_sites(H, W, N, 4))
    s.refresh(2)
    g = rng(9)
    field = feat().FeatureField(s, D, seed=2)
    field.features.mul_(100.0)  # unit size: the norm's eps plays no part
    tid = torch.rand((H * W, D), generator=g, device="cuda").topk(3, 1).indices.int().contiguous()
    tl = randn(g, H * W, 3)
    rw = (torch.rand(H * W, generator=g, device="cuda") < 0.9).float()
    field.update_lists()
    loss = field.loss_and_grads(tid, tl, 2.0, rw)
    p = [v.double().requires_grad_() for v in (field.features, field.gamma, field.beta)]
    ok = field.ids >= 0
    x = (p[0][field.ids.clamp(min=0).long()] * (field.weights.double() * ok)[..., None]).sum(1)
    xc = x - x.mean(1, keepdim=True)
    y = xc / torch.sqrt((xc * xc).mean(1, keepdim=True) + 1e-5) * p[1] + p[2]
    lq, lp = torch.log_softmax(tl.double() / 2.0, 1), torch.log_softmax(y / 2.0, 1)
    rows = 4.0 * rw.double() * (lq.exp() * (lq - lp.gather(1, tid.long()))).sum(1)
    rows.sum().backward()
    assert float((loss.double() - rows.detach()).norm()) <= 1e-5 * float(rows.detach().norm())
    for a, b in zip((field.grad_features, field.grad_gamma, field.grad_beta), p):
        assert float((a.double() - b.grad).norm()) <= 1e-5 * float(b.grad.norm())
    z = field.render()
    assert float((z.double() - y.detach()).norm()) <= 1e-5 * float(y.detach().norm())
    losses = fit.run_features(field, tid, tl, iterations=3, temperature=2.0, row_weight=rw)
    assert len(losses) == 3 and all(np.isfinite(losses))
    assert fit.run_features(field, tid, tl, iterations=0) == []
    s.close()


@pytest.mark.parametrize("D", [4, 64, 65, 300])
def test_empty_slots_beside_infinities(D):
    """Gradients of empty slots are 0 and rows without pairs give 0, also
    where the row that comes back holds infinities or NaN."""
    f = feat()
    g = rng(D)
    T, K, E = 40, 8, 9
    ids = make_ids(g, T, K, E, 0.4)
    w = torch.rand((T, K), generator=g, device="cuda")
    F, dout = randn(g, E, D), randn(g, T, D)
    dout[::3] = float("inf")
    dout[1::3] = float("nan")
    r = f.Route(T, K, E).build(ids)
    empty = r.place < 0
    _, dw = f.blend_backward(dout, F, ids, w, r)
    assert bool((dw[empty] == 0).all()) and not bool(torch.isfinite(dw[::3][~empty[::3]]).any())
    y = randn(g, T * K, D)
    for dw in (r.combine_backward(dout, y, w)[1], r.dispatch_backward(y, dout, w)[1]):
        assert bool((dw[empty] == 0).all())
        assert bool(torch.isfinite(dw[2::3]).all())


@pytest.mark.parametrize("T,E,D,dt", [(300000, 3000, 64, "f32"), (400001, 5, 48, "f32"), (262144, 200000, 70, "bf16"),
                                      (1100000, 40000, 33, "f16")])
def test_blend_backward_beyond_the_cache(T, E, D, dt):
    """Enough rows that the chunks are taken in the order of the rows: the
    same sums, sites with few, many and no pairs among them."""
    f, t = feat(), TYPES[dt]
    g = rng(T)
    ids = make_ids(g, T, 8, E, 0.05)
    valid = (ids >= 0) & (ids < E)
    w = torch.rand((T, 8), generator=g, device="cuda")
    dout = randn(g, T, D, dtype=t)
    F = randn(g, E, D, dtype=t)
    r = f.Route(T, 8, E).build(ids)
    dF, dw = f.blend_backward(dout, F, ids, w, r)
    ref, big = torch.zeros((E, D), device="cuda").double(), torch.zeros((E, D), device="cuda").double()
    for k in range(8):
        s = dout.double() * torch.where(valid[:, k], w[:, k].double(), 0.0)[:, None]
        at = torch.where(valid[:, k], ids[:, k], 0).long()
        ref.index_add_(0, at, s)
        big.index_add_(0, at, s.abs())
    count = (r.offsets[1:] - r.offsets[:-1])[:, None].double()
    # chunks of at most 4096 pairs, then at most 8192 partial rows by eight warps
    close(dF, ref, torch.minimum(count + 1, torch.tensor(4096.0 + 1100, device="cuda").double()) * U * big)
    dF2, dw2 = f.blend_backward(dout, F, ids, w, r)
    assert torch.equal(dF, dF2) and torch.equal(dw, dw2)


@pytest.mark.parametrize("kind", ["random", "coherent", "one", "none", "sorted", "reversed", "two"])
@pytest.mark.parametrize("T,K,E", [(786432, 8, 1024), (786433, 8, 5000), (900001, 7, 131072),
                                   (6300001, 1, (1 << 20) - 1), (131073, 8, 5000), (1048577, 1, 1 << 20),
                                   (790000, 8, 1 << 21), (1600000, 4, 60000)])
def test_route_of_many_pairs(T, K, E, kind):
    """From 3 * 2^21 pairs and 1024 sites on the tiles' runs are sorted: the same
    whole numbers, whatever the runs are."""
    g = rng(T + E)
    j = torch.arange(T * K, device="cuda")
    ids = {"random": lambda: torch.randint(0, E, (T * K,), generator=g, device="cuda"),
           "coherent": lambda: (j // 40 * 7919 + torch.randint(0, 6, (T * K,), generator=g, device="cuda")) % E,
           "one": lambda: torch.full_like(j, E - 1), "none": lambda: torch.full_like(j, E + 3),
           "sorted": lambda: j * E // (T * K), "reversed": lambda: E - 1 - j * E // (T * K),
           "two": lambda: (j & 1) * (E - 1)}[kind]()
    if kind in ("random", "coherent"):
        ids = torch.where(torch.rand(T * K, generator=g, device="cuda") < 0.03, -1, ids)
    ids = ids.int().view(T, K).contiguous()
    r = feat().Route(T, K, E)
    r.workspace.fill_(255)
    r.build(ids)
    flat = ids.view(-1).long()
    key = torch.where((flat >= 0) & (flat < E), flat, E)
    skey, perm = torch.sort(key, stable=True)
    m = int((key < E).sum())
    pos = torch.arange(T * K, device="cuda")
    place = torch.empty_like(pos)
    place[perm] = pos
    assert torch.equal(r.order.long(), torch.where(pos < m, perm, -1))
    assert torch.equal(r.place.view(-1).long(), torch.where(key < E, place, -1))
    assert torch.equal(r.offsets.long(), torch.searchsorted(skey, torch.arange(E + 1, device="cuda")))


def _graphed(call):
    """call() captured and replayed twice after its inputs were put back."""
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call()  # set-up outside the capture
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = call()
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    return out


def test_captured_large_forms():
    """The forms for large sizes replay to the eager bits: clusters of a long
    row, the sort by runs, segment sums of far rows, wide rows' norm."""
    f = feat()
    g = rng(21)
    z, tid, tl = randn(g, 2, 90001), torch.randint(0, 90001, (2, 9), generator=g, device="cuda").int(), randn(g, 2, 9)
    want = f.distill(z, tid, tl)
    got = _graphed(lambda: f.distill(z, tid, tl))
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    T, E, D = 800000, 5000, 24
    ids = ((torch.arange(T * 8, device="cuda") // 50 * 77 + torch.randint(0, 5, (T * 8,), generator=g, device="cuda"))
           % E).int().view(T, 8).contiguous()
    w = torch.rand((T, 8), generator=g, device="cuda")
    F, dout = randn(g, E, D), randn(g, T, D)
    r, r2 = f.Route(T, 8, E).build(ids), f.Route(T, 8, E)
    want = f.blend_backward(dout, F, ids, w, r)
    got = _graphed(lambda: f.blend_backward(dout, F, ids, w, r2.build(ids)))
    assert torch.equal(r.order, r2.order) and torch.equal(r.place, r2.place) and torch.equal(r.offsets, r2.offsets)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    x, dy = randn(g, 900, 4096, dtype=torch.bfloat16), randn(g, 900, 4096, dtype=torch.bfloat16)
    gamma = randn(g, 4096)
    y, m, rs = f.layer_norm(x, gamma, None)
    want = f.layer_norm_backward(dy, x, gamma, m, rs)
    got = _graphed(lambda: f.layer_norm_backward(dy, x, gamma, *f.layer_norm(x, gamma, None)[1:]))
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_offsets_beyond_32_bits():
    """Matrices of more than 4 GB: their last rows against the formulas."""
    f = feat()
    g = rng(31)
    bf = torch.bfloat16
    # 1,300,000 pairs of 2048: 5.3 GB on the pairs' side
    T, K, D, E = 162500, 8, 2048, 16
    ids = torch.randint(0, E, (T, K), generator=g, device="cuda").int()
    x = torch.randn((T, D), generator=g, device="cuda", dtype=bf)
    r = f.Route(T, K, E).build(ids)
    xs = r.dispatch(x)
    at = torch.cat([torch.arange(50, device="cuda"), torch.arange(T * K - 50, T * K, device="cuda")])
    assert torch.equal(xs[at], x[r.order[at].long() // K])
    back = r.combine(xs)
    t = torch.arange(T - 40, T, device="cuda")
    # eight equal rows: sums of a bfloat16 with itself
    close(back[t], 8.0 * x[t].double(), 8 * U * 8 * x[t].double().abs())
    del xs, back, x, r, ids
    torch.cuda.empty_cache()
    # 20,000 rows of 131,072 classes: 5.2 GB
    T, V, M = 20000, 131072, 4
    z = torch.randn((T, V), generator=g, device="cuda", dtype=bf)
    tid, tl = torch.randint(0, V, (T, M), generator=g, device="cuda").int(), randn(g, T, M)
    z1, rw = z[-3:].clone(), torch.ones(3, device="cuda")
    loss, dz = f.distill(z, tid, tl, dlogits=z)
    check_distill(z1, tid[-3:], tl[-3:], 1.0, rw, M, V, loss[-3:], dz[-3:])
    del z, dz
    torch.cuda.empty_cache()
    # 700,000 rows of 4096: 5.7 GB
    R, D = 700000, 4096
    x = torch.randn((R, D), generator=g, device="cuda", dtype=bf)
    x1 = x[-5:].clone()
    y, m, rs = f.layer_norm(x, out=x)
    want, m1, rs1 = f.layer_norm(x1)
    # five rows alone may be shared out over other lanes: one rounding apart
    assert float((y[-5:].double() - want.double()).abs().max()) <= 2.0 ** -8 * 2 * float(want.double().abs().max())
    assert float((m[-5:] - m1).abs().max()) <= (D / 32 + 20) * U * float(x1.float().abs().mean(1).max()) * 2


def test_many_experts_few_rows():
    """More experts than pairs, a key of 24 bits."""
    f = feat()
    E = (1 << 23) + 5
    ids = torch.tensor([[E - 1, 3], [-1, E], [3, 1 << 22]], dtype=torch.int32, device="cuda")
    r = f.Route(3, 2, E).build(ids)
    assert r.order.tolist() == [1, 4, 5, 0, -1, -1] and r.place.tolist() == [[3, 0], [-1, -1], [1, 2]]
    assert r.offsets[[0, 3, 4, 1 << 22, (1 << 22) + 1, E - 1, E]].tolist() == [0, 0, 2, 2, 3, 3, 4]
