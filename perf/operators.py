"""Timed cases of the feature-field operators: route, exchange, blend, layer norm, distill.

A feature field gives every site D channels beside its colour.  Pixels are the
rows (tokens), sites the experts, and a row's K candidate ids with their
softmax weights are the router's choice.  ``run`` computes the operators either
in elementary torch operations (``own = False``) or through
``soft_voronoi_render_b200.features`` (``own = True``).
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------

def listed():
    return [
        # routing one row: a single query against a small set of experts, all latency
        dict(name="route_token", op="route", layout="router", T=1, K=8, E=64),
        # the lists of the 2048 x 2048 frame with 131,072 sites, as a fit sorts them after a candidate update
        dict(name="route_full", op="route", layout="image", W=2048, T=2048 * 2048, K=8, E=131072),
        # one row out to its experts and back while serving
        dict(name="exchange_token", op="exchange", layout="router", T=1, K=4, E=64, D=1024, dtype="f16",
             weighted="combine", step=False),
        # a ragged training batch with the weights applied on the way out; nothing is a multiple of anything
        dict(name="exchange_ragged", op="exchange", layout="router", T=1021, K=3, E=37, D=203, dtype="f32",
             weighted="dispatch", step=True),
        # a full training batch through top-8 experts
        dict(name="exchange_step", op="exchange", layout="router", T=16384, K=8, E=128, D=2048, dtype="bf16",
             weighted="combine", step=True),
        # rendering 64 channels of a fitted 768 x 512 field with 50,000 sites
        dict(name="blend_frame", op="blend", layout="image", W=768, T=768 * 512, K=8, E=50000, D=64, dtype="f16",
             step=False),
        # a fitting step of 32 channels on the 2048 x 2048 frame: lists sorted, blend, gradients
        dict(name="blend_step", op="blend", layout="image", W=2048, T=2048 * 2048, K=8, E=131072, D=32, dtype="bf16",
             step=True),
        # every pixel's 64 blended channels normalised, forward and backward (768 x 512)
        dict(name="norm_frame", op="norm", R=768 * 512, D=64, dtype="f32", step=True),
        # wide rows of a transformer's training batch, an odd number of them
        dict(name="norm_wide", op="norm", R=8191, D=4096, dtype="bf16", step=True),
        # every pixel's 150 class scores against the teacher's 8 best classes (768 x 512)
        dict(name="distill_frame", op="distill", T=768 * 512, V=150, M=8, dtype="f32", tau=2.0, step=True),
        # one row over a large vocabulary: work split along the row
        dict(name="distill_token", op="distill", T=1, V=128000, M=32, dtype="bf16", tau=1.0, step=True),
        # a batch over an odd vocabulary
        dict(name="distill_vocab", op="distill", T=4096, V=50001, M=32, dtype="bf16", tau=1.0, step=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "exchange", "blend", "norm", "distill"])
    dtype = rng.choice(["f32", "bf16", "f16"])
    step = rng.random() < 0.6
    if op == "route":
        layout = rng.choice(["image", "router"])
        if layout == "image":
            W, H = _log(rng, 8, 2048), _log(rng, 8, 2048)
            return dict(op=op, layout=layout, W=W, T=W * H, K=8, E=_log(rng, 9, max(9, W * H // 8)))
        K = rng.randint(1, 8)
        return dict(op=op, layout=layout, T=_log(rng, 1, 65536), K=K, E=_log(rng, K, 512))
    if op == "exchange":
        K = rng.randint(1, 8)
        D = _log(rng, 5, 4096)
        if rng.random() < 0.5:
            D = -(-D // 8) * 8
        return dict(op=op, layout="router", T=_log(rng, 1, max(2, min(32768, (1 << 27) // (K * D)))), K=K,
                    E=_log(rng, K, 256), D=D, dtype=dtype, weighted=rng.choice(["combine", "dispatch"]), step=step)
    if op == "blend":
        D = _log(rng, 3, 256)
        if rng.random() < 0.5:
            D = -(-D // 8) * 8
        W = _log(rng, 8, 2048)
        H = _log(rng, 8, max(9, min(2048, (1 << 27) // (W * D))))
        return dict(op=op, layout="image", W=W, T=W * H, K=8, E=_log(rng, 9, max(9, W * H // 8)), D=D, dtype=dtype,
                    step=step)
    if op == "norm":
        D = _log(rng, 8, 8192)
        return dict(op=op, R=_log(rng, 1, min(1 << 19, (1 << 25) // D)), D=D, dtype=dtype, step=step)
    V = _log(rng, 4, 131072)
    return dict(op=op, T=_log(rng, 1, min(1 << 19, (1 << 27) // V)), V=V, M=rng.randint(1, min(V, 64)), dtype=dtype,
                tau=rng.choice([1.0, 2.0, 0.7]), step=step)


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------

def _gen(seed):
    return torch.Generator("cuda").manual_seed(seed)


def _randn(g, shape, dtype=torch.float32):
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def _image_lists(case, g):
    """Candidate lists as a converged fit holds them: the 8 nearest of the 9
    sites around a pixel on a jittered grid, ids in random order over the
    image, nearest first; cells beyond the border give empty slots (-1)."""
    W, T, E = case["W"], case["T"], case["E"]
    H = T // W
    gw = max(1, min(E, int(round(math.sqrt(E * W / H)))))
    gh = max(1, E // gw)
    ids = torch.randperm(E, generator=g, device="cuda")[:gw * gh].view(gh, gw)
    jit = torch.rand((2, gh, gw), generator=g, device="cuda")
    p = torch.arange(T, device="cuda")
    x, y = (p % W).float().add_(0.5).mul_(gw / W), (p // W).float().add_(0.5).mul_(gh / H)
    cx, cy = x.long().clamp_(max=gw - 1), y.long().clamp_(max=gh - 1)
    dist, cand = [], []
    for dy in (-1, 0, 1):
        for dx in (-1, 0, 1):
            qx, qy = cx + dx, cy + dy
            ok = (qx >= 0) & (qx < gw) & (qy >= 0) & (qy < gh)
            qx, qy = qx.clamp(0, gw - 1), qy.clamp(0, gh - 1)
            d = torch.hypot(x - qx - jit[0, qy, qx], y - qy - jit[1, qy, qx])
            dist.append(torch.where(ok, d, torch.inf))
            cand.append(torch.where(ok, ids[qy, qx], -1))
    dist, cand = torch.stack(dist, 1), torch.stack(cand, 1)
    dist, slot = dist.topk(8, dim=1, largest=False)
    cand = cand.gather(1, slot).int().contiguous()
    w = torch.softmax(-6.0 * dist, dim=1)
    return cand, torch.where(cand >= 0, w, 0.0).contiguous()


def _router_lists(case, g):
    """A top-K router's choice: distinct experts a row, some experts in more
    demand than others, a few slots dropped (-1) as beyond capacity."""
    T, K, E = case["T"], case["K"], case["E"]
    score = torch.rand((T, E), generator=g, device="cuda").add_(torch.rand(E, generator=g, device="cuda") * 0.5)
    top, ids = score.topk(K, dim=1)
    w = torch.softmax(4.0 * top, dim=1)
    drop = torch.rand((T, K), generator=g, device="cuda") < 0.02
    return torch.where(drop, -1, ids).int().contiguous(), w.contiguous()


def prepare(case, seed):
    g = _gen(seed)
    op, s = case["op"], {"case": case}
    if op in ("route", "exchange", "blend"):
        s["ids"], s["w"] = (_image_lists if case["layout"] == "image" else _router_lists)(case, g)
        T, K, E = case["T"], case["K"], case["E"]
        n = T * K
    if op == "exchange":
        D, dt = case["D"], DTYPES[case["dtype"]]
        s["x"], s["y"] = _randn(g, (T, D), dt), _randn(g, (n, D), dt)
        s["xs"] = torch.zeros((n, D), dtype=dt, device="cuda")  # rows behind the last pair stay as they are
        if case["step"]:
            s["dout"], s["dxs"] = _randn(g, (T, D), dt), _randn(g, (n, D), dt)
            s["dy"] = torch.zeros((n, D), dtype=dt, device="cuda")
    if op == "blend":
        D, dt = case["D"], DTYPES[case["dtype"]]
        s["F"] = _randn(g, (E, D), dt)
        if case["step"]:
            s["dout"] = _randn(g, (T, D), dt)
    if op == "norm":
        R, D, dt = case["R"], case["D"], DTYPES[case["dtype"]]
        # rows of different size and offset, as blended features have them
        s["x"] = (_randn(g, (R, D)) * (0.5 + torch.rand((R, 1), generator=g, device="cuda"))
                  + 0.5 * _randn(g, (R, 1))).to(dt)
        s["gamma"], s["beta"] = 1.0 + 0.1 * _randn(g, (D,)), 0.1 * _randn(g, (D,))
        if case["step"]:
            s["dy"] = _randn(g, (R, D), dt)
    if op == "distill":
        T, V, M, dt = case["T"], case["V"], case["M"], DTYPES[case["dtype"]]
        start = torch.randint(0, V, (T, 1), generator=g, device="cuda")
        hop = torch.randint(1, max(1, V // M) + 1, (T, 1), generator=g, device="cuda")
        tid = (start + hop * torch.arange(M, device="cuda")) % V  # M distinct classes a row
        tl = _randn(g, (T, M)).mul_(2.0).sort(dim=1, descending=True).values + 6.0
        if M > 1:  # some teachers hand out short lists
            short = torch.rand((T, M), generator=g, device="cuda") < 0.03
            short[:, 0] = False
            tid = torch.where(short, -1, tid)
        z = _randn(g, (T, V)).mul_(2.0)
        z.scatter_add_(1, tid.clamp(min=0), torch.where(tid >= 0, 0.7 * tl, 0.0))
        s["z"], s["tid"], s["tl"] = z.to(dt), tid.int().contiguous(), tl.contiguous()
        rw = torch.ones(T, device="cuda")
        if T > 8:  # padded rows count for nothing
            rw[torch.rand(T, generator=g, device="cuda") < 0.01] = 0.0
        s["rw"] = rw
    if own and op in ("route", "exchange", "blend"):
        from soft_voronoi_render_b200 import features
        s["route"] = features.Route(T, K, E)
    return s


# --------------------------------------------------------------------------
# the operators
# --------------------------------------------------------------------------

def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    from soft_voronoi_render_b200 import features
    c = s["case"]
    op = c["op"]
    if op == "route":
        r = s["route"].build(s["ids"])
        return {"offsets": r.offsets, "order": r.order, "place": r.place}
    if op == "exchange":
        forth, back = (s["w"], None) if c["weighted"] == "dispatch" else (None, s["w"])
        r = s["route"].build(s["ids"])
        res = {"xs": r.dispatch(s["x"], forth, out=s["xs"]), "out": r.combine(s["y"], back)}
        if c["step"]:
            dy, dw_back = r.combine_backward(s["dout"], s["y"], back, dy=s["dy"])
            dx, dw_forth = r.dispatch_backward(s["dxs"], s["x"], forth)
            res.update(dy=dy, dx=dx, dw=dw_forth if back is None else dw_back)
        return res
    if op == "blend":
        res = {"out": features.blend(s["F"], s["ids"], s["w"])}
        if c["step"]:
            r = s["route"].build(s["ids"])
            res["dF"], res["dw"] = features.blend_backward(s["dout"], s["F"], s["ids"], s["w"], r)
        return res
    if op == "norm":
        y, mean, rstd = features.layer_norm(s["x"], s["gamma"], s["beta"], 1e-5)
        res = {"y": y, "mean": mean, "rstd": rstd}
        if c["step"]:
            res["dx"], res["dgamma"], res["dbeta"] = features.layer_norm_backward(s["dy"], s["x"], s["gamma"], mean,
                                                                                  rstd)
        return res
    loss, dz = features.distill(s["z"], s["tid"], s["tl"], c["tau"], s["rw"], want_grad=c["step"])
    return {"loss": loss, "dz": dz} if c["step"] else {"loss": loss}


def _plain_route(ids, E):
    flat = ids.reshape(-1).long()
    n = flat.numel()
    key = torch.where((flat >= 0) & (flat < E), flat, E)
    order = torch.argsort(key, stable=True)
    count = torch.zeros(E + 1, dtype=torch.long, device=key.device).index_add_(0, key, torch.ones_like(key))
    offsets = torch.zeros(E + 1, dtype=torch.long, device=key.device)
    offsets[1:] = count[:E].cumsum(0)
    pos = torch.arange(n, device=key.device)
    place = torch.empty_like(pos)
    place[order] = pos
    place = torch.where(key < E, place, -1)
    order = torch.where(pos < offsets[E], order, -1)
    return offsets.int(), order.int(), place.int().view(ids.shape)


def _run_plain(s):
    c = s["case"]
    op = c["op"]
    if op == "route":
        offsets, order, place = _plain_route(s["ids"], c["E"])
        return {"offsets": offsets, "order": order, "place": place}
    if op == "exchange":
        return _plain_exchange(s, c)
    if op == "blend":
        return _plain_blend(s, c)
    if op == "norm":
        x, dt = s["x"].float(), s["x"].dtype
        mean = x.mean(1)
        xc = x - mean[:, None]
        rstd = 1.0 / torch.sqrt((xc * xc).mean(1) + 1e-5)
        xh = xc * rstd[:, None]
        res = {"y": (xh * s["gamma"] + s["beta"]).to(dt), "mean": mean, "rstd": rstd}
        if c["step"]:
            dy = s["dy"].float()
            gd = dy * s["gamma"]
            dx = rstd[:, None] * (gd - gd.mean(1, keepdim=True) - xh * (gd * xh).mean(1, keepdim=True))
            # sums over every row: 64 bits
            res.update(dx=dx.to(dt), dgamma=(dy * xh).sum(0, dtype=torch.float64).float(),
                       dbeta=dy.sum(0, dtype=torch.float64).float())
        return res
    return _plain_distill(s, c)


def _plain_exchange(s, c):
    T, K, E = c["T"], c["K"], c["E"]
    offsets, order, place = _plain_route(s["ids"], E)
    valid = place >= 0
    at = place.clamp(min=0).long()
    w = torch.where(valid, s["w"], 0.0)
    one = valid.float()
    forth, back = (w, one) if c["weighted"] == "dispatch" else (one, w)
    dt = s["x"].dtype
    x = s["x"].float()

    def spread(rows, weights):  # rows[t] times its weight to every place of t; the rest stays 0
        out = torch.zeros((T * K, rows.shape[1]), dtype=dt, device="cuda")
        for k in range(K):
            v = valid[:, k]
            out[at[v, k]] = (rows[v] * weights[v, k, None]).to(dt)
        return out

    def gather(pairs, weights):
        out = torch.zeros((T, pairs.shape[1]), device="cuda")
        for k in range(K):
            out += torch.where(valid[:, k, None], pairs[at[:, k]].float() * weights[:, k, None], 0.0)
        return out

    def dots(pairs, rows):
        return torch.stack([torch.where(valid[:, k], (pairs[at[:, k]].float() * rows).sum(1), 0.0)
                            for k in range(K)], 1)

    res = {"xs": spread(x, forth), "out": gather(s["y"], back).to(dt)}
    if c["step"]:
        dout = s["dout"].float()
        res["dy"] = spread(dout, back)
        res["dx"] = gather(s["dxs"], forth).to(dt)
        res["dw"] = dots(s["dxs"], x) if c["weighted"] == "dispatch" else dots(s["y"], dout)
    return res


def _plain_blend(s, c):
    T, K, E, dt = c["T"], c["K"], c["E"], s["F"].dtype
    F, ids = s["F"].float(), s["ids"].long()
    valid = (ids >= 0) & (ids < E)
    at = torch.where(valid, ids, 0)
    w = torch.where(valid, s["w"], 0.0)
    out = torch.zeros((T, F.shape[1]), device="cuda")
    for k in range(K):
        out += F[at[:, k]] * w[:, k, None]
    res = {"out": out.to(dt)}
    del out
    if c["step"]:
        dout = s["dout"].float()
        dF = torch.zeros(F.shape, dtype=torch.float64, device="cuda")  # a site's sum may be long
        dw = torch.empty((T, K), device="cuda")
        for k in range(K):
            dF.index_add_(0, at[:, k], (dout * w[:, k, None]).double())
            dw[:, k] = torch.where(valid[:, k], (F[at[:, k]] * dout).sum(1), 0.0)
        res["dF"], res["dw"] = dF.float(), dw
    return res


def _plain_distill(s, c):
    tau, z = c["tau"], s["z"].float() / c["tau"]
    T, V = z.shape
    tid, rw = s["tid"].long(), s["rw"]
    valid = (tid >= 0) & (tid < V) & (s["tl"] > -torch.inf)
    at = torch.where(valid, tid, 0)
    tl = torch.where(valid, s["tl"] / tau, -torch.inf)
    some = valid.any(1) & (rw != 0)
    m = tl.max(1, keepdim=True).values
    q = torch.where(valid, torch.exp(tl - m), 0.0)
    qs = q.sum(1, keepdim=True)
    q = q / qs
    logq = tl - m - torch.log(qs)
    zm = z.max(1, keepdim=True).values
    e = torch.exp(z - zm)
    es = e.sum(1, keepdim=True)
    logp = z.gather(1, at) - zm - torch.log(es)
    loss = torch.where(q > 0, q * (logq - logp), 0.0).sum(1)
    res = {"loss": torch.where(some, rw * tau * tau * loss, 0.0)}
    if c["step"]:
        e /= es
        e.scatter_add_(1, at, torch.where(valid, -q, 0.0))
        res["dz"] = torch.where(some[:, None], (rw * tau)[:, None] * e, 0.0).to(s["z"].dtype)
    return res


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------

def exact(case, seed):
    op = case["op"]
    if op == "route":
        return None  # whole numbers, equal or wrong
    s = prepare(case, seed)
    f8 = torch.float64
    if op == "norm":
        x = s["x"].to(f8)
        var, mean = torch.var_mean(x, 1, correction=0, keepdim=True)
        rstd = torch.rsqrt(var + 1e-5)
        g = s["gamma"].to(f8)
        y = (x - mean) * rstd * g + s["beta"].to(f8)
        res = {"y": y, "mean": mean[:, 0], "rstd": rstd[:, 0]}
        if case["step"]:
            xh, dy, D = (x - mean) * rstd, s["dy"].to(f8), case["D"]
            a = dy * g
            res["dx"] = (D * a - a.sum(1, keepdim=True) - xh * torch.einsum("rd,rd->r", a, xh)[:, None]) * rstd / D
            res["dgamma"] = torch.einsum("rd,rd->d", dy, xh)
            res["dbeta"] = torch.einsum("rd->d", dy)
        return res
    if op == "distill":
        tau, T, V, M = case["tau"], case["T"], case["V"], case["M"]
        loss, dz = [], []
        step = max(1, (1 << 26) // V)
        for a in range(0, T, step):
            z, tid = s["z"][a:a + step].to(f8) / tau, s["tid"][a:a + step].long()
            tl, rw = s["tl"][a:a + step].to(f8) / tau, s["rw"][a:a + step].to(f8)
            logp = torch.log_softmax(z, 1)
            q = torch.zeros((z.shape[0], V + 1), dtype=f8, device="cuda")  # the last column takes the empty slots
            lq = torch.log_softmax(torch.where(tid >= 0, tl, -torch.inf), 1)
            q.scatter_(1, torch.where(tid >= 0, tid, V), lq.exp())
            q = q[:, :V]
            loss.append(rw * tau * tau * (torch.special.xlogy(q, q) - q * logp).sum(1))
            if case["step"]:
                dz.append((logp.exp() - q) * (rw * tau)[:, None])
        res = {"loss": torch.cat(loss)}
        if case["step"]:
            res["dz"] = torch.cat(dz)
        return res
    T, K, E, D = case["T"], case["K"], case["E"], case["D"]
    ids = s["ids"].long()
    live = (ids >= 0)
    w = s["w"].to(f8) * live
    if op == "blend":
        F = torch.cat([s["F"].to(f8), torch.zeros((1, D), dtype=f8, device="cuda")])  # row E: nothing
        at = torch.where(live, ids, E)
        out = torch.empty((T, D), dtype=f8, device="cuda")
        step = max(1, (1 << 25) // (K * D))
        dF, dw = torch.zeros((E + 1, D), dtype=f8, device="cuda"), torch.empty((T, K), dtype=f8, device="cuda")
        for a in range(0, T, step):
            rows = F[at[a:a + step]]
            out[a:a + step] = torch.einsum("tk,tkd->td", w[a:a + step], rows)
            if case["step"]:
                go = s["dout"][a:a + step].to(f8)
                dw[a:a + step] = torch.einsum("td,tkd->tk", go, rows)
                dF.index_add_(0, at[a:a + step].reshape(-1), (w[a:a + step, :, None] * go[:, None]).reshape(-1, D))
        return {"out": out, "dF": dF[:E], "dw": dw} if case["step"] else {"out": out}
    # exchange: the pairs of each expert in turn
    flat = ids.reshape(-1)
    pairs = torch.cat([(flat == e).nonzero()[:, 0] for e in range(E)])
    m, tok = pairs.numel(), pairs // K
    forth = case["weighted"] == "dispatch"
    wp = w.reshape(-1)[pairs][:, None]
    ones = torch.ones_like(wp)
    wf, wb = (wp, ones) if forth else (ones, wp)
    xs = torch.zeros((T * K, D), dtype=f8, device="cuda")
    xs[:m] = s["x"].to(f8)[tok] * wf
    out = torch.zeros((T, D), dtype=f8, device="cuda").index_add_(0, tok, s["y"][:m].to(f8) * wb)
    res = {"xs": xs, "out": out}
    if case["step"]:
        dy = torch.zeros((T * K, D), dtype=f8, device="cuda")
        dy[:m] = s["dout"].to(f8)[tok] * wb
        res["dy"] = dy
        res["dx"] = torch.zeros((T, D), dtype=f8, device="cuda").index_add_(0, tok, s["dxs"][:m].to(f8) * wf)
        a, b = (s["dxs"], s["x"]) if forth else (s["y"], s["dout"])
        dw = torch.zeros(T * K, dtype=f8, device="cuda")
        dw[pairs] = torch.einsum("md,md->m", a[:m].to(f8), b.to(f8)[tok])
        res["dw"] = dw.view(T, K)
    return res


# --------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------

def work(case):
    op = case["op"]
    if op == "norm":
        R, D, b = case["R"], case["D"], BYTES[case["dtype"]]
        if not case["step"]:
            return {"bytes": 2 * R * D * b + 8 * R + 8 * D, "flops": 8 * R * D}
        return {"bytes": 4 * R * D * b + 8 * R + 16 * D, "flops": 20 * R * D}
    if op == "distill":
        T, V, M, b = case["T"], case["V"], case["M"], BYTES[case["dtype"]]
        if not case["step"]:
            return {"bytes": T * V * b + 8 * T * M + 8 * T, "flops": 4 * T * V}
        return {"bytes": 2 * T * V * b + 8 * T * M + 8 * T, "flops": 6 * T * V}
    T, K, E = case["T"], case["K"], case["E"]
    n = T * K
    if op == "route":
        return {"bytes": 12 * n + 4 * (E + 1), "flops": n}
    D, b = case["D"], BYTES[case["dtype"]]
    if op == "exchange":
        # ids and weights in; x and y in, xs and out out; the step adds dout and dxs in, dy, dx and dw out
        once = 2 * (T + n) * D * b
        if not case["step"]:
            return {"bytes": once + 8 * n, "flops": 2 * n * D}
        return {"bytes": 2 * once + 12 * n, "flops": 7 * n * D}
    if not case["step"]:
        return {"bytes": (T + E) * D * b + 8 * n, "flops": 2 * n * D}
    return {"bytes": (2 * T + E) * D * b + 4 * E * D + 12 * n, "flops": 6 * n * D}
