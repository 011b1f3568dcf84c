"""Feature fields: rows routed, blended, normalised and learned from a teacher.

A site may carry D channels beside its colour; pixels (rows) blend the rows
of their candidate sites (experts) with the render's softmax weights, which
``Sad.blend_weights`` hands out.  Every function here checks its tensors,
allocates its outputs where none are given and forwards to the C ABI
(``include/sad.h``, "Feature fields") on the current stream of the tensors'
device; no step of the computation runs in Python.

Row matrices are 2-D tensors of float32, bfloat16 or float16 whose rows are
consecutive elements (any row distance).  ids and places are dense int32, an id
outside [0, n_sites) is an empty slot; weights are dense float32.
"""
from __future__ import annotations

import functools

import torch

from . import _lib
from ._lib import SAD_ERR_INVALID_ARG, SAD_ERR_UNSUPPORTED, SadError

__all__ = ["Route", "blend", "blend_backward", "layer_norm", "layer_norm_backward", "distill", "FeatureField"]

_TYPES = {torch.float32: _lib.SAD_F32, torch.bfloat16: _lib.SAD_BF16, torch.float16: _lib.SAD_F16}


def _refuse(text: str):
    raise SadError(SAD_ERR_INVALID_ARG, text)


def _rows(name: str, x, shape=None, like=None):
    """Checks a row matrix; returns its row distance."""
    if not isinstance(x, torch.Tensor) or x.dim() != 2:
        _refuse(f"{name} must be a 2-D tensor")
    if x.dtype not in _TYPES:
        raise SadError(SAD_ERR_UNSUPPORTED, f"{name}: type {x.dtype} is not float32, bfloat16 or float16")
    if not x.is_cuda:
        _refuse(f"{name} must be on a CUDA device")
    if like is not None and (x.dtype != like.dtype or x.device != like.device):
        _refuse(f"{name} must have the type and the device of the other rows")
    T, D = x.shape
    if shape is not None and (T, D) != shape:
        _refuse(f"{name} has shape {(T, D)}, expected {tuple(shape)}")
    if D < 1:
        _refuse(f"{name} has no columns")
    if x.is_contiguous():
        return D
    ld, step = x.stride()
    if (D > 1 and step != 1) or (T > 1 and ld < D):
        _refuse(f"{name}: a row's elements must be consecutive and rows must not overlap")
    return ld if T > 1 else D


def _dense(name, x, dtype, shape, device):
    if not isinstance(x, torch.Tensor) or x.dtype != dtype or x.shape != shape:
        _refuse(f"{name} must be a {dtype} tensor of shape {tuple(shape)}")
    if x.device != device or not x.is_contiguous():
        _refuse(f"{name} must be dense and on {device}")


# The current stream's handle by device index.  torch.cuda.current_stream()
# builds a Stream object first, 3 us of a call's 10.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)


def _run(device, call, *args):
    """call(*args, stream) on the current stream of the tensors' device, made
    current for the call where it is not; raises on a non-zero status."""
    index = device.index
    if index == torch.cuda.current_device():
        status = call(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            status = call(*args, _raw_stream(index))
    if status:
        raise SadError(status, _lib.sad_feature_error())


def _at(x):
    return None if x is None else x.data_ptr()


def _float32(x, *shape):
    """An uninitialised float32 tensor beside x."""
    return x.new_empty(shape) if x.dtype is torch.float32 else x.new_empty(shape, dtype=torch.float32)


# workspace sizes are functions of the sizes alone
_blend_bytes = functools.lru_cache(256)(_lib.sad_blend_workspace_bytes)
_norm_bytes = functools.lru_cache(256)(_lib.sad_layer_norm_workspace_bytes)


class Route:
    """Rows sorted by expert: the buffers of one routing, and the row
    exchange that goes by it.

    ``build`` fills ``offsets`` (n_sites + 1), ``order`` (n_rows * K) and
    ``place`` (n_rows, K) for the ids it is given, in stream order; the calls
    after it go by those until the next build.  A Route owns one workspace (up
    to 28 bytes a pair): builds of one Route must not overlap on the GPU (use
    one Route per stream, and one per captured graph that may run beside
    another).
    """

    def __init__(self, n_rows: int, K: int, n_sites: int, device="cuda"):
        self.T, self.K, self.E = int(n_rows), int(K), int(n_sites)
        ws = _lib.sad_route_workspace_bytes(self.T, self.K, self.E)
        device = torch.device(device)
        if device.type != "cuda":
            _refuse(f"a route must be on a CUDA device, not on {device}")
        if not torch.cuda.is_available():
            raise SadError(_lib.SAD_ERR_CUDA, "no CUDA device is available")
        i32 = dict(dtype=torch.int32, device=device)
        self.offsets = torch.zeros(self.E + 1, **i32)
        self.order = torch.full((self.T * self.K,), -1, **i32)
        self.place = torch.full((self.T, self.K), -1, **i32)
        self.device = self.offsets.device
        self.workspace = torch.empty(ws, dtype=torch.uint8, device=device)

    @property
    def _outputs(self):
        return (self.offsets.data_ptr(), self.order.data_ptr(), self.place.data_ptr(), self.workspace.data_ptr(),
                self.workspace.numel())

    def build(self, ids) -> "Route":
        _dense("ids", ids, torch.int32, (self.T, self.K), self.device)
        _run(self.device, _lib.load().sad_route, ids.data_ptr(), self.T, self.K, self.E, *self._outputs)
        return self

    def _weights(self, weights):
        if weights is not None:
            _dense("weights", weights, torch.float32, (self.T, self.K), self.device)

    def _here(self, name, x):
        if x.device != self.device:
            _refuse(f"{name} is on {x.device}, the route on {self.device}")

    def dispatch(self, x, weights=None, out=None):
        """Rows out to their experts: (n_rows * K, D), row ``place[t, k]`` =
        weights[t, k] x[t].  Rows behind the last pair (offsets[n_sites]) are
        left as they were in ``out``, and undefined without it."""
        ldx = _rows("x", x)
        self._here("x", x)
        D = x.shape[1]
        if x.shape[0] != self.T:
            _refuse(f"x has {x.shape[0]} rows, the route {self.T}")
        self._weights(weights)
        ldo = D
        if out is None:
            out = x.new_empty((self.T * self.K, D))
        else:
            ldo = _rows("out", out, (self.T * self.K, D), x)
        _run(self.device, _lib.load().sad_dispatch, _TYPES[x.dtype], x.data_ptr(), ldx, _at(weights),
             self.place.data_ptr(), self.T, self.K, D, out.data_ptr(), ldo)
        return out

    def dispatch_backward(self, dxs, x=None, weights=None, dx=None):
        """(dx, dweights): dx[t] = sum of weights dxs[place]; dweights = <dxs[place],
        x[t]> when x is given, else None."""
        ld = _rows("dxs", dxs)
        self._here("dxs", dxs)
        D = dxs.shape[1]
        if dxs.shape[0] != self.T * self.K:
            _refuse(f"dxs has {dxs.shape[0]} rows, the route {self.T * self.K} pairs")
        self._weights(weights)
        ldx, dw = 0, None
        if x is not None:
            ldx = _rows("x", x, (self.T, D), dxs)
            dw = _float32(x, self.T, self.K)
        lddx = D
        if dx is None:
            dx = dxs.new_empty((self.T, D))
        else:
            lddx = _rows("dx", dx, (self.T, D), dxs)
        _run(self.device, _lib.load().sad_dispatch_backward, _TYPES[dxs.dtype], dxs.data_ptr(), ld, _at(x), ldx,
             _at(weights), self.place.data_ptr(), self.T, self.K, D, dx.data_ptr(), lddx, _at(dw))
        return dx, dw

    def combine(self, y, weights=None, out=None):
        """Rows back from their experts: out[t] = sum of weights[t, k]
        y[place[t, k]]; a row without a pair gives 0."""
        ldy = _rows("y", y)
        self._here("y", y)
        D = y.shape[1]
        if y.shape[0] != self.T * self.K:
            _refuse(f"y has {y.shape[0]} rows, the route {self.T * self.K} pairs")
        self._weights(weights)
        ldo = D
        if out is None:
            out = y.new_empty((self.T, D))
        else:
            ldo = _rows("out", out, (self.T, D), y)
        _run(self.device, _lib.load().sad_combine, _TYPES[y.dtype], y.data_ptr(), ldy, _at(weights),
             self.place.data_ptr(), self.T, self.K, D, out.data_ptr(), ldo)
        return out

    def combine_backward(self, dout, y=None, weights=None, dy=None):
        """(dy, dweights): dy[place[t, k]] = weights[t, k] dout[t] (rows behind
        the last pair as in ``dispatch``); dweights = <y[place], dout[t]> when
        y is given, else None."""
        ld = _rows("dout", dout)
        self._here("dout", dout)
        D = dout.shape[1]
        if dout.shape[0] != self.T:
            _refuse(f"dout has {dout.shape[0]} rows, the route {self.T}")
        self._weights(weights)
        ldy, dw = 0, None
        if y is not None:
            ldy = _rows("y", y, (self.T * self.K, D), dout)
            dw = _float32(y, self.T, self.K)
        lddy = D
        if dy is None:
            dy = dout.new_empty((self.T * self.K, D))
        else:
            lddy = _rows("dy", dy, (self.T * self.K, D), dout)
        _run(self.device, _lib.load().sad_combine_backward, _TYPES[dout.dtype], dout.data_ptr(), ld, _at(y), ldy,
             _at(weights), self.place.data_ptr(), self.T, self.K, D, dy.data_ptr(), lddy, _at(dw))
        return dy, dw


def _lists(ids, weights, device):
    if not isinstance(ids, torch.Tensor) or ids.dim() != 2:
        _refuse("ids must be a 2-D tensor")
    _dense("ids", ids, torch.int32, ids.shape, device)
    _dense("weights", weights, torch.float32, ids.shape, device)
    return ids.shape


def blend(F, ids, weights, out=None):
    """Rows that a site's pixels share: out[t] = sum of weights[t, k]
    F[ids[t, k]], F (n_sites, D)."""
    ldf = _rows("F", F)
    T, K = _lists(ids, weights, F.device)
    E, D = F.shape
    ldo = D
    if out is None:
        out = F.new_empty((T, D))
    else:
        ldo = _rows("out", out, (T, D), F)
    _run(F.device, _lib.load().sad_blend, _TYPES[F.dtype], F.data_ptr(), ldf, E, ids.data_ptr(), weights.data_ptr(),
         T, K, D, out.data_ptr(), ldo)
    return out


def blend_backward(dout, F, ids, weights, route=None, dF=None):
    """(dF, dweights) of ``blend``: dF (n_sites, D) float32 sums each site's
    pairs in order, by a Route built for these ids (None without one);
    dweights (T, K) float32."""
    ld, ldf = _rows("dout", dout), _rows("F", F, None, dout)
    T, K = _lists(ids, weights, F.device)
    E, D = F.shape
    if tuple(dout.shape) != (T, D):
        _refuse(f"dout has shape {tuple(dout.shape)}, expected {(T, D)}")
    dev = F.device
    dw = weights.new_empty((T, K))
    offsets = order = ws = None
    nbytes = 0
    if route is not None:
        if (route.T, route.K, route.E) != (T, K, E) or route.device != dev:
            _refuse("the route was made for other sizes or another device")
        offsets, order = route.offsets, route.order
        if dF is None:
            dF = weights.new_empty((E, D))
        else:
            _dense("dF", dF, torch.float32, (E, D), dev)
        nbytes = _blend_bytes(T, K, E, D)
        ws = weights.new_empty(-(-nbytes // 4))
    elif dF is not None:
        _refuse("dF needs a route")
    _run(dev, _lib.load().sad_blend_backward, _TYPES[F.dtype], dout.data_ptr(), ld, F.data_ptr(), ldf, E,
         ids.data_ptr(), weights.data_ptr(), _at(offsets), _at(order), T, K, D, _at(dF), dw.data_ptr(), _at(ws), nbytes)
    return dF, dw


def layer_norm(x, gamma=None, beta=None, eps: float = 1e-5, out=None):
    """(y, mean, rstd) of every row of x; gamma and beta (D) float32 or None.
    ``out`` may be x."""
    ldx = _rows("x", x)
    T, D = x.shape
    dev = x.device
    for name, v in (("gamma", gamma), ("beta", beta)):
        if v is not None:
            _dense(name, v, torch.float32, (D,), dev)
    ldy = D
    if out is None:
        out = x.new_empty((T, D))
    else:
        ldy = _rows("out", out, (T, D), x)
    like = x if gamma is None else gamma
    mean, rstd = _float32(like, T), _float32(like, T)
    _run(dev, _lib.load().sad_layer_norm, _TYPES[x.dtype], x.data_ptr(), ldx, _at(gamma), _at(beta), eps, T, D,
         out.data_ptr(), ldy, mean.data_ptr(), rstd.data_ptr())
    return out, mean, rstd


def layer_norm_backward(dy, x, gamma, mean, rstd, want_affine: bool = True, dx=None, dgamma=None, dbeta=None):
    """(dx, dgamma, dbeta) from the saved mean and rstd; without
    ``want_affine`` the last two are None.  ``dx`` may be dy; ``dgamma`` and
    ``dbeta``, dense float32, are given together."""
    ld, ldx = _rows("dy", dy), _rows("x", x, None, dy)
    T, D = x.shape
    dev = x.device
    if tuple(dy.shape) != (T, D):
        _refuse(f"dy has shape {tuple(dy.shape)}, expected {(T, D)}")
    if gamma is not None:
        _dense("gamma", gamma, torch.float32, (D,), dev)
    _dense("mean", mean, torch.float32, (T,), dev)
    _dense("rstd", rstd, torch.float32, (T,), dev)
    lddx = D
    if dx is None:
        dx = x.new_empty((T, D))
    else:
        lddx = _rows("dx", dx, (T, D), x)
    ws, nbytes = None, 0
    if (dgamma is None) != (dbeta is None) or (dgamma is not None and not want_affine):
        _refuse("dgamma and dbeta are given together, and wanted")
    if want_affine:
        if dgamma is None:
            dgamma, dbeta = mean.new_empty(D), mean.new_empty(D)
        else:
            _dense("dgamma", dgamma, torch.float32, (D,), dev)
            _dense("dbeta", dbeta, torch.float32, (D,), dev)
        nbytes = _norm_bytes(T, D)
        ws = mean.new_empty(-(-nbytes // 4))
    _run(dev, _lib.load().sad_layer_norm_backward, _TYPES[x.dtype], dy.data_ptr(), ld, x.data_ptr(), ldx, _at(gamma),
         mean.data_ptr(), rstd.data_ptr(), T, D, dx.data_ptr(), lddx, _at(dgamma), _at(dbeta), _at(ws), nbytes)
    return dx, dgamma, dbeta


def distill(logits, teacher_ids, teacher_logits, temperature: float = 1.0, row_weight=None, want_grad: bool = True,
            dlogits=None):
    """(loss (T), dlogits (T, V) or None): the divergence of softmax(logits /
    temperature) from the teacher's over its top classes, times temperature^2
    and the row's weight, and its gradient (sad_distill in include/sad.h has
    the formulas and what empty rows give).  ``dlogits`` may be logits."""
    ld = _rows("logits", logits)
    T, V = logits.shape
    dev = logits.device
    if not isinstance(teacher_ids, torch.Tensor) or teacher_ids.dim() != 2 or teacher_ids.shape[0] != T:
        _refuse(f"teacher_ids must have {T} rows")
    M = teacher_ids.shape[1]
    _dense("teacher_ids", teacher_ids, torch.int32, (T, M), dev)
    _dense("teacher_logits", teacher_logits, torch.float32, (T, M), dev)
    if row_weight is not None:
        _dense("row_weight", row_weight, torch.float32, (T,), dev)
    lddz = V
    if dlogits is not None:
        lddz = _rows("dlogits", dlogits, (T, V), logits)
    elif want_grad:
        dlogits = logits.new_empty((T, V))
    loss = teacher_logits.new_empty(T)
    _run(dev, _lib.load().sad_distill, _TYPES[logits.dtype], logits.data_ptr(), ld, teacher_ids.data_ptr(),
         teacher_logits.data_ptr(), _at(row_weight), T, V, M, float(temperature), loss.data_ptr(), _at(dlogits), lddz)
    return loss, dlogits


class FeatureField:
    """D channels for every site of a ``Sad``, blended per pixel by the
    render's weights and layer-normalised (convex blending shrinks rows where
    unlike sites meet; the norm undoes it).

    ``features`` (N, D), ``gamma`` and ``beta`` (D) are float32 and the
    caller's to optimise; ``loss_and_grads`` fills ``grad_features``,
    ``grad_gamma`` and ``grad_beta``, the same buffers at every call.
    ``update_lists`` takes the current
    candidate lists; call it after the lists or the sites changed, with their
    routing before a captured step is replayed.  The sites themselves are
    fitted by the colour loss and not moved here.
    """

    def __init__(self, sad, D: int, seed: int = 1, eps: float = 1e-5):
        if D < 1:
            _refuse(f"D = {D} is below 1")
        self.sad, self.D, self.eps = sad, int(D), float(eps)
        f32 = dict(dtype=torch.float32, device=sad.device)
        gen = torch.Generator(sad.device).manual_seed(seed)
        self.features = torch.randn((sad.N, self.D), generator=gen, **f32).mul_(0.01)
        self.gamma, self.beta = torch.ones(self.D, **f32), torch.zeros(self.D, **f32)
        self.grad_features = torch.zeros((sad.N, self.D), **f32)
        self.grad_gamma, self.grad_beta = torch.zeros(self.D, **f32), torch.zeros(self.D, **f32)
        self.ids = torch.full((sad.P, 8), -1, dtype=torch.int32, device=sad.device)
        self.weights = torch.zeros((sad.P, 8), **f32)
        self.route = Route(sad.P, 8, sad.N, sad.device)
        self._routed = True           # by what has run: no lists yet, and no pairs in the route
        self._unrouted_graph = False  # whether a replay may leave the route behind the lists

    def update_lists(self, route: bool = True) -> None:
        """The lists' ids and weights, and (for fitting) their routing; without
        ``route`` the next ``loss_and_grads`` routes them."""
        self.sad.blend_weights(self.ids, self.weights)
        if route:
            self.route.build(self.ids)
        if not torch.cuda.is_current_stream_capturing():
            self._routed = route
        elif not route:
            self._unrouted_graph = True

    def render(self):
        """The field's (P, D) rows: class logits, or an embedding."""
        return layer_norm(blend(self.features, self.ids, self.weights), self.gamma, self.beta, self.eps)[0]

    def loss_and_grads(self, teacher_ids, teacher_logits, temperature: float = 1.0, row_weight=None):
        """The pixels' distillation losses (P); the D channels are the
        teacher's classes.  Gradients are those of the losses' sum."""
        if not self._routed or self._unrouted_graph:
            self.route.build(self.ids)
            self._routed = self._routed or not torch.cuda.is_current_stream_capturing()
        x = blend(self.features, self.ids, self.weights)
        y, mean, rstd = layer_norm(x, self.gamma, self.beta, self.eps)
        loss, dy = distill(y, teacher_ids, teacher_logits, temperature, row_weight, dlogits=y)
        dx, _, _ = layer_norm_backward(dy, x, self.gamma, mean, rstd, dx=dy, dgamma=self.grad_gamma,
                                       dbeta=self.grad_beta)
        blend_backward(dx, self.features, self.ids, self.weights, self.route, dF=self.grad_features)
        return loss
