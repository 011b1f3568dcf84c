"""What the feature-field calls refuse, before anything is launched: through
the C ABI with addresses that are never read, and through the Python
functions with CPU tensors."""
import pytest
import torch

from soft_voronoi_render_b200 import _lib, features, fit

BAD, UNS, CAP = _lib.SAD_ERR_INVALID_ARG, _lib.SAD_ERR_UNSUPPORTED, _lib.SAD_ERR_CAPACITY
A = [0x100000 * (q + 1) for q in range(16)]  # aligned addresses that nothing reads


def refused(status, word, f, *args):
    with pytest.raises(_lib.SadError) as e:
        f(*args)
    assert e.value.status == status and word in str(e.value), str(e.value)
    assert word in _lib.sad_feature_error()


def with_arg(args, at, value):
    a = list(args)
    a[at] = value
    return a


def each(f, good, cases):
    for at, value, status, word in cases:
        refused(status, word, f, *with_arg(good, at, value))


def test_sizes():
    refused(BAD, "negative", _lib.sad_route_workspace_bytes, -1, 8, 8)
    refused(BAD, "below 1", _lib.sad_route_workspace_bytes, 4, 0, 8)
    refused(UNS, "exceeds 8", _lib.sad_route_workspace_bytes, 4, 9, 8)
    refused(CAP, "2^31", _lib.sad_route_workspace_bytes, 1 << 28, 8, 8)
    refused(BAD, "n_sites", _lib.sad_route_workspace_bytes, 4, 8, 0)
    refused(BAD, "n_sites", _lib.sad_route_workspace_bytes, 4, 8, 1 << 30)
    refused(BAD, "D = 0", _lib.sad_blend_workspace_bytes, 4, 8, 8, 0)
    refused(UNS, "16384", _lib.sad_layer_norm_workspace_bytes, 4, 16385)
    refused(BAD, "n_rows", _lib.sad_layer_norm_workspace_bytes, -1, 4)
    assert _lib.sad_route_workspace_bytes(0, 1, 1) >= 0
    assert _lib.sad_route_workspace_bytes(((1 << 31) - 1) // 8, 8, (1 << 30) - 1) > 1 << 31


def test_route():
    ws = _lib.sad_route_workspace_bytes(100, 8, 50)
    good = [A[0], 100, 8, 50, A[1], A[2], A[3], A[4], ws]
    each(_lib.sad_route, good, [
        (0, None, BAD, "ids is NULL"), (0, A[0] + 2, BAD, "ids is not 4-byte aligned"),
        (1, -3, BAD, "negative"), (2, 9, UNS, "exceeds 8"), (3, 0, BAD, "n_sites"), (4, None, BAD, "offsets is NULL"),
        (5, None, BAD, "order is NULL"), (6, A[3] + 1, BAD, "place is not"), (7, None, BAD, "workspace is NULL"),
        (7, A[4] + 8, BAD, "16-byte"), (8, ws - 1, BAD, "workspace has")])


def test_exchange():
    good = [_lib.SAD_BF16, A[0], 64, A[1], A[2], 10, 4, 64, A[3], 64]
    for f, rows, out in ((_lib.sad_dispatch, "x", "xs"), (_lib.sad_combine, "y", "out")):
        each(f, good, [
            (0, 3, UNS, "type 3"), (0, -1, UNS, "type"), (1, None, BAD, rows + " is NULL"),
            (1, A[0] + 1, BAD, rows + " is not aligned"), (2, 63, BAD, rows + ": 63"), (3, A[1] + 2, BAD, "weights"),
            (4, None, BAD, "place is NULL"), (5, -1, BAD, "negative"), (6, 0, BAD, "K = 0"), (6, 9, UNS, "K = 9"),
            (7, 0, BAD, "D = 0"), (7, 1 << 30, UNS, "2^30"), (8, None, BAD, out + " is NULL"),
            (9, 5, BAD, out + ": 5"), (2, 1 << 41, BAD, "too large")])
    good = [_lib.SAD_F32, A[0], 64, A[1], 64, A[2], A[3], 10, 4, 64, A[4], 64, A[5]]
    for f, a, b, c in ((_lib.sad_dispatch_backward, "dxs", "x", "dx"), (_lib.sad_combine_backward, "dout", "y", "dy")):
        each(f, good, [
            (1, None, BAD, a + " is NULL"), (3, None, BAD, b + " is NULL"), (4, 7, BAD, b + ": 7"),
            (6, None, BAD, "place is NULL"), (10, None, BAD, c + " is NULL"), (11, 63, BAD, c + ": 63"),
            (12, A[5] + 2, BAD, "dweights")])


def test_blend():
    good = [_lib.SAD_F16, A[0], 32, 50, A[1], A[2], 10, 8, 32, A[3], 32]
    each(_lib.sad_blend, good, [
        (1, None, BAD, "F is NULL"), (2, 31, BAD, "F: 31"), (3, 0, BAD, "n_sites"), (4, None, BAD, "ids is NULL"),
        (5, None, BAD, "weights is NULL"), (9, None, BAD, "out is NULL"), (6, 1 << 29, CAP, "2^31")])
    ws = max(16, _lib.sad_blend_workspace_bytes(10, 8, 50, 32))
    good = [_lib.SAD_F16, A[0], 32, A[1], 32, 50, A[2], A[3], A[4], A[5], 10, 8, 32, A[6], A[7], A[8], ws]
    each(_lib.sad_blend_backward, good, [
        (1, None, BAD, "dout is NULL"), (3, None, BAD, "F is NULL"), (6, None, BAD, "ids is NULL"),
        (7, None, BAD, "weights is NULL"), (8, None, BAD, "offsets is NULL"), (9, None, BAD, "order is NULL"),
        (13, A[6] + 2, BAD, "dF"), (14, A[7] + 1, BAD, "dweights")])


def test_layer_norm():
    good = [_lib.SAD_F32, A[0], 64, A[1], A[2], 1e-5, 10, 64, A[3], 64, A[4], A[5]]
    each(_lib.sad_layer_norm, good, [
        (0, 7, UNS, "type"), (1, None, BAD, "x is NULL"), (2, 1, BAD, "x: 1"), (3, A[1] + 2, BAD, "gamma"),
        (5, -1.0, BAD, "eps"), (5, float("nan"), BAD, "eps"), (6, -1, BAD, "n_rows"), (7, 0, BAD, "D = 0"),
        (7, 16385, UNS, "16384"), (8, None, BAD, "y is NULL"), (10, A[4] + 1, BAD, "mean")])
    refused(BAD, "another row distance", _lib.sad_layer_norm, *with_arg(with_arg(good, 8, A[0]), 9, 65))
    ws = _lib.sad_layer_norm_workspace_bytes(10, 64)
    good = [_lib.SAD_F32, A[0], 64, A[1], 64, A[2], A[3], A[4], 10, 64, A[5], 64, A[6], A[7], A[8], ws]
    each(_lib.sad_layer_norm_backward, good, [
        (1, None, BAD, "dy is NULL"), (3, None, BAD, "x is NULL"), (6, None, BAD, "mean is NULL"),
        (7, None, BAD, "rstd is NULL"), (10, None, BAD, "dx is NULL"), (12, None, BAD, "together"),
        (14, None, BAD, "workspace is NULL"), (15, ws - 1, BAD, "workspace has")])


def test_distill():
    good = [_lib.SAD_BF16, A[0], 100, A[1], A[2], A[3], 10, 100, 8, 1.0, A[4], A[5], 100]
    each(_lib.sad_distill, good, [
        (1, None, BAD, "logits is NULL"), (2, 99, BAD, "logits: 99"), (3, None, BAD, "teacher_ids is NULL"),
        (4, None, BAD, "teacher_logits is NULL"), (5, A[3] + 1, BAD, "row_weight"), (6, -1, BAD, "n_rows"),
        (7, 0, BAD, "V = 0"), (8, 0, BAD, "M = 0"), (8, 129, UNS, "128"), (9, 0.0, BAD, "tau"),
        (9, float("nan"), BAD, "tau"), (9, -1.0, BAD, "tau"), (9, float("inf"), BAD, "tau"),
        (10, None, BAD, "loss is NULL"), (11, A[5] + 1, BAD, "dlogits"), (12, 9, BAD, "dlogits: 9")])
    refused(BAD, "another row distance", _lib.sad_distill, *with_arg(with_arg(good, 11, A[0]), 12, 101))


def test_blend_weights_needs_bound_buffers():
    ctx = _lib.sad_create(8, 8, 16)
    try:
        with pytest.raises(_lib.SadError) as e:
            _lib.sad_blend_weights(ctx, A[0], A[1])
        assert e.value.status == _lib.SAD_ERR_NOT_BOUND
    finally:
        _lib.sad_destroy(ctx)


def test_messages_belong_to_the_thread():
    import threading
    refused(BAD, "below 1", _lib.sad_route_workspace_bytes, 4, 0, 8)
    seen = []
    t = threading.Thread(target=lambda: seen.append(_lib.sad_feature_error()))
    t.start()
    t.join()
    assert seen == [""] and "below 1" in _lib.sad_feature_error()


def test_python_refuses_tensors_before_any_call():
    x = torch.zeros((4, 8))
    i, w = torch.zeros((4, 2), dtype=torch.int32), torch.zeros((4, 2))
    for f, args in ((features.blend, (x, i, w)), (features.layer_norm, (x,)), (features.distill, (x, i, w)),
                    (features.layer_norm_backward, (x, x, None, w[:, 0], w[:, 0])),
                    (features.blend_backward, (x, x, i, w))):
        with pytest.raises(_lib.SadError) as e:
            f(*args)
        assert e.value.status == BAD and "CUDA device" in str(e.value)
    with pytest.raises(_lib.SadError) as e:
        features.layer_norm(torch.zeros(4))
    assert "2-D" in str(e.value)
    with pytest.raises(_lib.SadError) as e:
        features.layer_norm(x.double())
    assert e.value.status == UNS
    with pytest.raises(_lib.SadError) as e:
        features.Route(4, 9, 8)
    assert e.value.status == UNS
    assert callable(fit.run_features)
