"""More of what the feature-field functions refuse before any call."""
import pytest

from soft_voronoi_render_b200 import _lib, features


def test_a_route_needs_a_cuda_device():
    for device in ("cpu", "meta"):
        with pytest.raises(_lib.SadError) as e:
            features.Route(4, 2, 8, device=device)
        assert e.value.status == _lib.SAD_ERR_INVALID_ARG and "CUDA device" in str(e.value)
