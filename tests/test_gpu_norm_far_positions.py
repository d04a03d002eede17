"""Angles at the far end of the stated range of positions (1e7, shift included), against the fp64 oracle
with the tolerances of test_gpu_norm_rope.py.  Whole numbers up to 2^24 are exact in fp32, and the oracle's
own angle is good to 1e7 * 2^-53 radians."""
import numpy as np
import pytest
import torch

from tests.test_gpu_norm_rope import _case, _check_grad, _check_y, _bf16, _gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def h3():
    import __graft_entry__

    __graft_entry__.build()
    import packed_varlen_attention_modality_gb300 as h3

    h3.load_library()
    return h3


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    torch.cuda.set_device(0)
    return torch.device("cuda", 0)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("far, frames", [(9_999_400, (0.0, 0.0)), (-9_999_999, (0.0, 0.0)),
                                         (3_000_000, (238.0, 4_199_000.0))])  # 3e6 + 4.199e6 * 40 / 24 < 1e7
def test_positions_up_to_the_stated_range(h3, dev, far, frames, dim):
    q, k, qw, kw, where = _case((97, 3, 2, dim, True, 2, torch.float32, False), seed=31, far=far)
    where["pos"][:, 1:] += far  # the other two coordinates as well
    where["start_frames"] = np.array(frames, dtype=np.float32)
    on = {n: _gpu(dev, x) for n, x in where.items()}
    args = [_gpu(dev, x) for x in (q, k, qw, kw)]
    yq, yk = h3.qk_norm_rope(*args, **on)
    _check_y(yq, q, qw, where)
    _check_y(yk, k, kw, where)
    rng = np.random.default_rng(32)
    dy = [_bf16(rng, *x.shape) for x in (q, k)]
    dq, dk, dqw, dkw = h3.qk_norm_rope_bwd(*(t.to(dev) for t in dy), *args, **on)
    _check_grad(dq, dqw, dy[0], q, qw, where)
    _check_grad(dk, dkw, dy[1], k, kw, where)
