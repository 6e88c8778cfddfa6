"""What the bound by norm tells apart, on a model of the tree attention's arithmetic (CPU)."""
import numpy as np
import pytest
import torch

from spec_util import make_tree_case, tree_attention
from tree_accuracy import NORM_BOUND, attention64, model, norm_errors


def test_attention64_is_the_plain_form():
    c = make_tree_case(50, 2, 7, 4, 2, 64, [40, 300], poison=False)
    o, lse, _, _ = tree_attention(c["q64"], c["k64"], c["v64"], c["vis"], c["lens"], c["trees"], 0.2, 1.5)
    got, got_lse = attention64(c, 0.2, vs=1.5)
    assert np.allclose(got.numpy(), o, rtol=1e-11, atol=1e-13) and np.allclose(got_lse.numpy(), lse, rtol=1e-11)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D", [64, 128])
def test_the_bound_by_norm_sees_a_lost_part_and_a_lost_flush(dtype, D):
    c = make_tree_case(51, 1, 8, 1, 1, D, [40000], dtype=dtype, poison=False)
    c["vis"][:] = True
    ref, _ = attention64(c, D ** -0.5)
    off = lambda **kw: norm_errors(torch.from_numpy(model(c["q64"][0, :, 0], c["k64"][0][:, 0], c["v64"][0][:, 0],  # noqa: E731
                                                          D ** -0.5, dtype, **kw))[None, :, None], ref)[0]
    assert off() <= NORM_BOUND
    assert off(parts=1) > 4 * NORM_BOUND
    assert off(flush=1 << 30) > 1.5 * NORM_BOUND
