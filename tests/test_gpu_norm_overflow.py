"""Rows of the norm whose sums pass float32's range: y of a layer norm is NaN there, and the other rows
are what they are without them."""

import pytest
import torch

import combine_shuffling_amd as cs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("H", [40, 264, 2056, 16384])
def test_sums_past_the_range_stay_in_their_rows(H):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    dev = torch.device("cuda:0")
    p = cs.Plan(9, H, 4, 1, 2)
    g = torch.Generator(device=dev)
    g.manual_seed(H)
    x = torch.randn(9, H, generator=g, device=dev)
    huge = x.clone()
    huge[2], huge[7] = 3e38, -3e38
    rows = [0, 1, 3, 4, 5, 6, 8]
    for kind in ("layer", "rms"):
        y, _, stats = p.norm(x, kind=kind, save_stats=True)
        z, _, others = p.norm(huge, kind=kind, save_stats=True)
        assert torch.equal(y[rows], z[rows]) and torch.equal(stats[rows], others[rows])
        if kind == "layer":
            assert torch.isnan(z[[2, 7]]).all()
        else:       # the squares' sum: rstd 0
            assert (z[[2, 7]] == 0).all() and (others[[2, 7], 1] == 0).all()
