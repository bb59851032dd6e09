"""The gated layer's operators on the GPU where their kernels take other ways than at the sizes of test_gpu_gated.py: values
that are not finite beside lanes without channels."""
import pytest
import torch

import selective_state_space_chunked_amd as ssm

from .test_gpu_gated import DEV, gen, norm_inputs

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------------------
# group norm
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("G,per", [(4, 24), (5, 3), (3, 65), (2, 520), (2, 519), (2, 2056), (2, 2501)])
def test_norm_non_finite_values_stay_in_their_group(G, per, dtype):
    """What is not finite in x, z or gy of one group of one row, or in w and bias of one channel, reaches that group's (that
    channel's group's) results and no other's: groups whose last lanes have no channels among them."""
    r = gen(G + per)
    T, C = 9, G * per
    t, gy = norm_inputs(T, C, dtype, r)
    ref = {**ssm.group_norm_fwd(groups=G, silu=True, **t), **ssm.group_norm_bwd(gy=gy, groups=G, silu=True, **t)}
    for name in ("x", "z", "gy", "w", "bias"):
        for at in (0, per, C - 1):
            for bad in (float("nan"), float("inf"), -float("inf")):
                u = {**t, "gy": gy}
                u[name] = u[name].clone()
                rows = slice(None) if name in ("w", "bias") else 5
                u[name][(at,) if name in ("w", "bias") else (5, at)] = bad
                g = u.pop("gy")
                got = {**ssm.group_norm_fwd(groups=G, silu=True, **u), **ssm.group_norm_bwd(gy=g, groups=G, silu=True, **u)}
                own = slice(at // per * per, (at // per + 1) * per)
                for k in ref:
                    keep = torch.ones_like(ref[k], dtype=torch.bool)
                    if k in ("gw", "gbias"):
                        keep[own] = False
                    else:
                        keep[rows, own] = False
                    assert torch.equal(got[k][keep], ref[k][keep]), (name, at, bad, k)
