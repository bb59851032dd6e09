"""Host side of the gated layer's operators: which kernels the library holds, arguments that no field holds.  No GPU."""
import re

import pytest
import torch

import selective_state_space_chunked_amd as ssm
from selective_state_space_chunked_amd import binding as B


def kernels(name):
    """Template arguments of a kernel's instances in the built library, mangled."""
    B.lib()
    with open(B.LIB_PATH, "rb") as f:
        return set(m.decode() for m in re.findall(name.encode() + rb"I(\w+?)EEvNS_", f.read()))


def norm_forms(most):
    """Types, lanes of a team, channels of a vector and vectors of a lane that some group of 1 to 8192 channels takes,
    mangled: as norm_validate chooses them, for either outcome of its question whether the rows are few."""
    forms = set()
    for per in range(1, 8193):
        v = most if per % most == 0 else 1
        nv = per // v
        for few in (False, True):
            if v > 1:
                r = 1 if nv <= 64 or 128 < nv <= 256 or 512 < nv <= 1024 else 2
            else:
                r = 2 if nv <= 128 and few else 8
            lanes = -(-nv // r)
            forms.add((64 if lanes <= 64 else 256 if lanes <= 256 else 1024, v, r))
    return {f"{'t' if most == 8 else 'f'}Li{t}ELi{v}ELi{r}E" for t, v, r in forms}


def test_every_group_norm_kernel_is_reached():
    for name in ("norm_fwd_kernel", "norm_bwd_kernel"):
        assert kernels(name) == norm_forms(8) | norm_forms(4), name


@pytest.mark.parametrize("groups", [2**63, -2**63 - 1, 10**30])
def test_norm_refuses_counts_of_groups_past_64_bits(groups):
    x = torch.zeros(4, 6)
    with pytest.raises(ValueError, match="groups"):
        ssm.group_norm_fwd(x=x, groups=groups)
    with pytest.raises(ValueError, match="groups"):
        ssm.group_norm_bwd(gy=x, x=x, groups=groups)
