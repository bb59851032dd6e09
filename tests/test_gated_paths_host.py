"""Host side of the gated layer's operators: which kernels the library holds, arguments that no field holds, the
stated limits.  No GPU."""
import ctypes
import re

import pytest
import torch

import selective_state_space_chunked_amd as ssm
from selective_state_space_chunked_amd import binding as B

from .test_gated_host import code, gated_args, norm_args, tgated_args


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


def test_operations_tell_the_library():
    """What a caller that looks the entry points up may ask: the operations that came under the same version."""
    L, n = B.lib(), ctypes.c_size_t(0)
    for op, args in ((B.SSM_OP_GATED_FWD, gated_args()), (B.SSM_OP_GATED_BWD, gated_args()), (B.SSM_OP_TOKENS_GATED, tgated_args()),
                     (B.SSM_OP_GROUP_NORM_BWD, norm_args())):
        assert L.ssm_workspace_bytes(op, ctypes.byref(args), ctypes.byref(n)) == 0
    assert L.ssm_workspace_bytes(B.SSM_OP_GROUP_NORM_BWD + 1, ctypes.byref(norm_args()), ctypes.byref(n)) == code("UNSUPPORTED")


@pytest.mark.parametrize("over,ok", [
    (dict(batch=65535, channels=1, length=1), True), (dict(batch=65536, channels=1, length=1), False),
    (dict(batch=1, channels=(1 << 24) - 1, length=1), True), (dict(batch=1, channels=1 << 24, length=1), False),
    (dict(batch=1, channels=1, length=(1 << 31) - (1 << 16) - 1), True), (dict(batch=1, channels=1, length=(1 << 31) - (1 << 16)), False),
    (dict(batch=32, channels=(1 << 23) - 3, length=1), True), (dict(batch=32, channels=(1 << 23) - 2, length=1), False)])
def test_gated_sizes_are_the_stated_ones(over, ok):
    L, n = B.lib(), ctypes.c_size_t(0)
    dense = (over["channels"] * over["length"], over["length"])
    a = gated_args(x_stride=dense, r_stride=dense, i_stride=dense, **over)
    assert L.ssm_workspace_bytes(B.SSM_OP_GATED_BWD, ctypes.byref(a), ctypes.byref(n)) == (0 if ok else code("SHAPE"))
