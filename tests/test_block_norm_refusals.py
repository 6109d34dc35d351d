"""What the block norm's calls refuse, before anything is launched (no device needed)."""
import math

import pytest
import torch

from kda_delta_rule_chunkwise_b200 import binding
from kda_delta_rule_chunkwise_b200 import build as kbuild

BAD, NOT, OK = binding.KDA_ERR_INVALID_ARG, binding.KDA_ERR_UNSUPPORTED, binding.KDA_OK
F32, BF16 = binding.KDA_F32, binding.KDA_BF16


@pytest.fixture(scope="module")
def lib():
    kbuild.build()
    return binding.load()


def norm(lib, **kw):
    a = dict(x=16, y=32, gate=48, w_post=64, w_pre=80, rows=4, width=64, scale=1.0, eps=1e-6, x_dtype=F32, dtype=BF16,
             x_new=96, h=112, stream=None)
    a.update(kw)
    return lib.kda_block_norm(*a.values())


def back(lib, **kw):
    a = dict(x=16, y=32, gate=48, w_post=64, w_pre=80, dx_new=96, dh=112, rows=4, width=64, scale=1.0, eps=1e-6,
             x_dtype=F32, dtype=BF16, dx=128, dy=144, dgate=160, dw_post=176, dw_pre=192, workspace=208,
             workspace_bytes=1 << 30, stream=None)
    a.update(kw)
    return lib.kda_block_norm_backward(*a.values())


@pytest.mark.parametrize("call", [norm, back])
@pytest.mark.parametrize("bad", [dict(rows=-1), dict(width=0), dict(width=-8), dict(scale=math.inf), dict(scale=math.nan),
                                 dict(eps=0.0), dict(eps=-1.0), dict(eps=math.nan), dict(eps=math.inf), dict(x_dtype=5),
                                 dict(dtype=-1), dict(x=None), dict(y=None), dict(w_post=None), dict(w_pre=None)])
def test_refuses(lib, call, bad):
    assert call(lib, **bad) == BAD


@pytest.mark.parametrize("call", [norm, back])
@pytest.mark.parametrize("bad", [dict(width=16385), dict(x_dtype=BF16, dtype=F32), dict(rows=2 ** 31)])
def test_does_not_support(lib, call, bad):
    assert call(lib, **bad) == NOT


def test_outputs_and_workspace(lib):
    assert norm(lib, x_new=None) == BAD and norm(lib, h=None) == BAD and norm(lib, rows=0, x=None, h=None) == OK
    for bad in (dict(dx=None), dict(dy=None), dict(dgate=None), dict(dw_post=None), dict(dw_pre=None), dict(workspace=None),
                dict(workspace=210)):
        assert back(lib, **bad) == BAD
    f = lib.kda_block_norm_backward_workspace_bytes
    assert back(lib, workspace_bytes=f(4, 64) - 1) == BAD
    assert f(0, 64) == 0 and f(-1, 64) == 0 and f(4, 0) == 0 and f(10 ** 6, 4096) == 444 * 2 * 4096 * 4
    assert f(10 ** 6, 64) == 444 * 16 * 2 * 64 * 4 and f(1, 64) == 16 * 2 * 64 * 4


def test_binding_refuses():
    x, w = torch.zeros(4, 64), torch.zeros(64)
    with pytest.raises(ValueError, match="CUDA"):
        binding.kda_block_norm(x, x, None, w, w)
    with pytest.raises(ValueError, match="bf16 or fp32"):
        binding.kda_block_norm(x.half(), x, None, w, w)
    with pytest.raises(ValueError, match="last dimension"):
        binding.kda_block_norm(torch.zeros(()), x, None, w, w)
