"""What the gated-delta-rule calls refuse, before anything is launched (no device needed)."""
import pytest
import torch

from kda_delta_rule_chunkwise_b200 import binding
from kda_delta_rule_chunkwise_b200 import build as kbuild

BAD, NOT = binding.KDA_ERR_INVALID_ARG, binding.KDA_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    kbuild.build()
    return binding.load()


def prefill(lib, **kw):
    a = dict(q=16, k=32, v=48, g=64, beta=80, state_in=None, cu=None, B=1, T=16, N=1, Hk=2, H=4, dk=128, dv=128,
             dtype=binding.KDA_BF16, o=96, state_out=None, workspace=256, workspace_bytes=1 << 40, stream=None)
    a.update(kw)
    return lib.kda_gdr_chunk_prefill(*a.values())


@pytest.mark.parametrize("bad", [
    dict(B=-1), dict(T=-1), dict(N=-1), dict(N=2), dict(Hk=0), dict(H=0), dict(Hk=3), dict(dk=0), dict(dv=-64),
    dict(dtype=2), dict(cu=4, B=2, N=2), dict(q=None), dict(k=None), dict(v=None), dict(g=None), dict(beta=None),
    dict(o=None), dict(q=17), dict(k=40), dict(v=8), dict(o=100), dict(state_in=4), dict(state_out=8),
    dict(workspace=None), dict(workspace=272), dict(workspace_bytes=100)])
def test_prefill_refuses(lib, bad):
    assert prefill(lib, **bad) == BAD


@pytest.mark.parametrize("bad", [dict(dk=96), dict(dv=32), dict(dk=256), dict(T=2 ** 31), dict(B=2 ** 16, N=2 ** 16, T=2 ** 16),
                                 dict(cu=4, N=2 ** 28)])
def test_prefill_does_not_support(lib, bad):
    assert prefill(lib, **bad) == NOT


def test_prefill_workspace(lib):
    f = lib.kda_gdr_prefill_workspace_bytes
    need = f(100, 2, 2, 4, 128, 64, binding.KDA_BF16)
    assert need > 0 and need % 256 == 0 and f(100, 3, 2, 4, 128, 64, binding.KDA_BF16) > need
    assert f(100, 2, 2, 4, 128, 64, binding.KDA_F32) == 0 and f(100, 2, 3, 4, 128, 64, binding.KDA_BF16) == 0
    assert prefill(lib, workspace_bytes=f(16, 1, 2, 4, 128, 128, binding.KDA_BF16) - 1) == BAD


def test_prefill_of_nothing(lib):
    assert prefill(lib, B=0, N=0, q=None, k=None, v=None, g=None, beta=None, o=None) == binding.KDA_OK


def decode(lib, **kw):
    a = dict(q=16, k=32, v=48, g=64, beta=80, state=96, slots=None, lens=None, N=4, P=4, L=1, Hk=2, H=4, dk=128, dv=64,
             dtype=binding.KDA_BF16, update=1, o=112, stream=None)
    a.update(kw)
    return lib.kda_gdr_decode(*a.values())


@pytest.mark.parametrize("bad", [dict(N=-1), dict(P=-1), dict(P=3), dict(L=-1), dict(H=5), dict(dtype=9), dict(q=None),
                                 dict(state=None), dict(o=None), dict(state=100), dict(Hk=0)])
def test_decode_refuses(lib, bad):
    assert decode(lib, **bad) == BAD


def test_decode_sizes(lib):
    assert decode(lib, dk=32) == NOT and decode(lib, N=2 ** 27, P=2 ** 27) == NOT
    assert decode(lib, N=0, P=0) == binding.KDA_OK and decode(lib, L=0) == binding.KDA_OK


def backward(lib, **kw):
    a = dict(q=16, k=32, v=48, g=64, beta=80, state_in=None, cu=None, B=1, T=16, N=1, Hk=2, H=4, dk=128, dv=128,
             dtype=binding.KDA_BF16, dout=96, dstate_out=None, dq=112, dk_out=128, dv_out=144, dg=160, dbeta=176,
             dstate_in=None, workspace=256, workspace_bytes=1 << 40, stream=None)
    a.update(kw)
    return lib.kda_gdr_backward(*a.values())


@pytest.mark.parametrize("bad", [
    dict(B=-1), dict(N=2), dict(Hk=3), dict(dtype=2), dict(q=None), dict(dout=None), dict(dq=None), dict(dk_out=None),
    dict(dv_out=None), dict(dg=None), dict(dbeta=None), dict(dout=100), dict(dv_out=8), dict(dstate_out=4),
    dict(workspace=None), dict(workspace=272), dict(workspace_bytes=1000)])
def test_backward_refuses(lib, bad):
    assert backward(lib, **bad) == BAD


@pytest.mark.parametrize("bad", [dict(dk=96), dict(dv=256), dict(T=2 ** 31)])
def test_backward_does_not_support(lib, bad):
    assert backward(lib, **bad) == NOT


def test_backward_workspace(lib):
    f = lib.kda_gdr_backward_workspace_bytes
    for t in (binding.KDA_BF16, binding.KDA_F32):
        need = f(100, 2, 2, 4, 128, 64, t)
        assert need > 0 and need % 256 == 0 and f(100, 3, 2, 4, 128, 64, t) > need
        assert f(-1, 2, 2, 4, 128, 64, t) == 0 and f(100, 2, 3, 4, 128, 64, t) == 0 and f(100, 2, 2, 4, 96, 64, t) == 0
        assert backward(lib, dtype=t, workspace_bytes=f(16, 1, 2, 4, 128, 128, t) - 1) == BAD
    assert backward(lib, B=0, N=0) == binding.KDA_OK


def test_binding_refuses_other_shapes_types_and_devices():
    q = torch.zeros(1, 4, 2, 64, dtype=torch.bfloat16)
    v, g = torch.zeros(1, 4, 4, 64, dtype=torch.bfloat16), torch.zeros(1, 4, 4, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        binding.kda_gdr_chunk_prefill(q, q, v, g, g)
    with pytest.raises(ValueError, match="bf16 or fp32"):
        binding.kda_gdr_chunk_prefill(q.half(), q, v, g, g)
    with pytest.raises(ValueError, match="four dimensions"):
        binding.kda_gdr_decode(q[0], q[0], v[0], g[0], g[0], torch.zeros(1, 4, 64, 64))
    for bad, match in ((q[:, :2], "shape"), (q.float(), "must be torch.bfloat16")):
        with pytest.raises(ValueError, match=match):
            binding._want("k", bad, q.shape, q.dtype, q.device)
    with pytest.raises(ValueError, match="contiguous"):
        binding._want("k", q.transpose(1, 2), (1, 2, 4, 64), q.dtype, q.device)


def test_binding_refuses_a_stream_of_another_device():
    class Elsewhere:
        device = torch.device("cuda", 7)
    q = torch.zeros(1, 4, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="stream"):
        binding.kda_gdr_chunk_prefill(q, q, q, q, q, stream=Elsewhere())


def test_binding_takes_every_argument_by_name():
    """All arguments by keyword, with and without a stream: refused for the tensors' sake alone."""
    class Elsewhere:
        device = torch.device("cuda", 7)
    q = torch.zeros(1, 4, 2, 64, dtype=torch.bfloat16)
    x = torch.zeros(3, 64, dtype=torch.bfloat16)
    calls = [(binding.kda_gdr_chunk_prefill, dict(beta=q, g=q, v=q, k=q, q=q)),
             (binding.kda_gdr_decode, dict(q=q, k=q, v=q, g=q, beta=q, state=q)),
             (binding.kda_gdr_backward, dict(q=q, k=q, v=q, g=q, beta=q, state_in=None, cu_seqlens=None, dout=q)),
             (binding.kda_block_norm, dict(eps=1e-6, x=x, y=x, gate=None, w_post=x, w_pre=x)),
             (binding.kda_block_norm_backward, dict(x=x, y=x, gate=None, w_post=x, w_pre=x, dx_new=x, dh=x))]
    for call, arguments in calls:
        with pytest.raises(ValueError):
            call(**arguments)
        with pytest.raises(ValueError, match="the stream is on"):
            call(**arguments, stream=Elsewhere())


@pytest.mark.parametrize("strided", [torch.zeros(1, dtype=torch.uint8).expand(4096), torch.zeros(8192, dtype=torch.uint8)[::2]])
def test_a_workspace_with_strides_is_refused(strided):
    """Its element count says nothing about the memory behind its address."""
    with pytest.raises(ValueError, match="workspace must be contiguous"):
        binding._space(strided, 1024, strided.device)
    whole = torch.zeros(4096, dtype=torch.uint8)
    assert binding._space(whole, 1024, whole.device) == (whole, 4096) and binding._space(None, 0, whole.device) == (None, 0)


def test_second_derivatives_are_refused_not_dropped(monkeypatch):
    """With stand-ins for the kernels: y^2 and its gradient."""
    monkeypatch.setattr(binding, "kda_block_norm", lambda x, y, *_, **__: (x * x, y * y))
    monkeypatch.setattr(binding, "kda_block_norm_backward",
                        lambda x, y, g, wo, wi, a, b, **_: (2 * x * a, 2 * y * b, None, wo * 0, wi * 0))
    x, y, w = (torch.randn(4, requires_grad=True) for _ in range(3))
    a, b = binding.kda_block_norm_autograd(x, y, None, w, w)
    grads = torch.autograd.grad(a.sum() + b.sum(), (x, y, w), create_graph=True)
    assert torch.equal(grads[0], 2 * x) and torch.equal(grads[1], 2 * y) and (grads[2] == 0).all()
    with pytest.raises(RuntimeError, match="second derivative"):
        (a.sum() + grads[1].square().sum()).backward()
    a, b = binding.kda_block_norm_autograd(x, y, None, w, w)
    (a.sum() + b.sum()).backward()
    assert torch.equal(x.grad, 2 * x) and not x.grad.requires_grad


def test_sizes_whose_workspace_no_number_holds_are_refused(lib):
    """2^26 chunks of 2^27 heads are more bytes than 64 bits count: a wrapped sum would take any workspace."""
    huge = dict(T=2 ** 31 - 128, Hk=1, H=2 ** 27, workspace_bytes=2 ** 63)
    assert prefill(lib, **huge) == NOT and backward(lib, **huge) == NOT
    for f in (lib.kda_gdr_prefill_workspace_bytes, lib.kda_gdr_backward_workspace_bytes):
        assert f(2 ** 31 - 128, 1, 1, 2 ** 27, 128, 128, binding.KDA_BF16) == 0
        assert f(2 ** 31 - 128, 1, 1, 2 ** 9, 128, 128, binding.KDA_BF16) > 2 ** 40
