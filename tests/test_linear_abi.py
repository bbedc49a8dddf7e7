"""Refusals of the norm with rotation and of linear attention (no GPU: every
call fails its checks before anything is launched)."""
import pytest

from gated_delta_rule_49_gb300 import binding, build

F = 0x10000  # aligned, never read
INV, UNS, ALI, WS = (binding.GDN_ERR_INVALID_ARG, binding.GDN_ERR_UNSUPPORTED,
                     binding.GDN_ERR_ALIGNMENT, binding.GDN_ERR_WORKSPACE)


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load()


def norm(lib, back=False, **kw):
    a = dict(q=F, k=F, wq=F, wk=F, pos=F, f=F, dyq=F, dyk=F, yq=F + 4096, yk=F + 8192, dwq=F, dwk=F,
             N=3, Hq=4, Hk=2, D=128, R=64, ldq=512, ldk=256, norm=0, pair=0, eps=1e-6, dt=0,
             ws=F, wsb=1 << 30)
    a.update(kw)
    ins = [a[x] for x in ("q", "k", "wq", "wk", "pos", "f")]
    sizes = [a[x] for x in ("N", "Hq", "Hk", "D", "R", "ldq", "ldk", "norm", "pair", "eps", "dt")]
    if not back:
        return lib.gdn_qk_norm_rotate(*ins, a["yq"], a["yk"], *sizes, None)
    return lib.gdn_qk_norm_rotate_backward(*ins, a["dyq"], a["dyk"], a["yq"], a["yk"], a["dwq"],
                                           a["dwk"], *sizes, a["ws"], a["wsb"], None)


@pytest.mark.parametrize("back", [False, True])
def test_norm_refusals(lib, back):
    for kw, want in ((dict(D=96), UNS), (dict(D=512), UNS), (dict(R=24), UNS), (dict(R=256), INV),
                     (dict(R=-16), INV), (dict(N=-1), INV), (dict(N=1 << 50), INV),
                     (dict(Hq=-1), INV), (dict(Hk=1 << 20), INV), (dict(dt=2), INV),
                     (dict(norm=2), INV), (dict(pair=-1), INV), (dict(eps=-1.0), INV),
                     (dict(eps=float("nan")), INV), (dict(ldq=511), INV), (dict(ldq=500), INV),
                     (dict(ldk=260), INV), (dict(q=None), INV), (dict(k=None), INV),
                     (dict(pos=None), INV), (dict(f=None), INV), (dict(yq=None), INV),
                     (dict(q=F + 2), ALI), (dict(wk=F + 4), ALI), (dict(pos=F + 8), ALI),
                     (dict(yk=F + 8), ALI)):
        assert norm(lib, back, **kw) == want, kw


def test_norm_in_place_needs_dense_rows(lib):
    assert norm(lib, yq=F, ldq=768) == INV
    assert norm(lib, yk=F, ldk=768) == INV


def test_norm_backward_refusals(lib):
    assert norm(lib, True, wq=None) == INV  # a gradient of a weight that is not there
    assert norm(lib, True, dyk=None) == INV
    assert norm(lib, True, dyq=F + 4) == ALI
    assert norm(lib, True, ws=None) == WS
    assert norm(lib, True, wsb=16) == WS


def test_norm_of_nothing(lib):
    assert norm(lib, N=0) == binding.GDN_OK
    assert norm(lib, Hq=0, Hk=0, q=None, k=None) == binding.GDN_OK
    assert norm(lib, True, N=0, dwq=None, dwk=None) == binding.GDN_OK


def prefill(lib, **kw):
    a = dict(q=F, k=F, v=F, al=F, S0=None, o=F, ST=F, off=None, B=2, T=5, Hq=2, H=4, K=128, V=128,
             ldq=256, ldk=256, ldv=512, scale=1.0, dt=0, ws=None, wsb=0)
    a.update(kw)
    return lib.gdn_linear_prefill(*a.values(), None)


def backward(lib, **kw):
    a = dict(q=F, k=F, v=F, al=F, do=F, S0=None, dST=None, dq=F, dk=F, dv=F, dS0=None, off=None,
             B=2, T=5, Hq=4, H=4, K=128, V=128, ldq=512, ldk=512, ldv=512, scale=1.0, dt=0, ws=None,
             wsb=0)
    a.update(kw)
    return lib.gdn_linear_backward(*a.values(), None)


@pytest.mark.parametrize("call", [prefill, backward])
def test_linear_refusals(lib, call):
    for kw, want in ((dict(K=96), UNS), (dict(K=128, V=64), UNS), (dict(K=32, V=64), UNS),
                     (dict(K=0), INV), (dict(B=-1), INV), (dict(T=-1), INV), (dict(H=-1), INV),
                     (dict(Hq=3), INV), (dict(Hq=0), INV), (dict(dt=3), INV), (dict(ldq=8), INV),
                     (dict(ldk=516), INV), (dict(ldv=508), INV), (dict(B=1 << 20, H=64, Hq=64, ldq=8192, ldk=8192, ldv=8192), INV),
                     (dict(k=None), INV), (dict(v=None), INV), (dict(q=None), INV),
                     (dict(al=None), INV), (dict(v=F + 8), ALI), (dict(S0=F + 4), ALI),
                     (dict(off=F + 4), ALI)):
        assert call(lib, **kw) == want, kw
    assert call(lib, B=0) == binding.GDN_OK


def test_linear_wants_an_output(lib):
    assert prefill(lib, o=None, ST=None) == INV
    assert backward(lib, dq=None, dk=None, dv=None) == INV
    assert backward(lib, do=None) == INV


def test_linear_workspace(lib):
    size = binding.gdn_linear_prefill_workspace_size
    # a long sequence on one head is cut; enough sequences are not
    need = size(1, 65536, 1, 32, 32, False, binding.GDN_FP32)
    assert need > 0
    assert size(64, 4096, 16, 128, 128, False, binding.GDN_FP32) == 0
    assert size(1, 65536, 1, 96, 32, False, binding.GDN_FP32) == 0
    one = dict(B=1, T=65536, Hq=1, H=1, K=32, V=32, ldq=32, ldk=32, ldv=32, dt=1)
    assert prefill(lib, **one) == WS
    assert prefill(lib, **one, ws=F, wsb=need - 1) == WS
    assert backward(lib, **one) == WS
    # the parts of shared gradients
    back = binding.gdn_linear_backward_workspace_size
    assert back(2, 5, 1, 4, 64, 128, False, 0) >= 2 * 5 * 4 * 64 * 4
    assert backward(lib, Hq=1, ws=F, wsb=8) == WS


def test_step_refusals(lib):
    def step(**kw):
        a = dict(q=F, k=F, v=F, al=F, S=F, So=F, o=F, B=2, Hq=2, H=4, K=64, V=128, scale=1.0, dt=0)
        a.update(kw)
        return lib.gdn_linear_decode_step(*a.values(), None)

    for x in ("q", "k", "v", "al", "S", "So", "o"):
        assert step(**{x: None}) == INV
        assert step(**{x: F + 4}) == ALI
    assert step(K=48) == UNS
    assert step(Hq=3) == INV
    assert step(dt=9) == INV
    assert step(B=-2) == INV
    assert step(B=0) == binding.GDN_OK


def test_wrapper_refusals(lib):
    """Shapes, types and strides that the C boundary cannot see."""
    torch = pytest.importorskip("torch")
    q, v = torch.zeros(2, 5, 2, 64), torch.zeros(2, 5, 4, 128)
    al = torch.ones(4)

    def refuses(f, *a, **kw):
        with pytest.raises(binding.GDNError) as e:
            f(*a, **kw)
        assert e.value.status == INV

    refuses(binding.linear_prefill, q, q, v, torch.ones(3))
    refuses(binding.linear_prefill, q, q, v, al.double())
    refuses(binding.linear_prefill, q, q[:, :4], v, al)
    refuses(binding.linear_prefill, q, q, v[:, :4], al)
    refuses(binding.linear_prefill, q, q, v.bfloat16(), al)
    refuses(binding.linear_prefill, q.transpose(-1, -2).contiguous().transpose(-1, -2), q, v, al)
    refuses(binding.linear_prefill, q, q, v.transpose(1, 2).contiguous().transpose(1, 2), al)
    refuses(binding.linear_prefill, torch.zeros(2, 7, 2, 64)[:, :5], q, v, al)  # uneven tokens
    refuses(binding.linear_prefill, q, q, v, al, S0=torch.zeros(2, 4, 64, 128))
    refuses(binding.linear_prefill, q, q, v, al, offsets=torch.zeros(3, dtype=torch.int32))
    refuses(binding.linear_prefill, q[0], q[0], v[0], al, offsets=torch.zeros(3, dtype=torch.int64))
    refuses(binding.linear_backward, q, q, v, al, v[:, :, :2])
    refuses(binding.linear_backward, q, q, v, al, v.transpose(0, 1).contiguous().transpose(0, 1))
    refuses(binding.linear_decode_step, q[:, 0], q[:, 0], v[:, 0], al, torch.zeros(2, 4, 128, 64))
    pos, f = torch.zeros(2, 5, dtype=torch.int64), torch.ones(32)
    refuses(binding.qk_norm_rotate, q, q, pos.int(), f)
    refuses(binding.qk_norm_rotate, q, q, pos[:, :4], f)
    refuses(binding.qk_norm_rotate, q, q[..., :32], pos, f)
    refuses(binding.qk_norm_rotate, q, q, pos, f, norm="max")
    refuses(binding.qk_norm_rotate, q, q, pos, f, pairing="thirds")
    refuses(binding.qk_norm_rotate, q, q, pos, f, wq=torch.ones(63))
    refuses(binding.qk_norm_rotate, q, q, pos, f, out=(q, q.bfloat16()))
    refuses(binding.qk_norm_rotate_backward, q, q, pos, f, q, q[:, :4])
