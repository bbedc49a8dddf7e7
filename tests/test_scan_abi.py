"""Refusals of the gated linear recurrence and of the layer norm (no GPU: every
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


def prefill(lib, **kw):
    a = dict(x=F, gate=F, h0=None, h=F + 4096, hT=F, states=None, off=None, B=2, T=5, D=64, ldx=64,
             ldg=128, kind=1, dt=0, ws=None, wsb=0)
    a.update(kw)
    return lib.gdn_scan_prefill(*a.values(), None)


def backward(lib, **kw):
    a = dict(x=F, gate=F, dh=F, h0=None, dhT=None, states=F, dx=F + 4096, dgate=F + 8192, dh0=None,
             off=None, B=2, T=5, D=64, ldx=64, ldg=128, kind=1, dt=0, ws=None, wsb=0)
    a.update(kw)
    return lib.gdn_scan_backward(*a.values(), None)


def step(lib, **kw):
    a = dict(x=F + 64, gate=F + 128, h=F, h_out=F, y=F + 4096, B=2, D=64, ldx=64, ldg=128, kind=1, dt=0)
    a.update(kw)
    return lib.gdn_scan_decode_step(*a.values(), None)


@pytest.mark.parametrize("call", [prefill, backward, step])
def test_shared_refusals(lib, call):
    for kw, want in ((dict(D=60), UNS), (dict(D=-8), INV), (dict(B=-1), INV), (dict(dt=2), INV),
                     (dict(kind=2), INV), (dict(kind=-1), INV), (dict(ldx=56), INV),
                     (dict(ldg=56), INV), (dict(ldx=68), INV), (dict(ldg=68), INV),
                     (dict(ldx=66, dt=1), INV), (dict(kind=0, ldg=66), INV),
                     (dict(ldx=1 << 40), INV), (dict(x=F + 8), ALI), (dict(gate=F + 4), ALI),
                     (dict(x=None), INV), (dict(gate=None), INV)):
        assert call(lib, **kw) == want, kw
    assert call(lib, B=0) == binding.GDN_OK
    assert call(lib, D=0, ldx=0, ldg=0) == binding.GDN_OK


def test_prefill_refusals(lib):
    for kw, want in ((dict(T=-1), INV), (dict(h=None, hT=None), INV), (dict(h=F), INV),
                     (dict(B=1 << 20, T=1 << 12), INV), (dict(T=(1 << 31) - 1, B=1), INV),
                     (dict(h=F + 8), ALI), (dict(h0=F + 4), ALI), (dict(hT=F + 8), ALI),
                     (dict(states=F + 4), ALI), (dict(off=F + 4), ALI), (dict(off=F), WS),
                     (dict(off=F, ws=F, wsb=16), WS), (dict(off=F, ws=F + 8, wsb=4096), ALI),
                     (dict(h0=F + 4096), INV), (dict(hT=F + 4096), INV), (dict(states=F), INV),
                     (dict(h0=F + 64, states=F + 64), INV), (dict(states=F + 4096), INV),
                     (dict(off=F, ws=F, wsb=4096, B=(1 << 31) - 1, D=8), INV)):
        assert prefill(lib, **kw) == want, kw


def test_backward_refusals(lib):
    for kw, want in ((dict(T=-1), INV), (dict(dh=None), INV), (dict(dx=None), INV),
                     (dict(dgate=None), INV), (dict(dx=F), INV), (dict(dgate=F), INV),
                     (dict(dgate=F + 4096), INV), (dict(dhT=F, dh0=F), INV), (dict(dh=F + 2), ALI), (dict(dhT=F + 4), ALI),
                     (dict(dh0=F + 4), ALI), (dict(states=F + 4), ALI), (dict(states=None), WS),
                     (dict(states=None, ws=F, wsb=16), WS), (dict(off=F), WS),
                     (dict(h0=F + 64, dh0=F + 64), INV)):
        assert backward(lib, **kw) == want, kw
    size = binding.gdn_scan_backward_workspace_size
    assert size(2, 5, 64, False, True) == 0
    assert size(2, 65, 64, False, False) >= 2 * 2 * 64 * 4
    assert size(2, 65, 64, True, True) >= 65 * 4
    assert size(2, 65, 64, True, False) >= 65 * 4 + 2 * 64 * 4
    assert size(0, 65, 64, True, False) == 0
    assert binding.gdn_scan_prefill_workspace_size(3, 65, 64, False) == 0
    assert binding.gdn_scan_prefill_workspace_size(3, 65, 64, True) >= 65 * 4


def test_step_refusals(lib):
    for kw, want in ((dict(h=None), INV), (dict(h_out=None), INV), (dict(y=F), INV),
                     (dict(y=F + 64), INV), (dict(y=F + 128), INV),
                     (dict(h_out=F + 64), INV), (dict(h_out=F + 128), INV),
                     (dict(h=F + 4), ALI), (dict(h_out=F + 4), ALI), (dict(y=F + 2), ALI)):
        assert step(lib, **kw) == want, kw


def norm(lib, **kw):
    a = dict(x=F, res=F, w=F, b=F, y=F + 4096, s=F + 8192, stats=F, N=3, D=64, ldx=64, ldr=128,
             eps=1e-5, dt=0)
    a.update(kw)
    return lib.gdn_layer_norm(*a.values(), None)


def norm_backward(lib, **kw):
    a = dict(s=F, dy=F, stats=F, w=F, ds=F, dx=F + 4096, dw=F + 4096, db=F + 8192, N=3, D=64,
             lds=64, dt=0, ws=F, wsb=1 << 30)
    a.update(kw)
    return lib.gdn_layer_norm_backward(*a.values(), None)


def test_layer_norm_refusals(lib):
    for kw, want in ((dict(N=-1), INV), (dict(N=1 << 50), INV), (dict(D=-8), INV),
                     (dict(D=60), UNS), (dict(D=16392), UNS), (dict(dt=2), INV),
                     (dict(eps=-1.0), INV), (dict(eps=float("nan")), INV), (dict(ldx=56), INV),
                     (dict(ldx=68), INV), (dict(ldr=56), INV), (dict(ldr=130), INV),
                     (dict(x=None), INV), (dict(y=None), INV), (dict(res=None), INV),
                     (dict(s=F + 4096), INV), (dict(y=F, ldx=128), INV), (dict(s=F), INV),
                     (dict(y=F, res=F + 64, ldx=72), INV)):
        assert norm(lib, **kw) == want, kw
    for x in ("x", "res", "w", "b", "y", "s", "stats"):
        assert norm(lib, **{x: F + 8}) == ALI, x
    assert norm(lib, N=0) == binding.GDN_OK
    assert norm(lib, D=0, ldx=0, ldr=0) == binding.GDN_OK


def test_layer_norm_backward_refusals(lib):
    for kw, want in ((dict(N=-1), INV), (dict(D=60), UNS), (dict(D=16392), UNS), (dict(dt=-1), INV),
                     (dict(lds=56), INV), (dict(lds=68), INV), (dict(s=None), INV),
                     (dict(dy=None), INV), (dict(stats=None), INV), (dict(dx=None), INV),
                     (dict(db=F + 4096), INV), (dict(dx=F, lds=128), INV), (dict(ws=None), WS),
                     (dict(wsb=16), WS)):
        assert norm_backward(lib, **kw) == want, kw
    for x in ("s", "dy", "stats", "w", "ds", "dx", "dw", "db", "ws"):
        assert norm_backward(lib, **{x: F + 8}) == ALI, x
    assert norm_backward(lib, N=0, dw=None, db=None) == binding.GDN_OK
    assert binding.gdn_layer_norm_backward_workspace_size(0, 64) == 0
    assert binding.gdn_layer_norm_backward_workspace_size(5, 64) >= 2 * 64 * 4


def test_wrapper_refusals(lib):
    """Shapes, types, strides and devices that the C boundary cannot see."""
    torch = pytest.importorskip("torch")
    x, g, h = torch.zeros(2, 5, 64), torch.zeros(2, 5, 64), torch.zeros(2, 64)

    def refuses(f, *a, **kw):
        with pytest.raises(binding.GDNError) as e:
            f(*a, **kw)
        assert e.value.status == INV
        return str(e.value)

    off = torch.tensor([0, 3, 5], dtype=torch.int32)
    for f, more in ((binding.scan_prefill, ()), (binding.scan_backward, (x,))):
        refuses(f, x, g, *more, kind="tanh")
        refuses(f, x, g[:, :4], *more)
        refuses(f, x, g.bfloat16(), *more)
        refuses(f, x.bfloat16(), g.bfloat16(), *more, kind="decay")
        refuses(f, x, g, *more, h0=torch.zeros(2, 60))
        refuses(f, x, g, *more, h0=h.double())
        refuses(f, x, g, *more, offsets=off)
        refuses(f, x[0], g[0], *(z[0] for z in more), offsets=off.long())
        refuses(f, x.transpose(1, 2).contiguous().transpose(1, 2), g, *more)
        refuses(f, torch.zeros(2, 7, 64)[:, :5], g, *more)  # uneven tokens
        refuses(f, torch.zeros(1, 5, 64).expand(2, 5, 64), g, *more)
        refuses(f, x, torch.zeros(2, 1, 64).expand(2, 5, 64), *more)
        assert "on the CPU" in refuses(f, x, g, *more)
    refuses(binding.scan_prefill, x, g, out_state=torch.zeros(2, 5, 64))
    refuses(binding.scan_backward, x, g, x[:, :4])
    refuses(binding.scan_backward, x, g, x, states=torch.zeros(2, 2, 64))
    refuses(binding.scan_backward, x, g, x, dh_T=torch.zeros(3, 64))
    refuses(binding.scan_decode_step, x, g, h)
    refuses(binding.scan_decode_step, x[:, 0], g[:, 0], h[:1])
    refuses(binding.scan_decode_step, x[:, 0], g[:, 0], h.bfloat16())
    refuses(binding.scan_decode_step, x[:, 0], g[:, 0], h, kind="rate")
    refuses(binding.scan_decode_step, x[:, 0], g[:, 0], h, y=torch.zeros(2, 60))
    assert "on the CPU" in refuses(binding.scan_decode_step, x[:, 0], g[:, 0], h)
    w, st = torch.ones(64), torch.zeros(2, 5, 2)
    refuses(binding.layer_norm, x, w.bfloat16())
    refuses(binding.layer_norm, x, torch.ones(60))
    refuses(binding.layer_norm, x, w, w, residual=x[:, :4])
    refuses(binding.layer_norm, x, w, w, residual=x.bfloat16())
    refuses(binding.layer_norm, x, w, residual=x, out=(x, None))
    refuses(binding.layer_norm, x, w, out=(x.bfloat16(), None))
    refuses(binding.layer_norm, torch.zeros(1, 5, 64).expand(2, 5, 64), w)
    refuses(binding.layer_norm_backward, x, x[:, :4], st, w)
    refuses(binding.layer_norm_backward, x, x, torch.zeros(2, 5), w)
    refuses(binding.layer_norm_backward, x, x, st, w, ds=x.bfloat16())
    assert "on the CPU" in refuses(binding.layer_norm, x, w)
    assert "on the CPU" in refuses(binding.layer_norm_backward, x, x, st, w)
