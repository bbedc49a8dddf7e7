"""Calls whose `stream` argument is not torch's current stream: what they
allocate for themselves is theirs until that stream is done with it."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    torch = pytest.importorskip("torch")
    from gated_delta_rule_49_gb300 import binding
    binding.load()
    return torch


def calls(torch):
    """name: (the C call that gets the workspace, a call given the stream), each with scratch
    memory of its own."""
    from gated_delta_rule_49_gb300 import binding
    g = torch.Generator(device="cuda").manual_seed(0)

    def normal(*shape, dtype=torch.bfloat16):
        return torch.randn(shape, generator=g, device="cuda").to(dtype)

    q, k, v, do = (normal(1, 3000, 2, 128) for _ in range(4))
    alpha = torch.tensor([0.9, 0.999], device="cuda")
    pos, f = torch.arange(3000, device="cuda")[None], torch.ones(64, device="cuda")
    w = torch.ones(128, device="cuda")
    unit = torch.nn.functional.normalize
    at, bt = (torch.rand((1, 3000, 2), generator=g, device="cuda") * 0.1 + 0.9 for _ in range(2))
    qn, kn = unit(q.float(), dim=-1).bfloat16(), unit(k.float(), dim=-1).bfloat16()
    channel = torch.rand((1, 3000, 2, 128), generator=g, device="cuda") * 0.1 + 0.9
    state = torch.randn(1, 2, 128, 128, generator=g, device="cuda")
    gram = binding.channel_gram(kn, qn)
    idx = torch.stack([torch.randperm(128, generator=g, device="cuda")[:64].sort()[0]] * 2).int()
    return {
        "linear_prefill": ("gdn_linear_prefill", lambda s: binding.linear_prefill(
            q, k, v, alpha, stream=s)),
        "linear_backward": ("gdn_linear_backward", lambda s: binding.linear_backward(
            q, k, v, alpha, do, stream=s)),
        "qk_norm_rotate_backward": (
            "gdn_qk_norm_rotate_backward", lambda s: binding.qk_norm_rotate_backward(
                q, k, pos, f, q, k, w, w, stream=s)),
        "prefill": ("gdn_prefill", lambda s: binding.prefill(qn, kn, v, at, bt, stream=s)),
        "prefill_gated_chunked": (
            "gdn_prefill_gated_chunked", lambda s: binding.prefill_gated_chunked(
                qn, kn, v, channel, bt, stream=s)),
        "prefill_truncated": ("gdn_prefill_truncated", lambda s: binding.prefill_truncated(
            qn, kn, v, at, bt, seg_len=1500, stream=s)),
        "prefill_gathered": ("gdn_prefill_gathered", lambda s: binding.prefill_gathered(
            qn, kn, idx, v, at, bt, stream=s)),
        "channel_gram": ("gdn_channel_gram", lambda s: binding.channel_gram(qn, kn, stream=s)),
        # without scratch memory
        "qk_norm_rotate": (None, lambda s: binding.qk_norm_rotate(q, k, pos, f, w, w, stream=s)),
        "linear_decode_step": (None, lambda s: binding.linear_decode_step(
            q[:, 0], k[:, 0], v[:, 0], alpha, state, stream=s)),
        "decode_step": (None, lambda s: binding.decode_step(
            qn[:, 0], kn[:, 0], v[:, 0], at[:, 0], bt[:, 0], state, stream=s)),
        "prefill_gated": (None, lambda s: binding.prefill_gated(
            qn[:, :40].contiguous(), kn[:, :40].contiguous(), v[:, :40].contiguous(),
            channel[:, :40].contiguous(), bt[:, :40].contiguous(), stream=s)),
        "gather_normalize": (None, lambda s: binding.gather_normalize(qn, idx, stream=s)),
        "drrqr_select": (None, lambda s: binding.drrqr_select(gram, 64, stream=s)),
        "state_rank": (None, lambda s: binding.state_rank(state, stream=s)),
        "state_truncate": (None, lambda s: binding.state_truncate(
            state, 32, want_sigma=True, stream=s)),
    }


SCRATCH = ["linear_prefill", "linear_backward", "qk_norm_rotate_backward", "prefill",
         "prefill_gated_chunked", "prefill_truncated", "prefill_gathered", "channel_gram"]
NAMES = SCRATCH + ["qk_norm_rotate", "linear_decode_step", "decode_step", "prefill_gated",
                   "gather_normalize", "drrqr_select", "state_rank", "state_truncate"]


def tensors(x):
    return [y for y in (x if isinstance(x, tuple) else (x,)) if y is not None]


@pytest.mark.parametrize("as_handle", [False, True])
@pytest.mark.parametrize("name", SCRATCH)
def test_workspace_is_not_given_out_while_in_use(torch, name, as_handle, monkeypatch):
    """The other stream is busy when the call is made, so that its kernels have not run when the
    current stream allocates again; what it then writes must not be theirs."""
    from gated_delta_rule_49_gb300 import binding
    c_call, run = calls(torch)[name]
    want = [x.clone() for x in tensors(run(None))]
    torch.cuda.synchronize()
    taken = []
    whole = getattr(binding, c_call)

    def spy(*a, **kw):
        for x in list(a) + list(kw.values()):
            if isinstance(x, torch.Tensor) and x.dtype is torch.uint8:
                taken.append((x.data_ptr(), x.numel()))
        return whole(*a, **kw)

    monkeypatch.setattr(binding, c_call, spy)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        torch.cuda._sleep(2_000_000)
    got = tensors(run(s.cuda_stream if as_handle else s))
    (at, size), = taken
    again = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in (size, size, size)]
    torch.cuda.synchronize()
    for x in again:
        assert x.data_ptr() + x.numel() <= at or at + size <= x.data_ptr()
    assert len(got) == len(want) and all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("name", NAMES)
def test_outputs_that_are_dropped_at_once(torch, name):
    """An output that the caller lets go of is not given out before it has been written."""
    run = calls(torch)[name][1]
    sizes = [(x.shape, x.dtype) for x in tensors(run(None))]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        torch.cuda._sleep(2_000_000)
    run(s)
    again = [torch.zeros(shape, dtype=dtype, device="cuda") for shape, dtype in sizes]
    torch.cuda.synchronize()
    assert not any(x.any() for x in again)


def test_both_streams_at_work(torch):
    """Two cut prompts on two streams, and a third on the current one, with other inputs each."""
    from gated_delta_rule_49_gb300 import binding
    g = torch.Generator(device="cuda").manual_seed(1)
    alpha = torch.tensor([0.99, 0.9999], device="cuda")
    sets = [[torch.randn(1, 9000, 2, 128, generator=g, device="cuda").bfloat16() for _ in range(3)]
            for _ in range(3)]
    want = [binding.linear_prefill(*x, alpha) for x in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream(), None]
    for _ in range(10):
        got = [binding.linear_prefill(*x, alpha, stream=s) for x, s in zip(sets, streams)]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(x, y) for x, y in zip(a, b))
