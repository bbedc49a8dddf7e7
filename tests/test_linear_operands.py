"""Operands of linear attention and of the norm with rotation that the wrappers
must turn away themselves: the C boundary sees one token stride and trusts it
(no GPU: every call fails before anything is launched)."""
import pytest

from gated_delta_rule_49_gb300 import binding, build

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return binding.load()


def refused(why, f, *a, **kw):
    with pytest.raises(binding.GDNError, match=why) as e:
        f(*a, **kw)
    assert e.value.status == binding.GDN_ERR_INVALID_ARG


# tokens 2 x 5 of 4 heads; what has no memory of its own for every token
BROADCAST = {
    "over the tokens of each sequence": lambda D: torch.zeros(2, 1, 4, D).expand(2, 5, 4, D),
    "over all tokens": lambda D: torch.zeros(1, 1, 4, D).expand(2, 5, 4, D),
    "over the sequences": lambda D: torch.zeros(1, 5, 4, D).expand(2, 5, 4, D),
    "tokens that overlap": lambda D: torch.zeros(10 * 4 * D).as_strided(
        (2, 5, 4, D), (5 * 2 * D, 2 * D, D, 1)),
}


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("how", BROADCAST)
def test_broadcast_tokens_are_refused(how, D):
    x, bad = torch.zeros(2, 5, 4, D), BROADCAST[how](D)
    alpha, pos, f = torch.ones(4), torch.zeros(2, 5, dtype=torch.int64), torch.ones(16)
    for i in range(3):
        ops = [bad if j == i else x for j in range(3)]
        refused("evenly", binding.linear_prefill, *ops, alpha)
        refused("evenly", binding.linear_backward, *ops, alpha, x)
    for q, k in ((bad, x), (x, bad), (bad, None)):
        refused("evenly", binding.qk_norm_rotate, q, k, pos, f)
        refused("evenly", binding.qk_norm_rotate_backward, q, k, pos, f, x, None if k is None else x)


def test_broadcast_packed_tokens_are_refused():
    x, bad = torch.zeros(7, 4, 64), torch.zeros(4, 64).expand(7, 4, 64)
    alpha, offsets = torch.ones(4), torch.tensor([0, 3, 7], dtype=torch.int32)
    for i in range(3):
        ops = [bad if j == i else x for j in range(3)]
        refused("evenly", binding.linear_prefill, *ops, alpha, offsets=offsets)
        refused("evenly", binding.linear_backward, *ops, alpha, x, offsets=offsets)


def test_strides_of_what_has_memory():
    """Slices of a projection, single tokens and single sequences keep their strides."""
    def stride(x):
        return binding._token_stride("test", "x", x, x.dtype, x.get_device())

    wide = torch.zeros(2, 5, 6, 64)
    assert stride(wide[:, :, 1:4]) == 6 * 64
    assert stride(wide[:, :1, 1:4]) == 5 * 6 * 64
    assert stride(wide[1:, :, 2:4]) == 6 * 64
    assert stride(wide[:1, :1, 1:4]) == 3 * 64  # one token: any
    assert stride(torch.zeros(1, 1, 4, 64).expand(1, 1, 4, 64)) == 4 * 64
    assert stride(wide[:0, :, :3]) == 3 * 64
    assert stride(wide[:, :, 2:3]) == 6 * 64
    assert stride(wide[1, 2, 1:4]) == 3 * 64  # no leading dimension


def test_host_tensors_are_refused():
    """All on the CPU, so that they agree with one another: host pointers must not reach a kernel."""
    q, v, S = torch.zeros(2, 5, 4, 64), torch.zeros(2, 5, 4, 128), torch.zeros(2, 4, 128, 64)
    alpha, pos, f = torch.ones(4), torch.zeros(2, 5, dtype=torch.int64), torch.ones(32)
    refused("on the CPU", binding.linear_prefill, q, q, v, alpha, S0=S)
    refused("on the CPU", binding.linear_prefill, q[0], q[0], v[0], alpha,
            offsets=torch.tensor([0, 5], dtype=torch.int32))
    refused("on the CPU", binding.linear_backward, q, q, v, alpha, v)
    refused("on the CPU", binding.linear_decode_step, q[:, 0].contiguous(), q[:, 0].contiguous(),
            v[:, 0].contiguous(), alpha, S)
    refused("on the CPU", binding.qk_norm_rotate, q, q, pos, f)
    refused("on the CPU", binding.qk_norm_rotate_backward, q, q, pos, f, q, q)


def test_addresses_of_any_whole_number_type():
    """A raw address may come as a subclass of int (an enum's, a wrapper's own)."""
    class Address(int):
        pass

    assert binding._ptr(Address(0x10000)) == 0x10000
    assert binding._ptr(0x10000) == 0x10000 and binding._ptr(None) is None
    x = torch.zeros(4)
    assert binding._ptr(x) == x.data_ptr()
