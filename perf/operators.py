"""Cases of the query/key norm with rotation and of linear attention with a decay for each head.

``run`` computes an operator either in its plain form (elementary torch
operations in 32 bits, rounded once at the end) or through the library.

Norm and rotation, for every token and head (x one head's channels):

    r = (c sum x^2 + eps)^(-1/2),  c = 1/D ("rms") or 1 ("l2")
    y = rotate(w * x * r)          pairs (i, i + R/2) or (2i, 2i + 1), i < R/2,
                                   by the angle pos * inv_freq[i]

Linear attention, for every sequence and head (a = alpha[h]):

    S_t = a S_{t-1} + v_t k_t^T,   o_t = scale S_t q_t
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
EPS = 1e-6
BASE = 10000.0


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one token of one user on its way into the step below: launch latency
        dict(name="norm-step", op="norm", B=1, T=1, Hq=16, Hk=16, D=128, R=128, norm="rms",
             pairing="half", weight=True, first=70000, dtype="bf16"),
        # the queries and keys of a batch of prompts
        dict(name="norm-prompt", op="norm", B=8, T=4096, Hq=16, Hk=16, D=128, R=128, norm="rms",
             pairing="half", weight=True, first=0, dtype="bf16"),
        # odd lengths in float32: fewer key heads, half of the channels rotated, adjacent pairs
        dict(name="norm-odd-fp32", op="norm", B=3, T=1003, Hq=12, Hk=4, D=64, R=32, norm="l2",
             pairing="adjacent", weight=False, first=500, dtype="fp32"),
        # the same layer in a training step: gradients of both inputs and both weights
        dict(name="norm-train", op="norm_back", B=8, T=4096, Hq=16, Hk=16, D=128, R=128,
             norm="rms", pairing="half", weight=True, first=0, dtype="bf16"),
        # answering one user, a token at a time
        dict(name="step-1", op="step", B=1, Hq=16, H=16, K=128, V=128, dtype="bf16"),
        # answering a full batch of users
        dict(name="step-64", op="step", B=64, Hq=16, H=16, K=128, V=128, dtype="bf16"),
        # a batch of prompts, end states kept for the answers
        dict(name="prompt", op="prefill", B=8, T=4096, Hq=16, H=16, K=128, V=128, start=False,
             state=True, dtype="bf16"),
        # one very long prompt
        dict(name="long", op="prefill", B=1, T=65536, Hq=16, H=16, K=128, V=128, start=False,
             state=True, dtype="bf16"),
        # prompts of very different lengths packed one after another, keys of half the width shared
        # by two heads, continuing from earlier states; one has no tokens, one a single one
        dict(name="packed", op="packed", lens="1,0,700,64,129,2048,127,5,1530,333,128,911",
             Hq=8, H=16, K=64, V=128, start=True, dtype="bf16"),
        # the smallest recurrence, in float32
        dict(name="tiny-fp32", op="prefill", B=1, T=256, Hq=1, H=1, K=32, V=32, start=False,
             state=True, dtype="fp32"),
        # a training step on full sequences
        dict(name="train", op="back", B=8, T=4096, Hq=16, H=16, K=128, V=128, start=False,
             dtype="bf16"),
        # a short odd training window that starts from a carried state, in float32
        dict(name="train-odd-fp32", op="back", B=2, T=391, Hq=2, H=4, K=64, V=128, start=True,
             dtype="fp32"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm_back", "step", "prefill", "packed", "back"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    if op in ("norm", "norm_back"):
        D = rng.choice([64, 128, 128, 256])
        Hq = rng.choice([1, 4, 6, 12, 16])
        Hk = rng.choice([h for h in (1, 2, 4, 6, 16) if h <= Hq])
        most = 8 * 4096 * 32 * 128 // ((Hq + Hk) * D) // (2 if dtype == "fp32" else 1)
        T = _log_int(rng, 1, min(most, 16384))
        return dict(op=op, B=_log_int(rng, 1, max(1, min(16, most // T))), T=T, Hq=Hq, Hk=Hk, D=D,
                    R=rng.choice([D, D // 2]), norm=rng.choice(["rms", "l2"]),
                    pairing=rng.choice(["half", "adjacent"]), weight=rng.random() < 0.7,
                    first=rng.randrange(100000), dtype=dtype)
    K, V = rng.choice([(64, 64), (64, 128), (128, 128), (128, 128)])
    H = rng.choice([1, 2, 4, 8, 16])
    Hq = rng.choice([h for h in (H, H, H // 2) if h >= 1])
    if op == "step":
        return dict(op=op, B=_log_int(rng, 1, 128), Hq=Hq, H=H, K=K, V=V, dtype=dtype)
    most = 8 * 4096 * 16 // H // (8 if dtype == "fp32" else 1)
    if op == "packed":
        lens, left = [], min(most, 16384)
        for _ in range(rng.randint(1, 12)):
            n = min(left, rng.choice([0, 1, _log_int(rng, 2, 4096), _log_int(rng, 2, 4096)]))
            lens.append(n)
            left -= n
        if sum(lens) == 0:
            lens.append(rng.randint(1, 200))
        return dict(op=op, lens=",".join(map(str, lens)), Hq=Hq, H=H, K=K, V=V,
                    start=rng.random() < 0.5, dtype=dtype)
    T = _log_int(rng, 1, min(most, 32768 if dtype == "bf16" else 2048))
    B = _log_int(rng, 1, max(1, min(16, most // T)))
    case = dict(op=op, B=B, T=T, Hq=Hq, H=H, K=K, V=V, start=rng.random() < 0.5, dtype=dtype)
    if op == "prefill":
        case["state"] = rng.random() < 0.7
    return case


# ------------------------------------------------------------------ inputs

def _lens(case):
    return [int(n) for n in case["lens"].split(",")]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    dt = DTYPES[case["dtype"]]

    def normal(*shape, to=dt):
        return torch.randn(shape, generator=g, device="cuda").to(to)

    s = dict(case)
    if case["op"] in ("norm", "norm_back"):
        B, T, D, R = case["B"], case["T"], case["D"], case["R"]
        for n, h in (("q", case["Hq"]), ("k", case["Hk"])):
            s[n] = normal(B, T, h, D)
            s["w" + n] = 1 + 0.2 * normal(D, to=torch.float32) if case["weight"] else None
            if case["op"] == "norm_back":
                s["dy" + n] = normal(B, T, h, D)
        s["pos"] = (torch.arange(T, device="cuda") + case["first"]).repeat(B, 1)
        s["inv_freq"] = BASE ** (-torch.arange(0, R, 2, device="cuda", dtype=torch.float32) / R)
        return s
    H, Hq, K, V = case["H"], case["Hq"], case["K"], case["V"]
    # one decay a head, horizons from a few tokens to thousands
    u = torch.rand(H, generator=g, device="cuda")
    s["alpha"] = 1 - 2 ** -(0.5 + 11 * (torch.arange(H, device="cuda") + u) / H)
    s["scale"] = K ** -0.5
    if case["op"] == "step":
        B = case["B"]
        s.update(q=normal(B, Hq, K), k=normal(B, Hq, K), v=normal(B, H, V),
                 S=normal(B, H, V, K, to=torch.float32))
        s["S_out"], s["o"] = torch.empty_like(s["S"]), torch.empty_like(s["v"])
        return s
    if case["op"] == "packed":
        lens = _lens(case)
        lead, N = (sum(lens),), len(lens)
        s["offsets"] = torch.tensor([sum(lens[:i]) for i in range(N + 1)], dtype=torch.int32,
                                    device="cuda")
    else:
        lead, N = (case["B"], case["T"]), case["B"]
        s["offsets"] = None
    s.update(q=normal(*lead, Hq, K), k=normal(*lead, Hq, K), v=normal(*lead, H, V))
    s["S0"] = normal(N, H, V, K, to=torch.float32) if case["start"] else None
    if case["op"] == "back":
        s["do"] = normal(*lead, H, V)
        s["dS_T"] = normal(N, H, V, K, to=torch.float32) if case["start"] else None
    return s


# ------------------------------------------------------------------ plain forms

def _cos_sin(s):
    angle = s["pos"].double()[..., None] * s["inv_freq"].double()
    return angle.cos().float()[..., None, :], angle.sin().float()[..., None, :]


def _turn(x, cos, sin, s):
    half = s["R"] // 2
    if s["pairing"] == "half":
        a, b, rest = x[..., :half], x[..., half:2 * half], x[..., 2 * half:]
        return torch.cat([a * cos - b * sin, a * sin + b * cos, rest], -1)
    a, b, rest = x[..., :2 * half:2], x[..., 1:2 * half:2], x[..., 2 * half:]
    return torch.cat([torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2), rest], -1)


def _rnorm(x, s):
    c = 1 / s["D"] if s["norm"] == "rms" else 1.0
    return c, (c * (x * x).sum(-1, keepdim=True) + EPS).rsqrt()


def _norm(x, w, cos, sin, s):
    y = x.float()
    y = y * _rnorm(y, s)[1]
    return _turn(y if w is None else y * w, cos, sin, s).to(x.dtype)


def _norm_back(x, w, dy, cos, sin, s):
    xf = x.float()
    c, r = _rnorm(xf, s)
    g = _turn(dy.float(), cos, -sin, s)
    dw = None if w is None else (g * xf * r).flatten(0, -2).sum(0)
    g = g if w is None else g * w
    dx = r * (g - c * r * r * xf * (xf * g).sum(-1, keepdim=True))
    return dx.to(x.dtype), dw


def _core(q, k, v, a):
    """sum_{s <= t} a^(t - s) (q_t . k_s) v_s and the end state, from a zero start; q, k [N, H, T, *]."""
    N, H, T, _ = q.shape
    C = min(128, T)
    n = -(-T // C)
    q, k, v = (torch.nn.functional.pad(x, (0, 0, n * C - T, 0)).unflatten(2, (n, C))
               for x in (q, k, v))
    i = torch.arange(C, device=q.device)
    lag = i[:, None] - i
    within = torch.where(lag >= 0, a[:, None, None] ** lag.clamp(min=0), 0.0)
    written = (v * (a[:, None] ** (C - 1 - i))[:, None, :, None]).transpose(-1, -2) @ k
    j = torch.arange(n, device=q.device)
    gap = j[:, None] - 1 - j
    carry = torch.where(gap >= 0, a[:, None, None] ** (C * gap.clamp(min=0)), 0.0)
    start = (carry @ written.flatten(-2)).view_as(written)
    o = ((q @ k.transpose(-1, -2)) * within[:, None]) @ v
    o = o + (a[:, None] ** (i + 1))[:, None, :, None] * (q @ start.transpose(-1, -2))
    end = a[:, None, None] ** C * start[:, :, -1] + written[:, :, -1]
    return o.flatten(2, 3)[:, :, n * C - T:], end


def _heads(x, H):
    """[N, T, Hx, D] -> [N, H, T, D] in 32 bits, each of the Hx heads repeated for its group."""
    return x.float().repeat_interleave(H // x.shape[2], 2).transpose(1, 2)


def _prefill(q, k, v, a, S0, scale, n):
    """Dense linear attention; the n real tokens (one number a sequence) stand at the end of T."""
    H, T = v.shape[2], v.shape[1]
    q, k, v = _heads(q, H), _heads(k, H), _heads(v, H)
    o, S = _core(q, k, v, a)
    if S0 is not None:
        past = torch.arange(T, device=v.device) + 1 + n[:, None] - T
        o = o + (a[:, None] ** past.clamp(min=0)[:, None])[..., None] * (q @ S0.transpose(-1, -2))
        S = S + (a ** n[:, None])[..., None, None] * S0
    return (scale * o).transpose(1, 2), S


def _run_prefill(s):
    n = torch.full((s["B"],), s["T"], device="cuda")
    o, S = _prefill(s["q"], s["k"], s["v"], s["alpha"], s["S0"], s["scale"], n)
    o = o.to(s["v"].dtype)
    return (o, S) if s["state"] else o


def _run_packed(s):
    off = s["offsets"].long()
    n = off[1:] - off[:-1]
    T = max(1, max(_lens(s)))
    at = torch.arange(T, device="cuda") + (n - T)[:, None]  # token of each place, real ones last
    real = at >= 0
    where = (off[:-1, None] + at).clamp(min=0, max=s["v"].shape[0] - 1)
    q, k, v = (torch.where(real[..., None, None], s[x][where], 0.0) for x in "qkv")
    o, S = _prefill(q, k, v, s["alpha"], s["S0"], s["scale"], n)
    return o[real].to(s["v"].dtype), S


def _run_back(s):
    a, T, H, scale = s["alpha"], s["T"], s["H"], s["scale"]
    q, k, v, do = (_heads(s[x], H) for x in ("q", "k", "v", "do"))
    do = do * scale
    dq = _core(do, v, k, a)[0]
    q, k, v, do = (x.flip(2) for x in (q, k, v, do))
    dk = _core(v, do, q, a)[0]
    dv, end = _core(k, q, do, a)
    dS0 = None
    if s["S0"] is not None:
        late = (a[:, None] ** torch.arange(T, device="cuda"))[..., None]  # flipped tokens
        dq = dq + (late * a[:, None, None]) * (do.flip(2) @ s["S0"])
        dk = dk + late * (v @ s["dS_T"])
        dv = dv + late * (k @ s["dS_T"].transpose(-1, -2))
        dS0 = a[:, None, None] * end + (a ** T)[:, None, None] * s["dS_T"]
    dk, dv = dk.flip(2), dv.flip(2)
    group = (s["Hq"], H // s["Hq"])
    dq, dk = (x.unflatten(1, group).sum(2) for x in (dq, dk))
    return tuple(x.transpose(1, 2).to(s["v"].dtype) for x in (dq, dk, dv)) + (dS0,)


def _run_step(s):
    B, H, Hq = s["B"], s["H"], s["Hq"]
    q, k = (s[x].float().repeat_interleave(H // Hq, 1) for x in "qk")
    v = s["v"].float()
    S = s["alpha"][:, None, None] * s["S"] + v[..., :, None] * k[..., None, :]
    return (s["scale"] * (S * q[..., None, :]).sum(-1)).to(s["v"].dtype), S


def _run_norm(s):
    cos, sin = _cos_sin(s)
    return _norm(s["q"], s["wq"], cos, sin, s), _norm(s["k"], s["wk"], cos, sin, s)


def _run_norm_back(s):
    cos, sin = _cos_sin(s)
    dq, dwq = _norm_back(s["q"], s["wq"], s["dyq"], cos, sin, s)
    dk, dwk = _norm_back(s["k"], s["wk"], s["dyk"], cos, sin, s)
    return dq, dk, dwq, dwk


PLAIN = {"norm": _run_norm, "norm_back": _run_norm_back, "step": _run_step,
         "prefill": _run_prefill, "packed": _run_packed, "back": _run_back}


# ------------------------------------------------------------------ the framework's calls

def _run_own(s):
    from gated_delta_rule_49_gb300 import binding
    op = s["op"]
    if op == "norm":
        return binding.qk_norm_rotate(s["q"], s["k"], s["pos"], s["inv_freq"], s["wq"], s["wk"],
                                      norm=s["norm"], pairing=s["pairing"], eps=EPS)
    if op == "norm_back":
        return binding.qk_norm_rotate_backward(s["q"], s["k"], s["pos"], s["inv_freq"], s["dyq"],
                                               s["dyk"], s["wq"], s["wk"], norm=s["norm"],
                                               pairing=s["pairing"], eps=EPS)
    if op == "step":
        o = binding.linear_decode_step(s["q"], s["k"], s["v"], s["alpha"], s["S"],
                                       scale=s["scale"], S_out=s["S_out"], o=s["o"])
        return o, s["S_out"]
    if op == "back":
        return binding.linear_backward(s["q"], s["k"], s["v"], s["alpha"], s["do"], S0=s["S0"],
                                       dS_T=s["dS_T"], scale=s["scale"])
    state = s.get("state", True)
    o, S = binding.linear_prefill(s["q"], s["k"], s["v"], s["alpha"], S0=s["S0"],
                                  scale=s["scale"], offsets=s["offsets"], want_state=state)
    return (o, S) if state else o


def run(state):
    return _run_own(state) if own else PLAIN[state["op"]](state)


# ------------------------------------------------------------------ cost

def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    op = case["op"]
    if op in ("norm", "norm_back"):
        n = case["B"] * case["T"] * (case["Hq"] + case["Hk"]) * case["D"]
        return {"bytes": n * e * (2 if op == "norm" else 3) + 8 * case["B"] * case["T"],
                "flops": n * (8 if op == "norm" else 18)}
    H, Hq, K, V = case["H"], case["Hq"], case["K"], case["V"]
    state = 4 * V * K * H
    if op == "step":
        B = case["B"]
        return {"bytes": B * (2 * state + e * (2 * Hq * K + 2 * H * V)), "flops": 5 * B * H * V * K}
    if op == "packed":
        tokens, N = sum(_lens(case)), len(_lens(case))
    else:
        tokens, N = case["B"] * case["T"], case["B"]
    if op == "back":
        return {"bytes": tokens * e * (4 * Hq * K + 3 * H * V) + (3 * N * state if case["start"] else 0),
                "flops": 12 * tokens * H * V * K}
    states = (1 if case["start"] else 0) + (1 if case.get("state", True) else 0)
    return {"bytes": tokens * e * 2 * (Hq * K + H * V) + states * N * state,
            "flops": 4 * tokens * H * V * K}


# ------------------------------------------------------------------ 64 bits, from the definition

def _blocks(q, k, v, a, S, scale):
    """One block of tokens after another, the state carried between them; [N, T, H, *] in 64 bits."""
    outs, T, size = [], q.shape[1], 64
    for t in range(0, T, size):
        m = min(size, T - t)
        x, y, z = (u[:, t:t + m] for u in (q, k, v))
        i = torch.arange(m, device=a.device, dtype=torch.float64)
        decay = torch.tril(a[:, None, None] ** (i[:, None] - i).clamp(min=0))
        o = torch.einsum("nthk,nshk,hts,nshv->nthv", x, y, decay, z) if m == 1 else torch.einsum(
            "nhts,nshv->nthv", torch.einsum("nthk,nshk->nhts", x, y) * decay, z)
        past = (a[None] ** (i[:, None] + 1))[None, ..., None]
        outs.append(scale * (o + past * torch.einsum("nhvk,nthk->nthv", S, x)))
        left = (a[None] ** (m - 1 - i[:, None]))[None, ..., None]
        S = a[:, None, None] ** m * S + torch.einsum("nshv,nshk->nhvk", z * left, y)
    return torch.cat(outs, 1) if outs else torch.empty_like(v), S


def _exact_linear(q, k, v, a, S0, scale):
    H = v.shape[2]
    q, k = (x.repeat_interleave(H // x.shape[2], 2) for x in (q, k))
    if S0 is None:
        S0 = torch.zeros(v.shape[0], H, v.shape[3], k.shape[3], device=v.device, dtype=v.dtype)
    return _blocks(q, k, v, a, S0, scale)


def _exact_norm(x, w, s):
    x = x.double() if not x.dtype == torch.float64 else x
    D, R = s["D"], s["R"]
    size = (x.square().mean(-1, keepdim=True) if s["norm"] == "rms"
            else x.square().sum(-1, keepdim=True)) + EPS
    y = x / size.sqrt()
    if w is not None:
        y = y * w
    first = torch.arange(R // 2, device=x.device) * (1 if s["pairing"] == "half" else 2)
    second = first + (R // 2 if s["pairing"] == "half" else 1)
    angle = (s["pos"].double()[..., None] * s["inv_freq"].double())[..., None, :]
    z = torch.complex(y[..., first], y[..., second]) * torch.polar(torch.ones_like(angle), angle)
    out = y.clone()
    out[..., first] = z.real
    out[..., second] = z.imag
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        return _exact_norm(s["q"], _double(s["wq"]), s), _exact_norm(s["k"], _double(s["wk"]), s)
    if op == "norm_back":
        got = {}
        for x in "qk":  # the gradient of (y . dy), one input after the other
            leaf = s[x].double().requires_grad_()
            w = None if s["w" + x] is None else s["w" + x].double().requires_grad_()
            y = _exact_norm(leaf, w, s)
            got[x] = torch.autograd.grad(y, [leaf] + ([] if w is None else [w]),
                                         s["dy" + x].double())
        return (got["q"][0], got["k"][0], got["q"][1] if case["weight"] else None,
                got["k"][1] if case["weight"] else None)
    a = s["alpha"].double()
    q, k, v, S0 = (_double(s.get(x)) for x in ("q", "k", "v", "S0"))
    if op == "step":
        o, S = _exact_linear(q[:, None], k[:, None], v[:, None], a, s["S"].double(), s["scale"])
        return o[:, 0], S
    if op == "packed":
        outs, ends, t = [], [], 0
        for i, n in enumerate(_lens(case)):
            o, S = _exact_linear(q[None, t:t + n], k[None, t:t + n], v[None, t:t + n], a,
                                 None if S0 is None else S0[i:i + 1], s["scale"])
            outs.append(o[0])
            ends.append(S)
            t += n
        return torch.cat(outs), torch.cat(ends)
    if op == "prefill":
        o, S = _exact_linear(q, k, v, a, S0, s["scale"])
        return (o, S) if case["state"] else o
    parts = []
    for b in range(case["B"]):  # the gradient of (o . do + S_T . dS_T), sequence by sequence
        leaves = [x[b:b + 1].detach().requires_grad_() for x in (q, k, v)]
        if S0 is not None:
            leaves.append(S0[b:b + 1].detach().requires_grad_())
        o, S = _exact_linear(*leaves[:3], a, leaves[3] if S0 is not None else None, s["scale"])
        loss = (o * s["do"][b:b + 1].double()).sum()
        if S0 is not None:
            loss = loss + (S * s["dS_T"][b:b + 1].double()).sum()
        parts.append(torch.autograd.grad(loss, leaves))
    got = tuple(torch.cat(x) for x in zip(*parts))
    return got if S0 is not None else got + (None,)


def _double(x):
    return None if x is None else x.double()
