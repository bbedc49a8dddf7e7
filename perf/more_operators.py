"""Cases of the gated linear recurrence over channels and of the layer norm.

``run`` computes an operator either in its plain form (elementary torch
operations in 32 bits, rounded once at the end) or through the library.

Recurrence, for every sequence and channel:

    h_t = a_t h_{t-1} + b_t x_t
    "decay"     a_t is given (float32), b_t = 1
    "sigmoid"   a_t = 1 / (1 + exp(-g_t)), b_t = 1 - a_t

Layer norm, for every row (s = x, or x + residual rounded to the type):

    y = (s - mean) / sqrt(var + eps) * w + b
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
EPS = 1e-5
BLOCK = 64  # tokens between the states that a forward pass keeps for the gradients


# ------------------------------------------------------------------ cases

def listed():
    return [
        # answering one user, a token at a time: launch latency
        dict(name="scan-step-1", op="step", B=1, D=2048, kind="sigmoid", dtype="bf16"),
        # answering a full batch of users
        dict(name="scan-step-256", op="step", B=256, D=2048, kind="sigmoid", dtype="bf16"),
        # a batch of prompts, end states kept for the answers
        dict(name="scan-prompt", op="scan", B=8, T=4096, D=2048, kind="sigmoid", start=False,
             dtype="bf16"),
        # one very long prompt, with decays that the caller has formed
        dict(name="scan-long", op="scan", B=1, T=65536, D=2048, kind="decay", start=False,
             dtype="bf16"),
        # prompts of very different lengths packed one after another, continuing from earlier
        # states; one has no tokens, two a single one
        dict(name="scan-packed", op="packed", lens="1,0,700,64,129,2048,127,5,1530,1,128,911",
             D=2048, kind="sigmoid", start=True, dtype="bf16"),
        # a training step on full sequences: gradients of the inputs and the gates
        dict(name="scan-train", op="back", B=8, T=4096, D=2048, kind="sigmoid", start=False,
             dtype="bf16"),
        # a short odd training window that starts from a carried state, in float32
        dict(name="scan-train-odd-fp32", op="back", B=3, T=391, D=1000, kind="decay", start=True,
             dtype="fp32"),
        # one token on its way into a layer, with the sum that goes on past it
        dict(name="norm-step", op="norm", rows=1, D=2048, residual=True, bias=True, dtype="bf16"),
        # a batch of prompts on its way into a layer
        dict(name="norm-prompt", op="norm", rows=8 * 4096, D=2048, residual=True, bias=True,
             dtype="bf16"),
        # every head of a layer's output on its own
        dict(name="norm-heads", op="norm", rows=8 * 4096 * 16, D=128, residual=False, bias=False,
             dtype="bf16"),
        # a training step on full sequences: gradients of the input and of both weights, with the
        # gradient that comes past the layer
        dict(name="norm-train", op="norm_back", rows=8 * 4096, D=2048, residual=True, bias=True,
             dtype="bf16"),
        # odd rows of an odd width in float32
        dict(name="norm-train-odd-fp32", op="norm_back", rows=3 * 1003, D=1000, residual=False,
             bias=False, dtype="fp32"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["step", "scan", "packed", "back", "norm", "norm_back"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    most = 8 * 4096 * 2048 // (2 if dtype == "fp32" else 1)
    if op in ("norm", "norm_back"):
        D = rng.choice([64, 128, 512, 2048, 8 * _log_int(rng, 8, 1024)])
        return dict(op=op, rows=_log_int(rng, 1, most // D), D=D, residual=rng.random() < 0.6,
                    bias=rng.random() < 0.6, dtype=dtype)
    D = rng.choice([512, 2048, 8 * _log_int(rng, 8, 512)])
    kind = rng.choice(["decay", "sigmoid", "sigmoid"])
    if kind == "decay":
        most //= 2
    if op == "step":
        return dict(op=op, B=_log_int(rng, 1, 512), D=D, kind=kind, dtype=dtype)
    if op == "packed":
        lens, left = [], min(most // D, 16384)
        for _ in range(rng.randint(1, 12)):
            n = min(left, rng.choice([0, 1, _log_int(rng, 2, 4096), _log_int(rng, 2, 4096)]))
            lens.append(n)
            left -= n
        if sum(lens) == 0:
            lens.append(rng.randint(1, 200))
        return dict(op=op, lens=",".join(map(str, lens)), D=D, kind=kind,
                    start=rng.random() < 0.5, dtype=dtype)
    T = _log_int(rng, 1, min(most // D, 32768 if op == "scan" else 8192))
    B = _log_int(rng, 1, max(1, min(16, most // D // T)))
    return dict(op=op, B=B, T=T, D=D, kind=kind, start=rng.random() < 0.5, dtype=dtype)


# ------------------------------------------------------------------ inputs

def _lens(case):
    return [int(n) for n in case["lens"].split(",")]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    dt = DTYPES[case["dtype"]]
    D = case["D"]

    def normal(*shape, to=dt):
        return torch.randn(shape, generator=g, device="cuda").to(to)

    s = dict(case)
    if case["op"] in ("norm", "norm_back"):
        N = case["rows"]
        # channels of different sizes about means of their own, as a residual stream has them
        size = torch.exp(0.5 * normal(D, to=torch.float32))
        x = (normal(N, D, to=torch.float32) + 0.3 * normal(D, to=torch.float32)) * size
        s["w"] = 1 + 0.2 * normal(D, to=torch.float32)
        s["b"] = 0.1 * normal(D, to=torch.float32) if case["bias"] else None
        s["x"] = x.to(dt)
        s["residual"] = normal(N, D) if case["residual"] else None
        if case["op"] == "norm_back":
            # the sum and the statistics are the forward pass's
            s["x"] = _sum(s["x"], s["residual"])
            s["stats"] = _stats(s["x"].float())
            s["dy"] = normal(N, D)
            s["ds"] = normal(N, D) if case["residual"] else None
        return s
    if case["op"] == "step":
        lead, N = (case["B"],), case["B"]
    elif case["op"] == "packed":
        lens = _lens(case)
        lead, N = (sum(lens),), len(lens)
        s["offsets"] = torch.tensor([sum(lens[:i]) for i in range(N + 1)], dtype=torch.int32,
                                    device="cuda")
    else:
        lead, N = (case["B"], case["T"]), case["B"]
    s["x"] = normal(*lead, D)
    # horizons from a token or two to thousands, by channel
    gate = normal(*lead, D, to=torch.float32) + torch.linspace(0, 7.5, D, device="cuda")
    s["gate"] = torch.sigmoid(gate) if case["kind"] == "decay" else gate.to(dt)
    if case["op"] == "step":
        s["h"] = normal(N, D, to=torch.float32)
        s["h_out"], s["y"] = torch.empty_like(s["h"]), torch.empty_like(s["x"])
        return s
    s["h0"] = normal(N, D, to=torch.float32) if case["start"] else None
    if case["op"] == "back":
        s["dh"] = normal(*lead, D)
        s["dh_T"] = normal(N, D, to=torch.float32) if case["start"] else None
        # what the forward pass has kept: the state before every 64th token
        h = _before(_forward(s), s["h0"])
        s["states"] = h[:, ::BLOCK].contiguous()
    return s


# ------------------------------------------------------------------ plain forms

def _coefficients(s):
    """a and b x in 32 bits."""
    x = s["x"].float()
    if s["kind"] == "decay":
        return s["gate"], x
    g = s["gate"].float()
    return 1 / (1 + torch.exp(-g)), x / (1 + torch.exp(g))


def _doubling(a, u, dim):
    """h_t = a_t h_{t-1} + u_t from zero, by doubling the reach of each token."""
    T, reach = a.shape[dim], 1
    while reach < T:
        late = (slice(None),) * dim + (slice(reach, None),)
        soon = (slice(None),) * dim + (slice(None, T - reach),)
        keep = (slice(None),) * dim + (slice(None, reach),)
        u = torch.cat([u[keep], u[late] + a[late] * u[soon]], dim)
        a = torch.cat([a[keep], a[late] * a[soon]], dim)
        reach *= 2
    return u


def _forward(s):
    """[B, T, D] -> the states after each token."""
    a, u = _coefficients(s)
    if s["h0"] is not None:
        u = torch.cat([u[:, :1] + a[:, :1] * s["h0"][:, None], u[:, 1:]], 1)
    return _doubling(a, u, 1)


def _before(h, h0):
    first = torch.zeros_like(h[:, :1]) if h0 is None else h0[:, None]
    return torch.cat([first, h[:, :-1]], 1)


def _run_scan(s):
    h = _forward(s)
    return h.to(s["x"].dtype), h[:, -1].contiguous()


def _run_packed(s):
    a, u = _coefficients(s)
    off = s["offsets"].long()
    some = off[1:] > off[:-1]
    first = off[:-1][some]
    h0 = torch.zeros(len(off) - 1, s["D"], device="cuda") if s["h0"] is None else s["h0"]
    u, a = u.clone(), a.clone()
    u[first] += a[first] * h0[some]
    a[first] = 0
    h = _doubling(a, u, 0)
    end = h0.clone()
    end[some] = h[off[1:][some] - 1]
    return h.to(s["x"].dtype), end


def _run_back(s):
    a, _ = _coefficients(s)
    x, dh = s["x"].float(), s["dh"].float()
    if s["dh_T"] is not None:
        dh = torch.cat([dh[:, :-1], dh[:, -1:] + s["dh_T"][:, None]], 1)
    # G_t = dh_t + a_{t+1} G_{t+1}, the last token first
    later = torch.cat([torch.zeros_like(a[:, :1]), a[:, 1:].flip(1)], 1)
    G = _doubling(later, dh.flip(1), 1).flip(1)
    past = _before(_forward(s), s["h0"])
    dh0 = None if s["h0"] is None else a[:, 0] * G[:, 0]
    if s["kind"] == "decay":
        return G.to(s["x"].dtype), G * past, dh0
    b = 1 / (1 + torch.exp(s["gate"].float()))
    dt = s["x"].dtype
    return (G * b).to(dt), (G * (past - x) * a * b).to(dt), dh0


def _run_step(s):
    a, u = _coefficients(s)
    h = a * s["h"] + u
    return h.to(s["x"].dtype), h


def _sum(x, residual):
    return x if residual is None else (x.float() + residual.float()).to(x.dtype)


def _stats(s):
    """[N, 2]: mean and 1 / sqrt(var + eps) of each row."""
    mean = s.mean(-1, keepdim=True)
    var = (s - mean).square().mean(-1, keepdim=True)
    return torch.cat([mean, (var + EPS).rsqrt()], -1)


def _run_norm(s):
    z = _sum(s["x"], s["residual"])
    f = z.float()
    stats = _stats(f)
    y = (f - stats[:, :1]) * stats[:, 1:] * s["w"]
    if s["b"] is not None:
        y = y + s["b"]
    y = y.to(z.dtype)
    return y if s["residual"] is None else (y, z)


def _run_norm_back(s):
    mean, rstd = s["stats"][:, :1], s["stats"][:, 1:]
    dy = s["dy"].float()
    n = (s["x"].float() - mean) * rstd
    g = dy * s["w"]
    dx = rstd * (g - g.mean(-1, keepdim=True) - n * (g * n).mean(-1, keepdim=True))
    if s["ds"] is not None:
        dx = dx + s["ds"].float()
    return dx.to(s["x"].dtype), (dy * n).sum(0), dy.sum(0) if s["bias"] else None


PLAIN = {"step": _run_step, "scan": _run_scan, "packed": _run_packed, "back": _run_back,
         "norm": _run_norm, "norm_back": _run_norm_back}


# ------------------------------------------------------------------ the framework's calls

def _run_own(s):
    from gated_delta_rule_49_gb300 import binding
    op = s["op"]
    if op == "norm":
        y, z, _ = binding.layer_norm(s["x"], s["w"], s["b"], residual=s["residual"], eps=EPS)
        return y if z is None else (y, z)
    if op == "norm_back":
        return binding.layer_norm_backward(s["x"], s["dy"], s["stats"], s["w"], ds=s["ds"],
                                           want_db=s["bias"])
    if op == "step":
        y = binding.scan_decode_step(s["x"], s["gate"], s["h"], kind=s["kind"], h_out=s["h_out"],
                                     y=s["y"])
        return y, s["h_out"]
    if op == "back":
        return binding.scan_backward(s["x"], s["gate"], s["dh"], h0=s["h0"], dh_T=s["dh_T"],
                                     states=s["states"], kind=s["kind"])
    h, h_T, _ = binding.scan_prefill(s["x"], s["gate"], h0=s["h0"], kind=s["kind"],
                                     offsets=s.get("offsets"))
    return h, h_T


def run(state):
    return _run_own(state) if own else PLAIN[state["op"]](state)


# ------------------------------------------------------------------ cost

def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    op, D = case["op"], case["D"]
    if op in ("norm", "norm_back"):
        n = case["rows"] * D
        if op == "norm":
            return {"bytes": n * e * (4 if case["residual"] else 2) + 8 * D, "flops": 8 * n}
        return {"bytes": n * e * (4 if case["residual"] else 3) + 8 * case["rows"] + 12 * D,
                "flops": 13 * n}
    eg = 4 if case["kind"] == "decay" else e
    if op == "step":
        return {"bytes": case["B"] * D * (8 + 2 * e + eg), "flops": 8 * case["B"] * D}
    if op == "packed":
        tokens, N = sum(_lens(case)), len(_lens(case))
    else:
        tokens, N = case["B"] * case["T"], case["B"]
    states = 4 * N * D * (2 if case["start"] else 1)
    if op == "back":
        kept = 4 * N * -(-case["T"] // BLOCK) * D
        return {"bytes": tokens * D * (3 * e + 2 * eg) + kept + (2 * states if case["start"] else 0),
                "flops": 16 * tokens * D}
    return {"bytes": tokens * D * (2 * e + eg) + states, "flops": 8 * tokens * D}


# ------------------------------------------------------------------ 64 bits, from the definition

def _one_by_one(x, gate, h, kind):
    """The recurrence token by token; x, gate [T, N, D] in 64 bits.  (states after each, last)."""
    a = gate if kind == "decay" else torch.sigmoid(gate)
    outs = []
    for t in range(x.shape[0]):
        h = torch.addcmul(x[t], a[t], h) if kind == "decay" else torch.lerp(x[t], h, a[t])
        outs.append(h)
    return (torch.stack(outs) if outs else x), h


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        z = _sum(s["x"], s["residual"])
        y = _exact_norm(z.double(), s["w"].double(), _double(s["b"]))
        return y if s["residual"] is None else (y, z.double())
    if op == "norm_back":
        x, w = s["x"].double().requires_grad_(), s["w"].double().requires_grad_()
        y = _exact_norm(x, w, None)
        dx, dw = torch.autograd.grad(y, [x, w], s["dy"].double())
        if s["ds"] is not None:
            dx = dx + s["ds"].double()
        return dx, dw, s["dy"].double().sum(0) if s["bias"] else None
    x, gate, kind = s["x"].double(), s["gate"].double(), case["kind"]
    if op == "step":
        h = _one_by_one(x[None], gate[None], s["h"].double(), kind)[1]
        return h, h
    N = len(_lens(case)) if op == "packed" else case["B"]
    h0 = torch.zeros(N, case["D"], device="cuda", dtype=torch.float64)
    if s["h0"] is not None:
        h0 = s["h0"].double()
    if op == "packed":
        outs, ends, t = [], [], 0
        for i, n in enumerate(_lens(case)):
            h, end = _one_by_one(x[t:t + n, None], gate[t:t + n, None], h0[i:i + 1], kind)
            outs.append(h[:, 0])
            ends.append(end)
            t += n
        return torch.cat(outs), torch.cat(ends)
    if op == "scan":
        h, end = _one_by_one(x.transpose(0, 1), gate.transpose(0, 1), h0, kind)
        return h.transpose(0, 1), end
    leaves = [x.requires_grad_(), gate.requires_grad_(), h0.requires_grad_()]
    h, end = _one_by_one(x.transpose(0, 1), gate.transpose(0, 1), h0, kind)
    loss = (h.transpose(0, 1) * s["dh"].double()).sum()
    if s["dh_T"] is not None:
        loss = loss + (end * s["dh_T"].double()).sum()
    dx, dgate, dh0 = torch.autograd.grad(loss, leaves)
    return dx, dgate, dh0 if case["start"] else None


def _exact_norm(x, w, b):
    centred = x - x.sum(-1, keepdim=True) / x.shape[-1]
    y = centred / ((centred * centred).sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt() * w
    return y if b is None else y + b


def _double(x):
    return None if x is None else x.double()
