"""The feed-forward operators: what is measured, with their plain forms.

Three operators, as a transformer block uses them:

- ``linear``:   Y = act(X W^T + b) + alpha v + R, one linear with the
  activation, the steering add and the residual add in its epilogue;
- ``gated``:    H = act(X Wg^T + bg) * (X Wu^T + bu), the gated half of a
  feed-forward block, with the pre-activations kept where a training step
  needs them;
- ``backward``: the gradients of ``gated`` with respect to its inputs,
  weights and biases, from the kept pre-activations.

Weights are q8 (int8, one fp32 scale per output channel), q4 (nibbles in
groups of 32 along K, one fp16 scale per group), w8a8 (the q8 pack with int8
activations and one fp32 scale per token) or f16. Everything else is fp16.
"""
import math

import torch

own = False

D = "cuda"
FORMATS = ("q8", "q4", "w8a8", "f16")
ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")


def _linear(name, fmt, M, N, K, act, residual=True, steer=False):
    return {"name": name, "op": "linear", "fmt": fmt, "M": M, "N": N, "K": K, "act": act, "residual": residual,
            "steer": steer}


def _gated(name, fmt, M, N, K, act, save=False):
    return {"name": name, "op": "gated", "fmt": fmt, "M": M, "N": N, "K": K, "act": act, "save": save}


def _backward(name, M, N, K, act):
    return {"name": name, "op": "backward", "fmt": "f16", "M": M, "N": N, "K": K, "act": act}


def listed():
    return [
        # one token through the down projection of a d = 1024 block: latency
        _linear("linear_q8_m1_down", "q8", 1, 1024, 4096, "none"),
        # the attention output projection of the d = 1536 layer sequence, at
        # 2 x 216 latent frames, at the block whose residual stream is steered
        _linear("linear_w8a8_m432_out_steered", "w8a8", 432, 1536, 1536, "none", steer=True),
        # the down projection at the smallest weight format
        _linear("linear_q4_m432_down", "q4", 432, 1536, 6144, "none"),
        # the down projection over a long clip, the fastest precision
        _linear("linear_w8a8_m4096_down", "w8a8", 4096, 1536, 6144, "none"),
        # an ungated feed-forward's up projection over a long clip
        _linear("linear_f16_m4096_up", "f16", 4096, 6144, 1536, "gelu", residual=False),
        # one token through the gated half: both weight matrices are read once
        _gated("gated_q4_m1", "q4", 1, 6144, 1536, "silu"),
        # odd sizes in every direction
        _gated("gated_f16_m203_ragged", "f16", 203, 1040, 592, "gelu_tanh"),
        # a denoising step of the small block
        _gated("gated_q8_m432", "q8", 432, 4096, 1024, "gelu"),
        # a long clip, the fastest precision
        _gated("gated_w8a8_m4096", "w8a8", 4096, 6144, 1536, "silu"),
        # the forward pass of a training step: the pre-activations are kept
        _gated("gated_f16_m4096_train", "f16", 4096, 6144, 1536, "silu", save=True),
        # the backward pass at one clip's frames, and over a full batch
        _backward("backward_m432", 432, 4096, 1024, "gelu"),
        _backward("backward_m4096", 4096, 6144, 1536, "silu"),
    ]


def _log_int(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + step)))
    return max(lo, min(hi, int(v) // step * step))


def draw(rng):
    op = rng.choice(("linear", "gated", "gated", "backward", "linear"))
    fmt = "f16" if op == "backward" else rng.choice(FORMATS)
    step = 256 if fmt == "q4" else 16
    while True:
        M = _log_int(rng, 1, 4096)
        N = _log_int(rng, 256, 6144, 16)
        K = _log_int(rng, 256, 6144, step)
        if M * N * K <= 4096 * 6144 * 1536:
            break
    c = {"op": op, "fmt": fmt, "M": M, "N": N, "K": K, "act": rng.choice(ACTS)}
    if op == "linear":
        c["residual"] = rng.random() < 0.7
        c["steer"] = rng.random() < 0.3
        if c["act"] == "none" and not c["steer"]:
            c["residual"] = True
    elif op == "gated":
        c["save"] = rng.random() < 0.3
    return c


# ------------------------------------------------------------------ inputs --

def _pack_q8(w):
    """int8 codes and one fp32 scale per row: absmax / 127, half to even."""
    w = w.float()
    s = w.abs().amax(1) / torch.tensor(127.0, device=w.device)
    q = torch.where(s[:, None] > 0, w / s[:, None], torch.zeros_like(w))
    return q.round().clamp(-127, 127).to(torch.int8), s


def _pack_q4(w):
    """two codes + 8 per byte, even k in the low nibble; fp16 scale per 32."""
    n, k = w.shape
    g = w.float().view(n, k // 32, 32)
    s = (g.abs().amax(2) / torch.tensor(7.0, device=w.device)).half()
    f = s.float()[:, :, None]
    q = torch.where(f > 0, g / f, torch.zeros_like(g)).round().clamp(-7, 7).add(8).to(torch.uint8).view(n, k)
    return q[:, 0::2] | (q[:, 1::2] << 4), s


def prepare(case, seed):
    gen = torch.Generator(device=D)
    gen.manual_seed(seed)
    M, N, K, fmt = case["M"], case["N"], case["K"], case["fmt"]

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=gen, device=D).mul_(std)

    def weight():
        w = normal(N, K, std=0.02).half()
        if fmt in ("q8", "w8a8"):
            return _pack_q8(w)
        return _pack_q4(w) if fmt == "q4" else (w, None)

    st = {"case": case, "sx": None}
    x = normal(M, K)
    # a few input channels carry values far above the others', as they do in
    # trained transformers
    x[:, torch.randperm(K, generator=gen, device=D)[:max(1, K // 100)]] *= 5.0
    x = x.half()
    st["X"], st["sx"] = _pack_q8(x) if fmt == "w8a8" else (x, None)
    if case["op"] == "linear":
        st["W"], st["s"] = weight()
        st["bias"] = normal(N, std=0.1).half()
        st["R"] = normal(M, N).half() if case["residual"] else None
        st["v"] = torch.nn.functional.normalize(normal(N), dim=0) if case["steer"] else None
        st["out"] = torch.empty(M, N, dtype=torch.float16, device=D)
        return st
    st["Wg"], st["sg"] = weight()
    st["Wu"], st["su"] = weight()
    if case["op"] == "gated":
        st["bg"], st["bu"] = normal(N, std=0.1).half(), normal(N, std=0.1).half()
        st["out"] = torch.empty(M, N, dtype=torch.float16, device=D)
        st["save"] = (torch.empty_like(st["out"]), torch.empty_like(st["out"])) if case["save"] else None
        return st
    # what a forward pass kept: fp16 pre-activations
    st["G"] = (x.float() @ st["Wg"].float().t() + normal(N, std=0.1)).half()
    st["U"] = (x.float() @ st["Wu"].float().t() + normal(N, std=0.1)).half()
    st["dH"] = normal(M, N, std=0.05).half()
    return st


# ------------------------------------------------------------- plain forms --

ALPHA = 0.3
_C0, _C1 = math.sqrt(2 / math.pi), 0.044715


def _decode(fmt, W, s):
    """The weight's values in fp32 (for q8 and w8a8 without the row scale)."""
    if fmt != "q4":
        return W.float()
    lo, hi = (W & 15).float() - 8, (W >> 4).float() - 8
    n, k2 = W.shape
    codes = torch.stack((lo, hi), 2).view(n, k2 // 16, 32)
    return (codes * s.float()[:, :, None]).half().float().view(n, 2 * k2)  # the format's values are fp16


def _project(fmt, X, sx, W, s, bias):
    z = X.float() @ _decode(fmt, W, s).t()
    if sx is not None:
        z = z * sx[:, None]
    if fmt in ("q8", "w8a8"):
        z = z * s
    return z + bias.float()


def _act(z, act):
    if act == "relu":
        return z.clamp_min(0)
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * torch.erfc(z * -math.sqrt(0.5))
    if act == "gelu_tanh":
        return z / (1 + torch.exp(-2 * _C0 * (z + _C1 * z * z * z)))
    return z


def _act_grad(z, act):
    if act == "relu":
        return (z > 0).float()
    if act == "silu":
        s = 1 / (1 + torch.exp(-z))
        return s * (1 + z * (1 - s))
    if act == "gelu":
        return 0.5 * torch.erfc(z * -math.sqrt(0.5)) + z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi))
    if act == "gelu_tanh":
        s = 1 / (1 + torch.exp(-2 * _C0 * (z + _C1 * z * z * z)))
        return s + z * s * (1 - s) * (2 * _C0) * (1 + 3 * _C1 * z * z)
    return torch.ones_like(z)


def _plain(st, case):
    fmt, act = case["fmt"], case["act"]
    if case["op"] == "linear":
        y = _act(_project(fmt, st["X"], st["sx"], st["W"], st["s"], st["bias"]), act)
        if st["v"] is not None:
            y = y + ALPHA * st["v"]
        if st["R"] is not None:
            y = y + st["R"].float()
        return {"Y": y.half()}
    if case["op"] == "gated":
        g = _project(fmt, st["X"], st["sx"], st["Wg"], st["sg"], st["bg"])
        u = _project(fmt, st["X"], st["sx"], st["Wu"], st["su"], st["bu"])
        r = {"H": (_act(g, act) * u).half()}
        if case["save"]:
            r["G"], r["U"] = g.half(), u.half()
        return r
    x, g, u, dh = (st[k].float() for k in ("X", "G", "U", "dH"))
    dg, du = dh * u * _act_grad(g, act), dh * _act(g, act)
    return {"dX": (dg @ st["Wg"].float() + du @ st["Wu"].float()).half(),
            "dWg": (dg.t() @ x).half(), "dWu": (du.t() @ x).half(),
            "dbg": dg.sum(0).half(), "dbu": du.sum(0).half()}


def run(st):
    case = st["case"]
    if not own:
        return _plain(st, case)
    import int8_int4_b200 as aq
    if case["op"] == "linear":
        return {"Y": aq.qgemm_act(case["fmt"], st["X"], st["W"], st["s"], sx=st["sx"], bias=st["bias"],
                                  act=case["act"], residual=st["R"], steer_vec=st["v"], alpha=ALPHA,
                                  out=st["out"])}
    if case["op"] == "gated":
        h = aq.qgemm_gated(case["fmt"], st["X"], st["Wg"], st["sg"], st["Wu"], st["su"], sx=st["sx"],
                           bias_g=st["bg"], bias_u=st["bu"], act=case["act"], out=st["out"], save=st["save"])
        return {"H": h, "G": st["save"][0], "U": st["save"][1]} if case["save"] else {"H": h}
    dX, dWg, dWu, dbg, dbu = aq.gated_backward(st["dH"], st["X"], st["Wg"], st["Wu"], st["G"], st["U"],
                                               act=case["act"])
    return {"dX": dX, "dWg": dWg, "dWu": dWu, "dbg": dbg, "dbu": dbu}


# -------------------------------------------------- the definition, 64 bits --

def _values64(fmt, W, s):
    """The weight matrix itself: codes times scales."""
    if fmt == "f16":
        return W.double()
    if fmt != "q4":
        return W.double() * s.double().unsqueeze(1)
    w = torch.empty(W.shape[0], 2 * W.shape[1], dtype=torch.float64, device=W.device)
    w[:, 0::2] = W.remainder(16).double() - 8
    w[:, 1::2] = W.div(16, rounding_mode="floor").double() - 8
    return (w * s.double().repeat_interleave(32, 1)).half().double()


def _act64(z, act):
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "gelu":
        return z * torch.special.ndtr(z)
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z.pow(3))))
    return z


def exact(case, seed):
    st = prepare(case, seed)
    fmt, act = case["fmt"], case["act"]
    X = st["X"].double() if st["sx"] is None else st["X"].double() * st["sx"].double().unsqueeze(1)
    if case["op"] == "linear":
        y = _act64(torch.addmm(st["bias"].double(), X, _values64(fmt, st["W"], st["s"]).t()), act)
        if st["v"] is not None:
            # the strength is an fp32 number
            y = y + torch.tensor(ALPHA, dtype=torch.float32).item() * st["v"].double()
        return {"Y": y if st["R"] is None else y + st["R"].double()}
    if case["op"] == "gated":
        g = torch.addmm(st["bg"].double(), X, _values64(fmt, st["Wg"], st["sg"]).t())
        u = torch.addmm(st["bu"].double(), X, _values64(fmt, st["Wu"], st["su"]).t())
        h = _act64(g, act) * u
        return {"H": h, "G": g, "U": u} if case["save"] else {"H": h}
    g, u = st["G"].double().requires_grad_(), st["U"].double().requires_grad_()
    dg, du = torch.autograd.grad((_act64(g, act) * u * st["dH"].double()).sum(), (g, u))
    dx = torch.cat((dg, du), 1) @ torch.cat((st["Wg"], st["Wu"]), 0).double()
    return {"dX": dx, "dWg": (X.t() @ dg).t(), "dWu": (X.t() @ du).t(), "dbg": dg.sum(0), "dbu": du.sum(0)}


# -------------------------------------------------------------------- work --

def work(case):
    M, N, K, fmt = case["M"], case["N"], case["K"], case["fmt"]
    w = {"q8": N * K + 4 * N, "w8a8": N * K + 4 * N, "q4": N * K // 2 + N * K // 16, "f16": 2 * N * K}[fmt]
    x = M * K + 4 * M if fmt == "w8a8" else 2 * M * K
    mn = 2 * M * N
    if case["op"] == "linear":
        return {"bytes": x + w + 2 * N + mn + mn * case["residual"] + 4 * N * case["steer"], "flops": 2 * M * N * K}
    if case["op"] == "gated":
        return {"bytes": x + 2 * w + 4 * N + mn * (3 if case["save"] else 1), "flops": 4 * M * N * K}
    return {"bytes": 3 * mn + 2 * x + 4 * w + 4 * N, "flops": 8 * M * N * K}
