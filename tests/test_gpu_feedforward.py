"""The feed-forward operators on a B200, against their definitions in 64 bits:

- aria_qgemm_act:   Y = act(X W^T + b) + alpha v + R
- aria_qgemm_gated: H = act(X Wg^T + bg) * (X Wu^T + bu), and its kept G, U
- aria_gated_bwd:   the gradients of the latter

Tolerances, derived before the first run. A tensor-core sum of K products
starts from exact products and adds them to an fp32 accumulator in steps of
16 (32 for int8, exactly); taking every step to lose one unit 2^-23 of the
largest possible partial sum S = sum |x w|, plus 16 such units for the scales
and the bias, the pre-activation is off by at most
(K / 16 + 16) 2^-23 S =: dz. An activation with |act'| <= 1.13 passes on
1.13 dz, and its own fp32 evaluation is taken as 2^-18 relative. A product of
two such values is off by |u| 1.13 dg + |act(g)| du. The result is rounded
once to fp16: half a step, 2^-11 relative or 2^-25 absolute among the
subnormals. The backward pass's operands dG, dU are themselves rounded once
to fp16 (each off by 2^-11 relative), which the products pass on.
"""
import itertools

import pytest
import torch

import int8_int4_b200 as aq

pytestmark = pytest.mark.gpu

H16, SUB = 2.0 ** -11, 2.0 ** -25
FMTS = ("q8", "q4", "w8a8", "f16")
ACTS = tuple(aq.ACTS)


@pytest.fixture(scope="module", autouse=True)
def _lib():
    aq.load_library()   # raises if the CUDA library is missing: no fallback
    yield
    aq.device_status()


def gen(seed):
    return torch.Generator().manual_seed(seed)


def normal(seed, *shape, std=1.0):
    return (torch.randn(*shape, generator=gen(seed)) * std).half().cuda()


def weight(fmt, seed, N, K):
    """(packed, scales, value in 64 bits) of a random weight."""
    W = normal(seed, N, K, std=0.05)
    if fmt == "f16":
        return W, None, W.double()
    if fmt == "q4":
        P, S = aq.qpack("q4", W)
        codes = torch.stack((P & 15, P >> 4), 2).view(N, K).double() - 8
        v = codes * S.double().repeat_interleave(32, 1)
        return P, S, v.half().double()  # the format's values are fp16
    Wq, s = aq.qpack("q8", W)
    return Wq, s, Wq.double() * s.double()[:, None]


def acts(fmt, seed, M, K):
    """(X, sx, value in 64 bits)"""
    X = normal(seed, M, K)
    if fmt != "w8a8":
        return X, None, X.double()
    Xq, sx = aq.act_quant(X)
    return Xq, sx, Xq.double() * sx.double()[:, None]


def act64(z, act):
    return {"none": lambda: z, "relu": lambda: z.clamp_min(0), "silu": lambda: z * torch.sigmoid(z),
            "gelu": lambda: z * torch.special.ndtr(z),
            "gelu_tanh": lambda: 0.5 * z * (1 + torch.tanh((2 / torch.pi) ** 0.5 * (z + 0.044715 * z ** 3)))}[act]()


def project(x, w, b):
    """(z, dz): the pre-activation in 64 bits and its error bound."""
    z = x @ w.t()
    s = x.abs() @ w.abs().t()
    if b is not None:
        z, s = z + b.double(), s + b.double().abs()
    return z, (x.shape[1] / 16 + 16) * 2.0 ** -23 * s


def close(got, ref, tol):
    assert got.shape == ref.shape and not got.isnan().any()
    err = (got.double() - ref).abs()
    bad = err > tol
    assert not bad.any(), (int(bad.sum()), float((err / tol).max()), bad.nonzero()[:4].tolist())


def guarded(*shape):
    """A tensor inside a larger buffer of a known pattern, and a check that
    the buffer around it is untouched."""
    n = 1
    for d in shape:
        n *= d
    buf = torch.full((n + 512,), 1234.0, dtype=torch.float16, device="cuda")

    def check():
        assert (buf[:256] == 1234).all() and (buf[256 + n:] == 1234).all()
    return buf[256:256 + n].view(*shape), check


# ---------------------------------------------------------- activation, residual --

def check_act(fmt, M, N, K, act, residual, steer, bias=True, seed=0):
    X, sx, x = acts(fmt, seed + 1, M, K)
    W, s, w = weight(fmt, seed + 2, N, K)
    b = normal(seed + 3, N, std=0.1) if bias else None
    R = normal(seed + 4, M, N) if residual else None
    v = torch.randn(N, generator=gen(seed + 5)).cuda() if steer else None
    out, guard = guarded(M, N)
    Y = aq.qgemm_act(fmt, X, W, s, sx=sx, bias=b, act=act, residual=R, steer_vec=v, alpha=0.3, out=out)
    assert Y is out
    z, dz = project(x, w, b)
    a = act64(z, act)
    y = a
    if steer:
        y = y + torch.tensor(0.3, dtype=torch.float32).item() * v.double()
    if residual:
        y = y + R.double()
    parts = a.abs() + (y - a).abs()  # the fp32 sums round relative to their parts
    close(Y, y, 1.13 * dz + 2.0 ** -18 * a.abs() + 2.0 ** -22 * parts + H16 * y.abs() + SUB)
    guard()


SIZES = [(1, 16, 16), (1, 208, 512), (3, 1024, 4096), (9, 144, 256), (16, 1536, 1536), (17, 128, 256),
         (40, 400, 1040), (203, 1040, 592), (300, 6144, 512), (432, 1536, 1536), (600, 272, 768),
         (1500, 1552, 256)]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,N,K", SIZES)
def test_act_sizes(fmt, M, N, K):
    if fmt == "q4":
        K = (K + 255) // 256 * 256
    i = M + N + K
    check_act(fmt, M, N, K, ACTS[i % 5], residual=i % 3 != 0 or ACTS[i % 5] == "none", steer=i % 2 == 0)


# sizes where the linear runs on the token-major kernel, with tiles of 128, 192
# and 256 columns, and odd edges of both rows and columns
LARGE = [(1100, 1040, 2576), (4100, 1552, 2576), (3000, 1040, 6160), (1100, 6160, 2576)]


@pytest.mark.parametrize("fmt", ["f16", "w8a8"])
@pytest.mark.parametrize("M,N,K", LARGE)
@pytest.mark.parametrize("act,residual,steer", [("gelu", True, True), ("silu", False, False), ("none", True, False)])
def test_act_many_tokens(fmt, M, N, K, act, residual, steer):
    check_act(fmt, M, N, K, act, residual, steer)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M", [5, 150])
def test_act_functions(fmt, act, M):
    check_act(fmt, M, 256, 512, act, residual=False, steer=act == "none")
    check_act(fmt, M, 256, 512, act, residual=True, steer=True, bias=False, seed=50)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,N,K", [(4, 256, 256), (150, 384, 512), (432, 1536, 1536)])
def test_act_none_without_residual_is_the_plain_gemm(fmt, M, N, K):
    X, sx, _ = acts(fmt, 1, M, K)
    W, s, _ = weight(fmt, 2, N, K)
    b, v = normal(3, N), torch.randn(N, generator=gen(4)).cuda()
    ref = aq.qgemm(fmt, X, W, s, sx=sx, bias=b, steer_vec=v, alpha=0.3)
    got = aq.qgemm_act(fmt, X, W, s, sx=sx, bias=b, steer_vec=v, alpha=0.3)
    assert torch.equal(ref.view(torch.int16), got.view(torch.int16))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,N,K", [(4, 256, 1024), (130, 1536, 6144), (500, 1536, 512), (1100, 6160, 2560)])
def test_residual_in_place_and_strengths(fmt, M, N, K):
    X, sx, _ = acts(fmt, 1, M, K)
    W, s, _ = weight(fmt, 2, N, K)
    b, R, v = normal(3, N), normal(4, M, N), torch.randn(N, generator=gen(5)).cuda()
    call = lambda **k: aq.qgemm_act(fmt, X, W, s, sx=sx, bias=b, act="gelu", **k)
    plain = call(residual=R)
    inplace = R.clone()
    call(residual=inplace, out=inplace)
    assert torch.equal(plain, inplace)
    assert torch.equal(plain, call(residual=R, steer_vec=v, alpha=0.0))
    zero, some = torch.zeros(1, device="cuda"), torch.full((1,), 0.3, device="cuda")
    assert torch.equal(plain, call(residual=R, steer_vec=v, alpha_dev=zero, alpha=0.3))
    assert torch.equal(call(residual=R, steer_vec=v, alpha=0.3), call(residual=R, steer_vec=v, alpha_dev=some))
    assert torch.equal(plain, call(residual=R))  # the same bytes again


# ------------------------------------------------------------------------- gated --

def check_gated(fmt, M, N, K, act, save, bias=True, seed=0):
    X, sx, x = acts(fmt, seed + 1, M, K)
    Wg, sg, wg = weight(fmt, seed + 2, N, K)
    Wu, su, wu = weight(fmt, seed + 3, N, K)
    bg, bu = (normal(seed + 4, N, std=0.1), normal(seed + 5, N, std=0.1)) if bias else (None, None)
    out, guard = guarded(M, N)
    G, guard_g = guarded(M, N)
    U, guard_u = guarded(M, N)
    H = aq.qgemm_gated(fmt, X, Wg, sg, Wu, su, sx=sx, bias_g=bg, bias_u=bu, act=act, out=out,
                       save=(G, U) if save else None)
    g, dg = project(x, wg, bg)
    u, du = project(x, wu, bu)
    a = act64(g, act)
    close(H, a * u, u.abs() * 1.13 * dg + a.abs() * du + 1.13 * dg * du + 2.0 ** -18 * (a * u).abs()
          + H16 * (a * u).abs() + SUB)
    if save:
        close(G, g, dg + H16 * g.abs() + SUB)
        close(U, u, du + H16 * u.abs() + SUB)
    else:
        assert (G == 1234).all() and (U == 1234).all()
    for c in (guard, guard_g, guard_u):
        c()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,N,K", SIZES)
def test_gated_sizes(fmt, M, N, K):
    if fmt == "q4":
        K = (K + 255) // 256 * 256
    i = M + N + K
    check_gated(fmt, M, N, K, ACTS[i % 5], save=i % 2 == 0)


@pytest.mark.parametrize("fmt", ["f16", "w8a8"])
@pytest.mark.parametrize("M,N,K", [(130, 1040, 592), (300, 3088, 80), (1100, 1552, 80), (3000, 1040, 80)])
@pytest.mark.parametrize("save", [False, True])
def test_gated_tile_widths(fmt, M, N, K, save):
    """Token-major tiles of 128, 192 and 256 columns with odd edges."""
    check_gated(fmt, M, N, K, "gelu", save)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M", [5, 150])
def test_gated_functions(fmt, act, M):
    check_gated(fmt, M, 256, 512, act, save=True)
    check_gated(fmt, M, 256, 512, act, save=False, bias=False, seed=50)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M", [2, 15, 100, 433, 1030])
def test_gated_save_changes_nothing_and_repeats(fmt, M):
    N, K = 304, 512
    X, sx, _ = acts(fmt, 1, M, K)
    Wg, sg, _ = weight(fmt, 2, N, K)
    Wu, su, _ = weight(fmt, 3, N, K)
    G, U = torch.empty(M, N, dtype=torch.float16, device="cuda"), torch.empty(M, N, dtype=torch.float16, device="cuda")
    a = aq.qgemm_gated(fmt, X, Wg, sg, Wu, su, sx=sx)
    b = aq.qgemm_gated(fmt, X, Wg, sg, Wu, su, sx=sx, save=(G, U))
    assert torch.equal(a, b)
    c = aq.qgemm_gated(fmt, X, Wg, sg, Wu, su, sx=sx, save=(G, U))
    assert torch.equal(a, c)
    # the two projections are told apart, whichever weight lies first in memory
    swapped = aq.qgemm_gated(fmt, X, Wu, su, Wg, sg, sx=sx, act="none")
    assert torch.equal(swapped, aq.qgemm_gated(fmt, X, Wg, sg, Wu, su, sx=sx, act="none"))
    assert not torch.equal(a, aq.qgemm_gated(fmt, X, Wu, su, Wg, sg, sx=sx))


@pytest.mark.parametrize("M", [3, 200])
@pytest.mark.parametrize("sign", [1, -1])
def test_w8a8_accumulators_at_their_limit(M, sign):
    """K = 133136, every code at +-127: |acc| = 0.99999 * 2^31, exact in int32;
    its fp32 image and the scales are off by 2^-24 each, relative."""
    K, N = 133136, 32
    assert 2 ** 31 - 2 ** 18 < K * 127 ** 2 < 2 ** 31
    X = torch.full((M, K), 127, dtype=torch.int8, device="cuda")
    W = torch.full((N, K), 127 * sign, dtype=torch.int8, device="cuda")
    sx = torch.rand(M, generator=gen(1)).cuda() + 0.5
    sw = (torch.rand(N, generator=gen(2)).cuda() + 0.5) * 1e-8
    z = sx.double()[:, None] * sw.double() * (K * 127 ** 2 * sign)
    y = aq.qgemm_act("w8a8", X, W, sw, sx=sx, act="silu")
    close(y, act64(z, "silu"), (H16 + 2.0 ** -18 + 1.13 * 2.0 ** -21) * z.abs() + SUB)
    h = aq.qgemm_gated("w8a8", X, W, sw, W, sw, sx=sx, act="none")
    close(h, z * z, (H16 + 2.0 ** -20) * z * z + SUB)


@pytest.mark.parametrize("fmt", FMTS)
def test_long_and_narrow(fmt):
    """Many tiles per CTA: 9001 tokens, one column tile."""
    check_gated(fmt, 9001, 16, 256, "silu", save=True)
    check_act(fmt, 9001, 32, 256, "gelu", residual=True, steer=True)


# ---------------------------------------------------------------------- backward --

def grads64(dH, G, U, act):
    g, u = G.double().requires_grad_(), U.double().requires_grad_()
    return torch.autograd.grad((act64(g, act) * u * dH.double()).sum(), (g, u))


def bwd_inputs(M, N, K, seed=0):
    return (normal(seed + 1, M, N, std=0.1), normal(seed + 2, M, K), normal(seed + 3, N, K, std=0.05),
            normal(seed + 4, N, K, std=0.05), normal(seed + 5, M, N, std=1.5), normal(seed + 6, M, N, std=1.5))


BWD_SIZES = [(1, 16, 16), (2, 128, 64), (7, 208, 144), (64, 64, 64), (100, 272, 400), (129, 1040, 592),
             (432, 4096, 1024), (1000, 528, 272), (2100, 256, 1040), (4096, 512, 256), (9001, 32, 48)]


@pytest.mark.parametrize("M,N,K", BWD_SIZES)
def test_backward(M, N, K):
    for act in (ACTS if M * N * K < 1e7 else (ACTS[(M + N) % 5],)):
        dH, X, Wg, Wu, G, U = bwd_inputs(M, N, K)
        outs = [guarded(*s) for s in ((M, K), (N, K), (N, K), (N,), (N,))]
        r = aq.gated_backward(dH, X, Wg, Wu, G, U, act=act, out=tuple(o[0] for o in outs))
        dg, du = grads64(dH, G, U, act)
        # the operands: half a step of fp16, and their fp32 evaluation
        eg = (H16 + 2.0 ** -18) * dg.abs() + 2.0 ** -18 * (dH.double() * U.double()).abs() + SUB
        eu = (H16 + 2.0 ** -18) * du.abs() + SUB
        x, wg, wu = X.double(), Wg.double(), Wu.double()

        def product(pairs, k):
            ref = sum(a @ b for a, b, _ in pairs)
            s = sum(a.abs() @ b.abs() for a, b, _ in pairs)
            e = sum(ea @ b.abs() for _, b, ea in pairs)
            return ref, e + (k / 16 + 16) * 2.0 ** -23 * s + H16 * ref.abs() + SUB
        close(r[0], *product(((dg, wg, eg), (du, wu, eu)), 2 * N))
        close(r[1], *product(((dg.t(), x, eg.t()),), M))
        close(r[2], *product(((du.t(), x, eu.t()),), M))
        for got, d, e in ((r[3], dg, eg), (r[4], du, eu)):
            fp32 = e - H16 * d.abs()  # summed before the operands' rounding
            close(got, d.sum(0), fp32.sum(0) + M * 2.0 ** -24 * d.abs().sum(0) + H16 * d.sum(0).abs() + SUB)
        for _, check in outs:
            check()


@pytest.mark.parametrize("act", ACTS)
def test_backward_against_differences(act):
    """The gradients of sum(dH * H) along a random direction of every input,
    against the difference quotient of the forward definition."""
    M, N, K = 24, 96, 80
    X, Wg, Wu = normal(1, M, K), normal(2, N, K, std=0.1), normal(3, N, K, std=0.1)
    bg, bu, dH = normal(4, N, std=0.3), normal(5, N, std=0.3), normal(6, M, N, std=0.1)
    G, U = torch.empty_like(dH), torch.empty_like(dH)
    aq.qgemm_gated("f16", X, Wg, None, Wu, None, bias_g=bg, bias_u=bu, act=act, save=(G, U))
    got = aq.gated_backward(dH, X, Wg, Wu, G, U, act=act)
    at = [t.double() for t in (X, Wg, Wu, bg, bu)]

    def loss(p):
        return (dH.double() * act64(p[0] @ p[1].t() + p[3], act) * (p[0] @ p[2].t() + p[4])).sum()
    h = 1e-5  # the quotient of a smooth loss is off by h^2 times its third derivative
    for i, g in enumerate(got):
        d = torch.randn(at[i].shape, generator=gen(20 + i), dtype=torch.float64).cuda()
        up, dn = list(at), list(at)
        up[i], dn[i] = at[i] + h * d, at[i] - h * d
        want = (loss(up) - loss(dn)) / (2 * h)
        # each gradient element is off by about 3 * 2^-11 (operands, kept
        # pre-activations, result); the directional sum adds them in random
        # sign: 8 standard deviations. relu's kink may be crossed by the step
        # or by the rounding of G: |g| < 2^-10 happens to about 0.1 % of them.
        slack = 8 * 3 * H16 * float((g.double() * d).norm()) + (0.02 * float((g.double() * d).norm()) if act == "relu" else 0)
        assert abs(float((g.double() * d).sum() - want)) <= slack + 1e-6, (i, float((g.double() * d).sum()), float(want))


@pytest.mark.parametrize("want", [w for w in itertools.product((True, False), repeat=3) if any(w)])
def test_backward_parts(want):
    """Each subset of the gradients is what the full call gives: the same bytes,
    but for dX, whose sum over the channels may be divided differently (fp32
    sums that differ by their order, then one rounding: one step of fp16, of
    the sum's largest partial sums where it cancels)."""
    i, w, b = want
    for M, N, K in ((77, 144, 208), (1300, 400, 272), (2100, 1040, 256)):
        dH, X, Wg, Wu, G, U = bwd_inputs(M, N, K)
        full = aq.gated_backward(dH, X, Wg, Wu, G, U)
        part = aq.gated_backward(dH, X if w else None, Wg if i else None, Wu if i else None, G, U, input_grad=i,
                                 weight_grad=w, bias_grad=b)
        for k, (f, p, on) in enumerate(zip(full, part, (i, w, w, b, b))):
            assert (p is None) == (not on)
            if on and k:
                assert torch.equal(f, p)
            elif on:
                slack = 2.0 ** -10 * f.double().abs() + 2.0 ** -24 + 2.0 ** -20 * f.double().abs().max()
                assert ((f.double() - p.double()).abs() <= slack).all()


def test_backward_workspace_needs_no_preparation():
    dH, X, Wg, Wu, G, U = bwd_inputs(200, 144, 208)
    ref = aq.gated_backward(dH, X, Wg, Wu, G, U)
    n = aq.gated_backward_workspace_size(200, 144, 208)
    ws = torch.full((n + 256,), 255, dtype=torch.uint8, device="cuda")  # every fp16 and fp32 a NaN
    for _ in range(2):
        got = aq.gated_backward(dH, X, Wg, Wu, G, U, workspace=ws[:n])
        assert all(torch.equal(a, b) for a, b in zip(ref, got))
    assert (ws[n:] == 255).all()


# ---------------------------------------------------------------------- together --

def run_block(fmt, X, R, w, tmp):
    """The feed-forward half of a block: gated projections, then the down
    projection added to the residual stream in place."""
    aq.qgemm_gated(fmt, X[0], *w["g"], *w["u"], sx=X[1], out=tmp["h"])
    if fmt == "w8a8":
        h, sh = aq.act_quant(tmp["h"], out=(tmp["q"], tmp["s"]))
    else:
        h, sh = tmp["h"], None
    return aq.qgemm_act(fmt, h, *w["d"], sx=sh, residual=R, out=R)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M", [1, 16, 432])
def test_block_eager_and_captured(fmt, M):
    D, F = 256, 512
    w = {k: weight(fmt, i, n, kk)[:2] for i, (k, n, kk) in enumerate((("g", F, D), ("u", F, D), ("d", D, F)))}
    tmp = {"h": torch.empty(M, F, dtype=torch.float16, device="cuda"),
           "q": torch.empty(M, F, dtype=torch.int8, device="cuda"),
           "s": torch.empty(M, dtype=torch.float32, device="cuda")}
    xs = [acts(fmt, 10 + i, M, D)[:2] for i in range(3)]
    rs = [normal(20 + i, M, D) for i in range(3)]
    refs = []
    for x, r in zip(xs, rs):
        y = r.clone()
        for _ in range(3):  # three blocks in a row, each reading what the last one wrote
            run_block(fmt, x, y, w, tmp)
        refs.append(y)
    x = [None if t is None else t.clone() for t in xs[0]]
    R = rs[0].clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        run_block(fmt, x, R, w, tmp)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(3):
            run_block(fmt, x, R, w, tmp)
    for i in (1, 2, 0):
        for dst, src in zip(x, xs[i]):
            if dst is not None:
                dst.copy_(src)
        R.copy_(rs[i])
        graph.replay()
        assert torch.equal(R, refs[i])


@pytest.mark.parametrize("M", [1, 300, 1000])
def test_training_step_captured_while_an_eager_one_lives(M):
    N, K = 272, 208
    def step(X, Wg, Wu, dH, G, U, out, ws):
        aq.qgemm_gated("f16", X, Wg, None, Wu, None, save=(G, U))
        return aq.gated_backward(dH, X, Wg, Wu, G, U, out=out, workspace=ws)
    ins = [(normal(i, M, K), normal(i + 1, N, K, std=0.05), normal(i + 2, N, K, std=0.05), normal(i + 3, M, N)) for i in (1, 11)]
    new = lambda: ([torch.empty(M, N, dtype=torch.float16, device="cuda") for _ in range(2)],
                   tuple(torch.empty(*s, dtype=torch.float16, device="cuda") for s in ((M, K), (N, K), (N, K), (N,), (N,))),
                   torch.empty(aq.gated_backward_workspace_size(M, N, K), dtype=torch.uint8, device="cuda"))
    refs = []
    for t in ins:
        (G, U), out, ws = new()
        refs.append(step(*t, G, U, out, ws))
    static = [t.clone() for t in ins[0]]
    (G, U), out, ws = new()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(*static, G, U, out, ws)
    for k in (1, 0, 1):
        for a, b in zip(static, ins[k]):
            a.copy_(b)
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(out, refs[k]))


@pytest.mark.parametrize("M", [1, 16, 64, 100, 300])
def test_weights_written_by_the_preceding_kernel(M):
    """A training loop's forward right behind the update of its weights: the
    call that keeps G and U sees the weights that an ordinary kernel before it
    in the stream writes, eager and captured."""
    N, K = 1536, 512
    X, Wg, Wu = normal(1, M, K), normal(2, N, K, std=0.05), normal(3, N, K, std=0.05)
    g0, u0 = Wg.clone(), Wu.clone()
    G, U = (torch.empty(M, N, dtype=torch.float16, device="cuda") for _ in range(2))
    refs = []
    for k in (1.0, 0.5, -2.0):  # exact factors
        torch.cuda.synchronize()
        H = aq.qgemm_gated("f16", X, g0 * k, None, u0 * k, None, save=(G, U))
        torch.cuda.synchronize()
        refs.append((H.clone(), G.clone(), U.clone()))

    def run(i, k):
        torch.mul(u0, k, out=Wu)
        torch.mul(g0, k, out=Wg)
        return aq.qgemm_gated("f16", X, Wg, None, Wu, None, save=(G, U))
    graph = torch.cuda.CUDAGraph()
    outs = []
    with torch.cuda.graph(graph):
        for i, k in enumerate((1.0, 0.5, -2.0)):
            outs.append((run(i, k), G.clone(), U.clone()))
    for _ in range(20):
        for i, k in enumerate((1.0, 0.5, -2.0)):
            H = run(i, k)
            assert all(torch.equal(a, b) for a, b in zip((H, G, U), refs[i]))
        graph.replay()
        for i in range(3):
            assert all(torch.equal(a, b) for a, b in zip(outs[i], refs[i]))


def test_two_streams_at_once():
    """Independent calls on two streams, each with its own workspace."""
    M, N, K = 300, 528, 272
    sets = [bwd_inputs(M, N, K, seed=s) for s in (0, 100)]
    refs = [aq.gated_backward(*t) for t in sets]
    hs = [aq.qgemm_gated("f16", t[1], t[2], None, t[3], None) for t in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [[], []]
    for _ in range(4):
        for i, (t, s) in enumerate(zip(sets, streams)):
            got[i].append((aq.gated_backward(*t, stream=s), aq.qgemm_gated("f16", t[1], t[2], None, t[3], None, stream=s)))
    torch.cuda.synchronize()
    for i in range(2):
        for g, h in got[i]:
            assert torch.equal(h, hs[i]) and all(torch.equal(a, b) for a, b in zip(g, refs[i]))


def test_offsets_past_32_bits():
    """More than 2^31 elements in X's, H's and the gradients' rows: the last
    rows and columns against 64 bits (K is short: the size is in M N)."""
    M, N, K = 70000, 32768, 64
    assert M * N > 2 ** 31
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB of device memory")
    g = torch.Generator(device="cuda").manual_seed(3)
    r = lambda *s, std=1.0: (torch.randn(*s, generator=g, device="cuda", dtype=torch.float16) * std)
    X, Wg, Wu = r(M, K), r(N, K, std=0.1), r(N, K, std=0.1)
    G, U = torch.empty(M, N, dtype=torch.float16, device="cuda"), torch.empty(M, N, dtype=torch.float16, device="cuda")
    H = aq.qgemm_gated("f16", X, Wg, None, Wu, None, save=(G, U))
    rows = slice(M - 70, M)
    zg, dg = project(X[rows].double(), Wg.double(), None)
    zu, du = project(X[rows].double(), Wu.double(), None)
    a = act64(zg, "silu")
    close(G[rows], zg, dg + H16 * zg.abs() + SUB)
    close(U[rows], zu, du + H16 * zu.abs() + SUB)
    close(H[rows], a * zu, zu.abs() * 1.13 * dg + a.abs() * du + 1.13 * dg * du + (2.0 ** -18 + H16) * (a * zu).abs() + SUB)
    # in place on the residual: the whole of H is read and written
    tail, last = H[rows].double(), Wg.double()
    Wq, s = aq.qpack("q8", Wg)
    aq.qgemm_act("q8", X, Wq, s, act="relu", residual=H, out=H)
    z, dz = project(X[rows].double(), Wq.double() * s.double()[:, None], None)
    y = z.clamp_min(0) + tail
    close(H[rows], y, dz + 2.0 ** -18 * z.abs() + 2.0 ** -21 * (z.abs() + tail.abs()) + H16 * y.abs() + SUB)
    del tail, last, z, dz, y, a, zg, zu, dg, du
    dX, dWg, dWu, dbg, dbu = aq.gated_backward(H, X, Wg, Wu, G, U)
    gg, gu = grads64(H[rows], G[rows], U[rows], "silu")
    ref = gg @ Wg.double() + gu @ Wu.double()
    s = gg.abs() @ Wg.double().abs() + gu.abs() @ Wu.double().abs()
    # (the operands' rounding dominates: 2^-11 of every term, plus their evaluation)
    close(dX[rows], ref, (H16 + 2.0 ** -17 + (2 * N / 16 + 16) * 2.0 ** -23) * s + H16 * ref.abs() + SUB * N)
    cols = slice(N - 8, N)
    gg, gu = grads64(H[:, cols].contiguous(), G[:, cols].contiguous(), U[:, cols].contiguous(), "silu")
    for got, gw, d in ((dWg, dbg, gg), (dWu, dbu, gu)):
        ref, s = d.t() @ X.double(), d.abs().t() @ X.double().abs()
        fits = ref.abs() < 6e4  # sums over 70000 tokens may pass fp16's range
        close(torch.where(fits, got[cols].double(), ref), ref,
              (H16 + 2.0 ** -17 + (M / 16 + 16) * 2.0 ** -23) * s + H16 * ref.abs() + SUB * M)
        fits = d.sum(0).abs() < 6e4
        close(torch.where(fits, gw[cols].double(), d.sum(0)), d.sum(0),
              (2.0 ** -17 + M * 2.0 ** -24) * d.abs().sum(0) + H16 * d.sum(0).abs() + SUB)
