"""Short convolution, selective scan, gated norm and residual norm on the GPU, against
their float64 definitions (oracle.block_ops) and autograd of those.

Tolerances, relative in the 2-norm of a tensor:
  rounding the result to bf16 moves each value by at most half a step, 2^-8 of it;
  fp32 arithmetic of n roundings of 2^-24 each, of random sign, over terms whose 2-norm is
  up to 16 times the result's (signs cancel), gives 16 sqrt(n) 2^-24:
    conv and norms, n <= 16 per value (sums are trees):      4e-6
    scan of T <= 300 tokens, about 8 roundings a token:      5e-5
    gradients through the scan, twice the chain:             7e-5  (1e-4 is allowed, as in
    the chunk backward)
"""
import numpy as np
import pytest
import torch

import chunk_delta_rule_b200 as cdr
import oracle
from oracle import block_ops as ref

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
HALF = {BF: 2.0 ** -8, F32: 2.0 ** -24}
CONV, NORM, SCAN, SCAN_BWD = 4e-6, 4e-6, 5e-5, 1e-4


def check(name, got, want, tol):
    got, want = got.detach().double().cpu(), want.detach().double().cpu()
    assert got.shape == want.shape, (name, got.shape, want.shape)
    assert torch.equal(torch.isfinite(got), torch.isfinite(want)), name
    d, n = float((got - want).norm()), float(want.norm())
    assert d <= tol * n or n == 0 and d <= tol, f"{name}: off by {d / max(n, 1e-300):.3g} of its norm, {tol:.3g} allowed"


def gen(seed):
    return torch.Generator().manual_seed(seed)


def rnd(g, *shape, dtype=F32, std=1.0):
    return (torch.randn(shape, generator=g, dtype=torch.float64) * std).to(dtype)


def dev(d):
    return {k: (v.cuda() if isinstance(v, torch.Tensor) else v) for k, v in d.items()}


def grads(outs, cots, leaves):
    """d sum <out, cot> / d leaf for each leaf that is not None."""
    live = [l for l in leaves if l is not None]
    pairs = [(o, c) for o, c in zip(outs, cots) if c is not None and o.requires_grad]
    g = torch.autograd.grad([o for o, _ in pairs], live, [c.double() for _, c in pairs], allow_unused=True)
    g = iter([torch.zeros_like(l) if v is None else v for l, v in zip(live, g)])
    return [None if l is None else next(g) for l in leaves]


def leaf(t):
    return None if t is None else t.double().requires_grad_(True)


def bounds_of(lengths):
    b = [0]
    for n in lengths:
        b.append(b[-1] + n)
    return b


# ---------------------------------------------------------------- short convolution

def conv_inputs(tokens, nseq, C, W, dtype, seed, bias, state):
    g = gen(seed)
    return dict(x=rnd(g, tokens, C, dtype=dtype), weight=rnd(g, C, W, std=0.5), bias=rnd(g, C) if bias else None,
                init=rnd(g, nseq, W - 1, C, dtype=dtype) if state else None, dout=rnd(g, tokens, C, dtype=dtype),
                dfin=rnd(g, nseq, W - 1, C, dtype=dtype) if state else None)


CONV_CASES = [  # lengths (equal ones: also as a batch), C, W, dtype, bias, state, silu
    ([130], 64, 4, BF, True, True, True),
    ([33, 33, 33], 24, 4, F32, False, False, True),
    ([70, 70], 37, 4, BF, True, True, True),
    ([1, 1], 8, 4, BF, True, True, True),
    ([2, 2], 8, 4, F32, False, True, False),
    ([3, 3], 5, 3, F32, True, True, True),
    ([19, 19], 16, 2, BF, False, False, True),
    ([5, 0, 1, 2, 70, 3, 0], 40, 4, BF, True, True, True),
    ([0, 0, 17, 1], 9, 3, F32, True, False, True),
    ([200, 1, 1, 1, 64], 136, 2, F32, False, True, False),
    ([600, 41], 1, 4, BF, True, True, True),
]


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("lengths,C,W,dtype,bias,state,silu", CONV_CASES)
def test_conv(lengths, C, W, dtype, bias, state, silu, packed):
    if not packed and len(set(lengths)) > 1:
        pytest.skip("a batch has sequences of one length")
    b, n = bounds_of(lengths), len(lengths)
    h = conv_inputs(b[-1], n, C, W, dtype, 7 + len(lengths) * C, bias, state)
    d = dev(h)
    shape = (b[-1], C) if packed else (n, lengths[0], C)
    cu = torch.tensor(b, dtype=torch.int32, device="cuda") if packed else None
    out, fin = cdr.short_conv(d["x"].view(shape), d["weight"], d["bias"], d["init"], cu_seqlens=cu, silu=silu)
    x, w, bi, st = leaf(h["x"]), leaf(h["weight"]), leaf(h["bias"]), leaf(h["init"])
    ro, rf = ref.short_conv(x, w, bi, st, b, silu)
    check("out", out.view(-1, C), ro, CONV + HALF[dtype])
    check("final_state", fin, rf, 0.0)
    g = cdr.short_conv_bwd(d["x"].view(shape), d["weight"], d["dout"].view(shape), d["bias"], d["init"],
                           dfinal_state=d["dfin"], cu_seqlens=cu, silu=silu)
    rx, rw, rb, rs = grads([ro, rf], [h["dout"], h["dfin"]], [x, w, bi, st])
    check("dx", g["dx"].view(-1, C), rx, CONV + HALF[dtype])
    check("dweight", g["dweight"], rw, CONV)
    if bias:
        check("dbias", g["dbias"], rb, CONV)
    if state:
        check("dinitial_state", g["dinitial_state"], rs, CONV + HALF[dtype])
    else:
        assert g["dinitial_state"] is None
    torch.cuda.synchronize()
    assert cdr.get_last_error() == 0


@pytest.mark.parametrize("C,W,dtype", [(64, 4, BF), (13, 3, F32), (2048, 2, BF)])
def test_conv_steps_continue_a_prompt(C, W, dtype):
    B, T, steps = 3, 21, 5
    h = conv_inputs(B * (T + steps), B, C, W, dtype, 5, True, True)
    d = dev(h)
    x = d["x"].view(B, T + steps, C)
    whole, last = cdr.short_conv(x, d["weight"], d["bias"], d["init"])
    out, state = cdr.short_conv(x[:, :T].contiguous(), d["weight"], d["bias"], d["init"])
    outs = [out]
    for t in range(T, T + steps):
        outs.append(cdr.short_conv_step(x[:, t].contiguous(), d["weight"], state, d["bias"])[:, None])
    # the same products in the same order
    assert torch.equal(torch.cat(outs, 1), whole) and torch.equal(state, last)


# ---------------------------------------------------------------- selective scan

def scan_inputs(tokens, nseq, C, G, N, dtype, seed, opts):
    g = gen(seed)
    return dict(x=rnd(g, tokens, C, dtype=dtype), dt=rnd(g, tokens, C, dtype=dtype),
                A_log=torch.log(torch.arange(1, N + 1, dtype=F32)).expand(C, N).contiguous() + rnd(g, C, N, std=0.1),
                Bm=rnd(g, tokens, G, N, dtype=dtype), Cm=rnd(g, tokens, G, N, dtype=dtype),
                D=rnd(g, C) if "D" in opts else None, dt_bias=rnd(g, C) - 3 if "b" in opts else None,
                z=rnd(g, tokens, C, dtype=dtype) if "z" in opts else None,
                h0=rnd(g, nseq, C, N) if "h" in opts else None, dout=rnd(g, tokens, C, dtype=dtype),
                dh=rnd(g, nseq, C, N) if "h" in opts else None)


TOKEN_KEYS = ("x", "dt", "Bm", "Cm", "z", "dout")
IN_KEYS = ("x", "dt", "A_log", "Bm", "Cm", "D", "dt_bias", "z", "h0")


def scan_args(d, lead=None):
    """Positional and keyword arguments of selective_scan, token tensors in shape ``lead``."""
    v = {k: (t if t is None or lead is None or k not in TOKEN_KEYS else t.view(*lead, *t.shape[1:])) for k, t in d.items()}
    return [v[k] for k in ("x", "dt", "A_log", "Bm", "Cm")], {k: v[k] for k in ("D", "dt_bias", "z", "h0")}, v


def scan_reference(h, b, backward=True):
    l = [leaf(h[k]) for k in IN_KEYS]
    ro, rh = ref.selective_scan(*l[:5], D=l[5], dt_bias=l[6], z=l[7], h0=l[8], bounds=b)
    return ro, rh, dict(zip(IN_KEYS, grads([ro, rh], [h["dout"], h["dh"]], l))) if backward else None


SCAN_CASES = [  # lengths, C, G, N, dtype, options: D skip, dt bias, z gate, h states
    ([70], 64, 1, 16, BF, "Dbzh"),
    ([130, 130], 37, 1, 16, F32, "Dbzh"),
    ([9, 9, 9], 130, 2, 16, BF, "bh"),
    ([8, 8], 96, 3, 8, F32, "Dz"),
    ([1, 1], 33, 1, 16, F32, "Dbzh"),
    ([7], 6, 2, 8, BF, ""),
    ([65, 65], 40, 1, 32, F32, "Dbzh"),
    ([40], 20, 2, 64, BF, "Dbzh"),
    ([23], 10, 1, 128, F32, "bzh"),
    ([5, 0, 1, 16, 70, 17, 0, 8], 48, 1, 16, BF, "Dbzh"),
    ([3, 100, 0, 31], 35, 1, 8, F32, "Dbh"),
    ([250, 2, 47], 264, 2, 16, F32, "Dbzh"),
]


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("lengths,C,G,N,dtype,opts", SCAN_CASES)
def test_scan(lengths, C, G, N, dtype, opts, packed):
    if not packed and len(set(lengths)) > 1:
        pytest.skip("a batch has sequences of one length")
    b, n = bounds_of(lengths), len(lengths)
    h = scan_inputs(b[-1], n, C, G, N, dtype, 11 + C + N, opts)
    lead = (b[-1],) if packed else (n, lengths[0])
    cu = torch.tensor(b, dtype=torch.int32, device="cuda") if packed else None
    a, kw, v = scan_args(dev(h), lead)
    out, hf = cdr.selective_scan(*a, **kw, cu_seqlens=cu)
    ro, rh, rg = scan_reference(h, b)
    check("out", out.view(-1, C), ro, SCAN + HALF[dtype])
    check("h_final", hf, rh, SCAN)
    g = cdr.selective_scan_bwd(*a, v["dout"], **kw, dh_final=v["dh"], cu_seqlens=cu)
    for k in IN_KEYS:
        got = g["d" + k]
        if h[k] is None:
            assert got is None
            continue
        tol = SCAN_BWD + (HALF[dtype] if k in TOKEN_KEYS else 0.0)
        check("d" + k, got.view(h[k].shape), rg[k], tol)
    torch.cuda.synchronize()
    assert cdr.get_last_error() == 0


@pytest.mark.parametrize("lengths,C,G,N,dtype", [([1000], 33, 1, 16, F32), ([700, 700], 64, 2, 8, BF), ([1537], 24, 1, 64, BF),
                                                 ([3, 0, 900, 1, 0, 130, 640, 0], 40, 1, 16, F32),
                                                 ([256, 256, 0, 512, 31, 1], 16, 1, 32, BF), ([0, 0, 1500, 0], 10, 1, 128, F32)])
def test_scan_in_pieces(lengths, C, G, N, dtype):
    # few channels and many tokens: the split form.  Some sequences end, start or are empty
    # where a piece does; the state is carried in place.
    b, n = bounds_of(lengths), len(lengths)
    packed = len(set(lengths)) > 1
    assert cdr.library().comba_selective_scan_fwd_workspace_size(n, b[-1] if packed else lengths[0], C, G, N, int(packed)) > 0
    h = scan_inputs(b[-1], n, C, G, N, dtype, 5 + n, "Dbzh")
    h["dt_bias"] -= 2          # decays slow enough for the pieces to matter
    lead = (b[-1],) if packed else (n, lengths[0])
    cu = torch.tensor(b, dtype=torch.int32, device="cuda") if packed else None
    a, kw, v = scan_args(dev(h), lead)
    ro, rh, rg = scan_reference(h, b)
    out, hf = cdr.selective_scan(*a, **kw, cu_seqlens=cu)
    # twice the roundings of 300 tokens and more of them: sqrt(1600 / 300) times SCAN
    check("out", out.view(-1, C), ro, 3 * SCAN + HALF[dtype])
    check("h_final", hf, rh, 3 * SCAN)
    state = kw["h0"].clone()
    out2, _ = cdr.selective_scan(*a, **dict(kw, h0=state), h_final=state, cu_seqlens=cu)
    assert torch.equal(out2, out) and torch.equal(state, hf)
    g = cdr.selective_scan_bwd(*a, v["dout"], **kw, dh_final=v["dh"], cu_seqlens=cu)
    for k in IN_KEYS:
        check("d" + k, g["d" + k].view(h[k].shape), rg[k], 3 * SCAN_BWD + (HALF[dtype] if k in TOKEN_KEYS else 0.0))
    # without states and gate, and again: the same bits
    kw = dict(kw, h0=None, z=None)
    g, g2 = (cdr.selective_scan_bwd(*a, v["dout"], **kw, cu_seqlens=cu) for _ in range(2))
    assert all(torch.equal(g[k], g2[k]) for k in g if g[k] is not None)
    _, _, rg = scan_reference(dict(h, h0=None, z=None, dh=None), b)
    for k in ("x", "dt", "A_log", "Bm", "Cm", "D", "dt_bias"):
        check("d" + k, g["d" + k].view(h[k].shape), rg[k], 3 * SCAN_BWD + (HALF[dtype] if k in TOKEN_KEYS else 0.0))
    torch.cuda.synchronize()
    assert cdr.get_last_error() == 0


def test_scan_gradients_against_differences():
    # The kernel's gradient along a random direction of every input against a central
    # difference of the float64 definition: its error is h^2 times a third derivative of
    # order 1, with h = 1e-5 far below the fp32 gradients' 1e-4.
    b = bounds_of([21, 0, 12])
    h = scan_inputs(33, 3, 18, 2, 16, F32, 3, "Dbzh")
    a, kw, v = scan_args(dev(h))
    g = cdr.selective_scan_bwd(*a, v["dout"], **kw, dh_final=v["dh"], cu_seqlens=torch.tensor(b, dtype=torch.int32).cuda())
    gg = gen(77)
    for k in IN_KEYS:
        dir_ = torch.randn(h[k].shape, generator=gg, dtype=torch.float64)

        def loss(eps):
            l = [h[q].double() + (eps * dir_ if q == k else 0) for q in IN_KEYS]
            o, f = ref.selective_scan(*l[:5], D=l[5], dt_bias=l[6], z=l[7], h0=l[8], bounds=b)
            return float((o * h["dout"].double()).sum() + (f * h["dh"].double()).sum())

        want = (loss(1e-5) - loss(-1e-5)) / 2e-5
        got = float((g["d" + k].double().cpu() * dir_).sum())
        scale = float(g["d" + k].double().norm().cpu())   # of the projection's random sum
        assert abs(got - want) <= 3e-4 * scale, (k, got, want)


@pytest.mark.parametrize("T", [0, 1, 13])
def test_scan_steps_continue_a_prompt(T):
    B, C, G, N, steps = 2, 72, 2, 16, 4
    h = scan_inputs(B * (T + steps), B, C, G, N, BF, 21, "Dbzh")
    d = dev(h)
    cut = lambda k, s: None if d[k] is None else d[k].view(B, T + steps, *d[k].shape[1:])[:, s].contiguous()
    part = dict(d, **{k: cut(k, slice(0, T)) for k in TOKEN_KEYS})
    a, kw, _ = scan_args(part)
    out, state = cdr.selective_scan(*a, **kw)
    outs = [out]
    for t in range(T, T + steps):
        s = dict(d, **{k: cut(k, t) for k in TOKEN_KEYS})
        outs.append(cdr.selective_scan_step(s["x"], s["dt"], s["A_log"], s["Bm"], s["Cm"], state, D=s["D"],
                                            dt_bias=s["dt_bias"], z=s["z"])[:, None])
    b = [0, T + steps, 2 * (T + steps)]
    ro, rh, _ = scan_reference(h, b, backward=False)
    check("out", torch.cat(outs, 1).view(-1, C), ro, SCAN + HALF[BF])
    check("state", state, rh, SCAN)


def test_scan_state_carried_in_place_and_in_pieces():
    h = scan_inputs(60, 1, 48, 1, 16, F32, 9, "Dbzh")
    a, kw, v = scan_args(dev(h), (1, 60))
    whole, hf = cdr.selective_scan(*a, **kw)
    state = kw["h0"].clone()
    outs = []
    for s in (slice(0, 8), slice(8, 9), slice(9, 60)):
        p = {k: (t[:, s].contiguous() if k in TOKEN_KEYS and t is not None else t) for k, t in v.items()}
        pa, pk, _ = scan_args(dict(p, h0=state))
        o, hs = cdr.selective_scan(*pa, **pk, h_final=state)
        assert hs is state
        outs.append(o)
    check("out", torch.cat(outs, 1), whole, SCAN)
    check("state", state, hf, SCAN)


def test_scan_padding_tokens_leave_the_state():
    # dt = -inf: delta is 0, the state stays as it is and the token's own gradients vanish
    h = scan_inputs(20, 1, 16, 1, 16, F32, 4, "bh")
    h["dt"][12:] = -float("inf")
    a, kw, v = scan_args(dev(h), (1, 20))
    out, hf = cdr.selective_scan(*a, **kw)
    short = {k: (t[:12] if k in TOKEN_KEYS and t is not None else t) for k, t in h.items()}
    ro, rh, _ = scan_reference(short, [0, 12], backward=False)
    check("state", hf, rh, SCAN)
    check("out", out[0, :12], ro, SCAN)
    before = {k: (t[:, :12].contiguous() if k in TOKEN_KEYS and t is not None else t) for k, t in v.items()}
    ba, bk, _ = scan_args(before)
    assert torch.equal(hf, cdr.selective_scan(*ba, **bk)[1])     # not a bit moves
    g = cdr.selective_scan_bwd(*a, v["dout"], **kw, dh_final=v["dh"])
    for k in ("dx", "ddt", "dBm"):
        assert bool((g[k][0, 12:] == 0).all()), k
    assert all(bool(torch.isfinite(t).all()) for t in g.values() if t is not None)


def test_scan_extreme_decays():
    # A of -e^8 forgets at once, of -e^-12 hardly ever; large steps; all finite and right
    h = scan_inputs(200, 1, 32, 1, 16, F32, 15, "Dzh")
    h["A_log"][:8] = 8.0
    h["A_log"][8:16] = -12.0
    h["dt"][:, ::4] += 30.0
    a, kw, v = scan_args(dev(h), (1, 200))
    out, hf = cdr.selective_scan(*a, **kw)
    ro, rh, rg = scan_reference(h, [0, 200])
    check("out", out[0], ro, SCAN)
    check("h_final", hf, rh, SCAN)
    g = cdr.selective_scan_bwd(*a, v["dout"], **kw, dh_final=v["dh"])
    for k in IN_KEYS:
        if h[k] is not None:
            check("d" + k, g["d" + k].view(h[k].shape), rg[k], SCAN_BWD)


def test_nothing_behind_the_last_sequence_is_touched():
    b = [0, 9, 9, 25]
    tokens, C, N = 40, 24, 16
    cu = torch.tensor(b, dtype=torch.int32).cuda()
    h = conv_inputs(tokens, 3, C, 4, BF, 3, True, True)
    d = dev(h)
    out = torch.full((tokens, C), 7.0, dtype=BF, device="cuda")
    cdr.short_conv(d["x"], d["weight"], d["bias"], d["init"], cu_seqlens=cu, out=out)
    assert bool((out[25:] == 7).all())
    ro, _ = ref.short_conv(h["x"][:25], h["weight"], h["bias"], h["init"], b)
    check("conv", out[:25], ro, CONV + HALF[BF])
    h = scan_inputs(tokens, 3, C, 1, N, F32, 3, "Dbzh")
    h["x"][25:] = float("nan")          # what lies there does not reach the sums
    h["Bm"][25:] = float("nan")
    a, kw, v = scan_args(dev(h))
    out = torch.full((tokens, C), 7.0, device="cuda")
    cdr.selective_scan(*a, **kw, cu_seqlens=cu, out=out)
    assert bool((out[25:] == 7).all())
    short = {k: (t[:25] if k in TOKEN_KEYS and t is not None else t) for k, t in h.items()}
    ro, rh, rg = scan_reference(short, b)
    check("scan", out[:25], ro, SCAN)
    g = cdr.selective_scan_bwd(*a, v["dout"], **kw, dh_final=v["dh"], cu_seqlens=cu)
    for k in IN_KEYS:
        check("d" + k, g["d" + k][:25] if k in TOKEN_KEYS else g["d" + k], rg[k], SCAN_BWD)


def test_malformed_bounds_in_pieces_are_reported():
    cu = torch.tensor([0, 300, 5000, 800], dtype=torch.int32).cuda()
    lib, T, C, N = cdr.library(), 1000, 16, 16
    assert min(lib.comba_selective_scan_fwd_workspace_size(3, T, C, 1, N, 1),
               lib.comba_selective_scan_bwd_workspace_size(3, T, C, 1, N, 1)) > 0
    h = scan_inputs(T, 3, C, 1, N, F32, 3, "Dbzh")
    a, kw, v = scan_args(dev(h))
    out, _ = cdr.selective_scan(*a, **kw, cu_seqlens=cu)
    torch.cuda.synchronize()
    assert cdr.get_last_error() == -1
    g = cdr.selective_scan_bwd(*a, v["dout"], **kw, cu_seqlens=cu)
    torch.cuda.synchronize()
    assert cdr.get_last_error() == -1 and cdr.get_last_error() == 0
    first = {k: (t[:300] if k in TOKEN_KEYS and t is not None else t) for k, t in h.items()}
    ro, _, rg = scan_reference(dict(first, dh=None), [0, 300])
    check("out of the sound sequence", out[:300], ro, SCAN)
    check("its dx", g["dx"][:300], rg["x"], SCAN_BWD)


def test_tokens_without_any_sequence():
    cu = torch.zeros(1, dtype=torch.int32, device="cuda")     # N = 0
    d = dev(conv_inputs(30, 0, 16, 4, BF, 3, True, True))
    a, kw, v = scan_args(dev(scan_inputs(30, 0, 16, 1, 16, BF, 3, "Dbzh")))
    out = torch.full((30, 16), 7.0, dtype=BF, device="cuda")
    cdr.short_conv(d["x"], d["weight"], d["bias"], d["init"], cu_seqlens=cu, out=out)
    cdr.selective_scan(*a, **kw, cu_seqlens=cu, out=out)
    assert bool((out == 7).all())
    g = cdr.short_conv_bwd(d["x"], d["weight"], d["dout"], d["bias"], d["init"], cu_seqlens=cu)
    assert bool((g["dweight"] == 0).all()) and bool((g["dbias"] == 0).all())
    g = cdr.selective_scan_bwd(*a, v["dout"], **kw, cu_seqlens=cu)
    assert all(bool((g[k] == 0).all()) for k in ("dA_log", "dD", "ddt_bias"))
    torch.cuda.synchronize()
    assert cdr.get_last_error() == 0


def test_malformed_bounds_are_reported():
    # sequence 1 ends past the packed tokens, sequence 2 runs backwards
    cu = torch.tensor([0, 10, 300, 20], dtype=torch.int32).cuda()
    C, N = 16, 16
    d = dev(conv_inputs(20, 3, C, 4, BF, 3, True, True))
    ins = (d["x"], d["weight"])
    h = scan_inputs(20, 3, C, 1, N, BF, 3, "Dbzh")
    a, kw, v = scan_args(dev(h))
    for call in (lambda: cdr.short_conv(*ins, d["bias"], d["init"], cu_seqlens=cu),
                 lambda: cdr.short_conv(*ins, d["bias"], d["init"], cu_seqlens=cu, return_state=False),
                 lambda: cdr.short_conv_bwd(*ins, d["dout"], d["bias"], cu_seqlens=cu),
                 lambda: cdr.selective_scan(*a, **kw, cu_seqlens=cu),
                 lambda: cdr.selective_scan_bwd(*a, v["dout"], **kw, cu_seqlens=cu)):
        call()
        torch.cuda.synchronize()
        assert cdr.get_last_error() == -1
    assert cdr.get_last_error() == 0
    out, _ = cdr.selective_scan(*a, **kw, cu_seqlens=cu)
    cdr.get_last_error()
    ro, _ = ref.selective_scan(*[h[k][:10] if k in TOKEN_KEYS else h[k] for k in ("x", "dt", "A_log", "Bm", "Cm")],
                               D=h["D"], dt_bias=h["dt_bias"], z=h["z"][:10], h0=h["h0"], bounds=[0, 10])
    check("the sound sequence", out[:10], ro, SCAN + HALF[BF])


# ---------------------------------------------------------------- norms

WIDTHS = [1, 7, 8, 64, 100, 128, 129, 256, 1000, 2048, 2050, 4096, 5001, 8192]


@pytest.mark.parametrize("D", WIDTHS)
@pytest.mark.parametrize("dtype,rows", [(BF, 35), (F32, 1), (F32, 1300)])
def test_gated_norm(D, dtype, rows):
    if rows > 1000 and D > 2050:
        rows = 300
    g = gen(D + rows)
    x, gate, w, dout = rnd(g, rows, D, dtype=dtype), rnd(g, rows, D, dtype=dtype), rnd(g, D), rnd(g, rows, D, dtype=dtype)
    x[0] = 0          # a row of zeros: 1 / sqrt(eps)
    out = cdr.gated_norm(x.cuda(), gate.cuda(), w.cuda())
    l = [leaf(x), leaf(gate), leaf(w)]
    ro = ref.gated_norm(*l)
    check("out", out, ro, NORM + HALF[dtype])
    b = cdr.gated_norm_bwd(x.cuda(), gate.cuda(), w.cuda(), dout.cuda())
    rx, rg, rw = grads([ro], [dout], l)
    # the row of zeros has gradients of 1 / sqrt(eps) times the others': on its own
    check("dx row 0", b["dx"][0], rx[0], NORM + HALF[dtype])
    check("dx", b["dx"][1:], rx[1:], NORM + HALF[dtype])
    check("dgate", b["dgate"], rg, NORM + HALF[dtype])
    check("dweight", b["dweight"], rw, NORM)


@pytest.mark.parametrize("D", WIDTHS)
@pytest.mark.parametrize("dtype,rdtype,rows,opts", [(BF, BF, 35, "sp"), (BF, F32, 70, "p"), (F32, F32, 1, "s"),
                                                    (F32, F32, 700, "spd"), (BF, F32, 3, "d"), (BF, BF, 900, "d")])
def test_residual_norm(D, dtype, rdtype, rows, opts):
    if rows > 100 and D > 2050:
        rows = 170
    g = gen(D + rows)
    x, res = rnd(g, rows, D, dtype=dtype), rnd(g, rows, D, dtype=rdtype)
    w, sc, po = rnd(g, D), rnd(g, D) if "s" in opts else None, rnd(g, D) if "p" in opts else None
    dy, dh = rnd(g, rows, D, dtype=dtype), rnd(g, rows, D, dtype=rdtype) if "d" in opts else None
    c = lambda t: None if t is None else t.cuda()
    out, h = cdr.residual_norm(c(x), c(res), c(w), c(sc), c(po))
    l = [leaf(t) for t in (x, res, w, sc, po)]
    ro, rh = ref.residual_norm(*l, stored=h.cpu())
    check("h", h, rh, NORM + HALF[rdtype])
    check("out", out, ro, NORM + HALF[dtype])
    b = cdr.residual_norm_bwd(c(x), h, c(w), c(dy), c(dh), c(sc), c(po))
    rg = grads([ro, rh], [dy, dh], l)
    # gradients pass two chained norms: twice the roundings.  A width of 1 divides by the
    # value itself, so that its exact gradient is a difference of near equals: of eps only.
    tol = 2 * NORM
    if D > 1:
        check("dx", b["dx"], rg[0], tol + HALF[dtype])
        check("dresidual", b["dresidual"], rg[1], tol + HALF[rdtype])
        for k, want in (("dscale", rg[3]), ("dpost_weight", rg[4])):
            if want is None:
                assert b[k] is None
            else:
                check(k, b[k], want, tol)
    check("dweight", b["dweight"], rg[2], tol)
    # in place on the residual stream: the same values
    stream_t = c(res).clone()
    out2, h2 = cdr.residual_norm(c(x), stream_t, c(w), c(sc), c(po), h=stream_t)
    assert h2 is stream_t and torch.equal(h2, h) and torch.equal(out2, out)


def test_empty_calls():
    z = lambda *s, dtype=F32: torch.zeros(s, dtype=dtype, device="cuda")
    o, s = cdr.short_conv(z(2, 0, 8), z(8, 4), initial_state=z(2, 3, 8) + 5)
    assert o.shape == (2, 0, 8) and bool((s == 5).all())
    g = cdr.short_conv_bwd(z(2, 0, 8), z(8, 4), z(2, 0, 8), initial_state=z(2, 3, 8), dfinal_state=z(2, 3, 8) + 2)
    assert bool((g["dweight"] == 0).all()) and bool((g["dinitial_state"] == 2).all())
    o, h = cdr.selective_scan(z(2, 0, 8), z(2, 0, 8), z(8, 16), z(2, 0, 1, 16), z(2, 0, 1, 16), h0=z(2, 8, 16) + 3)
    assert bool((h == 3).all())
    g = cdr.selective_scan_bwd(z(2, 0, 8), z(2, 0, 8), z(8, 16), z(2, 0, 1, 16), z(2, 0, 1, 16), z(2, 0, 8),
                               h0=z(2, 8, 16), dh_final=z(2, 8, 16) + 4)
    assert bool((g["dh0"] == 4).all()) and bool((g["dA_log"] == 0).all())
    assert cdr.selective_scan(z(0, 5, 8), z(0, 5, 8), z(8, 16), z(0, 5, 1, 16), z(0, 5, 1, 16))[0].shape == (0, 5, 8)
    g = cdr.selective_scan_bwd(z(0, 5, 8), z(0, 5, 8), z(8, 16), z(0, 5, 1, 16), z(0, 5, 1, 16), z(0, 5, 8))
    assert bool((g["dA_log"] == 0).all())
    assert cdr.gated_norm(z(0, 64), z(0, 64), z(64)).shape == (0, 64)
    assert bool((cdr.gated_norm_bwd(z(0, 64), z(0, 64), z(64), z(0, 64))["dweight"] == 0).all())
    g = cdr.residual_norm_bwd(z(0, 64), z(0, 64), z(64), z(0, 64), scale=z(64), post_weight=z(64))
    assert all(bool((g[k] == 0).all()) for k in ("dweight", "dscale", "dpost_weight"))
    torch.cuda.synchronize()
    assert cdr.get_last_error() == 0


# ---------------------------------------------------------------- streams, graphs, repeats

def every_operator(seed, dtype=BF):
    """Closures over fresh inputs, one per operator call, each returning a list of tensors."""
    C, N, B, T = 136, 16, 2, 50
    c = dev(conv_inputs(B * T, B, C, 4, dtype, seed, True, True))
    x = c["x"].view(B, T, C)
    a, kw, v = scan_args(dev(scan_inputs(B * T, B, C, 2, N, dtype, seed, "Dbzh")), (B, T))
    g = gen(seed + 1)
    y, gate, dy = (rnd(g, 500, 128, dtype=dtype).cuda() for _ in range(3))
    w, sc, po = (rnd(g, 128).cuda() for _ in range(3))
    res, dh = rnd(g, 500, 128).cuda(), rnd(g, 500, 128).cuda()
    flat = lambda r: [t for t in (r.values() if isinstance(r, dict) else r if isinstance(r, tuple) else [r]) if t is not None]
    return {
        "conv": lambda **k: flat(cdr.short_conv(x, c["weight"], c["bias"], c["init"], **k)),
        "conv_bwd": lambda **k: flat(cdr.short_conv_bwd(x, c["weight"], c["dout"].view(B, T, C), c["bias"], c["init"], c["dfin"], **k)),
        "conv_step": lambda **k: flat(cdr.short_conv_step(x[:, 0].contiguous(), c["weight"], c["init"].clone(), c["bias"], **k)),
        "scan": lambda **k: flat(cdr.selective_scan(*a, **kw, **k)),
        "scan_bwd": lambda **k: flat(cdr.selective_scan_bwd(*a, v["dout"], **kw, dh_final=v["dh"], **k)),
        "scan_step": lambda **k: flat(cdr.selective_scan_step(*[t[:, 0].contiguous() if t.dim() > 2 else t for t in a],
                                                              kw["h0"].clone(), kw["D"], kw["dt_bias"], kw["z"][:, 0].contiguous(), **k)),
        "gated": lambda **k: flat(cdr.gated_norm(y, gate, w, **k)),
        "gated_bwd": lambda **k: flat(cdr.gated_norm_bwd(y, gate, w, dy, **k)),
        "residual": lambda **k: flat(cdr.residual_norm(y, res, w, sc, po, **k)),
        "residual_bwd": lambda **k: flat(cdr.residual_norm_bwd(y, res, w, dy, dh, sc, po, **k)),
    }


OPERATORS = ["conv", "conv_bwd", "conv_step", "scan", "scan_bwd", "scan_step", "gated", "gated_bwd", "residual", "residual_bwd"]


@pytest.mark.parametrize("name", OPERATORS)
def test_repeats_streams_and_graphs_give_the_same_bits(name):
    call, other = every_operator(1)[name], every_operator(2)[name]
    want, want2 = call(), other()
    again = call()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(want, again))
    # two calls at once, each on a stream of its own
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for s in (s1, s2):
        s.wait_stream(torch.cuda.current_stream())
    if name.endswith("step"):      # its closure clones on the current stream
        with torch.cuda.stream(s1):
            got = call()
        with torch.cuda.stream(s2):
            got2 = other()
    else:
        got, got2 = call(stream=s1), other(stream=s2)
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(want, got)) and all(torch.equal(p, q) for p, q in zip(want2, got2))
    # two captured graphs, replayed in turn and then at once
    graphs = []
    for f in (call, other):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            res = f()
        graphs.append((gr, res))
    for gr, res in graphs:
        for t in res:
            t.zero_()
    for _ in range(2):
        with torch.cuda.stream(s1):
            graphs[0][0].replay()
        with torch.cuda.stream(s2):
            graphs[1][0].replay()
        torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(want, graphs[0][1]))
    assert all(torch.equal(p, q) for p, q in zip(want2, graphs[1][1]))


def test_unaligned_token_tensors():
    # contiguous views that start 2 bytes into a 16-byte line: the scalar path
    for C, T in ((16, 40), (17, 33)):
        h = conv_inputs(T, 1, C, 4, BF, 5, True, False)
        buf = torch.empty(T * C + 1, dtype=BF, device="cuda")
        x = buf[1:].view(1, T, C)
        x.copy_(h["x"].view(1, T, C))
        out, _ = cdr.short_conv(x, h["weight"].cuda(), h["bias"].cuda())
        check("conv", out[0], ref.short_conv(h["x"], h["weight"], h["bias"], None, [0, T])[0], CONV + HALF[BF])
        w = torch.rand(C)
        out = cdr.gated_norm(x, x, w.cuda())
        check("gated", out[0], ref.gated_norm(h["x"], h["x"], w), NORM + HALF[BF])
        h = scan_inputs(T, 1, C, 1, 16, BF, 5, "Dbz")
        d = dev(h)
        x.copy_(h["x"].view(1, T, C))
        a, kw, _ = scan_args(d, (1, T))
        out, _ = cdr.selective_scan(x, *a[1:], **kw)
        check("scan", out[0], scan_reference(h, [0, T], False)[0], SCAN + HALF[BF])


# ---------------------------------------------------------------- together

def test_a_block_with_its_gradients():
    """residual_norm -> projection -> short_conv -> selective_scan -> gated_norm ->
    projection -> residual_norm, and back, against autograd of the definitions."""
    B, T, M, C, N, G, W, eps = 2, 37, 64, 96, 16, 1, 4, 1e-6
    g = gen(1234)
    h = {"x0": rnd(g, B * T, M), "stream": rnd(g, B * T, M), "w1": 1 + rnd(g, M, std=0.1), "w2": 1 + rnd(g, M, std=0.1),
         "sc": rnd(g, M), "po": 1 + rnd(g, M, std=0.1), "Wx": rnd(g, M, C, std=M ** -0.5), "Wdt": rnd(g, M, C, std=M ** -0.5),
         "Wg": rnd(g, M, C, std=M ** -0.5), "Wb": rnd(g, M, N, std=M ** -0.5), "Wc": rnd(g, M, N, std=M ** -0.5),
         "cw": rnd(g, C, W, std=0.5), "cb": rnd(g, C, std=0.1), "A_log": rnd(g, C, N, std=0.3), "D": rnd(g, C),
         "dtb": rnd(g, C) - 2, "gn": 1 + rnd(g, C, std=0.1), "Wo": rnd(g, C, M, std=C ** -0.5)}
    dy, dh = rnd(g, B * T, M), rnd(g, B * T, M)
    l = {k: leaf(v) for k, v in h.items()}
    b = [0, T, 2 * T]
    y1, s1 = ref.residual_norm(l["x0"], l["stream"], l["w1"])
    u, _ = ref.short_conv(y1 @ l["Wx"], l["cw"], l["cb"], None, b)
    m, _ = ref.selective_scan(u, y1 @ l["Wdt"], l["A_log"], (y1 @ l["Wb"])[:, None], (y1 @ l["Wc"])[:, None], l["D"], l["dtb"],
                              None, None, b)
    o = ref.gated_norm(m, y1 @ l["Wg"], l["gn"])
    y2, s2 = ref.residual_norm(o @ l["Wo"], s1, l["w2"], l["sc"], l["po"])
    want = dict(zip(l, grads([y2, s2], [dy, dh], list(l.values()))))
    # the library's calls; the projections' own gradients in float64 on the host values
    d = dev(h)
    dd = lambda t: t.double()
    prod = lambda p, q: (dd(p) @ dd(q)).float()
    k1, t1 = cdr.residual_norm(d["x0"], d["stream"], d["w1"])
    px, pdt, pg, pb, pc = (prod(k1, d[n]) for n in ("Wx", "Wdt", "Wg", "Wb", "Wc"))
    v3 = lambda t: t.view(B, T, -1)
    cu, _ = cdr.short_conv(v3(px), d["cw"], d["cb"])
    sa = (cu, v3(pdt), d["A_log"], v3(pb)[:, :, None], v3(pc)[:, :, None])
    sm, _ = cdr.selective_scan(*sa, D=d["D"], dt_bias=d["dtb"])
    go = cdr.gated_norm(sm.view(-1, C), pg, d["gn"])
    po = prod(go, d["Wo"])
    k2, t2 = cdr.residual_norm(po, t1, d["w2"], d["sc"], d["po"])
    check("out", k2, y2, SCAN)
    check("stream", t2, s2, SCAN)
    r2 = cdr.residual_norm_bwd(po, t2, d["w2"], dy.cuda(), dh.cuda(), d["sc"], d["po"])
    dWo, dgo = prod(go.t(), r2["dx"]), prod(r2["dx"], d["Wo"].t())
    rg = cdr.gated_norm_bwd(sm.view(-1, C), pg, d["gn"], dgo)
    rs = cdr.selective_scan_bwd(*sa, rg["dx"].view(B, T, C), D=d["D"], dt_bias=d["dtb"])
    rc = cdr.short_conv_bwd(v3(px), d["cw"], rs["dx"], d["cb"])
    back = {"Wx": rc["dx"].view(-1, C), "Wdt": rs["ddt"].view(-1, C), "Wg": rg["dgate"], "Wb": rs["dBm"].view(-1, N),
            "Wc": rs["dCm"].view(-1, N)}
    dk1 = sum(dd(t) @ dd(d[n]).t() for n, t in back.items()).float()
    r1 = cdr.residual_norm_bwd(d["x0"], t1, d["w1"], dk1, r2["dresidual"])
    got = {"x0": r1["dx"], "stream": r1["dresidual"], "w1": r1["dweight"], "w2": r2["dweight"], "sc": r2["dscale"],
           "po": r2["dpost_weight"], "cw": rc["dweight"], "cb": rc["dbias"], "A_log": rs["dA_log"], "D": rs["dD"],
           "dtb": rs["ddt_bias"], "gn": rg["dweight"], "Wo": dWo, **{n: prod(k1.t(), t) for n, t in back.items()}}
    for k in h:
        check("d" + k, got[k], want[k], SCAN_BWD)


def test_comba_block_prompt_then_decode():
    """short_conv of q, k, v -> the chunk forward -> gated_norm for a prompt, then one token
    through the single-token forms, against the definitions over all tokens."""
    B, T, H, D, W = 2, 67, 2, 128, 4
    C = 3 * H * D
    g = gen(99)
    x, w = rnd(g, B, T + 1, C, dtype=BF), rnd(g, C, W, std=0.5)
    la = (-0.1 * torch.rand(B, T + 1, H, generator=g)).float()
    be, dvec = torch.rand(B, T + 1, H, generator=g).float(), torch.rand(H, generator=g).float()
    gate, gw = rnd(g, B, T + 1, H, D, dtype=BF), 1 + rnd(g, D, std=0.1)

    def heads(u):
        q, k, v = u.reshape(*u.shape[:-1], 3, H, D).unbind(-3)
        unit = lambda t: torch.nn.functional.normalize(t.float(), dim=-1).to(BF)
        return unit(q).contiguous(), unit(k).contiguous(), v.contiguous()

    xd, wd = x.cuda(), w.cuda()
    u, conv_state = cdr.short_conv(xd[:, :T].contiguous(), wd)
    q, k, v = heads(u)
    o, S = cdr.chunk_fwd(q, k, v, la[:, :T].contiguous().cuda(), be[:, :T].contiguous().cuda(), dvec.cuda())
    y = cdr.gated_norm(o, gate[:, :T].contiguous().cuda(), gw.cuda())
    u1 = cdr.short_conv_step(xd[:, T].contiguous(), wd, conv_state)
    q1, k1, v1 = heads(u1)
    o1 = cdr.recurrent_step(q1, k1, v1, la[:, T].contiguous().cuda(), be[:, T].contiguous().cuda(), dvec.cuda(), S)
    y1 = cdr.gated_norm(o1, gate[:, T].contiguous().cuda(), gw.cuda())
    cu, _ = ref.short_conv(x.view(-1, C), w, None, None, [0, T + 1, 2 * (T + 1)])
    check("conv", torch.cat([u, u1[:, None]], 1).view(-1, C), cu, CONV + HALF[BF])
    cat = lambda p, r: torch.cat([p, r[:, None]], 1).cpu()
    ro, _ = oracle.recurrence(cat(q, q1), cat(k, k1), cat(v, v1), la, be, dvec)
    # the norm of what the recurrence gave: 5e-3 of the recurrence, and its own rounding
    want = ref.gated_norm(torch.from_numpy(np.asarray(ro)), gate, gw)
    check("block", cat(y, y1), want, 2 * 5e-3 + HALF[BF])


# ---------------------------------------------------------------- the caller's buffers, refusals

def test_the_callers_outputs_states_and_workspaces():
    C, B, T, N = 72, 2, 300, 16
    c = dev(conv_inputs(B * T, B, C, 4, BF, 8, True, True))
    x, lib = c["x"].view(B, T, C), cdr.library()
    want, wf = cdr.short_conv(x, c["weight"], c["bias"], c["init"])
    out, fin = torch.empty_like(x), torch.empty_like(c["init"])
    o, f = cdr.short_conv(x, c["weight"], c["bias"], c["init"], out=out, final_state=fin)
    assert o is out and f is fin and torch.equal(out, want) and torch.equal(fin, wf)
    assert cdr.short_conv(x, c["weight"], return_state=False)[1] is None
    ws = torch.empty(lib.comba_short_conv_bwd_workspace_size(B, T, C, 4, 0), dtype=torch.uint8, device="cuda")
    g, g2 = (cdr.short_conv_bwd(x, c["weight"], x, c["bias"], workspace=w) for w in (None, ws))
    assert all(torch.equal(g[k], g2[k]) for k in ("dx", "dweight", "dbias"))
    with pytest.raises(cdr.CombaError) as err:
        cdr.short_conv_bwd(x, c["weight"], x, c["bias"], workspace=ws[:16])
    assert err.value.status == -1
    a, kw, v = scan_args(dev(scan_inputs(B * T, B, C, 1, N, BF, 9, "Dbzh")), (B, T))
    want, wh = cdr.selective_scan(*a, **kw)
    out, hf = torch.empty_like(x), torch.empty_like(kw["h0"])
    ws = torch.empty(lib.comba_selective_scan_fwd_workspace_size(B, T, C, 1, N, 0) + 64, dtype=torch.uint8, device="cuda")
    o, h = cdr.selective_scan(*a, **kw, out=out, h_final=hf, workspace=ws)
    assert o is out and h is hf and torch.equal(out, want) and torch.equal(hf, wh)
    ws = torch.empty(lib.comba_selective_scan_bwd_workspace_size(B, T, C, 1, N, 0), dtype=torch.uint8, device="cuda")
    g, g2 = (cdr.selective_scan_bwd(*a, v["dout"], **kw, workspace=w) for w in (None, ws))
    assert all(torch.equal(g[k], g2[k]) for k in g)
    out = torch.empty_like(x)
    assert cdr.gated_norm(x, x, kw["D"], out=out) is out and torch.equal(out, cdr.gated_norm(x, x, kw["D"]))


def test_what_a_kernel_cannot_take_is_refused():
    x = torch.zeros(2, 6, 16, device="cuda")
    w, b = torch.zeros(16, 4, device="cuda"), torch.zeros(2, 6, 1, 16, device="cuda")
    A = torch.zeros(16, 16, device="cuda")
    for call in (lambda: cdr.short_conv(x.transpose(0, 1), w), lambda: cdr.short_conv(x, w.t().contiguous().t()),
                 lambda: cdr.short_conv(x, w, initial_state=torch.zeros(2, 2, 16, device="cuda")),
                 lambda: cdr.short_conv(x, w, out=x[:, :5]), lambda: cdr.short_conv(x, w.cpu()),
                 lambda: cdr.selective_scan(x[..., ::2], x[..., ::2], A[:8], b, b),
                 lambda: cdr.selective_scan(x, x, A, b, b[..., :8].contiguous()),
                 lambda: cdr.gated_norm(x, x.cpu(), A[0]), lambda: cdr.gated_norm(x[:, ::2], x[:, ::2], A[0]),
                 lambda: cdr.residual_norm(x, x[:1], A[0])):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: cdr.short_conv(x, w.bfloat16()), lambda: cdr.selective_scan(x, x.bfloat16(), A, b, b),
                 lambda: cdr.selective_scan(x, x, A, b.bfloat16(), b), lambda: cdr.gated_norm(x, x, A[0].bfloat16()),
                 lambda: cdr.residual_norm(x, x.bfloat16(), A[0])):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: cdr.short_conv(x, torch.zeros(16, 5, device="cuda")), lambda: cdr.short_conv(x, w, out=x),
                 lambda: cdr.selective_scan(x, x, A[:, :12].contiguous(), b[..., :12].contiguous(), b[..., :12].contiguous()),
                 lambda: cdr.selective_scan(x, x, A, b.repeat(1, 1, 3, 1), b.repeat(1, 1, 3, 1)),
                 lambda: cdr.gated_norm(x, x, A[0], out=x), lambda: cdr.gated_norm(x, x, A[0], eps=-1.0)):
        with pytest.raises(cdr.CombaError) as err:
            call()
        assert err.value.status == -1
    wide = torch.zeros(2, 8193, device="cuda")
    with pytest.raises(cdr.CombaError) as err:
        cdr.gated_norm(wide, wide, wide[0])
    assert err.value.status == -2


# ---------------------------------------------------------------- sizes past 32-bit offsets

def test_conv_and_norm_past_two_to_the_31_elements():
    T, C, tail = (1 << 20) + 37, 2056, 64          # 2.16e9 elements
    x = torch.randn(1, T, C, device="cuda", dtype=BF)
    w = torch.randn(C, 4, device="cuda") * 0.5
    out, fin = cdr.short_conv(x, w)
    assert torch.equal(fin[0], x[0, -3:])
    part, _ = cdr.short_conv(x[:, -tail:].contiguous(), w, initial_state=x[:, -tail - 3:-tail].contiguous())
    assert torch.equal(out[:, -tail:], part)
    g = cdr.short_conv_bwd(x, w, out)
    gp = cdr.short_conv_bwd(x[:, -tail:].contiguous(), w, out[:, -tail:].contiguous(),
                            initial_state=x[:, -tail - 3:-tail].contiguous())
    assert torch.equal(g["dx"][:, -tail:], gp["dx"])
    assert bool(torch.isfinite(g["dweight"]).all())
    del out, part, g, gp
    wn = torch.rand(C, device="cuda") + 0.5
    y = cdr.gated_norm(x, x, wn)
    assert torch.equal(y[:, -tail:], cdr.gated_norm(x[:, -tail:].contiguous(), x[:, -tail:].contiguous(), wn))
    b = cdr.gated_norm_bwd(x, x, wn, y)
    bp = cdr.gated_norm_bwd(x[:, -tail:].contiguous(), x[:, -tail:].contiguous(), wn, y[:, -tail:].contiguous())
    assert torch.equal(b["dx"][:, -tail:], bp["dx"]) and torch.equal(b["dgate"][:, -tail:], bp["dgate"])
    del b, bp
    o, h = cdr.residual_norm(x, y, wn, scale=wn)
    op, hp = cdr.residual_norm(x[:, -tail:].contiguous(), y[:, -tail:].contiguous(), wn, scale=wn)
    assert torch.equal(o[:, -tail:], op) and torch.equal(h[:, -tail:], hp)
    torch.cuda.synchronize()
    assert cdr.get_last_error() == 0


def test_scan_past_two_to_the_31_elements():
    T, C, N, tail = (1 << 20) + 48, 2056, 8, 96     # 2.16e9 elements, more in the states' table
    g = torch.Generator(device="cuda").manual_seed(1)
    rand = lambda *s: torch.randn(s, device="cuda", dtype=BF, generator=g)
    x, dt, Bm, Cm = rand(1, T, C), rand(1, T, C), rand(1, T, 1, N), rand(1, T, 1, N)
    A = torch.randn(C, N, device="cuda", generator=g) * 0.2
    bias = torch.full((C,), -4.0, device="cuda")
    cut = lambda t, s: t[:, s].contiguous()
    head, end = slice(0, T - tail), slice(T - tail, T)
    out, h = cdr.selective_scan(x, dt, A, Bm, Cm, dt_bias=bias)
    _, hm = cdr.selective_scan(*(cut(t, head) for t in (x, dt)), A, *(cut(t, head) for t in (Bm, Cm)), dt_bias=bias)
    po, ph = cdr.selective_scan(*(cut(t, end) for t in (x, dt)), A, *(cut(t, end) for t in (Bm, Cm)), dt_bias=bias, h0=hm)
    check("out", out[:, end], po, SCAN + HALF[BF])
    check("h_final", h, ph, SCAN)
    b = cdr.selective_scan_bwd(x, dt, A, Bm, Cm, out, dt_bias=bias)
    bp = cdr.selective_scan_bwd(*(cut(t, end) for t in (x, dt)), A, *(cut(t, end) for t in (Bm, Cm)), cut(out, end),
                                dt_bias=bias, h0=hm)
    for k in ("dx", "ddt", "dBm", "dCm"):
        check(k, b[k][:, end], bp[k], SCAN_BWD + 2 * HALF[BF])
    assert all(bool(torch.isfinite(b[k]).all()) for k in ("dA_log", "ddt_bias"))
    torch.cuda.synchronize()
    assert cdr.get_last_error() == 0


# ---------------------------------------------------------------- steps of many sequences

@pytest.mark.parametrize("B,C,W,dtype", [(1301, 936, 4, BF), (1303, 233, 3, F32)])
def test_conv_step_with_several_sequences_a_thread(B, C, W, dtype):
    # enough sequences for a thread to take four, and fewer for the last one
    h = conv_inputs(B, B, C, W, dtype, 41, True, True)
    d = dev(h)
    out = cdr.short_conv_step(d["x"], d["weight"], d["init"], d["bias"])
    ro, rf = ref.short_conv(h["x"], h["weight"], h["bias"], h["init"], list(range(B + 1)))
    check("out", out, ro, CONV + HALF[dtype])
    check("state", d["init"], rf, 0.0)


def test_conv_step_of_two_to_the_31_sequences():
    # small whole numbers: every product and sum is exact
    B = 2 ** 31 - 1
    x = (torch.arange(B, dtype=torch.int32, device="cuda") % 61).to(BF).view(B, 1)
    state = (torch.arange(B, dtype=torch.int32, device="cuda") % 59).to(BF).view(B, 1, 1)
    w = torch.tensor([[1.0, 2.0]], device="cuda")
    out = cdr.short_conv_step(x, w, state, silu=False)
    torch.cuda.synchronize()
    assert torch.equal(state.view(B, 1), x)
    x.mul_(2)
    out.sub_(x)             # 2 x + state is at most 178, exact in bf16, and so is the difference
    assert torch.equal(out.view(B), (torch.arange(B, dtype=torch.int32, device="cuda") % 59).to(BF))
    assert cdr.get_last_error() == 0


def test_packed_bounds_of_more_than_two_to_the_30_sequences():
    # nearly all of them empty; the tokens are in the last ones, the search ends behind 2^30
    N, T = 1_200_000_000, 300
    cu = torch.arange(N + 1, dtype=torch.int32, device="cuda").sub_(N - T).clamp_(min=0)
    cu[N - T + 100:N - T + 150] = 100       # empty ones and one of 50 tokens among those of one token
    h = conv_inputs(T, 1, 5, 2, F32, 43, True, False)
    d = dev(h)
    b = [0, *range(1, 101), *range(150, T + 1)]
    out, _ = cdr.short_conv(d["x"], d["weight"], d["bias"], cu_seqlens=cu, return_state=False)
    g = cdr.short_conv_bwd(d["x"], d["weight"], d["dout"], d["bias"], cu_seqlens=cu)
    x, w, bi = leaf(h["x"]), leaf(h["weight"]), leaf(h["bias"])
    ro, _ = ref.short_conv(x, w, bi, None, b)
    rx, rw, rb = grads([ro], [h["dout"]], [x, w, bi])
    check("out", out, ro, CONV)
    check("dx", g["dx"], rx, CONV)
    check("dweight", g["dweight"], rw, CONV)
    check("dbias", g["dbias"], rb, CONV)
    torch.cuda.synchronize()
    assert cdr.get_last_error() == 0


# ---------------------------------------------------------------- NaN, and decays past fp32

def same_where_finite(name, got, want, tol):
    """NaN exactly where the definition has NaN, and its values elsewhere."""
    got, want = got.detach().double().cpu(), want.detach().double().cpu()
    assert got.shape == want.shape, (name, got.shape, want.shape)
    assert torch.equal(got.isnan(), want.isnan()), f"{name}: NaN in {int(got.isnan().sum())} places, {int(want.isnan().sum())} expected"
    check(name, got.nan_to_num(nan=0.0), want.nan_to_num(nan=0.0), tol)


@pytest.mark.parametrize("where", ["dt", "dt_bias"])
@pytest.mark.parametrize("T,C,N,dtype", [(50, 5, 16, F32), (50, 8, 8, BF), (37, 5, 128, F32), (1000, 33, 16, F32)])
def test_a_nan_time_step_stays_one(T, C, N, dtype, where):
    # as in the definition: its channel's outputs and state from that token on, and the
    # gradients that they enter; 1000 tokens run in pieces
    lib = cdr.library()
    assert (lib.comba_selective_scan_fwd_workspace_size(1, T, C, 1, N, 0) > 0) == (T == 1000)
    assert lib.comba_selective_scan_bwd_workspace_size(1, T, C, 1, N, 0) > 0
    h = scan_inputs(T, 1, C, 1, N, dtype, 31, "Dbzh")
    h["dt_bias"] -= 2
    if where == "dt":
        h["dt"][2 * T // 5, 3] = float("nan")
    else:
        h["dt_bias"][3] = float("nan")
    a, kw, v = scan_args(dev(h), (1, T))
    out, hf = cdr.selective_scan(*a, **kw)
    ro, rh, rg = scan_reference(h, [0, T])
    assert bool(ro.isnan().any()) and not bool(ro.isnan().all())
    tol = 3 * SCAN + HALF[dtype]      # as for 1600 tokens in pieces
    same_where_finite("out", out[0], ro, tol)
    same_where_finite("h_final", hf, rh, tol)
    g = cdr.selective_scan_bwd(*a, v["dout"], **kw, dh_final=v["dh"])
    for k in IN_KEYS:
        same_where_finite("d" + k, g["d" + k].view(h[k].shape), rg[k], 3 * SCAN_BWD + (HALF[dtype] if k in TOKEN_KEYS else 0.0))
    # one token of two sequences, the second one without it
    one = {k: (torch.cat([t[2 * T // 5][None], t[:1]]) if k in TOKEN_KEYS else t) for k, t in h.items()}
    one["h0"] = torch.cat([h["h0"], h["h0"]])
    o = dev(one)
    out = cdr.selective_scan_step(o["x"], o["dt"], o["A_log"], o["Bm"], o["Cm"], o["h0"], D=o["D"], dt_bias=o["dt_bias"], z=o["z"])
    ro, rh, _ = scan_reference(one, [0, 1, 2], backward=False)
    same_where_finite("step", out, ro, SCAN + HALF[dtype])
    same_where_finite("state", o["h0"], rh, SCAN)


@pytest.mark.parametrize("T,N,dtype", [(16, 16, F32), (21, 16, F32), (21, 8, BF), (9, 64, F32), (1003, 16, F32)])
def test_decay_rates_past_the_largest_float(T, N, dtype):
    # exp(100) is infinite in fp32: such an entry forgets at once, whatever the length, but
    # for tokens with delta = 0, which leave it as it is
    C = 12
    h = scan_inputs(T, 1, C, 1, N, dtype, 17, "Dbzh")
    h["A_log"][:4] = 100.0
    a, kw, v = scan_args(dev(h), (1, T))
    out, hf = cdr.selective_scan(*a, **kw)
    ro, rh, rg = scan_reference(h, [0, T])
    assert all(bool(torch.isfinite(t).all()) for t in (ro, rh, *rg.values()))
    check("out", out[0], ro, 3 * SCAN + HALF[dtype])
    check("h_final", hf, rh, 3 * SCAN)
    g = cdr.selective_scan_bwd(*a, v["dout"], **kw, dh_final=v["dh"])
    for k in IN_KEYS:
        check("d" + k, g["d" + k].view(h[k].shape), rg[k], 3 * SCAN_BWD + (HALF[dtype] if k in TOKEN_KEYS else 0.0))
    # with tokens that leave the state as it is: their own gradients vanish
    h["dt"][T // 2:, 2:4] = -float("inf")
    h["h0"] *= 100
    a, kw, v = scan_args(dev(h), (1, T))
    _, _, rg = scan_reference(h, [0, T])
    g = cdr.selective_scan_bwd(*a, v["dout"], **kw, dh_final=v["dh"])
    for k in IN_KEYS:
        check("d" + k, g["d" + k].view(h[k].shape), rg[k], 3 * SCAN_BWD + (HALF[dtype] if k in TOKEN_KEYS else 0.0))
    h["A_log"][:2] = float("inf")
    a, kw, v = scan_args(dev(h), (1, T))
    out, hf = cdr.selective_scan(*a, **kw)
    ro, rh, _ = scan_reference(h, [0, T], backward=False)
    assert bool(torch.isfinite(rh).all())
    check("out", out[0], ro, 3 * SCAN + HALF[dtype])
    check("h_final", hf, rh, 3 * SCAN)
