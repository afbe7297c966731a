"""The operators around and beside the Comba recurrence, in plain PyTorch and as the library's calls.

Four operators of a recurrent token-mixer block, each with its backward and, where a model decodes with
it, its single-token form:

  short_conv     causal depthwise convolution over a few tokens, with SiLU, from and to a carried state
  selective_scan diagonal selective state space: h_t = exp(delta_t A) h_{t-1} + delta_t x_t B_t
  gated_norm     RMS norm of each head's output times SiLU of a gate
  residual_norm  a block's output (normed or not) scaled onto the residual stream, and the norm of the sum

`run` computes a case in plain form (fp32, rounded once at the end) or, with `own`, by the calls of
`chunk_delta_rule_b200`.  `exact` gives the same outputs in float64, computed another way.
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
EPS = 1e-6


# ---------------------------------------------------------------------------------- the cases

def listed():
    return [
        # training step of the convolution on q, k and v side by side (16 heads x 128 each), 1.3B layer
        dict(name="conv_train", kind="conv_train", dtype="bf16", batch=8, tokens=4096, channels=6144, taps=4, bias=False, silu=True),
        # a packed batch of prompts of mixed lengths, continued from earlier chunks' states
        dict(name="conv_packed", kind="conv_packed", dtype="fp32", seqs=25, tokens=32768, channels=2048, taps=4, bias=True, silu=True),
        # one decoded token of 256 sequences (32 heads x 128)
        dict(name="conv_step", kind="conv_step", dtype="bf16", batch=256, channels=4096, taps=4, bias=True, silu=True),
        # prompt or training forward of a 1.3B layer
        dict(name="scan_prompt", kind="scan_prompt", dtype="bf16", batch=8, tokens=4096, channels=2048, states=16, groups=1, gate=True),
        # one prompt of 64K tokens
        dict(name="scan_long", kind="scan_prompt", dtype="bf16", batch=1, tokens=65536, channels=2048, states=16, groups=1, gate=True),
        # a packed batch of prompts of mixed lengths, fp32
        dict(name="scan_packed", kind="scan_packed", dtype="fp32", seqs=25, tokens=32768, channels=2048, states=16, groups=2, gate=False),
        # training step (forward and backward) of a 340M layer
        dict(name="scan_train", kind="scan_train", dtype="bf16", batch=8, tokens=2048, channels=1024, states=16, groups=1, gate=True),
        # one decoded token of 256 sequences: the state's bandwidth
        dict(name="scan_step", kind="scan_step", dtype="bf16", batch=256, channels=4096, states=16, groups=1, gate=True),
        # training step of the norm of every head's output (16 heads x 128) with its gate, 1.3B layer
        dict(name="gated_norm_train", kind="gated_train", dtype="bf16", rows=8 * 4096 * 16, width=128),
        # the same for one decoded token of one sequence (32 heads x 128): latency
        dict(name="gated_norm_step", kind="gated", dtype="fp32", rows=32, width=128),
        # training step between two blocks of a 1.3B model: bf16 block output onto an fp32 residual stream
        dict(name="residual_norm_train", kind="residual_train", dtype="bf16", stream="fp32", rows=8 * 4096, width=2048, scale=True, post=True),
        # the same for one decoded token of 256 sequences, bf16 stream, no norm of the block's output
        dict(name="residual_norm_step", kind="residual", dtype="bf16", stream="bf16", rows=256, width=4096, scale=True, post=False),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["conv_train", "conv_packed", "conv_step", "scan_prompt", "scan_packed", "scan_train", "scan_step",
                       "gated_train", "gated", "residual_train", "residual"])
    case = dict(kind=kind, dtype=rng.choice(["bf16", "bf16", "fp32"]))
    op = kind.split("_")[0]
    if op in ("conv", "scan"):
        # whole heads (128), narrow odd widths and whatever lies between
        channels = rng.choice([128 * rng.randint(1, 32), 8 * rng.randint(4, 400), rng.randint(33, 2500)])
        groups = 1
        if op == "scan":
            groups = rng.choice([1, 1, 2, 4])
            channels = max(groups, channels // groups * groups)
        if kind.endswith("step"):
            case.update(batch=_log_int(rng, 1, 256), channels=channels)
        else:
            # tokens in all: up to 64K in one sequence, 16K for a backward through the scan
            total = _log_int(rng, 64, 16384 if kind == "scan_train" else 65536)
            if channels * total > 2048 * 65536:
                total = 2048 * 65536 // channels
            if kind.endswith("packed"):
                case.update(seqs=_log_int(rng, 1, 64), tokens=total, channels=channels)
            else:
                batch = rng.choice([1, 2, 3, 4, 8])
                case.update(batch=batch, tokens=max(1, total // batch), channels=channels)
        if op == "conv":
            case.update(taps=rng.choice([2, 3, 4]), bias=rng.random() < 0.5, silu=rng.random() < 0.8)
        else:
            case.update(states=rng.choice([8, 16, 16, 32]), groups=groups, gate=rng.random() < 0.7)
            if case["states"] > 16 and kind != "scan_step":
                case["tokens"] = max(1, case["tokens"] // 2)
    else:
        width = rng.choice([64, 128, 8 * rng.randint(8, 512), rng.randint(33, 4096)])
        most = (1 << 26) // width
        case.update(rows=_log_int(rng, 1, most), width=width)
        if op == "residual":
            case.update(stream=rng.choice(["fp32", case["dtype"]]), scale=rng.random() < 0.5, post=rng.random() < 0.5)
    return case


# ---------------------------------------------------------------------------------- the inputs

def _bounds(case, gen):
    """Start of each sequence on the joint token axis, and the end of the last: uniform batches and packed prompts."""
    if "seqs" not in case:
        return [case["tokens"] * i for i in range(case["batch"] + 1)]
    u = torch.rand(case["seqs"], generator=gen, dtype=torch.float64).add_(0.05).tolist()
    cuts, total = [0], sum(u)
    for v in u:
        cuts.append(cuts[-1] + v / total * case["tokens"])
    return [min(case["tokens"], int(c)) for c in cuts[:-1]] + [case["tokens"]]


def prepare(case, seed):
    host = torch.Generator().manual_seed(seed)
    gen = torch.Generator(device=DEV).manual_seed(seed)
    dt, kind = DTYPES[case["dtype"]], case["kind"]
    op = kind.split("_")[0]
    f32 = dict(device=DEV, dtype=torch.float32)

    def normal(*shape, dtype=dt, std=1.0):
        return torch.randn(shape, generator=gen, **f32).mul_(std).to(dtype)

    def uniform(*shape, lo=0.0, hi=1.0):
        return torch.rand(shape, generator=gen, **f32).mul_(hi - lo).add_(lo)

    s = dict(case=case)
    if op in ("conv", "scan"):
        c = case["channels"]
        if kind.endswith("step"):
            lead, n = (case["batch"],), case["batch"]
        else:
            cu = _bounds(case, host)
            n = len(cu) - 1
            s.update(starts=cu, cu=torch.tensor(cu, dtype=torch.int32, device=DEV))
            lead = (case["tokens"],) if "seqs" in case else (case["batch"], case["tokens"])
        s.update(x=normal(*lead, c), lead=lead, n=n)
        if kind.endswith("train"):
            s["dout"] = normal(*lead, c)
    if op == "conv":
        w = case["taps"]
        s["weight"] = uniform(c, w, lo=-1.0, hi=1.0).div_(math.sqrt(w)).mul_(1.7)
        s["bias"] = uniform(c, lo=-0.3, hi=0.3) if case["bias"] else None
        s["state"] = None if kind == "conv_train" else normal(n, w - 1, c)
    elif op == "scan":
        ns, g = case["states"], case["groups"]
        # time steps of 1e-3 .. 1e-1 at the bias, decay rates of 1 .. states
        step = torch.exp(uniform(c, lo=math.log(1e-3), hi=math.log(1e-1)))
        s["dt"] = normal(*lead, c)
        s["dt_bias"] = step + torch.log(-torch.expm1(-step))
        s["A_log"] = torch.log(torch.arange(1, ns + 1, **f32)).expand(c, ns) + uniform(c, ns, lo=-0.1, hi=0.1)
        s["Bm"], s["Cm"] = normal(*lead, g, ns), normal(*lead, g, ns)
        s["D"] = normal(c, dtype=torch.float32)
        s["z"] = normal(*lead, c) if case["gate"] else None
        s["h0"] = normal(n, c, ns, dtype=torch.float32)
        if kind == "scan_train":
            s["dh_final"] = normal(n, c, ns, dtype=torch.float32)
    elif op == "gated":
        r, d = case["rows"], case["width"]
        s.update(x=normal(r, d), gate=normal(r, d), weight=uniform(d, lo=0.5, hi=1.5))
        if kind.endswith("train"):
            s["dout"] = normal(r, d)
    else:
        r, d, st = case["rows"], case["width"], DTYPES[case["stream"]]
        s.update(x=normal(r, d), residual=normal(r, d, dtype=st, std=2.0), weight=uniform(d, lo=0.5, hi=1.5))
        s["scale"] = uniform(d, lo=0.1, hi=1.0) if case["scale"] else None
        s["post"] = uniform(d, lo=0.5, hi=1.5) if case["post"] else None
        if kind.endswith("train"):
            s.update(dy=normal(r, d), dh=normal(r, d, dtype=st))
    return s


# ---------------------------------------------------------------------------------- the plain forms

def _up(*ts):
    return [None if t is None else t.float() for t in ts]


def _silu(v):
    return v / (1 + torch.exp(-v))


def _dsilu(v):
    sg = 1 / (1 + torch.exp(-v))
    return sg * (1 + v * (1 - sg))


def _rows(starts):
    """Sequence of every token and its offset within it."""
    lens = torch.tensor([b - a for a, b in zip(starts, starts[1:])], device=DEV)
    seq = torch.repeat_interleave(torch.arange(len(lens), device=DEV), lens)
    first = torch.tensor(starts[:-1], device=DEV)
    return lens, first, seq, torch.arange(int(starts[-1]), device=DEV) - first[seq]


def _conv_forward(x, weight, bias, state, starts, silu):
    """Every sequence gets taps - 1 rows of state in front (zeros without one); a token's taps are rows of that axis."""
    w, c = weight.shape[1], weight.shape[0]
    lens, first, seq, off = _rows(starts)
    n = len(lens)
    ahead = x.new_zeros(n, w - 1, c) if state is None else state
    ext = torch.cat([ahead.reshape(n * (w - 1), c), x])
    o = off[:, None] + torch.arange(w, device=DEV) - (w - 1)
    at = torch.where(o < 0, seq[:, None] * (w - 1) + o + (w - 1), n * (w - 1) + first[seq][:, None] + o)
    taps = ext[at]
    pre = (taps * weight.t()).sum(1)
    pre = pre if bias is None else pre + bias
    last = lens[:, None] + torch.arange(w - 1, device=DEV) - (w - 1)
    sid = torch.arange(n, device=DEV)[:, None]
    keep = torch.where(last < 0, sid * (w - 1) + last + (w - 1), n * (w - 1) + first[:, None] + last)
    return (_silu(pre) if silu else pre), ext[keep], pre, taps


def _conv_backward(dout, pre, taps, weight, starts, silu):
    """dx of a token: its taps in the tokens after it, of the same sequence (no state and no state's gradient)."""
    w = weight.shape[1]
    lens, first, seq, off = _rows(starts)
    dpre = dout * _dsilu(pre) if silu else dout
    o = off[:, None] + (w - 1) - torch.arange(w, device=DEV)
    at = torch.where(o < lens[seq][:, None], first[seq][:, None] + o, len(seq))
    dx = (torch.cat([dpre, dpre.new_zeros(1, dpre.shape[1])])[at] * weight.t()).sum(1)
    return dx, (dpre[:, None] * taps).sum(0, dtype=torch.float64).t(), dpre.sum(0, dtype=torch.float64)


def _scan(a, u, longest):
    """h_t = a_t h_{t-1} + u_t along the first axis, by doubling; a is 0 where a sequence starts."""
    step = 1
    while step < longest:
        u[step:] += a[step:] * u[:-step]
        a[step:] = a[step:] * a[:-step]
        step *= 2
    return u


def _ssm(s):
    x, dt, bm, cm, z = _up(s["x"], s["dt"], s["Bm"], s["Cm"], s["z"])
    c, ns = s["A_log"].shape
    g = bm.shape[-2]
    flat = lambda t: None if t is None else t.reshape(-1, *t.shape[len(s["lead"]):])  # noqa: E731
    x, dt, bm, cm, z = map(flat, (x, dt, bm, cm, z))
    v = dt + s["dt_bias"]
    delta = torch.where(v > 20, v, torch.log1p(torch.exp(torch.clamp(v, max=20))))
    # a group's B and C for each of its channels
    per = lambda t: t[:, :, None, :].expand(-1, -1, c // g, -1).reshape(-1, c, ns)  # noqa: E731
    return x, v, delta, per(bm), per(cm), z, -torch.exp(s["A_log"])


def _scan_forward(s):
    x, v, delta, bm, cm, z, A = _ssm(s)
    starts = s["starts"]
    live = [i for i in range(s["n"]) if starts[i + 1] > starts[i]]
    at = torch.tensor([starts[i] for i in live], device=DEV)
    end = torch.tensor([starts[i + 1] - 1 for i in live], device=DEV)
    sid = torch.tensor(live, device=DEV)
    a = torch.exp(delta[..., None] * A)
    u = (delta * x)[..., None] * bm
    u[at] += a[at] * s["h0"][sid]
    cut = a.clone()
    cut[at] = 0
    h = _scan(cut, u, max(b - e for e, b in zip(starts, starts[1:])))
    del cut
    y = (h * cm).sum(-1) + s["D"] * x
    hf = s["h0"].clone()
    hf[sid] = h[end]
    out = y if z is None else y * _silu(z)
    return out, hf, (x, v, delta, bm, cm, z, A, a, h, y, at, end, sid)


def _scan_backward(s, kept):
    x, v, delta, bm, cm, z, A, a, h, y, at, end, sid = kept
    starts, g = s["starts"], s["Bm"].shape[-2]
    c, ns = s["A_log"].shape
    dout = s["dout"].float().reshape(-1, c)
    dy = dout if z is None else dout * _silu(z)
    dz = None if z is None else dout * y * _dsilu(z)
    dD = (dy * x).sum(0, dtype=torch.float64)
    dC = (h * dy[..., None]).reshape(-1, g, c // g, ns).sum(2)
    p = torch.empty_like(h)
    p[1:] = h[:-1]
    p[at] = s["h0"][sid]
    p *= a
    # the states' gradients, the other way along the tokens
    gr = dy[..., None] * cm
    gr[end] += s["dh_final"][sid]
    back = torch.zeros_like(a)
    back[:-1] = a[1:]
    back[end] = 0
    gr = _scan(back.flip(0), gr.flip(0), max(b - e for e, b in zip(starts, starts[1:]))).flip(0)
    del back
    dh0 = s["dh_final"].clone()
    dh0[sid] = a[at] * gr[at]
    dB = (gr * (delta * x)[..., None]).reshape(-1, g, c // g, ns).sum(2)
    du = (gr * bm).sum(-1)
    gp = gr * p
    ddelta = (gp * A).sum(-1) + du * x
    dA_log = (gp * delta[..., None]).sum(0, dtype=torch.float64) * A
    dx = du * delta + s["D"] * dy
    ddt = ddelta / (1 + torch.exp(-v))
    return dict(dx=dx, ddt=ddt, dA_log=dA_log, dBm=dB, dCm=dC, dD=dD, ddt_bias=ddt.sum(0, dtype=torch.float64), dz=dz, dh0=dh0)


def _rms(x):
    r = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS)
    return x * r, r


def _rms_back(dn, n, r):
    """Gradient of x r(x), from that of n = x r."""
    return r * (dn - n * (dn * n).mean(-1, keepdim=True))


def _to(t, like):
    return None if t is None else t.reshape(like.shape).to(like.dtype)


def _plain(s):
    case, kind = s["case"], s["case"]["kind"]
    f = torch.float32
    if kind in ("conv_train", "conv_packed"):
        c = case["channels"]
        x, state = _up(s["x"].reshape(-1, c), s["state"])
        out, last, pre, taps = _conv_forward(x, s["weight"], s["bias"], state, s["starts"], case["silu"])
        r = dict(out=_to(out, s["x"]))
        if kind == "conv_packed":
            return dict(r, state=last.to(s["x"].dtype))
        dx, dw, db = _conv_backward(s["dout"].float().reshape(-1, c), pre, taps, s["weight"], s["starts"], case["silu"])
        return dict(r, dx=_to(dx, s["x"]), dweight=dw.to(f), dbias=db.to(f) if case["bias"] else None)
    if kind == "conv_step":
        taps = torch.cat([s["state"], s["x"][:, None]], 1)
        pre = (taps.float() * s["weight"].t()).sum(1)
        pre = pre if s["bias"] is None else pre + s["bias"]
        s["state"].copy_(taps[:, 1:])
        return dict(out=_to(_silu(pre) if case["silu"] else pre, s["x"]), state=s["state"])
    if kind in ("scan_prompt", "scan_packed", "scan_train"):
        out, hf, kept = _scan_forward(s)
        r = dict(out=_to(out, s["x"]), h_final=hf)
        if kind != "scan_train":
            return r
        g = _scan_backward(s, kept)
        for k, like in (("dx", "x"), ("ddt", "dt"), ("dBm", "Bm"), ("dCm", "Cm"), ("dz", "z")):
            g[k] = _to(g[k], s[like]) if g[k] is not None else None
        for k in ("dA_log", "dD", "ddt_bias"):
            g[k] = g[k].to(f)
        return dict(r, **g)
    if kind == "scan_step":
        x, v, delta, bm, cm, z, A = _ssm(s)
        h = torch.exp(delta[..., None] * A) * s["h0"] + (delta * x)[..., None] * bm
        s["h0"].copy_(h)
        y = (h * cm).sum(-1) + s["D"] * x
        return dict(out=_to(y if z is None else y * _silu(z), s["x"]), h=s["h0"])
    if kind in ("gated", "gated_train"):
        x, gate = _up(s["x"], s["gate"])
        n, r = _rms(x)
        sg = _silu(gate)
        got = dict(out=_to(n * s["weight"] * sg, s["x"]))
        if kind == "gated":
            return got
        dout = s["dout"].float()
        dn = dout * s["weight"] * sg
        return dict(got, dx=_to(_rms_back(dn, n, r), s["x"]), dgate=_to(dout * n * s["weight"] * _dsilu(gate), s["x"]),
                    dweight=(dout * n * sg).sum(0, dtype=torch.float64).to(f))
    x, res = _up(s["x"], s["residual"])
    n, r = _rms(x) if case["post"] else (x, None)
    u = n * s["post"] if case["post"] else x
    h = (res + (u if s["scale"] is None else u * s["scale"])).to(s["residual"].dtype)
    m, q = _rms(h.float())
    got = dict(out=_to(m * s["weight"], s["x"]), h=h)
    if kind == "residual":
        return got
    dy, dh = _up(s["dy"], s["dh"])
    tot = dh + _rms_back(dy * s["weight"], m, q)
    du = tot if s["scale"] is None else tot * s["scale"]
    got.update(dresidual=_to(tot, h), dweight=(dy * m).sum(0, dtype=torch.float64).to(f))
    got.update(dscale=None if s["scale"] is None else (tot * u).sum(0, dtype=torch.float64).to(f))
    got.update(dpost=(du * n).sum(0, dtype=torch.float64).to(f) if case["post"] else None)
    return dict(got, dx=_to(_rms_back(du * s["post"], n, r) if case["post"] else du, s["x"]))


# ---------------------------------------------------------------------------------- the library's calls

def _library(s):
    import chunk_delta_rule_b200 as cdr

    case, kind = s["case"], s["case"]["kind"]
    if kind == "conv_train":
        a = dict(bias=s["bias"], silu=case["silu"])
        out, _ = cdr.short_conv(s["x"], s["weight"], return_state=False, **a)
        g = cdr.short_conv_bwd(s["x"], s["weight"], s["dout"], **a)
        return dict(out=out, dx=g["dx"], dweight=g["dweight"], dbias=g["dbias"])
    if kind == "conv_packed":
        out, last = cdr.short_conv(s["x"], s["weight"], bias=s["bias"], initial_state=s["state"], cu_seqlens=s["cu"], silu=case["silu"])
        return dict(out=out, state=last)
    if kind == "conv_step":
        out = cdr.short_conv_step(s["x"], s["weight"], s["state"], bias=s["bias"], silu=case["silu"])
        return dict(out=out, state=s["state"])
    if kind.startswith("scan"):
        a = dict(D=s["D"], dt_bias=s["dt_bias"], z=s["z"])
        ins = (s["x"], s["dt"], s["A_log"], s["Bm"], s["Cm"])
        if kind == "scan_step":
            out = cdr.selective_scan_step(*ins, s["h0"], **a)
            return dict(out=out, h=s["h0"])
        cu = s["cu"] if kind == "scan_packed" else None
        out, hf = cdr.selective_scan(*ins, h0=s["h0"], cu_seqlens=cu, **a)
        r = dict(out=out, h_final=hf)
        if kind == "scan_train":
            r.update(cdr.selective_scan_bwd(*ins, s["dout"], h0=s["h0"], dh_final=s["dh_final"], **a))
        return r
    if kind in ("gated", "gated_train"):
        r = dict(out=cdr.gated_norm(s["x"], s["gate"], s["weight"], eps=EPS))
        if kind == "gated_train":
            r.update(cdr.gated_norm_bwd(s["x"], s["gate"], s["weight"], s["dout"], eps=EPS))
        return r
    a = dict(scale=s["scale"], post_weight=s["post"], eps=EPS)
    out, h = cdr.residual_norm(s["x"], s["residual"], s["weight"], **a)
    r = dict(out=out, h=h)
    if kind == "residual_train":
        g = cdr.residual_norm_bwd(s["x"], h, s["weight"], s["dy"], dh=s["dh"], **a)
        r.update(dresidual=g["dresidual"], dweight=g["dweight"], dscale=g["dscale"], dpost=g["dpost_weight"], dx=g["dx"])
    return r


def run(state):
    return _library(state) if own else _plain(state)


# ---------------------------------------------------------------------------------- the costs

def work(case):
    kind, e = case["kind"], 2 if case["dtype"] == "bf16" else 4
    op = kind.split("_")[0]
    if op in ("conv", "scan"):
        c = case["channels"]
        step = kind.endswith("step")
        r = case["batch"] if step else case["tokens"] * (1 if "seqs" in case else case["batch"])
        n = case.get("seqs", case.get("batch"))
        el = r * c
        if op == "conv":
            w = case["taps"]
            par = c * (w + (1 if case["bias"] else 0)) * 4
            states = 0 if kind == "conv_train" else 2 * n * (w - 1) * c * e
            if kind == "conv_train":  # forward: x in, out; backward: x, dout in, dx
                return dict(bytes=5 * el * e + 3 * par, flops=el * (2 * w + 4) * 3)
            return dict(bytes=2 * el * e + states + par, flops=el * (2 * w + 4))
        ns, g = case["states"], case["groups"]
        z = 1 if case["gate"] else 0
        par = c * ns * 4 + 2 * c * 4
        fwd = el * e * (3 + z) + 2 * r * g * ns * e + 2 * n * c * ns * 4 + par
        flops = el * (7 * ns + 12)
        if kind != "scan_train":
            return dict(bytes=fwd, flops=flops)
        # x, dt, z, dout in, dx, ddt, dz out; B, C in, dB, dC out; h0, dh_final in, dh0 out
        bwd = el * e * (5 + 2 * z) + 4 * r * g * ns * e + 3 * n * c * ns * 4 + 2 * par
        return dict(bytes=fwd + bwd, flops=flops + el * (18 * ns + 30))
    r, d = case["rows"], case["width"]
    if op == "gated":
        train = kind.endswith("train")
        return dict(bytes=r * d * e * (3 + (5 if train else 0)) + d * 4 * (3 if train else 1), flops=r * d * (8 + (20 if train else 0)))
    er = 2 if case["stream"] == "bf16" else 4
    train = kind.endswith("train")
    el = 2 * e + 2 * er + ((3 * e + 3 * er) if train else 0)
    return dict(bytes=r * d * el + d * 4 * (1 + case["scale"] + case["post"]) * (3 if train else 1), flops=r * d * (8 + (24 if train else 0)))


# ---------------------------------------------------------------------------------- 64 bits

def _exact_conv(s, case):
    d = lambda t: None if t is None else t.double()  # noqa: E731
    c, w, train = case["channels"], case["taps"], case["kind"] == "conv_train"
    x = d(s["x"]).reshape(-1, c).requires_grad_(train)
    weight = d(s["weight"]).requires_grad_(train)
    bias = None if s["bias"] is None else d(s["bias"]).requires_grad_(train)
    outs, lasts = [], []
    if case["kind"] == "conv_step":
        cuts = list(range(case["batch"] + 1))
    else:
        cuts = s["starts"]
    with torch.set_grad_enabled(train):
        if case["kind"] == "conv_step":
            row = torch.cat([d(s["state"]), x[:, None]], 1)
            pre = torch.einsum("bwc,cw->bc", row, weight)
            pre = pre if bias is None else pre + bias
            return dict(out=torch.nn.functional.silu(pre) if case["silu"] else pre, state=row[:, 1:])
        for n, (a, b) in enumerate(zip(cuts, cuts[1:])):
            ahead = x.new_zeros(w - 1, c) if s["state"] is None else d(s["state"][n])
            row = torch.cat([ahead, x[a:b]])
            pre = sum(row[j:j + b - a] * weight[:, j] for j in range(w))
            outs.append(pre if bias is None else pre + bias)
            lasts.append(row[row.shape[0] - (w - 1):])
        pre = torch.cat(outs)
        out = torch.nn.functional.silu(pre) if case["silu"] else pre
    if not train:
        return dict(out=out.reshape(s["x"].shape), state=torch.stack(lasts))
    leaves = [x, weight] + ([] if bias is None else [bias])
    g = torch.autograd.grad(out, leaves, d(s["dout"]).reshape(-1, c))
    return dict(out=out.detach().reshape(s["x"].shape), dx=g[0].reshape(s["x"].shape), dweight=g[1], dbias=g[2] if bias is not None else None)


def _exact_scan(s, case):
    """Token by token, the recurrence and its adjoint as they are written down."""
    d = lambda t: None if t is None else t.double()  # noqa: E731
    c, ns, g = case["channels"], case["states"], case["groups"]
    A = -torch.exp(d(s["A_log"]))
    step, train = case["kind"] == "scan_step", case["kind"] == "scan_train"
    if step:
        spans = [(slice(None), 1)]
    elif "seqs" in case:
        spans = list(zip(s["starts"], s["starts"][1:]))
    else:
        spans = [(0, case["tokens"])]
    got = []
    for n, span in enumerate(spans):
        # [batch, time, ...]: a uniform batch at once, packed sequences one by one
        if step:
            cut = lambda t: None if t is None else d(t)[:, None]  # noqa: E731
        elif "seqs" in case:
            cut = lambda t: None if t is None else d(t[span[0]:span[1]])[None]  # noqa: E731
        else:
            cut = d
        x, dt, bm, cm, z = (cut(s[k]) for k in ("x", "dt", "Bm", "Cm", "z"))
        h = d(s["h0"][n:n + 1]) if "seqs" in case else d(s["h0"])
        delta = torch.nn.functional.softplus(dt + d(s["dt_bias"]), threshold=50)
        T = x.shape[1]
        heads = lambda t: t.repeat_interleave(c // g, dim=-2)  # noqa: E731
        ys, hs, as_ = [], [h], []
        for t in range(T):
            a = torch.exp(delta[:, t, :, None] * A)
            h = a * h + (delta[:, t] * x[:, t])[..., None] * heads(bm[:, t])
            ys.append((h * heads(cm[:, t])).sum(-1))
            if train:
                hs.append(h)
                as_.append(a)
        y = (torch.stack(ys, 1) if T else x) + d(s["D"]) * x
        act = 1.0 if z is None else torch.nn.functional.silu(z)
        r = dict(out=y * act, h_final=h)
        if train:
            dout = d(s["dout"])
            dy = dout * act
            sg = None if z is None else torch.sigmoid(z)
            r["dz"] = None if z is None else dout * y * (sg + z * sg * (1 - sg))
            r["dD"] = (dy * x).sum((0, 1))
            gh = d(s["dh_final"])
            dA = torch.zeros_like(A)
            ddel, dx, dB, dC = (torch.zeros_like(v) for v in (delta, x, bm, cm))
            for t in reversed(range(T)):
                gh = gh + dy[:, t, :, None] * heads(cm[:, t])
                dC[:, t] = (hs[t + 1] * dy[:, t, :, None]).unflatten(1, (g, c // g)).sum(2)
                dB[:, t] = (gh * (delta[:, t] * x[:, t])[..., None]).unflatten(1, (g, c // g)).sum(2)
                du = (gh * heads(bm[:, t])).sum(-1)
                dlog = gh * hs[t] * as_[t]
                ddel[:, t] = du * x[:, t] + (dlog * A).sum(-1)
                dA += (dlog * delta[:, t, :, None]).sum(0)
                dx[:, t] = du * delta[:, t]
                gh = gh * as_[t]
            ddt = ddel * torch.sigmoid(dt + d(s["dt_bias"]))
            r.update(dx=dx + d(s["D"]) * dy, ddt=ddt, dA_log=dA * A, dBm=dB, dCm=dC, ddt_bias=ddt.sum((0, 1)), dh0=gh)
        got.append(r)
    if step:
        return dict(out=got[0]["out"][:, 0], h=got[0]["h_final"])
    if "seqs" in case:
        return dict(out=torch.cat([r["out"][0] for r in got]), h_final=torch.cat([r["h_final"] for r in got]))
    return got[0]


def _exact_norm(s, case):
    train = case["kind"].endswith("train")
    leaf = lambda k: None if s.get(k) is None else s[k].double().requires_grad_(train)  # noqa: E731
    norm = lambda v: v / (v.pow(2).mean(-1, keepdim=True) + EPS).sqrt()  # noqa: E731
    with torch.set_grad_enabled(train):
        x, weight = leaf("x"), leaf("weight")
        if case["kind"].startswith("gated"):
            gate = leaf("gate")
            out = norm(x) * weight * torch.nn.functional.silu(gate)
            if not train:
                return dict(out=out)
            dx, dgate, dw = torch.autograd.grad(out, [x, gate, weight], s["dout"].double())
            return dict(out=out.detach(), dx=dx, dgate=dgate, dweight=dw)
        res, scale, post = leaf("residual"), leaf("scale"), leaf("post")
        u = x if post is None else norm(x) * post
        h = res + (u if scale is None else u * scale)
        # the norm reads the stream as it is stored
        kept = h + (h.detach().to(s["residual"].dtype).double() - h.detach())
        out = norm(kept) * weight
    if not train:
        return dict(out=out, h=h)
    names = [k for k, v in (("dx", x), ("dresidual", res), ("dweight", weight), ("dscale", scale), ("dpost", post)) if v is not None]
    leaves = [v for v in (x, res, weight, scale, post) if v is not None]
    g = torch.autograd.grad([out, h], leaves, [s["dy"].double(), s["dh"].double()])
    r = dict(out=out.detach(), h=h.detach(), dscale=None, dpost=None)
    r.update(zip(names, g))
    return r


def exact(case, seed):
    s = prepare(case, seed)
    op = case["kind"].split("_")[0]
    return (_exact_conv if op == "conv" else _exact_scan if op == "scan" else _exact_norm)(s, case)
