"""The operators around the recurrence on the host: refusals of the C ABI and of the
Python binding before anything reaches CUDA, and the definitions the GPU tests use."""
import ctypes

import pytest
import torch

import chunk_delta_rule_b200 as cdr
from chunk_delta_rule_b200 import build as cbuild
from oracle import block_ops as ref

# Fake, well-aligned, distinct "device" addresses: validation rejects before any CUDA
# call, so they are never dereferenced.
BASE, GB = 1 << 40, 1 << 30
EINVAL, EUNSUPPORTED, OK = -1, -2, 0


@pytest.fixture(scope="module")
def lib():
    cbuild.build()
    return cdr.library()


CALLS = {
    "comba_short_conv_fwd": (["x", "weight", "bias", "init", "out", "fin", "cu"],
                             dict(N=2, T=64, C=32, W=4, silu=1, dtype=0)),
    "comba_short_conv_bwd": (["x", "weight", "bias", "init", "dout", "dfin", "dx", "dweight", "dbias", "dinit", "cu"],
                             dict(N=2, T=64, C=32, W=4, silu=1, dtype=0, ws=BASE + 40 * GB, nws=1 << 24)),
    "comba_short_conv_step": (["x", "weight", "bias", "state", "out"], dict(B=2, C=32, W=4, silu=1, dtype=0)),
    "comba_selective_scan_fwd": (["x", "dt", "A_log", "Bm", "Cm", "D", "bias", "z", "h0", "out", "hf", "cu"],
                                 dict(n=2, T=4096, C=32, G=2, N=16, dtype=0, ws=BASE + 40 * GB, nws=1 << 24)),
    "comba_selective_scan_bwd": (["x", "dt", "A_log", "Bm", "Cm", "D", "bias", "z", "h0", "dout", "dhf", "dx", "ddt", "dA",
                                  "dBm", "dCm", "dD", "dbias", "dz", "dh0", "cu"],
                                 dict(n=2, T=64, C=32, G=2, N=16, dtype=0, ws=BASE + 40 * GB, nws=1 << 28)),
    "comba_selective_scan_step": (["x", "dt", "A_log", "Bm", "Cm", "D", "bias", "z", "h", "out"],
                                  dict(B=2, C=32, G=2, N=16, dtype=0)),
    "comba_gated_norm_fwd": (["x", "gate", "weight", "out"], dict(rows=8, D=64, eps=1e-6, dtype=0)),
    "comba_gated_norm_bwd": (["x", "gate", "weight", "dout", "dx", "dgate", "dweight"],
                             dict(rows=8, D=64, eps=1e-6, dtype=0, ws=BASE + 40 * GB, nws=1 << 24)),
    "comba_residual_norm_fwd": (["x", "res", "weight", "scale", "post", "out", "h"],
                                dict(rows=8, D=64, eps=1e-6, dtype=0, rdtype=1)),
    "comba_residual_norm_bwd": (["x", "h", "weight", "scale", "post", "dy", "dh", "dx", "dres", "dweight", "dscale", "dpost"],
                                dict(rows=8, D=64, eps=1e-6, dtype=0, rdtype=1, ws=BASE + 40 * GB, nws=1 << 24)),
}


def call(lib, name, **change):
    ptrs, sizes = CALLS[name]
    vals = {p: BASE + i * GB for i, p in enumerate(ptrs)}
    vals.update(sizes)
    assert set(change) <= set(vals), set(change) - set(vals)
    vals.update(change)
    args = [ctypes.c_void_p(vals[k]) if k in ptrs or k == "ws" else vals[k] for k in [*ptrs, *sizes]]
    return getattr(lib, name)(*args, ctypes.c_void_p(None))


def at(name, p, off=0):
    return BASE + CALLS[name][0].index(p) * GB + off


NORMS = ["comba_gated_norm_fwd", "comba_gated_norm_bwd", "comba_residual_norm_fwd", "comba_residual_norm_bwd"]
REFUSED = []
for _n, _required in [("comba_short_conv_fwd", ["x", "weight", "out"]),
                      ("comba_short_conv_bwd", ["x", "weight", "dout", "dx", "dweight", "ws"]),
                      ("comba_short_conv_step", ["x", "weight", "state", "out"]),
                      ("comba_selective_scan_fwd", ["x", "dt", "A_log", "Bm", "Cm", "out", "ws"]),
                      ("comba_selective_scan_bwd", ["x", "dt", "A_log", "Bm", "Cm", "dout", "dx", "ddt", "dA", "dBm", "dCm", "ws"]),
                      ("comba_selective_scan_step", ["x", "dt", "A_log", "Bm", "Cm", "h", "out"]),
                      ("comba_gated_norm_fwd", ["x", "gate", "weight", "out"]),
                      ("comba_gated_norm_bwd", ["x", "gate", "weight", "dout", "dx", "dgate", "dweight", "ws"]),
                      ("comba_residual_norm_fwd", ["x", "res", "weight", "out", "h"]),
                      ("comba_residual_norm_bwd", ["x", "h", "weight", "dy", "dx", "dres", "dweight", "ws"])]:
    REFUSED += [(_n, {_r: None}) for _r in _required]
    REFUSED += [(_n, {"x": BASE + 1}), (_n, {"dtype": 2}), (_n, {"dtype": -1})]
    if "ws" in _required:
        REFUSED += [(_n, dict(nws=64)), (_n, dict(ws=BASE + 40 * GB + 4)), (_n, dict(ws=BASE + 64))]
for _n in ("comba_short_conv_fwd", "comba_short_conv_bwd", "comba_short_conv_step"):
    REFUSED += [(_n, dict(W=1)), (_n, dict(W=5)), (_n, dict(C=-1)), (_n, {"weight": at(_n, "weight", 2)})]
for _n in ("comba_selective_scan_fwd", "comba_selective_scan_bwd", "comba_selective_scan_step"):
    REFUSED += [(_n, dict(N=12)), (_n, dict(N=256)), (_n, dict(N=0)), (_n, dict(G=3)), (_n, dict(G=0)),
                (_n, {"A_log": at(_n, "A_log", 4)}), (_n, {"Bm": at(_n, "Bm", 8)}), (_n, dict(C=-4))]
for _n in NORMS:
    REFUSED += [(_n, dict(rows=-1)), (_n, dict(D=-1)), (_n, dict(eps=-1.0)), (_n, dict(eps=float("nan"))),
                (_n, dict(rows=1 << 40, D=64))]
REFUSED += [
    ("comba_short_conv_fwd", dict(T=-1)), ("comba_short_conv_fwd", dict(N=-1)),
    ("comba_short_conv_fwd", dict(out=BASE + 16)),                                            # out on x
    ("comba_short_conv_fwd", dict(fin=at("comba_short_conv_fwd", "init"))),                   # final on initial state
    ("comba_short_conv_fwd", dict(fin=at("comba_short_conv_fwd", "out", 8))),
    ("comba_short_conv_bwd", dict(dx=at("comba_short_conv_bwd", "dout"))),
    ("comba_short_conv_bwd", dict(dinit=at("comba_short_conv_bwd", "dfin"))),
    ("comba_short_conv_step", dict(state=BASE + 64)),
    ("comba_selective_scan_fwd", dict(out=at("comba_selective_scan_fwd", "z"))),
    ("comba_selective_scan_fwd", dict(hf=at("comba_selective_scan_fwd", "h0", 16))),          # partial overlap
    ("comba_selective_scan_fwd", dict(h0=at("comba_selective_scan_fwd", "h0", 4))),
    ("comba_selective_scan_bwd", dict(z=None)), ("comba_selective_scan_bwd", dict(dz=None)),
    ("comba_selective_scan_bwd", dict(ddt=at("comba_selective_scan_bwd", "dx", 64))),
    ("comba_selective_scan_step", dict(out=at("comba_selective_scan_step", "h"))),
    ("comba_gated_norm_fwd", dict(out=BASE)), ("comba_gated_norm_bwd", dict(dgate=at("comba_gated_norm_bwd", "dx"))),
    ("comba_residual_norm_fwd", dict(rdtype=2)), ("comba_residual_norm_fwd", dict(dtype=1, rdtype=0)),
    ("comba_residual_norm_fwd", dict(h=at("comba_residual_norm_fwd", "res", 4))),             # not exactly in place
    ("comba_residual_norm_fwd", dict(h=BASE)), ("comba_residual_norm_bwd", dict(scale=None)),
    ("comba_residual_norm_bwd", dict(post=None)), ("comba_residual_norm_bwd", dict(dres=at("comba_residual_norm_bwd", "dh"))),
]


@pytest.mark.parametrize("name,change", REFUSED, ids=lambda v: str(v))
def test_refused_arguments(lib, name, change):
    assert call(lib, name, **change) == EINVAL


@pytest.mark.parametrize("name,change", [(n, dict(D=8193)) for n in NORMS] + [
    ("comba_selective_scan_fwd", dict(n=65536, T=1, cu=None)), ("comba_selective_scan_step", dict(B=65536))])
def test_sizes_beyond_the_limits(lib, name, change):
    assert call(lib, name, **change) == EUNSUPPORTED


@pytest.mark.parametrize("name,change", [
    ("comba_short_conv_fwd", dict(N=0)), ("comba_short_conv_fwd", dict(C=0)), ("comba_short_conv_step", dict(B=0)),
    ("comba_selective_scan_fwd", dict(n=0)), ("comba_selective_scan_fwd", dict(C=0)), ("comba_selective_scan_step", dict(B=0)),
    ("comba_gated_norm_fwd", dict(rows=0)), ("comba_gated_norm_fwd", dict(D=0)), ("comba_residual_norm_fwd", dict(rows=0))])
def test_empty_calls_do_nothing(lib, name, change):
    assert call(lib, name, **change) == OK


def test_workspace_sizes(lib):
    assert lib.comba_short_conv_bwd_workspace_size(0, 64, 32, 4, 0) == 0
    assert lib.comba_short_conv_bwd_workspace_size(2, 64, 32, 4, 0) > 0
    # N uniform sequences of T tokens, or T packed tokens
    assert lib.comba_short_conv_bwd_workspace_size(2, 64, 32, 4, 0) == lib.comba_short_conv_bwd_workspace_size(9, 128, 32, 4, 1)
    assert lib.comba_selective_scan_bwd_workspace_size(2, 64, 32, 5, 16, 0) == 0
    # few long sequences are cut into pieces; many, or short ones, are not
    assert lib.comba_selective_scan_fwd_workspace_size(1, 65536, 256, 1, 16, 0) > 0
    assert lib.comba_selective_scan_fwd_workspace_size(1, 65536, 256, 1, 16, 1) > 0
    assert lib.comba_selective_scan_fwd_workspace_size(64, 1024, 2048, 1, 16, 0) == 0
    assert lib.comba_selective_scan_fwd_workspace_size(1, 100, 256, 1, 16, 0) == 0
    assert (lib.comba_selective_scan_bwd_workspace_size(2, 4096, 32, 2, 16, 0)
            > lib.comba_selective_scan_bwd_workspace_size(2, 64, 32, 2, 16, 0) > 0)
    assert lib.comba_residual_norm_bwd_workspace_size(100, 64) == 3 * lib.comba_gated_norm_bwd_workspace_size(100, 64) > 0
    assert lib.comba_residual_norm_bwd_workspace_size(0, 64) == lib.comba_residual_norm_bwd_workspace_size(100, 8193) == 0


def test_the_binding_refuses_what_is_not_a_device_tensor():
    x, w = torch.zeros(2, 5, 8), torch.zeros(8, 4)
    with pytest.raises(ValueError, match="CUDA"):
        cdr.short_conv(x, w)
    with pytest.raises(ValueError, match="CUDA"):
        cdr.short_conv_bwd(x, w, x)
    with pytest.raises(ValueError, match="CUDA"):
        cdr.short_conv_step(x[:, 0], w, torch.zeros(2, 3, 8))
    b = torch.zeros(2, 5, 1, 16)
    with pytest.raises(ValueError, match="CUDA"):
        cdr.selective_scan(x, x, torch.zeros(8, 16), b, b)
    with pytest.raises(ValueError, match="CUDA"):
        cdr.selective_scan_step(x[:, 0], x[:, 0], torch.zeros(8, 16), b[:, 0], b[:, 0], torch.zeros(2, 8, 16))
    for f in (lambda: cdr.gated_norm(x, x, w[:, 0]), lambda: cdr.gated_norm_bwd(x, x, w[:, 0], x),
              lambda: cdr.residual_norm(x, x, w[:, 0]), lambda: cdr.residual_norm_bwd(x, x, w[:, 0], x)):
        with pytest.raises(ValueError, match="CUDA"):
            f()


def test_the_binding_refuses_types_and_ranks():
    with pytest.raises(TypeError, match="bf16 or fp32"):
        cdr.gated_norm(torch.zeros(2, 8, dtype=torch.float16), torch.zeros(2, 8, dtype=torch.float16), torch.zeros(8))
    with pytest.raises(TypeError, match="bf16 or fp32"):
        cdr.short_conv(torch.zeros(2, 5, 8, dtype=torch.float64), torch.zeros(8, 4))
    with pytest.raises(ValueError, match=r"\[B, T, C\]"):
        cdr.short_conv(torch.zeros(5, 8), torch.zeros(8, 4))
    with pytest.raises(ValueError, match="total_T"):
        cdr.selective_scan(torch.zeros(1, 5, 8), None, None, None, None, cu_seqlens=torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="cu_seqlens"):
        cdr.short_conv(torch.zeros(5, 8), torch.zeros(8, 4), cu_seqlens=torch.zeros(0, dtype=torch.int32))


def _doubles(*shapes):
    g = torch.Generator().manual_seed(3)
    return [torch.randn(s, generator=g, dtype=torch.float64).requires_grad_(True) for s in shapes]


def test_definitions_by_hand():
    # conv: taps 1, 10, 100 over 1, 2, 3 after a state of 7, 8
    x = torch.tensor([[1.0], [2.0], [3.0]])
    out, fin = ref.short_conv(x, torch.tensor([[1.0, 10.0, 100.0]]), torch.tensor([0.5]), torch.tensor([[[7.0], [8.0]]]), [0, 3], False)
    assert out[:, 0].tolist() == [187.5, 218.5, 321.5] and fin[0, :, 0].tolist() == [2.0, 3.0]
    # a shorter sequence keeps part of its state
    _, fin = ref.short_conv(x[:1], torch.ones(1, 3), None, torch.tensor([[[7.0], [8.0]]]), [0, 1])
    assert fin[0, :, 0].tolist() == [8.0, 1.0]
    # scan: with A_log = 0 and softplus(dt) = log 2, the decay is exp(-log 2) = 1/2
    dt = torch.full((2, 1), 0.0, dtype=torch.float64)      # softplus(0) = log 2
    one = torch.ones(2, 1, dtype=torch.float64)
    l2 = float(torch.log(torch.tensor(2.0, dtype=torch.float64)))
    o, h = ref.selective_scan(one, dt, torch.zeros(1, 1), one[:, :, None], one[:, :, None], torch.tensor([3.0]), None, None,
                              torch.tensor([[[4.0]]]), [0, 2])
    first = 2.0 + l2
    assert abs(float(o[0, 0]) - (first + 3)) < 1e-12 and abs(float(h[0, 0, 0]) - (first / 2 + l2)) < 1e-12
    assert float(ref.softplus(torch.tensor(-float("inf"), dtype=torch.float64))) == 0.0
    # norms: x = (3, 4) has mean square 12.5
    n = ref.gated_norm(torch.tensor([[3.0, 4.0]]), torch.full((1, 2), 1e3), torch.tensor([1.0, 2.0]), 0.0)
    assert torch.allclose(n, torch.tensor([[3000.0, 8000.0]], dtype=torch.float64) / 12.5 ** 0.5)
    out, h = ref.residual_norm(torch.tensor([[1.0, 2.0]]), torch.tensor([[1.0, 0.0]]), torch.ones(2), torch.tensor([2.0, 2.0]), None, 0.0)
    assert h.tolist() == [[3.0, 4.0]] and torch.allclose(out, h / 12.5 ** 0.5)


def test_gradients_of_the_definitions():
    x, w, b, s = _doubles((6, 3), (3, 3), (3,), (2, 2, 3))
    assert torch.autograd.gradcheck(lambda *a: ref.short_conv(*a, [0, 1, 6]), (x, w, b, s))
    x, dt, A, B, C, D, bias, z, h0 = _doubles((5, 4), (5, 4), (4, 2), (5, 2, 2), (5, 2, 2), (4,), (4,), (5, 4), (2, 4, 2))
    assert torch.autograd.gradcheck(lambda *a: ref.selective_scan(*a, [0, 3, 5]), (x, dt, A, B, C, D, bias, z, h0))
    x, g, w = _doubles((3, 5), (3, 5), (5,))
    assert torch.autograd.gradcheck(ref.gated_norm, (x, g, w))
    x, r, w, sc, po = _doubles((3, 5), (3, 5), (5,), (5,), (5,))
    assert torch.autograd.gradcheck(ref.residual_norm, (x, r, w, sc, po))


@pytest.mark.parametrize("G", [0, 3, -1, 64])
@pytest.mark.parametrize("name,none", [("comba_selective_scan_fwd", dict(n=0)), ("comba_selective_scan_bwd", dict(n=0)),
                                       ("comba_selective_scan_step", dict(B=0))])
def test_groups_that_do_not_divide_the_channels_are_refused_without_a_sequence(lib, name, none, G):
    assert call(lib, name, G=G, **none) == EINVAL


@pytest.mark.parametrize("wide", [2 ** 31, 2 ** 32 + 4])
def test_the_binding_refuses_dimensions_past_an_int(wide):
    # the C ABI takes them as int: what is wider must not arrive cut to its low 32 bits
    t = lambda *s: torch.zeros((1,) * len(s)).expand(s)     # no memory behind them
    w = torch.zeros(8, 4)
    a = torch.zeros(2, 8)
    for f in (lambda: cdr.short_conv(t(2, wide, 8), w), lambda: cdr.short_conv(t(2, 5, wide), w),
              lambda: cdr.short_conv_step(t(wide, 8), w, a), lambda: cdr.short_conv_step(t(2, wide), w, a),
              lambda: cdr.selective_scan_step(t(wide, 8), a, a, a, a, a), lambda: cdr.selective_scan_step(t(2, wide), a, a, a, a, a),
              lambda: cdr.gated_norm(t(3, wide), a, w), lambda: cdr.gated_norm_bwd(t(wide), a, w, a),
              lambda: cdr.residual_norm(t(3, wide), a, w), lambda: cdr.residual_norm_bwd(t(3, wide), a, w, a),
              lambda: cdr.short_conv(t(5, 8), w, cu_seqlens=t(wide + 1)),
              lambda: cdr.block_ops._filter(t(8, wide), 8, 0),
              lambda: cdr.block_ops._groups_states(t(2, wide, 16)), lambda: cdr.block_ops._groups_states(t(2, 1, wide))):
        with pytest.raises(ValueError, match=r"2\^31"):
            f()


# Sizes (sequences, T, C, N) with the measured times (us) of the scan's direct and split forms,
# forward and backward.
SCAN_FORMS = [
    ((1, 4096, 2048, 16), (322, 135), (1032, 561)), ((2, 4096, 2048, 16), (322, 250), (1036, 1079)),
    ((3, 4096, 2048, 16), (369, 363), (1291, 1568)), ((4, 4096, 2048, 16), (369, 473), (1303, 1340)),
    ((1, 512, 2048, 16), (47, 35), (146, 98)), ((2, 512, 2048, 16), (47, 43), (147, 164)),
    ((2, 1024, 2048, 16), (86, 74), (278, 297)), ((1, 16384, 64, 16), (1257, 45), (4059, 125)),
    ((2, 4096, 1024, 16), (322, 137), (1033, 516)), ((4, 4096, 1024, 16), (322, 250), (1063, 968)),
    ((6, 4096, 1024, 16), (369, 363), (1299, 1428)), ((1, 4096, 256, 16), (319, 37), (1022, 102)),
    ((16, 4096, 256, 16), (320, 244), (1068, 965)), ((3, 4096, 1920, 16), (365, 358), (1289, 1557)),
    ((1, 2048, 2048, 8), (256, 57), (770, 221)), ((1, 2048, 768, 32), (162, 60), (496, 195)),
    ((4, 2048, 768, 32), (190, 184), (627, 694)), ((1, 2048, 1024, 64), (133, 125), (561, 470)),
    ((2, 2048, 512, 64), (133, 127), (558, 475)), ((1, 2048, 512, 128), None, (514, 604)),
    ((1, 2048, 256, 128), (131, 80), (483, 324)),
]


@pytest.mark.parametrize("size,fwd,bwd", SCAN_FORMS, ids=lambda v: str(v))
def test_the_scan_takes_the_form_measured_to_be_faster(lib, size, fwd, bwd):
    n, T, C, N = size
    if fwd:
        split = lib.comba_selective_scan_fwd_workspace_size(n, T, C, 1, N, 0) > 0
        assert split == (fwd[1] < fwd[0])
    # the backward's workspace in the direct form: states, dB and dC of a channel block of
    # 512 / N channels, and one row of the parameters' sums for each sequence
    up = lambda v: -(-v // 256) * 256
    direct = (up((n * T // 8 + n + 2) * C * N * 4) + up(-(-C * N // 512) * n * T * 2 * N * 4) + up(n * C * N * 8) + up(n * 2 * C * 8))
    got = lib.comba_selective_scan_bwd_workspace_size(n, T, C, 1, N, 0)
    assert (got != direct) == (bwd[1] < bwd[0])
