"""The operators around the recurrence on the GPU against their 64-bit forms.

Every output and gradient of every case is held to ``_block_ref.close``: half a step of its type plus
K roundings of its terms' magnitudes.  K counts, for the longest chain of a case, one rounding per added
term for sums taken one after another and 64 for everything else; for the scan 64 + T + N, twice that in
the backward (its magnitudes carry each token's own roundings through the recursion).
"""

import numpy as np
import pytest
import torch

import oracle
from mlstm_chunkwise_attention_b200 import binding, block
from _block_ref import close, conv64, norm64, scan64

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
ACTS = {"none": block.ACT_NONE, "silu": block.ACT_SILU, "sigmoid": block.ACT_SIGMOID}
SCOPES = {"token": block.SCOPE_TOKEN, "sequence": block.SCOPE_SEQUENCE}


def rand(g, *shape, dtype=F32, scale=1.0):
    return (torch.randn(*shape, generator=g) * scale).to(dtype)


def dev(t, strided=False):
    """On the GPU; strided: as a slice of a wider tensor whose rows start at odd elements."""
    if t is None:
        return None
    if not strided:
        return t.cuda()
    wide = torch.full((*t.shape[:-1], t.shape[-1] + 5), float("nan"), dtype=t.dtype, device="cuda")
    wide[..., 3:-2] = t.cuda()
    return wide[..., 3:-2]


def d64(t):
    return None if t is None else t.double()


def heads(t, NH):
    """[B, T, D] as head-major [B, NH, T, d]."""
    B, T, D = t.shape
    return t.view(B, T, NH, D // NH).transpose(1, 2).contiguous()


def last(t):
    """Head-major back to [B, T, D]."""
    B, NH, T, d = t.shape
    return t.transpose(1, 2).reshape(B, T, NH * d)


# ---- short causal convolution --------------------------------------------------------------------

# B, T, NH, d, W, act, bias, carried, dtype, head-major, strided
CONV = [
    (1, 1, 1, 8, 4, "silu", True, False, BF, False, False),
    (2, 1, 2, 16, 4, "silu", True, True, F32, True, False),
    (1, 2, 1, 1, 4, "none", False, True, F32, False, False),      # shorter than the carried state
    (3, 3, 5, 7, 2, "silu", True, True, BF, True, False),         # odd heads: element accesses
    (2, 65, 3, 67, 3, "none", True, True, F32, True, False),      # one token past a run
    (2, 300, 4, 64, 4, "silu", True, False, BF, True, False),
    (2, 257, 2, 72, 3, "silu", False, True, BF, False, True),     # unaligned slices
    (1, 700, 1, 264, 2, "silu", True, True, F32, False, False),   # two channel blocks
]


def conv_case(B, T, NH, d, W, act, bias, carried, dtype, hm, strided, seed=0):
    g = torch.Generator().manual_seed(100 + seed + T)
    D = NH * d
    c = dict(x=rand(g, B, T, D, dtype=dtype), w=rand(g, D, W, scale=0.5),
             bias=rand(g, D, scale=0.3) if bias else None,
             state=rand(g, B, W - 1, D, dtype=dtype) if carried else None,
             dy=rand(g, B, T, D, dtype=dtype),
             dso=rand(g, B, W - 1, D, dtype=dtype) if carried else None)
    return c


@pytest.mark.parametrize("case", CONV, ids=[f"b{c[0]}t{c[1]}h{c[2]}d{c[3]}w{c[4]}" for c in CONV])
def test_conv_against_64_bits(case):
    B, T, NH, d, W, act, bias, carried, dtype, hm, strided = case
    c = conv_case(*case)
    x, w, b, st = dev(c["x"], strided), dev(c["w"]), dev(c["bias"]), dev(c["state"])
    y, so = block.causal_conv_forward(x, w, b, act=ACTS[act], state_in=st, want_state=True,
                                      heads=NH if hm else None)
    dy = dev(heads(c["dy"], NH)) if hm else dev(c["dy"], strided)
    got = block.causal_conv_backward(x, w, b, dy, act=ACTS[act], state_in=st, dstate_out=dev(c["dso"]),
                                     want_dstate=True)
    binding.check_device()
    ref = conv64(*(d64(c[k]) for k in ("x", "w", "bias", "state")), act, d64(c["dy"]), d64(c["dso"]))
    K = 64
    close(last(y) if hm else y, *ref["y"], K, "y")
    assert torch.equal(so.cpu().double(), ref["state"][0]), "the carried inputs are copies"
    close(got["dx"], *ref["dx"], K, "dx")
    close(got["dstate_in"], *ref["dstate_in"], K, "dstate_in")
    close(got["dweight"], *ref["dweight"], K + B * T, "dweight")
    if bias:
        close(got["dbias"], *ref["dbias"], K + B * T, "dbias")
    else:
        assert got["dbias"] is None


@pytest.mark.parametrize("dtype,d", [(BF, 64), (F32, 13)])
@pytest.mark.parametrize("W", [2, 3, 4])
def test_conv_pieces_and_steps_give_the_whole_sequence(dtype, d, W):
    """A prompt in two pieces, then single tokens, has the bits of one call over all tokens."""
    g = torch.Generator().manual_seed(7)
    B, T, NH = 2, 50, 3
    D = NH * d
    x, w, b = dev(rand(g, B, T, D, dtype=dtype)), dev(rand(g, D, W)), dev(rand(g, D))
    whole, end = block.causal_conv_forward(x, w, b, want_state=True)
    first, st = block.causal_conv_forward(x[:, :1], w, b, want_state=True)
    second, st = block.causal_conv_forward(x[:, 1:40], w, b, state_in=st, want_state=True)
    parts = [first, second]
    for t in range(40, T):
        parts.append(block.causal_conv_step(x[:, t], w, b, st)[:, None])
    assert torch.equal(torch.cat(parts, 1), whole) and torch.equal(st, end)
    # the head-major forms hold the same values
    hm, _ = block.causal_conv_forward(x, w, b, heads=NH)
    assert torch.equal(last(hm), whole)
    st2 = torch.zeros(B, W - 1, D, dtype=dtype, device="cuda")
    one = block.causal_conv_step(x[:, 0], w, b, st2, heads=NH)
    assert torch.equal(one.reshape(B, D), whole[:, 0])


# ---- selective scan ------------------------------------------------------------------------------

# B, T, D, N, G, gate, skip, bias, softplus, carried, dtype, strided
SCAN = [
    (1, 1, 8, 16, 1, True, True, True, True, False, BF, False),
    (2, 1, 1, 1, 1, False, False, False, False, True, F32, False),
    (2, 8, 16, 8, 1, True, True, True, True, True, F32, False),     # exactly one saved state
    (2, 9, 24, 5, 2, False, True, True, True, True, F32, False),    # padded states, odd groups
    (1, 33, 40, 16, 1, True, False, True, True, True, BF, False),   # one token past a tile
    (2, 47, 67 * 3, 12, 3, False, True, True, True, True, F32, True),
    (1, 300, 72, 16, 1, True, True, True, True, True, F32, False),
    (2, 130, 136, 16, 1, True, True, True, True, False, BF, False),  # ragged channel tiles
    (1, 65, 48, 32, 2, True, True, False, True, True, F32, False),
    (1, 70, 20, 64, 1, False, True, True, False, True, F32, False),
    (1, 1111, 24, 16, 1, True, True, True, True, True, F32, False),  # many segments, the last ragged
    (2, 530, 40, 6, 2, True, True, True, True, True, BF, False),     # several segments
    (2, 600, 256, 16, 256, False, True, True, True, True, F32, False),  # many tiles: segments in turn
    (5, 530, 256, 4, 256, True, False, True, True, True, BF, False),    # in turn in both directions
    (2, 64, 64, 20, 64, True, True, True, True, True, F32, False),   # a group per channel
    (1, 2943, 44, 12, 2, True, False, True, True, True, F32, False),  # long, and as many segments as fit
]


def scan_case(B, T, D, N, G, gate, skip, bias, softplus, carried, dtype, strided):
    g = torch.Generator().manual_seed(T + D)
    c = dict(x=rand(g, B, T, D, dtype=dtype),
             dt=(rand(g, B, T, D, scale=0.5) if softplus else rand(g, B, T, D).abs() * 0.2).to(dtype),
             A=-torch.exp(rand(g, D, N)), Bm=rand(g, B, T, G, N, dtype=dtype),
             Cm=rand(g, B, T, G, N, dtype=dtype), skip=rand(g, D) if skip else None,
             z=rand(g, B, T, D, dtype=dtype) if gate else None,
             dt_bias=(rand(g, D) - 2.0 if softplus else rand(g, D).abs() * 0.1) if bias else None,
             state=rand(g, B, D, N) if carried else None, dy=rand(g, B, T, D, dtype=dtype),
             dso=rand(g, B, D, N) if carried else None)
    return c


def scan_dev(c, strided=False):
    names = ("x", "dt", "Bm", "Cm", "z")
    return {k: dev(v, strided and k in names) for k, v in c.items()}


def scan_args(t):
    return (t["x"], t["dt"], t["A"], t["Bm"], t["Cm"])


def scan_kw(t, softplus):
    return dict(skip=t["skip"], z=t["z"], dt_bias=t["dt_bias"], softplus=softplus, state_in=t["state"])


@pytest.mark.parametrize("case", SCAN, ids=[f"b{c[0]}t{c[1]}d{c[2]}n{c[3]}g{c[4]}" for c in SCAN])
def test_scan_against_64_bits(case):
    B, T, D, N, G, gate, skip, bias, softplus, carried, dtype, strided = case
    c = scan_case(*case)
    t = scan_dev(c, strided)
    y, saved, end = block.selective_scan_forward(*scan_args(t), **scan_kw(t, softplus), want_state=True)
    alone, none, _ = block.selective_scan_forward(*scan_args(t), **scan_kw(t, softplus), keep_saved=False)
    got = block.selective_scan_backward(*scan_args(t), dev(c["dy"], strided), saved, **scan_kw(t, softplus),
                                        dstate_out=t["dso"], want_dstate=True)
    binding.check_device()
    assert none is None and torch.equal(alone, y)
    ref = scan64(*(d64(c[k]) for k in ("x", "dt", "A", "Bm", "Cm", "skip", "z", "dt_bias")), softplus,
                 d64(c["state"]), d64(c["dy"]), d64(c["dso"]))
    K = 64 + T + N  # T: where the scan is cut, the steps of a segment are summed before their exponential
    close(y, *ref["y"], K, "y")
    close(end, *ref["state"], K, "state")
    for name in ("dx", "ddt", "dstate_in", "dz"):
        if got[name] is not None:
            close(got[name], *ref[name], 2 * K, name)
    for name in ("dB", "dC"):
        close(got[name], *ref[name], 2 * K + D // G, name)
    for name in ("dA", "dskip", "ddt_bias"):
        if got[name] is not None:
            close(got[name], *ref[name], 2 * K + B * T, name)


@pytest.mark.parametrize("dtype,D,N", [(BF, 64, 16), (F32, 20, 7)])
def test_scan_pieces_and_steps_continue_a_sequence(dtype, D, N):
    """A prompt in two pieces, then single tokens, against 64 bits over the whole sequence."""
    B, T, G = 2, 60, 1
    c = scan_case(B, T, D, N, G, True, True, True, True, True, dtype, False)
    t = scan_dev(c)
    cut = lambda a, b: {k: (v[:, a:b] if k in ("x", "dt", "Bm", "Cm", "z") else v) for k, v in t.items()}
    p = cut(0, 11)
    y1, _, st = block.selective_scan_forward(*scan_args(p), **scan_kw(p, True), keep_saved=False,
                                             want_state=True)
    p = cut(11, 50)
    p["state"] = st
    y2, _, st = block.selective_scan_forward(*scan_args(p), **scan_kw(p, True), keep_saved=False,
                                             want_state=True)
    parts = [y1, y2]
    for i in range(50, T):
        parts.append(block.selective_scan_step(
            t["x"][:, i], t["dt"][:, i], t["A"], t["Bm"][:, i], t["Cm"][:, i], st, skip=t["skip"],
            z=t["z"][:, i], dt_bias=t["dt_bias"])[:, None])
    binding.check_device()
    ref = scan64(*(d64(c[k]) for k in ("x", "dt", "A", "Bm", "Cm", "skip", "z", "dt_bias")), True,
                 d64(c["state"]))
    close(torch.cat(parts, 1), *ref["y"], 64 + T + N, "y")
    close(st, *ref["state"], 64 + T + N, "state")


def test_scan_closed_decay_and_large_steps():
    """A step so large that the decay underflows forgets the state: y_t = C_t . (delta x B)_t."""
    B, T, D, N = 1, 20, 16, 16
    g = torch.Generator().manual_seed(3)
    x, Bm, Cm = rand(g, B, T, D), rand(g, B, T, 1, N), rand(g, B, T, 1, N)
    dt, A = torch.full((B, T, D), 50.0), torch.full((D, N), -10.0)
    t = [dev(v) for v in (x, dt, A, Bm, Cm)]
    y, saved, _ = block.selective_scan_forward(*t, state_in=dev(rand(g, B, D, N)))
    want = 50.0 * x.double() * (Bm * Cm).double().sum(-1)
    mag = 50.0 * x.double().abs() * (Bm * Cm).double().abs().sum(-1)
    close(y, want, mag, 64 + N, "y")
    dy = rand(g, B, T, D)
    got = block.selective_scan_backward(*t, dev(dy), saved)
    binding.check_device()
    assert not got["dA"].any(), "nothing passes a closed decay"


# ---- group norm ------------------------------------------------------------------------------------

# B, T, NH, d, scope, act, gated, affine, dtype, head-major, strided
NORM = [
    (1, 1, 1, 4, "token", "none", False, True, F32, True, False),
    (2, 1, 4, 64, "token", "sigmoid", True, True, BF, True, False),
    (2, 37, 3, 128, "token", "silu", True, True, BF, True, False),
    (2, 19, 2, 256, "token", "sigmoid", True, True, F32, True, False),
    (1, 33, 2, 512, "token", "silu", False, True, BF, False, False),
    (3, 21, 5, 67, "token", "silu", True, True, F32, False, True),
    (1, 50, 7, 17, "token", "none", False, False, BF, True, False),
    (2, 9, 1, 300, "token", "silu", False, True, F32, False, False),
    (1, 1, 2, 8, "sequence", "silu", False, True, F32, False, False),
    (2, 100, 4, 64, "sequence", "silu", False, True, BF, False, False),
    (2, 333, 5, 67, "sequence", "silu", False, True, F32, False, True),
    (1, 50, 2, 2056, "sequence", "none", False, True, F32, False, False),  # two channel blocks
    (2, 70, 3, 40, "sequence", "sigmoid", True, False, BF, True, False),
    (1, 3000, 1, 8, "sequence", "silu", True, True, F32, True, False),
    (8, 256, 128, 32, "sequence", "silu", False, True, BF, False, False),  # several chunks of groups
    (4, 200, 64, 64, "sequence", "sigmoid", True, True, F32, True, False),
]


def norm_case(B, T, NH, d, scope, act, gated, affine, dtype, hm, strided):
    g = torch.Generator().manual_seed(T + d)
    D = NH * d
    return dict(x=(rand(g, B, T, D) * 1.5 + 0.3).to(dtype), w=1 + rand(g, D, scale=0.2) if affine else None,
                b=rand(g, D, scale=0.2) if affine else None,
                gate=rand(g, B, T, D, dtype=dtype) if gated else None, dy=rand(g, B, T, D, dtype=dtype))


def run_norm(c, case, x=None):
    B, T, NH, d, scope, act, gated, affine, dtype, hm, strided = case
    if x is None:
        x = dev(heads(c["x"], NH)) if hm else dev(c["x"], strided)
    w, b, gate, dy = dev(c["w"]), dev(c["b"]), dev(c["gate"], strided), dev(c["dy"], strided)
    kw = dict(gate=gate, act=ACTS[act], scope=SCOPES[scope], groups=NH)
    y, stats = block.group_norm_forward(x, w, b, **kw)
    return y, block.group_norm_backward(x, w, b, dy, stats, **kw)


@pytest.mark.parametrize("case", NORM, ids=[f"{c[4]}_b{c[0]}t{c[1]}h{c[2]}d{c[3]}" for c in NORM])
def test_norm_against_64_bits(case):
    B, T, NH, d, scope, act, gated, affine, dtype, hm, strided = case
    c = norm_case(*case)
    y, got = run_norm(c, case)
    binding.check_device()
    part = lambda v: d64(v).view(B, T, NH, d)
    one, zero = torch.ones(NH, d, dtype=torch.float64), torch.zeros(NH, d, dtype=torch.float64)
    ref = norm64(part(c["x"]), d64(c["w"]).view(NH, d) if affine else one,
                 d64(c["b"]).view(NH, d) if affine else zero, part(c["gate"]) if gated else None, act, scope,
                 1e-5, part(c["dy"]))
    K = 64 + (d if scope == "token" else T + d)
    flat = lambda name: (v.reshape(B, T, NH * d) for v in ref[name])
    close(y, *flat("y"), K, "y")
    dx = last(got["dx"]) if hm else got["dx"]
    close(dx, *flat("dx"), 2 * K, "dx")
    if gated:
        close(got["dgate"], *flat("dgate"), K, "dgate")
    if affine:
        close(got["dweight"], *(v.flatten() for v in ref["dweight"]), K + B * T, "dweight")
        close(got["dbias"], *(v.flatten() for v in ref["dbias"]), K + B * T, "dbias")


# groups too large for the shared memory of a cluster (more than 2048 channels, or long), or nearly so
NORM_LARGE = [
    (1, 900, 3, 1000, "sequence", "silu", False, True, BF, False, False),
    (2, 480, 2, 1021, "sequence", "sigmoid", True, True, F32, True, False),   # element accesses
    (12, 33, 9, 2050, "sequence", "none", False, True, F32, False, True),     # several chunks of groups
    (2, 700, 2, 1024, "sequence", "silu", True, False, BF, True, False),
    (1, 1, 2, 2056, "sequence", "silu", False, True, BF, False, False),       # one token
    (5, 160, 32, 512, "sequence", "silu", False, True, F32, False, False),    # eight CTAs, two to an SM
    (1, 400, 2, 512, "sequence", "silu", False, True, F32, True, False),      # alone on their SMs: backward
    (1, 400, 2, 508, "sequence", "silu", True, True, F32, False, False),      # and forward
]


@pytest.mark.parametrize("case", NORM_LARGE, ids=[f"b{c[0]}t{c[1]}h{c[2]}d{c[3]}" for c in NORM_LARGE])
def test_norm_of_large_groups_against_64_bits(case):
    test_norm_against_64_bits(case)


def large_group_inputs(seed):
    case = (3, 40, 5, 2056, "sequence", "silu", True, True, BF, False, False)
    g = torch.Generator().manual_seed(seed)
    return {k: dev(rand(g, *v.shape, dtype=v.dtype)) for k, v in norm_case(*case).items()}


def run_large_group(t, stream=None):
    kw = dict(gate=t["gate"], act=block.ACT_SILU, scope=block.SCOPE_SEQUENCE, groups=5, stream=stream)
    y, stats = block.group_norm_forward(t["x"], t["w"], t["b"], **kw)
    return {"y": y, **block.group_norm_backward(t["x"], t["w"], t["b"], t["dy"], stats, **kw)}


def test_norms_of_large_groups_at_once_and_replayed():
    """CTAs that wait for one another's sums: two launches at once, and a graph of one replayed."""
    t = [large_group_inputs(s) for s in (1, 2)]
    want = [run_large_group(v) for v in t]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in t]
    got = [[run_large_group(v, s) for v, s in zip(t, streams)] for _ in range(3)]
    torch.cuda.synchronize()
    for rep in got:
        for a, b in zip(rep, want):
            same(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run_large_group(t[0])
    for k in t[0]:
        t[0][k].copy_(t[1][k])
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        same(out, want[1])
    binding.check_device()


@pytest.mark.parametrize("d", [64, 2056])
def test_norm_with_one_value_far_from_the_rest(d):
    """The first vector of a group lies 2^12 off: the others' distances keep their bits beside it."""
    g = torch.Generator().manual_seed(12)
    B, T, NH = 1, 200, 2
    x = rand(g, B, T, NH * d)
    x[:, 0, :8] += 4096.0
    x[:, :, d:] += 4096.0
    y, _ = block.group_norm_forward(dev(x), groups=NH, scope=block.SCOPE_SEQUENCE)
    one, zero = torch.ones(NH, d, dtype=torch.float64), torch.zeros(NH, d, dtype=torch.float64)
    ref, mag = norm64(d64(x).view(B, T, NH, d), one, zero, None, "none", "sequence", 1e-5)["y"]
    close(y, ref.reshape(B, T, -1), mag.reshape(B, T, -1), 64 + T + d, "y")


@pytest.mark.parametrize("scope", ["token", "sequence"])
def test_norm_of_values_far_from_zero(scope):
    """A common offset of 4096 leaves the statistics: squares are never subtracted.  fp32 holds the
    inputs to 2^-12 here, and the kernel gets those rounded inputs."""
    g = torch.Generator().manual_seed(11)
    B, T, NH, d = 1, 64, 2, 64
    x = rand(g, B, T, NH * d) + 4096.0
    y, _ = block.group_norm_forward(dev(x), groups=NH, scope=SCOPES[scope])
    one, zero = torch.ones(NH, d, dtype=torch.float64), torch.zeros(NH, d, dtype=torch.float64)
    ref, mag = norm64(d64(x).view(B, T, NH, d), one, zero, None, "none", scope, 1e-5)["y"]
    close(y, ref.reshape(B, T, -1), mag.reshape(B, T, -1), 64, "y")


def test_norm_of_constant_rows_is_the_bias():
    x = torch.full((2, 5, 24), 3.25, device="cuda")
    b = torch.arange(24.0, device="cuda")
    for scope in SCOPES.values():
        y, stats = block.group_norm_forward(x, None, b, groups=3, scope=scope)
        got = block.group_norm_backward(x, None, b, torch.ones_like(x), stats, groups=3, scope=scope)
        assert torch.equal(y, b.expand(2, 5, 24)) and torch.equal(got["dx"], torch.zeros_like(x))


# ---- how they are called ----------------------------------------------------------------------------

def all_calls(seed, dtype=BF, T=70):
    """One forward and backward of each operator on inputs of this seed: a flat dict of results."""
    g = torch.Generator().manual_seed(seed)
    B, NH, d, N = 2, 2, 64, 16
    D = NH * d
    ins = {"x": rand(g, B, T, D, dtype=dtype), "w": rand(g, D, 4), "b": rand(g, D),
           "dt": rand(g, B, T, D, dtype=dtype, scale=0.5), "A": -torch.exp(rand(g, D, N)),
           "Bm": rand(g, B, T, N, dtype=dtype), "Cm": rand(g, B, T, N, dtype=dtype),
           "z": rand(g, B, T, D, dtype=dtype), "dy": rand(g, B, T, D, dtype=dtype)}
    return {k: v.cuda() for k, v in ins.items()}


def run_all(t, stream=None):
    out = {}
    y, _ = block.causal_conv_forward(t["x"], t["w"], t["b"], stream=stream)
    out["conv"] = y
    out.update({"conv_" + k: v for k, v in block.causal_conv_backward(
        t["x"], t["w"], t["b"], t["dy"], stream=stream).items()})
    args, kw = (t["x"], t["dt"], t["A"], t["Bm"], t["Cm"]), dict(skip=t["b"], z=t["z"], dt_bias=t["b"])
    y, saved, end = block.selective_scan_forward(*args, **kw, want_state=True, stream=stream)
    out["scan"], out["scan_state"] = y, end
    out.update({"scan_" + k: v for k, v in block.selective_scan_backward(
        *args, t["dy"], saved, **kw, stream=stream).items()})
    for scope in SCOPES.values():
        kw = dict(gate=t["z"], act=block.ACT_SILU, scope=scope, groups=2)
        y, stats = block.group_norm_forward(t["x"], t["b"], t["b"], **kw, stream=stream)
        out[f"norm{scope}"] = y
        out.update({f"norm{scope}_" + k: v for k, v in block.group_norm_backward(
            t["x"], t["b"], t["b"], t["dy"], stats, **kw, stream=stream).items()})
    return {k: v for k, v in out.items() if v is not None}


def same(a, b):
    assert a.keys() == b.keys()
    for k in a:
        assert torch.equal(a[k], b[k]), k


def test_repeated_calls_have_the_same_bits():
    t = all_calls(1)
    first = run_all(t)
    for _ in range(3):
        same(run_all(t), first)


def test_calls_on_other_streams_at_once():
    t = [all_calls(s) for s in (1, 2)]
    want = [run_all(v) for v in t]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in t]
    got = [[run_all(v, s) for v, s in zip(t, streams)] for _ in range(3)]
    torch.cuda.synchronize()
    for rep in got:
        for a, b in zip(rep, want):
            same(a, b)


def test_captured_calls_replay_on_new_inputs():
    """Two graphs captured from the same code, replayed at once on their own inputs."""
    held = [all_calls(s) for s in (3, 4)]
    run_all(held[0])
    graphs, outs = [], []
    for t in held:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(run_all(t))
        graphs.append(g)
    fresh = [all_calls(s) for s in (5, 6)]
    want = [run_all(f) for f in fresh]
    for t, f in zip(held, fresh):
        for k in t:
            t[k].copy_(f[k])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in graphs]
    for g, s in zip(graphs, streams):
        with torch.cuda.stream(s):
            g.replay()
    torch.cuda.synchronize()
    for a, b in zip(outs, want):
        same(a, b)


def in_turn_inputs(seed):
    """Many channel tiles and several segments: both directions of the scan take work in turn."""
    case = (5, 530, 256, 4, 256, True, False, True, True, True, BF, False)
    g = torch.Generator().manual_seed(seed)
    c = scan_case(*case)
    for name in ("x", "z", "dy"):
        c[name] = rand(g, *c[name].shape, dtype=BF)
    return scan_dev(c)


def run_in_turn(t, stream=None):
    kw = dict(**scan_kw(t, True), stream=stream)
    y, saved, end = block.selective_scan_forward(*scan_args(t), **kw, want_state=True)
    got = block.selective_scan_backward(*scan_args(t), t["dy"], saved, **kw, dstate_out=t["dso"],
                                        want_dstate=True)
    return {"y": y, "end": end, **{k: v for k, v in got.items() if v is not None}}


def test_scans_in_turn_at_once_and_replayed():
    """CTAs that wait for one another within a launch: two such launches at once, and a graph of one
    replayed (its counters start again from zero each time)."""
    t = [in_turn_inputs(s) for s in (1, 2)]
    want = [run_in_turn(v) for v in t]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in t]
    got = [[run_in_turn(v, s) for v, s in zip(t, streams)] for _ in range(3)]
    torch.cuda.synchronize()
    for rep in got:
        for a, b in zip(rep, want):
            same(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run_in_turn(t[0])
    for k in t[0]:
        if t[0][k] is not None:
            t[0][k].copy_(t[1][k])
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        same(out, want[1])
    binding.check_device()


def test_offsets_beyond_32_bits():
    """Tensors of more than 2^31 elements: the last tokens are those of a call that starts there."""
    T, T0, D, NH = 280000, 279900, 8192, 64
    x = torch.empty(1, T, D, dtype=BF, device="cuda").normal_(generator=torch.Generator("cuda").manual_seed(1))
    assert x.numel() > 2 ** 31
    w, b = torch.randn(D, 4, device="cuda"), torch.randn(D, device="cuda")
    y, end = block.causal_conv_forward(x, w, b, want_state=True)
    _, st = block.causal_conv_forward(x[:, T0 - 3:T0], w, b, want_state=True)
    tail, end2 = block.causal_conv_forward(x[:, T0:], w, b, state_in=st, want_state=True)
    assert torch.equal(y[:, T0:], tail) and torch.equal(end, end2)
    got = block.causal_conv_backward(x, w, b, x)
    part = block.causal_conv_backward(x[:, T0:], w, b, x[:, T0:], state_in=st)
    assert torch.equal(got["dx"][:, T0:], part["dx"])
    del got, part
    for act in (block.ACT_NONE, block.ACT_SILU):
        y, stats = block.group_norm_forward(x, b, b, groups=NH, act=act)
        part, stats2 = block.group_norm_forward(x[:, T0:], b, b, groups=NH, act=act)
        assert torch.equal(y[:, T0:], part) and torch.equal(stats[:, T0:], stats2)
    got = block.group_norm_backward(x, b, b, x, stats, groups=NH, act=block.ACT_SILU)
    part = block.group_norm_backward(x[:, T0:], b, b, x[:, T0:], stats2, groups=NH, act=block.ACT_SILU)
    assert torch.equal(got["dx"][:, T0:], part["dx"])
    del got, part
    y, stats = block.group_norm_forward(x, b, b, groups=NH, scope=block.SCOPE_SEQUENCE)
    mean, rstd = stats[0, :, 0].repeat_interleave(D // NH), stats[0, :, 1].repeat_interleave(D // NH)
    want = (x[0, T0:].float() - mean) * rstd * b + b
    assert float((y[0, T0:].float() - want).abs().max()) <= 2.0 ** -8 * float(want.abs().max()) * 1.01
    del y
    A, Bm = -torch.ones(D, 1, device="cuda"), torch.ones(1, T, 1, dtype=BF, device="cuda")
    y, _, end = block.selective_scan_forward(x, x, A, Bm, Bm, keep_saved=False, want_state=True)
    # a step of softplus(x) on average forgets e^-0.8 a token: 400 tokens before T0 decide the state there
    _, _, st = block.selective_scan_forward(x[:, T0 - 400:T0], x[:, T0 - 400:T0], A, Bm[:, :400], Bm[:, :400],
                                            keep_saved=False, want_state=True)
    tail, _, end2 = block.selective_scan_forward(x[:, T0:], x[:, T0:], A, Bm[:, T0:], Bm[:, T0:], state_in=st,
                                                 keep_saved=False, want_state=True)
    # the same operations in other segments: fp32 states to 1e-5 of the largest, outputs to a bf16 step
    assert float((end - end2).abs().max()) <= 1e-5 * float(end.abs().max())
    assert float((y[:, T0:].float() - tail.float()).abs().max()) <= 2.0 ** -7 * float(tail.float().abs().max())
    binding.check_device()


def test_a_bad_batch_stays_alone():
    """NaN and infinities in one batch leave the other's outputs and gradients as they were."""
    t = all_calls(8)
    clean = run_all(t)
    for name in ("x", "dt", "Bm", "Cm", "z", "dy"):
        t[name][0, ::3] = float("nan")
        t[name][0, 1::3] = float("inf")
    dirty = run_all(t)
    batched = [k for k in clean if clean[k].shape[0] == 2 and clean[k].dim() > 1]
    assert len(batched) >= 15
    for k in batched:
        assert torch.equal(dirty[k][1], clean[k][1]), k


def test_outputs_stay_inside_their_rows():
    """Strided outputs through the C ABI: what lies between and behind the rows is left as it was."""
    g = torch.Generator().manual_seed(9)
    B, T, D, pad = 2, 41, 24, 8
    lib = binding.load()
    x, w = dev(rand(g, B, T, D, dtype=BF)), dev(rand(g, D, 4))
    A, Bm = dev(-torch.exp(rand(g, D, 16))), dev(rand(g, B, T, 16, dtype=BF))
    s = binding._stream_handle(None)

    def room():
        return torch.full((B, T + 3, D + pad), 7.0, dtype=BF, device="cuda")

    def untouched(o):
        return bool((o[:, T:] == 7.0).all() and (o[:, :, D:] == 7.0).all())

    def rows(o):
        return binding.Rows(o.data_ptr(), o.stride(0), o.stride(1), 12)

    o = room()
    assert lib.mlstm_conv_fwd(block._rows(x), w.data_ptr(), None, None, rows(o), None, B, T, 2, 12, 4, 1,
                              binding.BF16, s) == 0
    want, _ = block.causal_conv_forward(x, w)
    assert untouched(o) and torch.equal(o[:, :T, :D], want)
    o = room()
    p = block._scan_problem(x, x, A, Bm, Bm, None, None, None, True, None)
    assert lib.mlstm_scan_fwd(p, rows(o), None, None, None, 0, s) == 0
    want, _, _ = block.selective_scan_forward(x, x, A, Bm, Bm)
    assert untouched(o) and torch.equal(o[:, :T, :D], want)
    o = room()
    x2 = binding.Rows(x.data_ptr(), x.stride(0), x.stride(1), 12)
    assert lib.mlstm_group_norm_fwd(x2, None, None, None, rows(o), None, None, 0, B, T, 2, 12, 0, 1, 1e-5,
                                    binding.BF16, s) == 0
    want, _ = block.group_norm_forward(x, act=block.ACT_SILU, groups=2)
    assert untouched(o) and torch.equal(o[:, :T, :D], want)
    binding.check_device()


def test_empty_sequences_pass_states_through():
    x = torch.zeros(2, 0, 16, dtype=BF, device="cuda")
    w = torch.ones(16, 4, device="cuda")
    st = torch.randn(2, 3, 16, device="cuda").to(BF)
    y, so = block.causal_conv_forward(x, w, state_in=st, want_state=True)
    assert y.shape == (2, 0, 16) and torch.equal(so, st)
    got = block.causal_conv_backward(x, w, None, x, state_in=st, dstate_out=st, want_dstate=True)
    assert torch.equal(got["dstate_in"], st) and not got["dweight"].any()
    A, s0 = -torch.ones(16, 5, device="cuda"), torch.randn(2, 16, 5, device="cuda")
    Bm = torch.zeros(2, 0, 5, dtype=BF, device="cuda")
    y, saved, end = block.selective_scan_forward(x, x, A, Bm, Bm, state_in=s0, want_state=True)
    assert y.shape == x.shape and torch.equal(end, s0)
    got = block.selective_scan_backward(x, x, A, Bm, Bm, x, saved, state_in=s0, dstate_out=s0,
                                        want_dstate=True)
    assert torch.equal(got["dstate_in"], s0) and not got["dA"].any()
    b = torch.ones(16, device="cuda")
    for scope in SCOPES.values():
        y, stats = block.group_norm_forward(x, b, b, groups=2, scope=scope)
        got = block.group_norm_backward(x, b, b, x, stats, groups=2, scope=scope)
        assert y.shape == x.shape and not got["dweight"].any() and not got["dbias"].any()


def test_refusals_on_the_device():
    x = torch.zeros(2, 5, 16, dtype=BF, device="cuda")
    w = torch.zeros(16, 4, device="cuda")
    with pytest.raises(TypeError, match="float32"):
        block.causal_conv_forward(x, w.to(BF))
    with pytest.raises(ValueError, match="shape"):
        block.causal_conv_forward(x, w[:8])
    with pytest.raises(binding.MLSTMError):
        block.causal_conv_forward(x, torch.zeros(16, 7, device="cuda"))
    with pytest.raises(TypeError, match="dtype"):
        block.causal_conv_forward(x.half(), w)
    with pytest.raises(ValueError, match="last dimension"):
        block.causal_conv_forward(torch.zeros(2, 16, 5, dtype=BF, device="cuda").transpose(1, 2), w)
    with pytest.raises(ValueError, match="contiguous"):
        block.causal_conv_forward(x, w, state_in=torch.zeros(2, 16, 3, dtype=BF, device="cuda").transpose(1, 2))
    with pytest.raises(ValueError, match="heads"):
        block.causal_conv_forward(x, w, heads=3)
    A, Bm = torch.zeros(16, 4, device="cuda"), torch.zeros(2, 5, 4, dtype=BF, device="cuda")
    with pytest.raises(ValueError, match="groups"):
        block.selective_scan_forward(x, x, A, Bm.view(2, 5, 1, 4).expand(2, 5, 3, 4), Bm.view(2, 5, 1, 4).expand(2, 5, 3, 4))
    with pytest.raises(binding.MLSTMError):
        block.selective_scan_forward(x, x, torch.zeros(16, 65, device="cuda"),
                                     torch.zeros(2, 5, 65, dtype=BF, device="cuda"),
                                     torch.zeros(2, 5, 65, dtype=BF, device="cuda"))
    with pytest.raises(ValueError, match="saved"):
        block.selective_scan_backward(x, x, A, Bm, Bm, x, None)
    with pytest.raises(ValueError, match="saved"):
        block.selective_scan_backward(x, x, A, Bm, Bm, x, torch.zeros(16, device="cuda"))
    wide = torch.zeros(1, 2, 1, 520, device="cuda")
    with pytest.raises(binding.MLSTMError):
        block.group_norm_forward(wide)
    with pytest.raises(ValueError, match="gate"):
        block.group_norm_forward(x, groups=2, gate=x[:, :3])
    with pytest.raises(ValueError, match="stats"):
        block.group_norm_backward(x, None, None, x, None, groups=2)


def test_saved_states_are_refused_unless_contiguous():
    x = torch.zeros(2, 5, 16, dtype=BF, device="cuda")
    A, Bm = torch.zeros(16, 4, device="cuda"), torch.zeros(2, 5, 4, dtype=BF, device="cuda")
    _, saved, _ = block.selective_scan_forward(x, x, A, Bm, Bm)
    with pytest.raises(ValueError, match="contiguous"):
        block.selective_scan_backward(x, x, A, Bm, Bm, x, saved.repeat(2)[::2])


# ---- together, as a block uses them --------------------------------------------------------------

@pytest.mark.parametrize("variant", [binding.SIG, binding.EXP], ids=["sig", "exp"])
def test_block_around_the_cell(variant):
    """conv -> q, k; the cell; head-wise norm with an output gate: values and gradients.  Each stage is
    compared with 64 bits on the inputs it got from the stage before (the cell at its own parity bar)."""
    g = torch.Generator().manual_seed(21)
    B, T, NH, d, L = 2, 150, 2, 64, 64
    D = NH * d
    x, w, cb = rand(g, B, T, D), rand(g, D, 4, scale=0.5), rand(g, D, scale=0.1)
    ig, fg = rand(g, B, NH, T) - 1.0, rand(g, B, NH, T) + 3.0
    nw, nb, og, dy = 1 + rand(g, D, scale=0.1), rand(g, D, scale=0.1), rand(g, B, T, D), rand(g, B, T, D)
    X, W, CB, IG, FG, NW, NB, OG, DY = (dev(v) for v in (x, w, cb, ig, fg, nw, nb, og, dy))
    qk, _ = block.causal_conv_forward(X, W, CB, heads=NH)
    v = X.view(B, T, NH, d).transpose(1, 2).contiguous()
    h, saved = binding.forward(qk, qk, v, IG, FG, L, variant)
    kw = dict(gate=OG, act=block.ACT_SIGMOID)
    y, stats = block.group_norm_forward(h, NW, NB, **kw)
    gn = block.group_norm_backward(h, NW, NB, DY, stats, **kw)
    gc = binding.backward(qk, qk, v, IG, FG, h, gn["dx"], saved, L, variant)
    dqk = gc["dq"] + gc["dk"]
    gx = block.causal_conv_backward(X, W, CB, dqk)
    binding.check_device()
    # the convolution, and back through it
    ref = conv64(d64(x), d64(w), d64(cb), None, "silu", last(dqk).double().cpu())
    close(last(qk), *ref["y"], 64, "q, k")
    close(gx["dx"], *ref["dx"], 64, "dx")
    close(gx["dweight"], *ref["dweight"], 64 + B * T, "dweight")
    # the cell on those q and k
    for b in range(B):
        for hh in range(NH):
            one = lambda a: a[b, hh].double().cpu().numpy()
            li, lf = oracle.gate_logs(one(IG), one(FG), variant)
            want = oracle.chunkwise_forward(one(qk), one(qk), one(v), li, lf, variant, L)["h"]
            assert np.max(np.abs(one(h) - want)) <= 1e-4 * np.max(np.abs(want))
            back = oracle.parallel_backward(one(qk), one(qk), one(v), li, lf, variant, one(gn["dx"]))
            for name in ("dq", "dk", "dv"):
                assert np.max(np.abs(one(gc[name]) - back[name])) <= 1e-4 * np.max(np.abs(back[name])), name
    # the norm and gate on that h
    part = lambda a: d64(a.cpu()).view(B, T, NH, d)
    ref = norm64(last(h).double().cpu().view(B, T, NH, d), d64(nw).view(NH, d), d64(nb).view(NH, d), part(og),
                 "sigmoid", "token", 1e-5, part(dy))
    close(y, *(r.reshape(B, T, D) for r in ref["y"]), 64 + d, "y")
    close(last(gn["dx"]), *(r.reshape(B, T, D) for r in ref["dx"]), 2 * (64 + d), "dh")
    close(gn["dgate"], *(r.reshape(B, T, D) for r in ref["dgate"]), 64 + d, "dgate")


def test_block_prompt_then_tokens():
    """The same block in generation: a prompt, then single tokens through every operator's state, against
    one pass over the whole sequence.  The cell's two forms differ by delta = 2e-4 of its largest output
    (1e-4 each); through the norm that is at most rstd delta (2 + |xhat|), and |xhat| <= sqrt(d) = 8."""
    g = torch.Generator().manual_seed(22)
    B, T, T0, NH, d, L, var = 2, 80, 64, 2, 64, 64, binding.SIG
    D = NH * d
    x, w = dev(rand(g, B, T, D)), dev(rand(g, D, 4, scale=0.5))
    ig, fg = dev(rand(g, B, NH, T)), dev(rand(g, B, NH, T) + 3.0)
    og = dev(rand(g, B, T, D))

    def vals(xs, n):
        return xs.view(B, n, NH, d).transpose(1, 2).contiguous()

    qk, _ = block.causal_conv_forward(x, w, heads=NH)
    h, _ = binding.forward(qk, qk, vals(x, T), ig, fg, L, var)
    whole, stats = block.group_norm_forward(h, gate=og, act=block.ACT_SIGMOID)
    hmax = float(h.abs().max())
    xp = x[:, :T0]
    qk, cst = block.causal_conv_forward(xp, w, heads=NH, want_state=True)
    gates = [a[:, :, :T0].contiguous() for a in (ig, fg)]
    h, saved = binding.forward(qk, qk, vals(xp.contiguous(), T0), *gates, L, var)
    state = binding.final_state(qk, vals(xp.contiguous(), T0), saved, L, var)
    other = torch.empty_like(state)
    parts = [block.group_norm_forward(h, gate=og[:, :T0], act=block.ACT_SIGMOID)[0]]
    for t in range(T0, T):
        q1 = block.causal_conv_step(x[:, t], w, None, cst, heads=NH)
        h1 = binding.step(q1, q1, x[:, t].reshape(B, NH, d).contiguous(), ig[:, :, t].contiguous(),
                          fg[:, :, t].contiguous(), state, other, var)
        state, other = other, state
        parts.append(block.group_norm_forward(h1[:, :, None], gate=og[:, t:t + 1], act=block.ACT_SIGMOID)[0])
    binding.check_device()
    got = torch.cat(parts, 1)
    rstd = float(stats[..., 1].max())
    tol = 2e-4 * hmax * rstd * 10
    assert float((got - whole).abs().max()) <= tol
