"""The operators around the recurrence, without a GPU: their 64-bit forms' gradients against central
differences, the C entry points' argument errors (all before any launch), the empty problems, and
the Python functions' refusals."""

import ctypes
import os

import pytest
import torch

from mlstm_chunkwise_attention_b200 import binding as B
from mlstm_chunkwise_attention_b200 import block
from _block_ref import conv64, norm64, scan64


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(B.LIB_PATH):
        from mlstm_chunkwise_attention_b200 import _build
        _build.build()
    return B.load()


# ---- the 64-bit forms --------------------------------------------------------------------------

def _differences(fn, inputs, cotangents, grads, h=1e-6):
    """Central differences of sum <cotangent, output> in a random direction of each input."""
    g = torch.Generator().manual_seed(5)

    def loss(ins):
        out = fn(**ins)
        return float(sum((out[k][0] * c).sum() for k, c in cotangents.items()))

    for name, grad in grads.items():
        direction = torch.randn(inputs[name].shape, generator=g, dtype=torch.float64)
        up, down = dict(inputs), dict(inputs)
        up[name], down[name] = inputs[name] + h * direction, inputs[name] - h * direction
        slope = (loss(up) - loss(down)) / (2 * h)
        # the differences' own error: rounding 2^-52 |loss| / h, truncation of order h^2
        assert abs(slope - float((grad * direction).sum())) <= 1e-6 * max(1.0, abs(slope)), name


def _rand(g, *shape):
    return torch.randn(*shape, generator=g, dtype=torch.float64)


@pytest.mark.parametrize("act", ["none", "silu"])
@pytest.mark.parametrize("T", [1, 2, 9])
def test_conv_gradients_against_differences(act, T):
    g = torch.Generator().manual_seed(1)
    ins = dict(x=_rand(g, 2, T, 5), w=_rand(g, 5, 4), bias=_rand(g, 5), state=_rand(g, 2, 3, 5))
    cot = dict(y=_rand(g, 2, T, 5), state=_rand(g, 2, 3, 5))
    out = conv64(**ins, act=act, dy=cot["y"], dstate_out=cot["state"])
    _differences(lambda **k: conv64(**k, act=act), ins, cot,
                 dict(x=out["dx"][0], w=out["dweight"][0], bias=out["dbias"][0],
                      state=out["dstate_in"][0]))


@pytest.mark.parametrize("softplus", [True, False])
def test_scan_gradients_against_differences(softplus):
    g = torch.Generator().manual_seed(2)
    ins = dict(x=_rand(g, 2, 7, 6), dt=_rand(g, 2, 7, 6).abs() * 0.3, A=-_rand(g, 6, 3).abs(),
               Bm=_rand(g, 2, 7, 2, 3), Cm=_rand(g, 2, 7, 2, 3), skip=_rand(g, 6), z=_rand(g, 2, 7, 6),
               dt_bias=_rand(g, 6) * 0.1, state=_rand(g, 2, 6, 3))
    cot = dict(y=_rand(g, 2, 7, 6), state=_rand(g, 2, 6, 3))
    out = scan64(**ins, softplus=softplus, dy=cot["y"], dstate_out=cot["state"])
    _differences(lambda **k: scan64(**k, softplus=softplus), ins, cot,
                 dict(x=out["dx"][0], dt=out["ddt"][0], A=out["dA"][0], Bm=out["dB"][0],
                      Cm=out["dC"][0], skip=out["dskip"][0], z=out["dz"][0],
                      dt_bias=out["ddt_bias"][0], state=out["dstate_in"][0]))


@pytest.mark.parametrize("scope", ["token", "sequence"])
@pytest.mark.parametrize("act,gated", [("none", False), ("silu", False), ("sigmoid", True), ("silu", True)])
def test_norm_gradients_against_differences(scope, act, gated):
    g = torch.Generator().manual_seed(3)
    ins = dict(x=_rand(g, 2, 4, 3, 5), w=_rand(g, 3, 5), b=_rand(g, 3, 5),
               gate=_rand(g, 2, 4, 3, 5) if gated else None)
    cot = dict(y=_rand(g, 2, 4, 3, 5))
    fn = lambda **k: norm64(**k, act=act, scope=scope, eps=1e-5)
    out = norm64(**ins, act=act, scope=scope, eps=1e-5, dy=cot["y"])
    grads = dict(x=out["dx"][0], w=out["dweight"][0], b=out["dbias"][0])
    if gated:
        grads["gate"] = out["dgate"][0]
    _differences(fn, ins, cot, grads)


def test_scan_with_constant_gates_is_a_decayed_sum():
    """A closed form: delta = 1, A = log r, B = C = 1 gives y_t = sum_{s <= t} r^(t - s) x_s."""
    T, r = 6, 0.7
    x = torch.arange(1.0, T + 1, dtype=torch.float64).view(1, T, 1)
    one = torch.ones(1, T, 1, 1, dtype=torch.float64)
    A = torch.full((1, 1), float(torch.log(torch.tensor(r, dtype=torch.float64))), dtype=torch.float64)
    y = scan64(x, torch.ones_like(x), A, one, one, softplus=False)["y"][0].flatten()
    want = [sum(r ** (t - s) * (s + 1) for s in range(t + 1)) for t in range(T)]
    assert torch.allclose(y, torch.tensor(want, dtype=torch.float64), rtol=1e-12, atol=0)


# ---- the C entry points -------------------------------------------------------------------------

FAKE = 0x100000  # aligned addresses that no call dereferences: every one of these returns before a launch


def rows(ptr=FAKE, batch=4096, token=64, head=16):
    return B.Rows(ptr, batch, token, head)


def conv_fwd(lib, x=rows(), w=FAKE, bias=None, si=None, y=rows(), so=None, Bn=2, T=5, NH=4, d=16, W=4,
             act=block.ACT_SILU, dtype=B.BF16):
    return lib.mlstm_conv_fwd(x, w, bias, si, y, so, Bn, T, NH, d, W, act, dtype, None)


@pytest.mark.parametrize("kw,status", [
    (dict(Bn=-1), 1), (dict(T=-1), 1), (dict(NH=0), 1), (dict(d=0), 1), (dict(W=0), 1),
    (dict(dtype=5), 1), (dict(act=block.ACT_SIGMOID), 1), (dict(act=9), 1),
    (dict(W=1), 2), (dict(W=5), 2), (dict(Bn=1 << 15, T=1 << 15), 2), (dict(NH=1 << 13, d=1 << 12), 2),
    (dict(x=B.Rows(None, 0, 0, 0)), 1), (dict(x=rows(FAKE + 1)), 1), (dict(y=rows(FAKE + 1)), 1),
    (dict(w=None), 1), (dict(w=FAKE + 2), 1), (dict(bias=FAKE + 2), 1), (dict(si=FAKE + 1), 1),
    (dict(si=FAKE, so=FAKE), 1), (dict(si=FAKE, so=FAKE + 64), 1),
])
def test_conv_argument_errors(lib, kw, status):
    assert conv_fwd(lib, **kw) == status


def test_conv_backward_and_step_argument_errors(lib):
    need = lib.mlstm_conv_bwd_workspace_size(2, 5, 4, 16, 4, B.BF16)
    assert need > 0 and lib.mlstm_conv_bwd_workspace_size(2, 5, 4, 16, 7, B.BF16) == 0

    def bwd(dw=FAKE, ws=FAKE, nbytes=need, dso=None, dsi=None, dx=rows(), W=4, si=None):
        return lib.mlstm_conv_bwd(rows(), FAKE, None, si, rows(), dso, dx, dw, None, dsi, ws, nbytes, 2, 5,
                                  4, 16, W, block.ACT_SILU, B.BF16, None)

    assert bwd(dw=None) == 1 and bwd(dx=rows(None)) == 1 and bwd(W=9) == 2
    assert bwd(ws=None) == 3 and bwd(nbytes=need - 1) == 3 and bwd(ws=FAKE + 4) == 1
    assert bwd(dso=FAKE, dsi=FAKE + 8) == 1 and bwd(si=FAKE, dsi=FAKE + 8) == 1

    def step(si=FAKE, so=FAKE, Bn=2):
        return lib.mlstm_conv_step(rows(), FAKE, None, si, rows(), so, Bn, 4, 16, 4, block.ACT_SILU,
                                   B.BF16, None)

    assert step(si=None) == 1 and step(so=None) == 1 and step(so=FAKE + 32) == 1
    assert step(Bn=0) == 0


def scan_problem(**kw):
    p = B.ScanProblem()
    p.x, p.dt, p.z, p.b, p.c = rows(), rows(), B.Rows(None, 0, 0, 0), rows(), rows()
    p.a = FAKE
    p.B, p.T, p.D, p.G, p.N, p.softplus, p.dtype = 2, 5, 64, 1, 16, 1, B.BF16
    for k, v in kw.items():
        setattr(p, k, v)
    return p


@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), 1), (dict(T=-2), 1), (dict(D=0), 1), (dict(G=0), 1), (dict(N=0), 1), (dict(G=3), 1),
    (dict(dtype=2), 1), (dict(N=65), 2), (dict(B=1 << 16, T=1 << 14), 2),
    (dict(x=rows(None)), 1), (dict(dt=rows(FAKE + 1)), 1), (dict(b=rows(None)), 1), (dict(a=None), 1),
    (dict(z=rows(FAKE + 1)), 1), (dict(skip=FAKE + 1), 1), (dict(state_in=FAKE + 4), 1),
])
def test_scan_argument_errors(lib, kw, status):
    p = scan_problem(**kw)
    assert lib.mlstm_scan_fwd(p, rows(), None, None, None, 0, None) == status
    grads = B.ScanGrads()
    grads.dx = grads.ddt = grads.dz = grads.db = grads.dc = rows()
    grads.da = FAKE
    assert lib.mlstm_scan_bwd(p, rows(), FAKE, None, grads, FAKE, 1 << 40, None) == status


def test_scan_states_workspaces_and_step_errors(lib):
    p = scan_problem(state_in=FAKE)
    assert lib.mlstm_scan_fwd(None, rows(), None, None, None, 0, None) == 1
    assert lib.mlstm_scan_fwd(p, rows(), None, FAKE + 1024, None, 0, None) == 1  # overlapping states
    assert lib.mlstm_scan_fwd(p, rows(), FAKE + 8, None, None, 0, None) == 1  # misaligned saved
    assert lib.mlstm_scan_fwd(p, rows(None), None, None, None, 0, None) == 1
    assert lib.mlstm_scan_step(p, rows(), None, None) == 1
    assert lib.mlstm_scan_step(p, rows(), FAKE + 512, None) == 1
    assert lib.mlstm_scan_step(scan_problem(), rows(), FAKE, None) == 1    # no state
    grads = B.ScanGrads()
    grads.dx = grads.ddt = grads.db = grads.dc = rows()
    grads.da = FAKE
    need = lib.mlstm_scan_bwd_workspace_size(2, 5, 64, 1, 16, B.BF16)
    args = (scan_problem(), rows(), FAKE, None, grads, FAKE)
    assert need > 0 and lib.mlstm_scan_bwd(*args, need - 1, None) == 3
    assert lib.mlstm_scan_bwd(scan_problem(), rows(), None, None, grads, FAKE, need, None) == 1
    assert lib.mlstm_scan_bwd(scan_problem(z=rows()), *args[1:], need, None) == 1  # no dz
    grads.da = None
    assert lib.mlstm_scan_bwd(*args, need, None) == 1
    # a long sequence of few channels is cut into segments, and needs room for their states
    few = scan_problem(B=1, T=4096)
    need = lib.mlstm_scan_fwd_workspace_size(1, 4096, 64, 1, 16, B.BF16)
    assert need > 0 and lib.mlstm_scan_fwd(few, rows(), None, None, None, need, None) == 3
    assert lib.mlstm_scan_fwd(few, rows(), None, None, FAKE, need - 1, None) == 3
    assert lib.mlstm_scan_fwd(few, rows(), None, None, FAKE + 8, need, None) == 1
    assert lib.mlstm_scan_fwd_workspace_size(2, 5, 64, 1, 16, B.BF16) == 0
    # two saved states of 64 channels, 16 states each, for 5 (one group of eight) and 9 tokens
    assert lib.mlstm_scan_saved_size(2, 5, 64, 1, 16, B.BF16) == 2 * 1 * 64 * 16 * 4
    assert lib.mlstm_scan_saved_size(2, 9, 64, 1, 12, B.BF16) == 2 * 2 * 64 * 16 * 4


def norm_fwd(lib, x=rows(), w=None, bias=None, gate=None, y=rows(), stats=None, ws=None, nbytes=0, Bn=2,
             T=5, NH=4, d=16, scope=0, act=0, eps=1e-5, dtype=B.BF16):
    return lib.mlstm_group_norm_fwd(x, w, bias, gate, y, stats, ws, nbytes, Bn, T, NH, d, scope, act, eps,
                                    dtype, None)


@pytest.mark.parametrize("kw,status", [
    (dict(Bn=-1), 1), (dict(NH=0), 1), (dict(d=0), 1), (dict(scope=2), 1), (dict(act=3), 1),
    (dict(eps=0.0), 1), (dict(eps=float("nan")), 1), (dict(dtype=9), 1), (dict(d=513), 2),
    (dict(x=rows(None)), 1), (dict(y=rows(None)), 1), (dict(gate=rows(FAKE + 1)), 1),
    (dict(Bn=1 << 14, T=1 << 14, NH=1 << 6, d=1 << 8), 2), (dict(Bn=1 << 14, NH=1 << 14, d=1, scope=1), 2),
    (dict(w=FAKE + 1), 1), (dict(stats=FAKE + 4), 1),
    # a group too large for a cluster's shared memory needs a workspace
    (dict(d=4096, scope=1), 3), (dict(d=4096, scope=1, ws=FAKE, nbytes=4), 3),
    (dict(Bn=0), 0), (dict(T=0), 0),
])
def test_norm_argument_errors(lib, kw, status):
    assert norm_fwd(lib, **kw) == status


def test_norm_backward_argument_errors(lib):
    need = lib.mlstm_group_norm_workspace_size(2, 5, 4, 16, 0, B.BF16, 1)
    assert need > 0 and lib.mlstm_group_norm_workspace_size(2, 5, 4, 16, 0, B.BF16, 0) == 0

    def bwd(stats=FAKE, dx=rows(), gate=None, dgate=None, ws=FAKE, nbytes=need):
        return lib.mlstm_group_norm_bwd(rows(), None, None, gate, rows(), stats, dx, dgate, None, None, ws,
                                        nbytes, 2, 5, 4, 16, 0, 0, B.BF16, None)

    assert bwd(stats=None) == 1 and bwd(dx=rows(None)) == 1 and bwd(gate=rows()) == 1
    assert bwd(ws=None) == 3 and bwd(nbytes=need - 4) == 3 and bwd(ws=FAKE + 8) == 1
    # over a sequence: none in the forward where a cluster holds a group, else for what CTAs hand on
    assert lib.mlstm_group_norm_workspace_size(2, 5, 4, 16, 1, B.BF16, 0) == 0
    assert lib.mlstm_group_norm_workspace_size(2, 5, 4, 16, 1, B.BF16, 1) >= 2 * 2 * 4 * 16 * 4
    assert lib.mlstm_group_norm_workspace_size(2, 5, 4, 4096, 1, B.BF16, 0) > 0
    assert lib.mlstm_group_norm_stats_size(2, 5, 4, 16, 0) == 2 * 5 * 4 * 8
    assert lib.mlstm_group_norm_stats_size(2, 5, 4, 16, 1) == 2 * 4 * 8


def test_empty_problems_need_no_tensors(lib):
    none = B.Rows(None, 0, 0, 0)
    assert conv_fwd(lib, x=none, y=none, w=None, Bn=0) == 0
    assert conv_fwd(lib, x=none, y=none, w=None, T=0) == 0
    p = scan_problem(B=0, x=none, dt=none, b=none, c=none, a=None)
    assert lib.mlstm_scan_fwd(p, none, None, None, None, 0, None) == 0
    assert lib.mlstm_scan_step(p, none, None, None) == 0


# ---- the Python functions ----------------------------------------------------------------------

def test_python_functions_refuse_before_any_call():
    x = torch.zeros(2, 5, 8)
    w = torch.zeros(8, 4)
    with pytest.raises(ValueError, match="CUDA"):
        block.causal_conv_forward(x, w)
    with pytest.raises(ValueError, match="3 dimensions"):
        block.causal_conv_forward(x[0], w)
    with pytest.raises(ValueError, match="2 dimensions"):
        block.causal_conv_step(x, w, None, None)
    with pytest.raises(ValueError, match="CUDA"):
        block.selective_scan_forward(x, x, torch.zeros(8, 4), x[..., :4], x[..., :4])
    with pytest.raises(ValueError, match="state is required"):
        block.selective_scan_step(x[0], x[0], torch.zeros(8, 4), x[0, :, :4], x[0, :, :4], None)
    with pytest.raises(ValueError, match="do not divide"):
        block.group_norm_forward(x, groups=3)
    with pytest.raises(ValueError, match="3 dimensions"):
        block.group_norm_forward(x[0])
