"""The operators in a row as a state space block runs them: one convolution over x, B and C together, the
scan on slices of its output, a norm gated by z; values, gradients, and a prompt followed by single
tokens.  Each stage is held to its 64-bit form on the inputs that it got from the stage before."""

import pytest
import torch

from mlstm_chunkwise_attention_b200 import binding, block
from _block_ref import close, conv64, norm64, scan64

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def block_inputs(B, T, D, N, G, dtype):
    g = torch.Generator().manual_seed(D + T)
    r = lambda *s: torch.randn(*s, generator=g)
    W = D + 2 * G * N
    # one projection holds z, the convolution's channels and dt: all are read as slices
    c = dict(proj=r(B, T, D + W + D).to(dtype), w=0.5 * r(W, 4), cb=0.1 * r(W), A=-torch.exp(r(D, N)),
             skip=r(D), bias=r(D) - 2.0, nw=1 + 0.1 * r(D), nb=0.1 * r(D), dy=r(B, T, D).to(dtype))
    return {k: v.cuda() for k, v in c.items()}


def split(p, D, N, G):
    W = D + 2 * G * N
    return p[..., :D], p[..., D:D + W], p[..., D + W:]


def parts(u, D, N, G):
    """x, B, C of the convolution's output, as strided views."""
    per = (*u.shape[:-1], G, N)
    return u[..., :D], u[..., D:D + G * N].view(per), u[..., D + G * N:].view(per)


@pytest.mark.parametrize("B,T,D,N,G,dtype", [(2, 150, 128, 16, 1, F32), (2, 75, 136, 12, 2, BF),
                                             (1, 300, 64, 64, 1, BF), (1, 33, 15, 5, 3, F32)])
def test_block_values_and_gradients(B, T, D, N, G, dtype):
    c = block_inputs(B, T, D, N, G, dtype)
    z, xbc, dt = split(c["proj"], D, N, G)
    u, _ = block.causal_conv_forward(xbc, c["w"], c["cb"])
    x, Bm, Cm = parts(u, D, N, G)
    kw = dict(skip=c["skip"], dt_bias=c["bias"])
    h, saved, _ = block.selective_scan_forward(x, dt, c["A"], Bm, Cm, **kw)
    nk = dict(gate=z, act=block.ACT_SILU, groups=G)
    y, stats = block.group_norm_forward(h, c["nw"], c["nb"], **nk)
    gn = block.group_norm_backward(h, c["nw"], c["nb"], c["dy"], stats, **nk)
    gs = block.selective_scan_backward(x, dt, c["A"], Bm, Cm, gn["dx"], saved, **kw)
    du = torch.cat([gs["dx"], gs["dB"].reshape(B, T, G * N), gs["dC"].reshape(B, T, G * N)], -1)
    gx = block.causal_conv_backward(xbc, c["w"], c["cb"], du)
    binding.check_device()
    d = lambda v: v.double().cpu()
    ref = conv64(d(xbc), d(c["w"]), d(c["cb"]), None, "silu", d(du))
    close(u, *ref["y"], 64, "u")
    close(gx["dx"], *ref["dx"], 64, "d(xBC)")
    close(gx["dweight"], *ref["dweight"], 64 + B * T, "dweight")
    close(gx["dbias"], *ref["dbias"], 64 + B * T, "dbias")
    ref = scan64(d(x), d(dt), d(c["A"]), d(Bm), d(Cm), d(c["skip"]), None, d(c["bias"]), dy=d(gn["dx"]))
    K = 64 + T + N
    close(h, *ref["y"], K, "h")
    for name in ("dx", "ddt"):
        close(gs[name], *ref[name], 2 * K, name)
    for name in ("dB", "dC"):
        close(gs[name], *ref[name], 2 * K + D // G, name)
    for name in ("dA", "dskip", "ddt_bias"):
        close(gs[name], *ref[name], 2 * K + B * T, name)
    per = lambda v: d(v).view(B, T, G, D // G)
    ref = norm64(per(h), d(c["nw"]).view(G, -1), d(c["nb"]).view(G, -1), per(z), "silu", "token", 1e-5,
                 per(c["dy"]))
    K = 64 + D // G
    for got, name, k in ((y, "y", K), (gn["dx"], "dx", 2 * K), (gn["dgate"], "dgate", K)):
        close(got, *(v.reshape(B, T, D) for v in ref[name]), k, "norm " + name)
    for name in ("dweight", "dbias"):
        close(gn[name], *(v.flatten() for v in ref[name]), K + B * T, "norm " + name)


@pytest.mark.parametrize("D,N,G,dtype", [(128, 16, 1, BF), (15, 5, 3, F32)])
def test_block_prompt_then_tokens(D, N, G, dtype):
    """A prompt, then single tokens through the carried states.  The convolution has the bits of one call over
    all tokens; the scan and the norm are held to 64 bits of what it gave."""
    B, T, T0 = 2, 60, 41
    c = block_inputs(B, T, D, N, G, dtype)
    z, xbc, dt = split(c["proj"], D, N, G)
    kw = dict(skip=c["skip"], dt_bias=c["bias"])
    nk = dict(act=block.ACT_SILU, groups=G)
    whole, _ = block.causal_conv_forward(xbc, c["w"], c["cb"])
    u, cst = block.causal_conv_forward(xbc[:, :T0], c["w"], c["cb"], want_state=True)
    x, Bm, Cm = parts(u, D, N, G)
    h, _, st = block.selective_scan_forward(x, dt[:, :T0], c["A"], Bm, Cm, **kw, keep_saved=False, want_state=True)
    us, hs = [u], [h]
    ys = [block.group_norm_forward(h, c["nw"], c["nb"], gate=z[:, :T0], **nk)[0]]
    for t in range(T0, T):
        u = block.causal_conv_step(xbc[:, t], c["w"], c["cb"], cst)
        x, Bm, Cm = parts(u, D, N, G)
        h = block.selective_scan_step(x, dt[:, t], c["A"], Bm, Cm, st, **kw)
        us.append(u[:, None])
        hs.append(h[:, None])
        ys.append(block.group_norm_forward(h[:, None], c["nw"], c["nb"], gate=z[:, t:t + 1], **nk)[0])
    binding.check_device()
    u, h, y = (torch.cat(v, 1) for v in (us, hs, ys))
    assert torch.equal(u, whole)
    d = lambda v: v.double().cpu()
    x, Bm, Cm = parts(u, D, N, G)
    ref = scan64(d(x), d(dt), d(c["A"]), d(Bm), d(Cm), d(c["skip"]), None, d(c["bias"]))
    close(h, *ref["y"], 64 + T + N, "h")
    close(st, *ref["state"], 64 + T + N, "state")
    per = lambda v: d(v).view(B, T, G, D // G)
    ref = norm64(per(h), d(c["nw"]).view(G, -1), d(c["nb"]).view(G, -1), per(z), "silu", "token", 1e-5)
    close(y, *(v.reshape(B, T, D) for v in ref["y"]), 64 + D // G, "y")
