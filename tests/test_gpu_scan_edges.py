"""The selective scan where its numbers leave the ordinary range: decays of 0, infinite inputs, states that
grow or shrink by more than fp32's range within a segment, and cut forms at full width."""

import pytest
import torch

from mlstm_chunkwise_attention_b200 import binding, block
from _block_ref import close, scan64

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
INF = float("inf")


def inputs(B, T, D, N, G=1, dtype=F32, seed=0):
    """x, dt, A, B, C of a call, on the host."""
    g = torch.Generator().manual_seed(seed + T + D)
    r = lambda *s: torch.randn(*s, generator=g)
    return [r(B, T, D).to(dtype), (0.5 * r(B, T, D)).to(dtype), -torch.exp(r(D, N)),
            r(B, T, G, N).to(dtype), r(B, T, G, N).to(dtype)]


def both_ways(x, dt, A, Bm, Cm, **kw):
    y, saved, end = block.selective_scan_forward(x, dt, A, Bm, Cm, want_state=True, **kw)
    got = block.selective_scan_backward(x, dt, A, Bm, Cm, x, saved, want_dstate=True, **kw)
    binding.check_device()
    return {"y": y, "end": end, **{k: v for k, v in got.items() if v is not None}}


# ---- a decay of 0 ----------------------------------------------------------------------------------

# B, T, D, N, G: less than a tile, whole tiles, several segments at once, and segments in turn
CLOSED = [(1, 20, 16, 16, 1), (1, 32, 16, 16, 1), (2, 9, 24, 5, 2), (1, 300, 24, 16, 1), (5, 530, 256, 4, 256)]


@pytest.mark.parametrize("size", CLOSED, ids=["b%dt%dd%dn%dg%d" % s for s in CLOSED])
@pytest.mark.parametrize("rate", [-INF, -3e38], ids=["inf", "overflows_in_base_two"])
def test_an_infinite_rate_is_a_decay_of_zero(size, rate):
    """A = -inf, and a finite A whose product with log2 e is not: what A = -1e30 gives, whose decays are 0
    as well, for every step above 1e-28 (all of these are)."""
    t = [v.cuda() for v in inputs(*size)]
    res = []
    for v in (rate, -1e30):
        A = t[2].clone()
        A[:, size[3] // 2] = v
        res.append(both_ways(t[0], t[1], A, *t[3:]))
    for k in res[0]:
        assert torch.isfinite(res[0][k]).all(), k
        assert torch.equal(res[0][k], res[1][k]), k


def test_an_infinite_rate_in_steps_is_that_of_a_prompt():
    B, T, D, N = 2, 5, 24, 12
    x, dt, A, Bm, Cm = (v.cuda() for v in inputs(B, T, D, N))
    A[:, 3] = -INF
    dt[:, 2] = -200.0  # softplus underflows: a step of exactly 0, which leaves the states
    y, _, end = block.selective_scan_forward(x, dt, A, Bm, Cm, want_state=True)
    st = torch.zeros(B, D, N, device="cuda")
    steps = [block.selective_scan_step(x[:, i], dt[:, i], A, Bm[:, i], Cm[:, i], st) for i in range(T)]
    binding.check_device()
    ref = inputs(B, T, D, N)
    ref[2][:, 3] = -1e30
    ref[1][:, 2] = -200.0
    want = scan64(*(v.double() for v in ref))
    # delta of the third token is 1e-87 in 64 bits and 0 in fp32: times -1e30 no decay in either
    for got in (y, torch.stack(steps, 1)):
        close(got, *want["y"], 64 + T + N, "y")
    for got in (end, st):
        close(got, *want["state"], 64 + T + N, "state")


# ---- infinite inputs -------------------------------------------------------------------------------

def close_where_finite(got, ref, mag, K, what):
    """Infinities and NaN where the 64-bit form has them, the usual bound elsewhere."""
    g = got.double().cpu()
    assert torch.equal(g.isnan(), ref.isnan()), what
    wild = ~torch.isfinite(ref)
    assert torch.equal(g[wild].nan_to_num(0.0, INF, -INF), ref[wild].nan_to_num(0.0, INF, -INF)), what
    assert torch.isfinite(mag[~wild]).all(), what
    close(got.cpu()[~wild], ref[~wild], mag[~wild], K, what)


@pytest.mark.parametrize("where", ["x", "dt"])
@pytest.mark.parametrize("gate", [False, True], ids=["ungated", "gated"])
@pytest.mark.parametrize("size", [(1, 40, 16, 1, 1), (2, 40, 24, 5, 2), (1, 70, 16, 12, 1), (1, 40, 16, 16, 1),
                                  (1, 300, 24, 12, 1), (5, 530, 256, 3, 256)],
                         ids=lambda s: "b%dt%dd%dn%dg%d" % s)
def test_an_infinite_input_stays_infinite(size, gate, where):
    """x or the step infinite at one token, no skip: B and C of one sign, so the formula has infinities and
    no NaN in y and the state, in the prompt and in steps, whatever N is padded to."""
    B, T, D, N, G = size
    x, dt, A, Bm, Cm = inputs(*size)
    Bm, Cm = Bm.abs() + 0.1, Cm.abs() + 0.1
    x = x.abs() + 0.1
    (x if where == "x" else dt)[0, 10, 3] = INF
    z = torch.randn(B, T, D, generator=torch.Generator().manual_seed(1)) + 3.0 if gate else None
    t = [v.cuda() for v in (x, dt, A, Bm, Cm)]
    zd = None if z is None else z.cuda()
    y, _, end = block.selective_scan_forward(*t, z=zd, want_state=True)
    st = torch.zeros(B, D, N, device="cuda")
    steps = [block.selective_scan_step(t[0][:, i], t[1][:, i], t[2], t[3][:, i], t[4][:, i], st,
                                       z=None if z is None else zd[:, i]) for i in range(min(T, 60))]
    binding.check_device()
    ref = scan64(*(v.double() for v in (x, dt, A, Bm, Cm)), z=None if z is None else z.double())
    assert ref["y"][0].isinf().any() and not ref["y"][0].isnan().any()
    K = 64 + T + N
    close_where_finite(y, *ref["y"], K, "y")
    close_where_finite(end, *ref["state"], K, "state")
    n = len(steps)
    close_where_finite(torch.stack(steps, 1), *(v[:, :n] for v in ref["y"]), K, "steps")


@pytest.mark.parametrize("gate", [False, True], ids=["ungated", "gated"])
def test_an_infinite_input_without_skip_leaves_its_dx_finite(gate):
    """dx and dz of the token whose x is infinite: no skip, so nothing is added to dx (0 times dy) and y in
    dz is the infinite sum over states alone."""
    B, T, D, N = 1, 40, 16, 16
    x, dt, A, Bm, Cm = inputs(B, T, D, N)
    Bm, Cm = Bm.abs() + 0.1, Cm.abs() + 0.1
    x = x.abs() + 0.1
    x[0, 10, 3] = INF
    g = torch.Generator().manual_seed(2)
    dy = torch.rand(B, T, D, generator=g) + 0.1
    dy[0, 5, 7] = INF  # another channel's
    z = torch.rand(B, T, D, generator=g) + 0.5 if gate else None
    t = [v.cuda() for v in (x, dt, A, Bm, Cm)]
    zd = None if z is None else z.cuda()
    _, saved, _ = block.selective_scan_forward(*t, z=zd)
    got = block.selective_scan_backward(*t, dy.cuda(), saved, z=zd)
    binding.check_device()
    ref = scan64(*(v.double() for v in (x, dt, A, Bm, Cm)), z=None if z is None else z.double(),
                 dy=dy.double())
    for name in ("dx", "dz") if gate else ("dx",):
        assert not ref[name][0].isnan().any() and ref[name][0].isinf().any()
        close_where_finite(got[name], *ref[name], 2 * (64 + T + N), name)


@pytest.mark.parametrize("gate", [False, True], ids=["ungated", "gated"])
@pytest.mark.parametrize("size", [(1, 40, 16, 5, 1), (2, 40, 24, 12, 1), (1, 300, 24, 12, 1), (1, 40, 16, 16, 1)],
                         ids=lambda s: "b%dt%dd%dn%dg%d" % s)
def test_an_infinite_step_hands_nothing_back(size, gate):
    """An infinite step forgets the state (its decay is 0), so the tokens before it have the gradients of the
    sequence that ends there, however N is padded."""
    B, T, D, N, G = size
    at = T - 15
    x, dt, A, Bm, Cm = inputs(*size)
    dt[:, at] = INF
    g = torch.Generator().manual_seed(4)
    dy = torch.randn(B, T, D, generator=g)
    z = torch.randn(B, T, D, generator=g) if gate else None
    t = [v.cuda() for v in (x, dt, A, Bm, Cm)]
    zd = None if z is None else z.cuda()
    _, saved, _ = block.selective_scan_forward(*t, z=zd)
    got = block.selective_scan_backward(*t, dy.cuda(), saved, z=zd)
    binding.check_device()
    cut = lambda v: v[:, :at].double()
    ref = scan64(cut(x), cut(dt), A.double(), cut(Bm), cut(Cm), z=None if z is None else cut(z), dy=cut(dy))
    for name in ("dx", "ddt", "dz", "dB", "dC"):
        if got[name] is not None:
            r = [v.reshape(got[name][:, :at].shape) for v in ref[name]]
            close(got[name][:, :at].contiguous(), *r, 2 * (64 + T + N) + D // G, name)


# ---- decays beyond fp32's range --------------------------------------------------------------------

@pytest.mark.parametrize("log2_decay,state", [(4.1, 2.0 ** -66), (-4.1, 2.0 ** 60)], ids=["grows", "shrinks"])
@pytest.mark.parametrize("backwards", [False, True], ids=["state", "gradient"])
def test_a_segments_decay_beyond_the_range_of_fp32(log2_decay, state, backwards):
    """32 tokens, a segment where a short scan is cut at once, multiply a state by 2^131 or 2^-131 (or 16, a
    segment of the backward, from the other end the state's gradient): more than one fp32 number holds,
    but the state starts and ends inside its range."""
    T, D, N, on = 128, 8, 8, 16 if backwards else 32
    lib = binding.load()
    assert lib.mlstm_scan_fwd_workspace_size(1, T, D, 1, N, binding.FP32) > 0, "cut into segments"
    x = torch.zeros(1, T, D)
    A = torch.full((D, N), 1.0 if log2_decay > 0 else -1.0)
    one = torch.ones(1, T, 1, N)
    dt = torch.zeros(1, T, D)
    (dt[:, T - on:] if backwards else dt[:, :on]).fill_(abs(log2_decay) * 32 / on * 0.6931472)
    given = torch.full((1, D, N), state)
    t = [v.cuda() for v in (x, dt, A, one[:, :, 0], one[:, :, 0])]
    kw = dict(softplus=False, state_in=None if backwards else given.cuda())
    y, saved, end = block.selective_scan_forward(*t, **kw, want_state=True)
    got = block.selective_scan_backward(*t, torch.zeros_like(y), saved, **kw, want_dstate=True,
                                        dstate_out=given.cuda() if backwards else None)
    binding.check_device()
    ref = scan64(*(v.double() for v in (x, dt, A, one, one)), softplus=False,
                 state=None if backwards else given.double(), dy=torch.zeros(1, T, D, dtype=torch.float64),
                 dstate_out=given.double() if backwards else None)
    K = 64 + T + N
    if backwards:
        close(got["dstate_in"], *ref["dstate_in"], 2 * K, "dstate_in")
    else:
        close(end, *ref["state"], K, "state")
        close(y, *ref["y"], K, "y")


# ---- the cut forms and the wide accesses -----------------------------------------------------------

def test_segments_in_turn_at_full_width():
    """16-byte accesses, many live channels to a tile, B and C shared by all tiles: the training form, long
    enough for segments in turn in both directions (1280 tiles forward, 640 backward; two segments, the last
    one ragged).  The 64-bit form runs on the GPU."""
    B, T, D, N, G = 10, 530, 4096, 16, 1
    lib = binding.load()
    # in turn: the handed state [B, D, 16] and the counters; at once would hold two segments' states
    assert lib.mlstm_scan_fwd_workspace_size(B, T, D, G, N, binding.BF16) == B * D * 16 * 4 + 5376  # 1282 words
    g = torch.Generator("cuda").manual_seed(5)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")
    x, dt, z, dy = r(B, T, D).to(BF), (0.5 * r(B, T, D)).to(BF), r(B, T, D).to(BF), r(B, T, D).to(BF)
    A, Bm, Cm = -torch.exp(r(D, N)), r(B, T, G, N).to(BF), r(B, T, G, N).to(BF)
    skip, bias, st, dso = r(D), r(D) - 2.0, r(B, D, N), r(B, D, N)
    kw = dict(skip=skip, z=z, dt_bias=bias, state_in=st)
    y, saved, end = block.selective_scan_forward(x, dt, A, Bm, Cm, **kw, want_state=True)
    got = block.selective_scan_backward(x, dt, A, Bm, Cm, dy, saved, **kw, dstate_out=dso, want_dstate=True)
    binding.check_device()
    d = torch.Tensor.double
    ref = scan64(d(x), d(dt), d(A), d(Bm), d(Cm), d(skip), d(z), d(bias), True, d(st), d(dy), d(dso))
    ref = {k: (v.cpu(), m.cpu()) for k, (v, m) in ref.items()}
    K = 64 + T + N
    close(y, *ref["y"], K, "y")
    close(end, *ref["state"], K, "state")
    for name in ("dx", "ddt", "dstate_in", "dz"):
        close(got[name], *ref[name], 2 * K, name)
    for name in ("dB", "dC"):
        close(got[name], *ref[name], 2 * K + D // G, name)
    for name in ("dA", "dskip", "ddt_bias"):
        close(got[name], *ref[name], 2 * K + B * T, name)


# B, T, D, N, G, gate, dtype: more than 16 states with 16-byte accesses, whole and padded
MANY = [(2, 100, 128, 32, 1, True, BF), (2, 100, 128, 64, 2, True, BF), (1, 300, 64, 24, 1, False, BF),
        (1, 333, 64, 40, 1, True, BF), (2, 70, 64, 64, 1, True, F32), (1, 400, 96, 48, 2, False, F32)]


@pytest.mark.parametrize("case", MANY, ids=["b%dt%dd%dn%dg%d" % c[:5] for c in MANY])
def test_many_states_with_wide_accesses(case):
    B, T, D, N, G, gate, dtype = case
    x, dt, A, Bm, Cm = inputs(B, T, D, N, G, dtype)
    g = torch.Generator().manual_seed(6)
    r = lambda *s: torch.randn(*s, generator=g)
    dy, z, skip, bias = r(B, T, D).to(dtype), r(B, T, D).to(dtype) if gate else None, r(D), r(D) - 2.0
    st, dso = r(B, D, N), r(B, D, N)
    cuda = lambda v: None if v is None else v.cuda()
    t = [v.cuda() for v in (x, dt, A, Bm, Cm)]
    kw = dict(skip=cuda(skip), z=cuda(z), dt_bias=cuda(bias), state_in=cuda(st))
    y, saved, end = block.selective_scan_forward(*t, **kw, want_state=True)
    got = block.selective_scan_backward(*t, dy.cuda(), saved, **kw, dstate_out=dso.cuda(), want_dstate=True)
    binding.check_device()
    d = lambda v: None if v is None else v.double()
    ref = scan64(d(x), d(dt), d(A), d(Bm), d(Cm), d(skip), d(z), d(bias), True, d(st), d(dy), d(dso))
    K = 64 + T + N
    close(y, *ref["y"], K, "y")
    close(end, *ref["state"], K, "state")
    for name in ("dx", "ddt", "dstate_in", "dz"):
        if got[name] is not None:
            close(got[name], *ref[name], 2 * K, name)
    for name in ("dB", "dC"):
        close(got[name], *ref[name], 2 * K + D // G, name)
    for name in ("dA", "dskip", "ddt_bias"):
        close(got[name], *ref[name], 2 * K + B * T, name)


def test_an_infinite_state_crosses_segments():
    """A decay of 2^-43 a token leaves an infinite state infinite in every token, so in every segment too,
    although a segment's decay is far below fp32's smallest number."""
    B, T, D, N = 1, 300, 24, 16
    x, dt, _, Bm, Cm = inputs(B, T, D, N)
    x, Bm, Cm = x.abs() + 0.1, Bm.abs() + 0.1, Cm.abs() + 0.1
    x[0, 3, 5] = INF
    A, dt = torch.full((D, N), -30.0), torch.ones(B, T, D)
    y, _, end = block.selective_scan_forward(*(v.cuda() for v in (x, dt, A, Bm, Cm)), softplus=False,
                                             want_state=True)
    binding.check_device()
    ref = scan64(*(v.double() for v in (x, dt, A, Bm, Cm)), softplus=False)
    assert ref["y"][0][0, 3:, 5].isinf().all() and ref["y"][0].isinf().sum() == T - 3
    close_where_finite(y, *ref["y"], 64 + T + N, "y")
    close_where_finite(end, *ref["state"], 64 + T + N, "state")


def test_backward_offsets_beyond_32_bits():
    """The backward of a scan over more than 2^31 elements: its last tokens have the gradients of a call that
    starts there (with the state there), in other segments: to two bf16 steps of the largest."""
    T, T0, D = 280000, 279900, 8192
    g = torch.Generator("cuda").manual_seed(1)
    x = torch.empty(1, T, D, dtype=BF, device="cuda").normal_(generator=g)
    assert x.numel() > 2 ** 31
    A, one = -torch.ones(D, 1, device="cuda"), torch.ones(1, T, 1, dtype=BF, device="cuda")
    _, saved, _ = block.selective_scan_forward(x, x, A, one, one)
    got = block.selective_scan_backward(x, x, A, one, one, x, saved)
    got = {k: got[k][:, T0:].float() for k in ("dx", "ddt", "dB", "dC")}
    del saved
    # a step of softplus(x) on average forgets e^-0.8 a token: 400 tokens before T0 decide the state there
    lead, tail = slice(T0 - 400, T0), slice(T0, T)
    _, _, st = block.selective_scan_forward(x[:, lead], x[:, lead], A, one[:, lead], one[:, lead],
                                            keep_saved=False, want_state=True)
    args = (x[:, tail], x[:, tail], A, one[:, tail], one[:, tail])
    _, saved, _ = block.selective_scan_forward(*args, state_in=st)
    want = block.selective_scan_backward(*args, x[:, tail], saved, state_in=st)
    binding.check_device()
    for k in got:
        w = want[k].float()
        assert float((got[k] - w).abs().max()) <= 2.0 ** -7 * float(w.abs().max()), k
