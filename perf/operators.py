"""Cases and plain forms of the recurrent-block operators.

The operators stand around the gated linear recurrence of this package: the short causal
convolution before it, the selective state space scan beside it, and the group norm with an
activation or an output gate after it.  ``run`` computes one pass of a case, with elementary torch
operations in 32 bits, or, where ``own`` is true, with this package's calls.

Tensors are channels last, [B, T, NH * d], or head-major, [B, NH, T, d]; parameters are 32-bit.
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
DEVICE = "cuda"


def listed():
    return [
        # -- short causal convolution ------------------------------------------------------------
        # a prompt piece of one request that continues from the piece before it
        dict(name="conv_prompt_bf16", op="conv", mode="prompt", dtype="bf16", B=1, T=1000, NH=8,
             d=128, W=4, act="silu", bias=True, carried=True),
        # the layer before the cell at the headline training shape, into the head-major layout
        dict(name="conv_train_bf16", op="conv", mode="train", dtype="bf16", B=8, T=4096, NH=32,
             d=128, W=4, act="silu", bias=True, carried=False),
        # a ragged 32-bit training case: odd head dim (no wide accesses), three taps
        dict(name="conv_train_fp32_odd", op="conv", mode="train", dtype="fp32", B=2, T=577, NH=3,
             d=67, W=3, act="none", bias=True, carried=True),
        # one token of eight requests in generation
        dict(name="conv_step_bf16", op="conv", mode="step", dtype="bf16", B=8, T=1, NH=32, d=128,
             W=4, act="silu", bias=True, carried=True),
        # -- selective state space scan ----------------------------------------------------------
        # a training step of the scan as the mixer of the headline shape, with its output gate
        dict(name="scan_train_bf16", op="scan", mode="train", dtype="bf16", B=8, T=4096, NH=32,
             d=128, N=16, G=1, gate=True, carried=False),
        # a long prompt of one request: few rows, a long axis
        dict(name="scan_prompt_bf16", op="scan", mode="prompt", dtype="bf16", B=1, T=16384, NH=16,
             d=128, N=16, G=1, gate=True, carried=True),
        # a ragged 32-bit training case: odd channels, a state size that is no power of two, three
        # groups that share their B and C
        dict(name="scan_train_fp32_odd", op="scan", mode="train", dtype="fp32", B=2, T=577, NH=3,
             d=67, N=12, G=3, gate=False, carried=True),
        # one token of 64 requests in generation
        dict(name="scan_step_bf16", op="scan", mode="step", dtype="bf16", B=64, T=1, NH=32, d=128,
             N=16, G=1, gate=True, carried=True),
        # -- group norm with an activation or a gate ---------------------------------------------
        # the norm of every head's output and its output gate after the headline training cell
        dict(name="norm_train_bf16_token", op="norm", mode="train", dtype="bf16", B=8, T=4096,
             NH=32, d=128, scope="token", layout="heads", act="sigmoid", gate=True),
        # the same for one token of eight requests in generation
        dict(name="norm_step_bf16", op="norm", mode="step", dtype="bf16", B=8, T=1, NH=32, d=128,
             scope="token", layout="heads", act="sigmoid", gate=True),
        # group norm and SiLU of a channels-last map, statistics over all its positions
        dict(name="norm_train_bf16_sequence", op="norm", mode="train", dtype="bf16", B=4, T=8192,
             NH=16, d=256, scope="sequence", layout="last", act="silu", gate=False),
        # a ragged 32-bit map with odd groups
        dict(name="norm_train_fp32_odd", op="norm", mode="train", dtype="fp32", B=3, T=333, NH=5,
             d=67, scope="sequence", layout="last", act="silu", gate=False),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    """One more case: batches to 8 (64 for single tokens), lengths to 4096, up to 32 heads of up to
    128 channels, 2 to 4 taps, 1 to 32 states; every draw costs at most the largest listed case."""
    op = rng.choice(["conv", "scan", "norm"])
    mode = rng.choice(["train", "prompt", "step"] if op != "norm" else ["train", "train", "step"])
    c = dict(op=op, mode=mode, dtype=rng.choice(["bf16", "bf16", "fp32"]))
    c["B"] = _log_int(rng, 1, 64) if mode == "step" else rng.randint(1, 4)
    c["T"] = 1 if mode == "step" else _log_int(rng, 1, 4096)
    c["NH"] = _log_int(rng, 1, 32)
    c["d"] = rng.choice([64, 128, rng.randint(4 if op == "norm" else 1, 128)])
    if op == "conv":
        c.update(W=rng.randint(2, 4), act=rng.choice(["silu", "none"]), bias=rng.random() < 0.7,
                 carried=mode != "train" or rng.random() < 0.5)
    elif op == "scan":
        c.update(N=rng.choice([16, 16, rng.randint(1, 32)]), G=rng.choice([1, c["NH"]]),
                 gate=rng.random() < 0.5, carried=mode != "train" or rng.random() < 0.5)
    else:
        gate = rng.random() < 0.5
        c.update(scope="token" if mode == "step" else rng.choice(["token", "sequence"]),
                 layout=rng.choice(["heads", "last"]), gate=gate,
                 act=rng.choice(["silu", "sigmoid"] if gate else ["silu", "none"]))
    return c


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    B, T, NH, d = case["B"], case["T"], case["NH"], case["d"]
    D = NH * d
    full = B * T * D
    train = case["mode"] == "train"
    if case["op"] == "conv":
        W = case["W"]
        carried = B * (W - 1) * D * e
        wbytes = D * (W + case["bias"]) * 4
        nbytes = full * e * (4 if train else 2) + wbytes * (2 if train else 1)
        if case["carried"]:  # the state in, and the state (or, in training, its gradient too) out
            nbytes += carried * (4 if train else 2)
        flops = full * ((2 * W + 4) + (6 * W + 10 if train else 0))
    elif case["op"] == "scan":
        N, G = case["N"], case["G"]
        rows = 3 + case["gate"]  # x, dt, (z), y
        rows += (4 + case["gate"] - 1) if train else 0  # dy, dx, ddt, (dz)
        nbytes = full * e * rows + B * T * G * N * 2 * e * (2 if train else 1)
        nbytes += D * (N + 2) * 4 * (2 if train else 1)
        if case["carried"]:
            nbytes += B * D * N * 4 * (4 if train else 2)
        flops = full * N * (7 + (20 if train else 0))
    else:
        rows = 2 + case["gate"]  # x, (gate), y
        rows += (2 + case["gate"]) if train else 0  # dy, dx, (dgate)
        nbytes = full * e * rows + 2 * D * 4 * (2 if train else 1)
        flops = full * (10 + (20 if train else 0))
    return {"bytes": float(nbytes), "flops": float(flops)}


def prepare(case, seed):
    g = torch.Generator(device=DEVICE).manual_seed(int(seed))
    dt = DTYPES[case["dtype"]]
    B, T, NH, d = case["B"], case["T"], case["NH"], case["d"]
    D = NH * d

    def randn(*shape, scale=1.0, to=dt):
        return (torch.randn(*shape, generator=g, device=DEVICE) * scale).to(to)

    s = {"case": case}
    if case["op"] == "conv":
        W = case["W"]
        up = randn(B, T, 2 * D)  # an up-projection: the convolved half and the gate half
        s["x"] = up[:, 0, :D] if case["mode"] == "step" else up[..., :D]
        s["weight"] = (torch.rand(D, W, generator=g, device=DEVICE) * 2 - 1) / math.sqrt(W)
        s["bias"] = randn(D, scale=0.2, to=torch.float32) if case["bias"] else None
        s["state"] = randn(B, W - 1, D) if case["carried"] else None
        if case["mode"] == "train":
            s["dy"] = randn(B, NH, T, d)
            s["dstate_out"] = randn(B, W - 1, D) if case["carried"] else None
    elif case["op"] == "scan":
        N, G = case["N"], case["G"]
        xc = randn(B, T, D)
        s["x"] = torch.nn.functional.silu(xc.float()).to(dt)  # what the convolution hands over
        s["dt"] = randn(B, T, D, scale=0.5)
        # time steps log-uniform in [1e-3, 1e-1] before the token's own share
        u = torch.rand(D, generator=g, device=DEVICE) * math.log(100.0) + math.log(1e-3)
        s["dt_bias"] = torch.log(torch.expm1(torch.exp(u)))
        s["A"] = -(torch.arange(1, N + 1, device=DEVICE, dtype=torch.float32) *
                   torch.exp(randn(D, N, scale=0.2, to=torch.float32)))
        s["skip"] = 1.0 + randn(D, scale=0.1, to=torch.float32)
        bc = randn(B, T, 2 * G * N + 8)  # one projection holds B, C and eight more columns
        s["Bm"] = bc[..., :G * N].view(B, T, G, N)
        s["Cm"] = bc[..., G * N:2 * G * N].view(B, T, G, N)
        s["z"] = randn(B, T, 2 * D)[..., D:] if case["gate"] else None
        s["state"] = randn(B, D, N, scale=0.5, to=torch.float32) if case["carried"] else None
        if case["mode"] == "train":
            s["dy"] = randn(B, T, D)
            s["dstate_out"] = (randn(B, D, N, scale=0.5, to=torch.float32)
                               if case["carried"] else None)
        if case["mode"] == "step":
            for name in ("x", "dt", "Bm", "Cm", "z"):
                s[name] = s[name][:, 0] if s[name] is not None else None
    else:
        shape = (B, NH, T, d) if case["layout"] == "heads" else (B, T, D)
        scale = torch.exp(randn(B, *([NH, 1, 1] if case["layout"] == "heads" else [1, D]),
                                scale=0.3, to=torch.float32))
        x = torch.randn(*shape, generator=g, device=DEVICE) * scale + 0.1
        s["x"] = x.to(dt)
        s["weight"] = 1.0 + randn(D, scale=0.1, to=torch.float32)
        s["bias"] = randn(D, scale=0.1, to=torch.float32)
        s["gate"] = randn(B, T, D) if case["gate"] else None
        if case["mode"] == "train":
            s["dy"] = randn(B, T, D)
    return s


# ------------------------------------------------------------------------------------------------
# this package's calls
# ------------------------------------------------------------------------------------------------

def _run_own(s):
    from mlstm_chunkwise_attention_b200 import block
    c = s["case"]
    if c["op"] == "conv":
        act = {"silu": block.ACT_SILU, "none": block.ACT_NONE}[c["act"]]
        if c["mode"] == "step":
            state = s["state"].clone()
            y = block.causal_conv_step(s["x"], s["weight"], s["bias"], state, act=act)
            return {"y": y, "state": state}
        y, state = block.causal_conv_forward(s["x"], s["weight"], s["bias"], act=act,
                                             state_in=s["state"], want_state=c["carried"],
                                             heads=c["NH"])
        out = {"y": y, "state": state}
        if c["mode"] == "train":
            out.update(block.causal_conv_backward(s["x"], s["weight"], s["bias"], s["dy"], act=act,
                                                  state_in=s["state"], dstate_out=s["dstate_out"],
                                                  want_dstate=c["carried"]))
        return {k: v for k, v in out.items() if v is not None}
    if c["op"] == "scan":
        if c["mode"] == "step":
            state = s["state"].clone()
            y = block.selective_scan_step(s["x"], s["dt"], s["A"], s["Bm"], s["Cm"], state,
                                          skip=s["skip"], z=s["z"], dt_bias=s["dt_bias"])
            return {"y": y, "state": state}
        args = (s["x"], s["dt"], s["A"], s["Bm"], s["Cm"])
        kw = dict(skip=s["skip"], z=s["z"], dt_bias=s["dt_bias"], state_in=s["state"])
        y, saved, state = block.selective_scan_forward(*args, **kw, keep_saved=c["mode"] == "train",
                                                       want_state=c["carried"])
        out = {"y": y, "state": state}
        if c["mode"] == "train":
            out.update(block.selective_scan_backward(*args, s["dy"], saved, **kw,
                                                     dstate_out=s["dstate_out"],
                                                     want_dstate=c["carried"]))
        return {k: v for k, v in out.items() if v is not None}
    act = {"silu": block.ACT_SILU, "none": block.ACT_NONE, "sigmoid": block.ACT_SIGMOID}[c["act"]]
    scope = {"token": block.SCOPE_TOKEN, "sequence": block.SCOPE_SEQUENCE}[c["scope"]]
    kw = dict(gate=s["gate"], act=act, scope=scope, groups=c["NH"])
    y, stats = block.group_norm_forward(s["x"], s["weight"], s["bias"], **kw,
                                        keep_stats=c["mode"] == "train")
    out = {"y": y}
    if c["mode"] == "train":
        out.update(block.group_norm_backward(s["x"], s["weight"], s["bias"], s["dy"], stats, **kw))
    return {k: v for k, v in out.items() if v is not None}


# ------------------------------------------------------------------------------------------------
# plain forms
# ------------------------------------------------------------------------------------------------

def _sigmoid(v):
    return 1.0 / (1.0 + torch.exp(-v))


def _act(v, act):
    """The activation's value and its slope at v."""
    if act == "none":
        return v, torch.ones_like(v)
    sg = _sigmoid(v)
    if act == "sigmoid":
        return sg, sg * (1.0 - sg)
    return v * sg, sg * (1.0 + v * (1.0 - sg))


def _plain_conv(s):
    c = s["case"]
    io = DTYPES[c["dtype"]]
    B, T, NH, d, W = c["B"], c["T"], c["NH"], c["d"], c["W"]
    D = NH * d
    step = c["mode"] == "step"
    x = s["x"].float().view(B, T, D)
    w = s["weight"]
    before = s["state"].float() if s["state"] is not None else x.new_zeros(B, W - 1, D)
    seq = torch.cat([before, x], dim=1)  # token t of x is row t + W - 1
    pre = x.new_zeros(B, T, D) if s["bias"] is None else s["bias"].expand(B, T, D)
    for j in range(W):
        pre = pre + w[:, j] * seq[:, j:j + T]
    y, slope = _act(pre, c["act"])
    out = {"y": y.to(io).view(B, D) if step
           else y.view(B, T, NH, d).transpose(1, 2).contiguous().to(io)}
    if c["carried"]:
        out["state"] = seq[:, T:].to(io)
    if c["mode"] == "train":
        dp = s["dy"].float().transpose(1, 2).reshape(B, T, D) * slope
        dseq = torch.zeros_like(seq)
        dweight = torch.empty_like(w)
        for j in range(W):
            dseq[:, j:j + T] += w[:, j] * dp
            dweight[:, j] = (dp * seq[:, j:j + T]).sum((0, 1))
        if s["dstate_out"] is not None:
            dseq[:, T:] += s["dstate_out"].float()
        out["dx"] = dseq[:, W - 1:].to(io)
        out["dweight"] = dweight
        if s["bias"] is not None:
            out["dbias"] = dp.sum((0, 1))
        if c["carried"]:
            out["dstate_in"] = dseq[:, :W - 1].to(io)
    return out


def _plain_scan(s):
    c = s["case"]
    io = DTYPES[c["dtype"]]
    B, T, N, G = c["B"], c["T"], c["N"], c["G"]
    D = c["NH"] * c["d"]
    train, step = c["mode"] == "train", c["mode"] == "step"
    x = s["x"].float().view(B, T, G, D // G)
    raw = s["dt"].float().view(B, T, D) + s["dt_bias"]
    dt = torch.where(raw > 20.0, raw, torch.log1p(torch.exp(torch.minimum(raw, raw.new_tensor(20.0)))))
    dt = dt.view(B, T, G, D // G)
    A = s["A"].view(G, D // G, N)
    Bm = s["Bm"].float().view(B, T, G, 1, N)
    Cm = s["Cm"].float().view(B, T, G, 1, N)
    skip = s["skip"].view(G, D // G)
    h = s["state"].view(B, G, D // G, N) if s["state"] is not None else x.new_zeros(B, G, D // G, N)
    ys, hs = [], [h]
    for t in range(T):
        h = torch.exp(dt[:, t, ..., None] * A) * h + (dt[:, t] * x[:, t])[..., None] * Bm[:, t]
        ys.append((h * Cm[:, t]).sum(-1))
        if train:
            hs.append(h)
    y = torch.stack(ys, dim=1) + skip * x
    if s["z"] is not None:
        z = s["z"].float().view(B, T, G, D // G)
        zs, zslope = _act(z, "silu")
        o = y * zs
    else:
        o = y
    out = {"y": o.view(B, D).to(io) if step else o.view(B, T, D).to(io)}
    if c["carried"]:
        out["state"] = h.reshape(B, D, N).clone()
    if not train:
        return out
    dy = s["dy"].float().view(B, T, G, D // G)
    if s["z"] is not None:
        out["dz"] = (dy * y * zslope).view(B, T, D).to(io)
        dy = dy * zs
    gr = (s["dstate_out"].view(B, G, D // G, N).clone() if s["dstate_out"] is not None
          else x.new_zeros(B, G, D // G, N))
    dxs, ddts, dBs, dCs = [], [], [], []
    dA = x.new_zeros(G, D // G, N, dtype=torch.float64)
    for t in reversed(range(T)):
        gr = gr + dy[:, t, ..., None] * Cm[:, t]
        dCs.append((dy[:, t, ..., None] * hs[t + 1]).sum(2))
        a = torch.exp(dt[:, t, ..., None] * A)
        gah = gr * a * hs[t]
        gB = (gr * Bm[:, t]).sum(-1)
        dBs.append((gr * (dt[:, t] * x[:, t])[..., None]).sum(2))
        dA += (gah * dt[:, t, ..., None]).sum(0)
        ddts.append((gah * A).sum(-1) + gB * x[:, t])
        dxs.append(gB * dt[:, t])
        gr = gr * a
    ddt = torch.stack(ddts[::-1], dim=1).view(B, T, D) * _sigmoid(raw)
    out["dx"] = (torch.stack(dxs[::-1], dim=1) + skip * dy).view(B, T, D).to(io)
    out["ddt"] = ddt.to(io)
    out["dA"] = dA.view(D, N).float()
    out["dB"] = torch.stack(dBs[::-1], dim=1).to(io)
    out["dC"] = torch.stack(dCs[::-1], dim=1).to(io)
    out["dskip"] = (dy * x).sum((0, 1)).view(D)
    out["ddt_bias"] = ddt.sum((0, 1))
    if c["carried"]:
        out["dstate_in"] = gr.reshape(B, D, N)
    return out


def _plain_norm(s):
    c = s["case"]
    io = DTYPES[c["dtype"]]
    B, T, NH, d = c["B"], c["T"], c["NH"], c["d"]
    x = s["x"].float()
    x = x.transpose(1, 2) if c["layout"] == "heads" else x.view(B, T, NH, d)
    over = (3,) if c["scope"] == "token" else (1, 3)
    centred = x - x.mean(over, keepdim=True)
    rstd = 1.0 / torch.sqrt((centred * centred).mean(over, keepdim=True) + 1e-5)
    xhat = centred * rstd
    w, b = s["weight"].view(NH, d), s["bias"].view(NH, d)
    n = xhat * w + b
    if s["gate"] is not None:
        gt, gslope = _act(s["gate"].float().view(B, T, NH, d), c["act"])
        y = n * gt
    else:
        y, slope = _act(n, c["act"])
    out = {"y": y.reshape(B, T, NH * d).to(io)}
    if c["mode"] != "train":
        return out
    dy = s["dy"].float().view(B, T, NH, d)
    if s["gate"] is not None:
        out["dgate"] = (dy * n * gslope).reshape(B, T, NH * d).to(io)
        dn = dy * gt
    else:
        dn = dy * slope
    out["dweight"] = (dn * xhat).sum((0, 1)).view(-1)
    out["dbias"] = dn.sum((0, 1)).view(-1)
    dxh = dn * w
    dx = rstd * (dxh - dxh.mean(over, keepdim=True) - xhat * (dxh * xhat).mean(over, keepdim=True))
    out["dx"] = (dx.transpose(1, 2).contiguous().to(io) if c["layout"] == "heads"
                 else dx.reshape(B, T, NH * d).to(io))
    return out


def run(state):
    if own:
        return _run_own(state)
    return {"conv": _plain_conv, "scan": _plain_scan, "norm": _plain_norm}[state["case"]["op"]](state)


# ------------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ------------------------------------------------------------------------------------------------

def _grads64(value, leaves, cotangents):
    """Derivatives of sum over outputs of <cotangent, output> with respect to the leaves."""
    total = sum((o * w).sum() for o, w in zip(value, cotangents) if w is not None)
    return torch.autograd.grad(total, leaves)


def _exact_conv(case, s):
    B, T, NH, d, W = case["B"], case["T"], case["NH"], case["d"], case["W"]
    D = NH * d
    train = case["mode"] == "train"
    leaf = lambda v: v.double().clone().requires_grad_(train)
    outs = {}
    acc = None
    rows = []
    for b in range(B):  # one sequence at a time bounds the memory
        x = leaf(s["x"][b].reshape(T, D))
        w = leaf(s["weight"])
        bias = leaf(s["bias"]) if s["bias"] is not None else None
        st = leaf(s["state"][b]) if s["state"] is not None else None
        head = st if st is not None else torch.zeros(W - 1, D, dtype=torch.float64, device=x.device)
        seq = torch.cat([head, x])
        pre = (seq.unfold(0, W, 1) * w).sum(-1)  # [T, D]: the window ending at each token
        if bias is not None:
            pre = pre + bias
        y = pre * torch.sigmoid(pre) if case["act"] == "silu" else pre
        last = seq[T:]
        row = {"y": (y.reshape(D) if case["mode"] == "step"
                     else y.view(T, NH, d).permute(1, 0, 2)).detach()}
        if case["carried"]:
            row["state"] = last.detach()
        if train:
            dy = s["dy"][b].double().permute(1, 0, 2).reshape(T, D)
            dlast = s["dstate_out"][b].double() if s["dstate_out"] is not None else None
            leaves = [x, w] + ([bias] if bias is not None else []) + ([st] if st is not None else [])
            got = list(_grads64([y, last], leaves, [dy, dlast]))
            row["dx"] = got.pop(0)
            params = {"dweight": got.pop(0)}
            if bias is not None:
                params["dbias"] = got.pop(0)
            if st is not None:
                row["dstate_in"] = got.pop(0)
            acc = params if acc is None else {k: acc[k] + params[k] for k in acc}
        rows.append(row)
    for k in rows[0]:
        outs[k] = torch.stack([r[k] for r in rows])
    outs.update(acc or {})
    return outs


def _exact_scan(case, s):
    B, T, N, G = case["B"], case["T"], case["N"], case["G"]
    D = case["NH"] * case["d"]
    train = case["mode"] == "train"
    per = D // G
    A = s["A"].double()
    x = s["x"].double().reshape(B, T, D)
    raw = s["dt"].double().reshape(B, T, D) + s["dt_bias"].double()
    dt = torch.logaddexp(raw, torch.zeros_like(raw))
    Bm, Cm = s["Bm"].reshape(B, T, G, N), s["Cm"].reshape(B, T, G, N)
    widen = lambda m, t: m[:, t].double().repeat_interleave(per, 1)  # [B, D, N] of token t
    h = (s["state"].double() if s["state"] is not None
         else torch.zeros(B, D, N, dtype=torch.float64, device=x.device))
    trail = [h]
    y = torch.empty_like(x)
    for t in range(T):
        decay = torch.exp(torch.einsum("bd,dn->bdn", dt[:, t], A))
        h = torch.addcmul((dt[:, t] * x[:, t]).unsqueeze(2) * widen(Bm, t), decay, h)
        y[:, t] = torch.einsum("bdn,bdn->bd", h, widen(Cm, t))
        if train:
            trail.append(h)
    y = torch.addcmul(y, x, s["skip"].double().expand_as(x))
    outs = {"y": y}
    if s["z"] is not None:
        z = s["z"].double().reshape(B, T, D)
        sg = torch.sigmoid(z)
        outs["y"] = y * z * sg
    if case["mode"] == "step":
        outs["y"] = outs["y"].reshape(B, D)
    if case["carried"]:
        outs["state"] = h
    if not train:
        return outs
    dy = s["dy"].double()
    if s["z"] is not None:
        outs["dz"] = dy * y * (sg + z * sg * (1 - sg))
        dy = dy * z * sg
    gr = (s["dstate_out"].double() if s["dstate_out"] is not None
          else torch.zeros(B, D, N, dtype=torch.float64, device=x.device))
    dx, ddt = torch.empty_like(x), torch.empty_like(x)
    dB = torch.empty(B, T, G, N, dtype=torch.float64, device=x.device)
    dC = torch.empty_like(dB)
    dA = torch.zeros_like(A)
    for t in range(T - 1, -1, -1):
        gr = torch.addcmul(gr, dy[:, t].unsqueeze(2), widen(Cm, t))
        dC[:, t] = (dy[:, t].unsqueeze(2) * trail.pop()).view(B, G, per, N).sum(2)
        dB[:, t] = ((dt[:, t] * x[:, t]).unsqueeze(2) * gr).view(B, G, per, N).sum(2)
        back = gr * torch.exp(torch.einsum("bd,dn->bdn", dt[:, t], A))
        through = back * trail[-1]  # the gradient with respect to dt A
        gB = torch.einsum("bdn,bdn->bd", gr, widen(Bm, t))
        dx[:, t] = gB * dt[:, t]
        ddt[:, t] = gB * x[:, t] + torch.einsum("bdn,dn->bd", through, A)
        dA += torch.einsum("bdn,bd->dn", through, dt[:, t])
        gr = back
    ddt = ddt * torch.sigmoid(raw)
    outs.update(dx=torch.addcmul(dx, dy, s["skip"].double().expand_as(dy)), ddt=ddt, dA=dA, dB=dB,
                dC=dC, dskip=(dy * x).sum((0, 1)), ddt_bias=ddt.sum((0, 1)))
    if case["carried"]:
        outs["dstate_in"] = gr
    return outs


def _exact_norm(case, s):
    B, T, NH, d = case["B"], case["T"], case["NH"], case["d"]
    train = case["mode"] == "train"
    heads = case["layout"] == "heads"
    leaf = lambda v: v.double().clone().requires_grad_(train)
    rows, acc = [], None
    for b in range(B):
        x = leaf(s["x"][b])
        w, bias = leaf(s["weight"]), leaf(s["bias"])
        gate = leaf(s["gate"][b]) if s["gate"] is not None else None
        xg = x.permute(1, 0, 2) if heads else x.reshape(T, NH, d)
        if case["scope"] == "token":
            var, mean = torch.var_mean(xg, dim=2, unbiased=False, keepdim=True)
        else:
            var, mean = torch.var_mean(xg, dim=(0, 2), unbiased=False, keepdim=True)
        n = ((xg - mean) / torch.sqrt(var + 1e-5)).reshape(T, NH * d) * w + bias
        fn = {"none": lambda v: v, "silu": torch.nn.functional.silu, "sigmoid": torch.sigmoid}[case["act"]]
        y = n * fn(gate) if gate is not None else fn(n)
        row = {"y": y.detach()}
        if train:
            leaves = [x, w, bias] + ([gate] if gate is not None else [])
            got = list(_grads64([y], leaves, [s["dy"][b].double()]))
            row["dx"] = got[0]
            params = {"dweight": got[1], "dbias": got[2]}
            if gate is not None:
                row["dgate"] = got[3]
            acc = params if acc is None else {k: acc[k] + params[k] for k in acc}
        rows.append(row)
    outs = {k: torch.stack([r[k] for r in rows]) for k in rows[0]}
    outs.update(acc or {})
    return outs


def exact(case, seed):
    """What ``run`` returns, laid out the same, from the definitions in 64 bits."""
    s = prepare(case, seed)
    return {"conv": _exact_conv, "scan": _exact_scan, "norm": _exact_norm}[case["op"]](case, s)
