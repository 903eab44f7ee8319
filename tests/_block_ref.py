"""Plain 64-bit forms of the operators around the recurrence, with every gradient written out,
and the bound the kernels are held to.

Each form returns, beside its outputs, a magnitude for every output element: the same sums over
the absolute values of their terms (``mag``).  An output computed in fp32 as a sum of terms is off by
at most K 2^-24 mag, where K counts the roundings a term goes through, plus half a step of the I/O
dtype (``close`` below).  Exponentials and sigmoids of the kernels are good to a few 2^-22, so each
counts as 8 roundings; an exponent v adds |v| roundings, which the magnitudes carry.
"""

import torch

HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def close(got, ref, mag, K, what):
    """|got - ref| <= half a step of got's dtype + K roundings of the magnitude."""
    dtype = got.dtype
    got = got.detach().double().cpu()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert torch.isfinite(got).all(), f"{what}: non-finite values"
    # the rounding to the I/O dtype acts on the computed value, so its step is that of ref + error
    err = K * 2.0 ** -24 * mag
    bound = HALF_STEP[dtype] * (ref.abs() + err) + err + 1e-37
    over = (got - ref).abs() - bound
    worst = int(over.argmax())
    assert over.max() <= 0, (f"{what}: off by {float((got - ref).abs().flatten()[worst]):.3e} where "
                             f"{float(bound.flatten()[worst]):.3e} is allowed "
                             f"(value {float(ref.flatten()[worst]):.3e})")


def act64(v, act):
    """value, slope, and magnitudes of both."""
    if act == "none":
        one = torch.ones_like(v)
        return v, one, v.abs(), one
    s = torch.sigmoid(v)
    grow = 1.0 + v.abs()  # an exponential's relative error grows with its argument
    if act == "sigmoid":
        return s, s * (1 - s), s * grow, s * grow
    return v * s, s * (1 + v * (1 - s)), v.abs() * s * grow, s * grow * (1 + v.abs())


def conv64(x, w, bias, state, act, dy=None, dstate_out=None):
    """x [B, T, D], w [D, W], state [B, W - 1, D] or None, all fp64; dict name -> (value, mag)."""
    B, T, D = x.shape
    W = w.shape[1]
    st = state if state is not None else x.new_zeros(B, W - 1, D)
    seq = torch.cat([st, x], 1)
    pre = sum(w[:, j] * seq[:, j:j + T] for j in range(W))
    mag = sum((w[:, j] * seq[:, j:j + T]).abs() for j in range(W))
    if bias is not None:
        pre, mag = pre + bias, mag + bias.abs()
    y, slope, ymag, smag = act64(pre, act)
    # an error of the argument reaches y through a slope of at most 1.1
    out = {"y": (y, ymag + 1.1 * mag), "state": (seq[:, T:], seq[:, T:].abs())}
    if dy is not None:
        dp, dpm = dy * slope, dy.abs() * (smag + 0.5 * mag if act == "silu" else smag)
        dseq, dm = torch.zeros_like(seq), torch.zeros_like(seq)
        dw, dwm = torch.zeros_like(w), torch.zeros_like(w)
        for j in range(W):
            dseq[:, j:j + T] += w[:, j] * dp
            dm[:, j:j + T] += w[:, j].abs() * dpm
            dw[:, j] = (dp * seq[:, j:j + T]).sum((0, 1))
            dwm[:, j] = (dpm * seq[:, j:j + T].abs()).sum((0, 1))
        if dstate_out is not None:
            dseq[:, T:] += dstate_out
            dm[:, T:] += dstate_out.abs()
        out.update(dx=(dseq[:, W - 1:], dm[:, W - 1:]), dstate_in=(dseq[:, :W - 1], dm[:, :W - 1]),
                   dweight=(dw, dwm), dbias=(dp.sum((0, 1)), dpm.sum((0, 1))))
    return out


def scan64(x, dt, A, Bm, Cm, skip=None, z=None, dt_bias=None, softplus=True, state=None, dy=None,
           dstate_out=None):
    """x, dt, z [B, T, D]; A [D, N]; Bm, Cm [B, T, G, N]; dict name -> (value, mag)."""
    B, T, D = x.shape
    N, G = A.shape[1], Bm.shape[2]
    P = D // G
    raw = dt if dt_bias is None else dt + dt_bias
    rawm = dt.abs() if dt_bias is None else dt.abs() + dt_bias.abs()
    if softplus:
        delta = torch.logaddexp(raw, torch.zeros_like(raw))
        # relative errors of the exponential (its argument's size) and of the logarithm
        deltam = delta * (1 + rawm)
        dslope = torch.sigmoid(raw)
    else:
        delta, deltam, dslope = raw, rawm, torch.ones_like(raw)
    wide = lambda m, t: m[:, t].repeat_interleave(P, 1)  # [B, D, N]
    s = state if state is not None else x.new_zeros(B, D, N)
    sa = sm = s.abs()
    trail, sizes, mags, ys, ym = [s], [sa], [sm], [], []
    for t in range(T):
        e = torch.exp(delta[:, t, :, None] * A)
        # To first order an error of the state decays as the state does, and each step adds its own
        # roundings and the decay's: deltam |A| of its exponent, on a state of at most sa.
        s = e * s + (delta[:, t] * x[:, t])[..., None] * wide(Bm, t)
        sm = (e * (sm + (1 + deltam[:, t, :, None] * A.abs()) * sa)
              + (deltam[:, t] * x[:, t].abs())[..., None] * wide(Bm, t).abs())
        sa = e * sa + ((delta[:, t] * x[:, t])[..., None] * wide(Bm, t)).abs()
        trail.append(s)
        sizes.append(sa)
        mags.append(sm)
        ys.append((s * wide(Cm, t)).sum(-1))
        ym.append((sm * wide(Cm, t).abs()).sum(-1))
    y, ym = torch.stack(ys, 1) if T else x.clone(), torch.stack(ym, 1) if T else x.abs()
    if skip is not None:
        y, ym = y + skip * x, ym + (skip * x).abs()
    out = {"state": (s, sm)}
    if z is not None:
        zs, zsl, zm, zslm = act64(z, "silu")
        out["y"] = (y * zs, ym * zm.clamp_min(0) + y.abs() * zm)
    else:
        out["y"] = (y, ym)
    if dy is None:
        return out
    dym = dy.abs()
    if z is not None:
        out["dz"] = (dy * y * zsl, dy.abs() * (ym + y.abs()) * zslm)
        dy, dym = dy * zs, dy.abs() * zm
    g = dstate_out if dstate_out is not None else x.new_zeros(B, D, N)
    ga = gm = g.abs()
    dx, ddt, dB, dC = (torch.zeros_like(v) for v in (x, x, Bm, Cm))
    dxm, ddtm, dBm, dCm = (torch.zeros_like(v) for v in (x, x, Bm, Cm))
    dA, dAm = torch.zeros_like(A), torch.zeros_like(A)
    for t in range(T - 1, -1, -1):
        g = g + dy[:, t, :, None] * wide(Cm, t)
        gm = gm + dym[:, t, :, None] * wide(Cm, t).abs()
        ga = ga + dy[:, t, :, None].abs() * wide(Cm, t).abs()
        dC[:, t] = (dy[:, t, :, None] * trail[t + 1]).view(B, G, P, N).sum(2)
        dCm[:, t] = (dym[:, t, :, None] * mags[t + 1]).view(B, G, P, N).sum(2)
        dB[:, t] = ((delta[:, t] * x[:, t])[..., None] * g).view(B, G, P, N).sum(2)
        dBm[:, t] = ((deltam[:, t] * x[:, t].abs())[..., None] * gm).view(B, G, P, N).sum(2)
        e = torch.exp(delta[:, t, :, None] * A)
        power = 1 + deltam[:, t, :, None] * A.abs()
        u, um = g * e * trail[t], e * (gm * sizes[t] + ga * mags[t] + power * ga * sizes[t])
        gB, gBm = (g * wide(Bm, t)).sum(-1), (gm * wide(Bm, t).abs()).sum(-1)
        dA += (u * delta[:, t, :, None]).sum(0)
        dAm += (um * deltam[:, t, :, None]).sum(0)
        dx[:, t] = gB * delta[:, t]
        dxm[:, t] = gBm * deltam[:, t]
        ddt[:, t] = gB * x[:, t] + (u * A).sum(-1)
        ddtm[:, t] = gBm * x[:, t].abs() + (um * A.abs()).sum(-1)
        g, gm, ga = g * e, e * (gm + power * ga), e * ga
    if skip is not None:
        dx, dxm = dx + skip * dy, dxm + (skip * dy).abs() + skip.abs() * dym
    ddt, ddtm = ddt * dslope, ddtm * dslope * (1 + rawm)
    out.update(dx=(dx, dxm), ddt=(ddt, ddtm), dA=(dA, dAm), dB=(dB, dBm), dC=(dC, dCm),
               dskip=((dy * x).sum((0, 1)), (dym * x.abs()).sum((0, 1))),
               ddt_bias=(ddt.sum((0, 1)), ddtm.sum((0, 1))), dstate_in=(g, gm))
    return out


def norm64(x, w, b, gate, act, scope, eps, dy=None):
    """x [B, T, NH, d]; w, b [NH, d]; gate, dy [B, T, NH, d]; dict name -> (value, mag)."""
    over = (3,) if scope == "token" else (1, 3)
    mean = x.mean(over, keepdim=True)
    var = ((x - mean) ** 2).mean(over, keepdim=True)
    rstd = 1 / torch.sqrt(var + eps)
    xh = (x - mean) * rstd
    # the subtraction of the mean loses roundings of |x| and of the mean's own terms
    xm = xh.abs() + rstd * (x.abs() + x.abs().mean(over, keepdim=True))
    n, nm = xh * w + b, xm * w.abs() + b.abs()
    out = {}
    if gate is not None:
        gt, gsl, gtm, gslm = act64(gate, act)
        out["y"] = (n * gt, nm * gtm)
    else:
        y, slope, ymag, smag = act64(n, act)
        out["y"] = (y, ymag + 1.1 * nm)
    if dy is None:
        return out
    if gate is not None:
        out["dgate"] = (dy * n * gsl, dy.abs() * nm * gslm)
        dn, dnm = dy * gt, dy.abs() * gtm
    else:
        dn, dnm = dy * slope, dy.abs() * (smag + (0.5 * nm if act != "none" else 0))
    out["dweight"] = ((dn * xh).sum((0, 1)), (dnm * xm).sum((0, 1)))
    out["dbias"] = (dn.sum((0, 1)), dnm.sum((0, 1)))
    g, gm = dn * w, dnm * w.abs()
    out["dx"] = (rstd * (g - g.mean(over, keepdim=True) - xh * (g * xh).mean(over, keepdim=True)),
                 rstd * (gm + gm.mean(over, keepdim=True) + xm * (gm * xm).mean(over, keepdim=True)))
    return out
