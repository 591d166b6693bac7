"""Error bounds of the calls around the scan, worked out element by element in
fp64 from the inputs (never from a kernel's output).

u = 2^-24 is half a step of fp32.  Counted per operation, relative to its
result: an fp32 add, multiply or fma u; the hardware's exp2, rcp and sqrt one
step, 2u.  First order in u throughout; every bound is doubled once for the
terms of second order and for the reference's own rounding, and an fp32
denormal step is allowed on top.  An output is rounded once more, by half a
step of its type.
"""
from __future__ import annotations

import torch

F64 = torch.float64
U = 2.0 ** -24
TINY = 1e-37          # below this fp32 has no full precision


def _f64(t):
    return None if t is None else t.detach().cpu().to(F64)


def rounded(ref, err, dtype):
    """The allowance of an output of `dtype` whose fp32 value is off by `err`."""
    half = torch.finfo(dtype).eps / 2
    return 2 * err + half * (ref.abs() + 2 * err) + TINY


def check(got, ref, err, what):
    g = got.detach().cpu()
    tol = rounded(ref, err, g.dtype)
    d = (g.to(F64) - ref).abs()
    bad = ~(d <= tol)
    assert g.shape == ref.shape, (what, g.shape, ref.shape)
    if bad.any():
        at = tuple(int(i[0]) for i in bad.nonzero(as_tuple=True)) if g.dim() else ()
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {at}: "
                             f"{float(g[at])} for {float(ref[at])}, allowed {float(tol[at]):.3g}")


def _gates(ga, gx, A, ba, bx):
    """r, i, la, a, w in fp64, the relative errors of each in fp32, 1 - r and 1 - i."""
    za = ga + (ba if ba is not None else 0.0)
    zx = gx + (bx if bx is not None else 0.0)

    def sigma(gate, bias):
        # e = exp2(-gate log2e - bias log2e): the bias's product, the fused
        # sum and the constant's own rounding shift the exponent by
        # u (|bias| + |z| + |gate| + |bias|), at most u (2|z| + 3|bias|);
        # exp2 2u; 1 + e: u; rcp: 2u.  The error of e counts by its share of
        # 1 + e, at most 1.
        z = gate + bias
        return torch.sigmoid(z), (2 * z.abs() + 3 * bias.abs() + 2 + 1 + 2) * U

    zero = torch.zeros(1, dtype=F64)
    r, er = sigma(ga, ba if ba is not None else zero)
    i, ei = sigma(gx, bx if bx is not None else zero)
    la = A * r
    ela = er + 3 * U                               # A log2e, its constant, times r
    a = torch.exp(la)
    ea = la.abs() * ela + 2 * U                    # exp2
    w = torch.sqrt(-torch.expm1(2 * la))
    # -2 l a s(l^2) for l above -1/2 (-0.72 ln 2): l's error moves 1 - e^{2l}
    # by at most its own relative size; the rounding of a 2u (exp2), of s 3u
    # (three fma of falling weight, the constants, what is left out), of two
    # products 2u.  1 - a a below, at least 0.63: 2 a^2 ea + u over 0.63.  The
    # root halves, and adds 2u.
    ew = 0.5 * torch.where(la > -0.5, ela + 7 * U, (2 * a * a * ea + U) / 0.63) + 2 * U
    return r, i, la, a, w, er, ei, ela, ea, ew, torch.sigmoid(-za), torch.sigmoid(-zx)


def gated(x, gate_a, gate_x, A, bias_a=None, bias_x=None, h0=None, seq_lens=None):
    """err of y [B, L, D] and of the last state, and what the backward's bound needs."""
    x, ga, gx, A, ba, bx, h0 = (_f64(t) for t in (x, gate_a, gate_x, A, bias_a, bias_x, h0))
    B, L, D = x.shape
    r, i, la, a, w, er, ei, ela, ea, ew, c_r, c_i = _gates(ga, gx, A, ba, bx)
    b = (w * i * x).abs()
    eb = ew + ei + 2 * U
    h = h0 if h0 is not None else torch.zeros(B, D, dtype=F64)
    size, err = h.abs(), torch.zeros(B, D, dtype=F64)
    sizes, errs, before, before_err = [], [], [], []
    lens = None if seq_lens is None else seq_lens.cpu().to(torch.int64).clamp(0, L)
    for t in range(L):
        before.append(size)
        before_err.append(err)
        # size: the recurrence over magnitudes, at least every partial sum a
        # fold may form.  A token costs the error of its decay and of its
        # input, and a rounding each of a product of decays, of the fold and
        # of the run; the folds of groups and tiles add one for every 4.
        n_size = a[:, t] * size + b[:, t]
        n_err = a[:, t] * err + a[:, t] * size * (ea[:, t] + 3 * U) + b[:, t] * eb[:, t] + 3 * U * n_size
        if lens is not None:
            there = (t < lens)[:, None]
            n_size, n_err = torch.where(there, n_size, size), torch.where(there, n_err, err)
        size, err = n_size, n_err
        sizes.append(size)
        errs.append(err)
    stack = lambda v: torch.stack(v, 1) if L else torch.zeros(B, 0, D, dtype=F64)  # noqa: E731
    keep = dict(x=x, r=r, i=i, la=la, a=a, w=w, er=er, ei=ei, ela=ela, ea=ea, ew=ew, A=A, c_r=c_r, c_i=c_i,
                before=stack(before), before_err=stack(before_err), lens=lens)
    return stack(errs), err, keep


def gated_bwd(keep, dy, dh_last=None):
    """err of every gradient: {name: bound}."""
    k = keep
    x, r, i, la, a, w = (k[n] for n in ("x", "r", "i", "la", "a", "w"))
    B, L, D = x.shape
    dy = _f64(dy).abs()
    lens = k["lens"]
    there = torch.ones(B, L, 1, dtype=torch.bool)
    if lens is not None:
        there = torch.arange(L)[None, :, None] < lens[:, None, None]
        dy = torch.where(there, dy, torch.zeros_like(dy))
    q = _f64(dh_last).abs() if dh_last is not None else torch.zeros(B, D, dtype=F64)
    qe = torch.zeros(B, D, dtype=F64)
    G, Ge = torch.empty(B, L, D, dtype=F64), torch.empty(B, L, D, dtype=F64)
    for t in range(L - 1, -1, -1):
        G[:, t] = dy[:, t] + q
        Ge[:, t] = qe + 3 * U * G[:, t]
        n_q = a[:, t] * G[:, t]
        n_e = a[:, t] * Ge[:, t] + n_q * (k["ea"][:, t] + 3 * U)
        q = torch.where(there[:, t], n_q, q)
        qe = torch.where(there[:, t], n_e, qe)
    zero = torch.zeros_like(G)
    G, Ge = torch.where(there, G, zero), torch.where(there, Ge, zero)
    ix = i * x.abs()
    eix = k["ei"] + U
    first = la.abs() * a * k["before"]
    first_err = first * (k["ela"] + k["ea"] + 3 * U) + la.abs() * a * k["before_err"]
    law = torch.where(w > 0, la.abs() / w, zero)
    second = law * a * a * ix
    # formed as la a (h - a i x / w): the root's reciprocal (2u beside half the
    # error of w^2, which ew holds), the products, and the sum's rounding
    second_err = second * (k["ela"] + k["ew"] + 2 * k["ea"] + eix + 9 * U) + U * (first + second)
    E = G * (first + second)
    Ee = Ge * (first + second) + G * (first_err + second_err) + 2 * U * E
    c_r, c_i = k["c_r"], k["c_i"]
    ga, gx = E * c_r, G * w * ix * c_i
    # 1 - sigma = e sigma: relative errors of both, added
    # w = w^2 / w: one rounding more than the forward's root
    out = {"dx": (G * w * i, Ge * w * i + G * w * i * (k["ew"] + k["ei"] + 3 * U)),
           "dgate_a": (ga, Ee * c_r + ga * (2 * k["er"] + 2 * U)),
           "dgate_x": (gx, Ge * w * ix * c_i + gx * (k["ew"] + eix + 2 * k["ei"] + 4 * U))}
    # a sum of n terms: every term passes at most 16 (a run) + 2 (lanes) + 8
    # (wavefronts) + rows / 16 + 16 additions
    rows = B * -(-L // 128)
    depth = 42 + rows / 16
    res = {n: e for n, (_, e) in out.items()}
    add = lambda m, e: (e + depth * U * m).sum((0, 1))     # noqa: E731
    res["dbias_a"] = add(*out["dgate_a"])
    res["dbias_x"] = add(*out["dgate_x"])
    res["dA"] = add(E, Ee) / k["A"].abs() + U * E.sum((0, 1)) / k["A"].abs()
    res["dh0"] = qe
    return res


def _depth(D):
    # additions a term passes in a row's sum: a thread's share (32 elements, or
    # D / 1024 of a long row), six levels of lanes, sixteen wavefronts, and the
    # product with 1 / D
    return max(32, D / 1024 + 1) + 6 + 16 + 2


def norm(x, weight=None, bias=None, residual=None, eps=1e-5):
    """errs of y, mean, rstd, s, and what the backward's bound needs."""
    x, w, b, res = (_f64(t) for t in (x, weight, bias, residual))
    s = x if res is None else x + res
    es = U * s.abs() if res is not None else torch.zeros_like(s)
    D = s.shape[-1]
    k = _depth(D)
    mean = s.mean(-1, keepdim=True)
    em = es.mean(-1, keepdim=True) + k * U * s.abs().mean(-1, keepdim=True)
    c = s - mean
    ec = es + em + U * c.abs()
    var = (c * c).mean(-1, keepdim=True)
    ev = (2 * c.abs() * ec + ec * ec).mean(-1, keepdim=True) + k * U * var
    rstd = 1 / torch.sqrt(var + eps)
    er = 0.5 * (ev + U * (var + eps)) / (var + eps) + 3 * U            # relative: root and quotient
    n = c * rstd
    en = ec * rstd + n.abs() * (er + U)
    wa = w.abs() if w is not None else torch.ones(D, dtype=F64)
    y = n * (w if w is not None else 1.0) + (b if b is not None else 0.0)
    ey = wa * en + U * (y.abs() + wa * n.abs())
    return dict(y=ey, mean=em[..., 0], rstd=(er * rstd)[..., 0], s=es), \
        dict(n=n, en=en, rstd=rstd, er=er, w=wa, D=D)


def norm_bwd(keep, dy, dresidual_out=None, groups=256):
    n, en, rstd, er, w, D = (keep[k] for k in ("n", "en", "rstd", "er", "w", "D"))
    dy = _f64(dy)
    v = (dy * w).abs()
    na = n.abs()
    k = _depth(D)
    c1 = (v * na).mean(-1, keepdim=True)
    e1 = (v * en).mean(-1, keepdim=True) + (k + 2) * U * c1
    c2 = v.mean(-1, keepdim=True)
    e2 = (k + 1) * U * c2
    inner = v + c2 + na * c1
    ei = U * v + e2 + en * c1 + na * e1 + 3 * U * inner
    g = rstd * inner
    eg = rstd * ei + g * (er + U)
    if dresidual_out is not None:
        eg = eg + U * (g + _f64(dresidual_out).abs())
    flat = lambda t: t.reshape(-1, D)                        # noqa: E731
    rows = flat(dy).shape[0]
    # a term of a parameter's gradient: its workgroup's rows one after the
    # other, three joins of lanes, 16 of wavefronts, then the workgroups by
    # sixteens
    depth = -(-rows // max(1, min(groups, rows))) + 3 + 16 + groups / 16 + 16 + 1
    d = flat(dy).abs()
    return dict(dx=eg, dweight=(d * flat(en) + (depth + 1) * U * d * flat(na)).sum(0),
                dbias=(depth * U * d).sum(0))


def conv_bwd(x, weight, du, bias=None, state=None, silu=True, dstate_out=None):
    x, w, du, b, st, ds_out = (_f64(t) for t in (x, weight, du, bias, state, dstate_out))
    B, L, D = x.shape
    K = w.shape[1]
    full = torch.zeros(B, L + K - 1, D, dtype=F64)
    full[:, K - 1:] = x
    if st is not None:
        full[:, :K - 1] = st.transpose(1, 2)
    s = sum(w[:, k] * full[:, k:k + L] for k in range(K))
    size = sum((w[:, k] * full[:, k:k + L]).abs() for k in range(K))
    if b is not None:
        s, size = s + b, size + b.abs()
    es = (K + 1) * U * size
    if silu:
        sg, cs = torch.sigmoid(s), torch.sigmoid(-s)
        d = sg * (1 + s * cs)
        # sigma: relative (3|s| + 5) u; its value and 1 - sigma each carry
        # it; |d'| of the derivative is at most 1/2 + |s|/4 sigma (1 - sigma) < 0.6
        esg = (3 * s.abs() + 5) * U
        ed = 0.6 * es + sg * (esg + 3 * U) * (1 + s.abs() * cs) + sg * s.abs() * cs * (2 * esg + 2 * U)
        g, eg = (du * d).abs(), du.abs() * (ed + U * d.abs())
    else:
        g, eg = du.abs(), torch.zeros_like(du)
    dfull, efull = torch.zeros_like(full), torch.zeros_like(full)
    for k in range(K):
        dfull[:, k:k + L] += g * w[:, k].abs()
        efull[:, k:k + L] += eg * w[:, k].abs()
    efull += (K + 1) * U * dfull
    if ds_out is not None:
        efull[:, L:] += U * (dfull[:, L:] + ds_out.transpose(1, 2).abs())
    # a sum's term: a run of tokens, the workgroup's wavefronts, then the
    # cells by sixteens
    depth = 256 + 16 + (B * -(-L // 256)) / 16 + 16
    dw = torch.zeros(D, K, dtype=F64)
    for k in range(K):
        f = full[:, k:k + L].abs()
        dw[:, k] = (eg * f + (depth + 1) * U * g * f).sum((0, 1))
    return dict(dx=efull[:, K - 1:], dstate=efull[:, :K - 1].transpose(1, 2), dweight=dw,
                dbias=(eg + depth * U * g).sum((0, 1)))
