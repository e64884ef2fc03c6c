"""The layer's gradients in 64 bits, from the formulas, with the error that a
computation in 32 bits may add (for the tolerances of the training tests).

Tolerances are bounds, element by element, derived from the operations:
  * a product summed over K terms in fp32, in any order, with every addition
    rounded or cut: at most K * 2^-23 * sum |a_k b_k|;
  * a value stored in a type: half a step, eps / 2 of it (bf16 2^-8, fp32
    2^-24), relative to the value;
  * the logistic function and the few multiplications around it: the fast
    exponential is within 2 + 1.2 |z| units of 2^-23, so below 2^-18 of the
    value for |z| <= 20; larger |z| leave sig or 1 - sig below 3e-9;
  * errors of factors go through a product as |x| err(y) + |y| err(x), and
    through silu with |silu'| <= 1.1, |silu''| <= 0.5.
Each bound is widened by 1 % for the products of two errors.
"""
import torch

U = 2.0 ** -23
FAST = 2.0 ** -18
MORE = 1.01


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def random(g, *shape, dtype=torch.float32, scale=1.0):
    return (torch.randn(*shape, generator=g) * scale).to(dtype)


def offsets_of(sizes):
    return torch.tensor([0] + list(torch.tensor(sizes).cumsum(0)), dtype=torch.int32)


def segments(offsets):
    o = offsets.tolist()
    return [(e, o[e], o[e + 1]) for e in range(len(o) - 1)]


def mm(a, b, ea=None, eb=None):
    """a @ b and the error of computing it in 32 bits from operands that are
    off by at most ea and eb."""
    err = a.shape[1] * U * (a.abs() @ b.abs())
    if ea is not None:
        err = err + ea @ b.abs()
    if eb is not None:
        err = err + a.abs() @ eb
    return a @ b, err


def check(got, ref, err, dtype, what):
    """got (stored in dtype) within the arithmetic's error and half a step."""
    got = got.double().cpu()
    tol = MORE * err + half_step(dtype) * (ref.abs() + MORE * err) + 1e-38
    bad = ~((got - ref).abs() <= tol)
    assert got.shape == ref.shape, what
    assert not bad.any(), (
        f"{what}: {int(bad.sum())} of {bad.numel()} outside; worst "
        f"{float(((got - ref).abs() / tol).nan_to_num(nan=float('inf')).max()):.3g} x the bound")


def ffn_backward(x, offsets, wg, wu, wd, dy, dtype):
    """(value, error) pairs of dx, dw_gate, dw_up, dw_down; h, da and du are
    rounded to `dtype` as the library documents."""
    x, wg, wu, wd, dy = (t.double() for t in (x, wg, wu, wd, dy))
    hs = half_step(dtype)
    dx, edx = torch.zeros_like(x), torch.zeros_like(x)
    grads = [torch.zeros_like(w) for w in (wg, wu, wd)]
    errs = [torch.zeros_like(w) for w in (wg, wu, wd)]
    for e, lo, hi in segments(offsets):
        if lo == hi:
            continue
        xe, dye = x[lo:hi], dy[lo:hi]
        a, ea = mm(xe, wg[e].T)
        u, eu = mm(xe, wu[e].T)
        dh, edh = mm(dye, wd[e])
        sig = torch.sigmoid(a)
        silu = a * sig
        slope = sig * (1 + a * (1 - sig))
        h, da, du = silu * u, dh * u * slope, dh * silu
        eh = 1.1 * u.abs() * ea + silu.abs() * eu + FAST * h.abs()
        eda = (1.1 * (u.abs() * edh + dh.abs() * eu) + 0.5 * (dh * u).abs() * ea
               + FAST * 1.1 * (dh * u).abs())
        edu = silu.abs() * edh + 1.1 * dh.abs() * ea + FAST * du.abs()
        eh, eda, edu = (MORE * er + hs * (v.abs() + er) for v, er in
                        ((h, eh), (da, eda), (du, edu)))
        p, ep = mm(da, wg[e], ea=eda)
        q, eq = mm(du, wu[e], ea=edu)
        dx[lo:hi], edx[lo:hi] = p + q, ep + eq + U * (p.abs() + q.abs())
        for n, (l, r, el, er) in enumerate(((da, xe, eda, None), (du, xe, edu, None),
                                            (dye, h, None, eh))):
            grads[n][e], errs[n][e] = mm(l.T, r, None if el is None else el.T, er)
    return [(dx, edx)] + list(zip(grads, errs))


def combine_backward(dout, x, y, idx, gate, slot_row, n_routed, scale):
    """(value, error) of dy_perm (zeros where no slot points) and dgate."""
    T, k = idx.shape
    dout, x, y, gate = dout.double(), x.double(), y.double(), gate.double()
    rows = slot_row.view(T, k).long()
    dy = torch.zeros_like(y)
    dgate, err = torch.zeros(T, k).double(), torch.zeros(T, k).double()
    for t in range(T):
        for j in range(k):
            if idx[t, j] < n_routed:
                r = rows[t, j]
                dy[r] = scale * gate[t, j] * dout[t]
                dgate[t, j] = scale * (dout[t] @ y[r])
                err[t, j] = (x.shape[1] + 2) * U * abs(scale) * (dout[t].abs() @ y[r].abs())
            else:
                dgate[t, j] = dout[t] @ x[t]
                err[t, j] = (x.shape[1] + 2) * U * (dout[t].abs() @ x[t].abs())
    return (dy, 2 * U * dy.abs()), (dgate, err)


def input_backward(dout, x, w_router, idx, gate, slot_row, dgate, dx_perm, n_routed,
                   edgate=None, edx_perm=None):
    """(value, error) of dx and dw_router."""
    T, k = idx.shape
    dout, x, w, gate = dout.double(), x.double(), w_router.double(), gate.double()
    dgate, dxp = dgate.double(), dx_perm.double()
    edgate = torch.zeros_like(dgate) if edgate is None else edgate
    edxp = torch.zeros_like(dxp) if edx_perm is None else edx_perm
    mean = (gate * dgate).sum(1, keepdim=True)
    emean = ((gate * edgate).sum(1, keepdim=True)
             + (k + 2) * U * (gate * dgate).abs().sum(1, keepdim=True))
    dl = gate * (dgate - mean)
    edl = gate * (edgate + emean) + 3 * U * gate * (dgate.abs() + mean.abs())
    rows = slot_row.view(T, k).long()
    routed = idx < n_routed
    through = torch.where(routed[:, :, None], dxp[rows.clamp(min=0)], 0.0)
    ethrough = torch.where(routed[:, :, None], edxp[rows.clamp(min=0)], 0.0).sum(1)
    same = (torch.where(routed, 0.0, gate).sum(1, keepdim=True)) * dout
    we = w[idx.long()]
    dx = through.sum(1) + same + torch.einsum("tj,tjd->td", dl, we)
    size = through.abs().sum(1) + same.abs() + torch.einsum("tj,tjd->td", dl.abs(), we.abs())
    edx = ethrough + (2 * k + 4) * U * size + torch.einsum("tj,tjd->td", edl, we.abs())
    dense = torch.zeros(T, w.shape[0]).double().scatter(1, idx.long(), dl)
    edense = torch.zeros(T, w.shape[0]).double().scatter(1, idx.long(), edl)
    dw, edw = mm(dense.T, x, ea=edense.T)
    return (dx, edx), (dw, edw)


def route_by_hand(T, n_routed, n_zero, k, g, popular=None):
    """Random expert ids and gates, and the dispatch of them (rows ordered by
    expert, then token) -> idx, gate, slot_row, offsets."""
    E = n_routed + n_zero
    score = torch.randn(T, E, generator=g)
    if popular is not None:
        score[:, popular] += 100.0
    idx = torch.topk(score, k, dim=1).indices.int()
    gate = torch.softmax(torch.randn(T, k, generator=g), 1)
    slot_row = torch.full((T * k,), -1, dtype=torch.int32)
    flat = idx.reshape(-1)
    r, off = 0, [0]
    for e in range(n_routed):
        for s in torch.nonzero(flat == e).flatten().tolist():
            slot_row[s] = r
            r += 1
        off.append(r)
    return idx, gate, slot_row, torch.tensor(off, dtype=torch.int32)
