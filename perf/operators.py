"""Operators of the MoE layer's training pass, as measured cases.

Five operators, each in its plain form (elementary torch operations in 32 bits,
rounded once at the end) and as the framework's call:

* ``grouped``: matrix products grouped by expert over ragged row segments, in
  their three directions: ``fwd`` y[r] = W_e x[r], ``dx`` dx[r] = W_e^T dy[r],
  ``dw`` dW_e = sum over e's rows of dy[r] x[r]^T;
* ``ffn_backward``: gradients of the routed SwiGLU experts, recomputing the
  pre-activations from the dispatched rows;
* ``combine_backward``: gradients of the gate-weighted combine with respect to
  the expert outputs and the gates;
* ``input_backward``: gradients of the layer input (through the experts, the
  zero experts and the router) and of the router weights;
* ``adamw``: one AdamW step over many tensors, with states in 32 or 8 bits.
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"bf16": 2, "f32": 4}


# ------------------------------------------------------------------- cases --
def listed():
    return [
        # one projection of a decode step's experts: 64 tokens x top-8, about
        # four rows per expert, bound by streaming the weights
        dict(name="grouped_fwd_decode", op="grouped", form="fwd", rows=512, slack=0, groups=128,
             n_in=4096, n_out=1024, dtype="bf16", out="bf16", skew=0.0),
        # input gradient of one projection over a prefill-sized batch whose
        # expert load is skewed
        dict(name="grouped_dx_skewed", op="grouped", form="dx", rows=26215, slack=6553, groups=32,
             n_in=4096, n_out=1024, dtype="bf16", out="bf16", skew=0.5),
        # weight gradients of one projection kept in 32 bits, about 270 rows
        # per expert
        dict(name="grouped_dw_f32_out", op="grouped", form="dw", rows=17200, slack=7376, groups=64,
             n_in=6144, n_out=2048, dtype="bf16", out="f32", skew=0.0),
        # the tiny fp32 layer's experts
        dict(name="ffn_backward_tiny_f32", op="ffn_backward", T=128, d=256, N=8, Z=2, k=2, F=512,
             dtype="f32", skew=0.0),
        # a prefill-sized batch with skewed expert load
        dict(name="ffn_backward_skewed", op="ffn_backward", T=4096, d=4096, N=32, Z=8, k=8, F=1024,
             dtype="bf16", skew=0.5),
        # the large-expert-count layer's density (about 270 rows per expert)
        dict(name="ffn_backward_large", op="ffn_backward", T=2048, d=6144, N=64, Z=28, k=12,
             F=2048, dtype="bf16", skew=0.0),
        # gates' gradients for a decode-sized batch (latency)
        dict(name="combine_backward_small", op="combine_backward", T=64, d=4096, N=128, Z=32, k=8,
             F=1024, dtype="bf16", skew=0.0),
        # the large-expert-count layer's batch
        dict(name="combine_backward_large", op="combine_backward", T=8192, d=6144, N=256, Z=64,
             k=12, F=2048, dtype="bf16", skew=0.0),
        dict(name="input_backward_small", op="input_backward", T=64, d=4096, N=128, Z=32, k=8,
             F=1024, dtype="bf16", skew=0.0),
        dict(name="input_backward_large", op="input_backward", T=8192, d=6144, N=256, Z=64, k=12,
             F=2048, dtype="bf16", skew=0.0),
        # a router, its bias and many small odd-sized tensors (latency)
        dict(name="adamw_many_small", op="adamw", tensors=28, largest=80000, total=655360,
             bits=32, param="f32", grad="f32"),
        # the expert weights of a prefill-sized layer: bf16 weights with 32-bit
        # masters, states in 8 bits
        dict(name="adamw_experts_8bit", op="adamw", tensors=4, largest=134217728,
             total=402653184 + 655360, bits=8, param="bf16", grad="bf16"),
    ]


def _log(rng, lo, hi):
    return math.exp(rng.uniform(math.log(lo), math.log(hi)))


def _dim(rng, lo, hi, step):
    return max(step, int(_log(rng, lo, hi)) // step * step)


def draw(rng):
    op = rng.choice(["grouped", "grouped", "ffn_backward", "ffn_backward", "combine_backward",
                     "input_backward", "adamw"])
    skew = rng.choice([0.0, 0.0, 0.25, 0.5])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op == "adamw":
        tensors = rng.randint(1, 28)
        largest = int(_log(rng, 100, 60_000_000))
        total = largest + rng.randint(0, largest * min(tensors - 1, 3))
        param = rng.choice(["bf16", "f32"])
        return dict(op=op, tensors=tensors, largest=largest, total=total,
                    bits=rng.choice([8, 32]), param=param, grad=rng.choice([param, "f32"]))
    step = rng.choice([8, 64, 128])  # every size is a multiple of 8
    if op == "grouped":
        form = rng.choice(["fwd", "dx", "dw"])
        groups = int(_log(rng, 1, 256))
        small = dtype == "f32"
        n_in = _dim(rng, 64, 1024 if small else 6144, step)
        n_out = _dim(rng, 64, 1024 if small else 6144, step)
        most = min(24000, 3e9 / (n_in + n_out) / 4, (1.5e10 if small else 2e11) / n_in / n_out)
        rows = int(_log(rng, 1, most))
        out = dtype if form != "dw" else rng.choice([dtype, "f32"])
        return dict(op=op, form=form, rows=rows, slack=rng.choice([0, rng.randint(1, 500)]),
                    groups=groups, n_in=n_in, n_out=n_out, dtype=dtype, out=out, skew=skew)
    N = int(_log(rng, 1, 64 if op == "ffn_backward" else 256))
    Z = rng.randint(0, 1 + N // 3)
    k = rng.randint(1, min(12, N + Z))
    d = _dim(rng, 64, 6144, step)
    if op == "ffn_backward":
        small = dtype == "f32"
        if small:
            d = min(d, 1024)
        F = _dim(rng, 64, 512 if small else 2048, step)
        T = int(_log(rng, 1, max(2, min(2048, (2e9 if small else 1.5e11) / d / F / k))))
        return dict(op=op, T=T, d=d, N=N, Z=Z, k=k, F=F, dtype=dtype, skew=skew)
    T = int(_log(rng, 1, max(2, min(8192, 3e8 / d / k))))
    return dict(op=op, T=T, d=d, N=N, Z=Z, k=k, F=64, dtype=dtype, skew=skew)


# ------------------------------------------------------------------ inputs --
def _normal(g, *shape, dtype=torch.float32, scale=1.0):
    """Random normal values of any size, drawn in the type they are kept in."""
    return torch.randn(*shape, generator=g, device=DEV, dtype=dtype).mul_(scale)


def _popularity(g, n, skew):
    rank = torch.randperm(n, generator=g, device=DEV).float() + 1
    return skew * 3.0 * rank ** -1.1


def _routing(case, g):
    """Expert ids, gates and the dispatch of them: what the forward pass of the
    layer leaves behind (rows ordered by expert, then token)."""
    T, N, Z, k = case["T"], case["N"], case["Z"], case["k"]
    E = N + Z
    logits = _normal(g, T, E)
    bias = torch.zeros(E, device=DEV)
    bias[:N] = _popularity(g, N, case["skew"])
    idx = torch.topk(logits + bias, k, dim=1).indices
    gate = torch.softmax(torch.gather(logits, 1, idx), dim=1)
    flat = idx.reshape(-1)
    routed = flat < N
    order = torch.argsort(torch.where(routed, flat, E), stable=True)
    row = torch.empty_like(order)
    row[order] = torch.arange(T * k, device=DEV)
    slot_row = torch.where(routed, row, -1).int()
    counts = torch.bincount(flat, minlength=E)[:N]
    offsets = torch.zeros(N + 1, dtype=torch.int32, device=DEV)
    offsets[1:] = torch.cumsum(counts, 0)
    return idx.int(), gate, slot_row, offsets, int(counts.max()) if N else 0


def _sizes(case, g):
    """Numbers of elements of the adamw tensors: the largest one, and the rest
    shared unevenly, odd sizes among them."""
    n, rest = case["tensors"], case["total"] - case["largest"]
    if n == 1:
        return [case["largest"]]
    share = torch.rand(n - 1, generator=torch.Generator().manual_seed(n)).double() + 0.05
    cut = (share / share.sum() * rest).long().clamp(0, case["largest"]).tolist()
    return [case["largest"]] + cut


def _framework():
    import expert_routing_dispatch_router_b200 as moe

    return moe


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(int(seed))
    op = case["op"]
    s = dict(case=case)
    if op == "grouped":
        dt, G = DTYPES[case["dtype"]], case["groups"]
        rows, cap = case["rows"], case["rows"] + case["slack"]
        p = torch.softmax(_popularity(g, G, case["skew"]), 0)
        pick = torch.multinomial(p, rows, replacement=True, generator=g)
        counts = torch.bincount(pick, minlength=G)
        s["offsets"] = torch.zeros(G + 1, dtype=torch.int32, device=DEV)
        s["offsets"][1:] = torch.cumsum(counts, 0)
        s["longest"] = int(counts.max())
        n_in, n_out = case["n_in"], case["n_out"]
        if case["form"] != "dx":
            s["x"] = _normal(g, cap, n_in, dtype=dt)
        if case["form"] != "fwd":
            s["dy"] = _normal(g, cap, n_out, dtype=dt, scale=0.01)
        if case["form"] == "dw":
            s["out"] = torch.empty(G, n_out, n_in, dtype=DTYPES[case["out"]], device=DEV)
        else:
            s["w"] = _normal(g, G, n_out, n_in, dtype=dt, scale=n_in ** -0.5)
            s["out"] = torch.zeros(cap, n_out if case["form"] == "fwd" else n_in, dtype=dt,
                                   device=DEV)
        if own:
            moe = _framework()
            s["shape"] = moe.GroupedShape(cap, G, n_in, n_out, dt)
            s["ws"] = moe.alloc_grouped_workspace(s["shape"])
        return s
    if op == "adamw":
        sizes = _sizes(case, g)
        pdt, gdt = DTYPES[case["param"]], DTYPES[case["grad"]]
        s["params"] = [_normal(g, n, scale=0.02).to(pdt) for n in sizes]
        s["grads"] = [_normal(g, n, dtype=gdt, scale=0.01) for n in sizes]
        # the states after some steps (running means of such gradients), one
        # flat buffer of all tensors, each padded with zeros to whole blocks
        s["used"] = _flat([torch.ones(n, dtype=torch.bool, device=DEV) for n in sizes])
        m = torch.where(s["used"], _normal(g, s["used"].numel(), scale=0.003), 0.0)
        v = torch.where(s["used"], _normal(g, s["used"].numel(), scale=0.01).square_(), 0.0)
        s["master"] = [p.float() for p in s["params"]] if case["param"] == "bf16" else []
        s["hyper"] = dict(lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1)
        s["step"] = 10
        if case["bits"] == 8:
            s["m"], s["v"] = _quantise(m), _quantise(torch.sqrt(v), raise_small=True)
        else:
            s["m"], s["v"] = m, v
        if own:
            moe = _framework()
            s["opt"] = moe.AdamW(s["params"], s["grads"], state_bits=case["bits"],
                                 master=s["master"] or None)
            s["opt"].load_state(s["m"], s["v"], s["step"])
        return s
    # the layer's own operators
    dt = DTYPES[case["dtype"]]
    T, d, N, Z, k, F = (case[n] for n in ("T", "d", "N", "Z", "k", "F"))
    s["idx"], s["gate"], s["slot_row"], s["offsets"], s["longest"] = _routing(case, g)
    if op == "ffn_backward":
        s["x_perm"] = _normal(g, T * k, d, dtype=dt)
        s["dy_perm"] = _normal(g, T * k, d, dtype=dt, scale=0.01)
        s["w_gate"] = _normal(g, N, F, d, dtype=dt, scale=d ** -0.5)
        s["w_up"] = _normal(g, N, F, d, dtype=dt, scale=d ** -0.5)
        s["w_down"] = _normal(g, N, d, F, dtype=dt, scale=d ** -0.5)
        s["dx_perm"] = torch.zeros(T * k, d, dtype=dt, device=DEV)
        s["dw"] = [torch.empty_like(s[n]) for n in ("w_gate", "w_up", "w_down")]
    else:
        s["dout"] = _normal(g, T, d, dtype=dt, scale=0.01)
        s["x"] = _normal(g, T, d, dtype=dt)
        if op == "combine_backward":
            s["y_perm"] = _normal(g, T * k, d, dtype=dt, scale=0.5)
            s["dy_perm"] = torch.zeros(T * k, d, dtype=dt, device=DEV)
            s["dgate"] = torch.empty(T, k, device=DEV)
        else:
            s["w_router"] = _normal(g, N + Z, d, scale=d ** -0.5)
            s["dgate"] = _normal(g, T, k, scale=0.5)
            s["dx_perm"] = _normal(g, T * k, d, dtype=dt, scale=0.01)
            s["dx"] = torch.empty(T, d, dtype=dt, device=DEV)
            s["dw_router"] = torch.empty(N + Z, d, device=DEV)
    if own:
        moe = _framework()
        s["shape"] = moe.LayerShape(T, d, N, Z, k, F, dt, SCALE)
        s["ws"] = moe.alloc_backward_workspace(s["shape"])
    return s


SCALE = 2.5  # the layer's factor on the routed part


# ------------------------------------------------------------- plain forms --
def _padded(t, offsets, longest):
    """[groups, longest, cols] in 32 bits: each group's rows, then zeros."""
    at = torch.arange(longest, device=DEV)
    start, end = offsets[:-1].long()[:, None], offsets[1:].long()[:, None]
    row = (start + at).clamp(max=max(t.shape[0] - 1, 0))
    inside = (start + at < end)[:, :, None]
    return torch.where(inside, t[row].float(), 0.0)


def _ragged(p, offsets, rows, dtype):
    """The rows of [groups, longest, cols] back in their order; zeros behind the last."""
    r = torch.arange(rows, device=DEV)
    e = (torch.searchsorted(offsets.long(), r, right=True) - 1).clamp(0, p.shape[0] - 1)
    at = (r - offsets.long()[e]).clamp(0, p.shape[1] - 1)
    return torch.where((r < offsets[-1])[:, None], p[e, at], 0.0).to(dtype)


def _plain_grouped(s):
    case, off, longest = s["case"], s["offsets"], s["longest"]
    dt = DTYPES[case["out"]]
    if case["form"] == "fwd":
        y = _padded(s["x"], off, longest) @ s["w"].float().mT
        return _ragged(y, off, s["x"].shape[0], dt)
    if case["form"] == "dx":
        dx = _padded(s["dy"], off, longest) @ s["w"].float()
        return _ragged(dx, off, s["dy"].shape[0], dt)
    return (_padded(s["dy"], off, longest).mT @ _padded(s["x"], off, longest)).to(dt)


def _plain_ffn_backward(s):
    off, longest, dt = s["offsets"], s["longest"], s["x_perm"].dtype
    x, dy = _padded(s["x_perm"], off, longest), _padded(s["dy_perm"], off, longest)
    wg, wu, wd = s["w_gate"].float(), s["w_up"].float(), s["w_down"].float()
    a, u = x @ wg.mT, x @ wu.mT
    sig = 1.0 / (1.0 + torch.exp(-a))
    dh = dy @ wd
    da = dh * u * sig * (1.0 + a * (1.0 - sig))
    du = dh * a * sig
    dx = _ragged(da @ wg + du @ wu, off, s["x_perm"].shape[0], dt)
    return (dx, (da.mT @ x).to(dt), (du.mT @ x).to(dt), (dy.mT @ (a * sig * u)).to(dt))


def _plain_combine_backward(s):
    case = s["case"]
    T, k, N = case["T"], case["k"], case["N"]
    routed = (s["idx"] < N)[:, :, None]
    row = s["slot_row"].view(T, k).clamp(min=0).long()
    dout = s["dout"].float()
    seen = torch.where(routed, SCALE * s["y_perm"][row].float(), s["x"].float()[:, None, :])
    dgate = (seen * dout[:, None, :]).sum(-1)
    # every routed slot's row, in the order of the rows
    slot = s["slot_row"].long()
    at = torch.where(slot >= 0, slot, T * k)
    slot_of = torch.full((T * k + 1,), -1, dtype=torch.long, device=DEV)
    slot_of[at] = torch.arange(T * k, device=DEV)
    slot_of = slot_of[: T * k]
    used = torch.arange(T * k, device=DEV) < s["offsets"][-1]
    j = torch.where(used, slot_of, 0)
    dy = SCALE * s["gate"].view(-1)[j][:, None] * dout[j // k]
    return torch.where(used[:, None], dy, 0.0).to(s["y_perm"].dtype), dgate


def _plain_input_backward(s):
    case = s["case"]
    T, k, N, E = case["T"], case["k"], case["N"], case["N"] + case["Z"]
    gate, dgate, idx = s["gate"], s["dgate"], s["idx"].long()
    dlogit = gate * (dgate - (gate * dgate).sum(1, keepdim=True))
    dense = torch.zeros(T, E, device=DEV).scatter(1, idx, dlogit)
    routed = (idx < N)[:, :, None]
    row = s["slot_row"].view(T, k).clamp(min=0).long()
    through = torch.where(routed, s["dx_perm"][row].float(), 0.0).sum(1)
    same = torch.where(idx >= N, gate, 0.0).sum(1, keepdim=True) * s["dout"].float()
    dx = through + same + dense @ s["w_router"]
    return dx.to(s["x"].dtype), dense.mT @ s["x"].float()


BLOCK = 256  # values that share a scale


def _flat(tensors):
    """One buffer of all tensors, each padded with zeros to whole blocks."""
    return torch.cat([torch.nn.functional.pad(t, (0, -t.numel() % BLOCK)) for t in tensors])


def _parts(flat, tensors):
    """The tensors' values out of such a buffer."""
    padded = [-(-t.numel() // BLOCK) * BLOCK for t in tensors]
    return [f[: t.numel()] for f, t in zip(torch.split(flat, padded), tensors)]


def _quantise(t, raise_small=False):
    """Values in e4m3 with one 32-bit scale per block. With raise_small no
    positive value becomes zero: it takes the smallest step."""
    b = t.view(-1, BLOCK)
    scale = b.abs().amax(1, keepdim=True) / 448.0
    q = torch.where(scale > 0, b / torch.where(scale > 0, scale, 1.0), 0.0)
    if raise_small:
        q = torch.where((q > 0) & (q < 2.0 ** -9), 2.0 ** -9, q)
    q = q.clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return q.view(-1), scale.view(-1)


def _values(q):
    """The values that a quantised buffer stands for."""
    code, scale = q
    return (code.view(-1, BLOCK).float() * scale[:, None]).view(-1)


def _plain_adamw(s):
    h, bits = s["hyper"], s["case"]["bits"]
    s["step"] += 1
    c1, c2 = 1.0 - h["beta1"] ** s["step"], 1.0 - h["beta2"] ** s["step"]
    size, root = h["lr"] / c1, math.sqrt(c2)
    keep = 1.0 - h["lr"] * h["weight_decay"]
    g = _flat(s["grads"]).float()
    weights = s["master"] or s["params"]
    p = _flat(weights)
    m, v = s["m"], s["v"]
    if bits == 8:
        r = _values(v)
        m, v = _values(m), r * r
    m = m * h["beta1"] + g * (1.0 - h["beta1"])
    v = v * h["beta2"] + (g * (1.0 - h["beta2"])) * g
    r = torch.sqrt(v)
    p = p * keep - (m / (r / root + h["eps"])) * size
    new = _parts(p, weights)
    torch._foreach_copy_(s["params"], new)
    if s["master"]:
        torch._foreach_copy_(s["master"], new)
    if bits == 8:
        s["m"], s["v"] = _quantise(m), _quantise(r, raise_small=True)
        m, r = _values(s["m"]), _values(s["v"])
        return dict(params=s["params"], master=s["master"], m=m, root_v=r)
    s["m"], s["v"] = m, v
    return dict(params=s["params"], master=s["master"], m=m, v=v)


# --------------------------------------------------------------------- run --
def _own_run(s):
    moe, case = _framework(), s["case"]
    op = case["op"]
    if op == "grouped":
        if case["form"] == "fwd":
            return moe.grouped_matmul(s["shape"], s["x"], s["w"], s["offsets"], s["ws"],
                                      out=s["out"])
        if case["form"] == "dx":
            return moe.grouped_matmul_dx(s["shape"], s["dy"], s["w"], s["offsets"], s["ws"],
                                         out=s["out"])
        return moe.grouped_matmul_dw(s["shape"], s["dy"], s["x"], s["offsets"], s["ws"],
                                     out=s["out"])
    if op == "ffn_backward":
        return moe.expert_ffn_backward(
            s["shape"], s["x_perm"], s["offsets"], s["w_gate"], s["w_up"], s["w_down"],
            s["dy_perm"], s["ws"], dx_perm=s["dx_perm"], dw_gate=s["dw"][0], dw_up=s["dw"][1],
            dw_down=s["dw"][2])
    if op == "combine_backward":
        return moe.combine_backward(s["shape"], s["dout"], s["x"], s["y_perm"], s["idx"],
                                    s["gate"], s["slot_row"], dy_perm=s["dy_perm"],
                                    dgate=s["dgate"])
    if op == "input_backward":
        return moe.input_backward(s["shape"], s["dout"], s["x"], s["w_router"], s["idx"],
                                  s["gate"], s["slot_row"], s["dgate"], s["dx_perm"], s["ws"],
                                  dx=s["dx"], dw_router=s["dw_router"])
    moe.adamw_step(s["opt"], **s["hyper"])
    out = dict(params=s["params"], master=s["master"])
    if case["bits"] == 32:
        return dict(out, m=s["opt"].m, v=s["opt"].v)
    # the states are the optimizer's own buffers; what 8 bits hold (the second
    # moment by its root) is widened to the values that it stands for
    return dict(out, m=_values(s["opt"].m), root_v=_values(s["opt"].v))


def run(state):
    if own:
        return _own_run(state)
    return {"grouped": _plain_grouped, "ffn_backward": _plain_ffn_backward,
            "combine_backward": _plain_combine_backward,
            "input_backward": _plain_input_backward, "adamw": _plain_adamw}[
                state["case"]["op"]](state)


# -------------------------------------------------------------------- work --
def work(case):
    op = case["op"]
    if op == "grouped":
        es, G, rows = BYTES[case["dtype"]], case["groups"], case["rows"]
        n_in, n_out = case["n_in"], case["n_out"]
        flops = 2.0 * rows * n_in * n_out
        if case["form"] == "dw":
            return dict(bytes=rows * (n_in + n_out) * es + G * n_in * n_out * BYTES[case["out"]],
                        flops=flops)
        touched = G * (1.0 - (1.0 - 1.0 / G) ** rows)  # a group without rows needs no weights
        return dict(bytes=(rows * (n_in + n_out) + touched * n_in * n_out) * es, flops=flops)
    if op == "adamw":
        n = case["total"]
        each = 2 * BYTES[case["param"]] + BYTES[case["grad"]]  # weights in and out, gradient in
        if case["param"] == "bf16":
            each += 8 - 2  # the masters are read and written, the weights only written
        each += 16 if case["bits"] == 32 else 4 + 2 * 2 * 4 / 256
        return dict(bytes=n * each, flops=15.0 * n)
    es = BYTES[case["dtype"]]
    T, d, N, Z, k, F = (case[n] for n in ("T", "d", "N", "Z", "k", "F"))
    E = N + Z
    R = T * k * N / E  # routed rows (all of them where the load is not skewed away)
    if op == "ffn_backward":
        touched = N * (1.0 - (1.0 - 1.0 / N) ** R)
        return dict(bytes=(3 * R * d + 3 * touched * d * F + 3 * N * d * F) * es,
                    flops=8 * 2.0 * R * d * F)
    slots = T * k * 12.0  # expert id, gate, row
    if op == "combine_backward":
        return dict(bytes=(2 * T * d + 2 * R * d) * es + slots + T * k * 4, flops=3.0 * T * k * d)
    return dict(bytes=(3 * T * d + R * d) * es + 2 * E * d * 4 + slots + T * k * 4,
                flops=5.0 * T * k * d)


# ------------------------------------------------------------------- exact --
def exact(case, seed):
    """The operators by their definitions in 64 bits, group by group."""
    s = prepare(case, seed)
    return {"grouped": _exact_grouped, "ffn_backward": _exact_ffn_backward,
            "combine_backward": _exact_combine_backward,
            "input_backward": _exact_input_backward, "adamw": _exact_adamw}[case["op"]](s)


def _segments(s):
    off = s["offsets"].tolist()
    return [(e, off[e], off[e + 1]) for e in range(len(off) - 1)]


def _exact_grouped(s):
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
    for e, lo, hi in _segments(s):
        if s["case"]["form"] == "fwd":
            out[lo:hi] = torch.einsum("ri,oi->ro", s["x"][lo:hi].double(), s["w"][e].double())
        elif s["case"]["form"] == "dx":
            out[lo:hi] = torch.einsum("ro,oi->ri", s["dy"][lo:hi].double(), s["w"][e].double())
        else:
            out[e] = torch.einsum("ro,ri->oi", s["dy"][lo:hi].double(), s["x"][lo:hi].double())
    return out


def _exact_ffn_backward(s):
    dx = torch.zeros(s["x_perm"].shape, dtype=torch.float64, device=DEV)
    dwg, dwu, dwd = (torch.zeros(w.shape, dtype=torch.float64, device=DEV) for w in s["dw"])
    for e, lo, hi in _segments(s):
        x, dy = s["x_perm"][lo:hi].double(), s["dy_perm"][lo:hi].double()
        wg, wu, wd = (s[n][e].double() for n in ("w_gate", "w_up", "w_down"))
        a, u = x.mm(wg.t()), x.mm(wu.t())
        g = torch.sigmoid(a)
        dh = dy.mm(wd)
        dwd[e] = dy.t().mm(a * g * u)
        du = dh * (a * g)
        da = dh * u * (g + a * g * (1 - g))
        dwg[e], dwu[e] = da.t().mm(x), du.t().mm(x)
        dx[lo:hi] = da.mm(wg) + du.mm(wu)
    return dx, dwg, dwu, dwd


def _exact_combine_backward(s):
    N, T, k = s["case"]["N"], s["case"]["T"], s["case"]["k"]
    dy = torch.zeros(s["y_perm"].shape, dtype=torch.float64, device=DEV)
    dgate = torch.zeros(T, k, dtype=torch.float64, device=DEV)
    dout, x, gate = s["dout"].double(), s["x"].double(), s["gate"].double()
    rows = s["slot_row"].view(T, k).long()
    for j in range(k):
        on = s["idx"][:, j] < N
        r = rows[on, j]
        dy[r] = SCALE * gate[on, j, None] * dout[on]
        dgate[on, j] = SCALE * torch.einsum("td,td->t", s["y_perm"][r].double(), dout[on])
        dgate[~on, j] = torch.einsum("td,td->t", x[~on], dout[~on])
    return dy, dgate


def _exact_input_backward(s):
    N, T, k = s["case"]["N"], s["case"]["T"], s["case"]["k"]
    gate, dgate, x = s["gate"].double(), s["dgate"].double(), s["x"].double()
    w = s["w_router"].double()
    dlogit = gate * dgate - gate * torch.einsum("tj,tj->t", gate, dgate)[:, None]
    dx = torch.zeros(x.shape, dtype=torch.float64, device=DEV)
    dw = torch.zeros_like(w)
    rows = s["slot_row"].view(T, k).long()
    for j in range(k):
        e = s["idx"][:, j].long()
        on = e < N
        dx[on] += s["dx_perm"][rows[on, j]].double()
        dx[~on] += gate[~on, j, None] * s["dout"][~on].double()
        dx += dlogit[:, j, None] * w[e]
        dw.index_add_(0, e, dlogit[:, j, None] * x)
    return dx, dw


def _exact_adamw(s):
    h, t, eight = s["hyper"], s["step"] + 1, s["case"]["bits"] == 8
    m, v = (_values(s["m"]), _values(s["v"])) if eight else (s["m"], s["v"])
    m, v = m.double(), v.double()
    if eight:
        v = v.square()
    grads = torch.zeros_like(m)
    grads[s["used"]] = torch.cat(s["grads"]).double()
    m = h["beta1"] * m + (1 - h["beta1"]) * grads
    v = h["beta2"] * v + (1 - h["beta2"]) * grads.square()
    mh, vh = m / (1 - h["beta1"] ** t), v / (1 - h["beta2"] ** t)
    step = (h["lr"] * mh / (vh.sqrt() + h["eps"]))[s["used"]]
    start = [p.double() for p in s["master"] or s["params"]]
    new = [(1 - h["lr"] * h["weight_decay"]) * p - d
           for p, d in zip(start, torch.split(step, [p.numel() for p in start]))]
    out = dict(params=new, master=new if s["master"] else [])
    if eight:  # what 8 bits hold has no 64-bit value of its own
        return dict(out, m=None, root_v=None)
    return dict(out, m=m, v=v)
