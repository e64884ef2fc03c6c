"""Host-side tests of the training calls: the 64-bit gradients that the GPU
tests compare with agree with central differences of the layer itself, and the
library and its binding refuse bad arguments before anything is launched (so
these run without a GPU)."""
import ctypes

import pytest
import torch

import backward_helpers as ref
import expert_routing_dispatch_router_b200 as moe

P = ctypes.c_void_p
ST = P(0)


def _fake(addr=0x100000):
    return P(addr)


def _apart(n, step=1 << 40):
    """n addresses with room between them for any buffer of these tests."""
    return [P((i + 1) * step) for i in range(n)]


# ------------------------------------------------- formulas vs differences --
def _layer(x, w_r, wg, wu, wd, idx, n_routed, scale):
    """The layer in 64 bits for a fixed selection, token by token."""
    out = torch.zeros_like(x)
    for t in range(x.shape[0]):
        sel = idx[t].long()
        gate = torch.softmax(w_r[sel] @ x[t], 0)
        for j, e in enumerate(sel.tolist()):
            if e < n_routed:
                a, u = wg[e] @ x[t], wu[e] @ x[t]
                out[t] += scale * gate[j] * (wd[e] @ (a * torch.sigmoid(a) * u))
            else:
                out[t] += gate[j] * x[t]
    return out


@pytest.mark.parametrize("n_routed,n_zero,k", [(3, 2, 2), (2, 0, 1), (0, 3, 2)])
def test_reference_gradients_match_differences(n_routed, n_zero, k):
    g = torch.Generator().manual_seed(5)
    T, d, F, scale = 5, 8, 6, 1.7
    idx, _, slot_row, offsets = ref.route_by_hand(T, n_routed, n_zero, k, g)
    rnd = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    x, w_r, dout = rnd(T, d), rnd(n_routed + n_zero, d), rnd(T, d)
    wg, wu, wd = rnd(n_routed, F, d), rnd(n_routed, F, d), rnd(n_routed, d, F)
    gate = torch.softmax(torch.einsum("tjd,td->tj", w_r[idx.long()], x), 1)
    rows = slot_row.view(T, k).long()
    R = int(offsets[-1])
    x_perm, y_perm = torch.zeros(T * k, d).double(), torch.zeros(T * k, d).double()
    for t in range(T):
        x_perm[rows[t][rows[t] >= 0]] = x[t]
    for e, lo, hi in ref.segments(offsets):
        a, u = x_perm[lo:hi] @ wg[e].T, x_perm[lo:hi] @ wu[e].T
        y_perm[lo:hi] = (a * torch.sigmoid(a) * u) @ wd[e].T
    (dy, _), (dgate, _) = ref.combine_backward(dout, x, y_perm, idx, gate, slot_row, n_routed,
                                               scale)
    (dxp, _), (dwg, _), (dwu, _), (dwd, _) = ref.ffn_backward(x_perm, offsets, wg, wu, wd, dy,
                                                              torch.float32)
    (dx, _), (dw_r, _) = ref.input_backward(dout, x, w_r, idx, gate, slot_row, dgate, dxp,
                                            n_routed)
    assert R == int((idx < n_routed).sum())

    def loss():
        return float((_layer(x, w_r, wg, wu, wd, idx, n_routed, scale) * dout).sum())

    h = 1e-5
    for name, t, grad in (("x", x, dx), ("w_router", w_r, dw_r), ("w_gate", wg, dwg),
                          ("w_up", wu, dwu), ("w_down", wd, dwd)):
        flat, gf = t.view(-1), grad.reshape(-1)
        for i in torch.randperm(flat.numel(), generator=g)[:40].tolist():
            keep = float(flat[i])
            flat[i] = keep + h
            up = loss()
            flat[i] = keep - h
            down = loss()
            flat[i] = keep
            num = (up - down) / (2 * h)
            # h^2 / 6 of a third derivative of order 1e2, and rounding / h
            assert abs(num - float(gf[i])) <= 1e-7 * (1 + abs(num)), name


# ---------------------------------------------------------- C ABI refusals --
def grouped(rows=64, groups=4, n_in=64, n_out=32, dt=moe.MOE_BF16):
    return moe.MoEGrouped(rows, groups, n_in, n_out, dt)


def test_grouped_shapes_refused():
    L = moe.lib()
    assert L.moe_grouped_workspace_size(ctypes.byref(grouped())) >= 256
    for bad, code in ((grouped(rows=-1), 1), (grouped(groups=0), 1), (grouped(n_in=0), 1),
                      (grouped(n_out=-8), 1), (grouped(dt=9), 1), (grouped(n_in=60), 2),
                      (grouped(n_out=4), 2), (grouped(groups=1025), 2),
                      (grouped(rows=2 ** 31 - 1, n_in=65536), 2), (grouped(rows=2 ** 24 + 1), 2),
                      (grouped(groups=1024, n_in=1 << 17, n_out=1 << 17), 2)):
        assert L.moe_grouped_workspace_size(ctypes.byref(bad)) == 0
        for fn in (L.moe_grouped_matmul, L.moe_grouped_matmul_dx):
            assert fn(ctypes.byref(bad), *_apart(5), 256, ST) == code
        assert L.moe_grouped_matmul_dw(ctypes.byref(bad), *_apart(4), bad.dtype, _fake(), 256,
                                       ST) == code
    assert L.moe_grouped_matmul(None, *_apart(5), 256, ST) == 1
    assert L.moe_grouped_workspace_size(None) == 0


def test_grouped_matrix_sizes_have_a_limit():
    # behind it a row's chain of sums drifts past the rounding of its result, and
    # numbers of column tiles were multiplied past 32 bits (n_in behind 2^25)
    L = moe.lib()
    size = lambda c: L.moe_grouped_workspace_size(ctypes.byref(c))  # noqa: E731
    top = 1 << 20
    assert size(grouped(rows=1, groups=1, n_in=top, n_out=8)) >= 256
    assert size(grouped(rows=1, groups=1, n_in=8, n_out=top)) >= 256
    for big in (top + 8, 1 << 26, (1 << 31) - 8):
        for n_in, n_out in ((big, 8), (8, big)):
            bad = grouped(rows=1, groups=1, n_in=n_in, n_out=n_out)
            assert size(bad) == 0
            for fn in (L.moe_grouped_matmul, L.moe_grouped_matmul_dx):
                assert fn(ctypes.byref(bad), *_apart(5), 256, ST) == 2
            assert L.moe_grouped_matmul_dw(ctypes.byref(bad), *_apart(4), bad.dtype, _fake(), 256,
                                           ST) == 2
        for d, F in ((big, 8), (8, big)):
            c = ctypes.byref(cfg(T=1, d=d, N=1, Z=0, k=1, F=F))
            assert L.moe_backward_workspace_size(c) == 0


def test_grouped_pointers_refused():
    L = moe.lib()
    c = grouped()
    a, w, o, y, ws = _apart(5)
    for fn in (L.moe_grouped_matmul, L.moe_grouped_matmul_dx):
        assert fn(ctypes.byref(c), None, w, o, y, ws, 256, ST) == 1
        assert fn(ctypes.byref(c), a, w, P(o.value + 4), y, ws, 256, ST) == 1
        assert fn(ctypes.byref(c), a, w, o, y, None, 256, ST) == 3
        assert fn(ctypes.byref(c), a, w, o, y, ws, 255, ST) == 3
        assert fn(ctypes.byref(c), a, w, o, y, P(ws.value + 16), 256, ST) == 1
        # an output over an operand, the offsets or the workspace
        for out in (a, w, o, ws, P(a.value + 16)):
            assert fn(ctypes.byref(c), a, w, o, out, ws, 256, ST) == 1
    dw = L.moe_grouped_matmul_dw
    assert dw(ctypes.byref(c), a, w, o, y, 7, ws, 256, ST) == 1  # no such type
    f32 = grouped(dt=moe.MOE_F32)
    assert dw(ctypes.byref(f32), a, w, o, y, moe.MOE_BF16, ws, 256, ST) == 1
    assert dw(ctypes.byref(c), a, w, o, None, moe.MOE_BF16, ws, 256, ST) == 1
    assert dw(ctypes.byref(c), a, w, o, a, moe.MOE_BF16, ws, 256, ST) == 1
    # no rows: nothing to write, whatever the pointers
    empty = grouped(rows=0)
    assert L.moe_grouped_matmul(ctypes.byref(empty), *[None] * 5, 0, ST) == 0
    assert L.moe_grouped_matmul_dx(ctypes.byref(empty), *[None] * 5, 0, ST) == 0
    assert dw(ctypes.byref(empty), None, None, None, None, moe.MOE_BF16, None, 0, ST) == 1


def cfg(T=64, d=256, N=8, Z=2, k=2, F=512, dt=moe.MOE_BF16, s=1.0):
    return moe.MoEConfig(T, d, N, Z, k, F, dt, s)


def test_backward_configs_refused():
    L = moe.lib()
    n = L.moe_backward_workspace_size(ctypes.byref(cfg()))
    assert n > 0
    assert L.moe_backward_workspace_size(ctypes.byref(cfg(N=0))) > 0
    assert L.moe_backward_workspace_size(ctypes.byref(cfg(T=2 ** 23, d=128))) > 0
    for bad, code in ((cfg(k=11), 1), (cfg(d=12), 2), (cfg(F=20), 2), (cfg(T=-1), 1),
                      (cfg(T=2 ** 23 + 1, d=128), 2),
                      (cfg(dt=5), 1), (cfg(N=1100), 2), (cfg(s=float("nan")), 1)):
        assert L.moe_backward_workspace_size(ctypes.byref(bad)) == 0
        b = ctypes.byref(bad)
        assert L.moe_combine_backward(b, *_apart(8), ST) == code
        assert L.moe_expert_ffn_backward(b, *_apart(10), 1, _fake(), n, ST) == code
        assert L.moe_input_backward(b, *_apart(11), n, ST) == code
        assert L.moe_layer_backward(b, *_apart(17), 1, _fake(), n, ST) == code


def test_backward_pointers_refused():
    L = moe.lib()
    c = ctypes.byref(cfg())
    n = L.moe_backward_workspace_size(c)
    step = 1 << 40

    def each(fn, count, tail):
        """Every pointer missing, misaligned, and every output on top of the
        first input."""
        ok = _apart(count)
        for i in range(count):
            for bad in (None, P(ok[i].value + 8)):
                args = list(ok)
                args[i] = bad
                assert fn(c, *args, *tail) == 1, (fn.__name__, i)

    ws = P(50 * step)
    each(L.moe_combine_backward, 8, (ST,))
    each(L.moe_expert_ffn_backward, 10, (moe.MOE_BF16, ws, n, ST))
    each(L.moe_input_backward, 10, (ws, n, ST))
    each(L.moe_layer_backward, 17, (moe.MOE_BF16, ws, n, ST))
    for fn, count, dt, outs in ((L.moe_expert_ffn_backward, 10, True, range(6, 10)),
                                (L.moe_input_backward, 10, False, range(8, 10)),
                                (L.moe_layer_backward, 17, True, range(12, 17))):
        more = (moe.MOE_BF16,) if dt else ()
        ok = _apart(count)
        assert fn(c, *ok, *more, None, n, ST) == 3
        assert fn(c, *ok, *more, ws, n - 1, ST) == 3
        assert fn(c, *ok, *more, P(ws.value + 16), n, ST) == 1
        for o in outs:
            for onto in (ok[0], ws):
                args = list(ok)
                args[o] = onto
                assert fn(c, *args, *more, ws, n, ST) == 1, (fn.__name__, o)
        if dt:
            assert fn(c, *ok, 4, ws, n, ST) == 1
    for o in (6, 7):
        args = _apart(8)
        args[o] = args[2]
        assert L.moe_combine_backward(c, *args, ST) == 1
    # an f32 layer has f32 weight gradients only
    f = ctypes.byref(cfg(dt=moe.MOE_F32))
    nf = L.moe_backward_workspace_size(f)
    assert L.moe_expert_ffn_backward(f, *_apart(10), moe.MOE_BF16, ws, nf, ST) == 1
    # an empty batch: no rows to write; weight gradients still need a place
    e = ctypes.byref(cfg(T=0))
    assert L.moe_combine_backward(e, *[None] * 8, ST) == 0
    assert L.moe_expert_ffn_backward(e, *[None] * 10, moe.MOE_BF16, None, 0, ST) == 1
    assert L.moe_input_backward(e, *[None] * 11, 0, ST) == 1
    assert L.moe_layer_backward(e, *[None] * 17, moe.MOE_BF16, None, 0, ST) == 1
    z = ctypes.byref(cfg(N=0, T=0))
    assert L.moe_expert_ffn_backward(z, *[None] * 10, moe.MOE_BF16, None, 0, ST) == 0


def test_adamw_refusals():
    L = moe.lib()
    opt = moe.MoEAdamW(2, 32, moe.MOE_BF16, moe.MOE_F32, 8)
    good = dict(lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8, weight_decay=0.1)

    def call(o=opt, ptrs=None, **change):
        h = moe.MoEAdamWParams(**{**good, **change})
        t, m, ms, v, vs, st = ptrs or _apart(6)
        return L.moe_adamw_step(ctypes.byref(o), ctypes.byref(h), t, m, ms, v, vs, st, ST)

    nan, inf = float("nan"), float("inf")
    for change in (dict(beta1=1.0), dict(beta1=-0.1), dict(beta2=nan), dict(beta2=1.5),
                   dict(lr=-1e-3), dict(lr=inf), dict(eps=0.0), dict(eps=1e-60), dict(eps=-1.0),
                   dict(weight_decay=-0.1), dict(weight_decay=nan)):
        assert call(**change) == 1, change
    for bad in (moe.MoEAdamW(2, 16, 1, 0, 8), moe.MoEAdamW(2, 32, 3, 0, 8),
                moe.MoEAdamW(2, 32, 1, 3, 8), moe.MoEAdamW(-1, 32, 1, 0, 8),
                moe.MoEAdamW(2, 32, 1, 0, -1), moe.MoEAdamW(0, 32, 1, 0, 8)):
        assert call(bad) == 1
    for eps in (1e-38, 1e-45, 1e31, inf, nan):  # subnormal, or too large
        assert call(eps=eps) == 1, eps
    eight = moe.MoEAdamW(2, 8, 1, 0, 8)
    for i in range(6):  # overlapping states, scales, table or step count
        for j in range(i):
            ptrs = _apart(6)
            ptrs[i] = ptrs[j]
            assert call(eight, ptrs=ptrs) == 1
    for i in (0, 1, 3, 5):
        for p in (None, P(8)):
            ptrs = _apart(6)
            ptrs[i] = p
            assert call(ptrs=ptrs) == 1
    for i in (2, 4):  # the scales are needed with 8-bit states only
        ptrs = _apart(6)
        ptrs[i] = None
        assert call(eight, ptrs=ptrs) == 1
    assert L.moe_adamw_step(None, None, *_apart(6), ST) == 1


# --------------------------------------------------------- binding refusals --
def test_binding_refuses_host_tensors_and_bad_shapes():
    bf = torch.bfloat16
    gs = moe.GroupedShape(8, 2, 16, 8)
    x, w = torch.zeros(8, 16, dtype=bf), torch.zeros(2, 8, 16, dtype=bf)
    off, ws = torch.zeros(3, dtype=torch.int32), torch.zeros(256, dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA tensor"):
        moe.grouped_matmul(gs, x, w, off, ws)
    with pytest.raises(ValueError, match="dtype"):
        moe.grouped_matmul_dx(gs, x.float(), w, off, ws)
    with pytest.raises(ValueError, match="invalid or unsupported"):
        moe.alloc_grouped_workspace(moe.GroupedShape(8, 2, 12, 8), device="cpu")
    with pytest.raises(ValueError, match="CUDA tensor"):
        moe.AdamW([torch.zeros(4)], [torch.zeros(4)])
    with pytest.raises(ValueError, match="state_bits"):
        moe.AdamW([torch.zeros(4)], [torch.zeros(4)], state_bits=16)
    with pytest.raises(ValueError, match="at least one"):
        moe.AdamW([], [])
    with pytest.raises(ValueError, match="one gradient"):
        moe.AdamW([torch.zeros(4)], [])
    with pytest.raises(ValueError, match="dtype"):
        moe.AdamW([torch.zeros(4).half()], [torch.zeros(4)])


def test_overlapping_weights_are_refused():
    buf, other = torch.zeros(64), torch.zeros(64)
    refuse = moe.AdamW._refuse_overlaps
    refuse([buf[:32], buf[32:]], [other, other])  # shared gradients are only read
    refuse([buf[:0], buf], [other])
    for written, read in (([buf, buf], []), ([buf[:40], buf[32:]], []), ([buf], [buf]),
                          ([buf[32:]], [buf]), ([buf], [buf[8:16]]),
                          ([buf[8:16]], [buf, other])):
        with pytest.raises(ValueError, match="overlaps"):
            refuse(written, read)


def test_binding_calls_reach_the_library_with_an_empty_batch(monkeypatch):
    """With no tokens the calls that have nothing to write return before any
    pointer is looked at: host tensors stand in for device ones (the device
    check is relaxed for this test only)."""
    import types
    real = moe._need
    monkeypatch.setattr(moe, "_need", lambda t, n, dt, shape=None, on_device=True:
                        real(t, n, dt, shape, on_device=False))
    monkeypatch.setattr(moe, "_ws", lambda ws: (P(ws.data_ptr()), ws.numel()))
    monkeypatch.setattr(moe, "_on_current_device", lambda *tensors: None)
    st = types.SimpleNamespace(cuda_stream=0)
    bf = torch.bfloat16
    sh = moe.LayerShape(T=0, d=64, n_routed=2, n_zero=1, top_k=2, ffn=64)
    x, rows = torch.zeros(0, 64, dtype=bf), torch.zeros(0, 64, dtype=bf)
    idx, gate = torch.zeros(0, 2, dtype=torch.int32), torch.zeros(0, 2)
    dy, dgate = moe.combine_backward(sh, x, x, rows, idx, gate,
                                     torch.zeros(0, dtype=torch.int32), stream=st)
    assert dy.shape == (0, 64) and dgate.shape == (0, 2)
    gs = moe.GroupedShape(0, 2, 16, 8)
    w, off = torch.zeros(2, 8, 16, dtype=bf), torch.zeros(3, dtype=torch.int32)
    ws = torch.zeros(256, dtype=torch.uint8)
    assert moe.grouped_matmul(gs, torch.zeros(0, 16, dtype=bf), w, off, ws,
                              stream=st).shape == (0, 8)
    assert moe.grouped_matmul_dx(gs, torch.zeros(0, 8, dtype=bf), w, off, ws,
                                 stream=st).shape == (0, 16)


def test_tensors_of_another_device_are_refused(monkeypatch):
    import types
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    here, there = (types.SimpleNamespace(get_device=lambda d=d: d, device=f"cuda:{d}")
                   for d in (1, 0))
    moe._on_current_device(here, None, here)
    with pytest.raises(ValueError, match="cuda:0"):
        moe._on_current_device(here, there)


def test_the_struct_of_a_shape_is_the_callers_own():
    import copy
    import pickle
    for sh, field in ((moe.LayerShape(4, 64, 2, 1, 2, 32), "T"),
                      (moe.GroupedShape(4, 2, 64, 32), "rows")):
        c = sh.c()
        setattr(c, field, 1000)
        assert getattr(sh.c(), field) == 4 and sh == copy.deepcopy(sh)
        assert getattr(pickle.loads(pickle.dumps(sh)).c(), field) == 4
    sh = moe.GroupedShape(4, 2, 64, 32)
    sh.c().n_in = 60  # no longer changes what later calls see
    moe.alloc_grouped_workspace(sh, device="cpu")


# ------------------------------------- the optimizer's buffers, on the host --
@pytest.fixture
def host_adamw(monkeypatch):
    """The binding over host tensors, with a step that only notes its call (the
    device checks are relaxed for these tests only)."""
    import types
    real, calls = moe._need, []
    monkeypatch.setattr(moe, "_need", lambda t, n, dt, shape=None, on_device=True:
                        real(t, n, dt, shape, on_device=False))
    monkeypatch.setattr(moe, "_on_current_device", lambda *tensors: None)
    state = types.SimpleNamespace(capturing=False)
    monkeypatch.setattr(moe, "_capturing", lambda stream=None: state.capturing, raising=False)
    monkeypatch.setattr(moe, "lib", lambda: types.SimpleNamespace(
        moe_adamw_step=lambda *a: calls.append(a) or 0))
    state.calls, state.stream = calls, types.SimpleNamespace(cuda_stream=0)
    return state


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_refuses_buffers_that_moved(host_adamw, bits):
    bf = torch.bfloat16
    p, grad = torch.ones(300, dtype=bf), torch.ones(300, dtype=bf)
    opt = moe.AdamW([p], [grad], state_bits=bits, master=[p.float()])
    step = lambda: moe.adamw_step(opt, lr=1e-3, stream=host_adamw.stream)  # noqa: E731
    step()
    for t in (p, opt.master[0], opt.state, *((opt.m, opt.v) if bits == 32
                                             else (*opt.m, *opt.v))):
        keep = t.data
        t.data = keep.clone()
        with pytest.raises(ValueError, match="moved"):
            step()
        t.data = keep
    for name in ("m", "v"):  # a state put in another's place, of any size
        keep = getattr(opt, name)
        setattr(opt, name, torch.zeros(256) if bits == 32 else tuple(t.clone() for t in keep))
        with pytest.raises(ValueError, match="moved"):
            step()
        setattr(opt, name, keep)
    step()
    assert len(host_adamw.calls) == 2


def test_adamw_reads_gradients_where_they_lie(host_adamw):
    params = [torch.ones(300), torch.ones(0), torch.ones(5)]
    grads = [torch.ones(300), torch.ones(0), torch.ones(5)]
    opt = moe.AdamW(params, grads)
    step = lambda: moe.adamw_step(opt, lr=1e-3, stream=host_adamw.stream)  # noqa: E731
    seen = lambda: opt._table[:, 2].tolist()  # noqa: E731
    step()
    first, table = seen(), opt._table
    grads[0].data = torch.zeros(300)
    step()
    assert seen() == [grads[0].data_ptr(), grads[2].data_ptr()] != first
    other = torch.zeros(5)
    opt.grads[2] = other  # another tensor in its place
    step()
    assert seen() == [grads[0].data_ptr(), other.data_ptr()]
    assert opt._table[:, [0, 1, 3, 4, 5]].equal(table[:, [0, 1, 3, 4, 5]])
    # what construction refuses is refused here too, and the step is not made
    for bad, match in ((torch.zeros(6), "shape"), (torch.zeros(5, dtype=torch.bfloat16), "dtype"),
                       (torch.zeros(10)[::2], "contiguous"), (torch.zeros(6)[1:], "aligned"),
                       (params[0][:5], "overlaps")):
        opt.grads[2] = bad
        with pytest.raises(ValueError, match=match):
            step()
    opt.grads[2] = other
    step()
    assert len(host_adamw.calls) == 4
    # a captured step's table and gradients stay; a step under capture refuses
    host_adamw.capturing = True
    step()
    captured = opt._table
    opt.grads[2] = torch.zeros(5)
    with pytest.raises(ValueError, match="capture"):
        step()
    host_adamw.capturing = False
    step()
    assert opt._kept[0][0] is captured and opt._kept[0][1][2].data_ptr() == other.data_ptr()
    assert opt._table is not captured and len(opt._kept) == 1


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_refused_states_change_nothing(host_adamw, bits):
    opt = moe.AdamW([torch.ones(300)], [torch.ones(300)], state_bits=bits)
    e4 = torch.float8_e4m3fn
    one = lambda v, n=512, k=2: torch.full((n,), v) if bits == 32 else (  # noqa: E731
        torch.full((n,), v).to(e4), torch.full((k,), v))
    opt.load_state(one(0.5), one(0.25), 3)
    held = lambda: [opt.state[0].item()] + [t.float().tolist() for t in (  # noqa: E731
        (opt.m, opt.v) if bits == 32 else (*opt.m, *opt.v))]
    before = held()
    bad = [(one(1.0), one(1.0, 256, 1), 5), (one(1.0, 256, 1), one(1.0), 5),
           (one(1.0), one(1.0), -1)]
    if bits == 8:
        bad += [(one(1.0), one(1.0)[:1], 5), (one(1.0), torch.ones(512), 5),
                (one(1.0), (one(1.0)[0], torch.ones(3)), 5)]
    else:
        bad += [(one(1.0), one(1.0).double(), 5)]
    for m, v, step in bad:
        with pytest.raises(ValueError):
            opt.load_state(m, v, step)
        assert held() == before
    opt.load_state(one(1.0), one(2.0), 7)
    assert held()[0] == 7 and held() != before


# ------------------------------------------------------------- the sources --
def test_arrivals_on_another_cta_release_at_cluster_scope():
    """At a narrower scope nothing that a thread did before its arrival is
    ordered before what the other CTA does after its wait, and two CTAs of a pair
    hand accumulators and unit ids to each other by such arrivals."""
    import glob
    import os
    import re
    csrc = os.path.join(os.path.dirname(moe.__file__), "csrc")
    seen = 0
    for path in sorted(glob.glob(os.path.join(csrc, "*.cu*"))):
        with open(path) as f:
            text = f.read()
        for op in re.findall(r"mbarrier\.arrive[\w.:]*shared::cluster[\w.:]*", text):
            assert op.startswith("mbarrier.arrive.release.cluster."), (path, op)
            seen += 1
    assert seen > 0
