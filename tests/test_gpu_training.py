"""GPU tests of the training calls against 64-bit gradients (backward_helpers
derives the tolerances): grouped products in three directions, the experts',
combine's and input's backward passes, the whole layer, and AdamW steps."""
import math
import types

import pytest
import torch

import backward_helpers as ref
import expert_routing_dispatch_router_b200 as moe

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


def dev(*ts):
    out = [t.to(DEV) for t in ts]
    return out[0] if len(out) == 1 else out


# ------------------------------------------------------- grouped products --
# segment sizes around the tiles of every path, empty segments at both ends and
# in the middle, one row, one group
SIZES = [(1,), (0, 5, 0), (1, 63, 64, 65, 0, 2), (16, 15, 17, 31, 32, 33),
         (127, 128, 129, 255, 256, 257), (700, 0, 3), (0, 0), (3,) * 40]


def grouped_inputs(sizes, n_in, n_out, dtype, slack, seed):
    g = torch.Generator().manual_seed(seed)
    rows = sum(sizes) + slack
    x = ref.random(g, rows, n_in, dtype=dtype)
    dy = ref.random(g, rows, n_out, dtype=dtype)
    w = ref.random(g, len(sizes), n_out, n_in, dtype=dtype, scale=n_in ** -0.5)
    # what lies behind the last segment is never used
    x[sum(sizes):] = float("nan")
    dy[sum(sizes):] = float("inf")
    return x, dy, w, ref.offsets_of(sizes)


def check_grouped(sizes, n_in, n_out, dtype, slack=0, seed=1, dw_f32=False, spoil=None):
    x, dy, w, off = grouped_inputs(sizes, n_in, n_out, dtype, slack, seed)
    if spoil is not None:  # one group's rows and weights are not numbers
        lo, hi = int(off[spoil]), int(off[spoil + 1])
        x[lo:hi], dy[lo:hi], w[spoil] = float("nan"), float("inf"), float("-inf")
    rows, G = x.shape[0], len(sizes)
    sh = moe.GroupedShape(rows, G, n_in, n_out, dtype)
    ws = moe.alloc_grouped_workspace(sh)
    xd, dyd, wd, offd = dev(x, dy, w, off)
    y = torch.full((rows, n_out), 7.0, dtype=dtype, device=DEV)
    dx = torch.full((rows, n_in), 7.0, dtype=dtype, device=DEV)
    dw = torch.full((G, n_out, n_in), 7.0, dtype=F32 if dw_f32 else dtype, device=DEV)
    moe.grouped_matmul(sh, xd, wd, offd, ws, out=y)
    moe.grouped_matmul_dx(sh, dyd, wd, offd, ws, out=dx)
    moe.grouped_matmul_dw(sh, dyd, xd, offd, ws, out=dw)
    assert moe.read_device_error(ws) == 0
    x, dy, w = x.double(), dy.double(), w.double()
    for e, lo, hi in ref.segments(off):
        if e == spoil:
            continue
        ref.check(y[lo:hi], *ref.mm(x[lo:hi], w[e].T), dtype, f"y of {e}")
        ref.check(dx[lo:hi], *ref.mm(dy[lo:hi], w[e]), dtype, f"dx of {e}")
        ref.check(dw[e], *ref.mm(dy[lo:hi].T, x[lo:hi]), dw.dtype, f"dw of {e}")
        if lo == hi:
            assert int(dw[e].count_nonzero()) == 0
    R = sum(sizes)
    assert bool((y[R:] == 7.0).all()) and bool((dx[R:] == 7.0).all())


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("sizes", SIZES, ids=str)
def test_grouped_segments(sizes, dtype):
    check_grouped(sizes, 128, 192, dtype)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("n_in,n_out", [(8, 8), (8, 264), (264, 8), (72, 136), (200, 56),
                                        (520, 1032), (1024, 384)])
def test_grouped_odd_sizes(n_in, n_out, dtype):
    check_grouped((5, 0, 70, 1, 130), n_in, n_out, dtype, slack=37, seed=2)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_grouped_many_groups(dtype):
    g = torch.Generator().manual_seed(3)
    sizes = torch.randint(0, 4, (1024,), generator=g).tolist()
    check_grouped(tuple(sizes), 64, 72, dtype, slack=5)


@pytest.mark.parametrize("rows", [300, 2600])
def test_grouped_fp32_weight_gradient_of_bf16(rows):
    check_grouped((rows, 0, 9), 136, 264, BF, slack=3, dw_f32=True)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("n_in,n_out", [(128, 128), (72, 40)])
def test_grouped_values_of_one_group_stay_in_it(n_in, n_out, dtype):
    # infinities and NaN in a neighbour's rows and weights, and behind the last
    # segment, reach no other group (sizes that end inside every tile)
    check_grouped((13, 21, 150, 7), n_in, n_out, dtype, slack=64, seed=4, spoil=1)
    check_grouped((33, 1, 0, 90), n_in, n_out, dtype, slack=64, seed=5, spoil=3)


@pytest.mark.parametrize("dw_dtype", [F32, BF], ids=["f32", "bf16"])
def test_grouped_weight_gradient_of_a_long_segment_does_not_drift(dw_dtype):
    # terms of one sign, where sums that cut instead of rounding drift with
    # every step: 1024 rows are one chain of sums (every addition cut, 2^-23 of
    # the sum so far), and the chains' sums are added rounding (2^-24 each)
    sizes, I, O = (400_017, 1, 1023, 1025, 5000), 136, 72
    R = sum(sizes)
    g = torch.Generator(device=DEV).manual_seed(51)
    x, dy = ((torch.rand(R, n, generator=g, device=DEV) * 0.5 + 0.5).to(BF) for n in (I, O))
    off = dev(ref.offsets_of(sizes))
    sh = moe.GroupedShape(R, len(sizes), I, O)
    ws = moe.alloc_grouped_workspace(sh)
    out = torch.empty(len(sizes), O, I, dtype=dw_dtype, device=DEV)
    moe.grouped_matmul_dw(sh, dy, x, off, ws, out=out)
    assert moe.read_device_error(ws) == 0
    for e, lo, hi in ref.segments(off):
        want = sum(dy[i:min(i + 50_000, hi)].double().T @ x[i:min(i + 50_000, hi)].double()
                   for i in range(lo, hi, 50_000))
        n = hi - lo
        bound = (min(n, 1024) * ref.U + (n // 1024 + 1) * ref.U / 2) * want
        ref.check(out[e], want.cpu(), bound.cpu(), dw_dtype, f"dw of {n} rows")


def test_grouped_float_weight_gradient_of_a_long_segment_does_not_drift():
    # the most rows of a call, terms of one sign: in one chain the last terms
    # are below a step of the sum and are rounded all one way. Chains of 1024
    # rows and the sum of those chains, every addition rounded (2^-24 each)
    R, n = 1 << 24, 8
    g = torch.Generator(device=DEV).manual_seed(53)
    x, dy = (torch.rand(R, n, generator=g, device=DEV) * 0.5 + 0.5 for _ in range(2))
    off = dev(torch.tensor([0, 1000, R], dtype=torch.int32))
    sh = moe.GroupedShape(R, 2, n, n, F32)
    ws = moe.alloc_grouped_workspace(sh)
    dw = moe.grouped_matmul_dw(sh, dy, x, off, ws)
    assert moe.read_device_error(ws) == 0
    for e, lo, hi in ref.segments(off):
        want = sum(dy[i:min(i + 2 ** 20, hi)].double().T @ x[i:min(i + 2 ** 20, hi)].double()
                   for i in range(lo, hi, 2 ** 20))
        bound = (1024 + (hi - lo) // 1024 + 1) * ref.U / 2 * want
        ref.check(dw[e], want.cpu(), bound.cpu(), F32, f"dw of {hi - lo} rows")


@pytest.mark.parametrize("n_in,n_out", [(1 << 20, 8), (8, 1 << 20)])
def test_grouped_widest_matrices(n_in, n_out):
    # terms of one sign; a product of 2^20 terms is 2^16 additions of 16, each
    # cut by up to 2^-23 of a sum so far that is half the last one on average
    R, off = 5, torch.tensor([0, 2, 5], dtype=torch.int32)
    g = torch.Generator().manual_seed(52)
    x, dy, w = ((torch.rand(*s, generator=g) * 0.5 + 0.5).to(BF)
                for s in ((R, n_in), (R, n_out), (2, n_out, n_in)))
    sh = moe.GroupedShape(R, 2, n_in, n_out)
    ws = moe.alloc_grouped_workspace(sh)
    xd, dyd, wd, offd = dev(x, dy, w, off)
    y = moe.grouped_matmul(sh, xd, wd, offd, ws)
    dx = moe.grouped_matmul_dx(sh, dyd, wd, offd, ws)
    dw = moe.grouped_matmul_dw(sh, dyd, xd, offd, ws)
    assert moe.read_device_error(ws) == 0
    x, dy, w = x.double(), dy.double(), w.double()
    for e, lo, hi in ref.segments(off):
        for got, want, terms in ((y[lo:hi], x[lo:hi] @ w[e].T, n_in),
                                 (dx[lo:hi], dy[lo:hi] @ w[e], n_out),
                                 (dw[e], dy[lo:hi].T @ x[lo:hi], 16)):
            ref.check(got, want, max(terms // 16, 16) * ref.U / 2 * want, BF, f"{terms} terms")


def test_grouped_large_batches():
    # enough rows per group for the largest tiles of every path
    check_grouped((1030, 511, 0, 1290), 512, 768, BF, slack=100, seed=6)
    check_grouped((4100,), 264, 520, BF, seed=7)


def test_grouped_offsets_outside_the_rows_stay_in_bounds():
    # offsets are clamped: past the capacity they mean the last row, a segment
    # that ends before it starts is empty
    for dtype in (BF, F32):
        sh = moe.GroupedShape(40, 3, 64, 64, dtype)
        ws = moe.alloc_grouped_workspace(sh)
        g = torch.Generator().manual_seed(8)
        x, w = ref.random(g, 40, 64, dtype=dtype), ref.random(g, 3, 64, 64, dtype=dtype)
        off = torch.tensor([-5, 30, 20, 900], dtype=torch.int32)
        y = torch.full((40, 64), 7.0, dtype=dtype, device=DEV)
        xd, wd, offd = dev(x, w, off)
        moe.grouped_matmul(sh, xd, wd, offd, ws, out=y)
        dw = moe.grouped_matmul_dw(sh, xd, xd, offd, ws)
        assert moe.read_device_error(ws) == 0
        ref.check(y[:20], *ref.mm(x[:20].double(), w[0].double().T), dtype, "first")
        assert int(dw[1].count_nonzero()) == 0


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("off", [(-5, 30, 20, 900), (0, 300, 0, 300, 0, 300, 0),
                                 (250, 10, 260, 255, 270, 2 ** 31 - 1), (0, 290, 40, 120, 295)],
                         ids=str)
def test_grouped_offsets_that_fall_give_no_row_to_two_groups(off, dtype):
    # an offset counts as the largest up to it, within the rows; rows before
    # the first segment and behind the last are left as they were
    R, I, O, G = 300, 136, 72, len(off) - 1
    ends = torch.tensor(off).clamp(0, R).cummax(0).values.int()
    sh = moe.GroupedShape(R, G, I, O, dtype)
    ws = moe.alloc_grouped_workspace(sh)
    g = torch.Generator().manual_seed(9)
    x, dy, w = (ref.random(g, *s, dtype=dtype) for s in ((R, I), (R, O), (G, O, I)))
    y, dx = (torch.full((R, n), 7.0, dtype=dtype, device=DEV) for n in (O, I))
    offd = torch.tensor(off, dtype=torch.int32, device=DEV)
    xd, dyd, wd = dev(x, dy, w)
    for _ in range(3):
        moe.grouped_matmul(sh, xd, wd, offd, ws, out=y)
        moe.grouped_matmul_dx(sh, dyd, wd, offd, ws, out=dx)
        dw = moe.grouped_matmul_dw(sh, dyd, xd, offd, ws)
    assert moe.read_device_error(ws) == 0
    x, dy, w = x.double(), dy.double(), w.double()
    for e, lo, hi in ref.segments(ends):
        ref.check(y[lo:hi], *ref.mm(x[lo:hi], w[e].T), dtype, f"y of {e}")
        ref.check(dx[lo:hi], *ref.mm(dy[lo:hi], w[e]), dtype, f"dx of {e}")
        ref.check(dw[e], *ref.mm(dy[lo:hi].T, x[lo:hi]), dtype, f"dw of {e}")
    for t in (y, dx):
        assert bool((t[:int(ends[0])] == 7.0).all()) and bool((t[int(ends[-1]):] == 7.0).all())


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_expert_ffn_backward_with_offsets_that_fall(dtype):
    T, d, N, F = 90, 64, 4, 40
    off = torch.tensor([0, 70, 30, 85, 20], dtype=torch.int32)  # as 0, 70, 70, 85, 85
    g = torch.Generator().manual_seed(12)
    mk = lambda *s, sc=1.0: ref.random(g, *s, dtype=dtype, scale=sc)  # noqa: E731
    x, dy = mk(T, d), mk(T, d)
    wg, wu, wd = (mk(*s, sc=d ** -0.5) for s in ((N, F, d), (N, F, d), (N, d, F)))
    sh = moe.LayerShape(T, d, N, 1, 1, F, dtype)
    ws = moe.alloc_backward_workspace(sh)
    dx = torch.full(x.shape, 7.0, dtype=dtype, device=DEV)
    got = moe.expert_ffn_backward(sh, *dev(x, off, wg, wu, wd, dy), ws, dx_perm=dx)
    assert moe.read_device_error(ws) == 0
    want = ref.ffn_backward(x[:85], off.cummax(0).values, wg, wu, wd, dy[:85], dtype)
    ref.check(got[0][:85], *want[0], dtype, "dx")
    assert bool((got[0][85:] == 7.0).all())
    for a, (v, err) in zip(got[1:], want[1:]):
        ref.check(a, v, err, dtype, "weight gradient")


# ------------------------------------------------------- experts' backward --
def ffn_case(T, d, N, Z, k, F, dtype, seed, popular=None):
    g = torch.Generator().manual_seed(seed)
    idx, gate, slot_row, off = ref.route_by_hand(T, N, Z, k, g, popular)
    mk = lambda *s, sc=1.0: ref.random(g, *s, dtype=dtype, scale=sc)  # noqa: E731
    x_perm, dy = mk(T * k, d), mk(T * k, d)
    wg, wu, wd = (mk(*s, sc=d ** -0.5) for s in ((N, F, d), (N, F, d), (N, d, F)))
    return idx, gate, slot_row, off, x_perm, dy, wg, wu, wd


FFN = [dict(T=1, d=64, N=3, Z=1, k=2, F=32), dict(T=40, d=128, N=5, Z=2, k=3, F=64),
       dict(T=33, d=72, N=4, Z=0, k=1, F=40), dict(T=150, d=256, N=8, Z=2, k=2, F=384),
       dict(T=300, d=264, N=3, Z=1, k=2, F=136), dict(T=700, d=512, N=4, Z=1, k=3, F=256),
       dict(T=64, d=64, N=2, Z=6, k=2, F=64), dict(T=5, d=8, N=2, Z=0, k=1, F=8),
       dict(T=9, d=2048, N=3, Z=0, k=2, F=512)]


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("case", FFN, ids=lambda c: "-".join(str(v) for v in c.values()))
def test_expert_ffn_backward(case, dtype):
    idx, gate, slot_row, off, x, dy, wg, wu, wd = ffn_case(**case, dtype=dtype, seed=10)
    R = int(off[-1])
    x[R:], dy[R:] = float("nan"), float("nan")
    sh = moe.LayerShape(case["T"], case["d"], case["N"], case["Z"], case["k"], case["F"], dtype)
    ws = moe.alloc_backward_workspace(sh)
    dx = torch.full(x.shape, 7.0, dtype=dtype, device=DEV)
    got = moe.expert_ffn_backward(sh, *dev(x, off, wg, wu, wd, dy), ws, dx_perm=dx)
    assert moe.read_device_error(ws) == 0
    want = ref.ffn_backward(x[:R], off, wg, wu, wd, dy[:R], dtype)
    ref.check(got[0][:R], *want[0], dtype, "dx")
    assert bool((got[0][R:] == 7.0).all())
    for name, a, (v, err) in zip(("dw_gate", "dw_up", "dw_down"), got[1:], want[1:]):
        assert a.dtype == dtype
        ref.check(a, v, err, dtype, name)


def test_expert_ffn_backward_fp32_gradients_and_hot_expert():
    case = dict(T=600, d=256, N=6, Z=1, k=2, F=256)
    idx, gate, slot_row, off, x, dy, wg, wu, wd = ffn_case(**case, dtype=BF, seed=11, popular=2)
    R = int(off[-1])
    sh = moe.LayerShape(600, 256, 6, 1, 2, 256, BF)
    ws = moe.alloc_backward_workspace(sh)
    grads = [torch.full(w.shape, 7.0, device=DEV) for w in (wg, wu, wd)]
    got = moe.expert_ffn_backward(sh, *dev(x, off, wg, wu, wd, dy), ws, dw_gate=grads[0],
                                  dw_up=grads[1], dw_down=grads[2])
    assert moe.read_device_error(ws) == 0 and got[1] is grads[0]
    want = ref.ffn_backward(x[:R], off, wg, wu, wd, dy[:R], BF)
    for a, (v, err) in zip(grads, want[1:]):
        ref.check(a, v, err, F32, "fp32 gradient")


# -------------------------------------------------- combine and the input --
LAYER = [dict(T=1, d=64, N=3, Z=1, k=2), dict(T=37, d=72, N=5, Z=3, k=4),
         dict(T=20, d=520, N=0, Z=4, k=3), dict(T=65, d=136, N=40, Z=0, k=12),
         dict(T=12, d=4104, N=30, Z=10, k=32), dict(T=300, d=64, N=4, Z=2, k=1),
         dict(T=1500, d=72, N=3, Z=2, k=3), dict(T=2100, d=136, N=5, Z=2, k=3),
         dict(T=2049, d=520, N=0, Z=9, k=9), dict(T=40, d=64, N=1000, Z=24, k=32)]
IDS = lambda c: "-".join(str(v) for v in c.values())  # noqa: E731


def layer_case(c, dtype, seed, popular=None):
    g = torch.Generator().manual_seed(seed)
    T, d, N, Z, k = (c[n] for n in ("T", "d", "N", "Z", "k"))
    idx, gate, slot_row, off = ref.route_by_hand(T, N, Z, k, g, popular)
    dout, x = ref.random(g, T, d, dtype=dtype), ref.random(g, T, d, dtype=dtype)
    rows = ref.random(g, T * k, d, dtype=dtype)
    rows[int(off[-1]):] = float("nan")  # behind the routed rows
    w_r = ref.random(g, N + Z, d, scale=d ** -0.5)
    dgate = ref.random(g, T, k)
    return idx, gate, slot_row, off, dout, x, rows, w_r, dgate


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("c", LAYER, ids=IDS)
def test_combine_backward(c, dtype):
    idx, gate, slot_row, off, dout, x, y, _, _ = layer_case(c, dtype, 20)
    T, d, N, Z, k = (c[n] for n in ("T", "d", "N", "Z", "k"))
    sh = moe.LayerShape(T, d, N, Z, k, 8, dtype, 2.5)
    dy = torch.full(y.shape, 7.0, dtype=dtype, device=DEV)
    got, dgate = moe.combine_backward(sh, *dev(dout, x, y, idx, gate, slot_row), dy_perm=dy)
    R = int(off[-1])
    (v, ev), (g, eg) = ref.combine_backward(dout, x, y, idx, gate, slot_row, N, 2.5)
    ref.check(got[:R], v[:R], ev[:R].nan_to_num(), dtype, "dy_perm")
    assert bool((got[R:] == 7.0).all())
    ref.check(dgate, g, eg, F32, "dgate")


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("popular", [None, 1])
@pytest.mark.parametrize("c", LAYER, ids=IDS)
def test_input_backward(c, popular, dtype):
    idx, gate, slot_row, off, dout, x, rows, w_r, dgate = layer_case(c, dtype, 21, popular)
    T, d, N, Z, k = (c[n] for n in ("T", "d", "N", "Z", "k"))
    sh = moe.LayerShape(T, d, N, Z, k, 8, dtype, 2.5)
    ws = moe.alloc_backward_workspace(sh)
    dx, dw = moe.input_backward(sh, *dev(dout, x, w_r, idx, gate, slot_row, dgate, rows), ws)
    assert moe.read_device_error(ws) == 0
    want = ref.input_backward(dout, x, w_r, idx, gate, slot_row, dgate, rows, N)
    ref.check(dx, *want[0], dtype, "dx")
    ref.check(dw, *want[1], F32, "dw_router")
    unused = torch.bincount(idx.view(-1).long(), minlength=N + Z) == 0
    assert int(dw.cpu()[unused].count_nonzero()) == 0


def test_invalid_ids_stay_in_bounds_and_are_reported():
    c = dict(T=50, d=64, N=4, Z=2, k=3)
    idx, gate, slot_row, off, dout, x, rows, w_r, dgate = layer_case(c, BF, 22)
    rows = torch.where(rows.isnan(), 0.0, rows).to(BF)
    idx[3, 1], idx[7, 0] = 99, -4
    slot_row.view(50, 3)[3, 1] = slot_row.view(50, 3)[7, 0] = -1
    sh = moe.LayerShape(50, 64, 4, 2, 3, 8, BF)
    ws = moe.alloc_backward_workspace(sh)
    a = dev(dout, x, rows, idx, gate, slot_row)
    _, dg = moe.combine_backward(sh, *a)
    assert float(dg[3, 1]) == 0.0 and float(dg[7, 0]) == 0.0
    dx, _ = moe.input_backward(sh, a[0], a[1], dev(w_r), a[3], a[4], a[5], dev(dgate), a[2], ws)
    assert moe.read_device_error(ws) == 2
    assert moe.read_device_error(ws) == 0
    assert bool(torch.isfinite(dx).all())


def test_a_slot_with_an_invalid_id_adds_no_router_row():
    # not even zero times a row that holds no number
    c = dict(T=50, d=64, N=4, Z=2, k=3)
    idx, gate, slot_row, off, dout, x, rows, w_r, dgate = layer_case(c, BF, 23)
    rows = torch.where(rows.isnan(), 0.0, rows).to(BF)
    idx[5] = torch.tensor([1, -1, 2])
    slot_row.view(50, 3)[5] = torch.tensor([0, -1, 1])
    w_r[0] = float("nan")
    sh = moe.LayerShape(50, 64, 4, 2, 3, 8, BF)
    ws = moe.alloc_backward_workspace(sh)
    dx, _ = moe.input_backward(sh, *dev(dout, x, w_r, idx, gate, slot_row, dgate, rows), ws)
    assert moe.read_device_error(ws) == 2
    assert bool(torch.isfinite(dx[5]).all())


# ------------------------------------------------------------ whole layer --
def forward(ls, x, w_r, bias, wg, wu, wd):
    ws = moe.alloc_workspace(ls)
    idx, gate = moe.route(ls, x, w_r, bias, ws)
    _, off, _, slot_row, x_perm = moe.dispatch(ls, x, idx, ws)
    y_perm = moe.expert_ffn(ls, x_perm, off, wg, wu, wd, ws)
    out = moe.combine(ls, x, y_perm, idx, gate, slot_row)
    assert moe.read_device_error(ws) == 0
    return out, idx, gate, off, slot_row, x_perm, y_perm


def weights(ls, seed):
    g = torch.Generator().manual_seed(seed)
    N, F, d, dt = ls.n_routed, ls.ffn, ls.d, ls.act_dtype
    mk = lambda *s: ref.random(g, *s, dtype=dt, scale=d ** -0.5)  # noqa: E731
    x, dout = ref.random(g, ls.T, d, dtype=dt), ref.random(g, ls.T, d, dtype=dt)
    w_r = ref.random(g, ls.E, d, scale=d ** -0.5)
    return dev(x, dout, w_r, torch.zeros(ls.E), mk(N, F, d), mk(N, F, d), mk(N, d, F))


WHOLE = [moe.LayerShape(1, 128, 4, 2, 3, 128, BF, 2.0),
         moe.LayerShape(130, 256, 6, 2, 3, 128, BF, 9.0),
         moe.LayerShape(90, 72, 5, 1, 2, 40, BF, 1.0),
         moe.LayerShape(60, 128, 4, 2, 2, 64, F32, 1.5),
         moe.LayerShape(25, 64, 0, 3, 2, 8, F32, 1.0)]


@pytest.mark.parametrize("ls", WHOLE, ids=lambda s: f"{s.T}-{s.d}-{s.n_routed}-{s.act_dtype}")
def test_layer_backward(ls):
    x, dout, w_r, bias, wg, wu, wd = weights(ls, 30)
    _, idx, gate, off, slot_row, xp, yp = forward(ls, x, w_r, bias, wg, wu, wd)
    ws = moe.alloc_backward_workspace(ls)
    got = moe.layer_backward(ls, dout, x, w_r, wg, wu, wd, idx, gate, off, slot_row, xp, yp, ws)
    # the staged calls give the same, bit for bit
    dy, dgate = moe.combine_backward(ls, dout, x, yp, idx, gate, slot_row)
    if ls.n_routed:
        dxp, *dws = moe.expert_ffn_backward(ls, xp, off, wg, wu, wd, dy, ws)
    else:
        dxp, dws = torch.zeros_like(dy), [wg, wu, wd]
    dx, dw_r = moe.input_backward(ls, dout, x, w_r, idx, gate, slot_row, dgate, dxp, ws)
    assert moe.read_device_error(ws) == 0
    for a, b in zip(got, (dx, dw_r, *dws)):
        assert torch.equal(a, b)
    # and the formulas, from what the forward pass left
    c = lambda t: t.cpu()  # noqa: E731
    R = int(off[-1])
    (v, ev), (g, eg) = ref.combine_backward(c(dout), c(x), c(yp), c(idx), c(gate), c(slot_row),
                                            ls.n_routed, ls.routed_scale)
    ref.check(dy[:R], v[:R], ev[:R], ls.act_dtype, "dy")
    ref.check(dgate, g, eg, F32, "dgate")
    if ls.n_routed:
        want = ref.ffn_backward(c(xp)[:R], c(off), c(wg), c(wu), c(wd), c(dy)[:R], ls.act_dtype)
        for a, (w, e) in zip((dxp[:R], *dws), want):
            ref.check(a, w, e, ls.act_dtype, "expert gradient")
    want = ref.input_backward(c(dout), c(x), c(w_r), c(idx), c(gate), c(slot_row), c(dgate),
                              c(dxp), ls.n_routed)
    ref.check(dx, *want[0], ls.act_dtype, "dx")
    ref.check(dw_r, *want[1], F32, "dw_router")


def test_layer_gradient_against_differences():
    """The f32 layer's own forward pass, moved along random directions: the
    change of <dout, out> agrees with the gradients (the selection is fixed by
    a bias that no step can outweigh)."""
    ls = moe.LayerShape(48, 64, 4, 2, 2, 32, F32, 1.5)
    x, dout, w_r, bias, wg, wu, wd = weights(ls, 31)
    bias = dev(torch.tensor([300.0, 0, 100.0, 0, 0, 0]))
    _, idx, gate, off, slot_row, xp, yp = forward(ls, x, w_r, bias, wg, wu, wd)
    ws = moe.alloc_backward_workspace(ls)
    dx, dw_r, dwg, dwu, dwd = moe.layer_backward(ls, dout, x, w_r, wg, wu, wd, idx, gate, off,
                                                 slot_row, xp, yp, ws)
    args = dict(x=x, w_r=w_r, wg=wg, wu=wu, wd=wd)
    for name, grad in (("x", dx), ("w_r", dw_r), ("wg", dwg), ("wu", dwu), ("wd", dwd)):
        g = torch.Generator().manual_seed(32)
        step = dev(torch.randn(grad.shape, generator=g))
        step /= step.norm()
        h = 2.0 ** -5
        vals, size = [], 0.0
        for sign in (1, -1):
            moved = dict(args)
            moved[name] = args[name] + sign * h * step
            out = forward(ls, moved["x"], moved["w_r"], bias, moved["wg"], moved["wu"],
                          moved["wd"])[0]
            prod = dout.double() * out.double()
            vals.append(float(prod.sum()))
            size = max(size, float(prod.square().sum().sqrt()))
        num = (vals[0] - vals[1]) / (2 * h)
        want = float((grad.double() * step.double()).sum())
        # rounding: out is off by at most about (d + F) 2^-23 of its size per
        # element, at random, over the difference 2 h; truncation: h^2 / 6 of a
        # third derivative along a unit step that is below 20 times the first's
        # own scale |grad|
        tol = 96 * ref.U * size / h + 20 * h * h / 6 * float(grad.norm())
        assert abs(num - want) <= tol, (name, num, want, tol)


def test_results_do_not_change_from_run_to_run_or_with_the_stream():
    ls = moe.LayerShape(1200, 256, 8, 2, 3, 256, BF, 2.0)
    x, dout, w_r, bias, wg, wu, wd = weights(ls, 33)
    _, idx, gate, off, slot_row, xp, yp = forward(ls, x, w_r, bias, wg, wu, wd)
    ws = moe.alloc_backward_workspace(ls)
    args = (ls, dout, x, w_r, wg, wu, wd, idx, gate, off, slot_row, xp, yp)
    first = moe.layer_backward(*args, ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    again = moe.layer_backward(*args, ws)
    torch.cuda.synchronize()
    other = moe.layer_backward(*args, moe.alloc_backward_workspace(ls), stream=side)
    torch.cuda.synchronize()
    for a, b, c in zip(first, again, other):
        assert torch.equal(a, b) and torch.equal(a, c)


@pytest.mark.parametrize("sizes", [(900, 0, 1700, 330, 20, 64, 321, 257), (300,) * 24],
                         ids=["skewed", "even"])
def test_many_units_and_runs_give_the_same_result(sizes):
    # hundreds of work units per launch handed from CTA pair to CTA pair, of
    # one and of several tiles: every run equals the first bit for bit
    R, N, d, F = sum(sizes), len(sizes), 1024, 1024
    g = torch.Generator(device=DEV).manual_seed(34)
    mk = lambda *s, sc=1.0: (torch.randn(*s, generator=g, device=DEV) * sc).to(BF)  # noqa: E731
    off = dev(ref.offsets_of(sizes))
    sh = moe.LayerShape(R, d, N, 1, 1, F, BF)
    ws = moe.alloc_backward_workspace(sh)
    x, dy = mk(R, d), mk(R, d)
    wg, wu, wd = (mk(*s, sc=d ** -0.5) for s in ((N, F, d), (N, F, d), (N, d, F)))
    first = moe.expert_ffn_backward(sh, x, off, wg, wu, wd, dy, ws)
    again = [torch.empty_like(t) for t in first]
    for run in range(40):
        moe.expert_ffn_backward(sh, x, off, wg, wu, wd, dy, ws, *again)
        assert all(torch.equal(a, b) for a, b in zip(first, again)), run
    assert moe.read_device_error(ws) == 0


def test_empty_batch_gives_zero_weight_gradients():
    ls = moe.LayerShape(0, 64, 2, 1, 2, 32, BF)
    e = lambda *s, dt=BF: torch.empty(*s, dtype=dt, device=DEV)  # noqa: E731
    i32 = torch.int32
    wg, wu, wd, w_r = e(2, 32, 64), e(2, 32, 64), e(2, 64, 32), e(3, 64, dt=F32)
    off = torch.zeros(3, dtype=i32, device=DEV)
    ws = moe.alloc_backward_workspace(ls)
    idx, gate = e(0, 2, dt=i32), e(0, 2, dt=F32)
    full = lambda *s, dt=BF: torch.full(s, 7.0, dtype=dt, device=DEV)  # noqa: E731
    grads = moe.layer_backward(ls, e(0, 64), e(0, 64), w_r, wg, wu, wd, idx, gate, off,
                               e(0, dt=i32), e(0, 64), e(0, 64), ws,
                               dw_router=full(3, 64, dt=F32), dw_gate=full(2, 32, 64),
                               dw_up=full(2, 32, 64), dw_down=full(2, 64, 32))
    assert all(int(g.count_nonzero()) == 0 for g in grads)
    gs = moe.GroupedShape(0, 2, 16, 8)
    dw = moe.grouped_matmul_dw(gs, e(0, 8), e(0, 16), off, moe.alloc_grouped_workspace(gs),
                               out=full(2, 8, 16))
    assert int(dw.count_nonzero()) == 0


def test_two_calls_at_once_on_two_streams():
    ls = moe.LayerShape(700, 512, 6, 2, 3, 512, BF, 2.0)
    x, dout, w_r, bias, wg, wu, wd = weights(ls, 35)
    _, idx, gate, off, slot_row, xp, yp = forward(ls, x, w_r, bias, wg, wu, wd)
    args = (ls, dout, x, w_r, wg, wu, wd, idx, gate, off, slot_row, xp, yp)
    spaces = [moe.alloc_backward_workspace(ls) for _ in range(3)]
    want = moe.layer_backward(*args, spaces[2])
    sides = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [[torch.empty_like(t) for t in want] for _ in sides]
    torch.cuda.synchronize()
    for _ in range(10):
        for side, ws, out in zip(sides, spaces, outs):
            moe.layer_backward(*args, ws, *out, stream=side)
    torch.cuda.synchronize()
    for ws, out in zip(spaces, outs):
        assert moe.read_device_error(ws) == 0
        assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_an_output_dropped_at_once_is_not_handed_out_while_the_call_writes_it():
    ls = moe.LayerShape(700, 512, 0, 8, 3, 8, BF)
    x, dout, w_r, bias, *_ = weights(ls, 36)
    g = torch.Generator().manual_seed(36)
    idx, gate, slot_row, _ = ref.route_by_hand(700, 0, 8, 3, g)
    idx, gate, slot_row, dgate = dev(idx, gate, slot_row, ref.random(g, 700, 3))
    ws, rows = moe.alloc_backward_workspace(ls), torch.zeros(2100, 512, dtype=BF, device=DEV)
    args = (ls, dout, x, w_r, idx, gate, slot_row, dgate, rows, ws)
    want, _ = moe.input_backward(*args)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)  # about 10 ms: the call waits behind it
    dx, dw = moe.input_backward(*args, stream=side)
    del dw
    # the current stream asks for the same size while the call is outstanding
    mine = [torch.full((8, 512), 7.0, device=DEV) for _ in range(8)]
    torch.cuda.synchronize()
    assert all(bool((t == 7.0).all()) for t in mine) and torch.equal(dx, want)


def test_calls_on_a_forked_stream_are_captured():
    # outputs not given, some dropped at once, on a stream that joins the capture;
    # and the optimizer on a stream that is only a handle
    ls = moe.LayerShape(90, 128, 4, 2, 2, 64, BF, 2.0)
    x, dout, w_r, bias, wg, wu, wd = weights(ls, 37)
    _, idx, gate, off, slot_row, xp, yp = forward(ls, x, w_r, bias, wg, wu, wd)
    args = (ls, dout, x, w_r, wg, wu, wd, idx, gate, off, slot_row, xp, yp)
    ws = moe.alloc_backward_workspace(ls)
    want = moe.layer_backward(*args, ws)
    p, grad = torch.ones(500, device=DEV), torch.ones(500, device=DEV)
    opt = moe.AdamW([p], [grad])
    side = torch.cuda.Stream()
    handle = types.SimpleNamespace(cuda_stream=side.cuda_stream)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        moe.layer_backward(*args, ws, stream=side)  # all outputs dropped
        got = moe.layer_backward(*args, ws, stream=side)
        moe.adamw_step(opt, lr=0.5, stream=handle)
        torch.cuda.current_stream().wait_stream(side)
        copies = [t.clone() for t in got]
        del got
    assert opt._captured
    for _ in range(3):
        for t in copies:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(copies, want))
    assert int(opt.state[0]) == 3 and moe.read_device_error(ws) == 0
    with torch.cuda.stream(side):
        moe.adamw_step(opt, lr=0.5)
    y = moe.combine(ls, x, yp, idx, gate, slot_row, stream=handle)
    torch.cuda.synchronize()
    assert int(opt.state[0]) == 4 and torch.equal(y, moe.combine(ls, x, yp, idx, gate, slot_row))


# ------------------------------------------- positions behind 2^31 elements --
def test_grouped_rows_behind_two_to_the_31():
    R, I, O, G = 360_000, 6144, 64, 3  # x and dx hold 2.2 G elements
    g = torch.Generator(device=DEV).manual_seed(36)
    x = torch.randn(R, I, generator=g, device=DEV, dtype=BF)
    dy = torch.randn(R, O, generator=g, device=DEV, dtype=BF)
    w = torch.randn(G, O, I, generator=g, device=DEV, dtype=BF) * I ** -0.5
    off = torch.tensor([0, 1, R - 700, R], dtype=torch.int32, device=DEV)
    sh = moe.GroupedShape(R, G, I, O)
    ws = moe.alloc_grouped_workspace(sh)
    y = moe.grouped_matmul(sh, x, w, off, ws)
    dx = moe.grouped_matmul_dx(sh, dy, w, off, ws)
    dw = moe.grouped_matmul_dw(sh, dy, x, off, ws)
    assert moe.read_device_error(ws) == 0
    c = lambda t: t.double().cpu()  # noqa: E731
    for e, lo, hi in ((0, 0, 1), (1, 200_000, 200_040), (1, R - 720, R - 700), (2, R - 700, R)):
        ref.check(y[lo:hi], *ref.mm(c(x[lo:hi]), c(w[e]).T), BF, f"y {lo}")
        ref.check(dx[lo:hi], *ref.mm(c(dy[lo:hi]), c(w[e])), BF, f"dx {lo}")
    ref.check(dw[2], *ref.mm(c(dy[R - 700:]).T, c(x[R - 700:])), BF, "dw")


def test_layer_rows_behind_two_to_the_31():
    T, d, N, Z, k = 45_000, 6144, 8, 0, 8  # 2.2 G elements of rows
    g = torch.Generator(device=DEV).manual_seed(37)
    idx = torch.rand(T, N, generator=g, device=DEV).argsort(1).int()
    gate = torch.softmax(torch.randn(T, k, generator=g, device=DEV), 1)
    # every token chose all eight experts: row e T + t
    slot_row = (idx.long() * T + torch.arange(T, device=DEV)[:, None]).int().view(-1)
    mk = lambda *s: torch.randn(*s, generator=g, device=DEV, dtype=BF)  # noqa: E731
    dout, x, rows, w_r = mk(T, d), mk(T, d), mk(T * k, d), mk(N, d).float()
    dgate = torch.randn(T, k, generator=g, device=DEV)
    sh = moe.LayerShape(T, d, N, Z, k, 8, BF, 1.5)
    dy, dg = moe.combine_backward(sh, dout, x, rows, idx, gate, slot_row)
    ws = moe.alloc_backward_workspace(sh)
    dx, _ = moe.input_backward(sh, dout, x, w_r, idx, gate, slot_row, dgate, rows, ws)
    assert moe.read_device_error(ws) == 0
    pick = torch.tensor([0, 1, T // 2, T - 2, T - 1], device=DEV)
    local = torch.arange(5 * k, dtype=torch.int32)  # the picked tokens' rows, gathered
    at = slot_row.view(T, k)[pick].reshape(-1).long()
    c = lambda t: t.cpu()  # noqa: E731
    (v, ev), (gv, eg) = ref.combine_backward(c(dout[pick]), c(x[pick]), c(rows[at]), c(idx[pick]),
                                             c(gate[pick]), local, N, 1.5)
    ref.check(dy[at], v, ev, BF, "dy_perm")
    ref.check(dg[pick], gv, eg, F32, "dgate")
    want, _ = ref.input_backward(c(dout[pick]), c(x[pick]), c(w_r), c(idx[pick]), c(gate[pick]),
                                 local, c(dgate[pick]), c(rows[at]), N)
    ref.check(dx[pick], *want, BF, "dx")


def test_adamw_elements_behind_two_to_the_31():
    n = 2 ** 31 + 1000
    p = torch.ones(n, dtype=BF, device=DEV)
    grad = torch.zeros(n, dtype=BF, device=DEV)
    grad[-300:], grad[:10] = 1.0, -1.0
    opt = moe.AdamW([p], [grad], state_bits=8)
    moe.adamw_step(opt, lr=0.25, beta1=0.5, beta2=0.5)
    # the first step moves an element by lr in its gradient's direction
    assert bool((p[-300:] == 0.75).all()) and bool((p[:10] == 1.25).all())
    assert bool((p[2 ** 31 - 1000:-300] == 1.0).all()) and bool((p[10:2000] == 1.0).all())


# ------------------------------------------------------------------ AdamW --
HYPER = dict(lr=2e-3, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1)
SETS = [[1], [255, 256, 257], [3, 1, 7, 5000, 0, 12], [70000, 9]]


def widen(q):
    code, scale = q
    return code.float() * scale.repeat_interleave(256)


def narrow(t, root):
    """e4m3 codes with a scale per 256 values, step by step in 32 bits."""
    b = t.view(-1, 256)
    scale = b.abs().amax(1, keepdim=True) * torch.tensor(1 / 448, dtype=F32)
    q = torch.where(scale > 0, b / scale, torch.zeros_like(b))
    if root:
        q = torch.where((q > 0) & (q < 2.0 ** -9), torch.full_like(q, 2.0 ** -9), q)
    return q.clamp(-448, 448).to(torch.float8_e4m3fn).view(-1), scale.view(-1)


def flat(ts):
    return torch.cat([torch.nn.functional.pad(t.float(), (0, -t.numel() % 256)) for t in ts])


class Plain:
    """AdamW in 32 bits on the CPU, every operation rounded by itself."""

    def __init__(self, weights, bits):
        self.p, self.bits, self.t = flat(weights), bits, 0
        self.m, self.r2 = torch.zeros_like(self.p), torch.zeros_like(self.p)
        self.qm = self.qr = None

    def step(self, grads, lr, beta1, beta2, eps, weight_decay):
        self.t += 1
        g, c = flat(grads), lambda v: torch.tensor(v, dtype=F32)  # noqa: E731
        m, v = self.m, self.r2
        if self.bits == 8 and self.qm is not None:
            m, r = widen(self.qm), widen(self.qr)
            v = r * r
        self.m = m * c(beta1) + g * c(1 - beta1)
        self.r2 = v * c(beta2) + (g * c(1 - beta2)) * g
        r = self.r2.double().sqrt().float()  # correctly rounded (the CPU's float sqrt is not)
        root, size = c(math.sqrt(1 - beta2 ** self.t)), c(lr / (1 - beta1 ** self.t))
        self.p = self.p * c(1 - lr * weight_decay) - (self.m / (r / root + c(eps))) * size
        if self.bits == 8:
            self.qm, self.qr = narrow(self.m, False), narrow(r, True)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("pdt,gdt,master", [(F32, F32, False), (BF, BF, True), (BF, F32, True),
                                            (BF, BF, False), (F32, BF, False)],
                         ids=["f32", "bf16-master", "bf16-f32grad", "bf16", "f32-bf16grad"])
@pytest.mark.parametrize("sizes", SETS, ids=str)
def test_adamw_steps(sizes, pdt, gdt, master, bits):
    g = torch.Generator().manual_seed(40)
    params = [ref.random(g, n, dtype=pdt, scale=0.1) for n in sizes]
    start = [p.clone() for p in params]
    pd = [dev(p) for p in params]
    md = [dev(p.float()) for p in params] if master else None
    gd = [torch.empty(n, dtype=gdt, device=DEV) for n in sizes]
    opt = moe.AdamW(pd, gd, state_bits=bits, master=md)
    plain = Plain(start, bits)
    for step in range(4):
        grads = [ref.random(g, n, dtype=gdt, scale=10.0 ** -step) for n in sizes]
        if step == 2:
            grads = [torch.zeros_like(t) for t in grads]
        for a, b in zip(gd, grads):
            a.copy_(b)
        before = plain.p.clone()
        moe.adamw_step(opt, **HYPER)
        plain.step(grads, **HYPER)
        # the states come from explicitly rounded operations: equal bit for bit
        if bits == 32:
            assert torch.equal(opt.m.cpu(), plain.m) and torch.equal(opt.v.cpu(), plain.r2)
        else:
            for mine, want in ((opt.m, plain.qm), (opt.v, plain.qr)):
                assert torch.equal(mine[1].cpu(), want[1])
                assert torch.equal(mine[0].cpu().float(), want[0].float())
        # the weights: the coefficients are rounded from doubles (half a unit),
        # and the quotient, its product and the difference a few units more
        got = flat([t.cpu() for t in (md or pd)])
        moved = (plain.p - before).abs() + before.abs() * HYPER["lr"]
        if pdt == BF and not master:
            plain.p = plain.p.to(BF).float()
            tol = 2.0 ** -7 * plain.p.abs() + 16 * ref.U * moved
        else:
            tol = 16 * ref.U * moved + 2 * ref.U * plain.p.abs()
        assert bool(((got - plain.p).abs() <= tol + 1e-38).all()), step
        plain.p = got  # the next step starts from the same weights
        if master:
            for p, w in zip(pd, md):
                assert torch.equal(p, w.to(BF))
    assert int(opt.state[0]) == 4


def test_adamw_states_of_very_small_and_large_values():
    # blocks whose scale or its reciprocal lies far from one, subnormal second
    # moments among them: the 8-bit states still equal the formulas'
    g = torch.Generator().manual_seed(43)
    grad = ref.random(g, 4 * 256)
    for b, size in enumerate((1e-20, 1e-30, 1e17, 1e-3)):
        grad[256 * b:256 * (b + 1)] *= size
    p, gd = torch.zeros(1024, device=DEV), dev(grad)
    opt, plain = moe.AdamW([p], [gd], state_bits=8), Plain([torch.zeros(1024)], 8)
    for _ in range(3):
        moe.adamw_step(opt, **HYPER)
        plain.step([grad], **HYPER)
        for mine, want in ((opt.m, plain.qm), (opt.v, plain.qr)):
            assert torch.equal(mine[1].cpu(), want[1])
            assert torch.equal(mine[0].cpu().float(), want[0].float())


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_against_64_bits(bits):
    g = torch.Generator().manual_seed(41)
    n = 3000
    p, grad = ref.random(g, n, scale=0.1), ref.random(g, n)
    m, v = ref.random(g, n, scale=0.1), ref.random(g, n).square() + 0.01
    pad = -n % 256
    fm, fv = (torch.nn.functional.pad(t, (0, pad)) for t in (m, v))
    sm, sv = (fm, fv) if bits == 32 else (narrow(fm, False), narrow(fv.double().sqrt().float(), True))
    pd, gd = dev(p, grad)
    opt = moe.AdamW([pd], [gd], state_bits=bits)
    opt.load_state(*(dev(t) if bits == 32 else dev(*t) for t in (sm, sv)), step=6)
    moe.adamw_step(opt, **HYPER)
    m64 = (sm if bits == 32 else widen(sm))[:n].double()
    v64 = (sv if bits == 32 else widen(sv).double().square())[:n].double()
    h = HYPER
    m64 = h["beta1"] * m64 + (1 - h["beta1"]) * grad.double()
    v64 = h["beta2"] * v64 + (1 - h["beta2"]) * grad.double().square()
    upd = (m64 / (1 - h["beta1"] ** 7)) / ((v64 / (1 - h["beta2"] ** 7)).sqrt() + h["eps"])
    want = p.double() * (1 - h["lr"] * h["weight_decay"]) - h["lr"] * upd
    # fp32: a sum of two terms in m (2 units of its larger term, which may
    # cancel), 8 more units through root, quotients and product
    terms = h["beta1"] * sm[:n].abs().double() if bits == 32 else \
        h["beta1"] * widen(sm)[:n].abs().double()
    m_err = 2 * ref.U * (terms + 0.1 * grad.abs().double())
    scale = upd.abs() / m64.abs().clamp(min=1e-30)
    tol = h["lr"] * (scale * m_err + 16 * ref.U * upd.abs()) + 2 * ref.U * p.abs().double()
    assert bool(((pd.cpu().double() - want).abs() <= tol).all())


def test_adamw_refuses_weights_that_moved():
    p, grad = torch.ones(300, device=DEV), torch.ones(300, device=DEV)
    opt = moe.AdamW([p], [grad])
    memory = grad.data_ptr()
    grad.data = torch.zeros(300, device=DEV)  # the step's buffer stays alive
    assert torch.empty(300, device=DEV).data_ptr() != memory
    keep = p.data
    p.data = p.data.clone()
    with pytest.raises(ValueError, match="moved"):
        moe.adamw_step(opt, **HYPER)
    p.data = keep
    moe.adamw_step(opt, **HYPER)
    assert int(opt.state[0]) == 1 and bool((p < 1).all())


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_refuses_masters_and_states_that_moved(bits):
    p, grad = torch.ones(300, dtype=BF, device=DEV), torch.ones(300, dtype=BF, device=DEV)
    opt = moe.AdamW([p], [grad], state_bits=bits, master=[p.float()])
    parts = [opt.master[0], opt.state, *((opt.m, opt.v) if bits == 32 else (*opt.m, *opt.v))]
    for t in parts:  # as a loaded checkpoint would be put in their place
        keep = t.data
        t.data = keep.clone()
        with pytest.raises(ValueError, match="moved"):
            moe.adamw_step(opt, **HYPER)
        t.data = keep
    for name in ("m", "v"):  # a state of another size would be written past its end
        keep = getattr(opt, name)
        setattr(opt, name, torch.zeros(256, device=DEV) if bits == 32
                else tuple(t.clone() for t in keep))
        with pytest.raises(ValueError, match="moved"):
            moe.adamw_step(opt, **HYPER)
        setattr(opt, name, keep)
    assert int(opt.state[0]) == 0 and bool((p == 1).all())
    moe.adamw_step(opt, **HYPER)
    assert int(opt.state[0]) == 1 and bool((opt.master[0] < 1).all())


def test_adamw_steps_from_gradients_that_moved():
    # first gradients of one sign, then others in new memory of the other sign:
    # every step follows what the gradients hold; a replay reads its capture's
    # five quotients within 2 units of 2^-23, times lr and rounded: 5 * 2^-22
    at = lambda v: bool(((p - v).abs() <= 5 * 2.0 ** -22).all())  # noqa: E731
    p = torch.zeros(700, device=DEV)
    grad = torch.ones(700, device=DEV)
    opt = moe.AdamW([p], [grad])
    h = dict(lr=0.5, beta1=0.0, beta2=0.0)  # a step moves every weight by lr
    moe.adamw_step(opt, **h)
    assert at(-0.5)
    grad.data = torch.full((700,), -3.0, device=DEV)
    moe.adamw_step(opt, **h)
    assert at(0.0)
    opt.grads[0] = torch.full((700,), 2.0, device=DEV)
    moe.adamw_step(opt, **h)
    assert at(-0.5)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.adamw_step(opt, **h)
    kept = opt.grads[0]
    opt.grads[0] = torch.full((700,), -1.0, device=DEV)
    moe.adamw_step(opt, **h)
    assert at(0.0)
    kept.fill_(5.0)
    del kept
    graph.replay()
    assert at(-0.5) and int(opt.state[0]) == 5


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_step_of_no_elements_counts(bits):
    none = torch.empty(0, device=DEV)
    opt = moe.AdamW([none], [none.clone()], state_bits=bits)
    for _ in range(3):
        moe.adamw_step(opt, **HYPER)
    assert opt.state.tolist() == [3, 0]


def test_adamw_blocks_before_the_first_tensor_belong_to_none():
    # the tensor owns blocks 2 and 3; what lies before it in memory stays
    buf, grad = torch.ones(1024, device=DEV), torch.ones(1024, device=DEV)
    opt = moe.AdamW([buf], [grad])
    opt._table[0, 0] += 512 * 4
    opt._table[0, 2] += 512 * 4
    opt._table[0, 3], opt._table[0, 4] = 512, 2
    moe.adamw_step(opt, **HYPER)
    assert bool((buf[:512] == 1).all()) and bool((buf[512:] < 1).all())
    assert int(opt.m[:512].count_nonzero()) == 0 and bool((opt.m[512:] > 0).all())


def test_adamw_values_that_are_not_numbers_are_not_hidden():
    for bits in (32, 8):
        grad = torch.ones(600, device=DEV)
        grad[300] = float("nan")
        p = torch.ones(600, device=DEV)
        opt = moe.AdamW([p], [grad], state_bits=bits)
        moe.adamw_step(opt, lr=1e-2)
        assert bool(p[300].isnan()) and int(p.isnan().sum()) == 1
        m = opt.m if bits == 32 else widen(opt.m)
        assert bool(m[300].isnan())
        assert not bool(m[:256].isnan().any()) and not bool(m[512:].isnan().any())


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_step_is_captured_and_counts_on(bits):
    g = torch.Generator().manual_seed(42)
    p0 = [ref.random(g, n, dtype=BF) for n in (777, 2000)]
    grads = [dev(ref.random(g, n, dtype=BF)) for n in (777, 2000)]

    def fresh():
        p = [dev(t) for t in p0]
        return p, moe.AdamW(p, grads, state_bits=bits, master=[t.float() for t in p])

    p1, eager = fresh()
    for _ in range(5):
        moe.adamw_step(eager, **HYPER)
    p2, opt = fresh()
    moe.adamw_step(opt, **HYPER)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.adamw_step(opt, **HYPER)
    for _ in range(4):
        graph.replay()
    torch.cuda.synchronize()
    assert int(opt.state[0]) == 5
    for a, b in zip(p1 + eager.master, p2 + opt.master):
        assert torch.equal(a, b)


# ------------------------------------------------------------- all of it --
def train_step(ls, st):
    """Forward, backward and update of one layer, as a training loop has them."""
    idx, gate = moe.route(ls, st["x"], st["w_r"], st["bias"], st["fws"])
    _, off, _, slot_row, xp = moe.dispatch(ls, st["x"], idx, st["fws"])
    yp = moe.expert_ffn(ls, xp, off, *st["w"], st["fws"], y_perm=st["yp"])
    moe.combine(ls, st["x"], yp, idx, gate, slot_row, out=st["out"])
    torch.sub(st["out"], st["target"], out=st["dout"])
    moe.layer_backward(ls, st["dout"], st["x"], st["w_r"], *st["w"], idx, gate, off, slot_row,
                       xp, yp, st["bws"], dx=st["dx"], dw_router=st["dw_r"], dw_gate=st["dw"][0],
                       dw_up=st["dw"][1], dw_down=st["dw"][2])
    moe.adamw_step(st["opt"], lr=1e-3)
    moe.adamw_step(st["opt_r"], lr=1e-3)


def train_state(ls, seed):
    x, target, w_r, bias, wg, wu, wd = weights(ls, seed)
    st = dict(x=x, target=target, w_r=w_r, bias=bias, w=[wg, wu, wd],
              fws=moe.alloc_workspace(ls), bws=moe.alloc_backward_workspace(ls))
    st["out"], st["dout"], st["dx"] = (torch.empty_like(x) for _ in range(3))
    st["yp"] = torch.zeros(ls.T * ls.top_k, ls.d, dtype=ls.act_dtype, device=DEV)
    st["dw_r"], st["dw"] = torch.empty_like(w_r), [torch.empty_like(w) for w in st["w"]]
    st["opt"] = moe.AdamW(st["w"], st["dw"], state_bits=8, master=[w.float() for w in st["w"]])
    st["opt_r"] = moe.AdamW([w_r], [st["dw_r"]])
    return st


def test_training_steps_captured_and_eager_agree():
    ls = moe.LayerShape(200, 256, 6, 2, 3, 128, BF, 2.0)
    eager, st = train_state(ls, 50), train_state(ls, 50)
    for _ in range(4):
        train_step(ls, eager)
    train_step(ls, st)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        train_step(ls, st)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for s in (eager, st):
        assert moe.read_device_error(s["fws"]) == 0 and moe.read_device_error(s["bws"]) == 0
        assert all(bool(torch.isfinite(t).all()) for t in [s["dx"], s["dw_r"], *s["dw"], *s["w"]])
    for a, b in zip([eager["dx"], eager["w_r"], *eager["w"], *eager["dw"]],
                    [st["dx"], st["w_r"], *st["w"], *st["dw"]]):
        assert torch.equal(a, b)
