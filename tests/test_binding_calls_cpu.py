"""Every binding function reaches the library with the right arguments: with
an empty batch (T = 0) the library returns before it reads any pointer, so the
calls run here without a GPU. Host tensors stand in for device ones (the
binding's device checks are relaxed for this test only), and a stand-in
stream handle replaces torch's current stream."""
import types

import pytest
import torch

import expert_routing_dispatch_router_b200 as moe


@pytest.fixture
def relaxed(monkeypatch):
    real_need = moe._need

    def need(t, name, dtype, shape=None, on_device=True):
        real_need(t, name, dtype, shape, on_device=False)

    def ws_of(ws):
        return moe.ctypes.c_void_p(ws.data_ptr()), ws.numel() * ws.element_size()

    monkeypatch.setattr(moe, "_need", need)
    monkeypatch.setattr(moe, "_ws", ws_of)
    return types.SimpleNamespace(cuda_stream=0)


def test_every_call_with_an_empty_batch(relaxed):
    st = relaxed
    sh = moe.LayerShape(T=0, d=64, n_routed=2, n_zero=1, top_k=2, ffn=64)
    bf = torch.bfloat16
    x = torch.zeros(0, 64, dtype=bf)
    w_r, b = torch.zeros(3, 64), torch.zeros(3)
    wg, wd = torch.zeros(2, 64, 64, dtype=bf), torch.zeros(2, 64, 64, dtype=bf)
    ws = torch.zeros(moe.workspace_size(sh), dtype=torch.uint8)
    idx, gate = moe.route(sh, x, w_r, b, ws, stream=st)
    assert idx.shape == (0, 2) and gate.shape == (0, 2)
    moe.route_noalloc(sh, x, w_r, b, idx, gate, stream=st)
    counts, offsets, row_token, slot_row, x_perm = moe.dispatch(sh, x, idx, ws, stream=st)
    y = moe.expert_ffn(sh, x_perm, offsets, wg, wg, wd, ws, stream=st)
    out = moe.combine(sh, x, y, idx, gate, slot_row, stream=st)
    assert out.shape == (0, 64)
    out = moe.layer_forward(sh, x, w_r, b, wg, wg, wd, ws, stream=st)
    assert out.shape == (0, 64)
    moe.layer_forward_host(sh, x, w_r, b, wg, wg, wd, ws, torch.zeros(0, 64, dtype=bf),
                           stream=st)


def test_new_outputs_come_from_the_memory_of_their_own_stream(monkeypatch):
    """Every output that a call on another stream allocates is taken from that
    stream's memory, and the current stream is noted as its user: otherwise an
    output that the caller drops at once would be handed out again while the
    call still writes it. Device tensors are stand-ins here."""
    import contextlib
    current, side = (types.SimpleNamespace(cuda_stream=n, name=n) for n in (1, 2))
    active, made = [current], []

    class Fake:
        device = torch.device("cuda", 0)

        def __init__(self, dtype=None):
            self.dtype, self.owner, self.users = dtype, active[-1], []

        def record_stream(self, stream):
            self.users.append(stream)

    def empty(*shape, dtype, device):
        made.append(Fake(dtype))
        return made[-1]

    @contextlib.contextmanager
    def on(stream):
        active.append(stream)
        yield
        active.pop()

    class Library:
        def __getattr__(self, name):
            return lambda *args: 2 if name == "moe_ep_local_experts" else 0

    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: current)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device: side)
    monkeypatch.setattr(moe, "lib", lambda: Library())
    for name, value in (("_need", None), ("_on_current_device", None), ("_ptr", 0),
                        ("_ws", (0, 0))):
        monkeypatch.setattr(moe, name, lambda *a, value=value, **k: value)
    sh = moe.LayerShape(T=4, d=64, n_routed=2, n_zero=1, top_k=2, ffn=64)
    gs = moe.GroupedShape(8, 2, 16, 8)
    t = Fake()
    calls = [lambda **k: moe.route(sh, t, t, t, t, **k),
             lambda **k: moe.dispatch(sh, t, t, t, **k),
             lambda **k: moe.expert_ffn(sh, t, t, t, t, t, t, **k),
             lambda **k: moe.combine(sh, t, t, t, t, t, **k),
             lambda **k: moe.layer_forward(sh, t, t, t, t, t, t, t, **k),
             lambda **k: moe.ep_plan(sh, 0, 2, t, **k),
             lambda **k: moe.grouped_matmul(gs, t, t, t, t, **k),
             lambda **k: moe.grouped_matmul_dx(gs, t, t, t, t, **k),
             lambda **k: moe.grouped_matmul_dw(gs, t, t, t, t, **k),
             lambda **k: moe.combine_backward(sh, t, t, t, t, t, t, **k),
             lambda **k: moe.expert_ffn_backward(sh, t, t, t, t, t, t, t, **k),
             lambda **k: moe.input_backward(sh, t, t, t, t, t, t, t, t, t, **k),
             lambda **k: moe.layer_backward(sh, *[t] * 13, **k)]
    for call in calls:
        for stream in (current, side):
            made.clear()
            call(stream=stream)
            assert made and all(m.owner is stream for m in made)
            assert all((current in m.users) == (stream is side) for m in made)
    assert active == [current]
