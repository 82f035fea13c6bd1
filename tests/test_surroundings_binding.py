"""What the binding of the surrounding operators checks and keeps, on host tensors (no GPU needed): nothing here
reaches a launch."""
import ctypes

import pytest
import torch

from residual_binarized_weight_b200 import build as rbw_build
from residual_binarized_weight_b200 import rbw
from tests.test_surroundings_abi import A, B, K, M, N, backward, epilogue, grad, layer, linear, no_device, qat


@pytest.fixture(autouse=True)
def library():
    rbw_build.build()


def tensor(n=300, bits=32, **kw):
    p = torch.zeros(n)
    return rbw.AdamWTensor(p, torch.zeros(n), **(rbw.AdamWTensor.new_state(p, bits) | kw))


def test_the_optimizer_follows_what_is_assigned():
    """The table's row of a tensor whose gradient, state, rate or decay was assigned, as the next step takes it."""
    ts = [tensor(bits=b) for b in (32, 8, 32)]
    opt = rbw.AdamW(ts)
    old = [opt._table[i].grad for i in range(3)]
    new = torch.ones(300)
    ts[1].grad, ts[1].lr, ts[1].weight_decay = new, 0.5, 0.25
    with pytest.raises((rbw.RbError, ValueError, RuntimeError, AssertionError)):     # no device here, or not the tensors'
        opt.step(1)
    row = opt._table[1]
    assert row.grad == new.data_ptr() and row.lr == 0.5 and row.weight_decay == 0.25
    assert opt._table[0].grad == old[0] and opt._table[2].grad == old[2]
    ts[0].grad = torch.zeros(300, dtype=torch.bfloat16)
    opt._follow()
    assert (opt._table[0].grad, opt._table[0].grad_dtype) == (ts[0].grad.data_ptr(), rbw.RB_BF16)
    assert opt._table[0].exp_avg == ts[0].exp_avg.data_ptr()
    ts[2].exp_avg = torch.zeros(300)
    other = rbw.AdamW(ts)                                                            # a second list over the same tensors
    opt._follow()
    assert opt._table[2].exp_avg == other._table[2].exp_avg == ts[2].exp_avg.data_ptr()
    assert [bytes(x) for x in opt._table] == [bytes(x) for x in other._table]


@pytest.mark.parametrize("name,value", [
    ("grad", torch.zeros(299)), ("grad", torch.zeros(600)[::2]), ("grad", torch.zeros(300).half()), ("grad", None),
    ("exp_avg", torch.zeros(301)), ("exp_avg_sq", torch.zeros(300).to(torch.float8_e4m3fn)), ("param", torch.zeros(10))])
def test_the_optimizer_refuses_what_does_not_fit(name, value):
    t = tensor()
    opt = rbw.AdamW([t])
    before = bytes(opt._table)
    setattr(t, name, value)
    with pytest.raises(ValueError):
        opt.step(1)
    assert bytes(opt._table) == before


def test_a_list_stays_as_it_was_made():
    ts = [tensor(), tensor()]
    opt = rbw.AdamW(ts)
    ts.pop()
    assert len(opt.tensors) == 2
    with pytest.raises(TypeError):
        opt.tensors[0] = tensor()


def test_shapes_count_and_not_only_element_numbers(monkeypatch):
    """Scales and gradients whose elements would pair up wrongly; flat states and flat gradients still fit."""
    monkeypatch.setattr(rbw, "_current", lambda stream: (-1, 0))
    N, K, k = 64, 96, 2
    W, X = torch.zeros(N, K), torch.zeros(3, K, dtype=torch.bfloat16)
    g, h = torch.zeros(k, N), torch.zeros(k, K)
    for bad in (dict(g=torch.zeros(N, k)), dict(g=torch.zeros(k * N)), dict(h=torch.zeros(K, k)), dict(h=torch.zeros(1, k * K))):
        a = dict(g=g, h=h) | bad
        with pytest.raises(ValueError):
            rbw.qat_linear(W, a["g"], a["h"], k, X)
    p = torch.zeros(6, 50)
    state = rbw.AdamWTensor.new_state(p)
    for shape in ((50, 6), (300, 1), (3, 100)):
        with pytest.raises(ValueError):
            rbw.AdamWTensor(p, torch.zeros(shape), **state)
        with pytest.raises(ValueError):
            rbw.AdamWTensor(p, torch.zeros(6, 50), **(state | dict(exp_avg=torch.zeros(shape))))
    rbw.AdamWTensor(p, torch.zeros(6, 50), **state)
    rbw.AdamWTensor(p, torch.zeros(300), **state)
    rbw.AdamWTensor(torch.zeros(300), torch.zeros(6, 50), **state)
    rbw.AdamWTensor(p, torch.zeros(6, 50), **rbw.AdamWTensor.new_state(p, 8))


def test_memory_that_is_not_in_one_piece_is_refused(monkeypatch):
    """A workspace with gaps, whose bytes in between belong to others, and scales of another type or with gaps."""
    monkeypatch.setattr(rbw, "_current", lambda stream: (-1, 0))
    layer = rbw.PackedLayer(64, 96, 2, "cpu")
    X, d = torch.zeros(3, 96, dtype=torch.bfloat16), torch.zeros(3, 64, dtype=torch.bfloat16)
    for ws in (torch.zeros(1 << 20, 2, dtype=torch.uint8)[:, 0], torch.zeros(1 << 12, 1 << 8).t()):
        with pytest.raises(ValueError):
            rbw.linear(layer, X, ws=ws)
        with pytest.raises(ValueError):
            rbw.qat_linear(torch.zeros(64, 96), torch.zeros(2, 64), torch.zeros(2, 96), 2, X, ws=ws)
        with pytest.raises(ValueError):
            rbw.epilogue_backward(d, d, act="relu", ws=ws)
    rbw.PackedLayer(64, 96, 2, "cpu", g16=torch.zeros(2, 64, dtype=torch.int16))           # bits of fp16
    for bad in (torch.zeros(2, 64), torch.zeros(64, 2).half().t(), torch.zeros(2, 64, dtype=torch.bfloat16),
                torch.zeros(2, 64, dtype=torch.uint8)):
        with pytest.raises(ValueError):
            rbw.PackedLayer(64, 96, 2, "cpu", g16=bad)
        with pytest.raises(ValueError):
            rbw.PackedLayer(96, 64, 2, "cpu", h16=bad)


# ---------------------------------------------------------------- the C entry points, on made-up addresses
FAR = 0x8000000                                                # planes, g16 and h16 of their own


@pytest.fixture
def L():
    return rbw.lib()


def at(**kw):
    return ctypes.byref(epilogue(**kw))


@pytest.mark.parametrize("name,size", [("planes", 2 * 256 * 2 * 4), ("g16", 2 * N * 2), ("h16", 2 * K * 2)])
@pytest.mark.parametrize("m", [1, M])
def test_outputs_over_the_layer_are_refused(L, name, size, m):
    lay = ctypes.byref(layer(**{name: FAR}))
    out = m * N * 2
    for Y in (FAR, FAR + size - 16, FAR - out + 16):
        assert linear(L, lay=lay, Y=Y, m=m) == rbw.RB_ERR_ARG
        assert linear(L, lay=lay, ep=at(preact=Y, ld_preact=N), m=m) == rbw.RB_ERR_ARG


@pytest.mark.parametrize("name,size", [("w", N * K * 4), ("g", 2 * N * 4), ("h", 2 * K * 4)])
def test_outputs_over_the_latent_weight_are_refused(L, name, size):
    for Y in (FAR, FAR + size - 16, FAR - M * N * 2 + 16):
        assert qat(L, Y=Y, **{name: FAR}) == rbw.RB_ERR_ARG
        assert qat(L, ep=at(preact=Y, ld_preact=N), **{name: FAR}) == rbw.RB_ERR_ARG


def test_outputs_over_the_workspace_are_refused(L):
    need = rbw.linear_workspace_bytes(N, K, 2, M)
    for Y in (FAR, FAR + need - 16, FAR - M * N * 2 + 16):
        assert linear(L, ws=FAR, Y=Y) == rbw.RB_ERR_ARG
        assert linear(L, ws=FAR, ep=at(preact=Y, ld_preact=N)) == rbw.RB_ERR_ARG
    need = rbw.qat_linear_workspace_bytes(N, K, 2, M)
    for Y in (FAR, FAR + need - 16):
        assert qat(L, ws=FAR, Y=Y) == rbw.RB_ERR_ARG
    need = rbw.epilogue_backward_workspace_bytes(M, N)
    for p in (FAR, FAR + (need - 1) // 16 * 16):
        assert backward(L, grad(dP=p), ws=FAR) == rbw.RB_ERR_ARG
        assert backward(L, grad(dmul=p), ws=FAR) == rbw.RB_ERR_ARG
        assert backward(L, grad(dbias=p), ws=FAR) == rbw.RB_ERR_ARG


@no_device
def test_outputs_beside_the_layer_and_the_workspace_are_taken(L):
    assert linear(L, ws=FAR, Y=FAR - M * N * 2) == rbw.RB_ERR_UNSUPPORTED
    assert linear(L, ws=FAR, Y=FAR + rbw.linear_workspace_bytes(N, K, 2, M)) == rbw.RB_ERR_UNSUPPORTED
    assert linear(L, lay=ctypes.byref(layer(planes=FAR)), Y=FAR + 4096) == rbw.RB_ERR_UNSUPPORTED
    assert linear(L, ws=FAR, wsb=0, m=1, Y=FAR) == rbw.RB_ERR_UNSUPPORTED      # one token leaves it alone
    assert qat(L, w=FAR, Y=FAR + N * K * 4) == rbw.RB_ERR_UNSUPPORTED
    assert backward(L, grad(dP=A, dbias=None), ws=A) == rbw.RB_ERR_UNSUPPORTED  # no sums, no workspace
    assert backward(L, grad(dP=B), ws=FAR) == rbw.RB_ERR_UNSUPPORTED
