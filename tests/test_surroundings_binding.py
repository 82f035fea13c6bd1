"""What the binding of the surrounding operators checks and keeps, on host tensors (no GPU needed): nothing here
reaches a launch."""
import pytest
import torch

from residual_binarized_weight_b200 import build as rbw_build
from residual_binarized_weight_b200 import rbw


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
    ts[2].exp_avg = torch.zeros(300)
    other = rbw.AdamW(ts)                                                            # a second list over the same tensors
    opt._follow()
    assert opt._table[2].exp_avg == other._table[2].exp_avg == ts[2].exp_avg.data_ptr()


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
