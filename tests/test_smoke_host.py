"""The smoke check's own test of the routed training step: it passes on the formulas' values (plain
64-bit statements, CPU) and fails where a gradient is lost."""
import pytest
import torch

import __graft_entry__ as entry
import routed_ref as ref


def step():
    g = torch.Generator().manual_seed(3)
    T, E, k, d, lr = 96, 16, 6, 64, 1e-3
    x = torch.randn(T, d, generator=g).bfloat16()
    W = torch.randn(E, d, generator=g) / 8
    logits = x.float() @ W.t()
    idx, gate = ref.route(logits, k, score="sigmoid", groups=4, top_groups=2, group_top=2,
                          renorm=True)
    a = ref.assign(idx, E, T)
    rows = torch.zeros(E * T, d, dtype=torch.bfloat16)
    t, _, r = ref.rows_of(idx, a["slot"], a["kept"], T)
    rows[r] = x[t]
    rows = rows.view(E, T, d)
    ye = torch.randn(E, T, d, generator=g).bfloat16()
    dy = torch.randn(T, d, generator=g).bfloat16()
    _, dgate = ref.combine_backward(dy, ye, idx, gate, a["slot"], a["kept"])
    dgate = dgate.float()
    dlogits = ref.route_backward(logits, idx, dgate, score="sigmoid", renorm=True).float()
    dW = dlogits.t() @ x.float()
    zero = torch.zeros_like(W)
    after, _, _ = ref.adamw(W, dW, zero, zero, step=1, lr=lr, betas=(0.9, 0.999), eps=1e-8,
                            weight_decay=0.0)
    return dict(logits=logits, x=x, idx=idx, gate=gate.float(), slot=a["slot"],
                y=ref.gather(rows, idx, a["slot"], a["kept"], gate).bfloat16(),
                dx=ref.gather(rows, idx, a["slot"], a["kept"]).bfloat16(), dy=dy, ye=ye, dgate=dgate,
                dlogits=dlogits, dW=dW, before=W, after=after.float(), lr=lr)


def test_the_formulas_values_pass():
    entry.check_routed_step(**step())


@pytest.mark.parametrize("lost", ["dgate", "dlogits", "dW", "dx", "gate", "y"])
def test_a_lost_result_fails(lost):
    s = step()
    s[lost] = torch.zeros_like(s[lost])
    with pytest.raises(AssertionError):
        entry.check_routed_step(**s)


def test_gradients_that_vanish_through_all_fail():
    """No gradient of the weights: everything behind it is zero, and consistently so."""
    s = step()
    for name in ("dgate", "dlogits", "dW", "dy"):
        s[name] = torch.zeros_like(s[name])
    s["after"] = s["before"]
    with pytest.raises(AssertionError, match="nearly zero"):
        entry.check_routed_step(**s)


def test_a_step_in_the_wrong_direction_fails():
    s = step()
    s["after"] = 2 * s["before"] - s["after"]
    with pytest.raises(AssertionError, match="lr long"):
        entry.check_routed_step(**s)
