"""The inputs of tests/coherent_sink.py tell a backward that rounds once too often from
one that does not: each mistake, planted in 64-bit arithmetic, breaks its bound."""
import numpy as np
import pytest

from oracle import sink_oracle as so
from tests import coherent_sink as cs


@pytest.mark.parametrize("hd,T,Hq,seed", cs.CASES)
def test_planted_roundings_break_the_bounds(hd, T, Hq, seed):
    x = cs.inputs(hd, T, Hq, seed)
    q, k = (y[0].double().numpy() for y in x[:2])
    assert so.score_slack(q, k, hd ** -0.5) <= 0.8 * so.W
    ref, bound = cs.exact(*x)

    def breaks(name, **mistake):
        got = cs.exact(*x, **mistake)[0][name]
        return bool((np.abs(cs.bf16(got).double().numpy() - ref[name]) > bound[name]).any())

    for name in ref:
        assert not breaks(name)  # the last rounding alone
    assert breaks("dv", round_p=True)
    for name in ("dq", "dk"):
        assert breaks(name, round_ds=True) and breaks(name, round_o=True)


@pytest.mark.parametrize("hd,T,Hq,seed", cs.CASES[:1])
def test_the_formulas_are_the_oracles(hd, T, Hq, seed):
    x = cs.inputs(hd, T, Hq, seed)
    ref, _ = cs.exact(*x)
    g, _ = so.sink_window_attention_vjp(*[y.double().numpy() for y in x], cs.WINDOW, 1, hd ** -0.5)
    # 16 bits of P and dS
    for name, want in (("dq", g["dq"][0]), ("dk", g["dk"][0, 0, 0]), ("dv", g["dv"][0, 0, 0])):
        np.testing.assert_allclose(ref[name], want, rtol=2.0 ** -15, atol=1e-9)
