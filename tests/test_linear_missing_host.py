"""A call of the linear layers without one of the matrices that it needs says which, with the stand-ins of
test_devices_host.py (no GPU)."""

from tests.test_devices_host import _run
from tests.test_linear_devices_host import TENSORS


def test_a_missing_matrix_is_named():
    _run(TENSORS + """
    def without(call, names, args):
        for i, name in enumerate(names):
            given = list(args)
            given[i] = None
            with pytest.raises(ValueError, match=f"{name}.* must be given"):
                call(*given)
    without(tsg.gated_linear, ("x", "gate_weight", "up_weight", "y"), (x, w, w, y))
    without(tsg.gated_linear_grad, ("dy", "x", "gate_weight", "up_weight", "gate", "up"), (y, x, w, w, y, y, x))
    without(tsg.linear_cross_entropy, ("x", "weight"), (x, w, t, v, v))
    without(tsg.linear_cross_entropy_grad, ("dloss", "x", "weight"), (v, x, w, t, v, x))
    for call in (lambda: tsg.linear_cross_entropy(x, w, None, v, v), lambda: tsg.linear_cross_entropy(x, w, t, None, v),
                 lambda: tsg.linear_cross_entropy(x, w, t, v, None), lambda: tsg.linear_cross_entropy_grad(v, x, w, None, v, x),
                 lambda: tsg.linear_cross_entropy_grad(v, x, w, t, None, x)):
        with pytest.raises(ValueError, match="must be given"):
            call()
    assert not calls
    """)
