"""The gated projection's and the cross entropy's calls on tensors of a GPU that is
not the current one, with the stand-ins of test_devices_host.py (no GPU)."""

from tests.test_devices_host import _run

TENSORS = """
    KINDS["i64"] = (0, 64)
    x, w, y, v, t = tensor((4, 64), "bf16"), tensor((24, 64), "bf16"), tensor((4, 24), "bf16"), tensor((4,), "f32"), tensor((4,), "i64")
    calls_of = {
        "gated_linear": lambda **kw: tsg.gated_linear(x, w, w, y, gate=y, up=y, **kw),
        "gated_linear_grad": lambda **kw: tsg.gated_linear_grad(y, x, w, w, y, y, x, w, w, **kw),
        "linear_cross_entropy": lambda **kw: tsg.linear_cross_entropy(x, w, t, v, v, **kw),
        "linear_cross_entropy_grad": lambda **kw: tsg.linear_cross_entropy_grad(v, x, w, t, v, x, w, **kw)}
"""


def test_calls_run_on_their_tensors_device():
    _run(TENSORS + """
    for name, call in calls_of.items():
        for kw in ({}, {"stream": Stream(1)}):
            call(**kw)
            made(name)
    """)


def test_several_devices_are_refused():
    _run(TENSORS + """
    w0, y0, t0, v0 = tensor((24, 64), "bf16", dev=0), tensor((4, 24), "bf16", dev=0), tensor((4,), "i64", dev=0), tensor((4,), "f32", dev=0)
    for call in (lambda: tsg.gated_linear(x, w, w0, y), lambda: tsg.gated_linear(x, w, w, y0), lambda: tsg.gated_linear(x, w, w, y, up=y0),
                 lambda: tsg.gated_linear_grad(y, x, w, w, y, y0, x), lambda: tsg.gated_linear_grad(y, x, w, w, y, y, x, w, w0),
                 lambda: tsg.linear_cross_entropy(x, w, t0, v, v), lambda: tsg.linear_cross_entropy(x, w, t, v, v0),
                 lambda: tsg.linear_cross_entropy_grad(v0, x, w, t, v, x), lambda: tsg.linear_cross_entropy_grad(v, x, w, t, v, x, w0),
                 *(lambda c=c: c(stream=Stream(0)) for c in calls_of.values())):
        with pytest.raises(ValueError, match="device"):
            call()
    assert not calls and current[0] == 0
    """)
