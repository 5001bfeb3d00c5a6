"""What ``from linear_recurrence_gb300 import *`` brings: every operator of the ABI that the binding has."""


def test_every_operator_is_exported():
    import linear_recurrence_gb300 as m
    there = [n for n in m.SIGNATURES if callable(getattr(m, n, None))]
    assert {"sscan_fwd", "lattn_step", "qknorm_bwd", "state_move"} <= set(there)
    assert [n for n in there if n not in m.__all__] == []
    names = {}
    exec("from linear_recurrence_gb300 import *", names)
    assert all(names[n] is getattr(m, n) for n in m.__all__)
