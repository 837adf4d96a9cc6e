"""Which polynomials fsdp_orthogonalize takes, without a GPU: those that keep
singular values at or below 8 until the last step. A refused call enqueues
nothing, and neither does one that is refused for its workspace, which the call
looks at last."""
import numpy as np
import pytest

from hsdp_sharded_parameter_gb300 import capi as C

P = 1 << 20


def call(steps, a, b, c, rows=70, cols=90):
    rc = C.lib().fsdp_orthogonalize(rows, cols, C.FSDP_F32, P, cols, steps, a, b, c, 1.0, 1e-7, 2 * P, cols, 3 * P, 0, None)
    assert rc == C.FSDP_ERR_INVALID_ARG
    return C.lib().fsdp_last_error().decode()


def reach(steps, a, b, c):
    """The largest singular value that a step starts from, on a grid."""
    most = top = 1.0
    for _ in range(steps - 1):
        s = np.linspace(0, top, 20001)
        top = float(np.abs(a * s + b * s ** 3 + c * s ** 5).max())
        most = max(most, top)
        if most > 1e6:
            break
    return most


CASES = [(1, 256, 0, 0), (2, 256, 0, 0), (2, 8, 0, 0), (2, -8, 0, 0), (2, 8.01, 0, 0), (4, 2, 0, 0), (5, 2, 0, 0), (64, 1, 0, 0), (3, 0, -2.8, 0),
         (5, 4, -6, 3), (3, 4, -6, 3), (64, 3.4445, -4.7750, 2.0315), (64, 1.875, -1.25, 0.375), (64, 1.5, -0.5, 0), (64, 2, -1.5, 0.5),
         (64, 0, 0, 0), (64, 256, -256, 0), (2, 256, -256, 256), (1, 256, -256, 256), (64, -1, 0, 0), (64, 0.5, 0.25, -0.1), (9, 1.25, 0, 0), (11, 1.25, 0, 0),
         (2, 8.28721201814563, -23.595886519098837, 17.300387312530933), (3, 8.28721201814563, -23.595886519098837, 17.300387312530933)]


@pytest.mark.parametrize("case", CASES, ids=str)
@pytest.mark.parametrize("rows", [40, 70])
def test_polynomials_that_leave_the_range_are_refused(case, rows):
    message = call(*case, rows=rows)
    assert ("singular value" in message) == (reach(*case) > 8.0005), (message, reach(*case))
    assert "singular value" in message or "workspace" in message


def test_random_polynomials():
    rng = np.random.default_rng(5)
    for _ in range(300):
        case = (int(rng.integers(1, 8)), *(float(np.float32(v)) for v in rng.normal(size=3) * [4, 6, 3]))
        most = reach(*case)
        if abs(most - 8) < 0.01:
            continue  # the grid's own error
        assert ("singular value" in call(*case)) == (most > 8), (case, most)
