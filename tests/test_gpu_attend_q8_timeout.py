"""The failure path of kv_attend_q8's kernel for many rows, made to run on purpose without any
fault: kvrp_test_set_wait_limit shortens the limit of its pipeline waits to a cycle, so that
a wait that is not over at its first look gives up.  The launch then reports
KVRP_DEV_TIMEOUT, lets its copies and tensor-core work drain, frees its TMEM and returns, and
the next call on the same stream, with the default limit, is right."""
import pytest
import torch

from test_gpu_attend_q8 import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from position_invariant_kv_gb300.build import build
    build()
    import position_invariant_kv_gb300 as kvrp
    yield
    kvrp.kvrp_test_set_wait_limit(0)


@pytest.mark.parametrize("case", [dict(ctx=[300, 17], rows=[150, 40], hq=7, hkv=1, d=128),
                                  dict(ctx=[1200], rows=[90], hq=8, hkv=2, d=64)])
def test_short_wait_limit_reports_timeout_and_the_next_call_is_right(case):
    c = Case(**case)
    try:
        c.kvrp.kvrp_test_set_wait_limit(1)
        c.run()
    finally:
        c.kvrp.kvrp_test_set_wait_limit(0)
    torch.cuda.synchronize()                      # the launch returns
    assert int(c.status) & c.kvrp.KVRP_DEV_TIMEOUT
    c.status.zero_()
    c.run()
    c.check()
    assert int(c.status) == 0
