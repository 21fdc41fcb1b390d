"""mla_batch_plan's report of page numbers outside the pool, for the pages that
no row of the step lies on: the shared ones."""
import numpy as np
import pytest

from tests.test_gpu_paging import draw_plan, mla, plan_reference, run_plan, same  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bad", [-1, "num_blocks", 2 ** 31 - 1, -2 ** 31])
@pytest.mark.parametrize("B,at", [(1, 0), (40, 2), (40, 0)])
def test_a_shared_page_outside_the_pool_is_reported(mla, B, at, bad):  # noqa: F811
    c = draw_plan(51, B=B, bs=16, ctx_hi=100, new_hi=30, nshared=3, pad=4)
    assert run_plan(mla, **c)[1] == mla.MLA_OK
    c["shared"] = np.array(c["shared"])
    c["shared"][at] = c["num_blocks"] if bad == "num_blocks" else bad
    got, err = run_plan(mla, **c)
    assert err == mla.MLA_ERR_DEVICE_DATA
    same(got, plan_reference(**c))  # planned all the same: no new row lies on a shared page
    assert mla.mla_get_device_error() == mla.MLA_OK
