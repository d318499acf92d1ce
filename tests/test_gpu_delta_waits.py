"""The prefill's bounded waits: whatever the limit, every launch ends, the status tells, and the next call is whole."""
import pytest
import torch

import tests.test_gpu_delta as base
import weight_only_int4_fp32_b200 as lm

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("d", [64, 128])
def test_waits_that_run_out_end_every_launch(d):
    """The scan's copies are not issued, so each of its warps gives up within the limit, all lanes alike."""
    T, H = 500, 40
    f = lm.GatedDeltaRule(H, H, d, d, T, 2)
    a = base.make(T, H, H, d, d, True, 1)
    cu = torch.tensor([0, 333, T], dtype=torch.int32, device=DEV)
    st = base.pool(2, H, d, d, 1)
    want_s = st.clone()
    want = f.prefill(*a, want_s, cu)
    for limit in (1, 50, 1_000, 30_000, 1_000_000):  # ns
        f.test_set_wait(True, limit)
        f.prefill(*a, st.clone(), cu)
        assert f.status() == lm.LING_MOE_ERR_DEVICE_TIMEOUT
        f.test_set_wait(False)
        s = st.clone()
        assert torch.equal(f.prefill(*a, s, cu), want) and torch.equal(s, want_s) and f.status() == lm.LING_MOE_OK
    f.close()
