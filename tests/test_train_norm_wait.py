"""The layer norm's bounded wait for a row that is copied ahead (1 s of the
GPU's global timer).  MOE_DEBUG_NORM_SKIP_COPY leaves the copy of row T / 2
out: nothing is in flight against its barrier, and the wait for it runs out.
Nothing faults: the block leaves NaN for that row and its later ones, and in
the column sums; every other row is right, and the next call is clean."""
import time

import pytest
import torch

from nvfp4_mixture_experts_router_gb300 import api, build

from test_train_norm import EPS, backward, check_backward, check_forward, data, forward

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    api.lib()


def nan_rows(t):
    """Every row is NaN throughout or not at all; which ones are."""
    bad = torch.isnan(t.float())
    assert torch.equal(bad.all(1), bad.any(1))
    return bad.all(1)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,H", [(1300, 7168), (1300, 2047), (4000, 1032)])
def test_a_row_that_never_lands_becomes_nan(T, H, dt):
    x, gamma, beta, dy = data(T, H, dt)
    want = forward(x, gamma, beta)
    gone = torch.arange(T, device="cuda") == T // 2
    flag = api.MOE_DEBUG_NORM_SKIP_COPY | (api.MOE_DTYPE_F32 if dt == torch.float32 else api.MOE_DTYPE_BF16)
    L, stream = api.lib(), torch.cuda.current_stream().cuda_stream
    y, dx = torch.zeros_like(x), torch.zeros_like(x)
    mean, rstd = (torch.zeros(T, device="cuda") for _ in range(2))
    dg, db = (torch.zeros(H, device="cuda") for _ in range(2))
    ws = torch.zeros(api.moe_nvfp4_layer_norm_workspace_bytes(T, H), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    assert L.moe_nvfp4_layer_norm(T, H, flag, x.data_ptr(), H, gamma.data_ptr(), beta.data_ptr(), EPS, y.data_ptr(), H,
                                  mean.data_ptr(), rstd.data_ptr(), stream) == api.MOE_OK
    torch.cuda.synchronize()
    assert 0.9 <= time.perf_counter() - t0 < 30.0
    lost = nan_rows(y)
    assert bool(lost[gone].all()) and int(lost.sum()) <= T // 2
    assert torch.equal(torch.isnan(mean), lost) and torch.equal(torch.isnan(rstd), lost)
    assert torch.equal(y[~lost], want[0][~lost]) and torch.equal(mean[~lost], want[1][~lost])
    t0 = time.perf_counter()
    assert L.moe_nvfp4_layer_norm_backward(T, H, flag, dy.data_ptr(), H, x.data_ptr(), H, gamma.data_ptr(),
                                           want[1].data_ptr(), want[2].data_ptr(), dx.data_ptr(), H, dg.data_ptr(),
                                           db.data_ptr(), ws.data_ptr(), ws.numel(), stream) == api.MOE_OK
    torch.cuda.synchronize()
    assert 0.9 <= time.perf_counter() - t0 < 30.0
    clean = backward(dy, x, gamma, want[1], want[2])
    check_backward(dy, x, gamma, want[1], want[2], clean)
    lost = nan_rows(dx)
    assert bool(lost[gone].all()) and int(lost.sum()) <= T // 2
    assert torch.equal(dx[~lost], clean[0][~lost])
    assert bool(torch.isnan(dg).all()) and bool(torch.isnan(db).all())
    check_forward(x, gamma, beta, forward(x, gamma, beta))
