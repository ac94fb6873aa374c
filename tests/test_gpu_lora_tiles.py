"""GPU: fs_lora_add at the sizes at which its items change from one row tile to two: a row's
bits are the same on both sides."""
import numpy as np
import pytest

from tests.test_gpu_lora import check, make, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from continuous_transformer_decode_gb300 import build
    build.build()


@pytest.mark.parametrize("xb,yb", [(True, False), (True, True), (False, False), (False, True)])
@pytest.mark.parametrize("rank", [16, 64])
def test_rows_on_both_sides(rank, xb, yb):
    import torch
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    ads = 4
    most = 16 * (2 * sms - ads)  # rows whose items of one tile run at a time
    rng = np.random.default_rng(rank)
    c = make(rng, most + 600, 136, 69, ads, rank, xb, yb, np.sort(rng.integers(-1, ads, most + 600)))
    whole = run(c)
    check(c, whole)
    for n in (most - 1, most, most + 1, most + 17):
        rows = np.sort(rng.permutation(most + 600)[:n])
        d = dict(c, x=c["x"][rows].contiguous(), adapter=c["adapter"][rows].contiguous(), base=c["base"][rows].contiguous())
        assert torch.equal(run(d), whole[rows]), n
