"""lora_linear_w4 runs on the pool's GPU and refuses tensors that are on another one, without a GPU."""
import pytest

import heterogeneous_adapter_gemm_amd as hg
from tests.test_kv_host import FAKE, host_pool


class On:
    """Stands for a tensor of GPU ``index``."""

    def __init__(self, index):
        self.index = index

    def get_device(self):
        return self.index

    def data_ptr(self):
        return FAKE


def test_tensors_of_another_gpu_than_the_pools_are_refused():
    pool = host_pool()
    plan = pool.plan(token_slot=[-1])
    pool.pool.pages = On(0)
    for args in ([On(1)] * 4, [On(1), On(0), On(0), On(0)], [On(0), On(0), On(0), On(1)], [FAKE, On(1), FAKE, FAKE]):
        x, code, scale, y = args
        with pytest.raises(ValueError, match="one GPU"):
            pool.linear_w4(plan, 0, 0, x, code, scale, 64, y, stream=0)
        with pytest.raises(ValueError, match="one GPU"):
            hg.lora_linear_w4(pool.pool, plan, 0, 0, x, code, scale, 64, y, stream=0)
