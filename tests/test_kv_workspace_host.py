"""The workspace that kv_attention takes, without a GPU: by the rule that chooses its kernels."""
import pytest

import heterogeneous_adapter_gemm_amd as hg
from tests.test_kv_host import FAKE, batch, host_pool, refused


def attend(rows, size, head_dim=128, n_kv=2):
    """8 query heads: rows * 4 query rows of a KV head."""
    b = batch(head_dim=head_dim, n_heads=4 * n_kv, n_kv_heads=n_kv, max_rows=rows, n_rows=rows)
    width = 4 * n_kv * head_dim
    hg.lora_kv_attention(host_pool(4096).pool, b, FAKE, width, FAKE, width, 0.1, FAKE, size, stream=0)


@pytest.mark.parametrize("head_dim", [64, 128, 256])
def test_up_to_64_query_rows_take_the_workspace_of_few(head_dim):
    few = hg.lora_kv_workspace_bytes(batch(head_dim=head_dim, max_rows=4))
    many = hg.lora_kv_workspace_bytes(batch(head_dim=head_dim, max_rows=17))
    for rows in (1, 4, 5, 16):
        assert few <= hg.lora_kv_workspace_bytes(batch(head_dim=head_dim, max_rows=rows)) <= many
        refused(lambda: attend(rows, few - 1, head_dim), "workspace")
        refused(lambda: attend(rows, few, head_dim), "host-only")       # past the workspace's check
    for rows in (17, 1000):
        refused(lambda: attend(rows, many - 1, head_dim), "workspace")
        refused(lambda: attend(rows, many, head_dim), "host-only")
