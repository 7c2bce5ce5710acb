"""Requests of the engine over the KV calls: prompts and decode rows as the engine forms them, keys and values
in the pages that it holds for each request, attention over them in every layer, in 64 bits."""
import numpy as np
import pytest

from oracle import kv_model as KV
from tests.gpu_helpers import to_np
from tests.kv_bounds import FEW_ROWS, attention_bounds, outside
from tests.test_gpu_kv import _gpu, bf16, dev, say

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def test_requests_keep_their_tokens_in_the_engines_pages():
    import heterogeneous_adapter_gemm_amd as hg
    D, H, n_kv, layers = 64, 8, 2, 2
    g = np.random.default_rng(31)
    pool = hg.DevicePool(hg.LORA_BF16, 1024, 1024, g.permutation(1024), layers, [512], [512], 4, 16, 64, 8)
    npb = pool.kv_pages_per_block(n_kv, D)
    eng = hg.AdapterEngine(pool, lambda a: (8, 16.0, 0), lambda a, A, B: None, 1 << 22, 64, 4, max_running=8,
                           kv_pages_per_token=layers * npb)
    free0 = len(pool.free_list())
    for rid, (prompt, new) in enumerate([(17, 3), (1, 18), (33, 2), (16, 5)]):
        eng.submit(rid, -1, prompt, new)
    most = 4                                                     # blocks of the longest request
    cache = {}                                                   # request -> [layer][keys, values]: code, step, lo
    steps = 0
    while True:
        b, plan = eng.step()
        ids, rows = [int(i) for i in b["requests"]], [int(r) for r in b["rows"]]
        if not ids:
            eng.step_done()
            break
        say("engine step", steps, ids, rows)
        T = sum(rows)
        table = np.full((layers, len(ids), most, npb), -1, np.int32)
        lens = []
        for s, (rid, n) in enumerate(zip(ids, rows)):
            cache.setdefault(rid, [[[], []] for _ in range(layers)])
            had = sum(len(c[0]) for c in cache[rid][0][0])
            lens.append(had + n)
            nb = -(-lens[-1] // KV.BLOCK)
            pages = eng.kv_pages(rid)[:nb * layers * npb].reshape(nb, layers, npb)     # the request's own, block by block
            table[:, s, :nb] = pages.transpose(1, 0, 2)
        start = torch.from_numpy(np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)).cuda()
        for layer in range(layers):
            batch = hg.KvBatch(H, n_kv, D, start, torch.tensor(lens, dtype=torch.int32).cuda(),
                               torch.from_numpy(table[layer]).cuda(), T, max_rows=max(rows))
            q, k, v = bf16(g, T, H, D), bf16(g, T, n_kv, D), bf16(g, T, n_kv, D)
            out = torch.empty((T, H, D), dtype=torch.bfloat16, device="cuda")
            pool.kv_append(batch, dev(k), dev(v))
            pool.kv_attention(batch, dev(q), out, workspace=pool.kv_workspace(batch))
            torch.cuda.synchronize()
            got, at = to_np(out), 0
            new = KV.quantise(k), KV.quantise(v)
            few = True if max(rows) * H // n_kv <= FEW_ROWS else None
            for rid, n in zip(ids, rows):
                for side in range(2):
                    cache[rid][layer][side].append(tuple(x[at:at + n] for x in new[side]))
                key, val = (tuple(np.concatenate(x) for x in zip(*c)) for c in cache[rid][layer])
                want, bound, _ = attention_bounds(q[at:at + n], key, val, n_kv, D ** -0.5, few)
                assert not outside(got[at:at + n], want, bound).any(), (steps, layer, rid)
                at += n
        eng.step_done()
        steps += 1
    assert steps >= 18 and len(pool.free_list()) == free0        # every page went back
    eng.close()
