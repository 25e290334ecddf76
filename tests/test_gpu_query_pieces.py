"""Query attention whose units have one tile of rows and two by turns on the same CTA: what a unit
leaves in shared memory and tensor memory must not reach the next one."""
import pytest
import torch

from test_gpu_queries import Cache, check_query, queries, run_query, same

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hq,hk,d,dtype", [(8, 2, 128, "bf16"), (16, 16, 64, "fp16"), (4, 4, 128, "fp16")])
@pytest.mark.parametrize("many", [False, True])
def test_one_tile_then_two(hq, hk, d, dtype, many):
    """Sequences of one short tile of rows and of several, in turn: Q of the second tile comes to
    where the sums of a unit whose blocks the softmax sets share were.  In chunks and, of many
    sequences, as whole units."""
    n = 160 if many else 24
    q_lens = [(1, 200, 20, 150, 3)[i % 5] for i in range(n)]
    kv_lens = [(40, 130, 400, 64, 700)[i % 5] + i % 7 for i in range(n)]
    cache = Cache([kv_lens], hk, d, 16, dtype, seed=13)
    q = queries(sum(q_lens), hq, d, dtype, seed=14)
    out, lse = run_query(cache, q, q_lens, kv_lens)
    check_query(cache, q, q_lens, out, lse, pick=[0, 31, 32, 127, 128, 140, 199])
    for _ in range(10):
        again, lse2 = run_query(cache, q, q_lens, kv_lens)
        assert same(out, again) and same(lse, lse2)
