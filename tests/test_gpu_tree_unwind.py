"""Tree decode beside a wait that has run out elsewhere: its own waits may then give up at once.

Whatever they leave, the kernel returns with its copies landed and its tensor memory freed, the status keeps naming the
wait, and after a reset calls are right again."""
import pytest
import torch

from exact_long_context_tmem_b200 import attn as A
from tests.parity import device_clean
from tests.test_gpu_tree import KINDS, caches, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("n_q,lens", [(6, [4000] * 20), (40, [4000, 300, 128] * 8), (40, [60] * 90)])
def test_calls_after_a_timeout_return_and_calls_after_a_reset_are_right(cuda_device, kind, n_q, lens):
    dev = cuda_device
    d = make(kind, len(lens), n_q, 8, 2, lens, max(lens), seed=n_q)
    (k, v), sc = caches(d, kind, dev)
    args = d["q"].to(dev), k, v, d["kv_lens"].to(dev), d["mask"].to(dev)
    want = A.attn_decode_tree(*args, **sc)
    device_clean()
    try:
        assert A.attn_debug_wait_probe(1_000_000) == A.ATTN_ERR_TIMEOUT
        for _ in range(4):
            A.attn_decode_tree(*args, **sc)
        torch.cuda.synchronize()
    finally:
        status = A.attn_device_status(reset=True)
    assert status == (A.ATTN_ERR_TIMEOUT, 1)
    for _ in range(2):
        got = A.attn_decode_tree(*args, **sc)
        assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    device_clean()
