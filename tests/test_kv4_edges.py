"""The 4-bit paged cache on the CPU: what the binding and the library refuse, or decide, on the host."""
import pytest

import random_access_kv_fq_b200 as fq
from tests import kv4_ref as ref

torch = pytest.importorskip("torch")


def _call(**kw):
    q = torch.zeros(3, 4, 64, dtype=torch.float16)
    cache = torch.zeros(2, 2, 1, ref.unit_bytes(64, 32), dtype=torch.uint8)
    i = torch.zeros(2, dtype=torch.int32)
    return fq.fq_kv4_attn(q, cache, i[:, None], i, 32, **kw)


def test_query_counts_need_their_maximum():
    cu = torch.tensor([0, 1, 3], dtype=torch.int32)
    with pytest.raises(ValueError, match="max_q"):
        _call(cu_q=cu)
    for ok in (dict(cu_q=cu, max_q=2), dict(), dict(max_q=1)):  # as far as the tensors, which are not on a GPU
        with pytest.raises(ValueError, match="CUDA"):
            _call(**ok)
