"""What the header promises of row scores, eviction and draft verification at the
edges of its ranges, on the GPU."""

import numpy as np
import pytest
import torch

from quantized_kv_cache_08_gb300.cache import verify
from tests.kvq_testutil import need_gpu
from tests.test_rows_contract_host import ODD, odd_rows

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


# ------------------------------------------------------------------ verification

@pytest.mark.parametrize("dtype", [F32, BF])
def test_probabilities_of_a_draft_that_are_none(dtype):
    """A drafted token's own p and q: NaN and what is not above 0 are 0, what is above 1 is 1."""
    need_gpu()
    rows = [odd_rows(*c[:3]) for c in ODD]
    t, q, k, u = (torch.from_numpy(np.stack([r[i] for r in rows])) for i in range(4))
    accept, token = verify(t.to(dtype).cuda(), q.to(dtype).cuda(), k.cuda(), u.float().cuda())
    assert accept.tolist() == [2 if c[3] else 1 for c in ODD]
    assert token.tolist() == [6 if c[3] else 4 for c in ODD]
