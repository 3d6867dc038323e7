"""GPU tests of the 4-bit KV cache where it is easy to get wrong: values far past what
a block can hold, lengths past the page table, weights of one token, workspaces of
other calls, empty batches, and rows whose elements span fp16's range.  Each test
derives its own tolerance."""
import math

import pytest
import torch

from tests import kv4_reference as ref
from tests.test_gpu_kv4 import Setup, _aq

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("g", [2.0 ** -100, 2.0 ** -40, 2.0 ** -12, 1.0, 2.0 ** 20, 3e-30])
@pytest.mark.parametrize("dtype,rotate", [(F32, False), (BF16, False), (F32, True)])
def test_append_far_past_the_largest_value(g, dtype, rotate):
    """Values up to fp32's range saturate with their sign whatever the head's scale: bit for bit the
    documented steps, in which x / (g s) is an infinity of x's sign."""
    for amplitude in (g * 1e2, g * 1e6, 1e12, 1e30, 3e37):
        # (a rotation adds up to 64 values of up to nine times the amplitude: 576 x 5e35 is still in fp32's range)
        if not 1e-37 < amplitude < (5e35 if rotate else 1e38):
            continue
        st = Setup([40], 1, 64, dtype=dtype, rotate=rotate, seed=7, amplitude=amplitude, g=(g, g))
        # one block of every row far below the rest, so that both kinds of block are there
        st.K[..., 16:32] *= 1e-30
        st.V[..., 32:48] *= 1e-30
        _aq().attnq_kv4_append(st.cache, st.seqs, st.K.cuda(), st.V.cuda())
        K, V = st.read()
        k, v = st.held(0, 0)
        assert torch.equal(K[0, 0], k.float()) and torch.equal(V[0, 0], v.float())
        most = 6 * 448 * g
        if amplitude > 1e6 * most and not rotate:
            assert (V[0, 0, :, :32].abs() == most).any() and (V[0, 0] == -most).any()
