"""The waits of whole warps in the routed experts' kernels run out, with a short
limit, on barriers that nothing completes: every lane learns of it, the error
word is raised once, and the context stays usable."""
import pytest
import torch

import q4_weight_matmul_gb300 as q4k

pytestmark = pytest.mark.gpu
LIMIT = 2 ** 26 >> 16                 # of a wait, in 65536 cycles


def test_a_refused_call():
    q4k.build()
    assert q4k.lib().q4k_selftest_warp_waits(None, None) == 1
    assert q4k.lib().q4k_selftest_warp_waits(8, None) == 2


@pytest.mark.parametrize("own_stream", [False, True])
def test_waits_that_run_out(own_stream):
    q4k.build()
    assert q4k.q4k_device_error() == 0
    stream = torch.cuda.Stream() if own_stream else None
    out = q4k.q4k_selftest_warp_waits(stream=stream)
    assert q4k.q4k_device_error(stream) == 5 and q4k.q4k_device_error() == 0
    *got, state = out.cpu().tolist()
    for i, goes_on in enumerate([0, 0, 0, 1, 0, 1, 0]):
        assert got[i] == [goes_on] * 32, i
    raised, took = state[:7], state[8:15]
    # (the second wait finds the flag set and reports nothing again)
    assert raised == [0x101, 0x100, 0x101, 0, 0x101, 0, 0x101]
    for i in range(7):
        if i in (0, 2, 4):
            assert LIMIT <= took[i] + 1 and took[i] < 50 * LIMIT, (i, took[i])
        else:
            assert took[i] < LIMIT // 2, (i, took[i])
