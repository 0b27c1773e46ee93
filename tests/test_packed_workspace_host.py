"""Workspace sizes of the packed call: what the kernels that run need, and no more (no GPU needed)."""
import numpy as np
import pytest

import linear_attention_sequence_chunkwise_b200 as rn
from linear_attention_sequence_chunkwise_b200 import _build
from serving_util import FLAGS

FAKE = 0x10000  # never dereferenced: every call here is refused for its workspace


@pytest.fixture(scope="module", autouse=True)
def lib():
    _build.build()
    return rn.load()


def gamma(n):
    return np.linspace(0.95, 0.9999, n).astype(np.float32)


# tokens, seqs, heads, heads_kv, d_k, d_v
DIMS = [(16381, 2, 16, 16, 256, 512), (12289, 9, 8, 8, 128, 128), (16384, 64, 8, 8, 128, 128), (157, 6, 8, 8, 128, 128),
        (2999, 5, 8, 2, 80, 120), (1, 1, 1, 1, 64, 64), (1, 1, 1, 1, 1, 1), (700, 3, 4, 2, 64, 1024)]


@pytest.mark.parametrize("dims", DIMS)
def test_sizes(dims):
    every = rn.retnet_packed_workspace_size(dims)
    sizes = {}
    for dtype, flags in ((rn.BF16, 0), (rn.BF16, rn.F_PRECISE), (rn.F32, 0)):
        n = rn.retnet_packed_call_workspace_size(dims, dtype, flags, gamma(dims[3]))
        assert 0 < n <= every
        sizes[rn.retnet_packed_kernel(dims, dtype, flags, gamma(dims[3]))] = n
    assert max(sizes.values()) == every  # no larger than one of the calls needs


def test_the_tensor_core_call_keeps_one_copy_of_its_states():
    """Chunks of 128 tokens: fp16 states, and what is small beside them."""
    tokens, seqs, heads, kv, dk, dv = dims = (16381, 2, 16, 16, 256, 512)
    states = 2 * (tokens // 128 + seqs) * kv * dk * dv
    assert states <= rn.retnet_packed_call_workspace_size(dims, rn.BF16, FLAGS, gamma(kv)) <= states * 1.01


@pytest.mark.parametrize("dtype,flags", [(rn.BF16, 0), (rn.F32, 0)])
def test_a_smaller_workspace_is_refused(lib, dtype, flags):
    dims = (300, 3, 4, 2, 128, 64)
    d = rn.PackedDims(*dims, 5, 512, 256, 128, 256)
    n = rn.retnet_packed_call_workspace_size(dims, dtype, flags, gamma(2))
    assert lib.retnet_retention_packed(FAKE, FAKE, FAKE, FAKE, d, dtype, gamma(2).tobytes(), None, flags, FAKE, FAKE, None, FAKE,
                                       FAKE, n - 1, None) == 4


def test_refusals(lib):
    d = rn.PackedDims(300, 3, 4, 2, 128, 64, 5, 512, 256, 128, 256)
    assert lib.retnet_packed_call_workspace_size(d, rn.BF16, 0, gamma(2).tobytes(), None) == 1
    for dtype, flags, g, status in ((7, 0, gamma(2), 3), (rn.BF16, rn.F_NORM_R, gamma(2), 5), (rn.BF16, 0, np.ones(2), 4)):
        with pytest.raises(rn.RetnetError) as e:
            rn.retnet_packed_call_workspace_size((300, 3, 4, 2, 128, 64), dtype, flags, g)
        assert e.value.status == status
    with pytest.raises(rn.RetnetError):
        rn.retnet_packed_call_workspace_size((300, 3, 3, 2, 128, 64), rn.BF16, 0, gamma(2))
