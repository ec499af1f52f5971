"""GPU test of cache_evict with counts beyond 32 bits."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
needs_gpu = pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")

D = 128


@pytest.fixture(scope="module")
def lib():
    from long_context_prefill_dhsa_b200 import binding
    return binding


@pytest.fixture(autouse=True)
def _clean_status():
    yield
    from long_context_prefill_dhsa_b200 import binding
    if torch.cuda.is_available():
        assert binding.check_device_status() == 0


def _bf(rng, *shape):
    return torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(torch.bfloat16).cuda()


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


@needs_gpu
def test_counts_beyond_32_bits(lib):
    """Counts above the largest int mean all of it, and are not taken modulo 2^32."""
    rng = np.random.default_rng(61)
    cap = 40
    K, V = _bf(rng, 1, 1, cap, D), _bf(rng, 1, 1, cap, D)
    w = torch.from_numpy(rng.random((1, 1, cap)).astype(np.float32)).cuda()
    pos = torch.from_numpy(rng.permutation(cap).astype(np.int32)[None, None]).cuda()

    def kept(keep=8, **kw):
        index = torch.zeros(1, 1, min(keep, cap), dtype=torch.int32, device="cuda")
        lib.cache_evict(K.clone(), V.clone(), w.clone(), pos.clone(), _i32([cap]), keep, next_pos=_i32([cap]),
                        index=index, **kw)
        return index.tolist()

    plain = kept()
    first = [[list(range(8))]]                       # everything held: the first slots stay
    assert plain != first
    for big in (0x7fffffff, 1 << 31, 1 << 32, (1 << 40) + 3):
        assert kept(recent=big) == first, big
        assert kept(sinks=big) == first, big
    assert kept(keep=(1 << 32) + 5) == [[list(range(cap))]]
    for bad in (dict(keep=-(1 << 32) + 8), dict(sinks=-(1 << 32)), dict(recent=-(1 << 32) + 2), dict(sinks=-1), dict(keep=0)):
        with pytest.raises((ValueError, lib.DHSAError)):
            lib.cache_evict(K, V, w, pos, _i32([cap]), **{**dict(keep=8, next_pos=_i32([cap])), **bad})
