"""GPU test of a streamed prefill that fills the layers' caches."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
needs_gpu = pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")

D = 128


def _bf(rng, *shape):
    return torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(torch.bfloat16).cuda()


@needs_gpu
@pytest.mark.parametrize("rotary", [True, False])
def test_streamed_layers_fill_their_caches(rotary):
    """Each layer's cache holds that layer's K, rotated, and V, and decodes like one filled by hand."""
    from long_context_prefill_dhsa_b200 import binding, cache
    from long_context_prefill_dhsa_b200 import inputs as I
    B, Hq, Hkv, L = 2, 4, 2, 500
    w = I.custom(B=B, Hq=Hq, Hkv=Hkv, L=L, lo=20, hi=120, k=3, wid=902)
    d = I.make_inputs(w)
    off, nc = (torch.from_numpy(np.ascontiguousarray(d[x])).cuda() for x in ("off", "n_chunks"))
    f, m = cache.rotary_inv_freq(D, base=500000.0, scaling="wavelength", factor=8.0)
    kw = dict(inv_freq=f, rotary_factor=m) if rotary else {}
    rng = np.random.default_rng(80)
    layers = [[_bf(rng, B, H, L, D) for H in (Hq, Hkv, Hkv)] for _ in range(5)]
    host = [[x.cpu().pin_memory() for x in s] + [torch.empty(B, Hq, L, D, dtype=torch.bfloat16).pin_memory()]
            for s in layers]
    torch.cuda.synchronize()
    streamed = binding.HostStreamedPrefill(binding.DHSAPrefill(B, Hq, Hkv, L, off, nc, w.k, **kw))
    caches = []
    for i, h in enumerate(host):
        # made on the current stream right before; one layer is streamed without
        caches.append(None if i == 2 else cache.KVCache(B, Hq, Hkv, L + 20, f, rotary_factor=m))
        streamed.submit(*h, cache=caches[-1])
    streamed.synchronize()
    for (Q, K, V), h, c in zip(layers, host, caches):
        plain = binding.DHSAPrefill(B, Hq, Hkv, L, off, nc, w.k, **kw)
        assert torch.equal(h[3].cuda(), plain.run(Q, K, V))
        if c is None:
            continue
        want = cache.KVCache(B, Hq, Hkv, L + 20, f, rotary_factor=m)
        want.fill(plain.Kr if rotary else K, V)
        for name in ("K", "V", "weight", "pos", "lengths", "next_pos"):
            assert torch.equal(getattr(c, name), getattr(want, name)), name
        new = [_bf(rng, B, H, 3, D) for H in (Hq, Hkv, Hkv)]
        assert torch.equal(c.attend(c.extend(*new)), want.attend(want.extend(*new)))
    assert binding.check_device_status() == 0
