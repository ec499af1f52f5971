"""Host checks of the calls on a key/value cache, the rotary frequencies, and
pins of the cache oracle. No GPU."""
import ctypes
import math

import numpy as np
import pytest
import torch

from long_context_prefill_dhsa_b200 import binding, build, cache
from oracle import cache as oc

FAKE = 1 << 20   # a non-null, aligned stand-in pointer; never dereferenced
INV, UNS, WS = 1, 2, 5


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load()


def _call(fn, order, base, **change):
    args = dict(base, **change)
    return fn(*[args[n] for n in order])


def _strides(*s):
    return (ctypes.c_int64 * 3)(*s)


ROT = ("Q qs K ks V vs B Hq Hkv T d f rd inter tr factor positions start n_new Qo Ko kos Vo vos slots cap pos "
       "stream").split()
ROT_OK = dict(Q=FAKE, qs=None, K=FAKE, ks=None, V=FAKE, vs=None, B=2, Hq=4, Hkv=2, T=5, d=128, f=FAKE, rd=64, inter=0,
              tr=0, factor=1.0, positions=None, start=None, n_new=None, Qo=FAKE, Ko=FAKE, kos=None, Vo=FAKE, vos=None,
              slots=FAKE, cap=9, pos=None, stream=None)


@pytest.mark.parametrize("change,want", [
    (dict(Q=None), INV), (dict(Q=None, Qo=None, K=None, Ko=None, V=None, Vo=None), INV), (dict(K=None), INV),
    (dict(V=None), INV), (dict(K=None, Ko=None, pos=FAKE), INV), (dict(B=0), INV), (dict(Hq=0), INV),
    (dict(Hkv=-1), INV), (dict(T=0), INV), (dict(cap=0), INV), (dict(slots=None, cap=4), INV), (dict(d=64), UNS),
    (dict(f=None), INV), (dict(f=FAKE + 4), INV), (dict(rd=8), INV), (dict(rd=144), INV), (dict(rd=72), INV),
    (dict(factor=math.inf), INV), (dict(factor=math.nan), INV), (dict(Q=FAKE + 8), INV), (dict(Ko=FAKE + 2), INV),
    (dict(qs=_strides(640, 128, 4)), INV), (dict(kos=_strides(2304, 1152, 0)), INV),
    (dict(vos=_strides(2304, -1152, 128)), INV), (dict(Hkv=1 << 20, cap=1 << 20), INV),
])
def test_rotary_refusals(lib, change, want):
    assert _call(lib.dhsa_rotary_qkv, ROT, ROT_OK, **change) == want


TREE = ("Q K ks V vs B Hq Hkv T cap d lengths parents n_draft scale O lse w wo ws bytes stream").split()


@pytest.mark.parametrize("change,want", [
    (dict(Q=None), INV), (dict(K=None), INV), (dict(V=None), INV), (dict(O=None), INV), (dict(lengths=None), INV),
    (dict(w=FAKE), INV), (dict(wo=FAKE), INV), (dict(Hq=3), INV), (dict(T=0), INV), (dict(T=65), UNS),
    (dict(Hq=2 * 65), UNS), (dict(d=96), UNS), (dict(cap=0), INV), (dict(scale=0.0), INV), (dict(scale=-1.0), INV),
    (dict(scale=math.nan), INV), (dict(scale=math.inf), INV), (dict(K=FAKE + 2), INV),
    (dict(ks=_strides(1280, 128, 64)), INV), (dict(vs=_strides(1280, 132, 256)), INV), (dict(ws=None), WS),
    (dict(bytes=16), WS), (dict(ws=FAKE + 4), WS), (dict(O=FAKE), INV),
    (dict(w=FAKE, wo=FAKE, scale=9e-31), INV),
])
def test_tree_refusals(lib, change, want):
    ok = dict(Q=FAKE, K=FAKE, ks=None, V=FAKE, vs=None, B=2, Hq=4, Hkv=2, T=5, cap=50, d=128, lengths=FAKE,
              parents=None, n_draft=None, scale=0.1, O=FAKE + 4096, lse=None, w=None, wo=None, ws=FAKE,
              bytes=lib.dhsa_tree_attn_workspace_size(2, 4, 2, 5, 50, 0), stream=None)
    assert _call(lib.dhsa_tree_attn, TREE, ok, **change) == want


def test_workspace_queries(lib):
    ws = lib.dhsa_tree_attn_workspace_size
    assert lib.dhsa_tree_max_drafts() == 64
    assert ws(1, 4, 2, 1, 100, 0) > 0 and ws(1, 4, 2, 1, 100, 1) >= ws(1, 4, 2, 1, 100, 0)
    for bad in ((0, 4, 2, 1, 100), (1, 3, 2, 1, 100), (1, 4, 2, 0, 100), (1, 4, 2, 65, 100), (1, 4, 2, 1, 0)):
        assert ws(*bad, 0) == 0
    assert lib.dhsa_cache_evict_workspace_size(2, 3, 100) >= 4 * 2 * 3 * 100
    assert lib.dhsa_cache_evict_workspace_size(2, 0, 100) == 0


EV = ("K ks V vs w pos B Hkv cap d lengths n_draft accept keep sinks recent next wo po lo index ws bytes stream").split()


@pytest.mark.parametrize("change,want", [
    (dict(K=None), INV), (dict(V=None), INV), (dict(w=None), INV), (dict(pos=None), INV), (dict(lengths=None), INV),
    (dict(wo=None), INV), (dict(po=None), INV), (dict(lo=None), INV), (dict(lo=FAKE + 64), INV), (dict(keep=0), INV),
    (dict(keep=-1), INV), (dict(sinks=-1), INV), (dict(recent=-1), INV), (dict(recent=1, next=None), INV),
    (dict(n_draft=None), INV), (dict(accept=FAKE + 4), INV), (dict(d=64), UNS), (dict(V=FAKE + 8), INV),
    (dict(ks=_strides(6400, 0, 128)), INV), (dict(ws=None), WS), (dict(bytes=8), WS), (dict(B=-2), INV),
])
def test_evict_refusals(lib, change, want):
    ok = dict(K=FAKE, ks=None, V=FAKE, vs=None, w=FAKE, pos=FAKE, B=2, Hkv=2, cap=50, d=128, lengths=FAKE + 64,
              n_draft=FAKE, accept=FAKE, keep=10, sinks=0, recent=0, next=FAKE, wo=FAKE, po=FAKE, lo=FAKE, index=None,
              ws=FAKE, bytes=lib.dhsa_cache_evict_workspace_size(2, 2, 50), stream=None)
    assert _call(lib.dhsa_cache_evict, EV, ok, **change) == want


def test_binding_refuses_host_tensors_and_wrong_types():
    bf = torch.zeros(1, 2, 3, 128, dtype=torch.bfloat16)
    n = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        binding.rotary_qkv(bf, bf, torch.zeros(64, dtype=torch.float64))
    with pytest.raises(ValueError):
        binding.rotary_qkv(None, None, torch.zeros(64, dtype=torch.float64))
    with pytest.raises(ValueError):
        binding.tree_attn(bf, bf, bf, n)
    with pytest.raises(TypeError):
        binding.tree_attn(bf.float(), bf, bf, n)
    with pytest.raises(ValueError):
        binding.cache_evict(bf, bf, torch.zeros(1, 2, 3), torch.zeros(1, 2, 3, dtype=torch.int32), n, 2)


def test_inv_freq_scalings():
    plain, one = cache.rotary_inv_freq(64, base=10000.0, device="cpu")
    assert one == 1.0 and plain.dtype == torch.float64 and plain[0] == 1.0
    assert math.isclose(plain[-1].item(), 10000.0 ** (-62 / 64), rel_tol=1e-14)
    lin, _ = cache.rotary_inv_freq(64, scaling="linear", factor=4.0, device="cpu")
    assert torch.allclose(lin * 4, plain, rtol=1e-15, atol=0)
    ntk, _ = cache.rotary_inv_freq(64, scaling="ntk", factor=4.0, device="cpu")
    assert ntk[0] == 1.0 and math.isclose(ntk[-1].item(), plain[-1].item() / 4, rel_tol=1e-13)
    for kind in ("wavelength", "yarn"):
        f, m = cache.rotary_inv_freq(128, base=500000.0, scaling=kind, factor=8.0, device="cpu")
        base, _ = cache.rotary_inv_freq(128, base=500000.0, device="cpu")
        r = f / base
        assert r[0] == 1.0 and math.isclose(r[-1].item(), 1 / 8, rel_tol=1e-13)
        assert torch.all(r[1:] <= r[:-1] + 1e-15)
        assert math.isclose(m, 1.0 if kind == "wavelength" else 0.1 * math.log(8.0) + 1.0)
    for bad in (dict(rotary_dim=20), dict(rotary_dim=0), dict(rotary_dim=256), dict(rotary_dim=64, scaling="cubic"),
                dict(rotary_dim=64, base=1.0), dict(rotary_dim=64, factor=0.5)):
        with pytest.raises(ValueError):
            cache.rotary_inv_freq(device="cpu", **bad)


def test_oracle_rotation_pins():
    x = np.zeros((1, 1, 2, 128))
    x[..., 0], x[..., 1], x[..., 100] = 1.0, 2.0, 3.0
    f = [math.pi / 2] + [0.0] * 7
    r = oc.rotate(x, [[0, 1]], f, interleaved=True)
    assert np.allclose(r[0, 0, 1, :2], [-2.0, 1.0]) and r[0, 0, 1, 100] == 3.0 and np.array_equal(r[0, 0, 0], x[0, 0, 0])
    back = oc.rotate(r, [[0, 1]], f, interleaved=True, transpose=True)
    assert np.allclose(back, x)
    h = oc.rotate(x, [[0, 1]], f)          # half layout: element 0 pairs with element 8
    assert np.allclose(h[0, 0, 1, [0, 8]], [0.0, 1.0])


def test_oracle_rotation_gradient_by_differences():
    """transpose is the gradient: <dL/dX, dX> equals the change of <g, rotate(X)>."""
    rng = np.random.default_rng(3)
    X, g, dX = (rng.standard_normal((2, 3, 4, 128)) for _ in range(3))
    pos, f = rng.integers(0, 5000, (2, 4)), rng.random(32)
    for inter in (False, True):
        grad = oc.rotate(g, pos, f, inter, transpose=True, factor=1.3)
        h = 1e-6
        diff = (np.sum(g * oc.rotate(X + h * dX, pos, f, inter, factor=1.3)) -
                np.sum(g * oc.rotate(X - h * dX, pos, f, inter, factor=1.3))) / (2 * h)
        assert math.isclose(diff, np.sum(grad * dX), rel_tol=1e-7)


def test_oracle_tree_and_evict_pins():
    assert oc.ancestors([-1, 0, 0, 1], 4).tolist() == [[True, False, False, False], [True, True, False, False],
                                                       [True, False, True, False], [True, True, False, True]]
    assert np.array_equal(oc.ancestors(None, 3), np.tril(np.ones((3, 3), dtype=bool)))
    Q, K = np.zeros((2, 1, 4)), np.zeros((1, 3, 4))
    V = np.arange(12.0).reshape(1, 3, 4)
    O, lse, W, A, _ = oc.tree_attn(Q, K, V, 2, None, 1, 1.0)
    assert np.allclose(O[0, 0], V[0].mean(0)) and np.allclose(lse, math.log(3)) and np.allclose(W, 2 / 3)
    #            slot:  0    1    2    3    4    5
    w, pos = [0.5, 0.1, 0.1, 0.9, 0.2, 0.3], [0, 1, 2, 3, 4, 5]
    f = lambda **k: oc.evict_rows(w, pos, **dict(dict(length=5, n_draft=1, accept=None, keep=3, sinks=0, recent=0,
                                                    next_pos=None), **k))
    assert f() == [0, 3, 5]                       # kept 0, 3, 5: holes 1, 2 take 3, 5
    assert f(keep=6) == [0, 1, 2, 3, 4, 5]
    assert f(accept=0, keep=6) == [0, 1, 2, 3, 4]
    assert f(sinks=2, keep=2) == [0, 1]
    assert f(recent=2, next_pos=6, keep=3) == [3, 4, 5]      # 4 and 5 are held, 3 weighs most
    assert f(keep=4, accept=0, n_draft=1) == [0, 1, 4, 3]     # 1 and 2 tie: the lower slot stays
