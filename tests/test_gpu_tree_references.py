"""Attention of drafted tokens where a row's reference score has to be raised
in later key tiles, so that what O and the sums hold of earlier tiles is
scaled down: keys that climb in steps of 19 and 2.5 (in powers of two). The
first stays below the slack of 2^20 that a reference leaves, the second
passes it, and the earlier tiles still carry a good part of the row.
Rows follow the climb in full, nearly (no raise), not at all or downwards,
side by side. Against the fp64 oracle, with the tolerances of
test_gpu_cache.py (its head comment derives them)."""
import math

import numpy as np
import pytest
import torch

from oracle import cache as oc

pytestmark = pytest.mark.gpu
needs_gpu = pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")

U_BF, U = 2.0 ** -8, 2.0 ** -24
D = 128
# powers of two by which the halves of seven key tiles in a row stand above the first one
CLIMB = {
    "second-half": [(0, 0), (0, 0), (19, 21.5), (19, 21.5), (21, 20), (20, 21), (19, 20)],
    "first-half": [(0, 19), (0, 19), (21.5, 20), (21.5, 20), (19, 21), (20, 20), (21, 19)],
    "twice": [(0, 0), (0, 19), (19, 21.5), (21.5, 40), (42, 41), (42.5, 41), (41, 42)],
}
FOLLOWS = [1.0, 0.0, 0.9, 1.0, -1.0, 0.95, 0.0]      # of row r: FOLLOWS[5 r mod 7]


@pytest.fixture(scope="module")
def lib():
    from long_context_prefill_dhsa_b200 import binding
    yield binding
    if torch.cuda.is_available():
        assert binding.check_device_status() == 0


def climbing(rng, climb, B, Hkv, G, T, cap):
    """Q [B,Hkv*G,T,128] and K [B,Hkv,cap,128] as fp32 arrays."""
    Q = rng.standard_normal((B, Hkv, G * T, D)) * 0.1
    K = rng.standard_normal((B, Hkv, cap, D))
    level = np.array([CLIMB[climb][s // 128 % 7][s // 64 % 2] for s in range(cap)])
    Q[..., 0] = 4.0 * np.array([FOLLOWS[5 * r % 7] for r in range(G * T)])
    K[..., 0] = level * math.log(2.0) * math.sqrt(D) / 4.0
    return Q.reshape(B, Hkv * G, T, D).astype(np.float32), K.astype(np.float32)


ROWS = [(1, 1), (4, 2), (8, 8), (8, 13), (16, 8), (8, 25), (5, 60)]      # query heads of a kv head, tokens
PLACE = {        # sequences, kv heads, slots, heads compared
    "whole": (1, 2, 637, [(0, 0), (0, 1)]),                      # one CTA has all five tiles
    "whole-many": (32, 2, 1020, [(0, 0), (31, 1)]),              # eight
    "split": (1, 8, 12345, [(0, 0), (0, 5)]),                    # five to six tiles a CTA, joined afterwards
}


@needs_gpu
@pytest.mark.parametrize("rows", ROWS, ids=[f"{g}x{t}" for g, t in ROWS])
@pytest.mark.parametrize("climb", list(CLIMB))
@pytest.mark.parametrize("place", list(PLACE))
def test_references_raised_in_later_tiles(lib, place, climb, rows):
    G, T = rows
    B, Hkv, cap, compared = PLACE[place]
    rng = np.random.default_rng(70 + G * T)
    Q, K = (torch.from_numpy(x).to(torch.bfloat16).cuda() for x in climbing(rng, climb, B, Hkv, G, T, cap))
    V = torch.from_numpy(rng.standard_normal((B, Hkv, cap, D)).astype(np.float32)).to(torch.bfloat16).cuda()
    n = cap - T
    lengths = torch.full((B,), n, dtype=torch.int32, device="cuda")
    lse = torch.zeros(B, Hkv * G, T, device="cuda")
    w = torch.zeros(B, Hkv, cap, device="cuda")
    out = lib.tree_attn(Q, K, V, lengths, weight=w, lse=lse)
    plain = lib.tree_attn(Q, K, V, lengths)
    assert torch.equal(out, plain)
    for b, h in compared:
        of = slice(h * G, (h + 1) * G)
        f64 = lambda x: x.double().cpu().numpy()
        O, L, W, A, abs_s = oc.tree_attn(f64(Q[b, of]), f64(K[b, h:h + 1]), f64(V[b, h:h + 1]), n, None, T,
                                         1 / math.sqrt(D))
        e = 2 * 256 * U * abs_s + 2.0 ** -20
        assert np.all(np.abs(f64(out[b, of]) - O) <= (U_BF + e) * A + U_BF * np.abs(O) * (1 + U_BF) + 1e-30)
        assert np.all(np.abs(f64(lse[b, of]) - L) <= e + 4 * U * np.abs(L))
        assert np.all(np.abs(f64(w[b, h]) - W[0]) <= e * W[0] + 4 * U * W[0])
