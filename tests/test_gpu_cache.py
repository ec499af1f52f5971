"""GPU tests of the calls on a key/value cache (include/dhsa.h, 6 to 8) through
the binding, against the fp64 oracle in oracle/cache.py.

Tolerances are sums of the roundings each result goes through, u_bf = 2^-8
(bf16, half a step relative to the value) and u = 2^-24 (fp32):
* rotary: one bf16 rounding of the result; the fp32 cosine and sine carry at
  most 2 ulp plus the angle's 2^-25 half-turns, the two products and the sum
  three more roundings: under 16 u (|x| + |y|) factor.
* scores: products of bf16 are exact in fp32, 128 of them are added with at
  most one fp32 step (2 u) each: e_s = 256 u * scale * sum |q||k|, an absolute
  error of the exponent and so a relative one of p and of the denominator.
* O: each p is rounded to bf16 before the product with V (u_bf sum p|v|), and
  the result is (u_bf |O|); 2 e_s and 2^-20 (exponentials, sums of up to a few
  thousand terms) come on top, relative to sum p|v|.
* weight: no bf16 rounding: (2 e_s + 2^-20) of the added part, 2 u of the total.
"""
import math

import numpy as np
import pytest
import torch

from oracle import cache as oc

pytestmark = pytest.mark.gpu
needs_gpu = pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")

U_BF, U = 2.0 ** -8, 2.0 ** -24
D = 128


@pytest.fixture(scope="module")
def lib():
    from long_context_prefill_dhsa_b200 import binding
    return binding


@pytest.fixture(autouse=True)
def _clean_status(request):
    yield
    from long_context_prefill_dhsa_b200 import binding
    if torch.cuda.is_available() and "expects_flag" not in request.keywords:
        assert binding.check_device_status() == 0


def _bf(rng, *shape, scale=1.0):
    return torch.from_numpy((rng.standard_normal(shape) * scale).astype(np.float32)).to(torch.bfloat16).cuda()


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def _np(x):
    return x.double().cpu().numpy()


def _bits(x):
    return x.view(torch.int16 if x.element_size() == 2 else torch.int32)


# ----------------------------------------------------------------- rotary
ROT = [  # B, Hq, Hkv, T, rotary_dim, interleaved, transpose, factor, far, token_major
    (1, 1, 1, 1, 16, False, False, 1.0, 0, False),
    (1, 4, 2, 1, 128, False, False, 1.0, 1 << 20, False),
    (2, 3, 3, 7, 64, True, False, 1.25, 131071, True),
    (3, 8, 1, 65, 96, False, True, 1.0, 5000, True),
    (1, 16, 2, 1000, 112, True, True, 0.5, 2 ** 31 - 2000, False),
    (2, 5, 5, 333, 32, False, False, 1.0, 10, False),
]


@needs_gpu
@pytest.mark.parametrize("case", ROT, ids=[str(i) for i in range(len(ROT))])
def test_rotary(lib, case):
    B, Hq, Hkv, T, rd, inter, tr, factor, far, token_major = case
    rng = np.random.default_rng(T + rd)
    f = 500000.0 ** (-2.0 * np.arange(rd // 2) / rd)
    f[0] = 7.5      # more than one turn per position
    mk = lambda H: _bf(rng, B, T, H, D).transpose(1, 2) if token_major else _bf(rng, B, H, T, D)
    Q, K = mk(Hq), mk(Hkv)
    pos = rng.integers(0, far + 1, (B, T)).astype(np.int32)
    pos[0, 0] = far
    Qo, Ko, _ = lib.rotary_qkv(Q, K, torch.from_numpy(f).cuda(), positions=_i32(pos), interleaved=inter, transpose=tr,
                               factor=factor)
    for got, X in ((Qo, Q), (Ko, K)):
        x = _np(X)
        ref = oc.rotate(x, pos, f, inter, tr, factor)
        # |x| + |y| of each element's pair
        a = np.abs(x)
        s = a.copy()
        n = rd // 2
        i, j = (slice(0, rd, 2), slice(1, rd, 2)) if inter else (slice(0, n), slice(n, rd))
        s[..., i] = s[..., j] = a[..., i] + a[..., j]
        # an fp64 angle of the reference is itself off by 2^-53 of pos * f
        tol = U_BF * np.abs(ref) + (16 * U + far * 8.0 * 2.0 ** -52) * factor * s
        tol[..., rd:] = 0
        assert np.all(np.abs(_np(got) - ref) <= tol)
        assert torch.equal(_bits(got[..., rd:].contiguous()), _bits(X[..., rd:].contiguous()))


@needs_gpu
def test_rotary_positions_from_start_and_default(lib):
    rng = np.random.default_rng(1)
    Q = _bf(rng, 2, 4, 9, D)
    f = torch.from_numpy(10000.0 ** (-np.arange(64) / 64)).cuda()
    start = _i32([5, 70000])
    by_start, _, _ = lib.rotary_qkv(Q, None, f, start=start)
    by_pos, _, _ = lib.rotary_qkv(Q, None, f, positions=(start[:, None] + torch.arange(9, device="cuda").int()).int())
    assert torch.equal(by_start, by_pos)
    plain, _, _ = lib.rotary_qkv(Q, None, f)
    zero, _, _ = lib.rotary_qkv(Q, None, f, start=_i32([0, 0]))
    assert torch.equal(plain, zero)
    # position 0 leaves rows as they are; negative positions turn the other way
    neg, _, _ = lib.rotary_qkv(Q, None, f, positions=_i32(np.full((2, 9), -3)))
    ref = oc.rotate(_np(Q), np.full((2, 9), -3), f.cpu().numpy())
    assert np.all(np.abs(_np(neg) - ref) <= U_BF * np.abs(ref) + 32 * U * np.abs(_np(Q)).max())
    assert torch.equal(plain[:, :, 0], Q[:, :, 0])


@needs_gpu
def test_rotary_in_place_equals_out_of_place(lib):
    rng = np.random.default_rng(2)
    Q, K = _bf(rng, 2, 8, 50, D), _bf(rng, 2, 2, 50, D)
    f = torch.from_numpy(10000.0 ** (-np.arange(48) / 48)).cuda()
    want = lib.rotary_qkv(Q, K, f)
    lib.rotary_qkv(Q, K, f, Q_out=Q, K_out=K)
    assert torch.equal(Q, want[0]) and torch.equal(K, want[1])


@needs_gpu
@pytest.mark.parametrize("slot_major", [False, True])
def test_rotary_append_touches_only_new_slots(lib, slot_major):
    B, Hq, Hkv, T, cap = 3, 6, 2, 5, 40
    rng = np.random.default_rng(4)
    Q, K, V = _bf(rng, B, Hq, T, D), _bf(rng, B, Hkv, T, D), _bf(rng, B, Hkv, T, D)
    mk = lambda: (torch.full((B, cap, Hkv, D), 7.0, dtype=torch.bfloat16, device="cuda").transpose(1, 2) if slot_major
                  else torch.full((B, Hkv, cap, D), 7.0, dtype=torch.bfloat16, device="cuda"))
    Kc, Vc = mk(), mk()
    pc = torch.full((B, Hkv, cap), -9, dtype=torch.int32, device="cuda")
    Qo = torch.full_like(Q, 3.0)
    slots, n_new, start = [0, 17, 35], [5, 2, 0], [100, 200, 300]
    f = 10000.0 ** (-np.arange(64) / 64)
    lib.rotary_qkv(Q, K, torch.from_numpy(f).cuda(), V=V, start=_i32(start), slots=_i32(slots), n_new=_i32(n_new),
                   Q_out=Qo, K_out=Kc, V_out=Vc, pos_out=pc)
    pos = np.asarray(start)[:, None] + np.arange(T)
    rk, rq = oc.rotate(_np(K), pos, f), oc.rotate(_np(Q), pos, f)
    for b in range(B):
        n, s = n_new[b], slots[b]
        assert np.all(np.abs(_np(Kc)[b, :, s:s + n] - rk[b, :, :n]) <= U_BF * np.abs(rk[b, :, :n]) + 1e-5)
        assert np.all(np.abs(_np(Qo)[b, :, :n] - rq[b, :, :n]) <= U_BF * np.abs(rq[b, :, :n]) + 1e-5)
        assert torch.equal(Vc[b, :, s:s + n], V[b, :, :n])
        assert (pc[b, :, s:s + n].cpu().numpy() == pos[b, :n]).all()
        assert (Qo[b, :, n:] == 3.0).all()
        rest = [i for i in range(cap) if not s <= i < s + n]
        assert (Kc[b][:, rest] == 7.0).all() and (Vc[b][:, rest] == 7.0).all() and (pc[b][:, rest] == -9).all()


@needs_gpu
@pytest.mark.expects_flag
def test_rotary_slots_outside_the_cache_are_skipped_and_flagged(lib):
    rng = np.random.default_rng(5)
    K = _bf(rng, 2, 1, 4, D)
    Kc = torch.zeros(2, 1, 10, D, dtype=torch.bfloat16, device="cuda")
    f = torch.ones(8, dtype=torch.float64, device="cuda")
    lib.rotary_qkv(None, K, f, slots=_i32([8, -2]), K_out=Kc)
    with pytest.raises(lib.DHSAError) as e:
        lib.check_device_status()
    assert e.value.flags == lib.DEVFLAG_BAD_CACHE
    assert (Kc[0, 0, 8:] != 0).any(-1).all() and (Kc[0, 0, :8] == 0).all()
    assert (Kc[1, 0, :2] != 0).any(-1).all() and (Kc[1, 0, 2:] == 0).all()


@needs_gpu
def test_rotary_gradient(lib):
    """<g, rotate(x + dx)> - <g, rotate(x)> = <transpose(g), dx> within bf16."""
    rng = np.random.default_rng(6)
    B, H, T = 2, 4, 33
    f = 10000.0 ** (-np.arange(32) / 32)
    g, dx = _bf(rng, B, H, T, D), _bf(rng, B, H, T, D)
    fc = torch.from_numpy(f).cuda()
    for inter in (False, True):
        grad, _, _ = lib.rotary_qkv(g, None, fc, interleaved=inter, transpose=True)
        turned, _, _ = lib.rotary_qkv(dx, None, fc, interleaved=inter)
        a, b = np.sum(_np(grad) * _np(dx)), np.sum(_np(g) * _np(turned))
        # each side rounds every term once: u_bf of the sum of absolute terms
        assert abs(a - b) <= 1.01 * U_BF * (np.sum(np.abs(_np(grad) * _np(dx))) + np.sum(np.abs(_np(g) * _np(turned))))


# ----------------------------------------------------------------- tree attention
def _check_tree(lib, rng, B, Hq, Hkv, T, lengths, drafts, tree, weights, cap=None, scale=None, q_scale=1.0,
                slot_major=False, poison=True, in_place=False, sample=None):
    cap = cap or max(l + d for l, d in zip(lengths, drafts))
    Q = _bf(rng, B, Hq, T, D, scale=q_scale)
    mk = lambda: _bf(rng, B, cap, Hkv, D).transpose(1, 2) if slot_major else _bf(rng, B, Hkv, cap, D)
    K, V = mk(), mk()
    for b in range(B):
        if poison:
            K[b, :, lengths[b] + drafts[b]:] = float("nan")
            V[b, :, lengths[b] + drafts[b]:] = float("nan")
    parents = None
    if tree:
        parents = np.stack([[int(rng.integers(-1, t)) if t else -1 for t in range(T)] for _ in range(B)])
    out = torch.full_like(Q, 5.0)
    lse = torch.full((B, Hq, T), 5.0, device="cuda")
    w = torch.from_numpy(rng.random((B, Hkv, cap)).astype(np.float32)).cuda() if weights else None
    w0 = _np(w) if weights else None
    wo = None if not weights or in_place else torch.full_like(w, -3.0)
    got = lib.tree_attn(Q, K, V, _i32(lengths), parents=None if parents is None else _i32(parents),
                        n_draft=_i32(drafts), softmax_scale=scale, weight=w, weight_out=wo, out=out, lse=lse)
    assert got is out
    sc = 1 / math.sqrt(D) if scale is None else scale
    for b in range(B):
        n, t = lengths[b], drafts[b]
        assert (out[b, :, t:] == 5.0).all() and (lse[b, :, t:] == 5.0).all()
        heads = range(Hkv) if sample is None else sample
        G = Hq // Hkv
        for h in heads:
            q = _np(Q[b, h * G:(h + 1) * G])
            k, v = _np(K[b, h:h + 1, : n + t]), _np(V[b, h:h + 1, : n + t])
            O, L, W, A, abs_s = oc.tree_attn(q, k, v, n, None if parents is None else parents[b], t, sc)
            e = 2 * 256 * U * abs_s + 2.0 ** -20
            err = np.abs(_np(out[b, h * G:(h + 1) * G, :t]) - O)
            assert np.all(err <= (U_BF + e) * A + U_BF * np.abs(O) * (1 + U_BF) + 1e-30), (b, h, err.max())
            assert np.all(np.abs(_np(lse[b, h * G:(h + 1) * G, :t]) - L) <= e + 4 * U * np.abs(L))
            if weights:
                res = _np(w if in_place else wo)[b, h]
                old = np.concatenate([w0[b, h, :n], np.zeros(t)])
                assert np.all(np.abs(res[: n + t] - old - W[0]) <= e * W[0] + 4 * U * (old + W[0])), (b, h)
                assert np.array_equal(res[n + t:], w0[b, h, n + t:] if in_place else np.full(cap - n - t, -3.0))


TREE = [  # B, Hq, Hkv, T, lengths, drafts, tree, weights, options
    (1, 1, 1, 1, [0], [1], False, True, {}),
    (1, 2, 1, 1, [37], [1], False, False, {}),
    (3, 4, 2, 1, [127, 128, 129], [1, 1, 1], False, True, {"cap": 200}),
    (2, 8, 1, 5, [250, 251], [5, 5], True, True, {}),
    (4, 4, 4, 7, [0, 1, 300, 63], [7, 0, 3, 7], True, True, {"cap": 333}),
    (2, 14, 2, 2, [500, 13], [2, 1], False, True, {"slot_major": True}),
    (1, 16, 1, 8, [640], [8], True, False, {"in_place": False}),          # 128 rows exactly
    (1, 8, 2, 33, [1000], [33], True, True, {"in_place": True}),          # 132 rows
    (2, 8, 2, 64, [700, 5], [64, 20], True, True, {}),                    # 256 rows
    (1, 12, 1, 64, [390], [64], False, True, {}),                         # 768 rows, chain
    (1, 64, 1, 1, [1500], [1], False, True, {}),
    (1, 64, 1, 64, [300], [64], True, True, {}),                          # 4096 rows
    (5, 2, 1, 3, [0, 0, 1, 2, 3], [3, 2, 1, 0, 3], True, True, {"cap": 7}),
    (2, 4, 1, 4, [900, 257], [4, 4], True, True, {"q_scale": 20.0}),      # scores far apart
    (1, 4, 1, 4, [900], [4], True, True, {"scale": 1e-6}),
    (2, 4, 2, 3, [4000, 2500], [3, 3], True, True, {"cap": 4100}),
]


@needs_gpu
@pytest.mark.parametrize("case", TREE, ids=[f"{i}-" + "x".join(map(str, c[:4])) for i, c in enumerate(TREE)])
def test_tree_attn(lib, case):
    B, Hq, Hkv, T, lengths, drafts, tree, weights, opt = case
    _check_tree(lib, np.random.default_rng(sum(lengths) + T), B, Hq, Hkv, T, lengths, drafts, tree, weights, **opt)


@needs_gpu
def test_tree_attn_long(lib):
    """A context of many tiles over several heads and sequences, split over the device."""
    rng = np.random.default_rng(20)
    _check_tree(lib, rng, 2, 8, 2, 2, [30011, 17], [2, 2], True, True, sample=[1])
    _check_tree(lib, rng, 1, 8, 8, 20, [9001], [20], True, True, sample=[0, 7])


@needs_gpu
def test_tree_attn_defaults_and_repeat(lib):
    """n_draft None is T; the same call twice gives the same bits; parents of a chain equal None."""
    rng = np.random.default_rng(21)
    B, Hq, Hkv, T, cap = 2, 8, 2, 6, 3000
    Q, K, V = _bf(rng, B, Hq, T, D), _bf(rng, B, Hkv, cap, D), _bf(rng, B, Hkv, cap, D)
    lengths = _i32([2990, 1234])
    w = torch.zeros(B, Hkv, cap, device="cuda")
    runs = []
    for parents, nd in ((None, None), (_i32([[-1, 0, 1, 2, 3, 4]] * 2), _i32([6, 6])), (None, None)):
        wo = torch.zeros_like(w)
        runs.append((lib.tree_attn(Q, K, V, lengths, parents=parents, n_draft=nd, weight=w, weight_out=wo), wo))
    for o, wo in runs[1:]:
        assert torch.equal(o, runs[0][0]) and torch.equal(wo, runs[0][1])
    # the group's weights of one step sum to the number of its rows
    for b, n in enumerate((2996, 1240)):
        s = _np(runs[0][1])[b, :, :n].sum(-1)
        assert np.allclose(s, Hq // Hkv * T, rtol=1e-5)


@needs_gpu
def test_tree_attn_infinite_score_rows(lib):
    """A key whose score is far above all others takes the row alone; one far below takes nothing."""
    B, T, cap = 1, 1, 300
    Q = torch.zeros(B, 1, T, D, dtype=torch.bfloat16, device="cuda")
    Q[..., 0] = 3e4
    K = torch.zeros(B, 1, cap, D, dtype=torch.bfloat16, device="cuda")
    K[:, :, :, 0] = -3e4
    K[:, :, 200, 0] = 3e4
    V = _bf(np.random.default_rng(22), B, 1, cap, D)
    w = torch.zeros(B, 1, cap, device="cuda")
    out = lib.tree_attn(Q, K, V, _i32([299]), weight=w)
    assert torch.equal(out[0, 0, 0], V[0, 0, 200])
    assert w[0, 0, 200] == 1.0 and w.sum() == 1.0


@needs_gpu
@pytest.mark.expects_flag
def test_tree_attn_bad_lengths_and_parents_are_flagged(lib):
    rng = np.random.default_rng(23)
    B, T, cap = 2, 3, 50
    Q, K, V = _bf(rng, B, 2, T, D), _bf(rng, B, 1, cap, D), _bf(rng, B, 1, cap, D)
    good = lib.tree_attn(Q, K, V, _i32([20, 50]), n_draft=_i32([3, 0]))
    got = torch.zeros_like(Q)
    lib.tree_attn(Q, K, V, _i32([20, 70]), n_draft=_i32([9, 3]), out=got)
    with pytest.raises(lib.DHSAError) as e:
        lib.check_device_status()
    assert e.value.flags == lib.DEVFLAG_BAD_CACHE
    assert torch.equal(got[0], good[0]) and (got[1] == 0).all()
    lib.tree_attn(Q, K, V, _i32([-4, 48]), n_draft=_i32([1, 3]), out=got)
    with pytest.raises(lib.DHSAError) as e:
        lib.check_device_status()
    assert e.value.flags == lib.DEVFLAG_BAD_CACHE
    assert torch.equal(got[0, :, 0], V[0, 0, 0].expand(2, -1))       # nothing cached: the token itself
    roots = lib.tree_attn(Q, K, V, _i32([20, 20]), parents=_i32([[-1] * 3] * 2))
    bad = lib.tree_attn(Q, K, V, _i32([20, 20]), parents=_i32([[0, 1, 2], [-7, 5, 100]]))
    with pytest.raises(lib.DHSAError) as e:
        lib.check_device_status()
    assert e.value.flags == lib.DEVFLAG_BAD_TREE
    assert torch.equal(roots, bad)


# ----------------------------------------------------------------- eviction
def _check_evict(lib, rng, B, Hkv, cap, lengths, keep, n_draft=None, accept=None, sinks=0, recent=0, weight=None,
                 in_place=False, slot_major=False, with_index=True):
    mk = lambda: _bf(rng, B, cap, Hkv, D).transpose(1, 2) if slot_major else _bf(rng, B, Hkv, cap, D)
    K, V = mk(), mk()
    w = weight if weight is not None else rng.random((B, Hkv, cap)).astype(np.float32) ** 4
    w = torch.from_numpy(np.broadcast_to(w, (B, Hkv, cap)).copy()).cuda()
    pos = torch.from_numpy(np.argsort(rng.random((B, Hkv, cap)), -1).astype(np.int32)).cuda()
    next_pos = [cap + 3 * b for b in range(B)]
    K0, V0, w0, p0 = K.clone(), V.clone(), w.clone(), pos.clone()
    wo = w if in_place else torch.full_like(w, -3.0)
    po = pos if in_place else torch.full_like(pos, -3)
    index = torch.full((B, Hkv, min(keep, cap)), -7, dtype=torch.int32, device="cuda") if with_index else None
    out = lib.cache_evict(K, V, w, pos, _i32(lengths), keep, next_pos=_i32(next_pos) if recent else None,
                          n_draft=None if n_draft is None else _i32(n_draft),
                          accept=None if accept is None else torch.tensor(accept, dtype=torch.int64, device="cuda"),
                          sinks=sinks, recent=recent, weight_out=wo, pos_out=po, index=index)
    for b in range(B):
        for h in range(Hkv):
            src = oc.evict_rows(w0[b, h].cpu().numpy(), p0[b, h].cpu().numpy(), lengths[b],
                                0 if n_draft is None else n_draft[b], None if accept is None else accept[b], keep,
                                sinks, recent, next_pos[b] if recent else None)
            m = len(src)
            assert int(out[b]) == m
            s = torch.tensor(src, dtype=torch.int64, device="cuda")
            if with_index:
                assert torch.equal(index[b, h, :m].long(), s) and (index[b, h, m:] == -1).all(), (b, h)
            for got, old in ((K, K0), (V, V0)):
                assert torch.equal(_bits(got[b, h, :m].contiguous()), _bits(old[b, h][s]))
                assert torch.equal(_bits(got[b, h, m:].contiguous()), _bits(old[b, h, m:].contiguous()))
            assert torch.equal(_bits(wo[b, h, :m]), _bits(w0[b, h][s])) and torch.equal(po[b, h, :m], p0[b, h][s])
            if in_place:
                assert torch.equal(_bits(wo[b, h, m:]), _bits(w0[b, h, m:])) and torch.equal(po[b, h, m:], p0[b, h, m:])
            else:
                assert (wo[b, h, m:] == -3).all() and (po[b, h, m:] == -3).all()


NAN, INF = float("nan"), float("inf")
EVICT = [  # B, Hkv, cap, lengths, keep, options
    (1, 1, 1, [1], 1, {}),
    (1, 1, 1, [0], 5, {}),
    (2, 3, 70, [70, 11], 10, {"in_place": True}),
    (2, 1, 70, [64, 0], 64, {"n_draft": [6, 6], "accept": [0b101101, 0b000001]}),
    (2, 2, 80, [16, 1], 100, {"n_draft": [64, 64], "accept": [-1, -(1 << 63)]}),
    (1, 2, 500, [470], 1, {"n_draft": [30]}),
    (3, 2, 1000, [1000, 999, 501], 500, {"sinks": 4, "recent": 50, "in_place": True}),
    (1, 2, 1000, [1000], 20, {"recent": 100}),                       # more held than kept
    (2, 1, 3000, [2900, 40], 2899, {"slot_major": True}),
    (1, 1, 4099, [4099], 4098, {"with_index": False, "in_place": True}),
    (1, 2, 8193, [8193], 4000, {}),                                  # two blocks per head
    (1, 2, 40000, [39990], 7000, {"n_draft": [10], "accept": [0b1010101010], "sinks": 4, "recent": 32}),
    (2, 1, 70001, [70001, 1], 69000, {"in_place": True}),
]


@needs_gpu
@pytest.mark.parametrize("case", EVICT, ids=[str(i) for i in range(len(EVICT))])
def test_evict(lib, case):
    B, Hkv, cap, lengths, keep, opt = case
    _check_evict(lib, np.random.default_rng(cap + keep), B, Hkv, cap, lengths, keep, **opt)


@needs_gpu
@pytest.mark.parametrize("kind", ["equal", "two_values", "nan", "inf", "signs", "near", "zeros", "denormal"])
@pytest.mark.parametrize("cap", [97, 9000])
def test_evict_weights_at_the_edges(lib, kind, cap):
    rng = np.random.default_rng(cap)
    n = (1, 1, cap)
    w = {"equal": np.full(n, 0.25), "two_values": rng.integers(0, 2, n) * 0.5,
         "nan": np.where(rng.random(n) < 0.5, NAN, rng.random(n)),
         "inf": rng.choice([INF, -INF, 1.0, 0.0], n), "signs": rng.standard_normal(n),
         "near": 1.0 + rng.integers(0, 4, n) * 2.0 ** -23,
         "zeros": rng.choice([0.0, -0.0], n), "denormal": rng.integers(0, 9, n) * 1e-45}[kind].astype(np.float32)
    _check_evict(lib, rng, 1, 1, cap, [cap], cap // 3, weight=w)


@needs_gpu
def test_evict_last_block_out_of_reach_of_shared_memory(lib):
    """More slots per block than it holds keys for: the rest are ranked from memory."""
    rng = np.random.default_rng(30)
    cap = 8 * 48 * 1024 + 5000
    _check_evict(lib, rng, 1, 1, cap, [cap], 1000, sinks=2, recent=5)


@needs_gpu
@pytest.mark.expects_flag
def test_evict_bad_lengths_are_clamped_and_flagged(lib):
    rng = np.random.default_rng(31)
    K, V = _bf(rng, 2, 1, 20, D), _bf(rng, 2, 1, 20, D)
    w, pos = torch.rand(2, 1, 20, device="cuda"), torch.zeros(2, 1, 20, dtype=torch.int32, device="cuda")
    out = lib.cache_evict(K, V, w, pos, _i32([25, 15]), 18, n_draft=_i32([3, 9]))
    with pytest.raises(lib.DHSAError) as e:
        lib.check_device_status()
    assert e.value.flags == lib.DEVFLAG_BAD_CACHE
    assert out.tolist() == [18, 18]


# ----------------------------------------------------------------- together
def _cache(B, Hq, Hkv, cap, **kw):
    from long_context_prefill_dhsa_b200 import cache
    f, m = cache.rotary_inv_freq(128, base=500000.0, scaling="wavelength", factor=8.0)
    return cache.KVCache(B, Hq, Hkv, cap, f, rotary_factor=m, **kw)


@needs_gpu
def test_prefill_then_decode_with_drafts_and_eviction(lib):
    """Prefill with rotary positions, fill and score the cache, evict, then
    three drafted steps with commits, each step checked against the oracle on
    the state the step started from."""
    from long_context_prefill_dhsa_b200 import inputs as I
    w = I.custom(B=2, Hq=4, Hkv=2, L=700, lo=20, hi=120, k=3, wid=900)
    d = I.make_inputs(w)
    off, nc = (torch.from_numpy(np.ascontiguousarray(d[x])).cuda() for x in ("off", "n_chunks"))
    rng = np.random.default_rng(40)
    c = _cache(2, 4, 2, 400 + 320, sinks=4, recent=16)
    layer = lib.DHSAPrefill(2, 4, 2, 700, off, nc, w.k, inv_freq=c.inv_freq, rotary_factor=c.rotary_factor)
    Q, K = (_bf(rng, 2, 700, H, D).transpose(1, 2) for H in (4, 2))
    V = _bf(rng, 2, 2, 700, D)
    O = layer.run(Q, K, V)
    # the rotated prefill equals rotating first and prefilling then
    Qr, Kr, _ = lib.rotary_qkv(Q, K, c.inv_freq, factor=c.rotary_factor)
    plain = lib.DHSAPrefill(2, 4, 2, 700, off, nc, w.k)
    assert torch.equal(O, plain.run(Qr, Kr, V))
    c.fill(layer.Kr, V)
    c.observe(layer.Qr[:, :, -32:].contiguous())
    assert torch.allclose(c.weight[:, :, :700].sum(-1), torch.full((2, 2), 64.0, device="cuda"), rtol=1e-4)
    c.commit(_i32([0, 0]), keep=400)
    assert c.lengths.tolist() == [400, 400] and c.next_pos.tolist() == [700, 700]
    for step in range(3):
        T = (1, 9, 16)[step]
        parents = None if T == 1 else _i32([[t - 1 - (t % 3 == 2) if t else -1 for t in range(T)]] * 2)
        depth = None if T == 1 else _i32([[sum(1 for _ in _up(parents[0].tolist(), t)) for t in range(T)]] * 2)
        q, k, v = _bf(rng, 2, 4, T, D), _bf(rng, 2, 2, T, D), _bf(rng, 2, 2, T, D)
        n0, p0 = c.lengths.tolist(), c.next_pos.clone()
        w0 = _np(c.weight)
        qr = c.extend(q, k, v, depth=depth)
        out = c.attend(qr, parents=parents)
        at = (p0[:, None].cpu().numpy() + (np.zeros((2, 1)) if depth is None else depth.cpu().numpy())).astype(np.int64)
        f = c.inv_freq.cpu().numpy()
        ref = oc.rotate(_np(k), at, f, factor=c.rotary_factor)
        for b in range(2):
            new = _np(c.K)[b, :, n0[b]: n0[b] + T]
            assert np.all(np.abs(new - ref[b]) <= U_BF * np.abs(ref[b]) + 1e-5)
            assert (c.pos[b, :, n0[b]: n0[b] + T].cpu().numpy() == at[b]).all()
            G = 2
            for h in range(2):
                Or, _, W, A, abs_s = oc.tree_attn(_np(qr[b, h * G:(h + 1) * G]), _np(c.K[b, h:h + 1]),
                                                  _np(c.V[b, h:h + 1]), n0[b],
                                                  None if parents is None else parents[b].tolist(), T, 1 / math.sqrt(D))
                e = 512 * U * abs_s + 2.0 ** -20
                assert np.all(np.abs(_np(out[b, h * G:(h + 1) * G]) - Or) <= (U_BF + e) * A + 1.01 * U_BF * np.abs(Or))
                old = np.concatenate([w0[b, h, : n0[b]], np.zeros(T)])
                assert np.all(np.abs(_np(c.weight)[b, h, : n0[b] + T] - old - W[0]) <= e * W[0] + 4 * U * (old + W[0]))
        accept = None if T == 1 else torch.tensor([0b1011, 0b111], dtype=torch.int64, device="cuda")
        wb, pb, Kb = c.weight.cpu().numpy(), c.pos.cpu().numpy(), c.K.clone()
        nb = c.next_pos.tolist()
        c.commit(_i32([T, T]), accept=accept, keep=400)
        for b in range(2):
            for h in range(2):
                src = oc.evict_rows(wb[b, h], pb[b, h], n0[b], T, None if accept is None else int(accept[b]), 400, 4,
                                    16, nb[b])
                assert int(c.lengths[b]) == len(src) == 400
                assert torch.equal(c.K[b, h, : len(src)], Kb[b, h][torch.tensor(src, device="cuda")])
                assert (c.pos[b, h, : len(src)].cpu().numpy() == pb[b, h][src]).all()
    assert c.next_pos.tolist() == [700 + 1 + 3 + 3] * 2


def _up(parents, t):
    """The ancestors of t in a tree."""
    while parents[t] >= 0:
        t = parents[t]
        yield t


@needs_gpu
def test_captured_step_replays_like_eager_steps(lib):
    """A whole decoding step as a CUDA graph, replayed, against eager steps;
    two graphs share one cache's workspace, replayed in turn on a side stream."""
    rng = np.random.default_rng(41)
    B, Hq, Hkv, cap, T = 2, 8, 2, 300, 2
    prompt = [_bf(rng, B, Hkv, 200, D) for _ in range(2)]
    steps = [[_bf(rng, B, H, T, D) for H in (Hq, Hkv, Hkv)] for _ in range(4)]
    nd = _i32([T, T])

    def step(c, q, k, v, out, keep):
        qr = c.extend(q, k, v)
        c.attend(qr, out=out)
        c.commit(nd, keep=keep)

    eager, outs = _cache(B, Hq, Hkv, cap, recent=8), []
    eager.fill(*prompt)
    for i, (q, k, v) in enumerate(steps):
        o = torch.empty_like(q)
        step(eager, q, k, v, o, 202 - i % 2)
        outs.append(o)

    c = _cache(B, Hq, Hkv, cap, recent=8)
    c.fill(*prompt)
    bufs = [[x.clone() for x in steps[0]] + [torch.empty_like(steps[0][0])] for _ in range(2)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graphs = []
    with torch.cuda.stream(s):
        for i in range(2):
            step(c, *bufs[i], 202 - i)            # one eager run before capture
        for i in range(2):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                step(c, *bufs[i], 202 - i)
            graphs.append(g)
        c.fill(*prompt)
        c.lengths.fill_(200)
        for i, x in enumerate(steps):
            for dst, src in zip(bufs[i % 2], x):
                dst.copy_(src)
            graphs[i % 2].replay()
            assert torch.equal(bufs[i % 2][3], outs[i]), i
    s.synchronize()
    assert torch.equal(c.K[:, :, :201], eager.K[:, :, :201]) and torch.equal(c.pos[:, :, :201], eager.pos[:, :, :201])
    assert torch.equal(c.weight[:, :, :201], eager.weight[:, :, :201]) and torch.equal(c.lengths, eager.lengths)


@needs_gpu
def test_two_streams_with_their_own_workspaces(lib):
    rng = np.random.default_rng(42)
    sets = []
    for _ in range(2):
        Q, K, V = _bf(rng, 2, 8, 4, D), _bf(rng, 2, 2, 5000, D), _bf(rng, 2, 2, 5000, D)
        n = _i32([4990, 3333])
        sets.append((Q, K, V, n, lib.tree_attn(Q, K, V, n)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(20):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                Q, K, V, n, _ = sets[i]
                got[i].append(lib.tree_attn(Q, K, V, n))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o, sets[i][4]) for o in got[i])


@needs_gpu
def test_evict_more_slots_than_a_cluster_holds_keys_for(lib):
    """A cache so long that the largest cluster ranks the rest of its slots from memory."""
    rng = np.random.default_rng(33)
    cap = 16 * 48 * 1024 + 7000
    _check_evict(lib, rng, 1, 1, cap, [cap - 5], 900, n_draft=[5], accept=[0b10011], sinks=2, recent=5)


SPLIT = [  # as TREE, with caches long enough that several CTAs share an item
    (1, 4, 1, 1, [1100], [1], False, True, {"cap": 1101}),                    # a few rows, by items
    (1, 40, 1, 1, [2000], [1], False, True, {}),                              # 40 rows: K is read again
    (2, 8, 1, 9, [1500, 1029], [9, 4], True, True, {}),                       # 72 rows: both lane halves
    (1, 16, 2, 16, [2300], [16], True, True, {"slot_major": True}),           # 128 rows
    (3, 8, 2, 40, [1300, 0, 1290], [40, 0, 33], True, True, {"in_place": True}),   # 160 rows: two query tiles
    (1, 8, 1, 64, [1700], [64], False, True, {}),                             # 512 rows: two query blocks
    (40, 8, 4, 2, [1200 - 29 * b for b in range(40)], [b % 3 for b in range(40)], True, True, {"cap": 1210}),
    (40, 2, 1, 1, [1900] + [5] * 39, [1] * 40, False, True, {}),              # one long, many short
    (200, 1, 1, 1, [1500 if b in (3, 150) else 7 * b for b in range(200)], [int(b in (3, 150)) for b in range(200)],
     False, True, {"cap": 1600}),                                             # most sequences have no new token
    (150, 4, 1, 3, [(37 * b) % 1400 for b in range(150)], [3] * 150, True, False, {"cap": 1410}),
]


@needs_gpu
@pytest.mark.parametrize("case", SPLIT, ids=[f"{i}-" + "x".join(map(str, c[:4])) for i, c in enumerate(SPLIT)])
def test_tree_attn_split(lib, case):
    B, Hq, Hkv, T, lengths, drafts, tree, weights, opt = case
    _check_tree(lib, np.random.default_rng(sum(lengths) + T), B, Hq, Hkv, T, lengths, drafts, tree, weights, **opt)


@needs_gpu
def test_tree_attn_garbage_behind_the_rows_and_slots(lib):
    """Rows of missing tokens hold NaN queries, slots behind the last one NaN
    keys and values, weights of unused slots NaN: none of it shows."""
    rng = np.random.default_rng(24)
    for G, T, n in ((2, 4, 300), (8, 30, 2000)):
        cap = n + 77
        Q, K, V = _bf(rng, 2, G, T, D), _bf(rng, 2, 1, cap, D), _bf(rng, 2, 1, cap, D)
        nd = [T, T // 2]
        clean = torch.zeros(2, 1, cap, device="cuda")
        ref, wref = torch.zeros_like(Q), torch.zeros_like(clean)
        lib.tree_attn(Q, K, V, _i32([n, n - 200]), n_draft=_i32(nd), weight=clean, weight_out=wref, out=ref)
        nan = float("nan")
        w = clean.clone()
        Q[1, :, nd[1]:] = nan
        for b, end in enumerate((n + nd[0], n - 200 + nd[1])):
            K[b, :, end:] = nan
            V[b, :, end:] = nan
            w[b, :, end - nd[b]:] = nan
        got, wgot = torch.zeros_like(Q), torch.zeros_like(w)
        lib.tree_attn(Q, K, V, _i32([n, n - 200]), n_draft=_i32(nd), weight=w, weight_out=wgot, out=got)
        assert torch.equal(got, ref) and torch.equal(wgot, wref)


@needs_gpu
def test_streamed_and_graphed_prefill_with_rotary_positions(lib):
    from long_context_prefill_dhsa_b200 import inputs as I
    w = I.custom(B=1, Hq=4, Hkv=2, L=500, lo=20, hi=120, k=3, wid=901)
    d = I.make_inputs(w)
    off, nc = (torch.from_numpy(np.ascontiguousarray(d[x])).cuda() for x in ("off", "n_chunks"))
    f = torch.from_numpy(10000.0 ** (-np.arange(64) / 64)).cuda()
    mk = lambda: lib.DHSAPrefill(1, 4, 2, 500, off, nc, w.k, inv_freq=f, interleaved=True)
    rng = np.random.default_rng(43)
    steps = [[_bf(rng, 1, H, 500, D) for H in (4, 2, 2)] for _ in range(3)]
    want = [mk().run(*s).clone() for s in steps]
    streamed = lib.HostStreamedPrefill(mk())
    host = [[x.cpu().pin_memory() for x in s] + [torch.empty(1, 4, 500, D, dtype=torch.bfloat16).pin_memory()]
            for s in steps]
    torch.cuda.synchronize()
    for h in host:
        streamed.submit(*h)
    streamed.synchronize()
    graphed = lib.GraphedPrefill(mk(), *[x.clone() for x in steps[0]])
    for s, h, o in zip(steps, host, want):
        for dst, src in zip((graphed.Q, graphed.K, graphed.V), s):
            dst.copy_(src)
        assert torch.equal(graphed.replay(), o) and torch.equal(h[3].cuda(), o)


@needs_gpu
def test_calls_on_a_side_stream_and_with_a_callers_workspace(lib):
    """A workspace full of NaN, a side stream: the same bits as the plain call."""
    rng = np.random.default_rng(44)
    B, Hq, Hkv, T, cap = 2, 8, 2, 3, 5000
    Q, K, V = _bf(rng, B, Hq, T, D), _bf(rng, B, Hkv, cap, D), _bf(rng, B, Hkv, cap, D)
    n, w = _i32([4990, 2000]), torch.rand(B, Hkv, cap, device="cuda")
    wo = torch.zeros_like(w)
    want = lib.tree_attn(Q, K, V, n, weight=w, weight_out=wo)
    size = lib.load().dhsa_tree_attn_workspace_size(B, Hq, Hkv, T, cap, 1)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")
        got_w = torch.zeros_like(w)
        got = lib.tree_attn(Q, K, V, n, weight=w, weight_out=got_w, workspace=ws)
    s.synchronize()
    assert torch.equal(got, want) and torch.equal(got_w, wo)
    with pytest.raises(lib.DHSAError):
        lib.tree_attn(Q, K, V, n, weight=w, workspace=ws[: size - 256])
    with pytest.raises(ValueError):
        lib.tree_attn(Q, K, V, n.cpu(), weight=w)
    with pytest.raises(ValueError):
        lib.tree_attn(Q, K[:, :, :, ::1].transpose(2, 3), V, n)
    with pytest.raises(lib.DHSAError):
        lib.tree_attn(Q, K, V, n, out=Q)


@needs_gpu
def test_layers_share_a_workspace(lib):
    """Two caches with one workspace, stepped in turn, against two with their own."""
    from long_context_prefill_dhsa_b200 import cache
    rng = np.random.default_rng(45)
    B, Hq, Hkv, cap = 2, 8, 2, 1500
    ws = torch.empty(cache.KVCache.workspace_size(B, Hq, Hkv, cap), dtype=torch.uint8, device="cuda")
    pairs = [[_cache(B, Hq, Hkv, cap, recent=4, workspace=w) for _ in range(2)] for w in (ws, None)]
    prompts = [[_bf(rng, B, Hkv, 1400, D) for _ in range(2)] for _ in range(2)]
    for layers in pairs:
        for c, x in zip(layers, prompts):
            c.fill(*x)
    for T in (1, 5, 40):
        x = [[_bf(rng, B, H, T, D) for H in (Hq, Hkv, Hkv)] for _ in range(2)]
        outs = []
        for layers in pairs:
            for c, (q, k, v) in zip(layers, x):
                outs.append(c.attend(c.extend(q, k, v)))
                c.commit(_i32([T, T]), keep=1398)
        assert torch.equal(outs[0], outs[2]) and torch.equal(outs[1], outs[3])
    for a, b in zip(*pairs):
        assert torch.equal(a.K, b.K) and torch.equal(a.weight, b.weight) and torch.equal(a.pos, b.pos)


@needs_gpu
@pytest.mark.parametrize("scale", [1e-38, 1e-30, 1e30])
def test_tree_attn_extreme_scales(lib, scale):
    """A scale so small that every slot weighs the same, one so large that the best slot takes all."""
    rng = np.random.default_rng(46)
    n = 700
    Q, K, V = _bf(rng, 1, 2, 1, D), _bf(rng, 1, 1, n + 1, D), _bf(rng, 1, 1, n + 1, D)
    out = lib.tree_attn(Q, K, V, _i32([n]), softmax_scale=scale)
    s = _np(K[0, 0]) @ _np(Q[0, :, 0]).T
    v = _np(V[0, 0])
    for h in range(2):
        want = v.mean(0) if scale < 1 else v[s[:, h].argmax()]
        tol = U_BF * (np.abs(v).mean(0) + np.abs(want)) * 1.01 if scale < 1 else 0
        assert np.all(np.abs(_np(out[0, h, 0]) - want) <= tol)


@needs_gpu
@pytest.mark.parametrize("T", [1, 12])          # 4 and 48 rows of a head: scores kept, and computed again
@pytest.mark.parametrize("scale", [1e-30, 1e30])
def test_slot_weights_at_extreme_scales(lib, scale, T):
    """Every slot that a token sees gets the same weight, or the best one all of it.

    Small: the exponent -log2 l, |log2 l| < 9.6, passes through a handful of fp32 operations (log2,
    a division, three parts, two sums, a product: 8 half steps of it at most, twice that if the tensor
    core truncates), and log2, exp2 and 1 / l add 2^-22 each: 9.6 ln 2 * 16 U + 3 * 2^-22 < 8e-6."""
    rng = np.random.default_rng(47)
    n = 700
    Q, K, V = _bf(rng, 1, 4, T, D), _bf(rng, 1, 1, n + T, D), _bf(rng, 1, 1, n + T, D)
    w = torch.zeros(1, 1, n + T, device="cuda")
    lib.tree_attn(Q, K, V, _i32([n]), softmax_scale=scale, weight=w)
    s = _np(Q[0]) @ _np(K[0, 0]).T
    want = np.zeros(n + T)
    for h in range(4):
        for t in range(T):
            if scale < 1:
                want[: n + t + 1] += 1 / (n + t + 1)
            else:
                want[s[h, t, : n + t + 1].argmax()] += 1
    got = _np(w[0, 0])
    assert np.all(np.abs(got - want) <= (8e-6 * want if scale < 1 else 0))


def _three_calls(lib, rng):
    """Arguments of the three calls with every optional one, caches as views of slot-major storage."""
    B, Hq, Hkv, T, cap = 2, 4, 2, 3, 40
    cache = lambda: _bf(rng, B, cap, Hkv, D).transpose(1, 2)
    f = torch.from_numpy(10000.0 ** (-np.arange(64) / 64)).cuda()
    n, t = _i32([20, 31]), _i32([3, 2])
    wt = lambda: torch.from_numpy(rng.random((B, Hkv, cap)).astype(np.float32)).cuda()
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")
    return {
        "rotary_qkv": dict(Q=_bf(rng, B, T, Hq, D).transpose(1, 2), K=_bf(rng, B, T, Hkv, D).transpose(1, 2), inv_freq=f,
                           V=_bf(rng, B, Hkv, T, D), start=n.clone(), n_new=t, slots=n, Q_out=torch.zeros_like(_bf(rng, B, Hq, T, D)),
                           K_out=cache(), V_out=cache(), pos_out=i32(B, Hkv, cap), factor=1, interleaved=True),
        "tree_attn": dict(Q=_bf(rng, B, Hq, T, D), K=cache(), V=cache(), lengths=n, parents=_i32([[-1, 0, 0], [-1, 0, 1]]),
                          n_draft=t, softmax_scale=0.25, weight=wt(), weight_out=wt(), out=_bf(rng, B, Hq, T, D),
                          lse=torch.zeros(B, Hq, T, device="cuda")),
        "cache_evict": dict(K=cache(), V=cache(), weight=wt(), pos=i32(B, Hkv, cap), lengths=n, keep=12, next_pos=n + 3,
                            n_draft=t, accept=torch.tensor([5, 1], device="cuda"), sinks=0, recent=4, weight_out=wt(),
                            pos_out=i32(B, Hkv, cap), lengths_out=i32(B), index=i32(B, Hkv, 12)),
    }


class _TakesNothing:
    def __getattr__(self, name):
        return lambda *a: None


@needs_gpu
@pytest.mark.parametrize("name", ["rotary_qkv", "tree_attn", "cache_evict"])
@pytest.mark.parametrize("optional", [True, False])
def test_calls_with_their_checks_in_python(lib, monkeypatch, name, optional):
    """The compiled checks take an ordinary call, and make the same one as the checks in Python."""
    results = []
    for python in (False, True):
        a = _three_calls(lib, np.random.default_rng(51))[name]
        if not optional:
            for k in ("Q_out", "K_out", "V_out", "pos_out", "slots", "n_new", "out", "lse", "weight_out", "lengths_out",
                      "index", "softmax_scale"):
                a.pop(k, None)
        if name == "tree_attn" and not optional:
            a["n_draft"], a["parents"] = None, None     # rows of missing tokens of a new `out` hold anything
        lib._load_marshal()
        with monkeypatch.context() as m:
            if python:
                m.setattr(lib, "_marshal", _TakesNothing())
            else:
                real, taken = lib._marshal, []

                class Watch:
                    def __getattr__(self, n):
                        def call(*x):
                            taken.append(getattr(real, n)(*x))
                            return taken[-1]
                        return call
                m.setattr(lib, "_marshal", Watch())
            r = getattr(lib, name)(**a)
            assert python or (len(taken) == 1 and taken[0] is not None and type(taken[0]) is not int)
        tensors = [x for x in a.values() if isinstance(x, torch.Tensor)]
        results.append(tensors + list(r if isinstance(r, tuple) else (r,)))
        if name == "rotary_qkv" and optional:
            assert r[0] is a["Q_out"] and r[1] is a["K_out"] and r[2] is a["V_out"]
        elif optional:
            assert r is (a["out"] if name == "tree_attn" else a["lengths_out"])
    for x, y in zip(*results):
        assert torch.equal(x, y)


@needs_gpu
@pytest.mark.parametrize("name", ["rotary_qkv", "tree_attn", "cache_evict"])
def test_every_tensor_is_checked(lib, name):
    """Each tensor of each call with another type, shape, layout or place is refused, before anything runs."""
    good = _three_calls(lib, np.random.default_rng(52))[name]
    rows = {"Q", "K", "V", "K_out", "V_out"} - ({"Q"} if name == "tree_attn" else set())
    for key, t in good.items():
        if not isinstance(t, torch.Tensor):
            continue
        other = torch.float64 if t.dtype != torch.float64 else torch.float32
        bad = [t.to(other), torch.cat([t, t], -1), t.cpu(), t.tolist()]
        wide = torch.zeros(*t.shape, 2, dtype=t.dtype, device="cuda")[..., 0]        # elements two apart
        if t.dim() > 1 or t.numel() > 1:
            bad.append(wide)
        if key not in rows and t.dim() > 1:
            bad.append(torch.zeros(*t.shape[1:], t.shape[0], dtype=t.dtype, device="cuda").movedim(-1, 0))
        for b in bad:
            if key == "inv_freq" and b is bad[1]:
                b = torch.cat([t, t])                # 256 rotated elements of 128
            with pytest.raises((TypeError, ValueError, lib.DHSAError)):
                getattr(lib, name)(**{**good, key: b})
    for key in {"rotary_qkv": ["inv_freq"], "tree_attn": ["Q", "K", "V", "lengths"],
                "cache_evict": ["K", "V", "weight", "pos", "lengths"]}[name]:
        with pytest.raises((TypeError, ValueError, AttributeError, lib.DHSAError)):
            getattr(lib, name)(**{**good, key: None})
    torch.cuda.synchronize()


@needs_gpu
@pytest.mark.parametrize("case", [
    (1, 1, 800_000, [799_990], 100_000, {"n_draft": [10], "accept": [0b1100110011], "sinks": 4, "recent": 64}),
    (2, 1, 790_000, [790_000, 17], 700_001, {"in_place": True, "with_index": False}),    # 49K slots a block
    (3, 5, 131_072, [131_072, 131_000, 70_000], 5000, {"recent": 32}),     # more heads than clusters of 16 at a time
], ids=["1x800k", "2x790k", "15x128k"])
def test_evict_blocks_with_more_slots_than_keys_and_many_heads(lib, case):
    B, Hkv, cap, lengths, keep, opt = case
    _check_evict(lib, np.random.default_rng(cap), B, Hkv, cap, lengths, keep, **opt)
