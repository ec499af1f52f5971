"""Bounded waits of the attention of drafted tokens, made to run out.

The library's test hook (include/dhsa.h, 5) keeps the kernels from loading
any key tile, so the waits for the first tile run out after a short limit:
before any MMA, with no copy in flight. The call returns, the flag is
reported, what the joining kernels read of an unwritten workspace stays in
range, and the next call is correct. Nothing traps."""
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


def _bf(rng, *shape):
    return torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(torch.bfloat16).cuda()


def _flags(lib):
    try:
        return lib.check_device_status()
    except lib.DHSAError as e:
        return e.flags


CASES = [  # B, Hq, Hkv, T, slots, weights
    (1, 2, 1, 1, 300, False),        # a whole item a CTA: nothing joins
    (2, 8, 2, 1, 5000, True),        # shared items, weights from the kept scores
    (2, 8, 2, 3, 5000, False),       # shared items, rows joined
    (1, 8, 1, 12, 500, True),        # 96 rows: weights from K again
    (1, 8, 1, 12, 5000, True),
    (1, 8, 2, 50, 3000, True),       # 200 rows: two query tiles a CTA
    (2, 16, 2, 40, 600, False),      # 320 rows: two query blocks
]


@needs_gpu
@pytest.mark.parametrize("fill", ["zeros", "ones", "random"])
@pytest.mark.parametrize("case", CASES, ids=["x".join(map(str, c[:5])) for c in CASES])
def test_waits_run_out_then_recover(lib, case, fill):
    B, Hq, Hkv, T, n, weights = case
    rng = np.random.default_rng(90 + T)
    cap = n + T + 3
    Q, K, V = _bf(rng, B, Hq, T, D), _bf(rng, B, Hkv, cap, D), _bf(rng, B, Hkv, cap, D)
    lengths = torch.full((B,), n, dtype=torch.int32, device="cuda")
    w = torch.rand(B, Hkv, cap, device="cuda") if weights else None
    size = lib.load().dhsa_tree_attn_workspace_size(B, Hq, Hkv, T, cap, weights)
    lo, hi = {"zeros": (0, 1), "ones": (255, 256), "random": (0, 256)}[fill]
    left = torch.randint(lo, hi, (size + 4096,), dtype=torch.uint8, device="cuda")     # by an earlier call, say
    space = left.clone()

    def call():
        out = torch.full_like(Q, 7.0)
        wo = torch.full_like(w, -3.0) if weights else None
        lib.tree_attn(Q, K, V, lengths, weight=w, weight_out=wo, out=out, workspace=space[:size])
        return out, wo

    want, want_w = call()
    assert _flags(lib) == 0
    space.copy_(left)
    torch.cuda.synchronize()
    lib.debug_arm_wait_timeout(1, 50_000)            # 50 us
    out, wo = call()
    assert _flags(lib) == lib.DEVFLAG_WAIT_TIMEOUT
    assert torch.equal(space[size:], left[size:])
    if cap <= 640:                                   # whole items: no kernel writes their rows
        assert (out == 7.0).all()
    if weights:
        assert (wo[..., n + T:] == -3.0).all()       # nothing behind the last slot
    # the hook is one-shot
    again, again_w = call()
    assert _flags(lib) == 0
    assert torch.equal(again, want) and (not weights or torch.equal(again_w, want_w))


@needs_gpu
def test_a_disarmed_hook_changes_nothing(lib):
    rng = np.random.default_rng(91)
    Q, K, V = _bf(rng, 1, 4, 2, D), _bf(rng, 1, 2, 900, D), _bf(rng, 1, 2, 900, D)
    lengths = torch.full((1,), 890, dtype=torch.int32, device="cuda")
    want = lib.tree_attn(Q, K, V, lengths)
    lib.debug_arm_wait_timeout(1, 50_000)
    lib.debug_arm_wait_timeout(0)
    assert torch.equal(lib.tree_attn(Q, K, V, lengths), want)
    # armed for the routing, the attention does not take it
    lib.debug_arm_wait_timeout(2, 50_000)
    assert torch.equal(lib.tree_attn(Q, K, V, lengths), want)
    lib.debug_arm_wait_timeout(0)
    assert _flags(lib) == 0
