"""GPU tests of KVCache.commit where the budget is about as large as what is
held. Expected positions are worked out from the positions alone, not from
the order in which commit does its steps."""
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


# sinks, recent, keep, tokens of each step, tokens accepted (the first ones of the chain), of two sequences.
# Where keep <= sinks + recent + accepted, the sinks and the last keep - sinks positions are what stays.
WINDOW = [
    (4, 8, 12, [1, 1, 1, 1, 1], [(1, 1)] * 5),                # a budget of exactly sinks + recent
    (4, 8, 12, [5, 3, 7], [(3, 1), (0, 3), (7, 2)]),          # drafts, some of them accepted
    (4, 8, 13, [3, 3], [(3, 2), (2, 3)]),                     # room for some of the earlier window
    (4, 8, 7, [1, 4], [(1, 1), (4, 2)]),                      # less than sinks + recent
    (4, 8, 6, [9], [(9, 5)]),                                 # more accepted than there is room for
    (0, 0, 6, [10, 1], [(10, 7), (1, 1)]),                    # the same with nothing held by request
    (0, 16, 16, [1, 64, 2], [(1, 1), (64, 20), (1, 2)]),      # no sinks, a whole step of drafts
]


@needs_gpu
@pytest.mark.parametrize("track", [False, True], ids=["unweighted", "weighted"])
@pytest.mark.parametrize("case", WINDOW, ids=[str(i) for i in range(len(WINDOW))])
def test_the_newest_tokens_stay_when_the_budget_is_what_is_held(lib, case, track):
    from long_context_prefill_dhsa_b200 import cache
    sinks, recent, keep, steps, accepted = case
    rng = np.random.default_rng(60 + keep)
    B, Hq, Hkv, cap, L = 2, 4, 2, 160, 40
    f, m = cache.rotary_inv_freq(128)
    c = cache.KVCache(B, Hq, Hkv, cap, f, rotary_factor=m, track_weight=track, sinks=sinks, recent=recent)
    c.fill(_bf(rng, B, Hkv, L, D), _bf(rng, B, Hkv, L, D))
    if track:
        c.observe(_bf(rng, B, Hq, 8, D))
    # the rows that belong to each position
    at = [{p: (c.K[b, :, p].clone(), c.V[b, :, p].clone()) for p in range(L)} for b in range(B)]
    seen = [L] * B
    for step, T in enumerate(steps):
        n0 = c.lengths.tolist()
        q = c.extend(_bf(rng, B, Hq, T, D), _bf(rng, B, Hkv, T, D), _bf(rng, B, Hkv, T, D))
        c.attend(q)
        acc = [min(a, T) for a in accepted[step]]
        for b in range(B):
            for t in range(acc[b]):
                at[b][seen[b] + t] = (c.K[b, :, n0[b] + t].clone(), c.V[b, :, n0[b] + t].clone())
            seen[b] += acc[b]
        bits = [(1 << a) - 1 if a < 64 else -1 for a in acc]
        c.commit(_i32([T] * B), accept=torch.tensor(bits, dtype=torch.int64, device="cuda"), keep=keep)
        assert c.next_pos.tolist() == seen
        for b in range(B):
            if sinks + recent + acc[b] < keep:
                continue               # room left over, which goes by weight
            want = sorted(set(range(min(sinks, keep))) | set(range(seen[b] - (keep - sinks), seen[b])))
            for h in range(Hkv):
                n = int(c.lengths[b])
                pos = c.pos[b, h, :n].tolist()
                assert sorted(pos) == want, (step, b, h)
                for s, p in enumerate(pos):
                    assert torch.equal(c.K[b, h, s], at[b][p][0][h]) and torch.equal(c.V[b, h, s], at[b][p][1][h])


@needs_gpu
def test_a_captured_step_with_a_budget_of_what_is_held(lib):
    """A drafted step captured once and replayed with other drafts and other accepted ones."""
    from long_context_prefill_dhsa_b200 import cache
    sinks, recent, keep, T, B, Hq, Hkv, L = 4, 8, 12, 5, 2, 4, 2, 40
    rng = np.random.default_rng(62)
    f, m = cache.rotary_inv_freq(128)
    c = cache.KVCache(B, Hq, Hkv, 64, f, rotary_factor=m, sinks=sinks, recent=recent)
    q, k, v = _bf(rng, B, Hq, T, D), _bf(rng, B, Hkv, T, D), _bf(rng, B, Hkv, T, D)
    n_new, accept = _i32([T] * B), torch.zeros(B, dtype=torch.int64, device="cuda")

    def step():
        c.attend(c.extend(q, k, v))
        c.commit(n_new, accept=accept, keep=keep)

    def start():
        c.fill(prompt, prompt)
        c.commit(_i32([0] * B), keep=keep)

    prompt = _bf(rng, B, Hkv, L, D)
    start()
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    start()
    seen = [L] * B
    for acc in ((5, 1), (0, 2), (3, 5), (1, 0), (5, 5)):
        for x in (q, k, v):
            x.copy_(_bf(rng, *x.shape))
        accept.copy_(torch.tensor([(1 << a) - 1 for a in acc], device="cuda"))
        g.replay()
        for b in range(B):
            seen[b] += acc[b]
            want = list(range(sinks)) + list(range(seen[b] - recent, seen[b]))
            for h in range(Hkv):
                assert sorted(c.pos[b, h, : int(c.lengths[b])].tolist()) == want
    assert c.next_pos.tolist() == seen
