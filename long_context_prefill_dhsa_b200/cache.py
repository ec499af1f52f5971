"""The key/value cache of a layer after its prefill: rotary frequencies, and
KVCache, which chains the cache's calls (binding.rotary_qkv, tree_attn,
cache_evict) for one layer with buffers allocated once.
"""
from __future__ import annotations

import math
from typing import Optional

import torch

from . import binding


def rotary_inv_freq(rotary_dim: int, base: float = 10000.0, scaling: Optional[str] = None, factor: float = 1.0,
                    original: int = 8192, low: float = 1.0, high: float = 4.0, beta_fast: float = 32.0,
                    beta_slow: float = 1.0, device="cuda"):
    """(inv_freq, factor) of rotary positions, as binding.rotary_qkv takes them:
    float64 [rotary_dim/2] radians per position, and the factor on cos and sin.

    inv_freq[i] = base ** (-2 i / rotary_dim), rescaled for contexts `factor`
    times longer than the `original` one:
      None          not rescaled
      "linear"      divided by factor
      "ntk"         base * factor ** (rotary_dim / (rotary_dim - 2)): the last
                    pair is stretched by factor, the first not at all
      "wavelength"  pairs with fewer than `low` turns over the original context
                    divided by factor, those with more than `high` kept, a
                    linear blend in between
      "yarn"        the same idea with a ramp over the pair index between
                    beta_fast and beta_slow turns, and cos and sin times
                    0.1 ln(factor) + 1
    """
    if rotary_dim < 16 or rotary_dim > 128 or rotary_dim % 16:
        raise ValueError("rotary_dim: a multiple of 16 from 16 to 128")
    if base <= 1 or factor < 1:
        raise ValueError("base must be above 1 and factor at least 1")
    if scaling == "ntk":
        base = base * factor ** (rotary_dim / (rotary_dim - 2))
    f = [base ** (-2.0 * i / rotary_dim) for i in range(rotary_dim // 2)]
    mscale = 1.0
    if scaling == "linear":
        f = [x / factor for x in f]
    elif scaling == "wavelength":
        if not low < high:
            raise ValueError("low must be below high")
        keep = [min(1.0, max(0.0, (original * x / (2 * math.pi) - low) / (high - low))) for x in f]
        f = [k * x + (1 - k) * x / factor for k, x in zip(keep, f)]
    elif scaling == "yarn":
        def at(turns):
            return rotary_dim * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(base))
        first, last = max(math.floor(at(beta_fast)), 0), min(math.ceil(at(beta_slow)), rotary_dim - 1)
        ramp = [min(1.0, max(0.0, (i - first) / max(last - first, 1e-3))) for i in range(len(f))]
        f = [(1 - r) * x + r * x / factor for r, x in zip(ramp, f)]
        mscale = 0.1 * math.log(factor) + 1.0
    elif scaling not in (None, "ntk"):
        raise ValueError(f"unknown scaling {scaling!r}")
    return torch.tensor(f, dtype=torch.float64, device=device), mscale


class KVCache:
    """Cached keys and values of one layer, from its prefill on.

    A step of T new tokens (T = 1: decoding; more: a drafted tree) is
      q = cache.extend(Q, K, V, depth)     rotary positions; K, V into the slots after the cached ones
      O = cache.attend(q, parents)         attention over the cache and the step's own tokens
      cache.commit(T, accept, keep)        accepted tokens stay, the rest is dropped; at most `keep` slots stay,
                                           the first `sinks` and the last `recent` positions first

    K, V [B,Hkv,cap,128], weight (fp32) and pos (int32) [B,Hkv,cap], lengths
    and next_pos (int32 [B]) are the state; every call runs on the current
    stream and none synchronises. Not for use from two streams at once.
    Caches used one after the other (the layers of a model) can share one
    `workspace` (uint8, workspace_size bytes). Tokens that lead past `cap` are
    not stored and raise DHSA_DEVFLAG_BAD_CACHE (binding.check_device_status).
    """

    def __init__(self, B: int, Hq: int, Hkv: int, cap: int, inv_freq: torch.Tensor, interleaved: bool = False,
                 rotary_factor: float = 1.0, softmax_scale: Optional[float] = None, track_weight: bool = True,
                 sinks: int = 0, recent: int = 0, workspace: Optional[torch.Tensor] = None, device="cuda"):
        dev = torch.device(device)
        self.B, self.Hq, self.Hkv, self.cap = B, Hq, Hkv, cap
        self.inv_freq, self.interleaved, self.rotary_factor = inv_freq, interleaved, rotary_factor
        self.scale, self.track_weight, self.sinks, self.recent = softmax_scale, track_weight, sinks, recent
        # zeros, not empty: a fresh cache has no unkept slot that could hold NaN weights
        self.K = torch.zeros((B, Hkv, cap, 128), dtype=torch.bfloat16, device=dev)
        self.V = torch.zeros_like(self.K)
        self.weight = torch.zeros((B, Hkv, cap), dtype=torch.float32, device=dev)
        self.pos = torch.zeros((B, Hkv, cap), dtype=torch.int32, device=dev)
        self.lengths = torch.zeros(B, dtype=torch.int32, device=dev)
        self._lengths_next = torch.zeros_like(self.lengths)
        self.next_pos = torch.zeros_like(self.lengths)
        self._ws = workspace if workspace is not None else torch.empty(
            self.workspace_size(B, Hq, Hkv, cap, track_weight), dtype=torch.uint8, device=dev)
        self._bits = torch.arange(binding.tree_max_drafts(), dtype=torch.int64, device=dev)
        self._prompt: Optional[int] = None      # tokens of a prompt that nothing has followed yet
        self._arange = torch.arange(cap, dtype=torch.int32, device=dev)

    @staticmethod
    def workspace_size(B: int, Hq: int, Hkv: int, cap: int, track_weight: bool = True) -> int:
        """Bytes of workspace that steps of any number of tokens need. What a
        step needs depends on its number of tokens, and not only upwards: up
        to 32 rows (query heads of a kv head x tokens) its scores are kept,
        4 bytes per row and slot."""
        lib = binding.load()
        return max(lib.dhsa_cache_evict_workspace_size(B, Hkv, cap),
                   *(lib.dhsa_tree_attn_workspace_size(B, Hq, Hkv, T, cap, track_weight)
                     for T in range(1, lib.dhsa_tree_max_drafts() + 1)))

    def fill(self, K: torch.Tensor, V: torch.Tensor):
        """Start over from a prompt: K (rotated) and V [B,Hkv,L,128] take slots 0 .. L-1."""
        L = K.shape[2]
        if L > self.cap:
            raise ValueError(f"fill: {L} tokens, capacity {self.cap}")
        self.K[:, :, :L].copy_(K)
        self.V[:, :, :L].copy_(V)
        self.weight.zero_()
        self.pos[:, :, :L].copy_(self._arange[:L])
        self.lengths.fill_(L)
        self.next_pos.fill_(L)
        self._prompt = L

    def observe(self, Q: torch.Tensor):
        """Score the cached slots by the attention of the prompt's last tokens:
        Q (rotated) [B,Hq,w,128], w <= 64, the queries of the last w slots.
        Right after fill."""
        if not self.track_weight:
            raise ValueError("observe: the cache keeps no weights")
        if self._prompt is None or Q.shape[2] > self._prompt:
            raise ValueError("observe: comes right after fill, with at most the prompt's tokens")
        return binding.tree_attn(Q, self.K, self.V, self.lengths - Q.shape[2], softmax_scale=self.scale,
                                 weight=self.weight, workspace=self._ws)

    def extend(self, Q: torch.Tensor, K: torch.Tensor, V: torch.Tensor, depth: Optional[torch.Tensor] = None,
               n_new: Optional[torch.Tensor] = None) -> torch.Tensor:
        """Rotate Q [B,Hq,T,128] and K, and put K, V [B,Hkv,T,128] into the slots
        after the cached ones. depth (int32 [B,T]) is each token's distance
        from the next position (None: 0 .. T-1). Returns the rotated Q."""
        self._prompt = None
        at = {"start": self.next_pos} if depth is None else {"positions": self.next_pos[:, None] + depth}
        q, _, _ = binding.rotary_qkv(Q, K, self.inv_freq, V=V, n_new=n_new, slots=self.lengths,
                                     interleaved=self.interleaved, factor=self.rotary_factor, K_out=self.K,
                                     V_out=self.V, pos_out=self.pos, **at)
        return q

    def attend(self, Q: torch.Tensor, parents: Optional[torch.Tensor] = None,
               n_draft: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None) -> torch.Tensor:
        """Attention of the step's tokens (rotated Q) over the cache and their
        own ancestors; adds the slots' attention weights when they are tracked."""
        return binding.tree_attn(Q, self.K, self.V, self.lengths, parents=parents, n_draft=n_draft,
                                 softmax_scale=self.scale, weight=self.weight if self.track_weight else None,
                                 out=out, workspace=self._ws)

    def commit(self, n_draft: torch.Tensor, accept: Optional[torch.Tensor] = None, keep: Optional[int] = None):
        """End a step: of each sequence's n_draft (int32 [B]) new tokens those
        with their bit in accept (int64 [B]; None: all) stay, and of all slots
        the `keep` (None: all) that rank first by held, then weight, slot. Held are
        positions below `sinks`, the accepted tokens and the `recent`
        positions before them; where these are more than `keep`, the sinks and
        the last keep - sinks positions."""
        self._prompt = None
        added = n_draft
        if accept is not None:
            bit = (accept[:, None] >> self._bits) & (self._bits < n_draft[:, None])
            added = bit.sum(-1, dtype=torch.int32)
        # cache_evict lets the lower slot win among held ones, and the newest
        # tokens are in the highest: it must not be given more than `keep` of them
        held_from, recent = self.next_pos, self.recent
        if keep is not None and self.sinks + recent + self._bits.numel() > keep:
            room = min(max(keep - self.sinks, 0), 0x7fffffff)
            held_from = torch.maximum(self.next_pos - min(recent, 0x7fffffff), self.next_pos + added - room)
            recent = 0
        binding.cache_evict(self.K, self.V, self.weight, self.pos, self.lengths, self.cap if keep is None else keep,
                            next_pos=held_from, n_draft=n_draft, accept=accept, sinks=self.sinks,
                            recent=recent, lengths_out=self._lengths_next, workspace=self._ws)
        self.next_pos += added
        self.lengths.copy_(self._lengths_next)      # the same tensor every step, so that a step can be captured
