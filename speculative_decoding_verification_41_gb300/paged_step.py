"""A speculative serving step on a paged key-value cache, all on the device: the
drafter proposes (dspark_draft_markov), the scheduler gives each request a verify
length (dspark_schedule), pages are reserved for the tokens to verify
(dspark_pages_reserve), the target runs over them (dspark_kv_append,
dspark_paged_attention), dspark_verify judges the drafts and dspark_pages_release
takes back the pages that only rejected tokens used.

No call waits for the host and every shape is fixed by the batch, so a step can
be captured in a CUDA graph and replayed. `ToyTarget` stands for the target: one
attention layer with random weights.

    python -m speculative_decoding_verification_41_gb300.paged_step
"""
from __future__ import annotations

import torch

from . import binding, paged


class PagedCache:
    """Keys and values of B requests in pages, and the books about them. The lengths
    and the free pages are updated in place."""

    def __init__(self, B: int, num_pages: int, page_size: int, max_pages: int, Hkv: int, D: int,
                 max_new: int, dtype=torch.bfloat16, device="cuda"):
        dev = torch.device(device)
        i32 = dict(dtype=torch.int32, device=dev)
        self.B, self.page_size, self.max_new = B, page_size, max_new
        self.k = torch.zeros(num_pages, page_size, Hkv, D, dtype=dtype, device=dev)
        self.v = torch.zeros_like(self.k)
        self.block_table = torch.zeros(B, max_pages, **i32)
        self.free_pages = torch.arange(num_pages, **i32)
        self.free_count = torch.full((1,), num_pages, **i32)
        self.context_len = torch.zeros(B, **i32)
        self.rows = paged.ReserveBuffers(B, B * max_new, dev)
        self.rows.free_count = self.free_count
        self._kept = paged.ReleaseBuffers(B, dev)
        self._kept.context_len, self._kept.free_count = self.context_len, self.free_count
        self._append_status = torch.zeros(1, **i32)
        self._attention = None

    def reserve(self, new_len: torch.Tensor, extra: int = 1) -> dict:
        """Pages for new_len[r] + extra tokens; the rows of the step (dspark_pages_reserve)."""
        return paged.dspark_pages_reserve(
            self.context_len, new_len, self.block_table, self.free_pages, self.free_count,
            page_size=self.page_size, max_tokens=self.B * self.max_new, extra=extra,
            buffers=self.rows)

    def append(self, k: torch.Tensor, v: torch.Tensor) -> None:
        paged.dspark_kv_append(k, v, self.rows.slot_map, self.k, self.v,
                               device_status=self._append_status)

    def attend(self, q: torch.Tensor) -> torch.Tensor:
        """Attention of the step's rows. The result is a buffer that the next call for rows of this
        shape overwrites (another layer's): copy what has to outlive it."""
        n, Hq, D = q.shape
        if self._attention is None or self._attention.out.shape != q.shape:
            self._attention = paged.AttentionBuffers(n, Hq, self.k.shape[2], D, self.max_new,
                                                     q.dtype, q.device)
        return paged.dspark_paged_attention(
            q, self.k, self.v, self.block_table, self.rows.context_len, self.rows.row_off,
            scale=D ** -0.5, max_new=self.max_new, buffers=self._attention)["out"]

    def release(self, kept_len: torch.Tensor, extra: int = 1) -> None:
        """Keep kept_len[r] + extra of the reserved tokens (-1: the request is finished)."""
        paged.dspark_pages_release(self.context_len, self.rows.context_len, kept_len,
                                   self.block_table, self.free_pages, self.free_count,
                                   page_size=self.page_size, extra=extra, buffers=self._kept)

    def statuses(self) -> list:
        """The cache's calls' device status words (synchronises): reserve, append, release and, once
        it has run, the attention. The verification's is in speculative_step's result."""
        words = [self.rows.device_status, self._append_status, self._kept.device_status]
        if self._attention is not None:
            words.append(self._attention.device_status)
        return [int(w.item()) for w in words]


class ToyTarget:
    """One attention layer over token embeddings, random weights: keys and values of a token
    depend on the token alone, logits on what its query finds in the cache."""

    def __init__(self, V: int, Hq: int, Hkv: int, D: int, dtype=torch.bfloat16, seed: int = 0,
                 device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        make = lambda *s: torch.randn(*s, generator=g, device=device)
        width = 64
        self.embed = make(V, width).to(dtype)
        self.wq = (make(width, Hq * D) / 8).to(dtype)
        self.wk = (make(width, Hkv * D) / 8).to(dtype)
        self.wv = (make(width, Hkv * D) / 8).to(dtype)
        self.head = (make(Hq * D, V) / 8).to(dtype)
        self.Hq, self.Hkv, self.D = Hq, Hkv, D

    def qkv(self, tokens: torch.Tensor):
        x = self.embed[tokens]
        n = tokens.numel()
        return ((x @ self.wq).view(n, self.Hq, self.D), (x @ self.wk).view(n, self.Hkv, self.D),
                (x @ self.wv).view(n, self.Hkv, self.D))

    def logits(self, attended: torch.Tensor) -> torch.Tensor:
        return attended.flatten(1) @ self.head


def speculative_step(cache: PagedCache, target: ToyTarget, anchors: torch.Tensor,
                     draft_tokens: torch.Tensor, draft_logits: torch.Tensor,
                     verify_len: torch.Tensor, uniforms: torch.Tensor, temperature: float) -> dict:
    """One target pass over each request's anchor and its first verify_len[r] drafts, the
    verification, and the roll back. draft_tokens [B, gamma], draft_logits [B, gamma, V].

    Returns dspark_verify's outputs, and
      served [B] bool: which requests got rows. The others (out of pages or of room in their
        block table, reserve_status says why) are as they were before the step: their anchor is
        still to be run, their accepted_len is 0, their emitted_tokens are -1, and device_status is
        DSPARK_ERR_BAD_DATA because of them;
      next_anchors [B]: emitted_tokens at accepted_len, the same anchor where not served;
      reserve_status [1]: dspark_pages_reserve's status."""
    B, gamma = draft_tokens.shape
    dev = anchors.device
    rows = cache.reserve(verify_len)
    row_off = rows["row_off"]
    served = row_off[1:] > row_off[:-1]
    # the token of every row: position 0 of a request is its anchor
    i = torch.arange(B * cache.max_new, device=dev)
    r = torch.searchsorted(row_off[1:], i, right=True).clamp(max=B - 1)
    j = (i - row_off[r]).clamp(0, gamma)
    tokens = torch.cat([anchors[:, None], draft_tokens], 1)[r, j].long()
    q, k, v = target.qkv(tokens)
    cache.append(k, v)
    logits = target.logits(cache.attend(q))
    out = binding.dspark_verify(
        logits, draft_logits.reshape(B * gamma, -1), draft_tokens, verify_len, uniforms,
        temperature, row_off, torch.arange(B + 1, device=dev, dtype=torch.int64) * gamma)
    cache.release(out["accepted_len"])
    last = out["emitted_tokens"].gather(1, out["accepted_len"].long()[:, None])[:, 0]
    return {**out, "served": served, "next_anchors": torch.where(served, last, anchors),
            "reserve_status": rows["device_status"].clone()}


def demo(B: int = 32, gamma: int = 4, V: int = 4096, steps: int = 8, device="cuda") -> dict:
    """A few steps with the Markov drafter, the scheduler and the toy target."""
    from . import workloads
    dev = torch.device(device)
    g = torch.Generator(device=dev).manual_seed(1)
    target = ToyTarget(V, 16, 4, 64, device=dev)
    cache = PagedCache(B, num_pages=B * 8, page_size=16, max_pages=16, Hkv=4, D=64,
                       max_new=gamma + 1, device=dev)
    d = workloads.make_markov_draft(B, gamma, V, 64, temperature=1.0, seed=2, device=dev)
    profile = torch.from_numpy(
        workloads.step_time_profile(B * (gamma + 1) + 1, base_ms=1.0, slope_ms=0.002)).to(dev)
    anchors, emitted = d.anchors, 0
    for _ in range(steps):
        u = torch.rand(B, gamma, generator=g, device=dev)
        draft = binding.dspark_draft_markov(d.base_logits, d.w1, d.w2t, anchors, u, 1.0)
        conf = 0.5 + 0.5 * torch.rand(B, gamma, generator=g, device=dev)
        ell = binding.dspark_schedule(conf, profile)["verify_len"]
        out = speculative_step(cache, target, anchors, draft["draft_tokens"],
                               draft["draft_logits"], ell,
                               torch.rand(B, gamma + 1, generator=g, device=dev), 1.0)
        anchors = out["next_anchors"]
        emitted += int((out["accepted_len"].long() + out["served"]).sum().item())
    held = int(((cache.context_len + 15) // 16).sum().item())
    return {"tokens": emitted, "cached": int(cache.context_len.sum().item()),
            "pages_held": held, "pages_free": int(cache.free_count.item()),
            "statuses": cache.statuses()}


if __name__ == "__main__":
    print(demo())
