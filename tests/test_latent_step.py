"""The latent-attention operators together, as a speculative serving loop runs
them: prompts, then steps of metadata, attention of the drafted tokens and their
verification, each step one replay of a captured graph."""
import math

import numpy as np
import pytest
import torch

import split_kv_paged_gqa_gb300 as fd
from oracle.latent_ref import latent_decode_ref, latent_prefill_ref, verify_draft_ref

BF, F32, I32, I64 = torch.bfloat16, torch.float32, torch.int32, torch.int64
SCALE = 1.0 / math.sqrt(192)
H, P, K, V, POOL, SLOTS = 16, 16, 3, 499, 7, 40 * 16


def f64(t):
    return t.detach().double().cpu().numpy()


def within(out, lse, ref):
    o, s, tol, ltol = ref
    live = np.isfinite(s)
    assert np.array_equal(np.isneginf(f64(lse)), ~live)
    assert (np.abs(f64(out) - o) <= tol).all() and (np.abs(f64(lse)[live] - s[live]) <= ltol[live]).all()


class Engine:
    """One latent-attention layer over a token pool; row 3 of the batch is padding."""

    def __init__(self, prompts, seed):
        g = torch.Generator().manual_seed(seed)
        rand = lambda *n, s=1.0: (torch.randn(*n, generator=g) * s).to(BF).cuda()   # noqa: E731
        self.rows = rand(V, 576)                                  # a token's cache row
        self.queries = rand(V, H, 192)
        self.up_k, self.up_v = rand(H, 128, 512, s=512 ** -0.5), rand(H, 128, 512, s=512 ** -0.5)
        self.head = rand(H * 128, V, s=0.05)
        self.guess = torch.randint(V, (V,), generator=g).cuda()   # the lookup that drafts the next token
        B = len(prompts) + 1
        order = torch.randperm(POOL * SLOTS // P, generator=g)    # pages of the pool, in any order
        self.req_to_token = (order.view(POOL, -1, 1) * P + torch.arange(P)).reshape(POOL, SLOTS).to(I32).cuda()
        self.pool = torch.tensor([4, 0, 6, -1], dtype=I64).cuda()
        self.active = self.pool >= 0
        self.cache = torch.full((POOL * SLOTS // P, P, 576), math.nan, dtype=BF, device="cuda")
        z = lambda *n, dtype=I32: torch.zeros(*n, dtype=dtype, device="cuda")   # noqa: E731
        self.lens, self.keys, self.last = z(B), z(B), z(B, dtype=I64)
        self.tokens, self.uniforms = z(B, K + 1, dtype=I64), z(B, K + 1, dtype=F32)
        self.table, self.seqlens, self.cu_k, self.cu_q = z(B, SLOTS // P), z(B), z(B + 1), z(B + 1)
        self.q, self.attn, self.lse = z(B, K + 1, H, 576, dtype=BF), z(B, K + 1, H, 512, dtype=BF), z(B, K + 1, H, dtype=F32)
        self.probs, self.drafts = z(B, K + 1, V, dtype=F32), z(B, K)
        self.out_tokens, self.emitted, self.status = z(B, K + 1), z(B), z(1)
        self.plan = fd.fd_latent_plan_create(0, B, K + 1, H, P, SCALE)
        self.prompt(prompts)

    def prompt(self, prompts):
        """The prompts' cache rows, and their attention in the expanded form."""
        n = [len(p) for p in prompts]
        tok = torch.cat(prompts).cuda()
        rows = self.rows[tok]
        at = torch.cat([self.req_to_token[int(r), :k] for r, k in zip(self.pool, n)]).long()
        self.cache.view(-1, 576)[at] = rows
        cu = torch.tensor(np.concatenate([[0], np.cumsum(n)]), dtype=I32).cuda()
        k = torch.einsum("sc,hdc->shd", rows[:, :512], self.up_k)
        v = torch.einsum("sc,hdc->shd", rows[:, :512], self.up_v)
        a = dict(q=self.queries[tok], k_nope=k, k_pe=rows[:, 512:], v=v)
        out = torch.empty(sum(n), H, 128, dtype=BF, device="cuda")
        lse = torch.empty(sum(n), H, device="cuda")
        fd.fd_prefill_latent(**a, cu_seqlens_q=cu, cu_seqlens_k=cu, max_seqlen_q=max(n), softmax_scale=SCALE, out=out,
                             lse=lse, status=self.status)
        within(out, lse, latent_prefill_ref(*(f64(a[x]) for x in ("q", "k_nope", "k_pe", "v")), cu.cpu().numpy(),
                                            cu.cpu().numpy(), SCALE))
        ends = cu[1:].long() - 1
        self.lens[:-1] = torch.tensor(n, dtype=I32).cuda()
        self.last[:-1] = (out[ends].reshape(-1, H * 128) @ self.head).argmax(-1)

    def step(self):
        """K drafted tokens behind the last one: written to the cache, attended, verified."""
        t = self.last
        for i in range(K + 1):
            self.tokens[:, i] = t
            t = self.guess[t]
        self.drafts.copy_(self.tokens[:, 1:])
        self.keys.copy_((self.lens + K + 1) * self.active)
        pos = self.lens[:, None].long() + torch.arange(K + 1, device="cuda")
        slot = self.req_to_token[self.pool.clamp(min=0)[:, None], pos]
        rows = self.rows[self.tokens]
        live = slice(0, self.tokens.shape[0] - 1)                 # (the padding row owns no slots)
        self.cache.view(-1, 576).index_copy_(0, slot[live].reshape(-1).long(), rows[live].reshape(-1, 576))
        fd.fd_graph_metadata(self.req_to_token, self.pool, self.keys, P, "strided", None, K + 1, self.table, self.seqlens,
                             self.cu_k, self.cu_q, self.status)
        raw = self.queries[self.tokens]
        self.q[..., :512] = torch.einsum("bthd,hdc->bthc", raw[..., :128], self.up_k)
        self.q[..., 512:] = raw[..., 128:]
        fd.fd_decode_latent(self.q, self.cache, self.table, self.seqlens, K + 1, self.attn, self.lse)
        heads = torch.einsum("bthc,hdc->bthd", self.attn, self.up_v).flatten(2)
        torch.softmax((heads @ self.head).float(), -1, out=self.probs)
        fd.fd_verify_draft(self.probs, None, self.drafts, None, self.uniforms, self.out_tokens, self.emitted, self.status)
        self.lens += self.emitted * self.active
        self.last.copy_(self.out_tokens.gather(1, self.emitted[:, None].long() - 1)[:, 0])

    def state(self):
        return [x.clone() for x in (self.lens, self.last, self.out_tokens, self.emitted, self.attn, self.lse, self.probs)]


def prompts(seed):
    g = torch.Generator().manual_seed(seed)
    return [torch.randint(V, (n,), generator=g) for n in (77, 1, 300)]


@pytest.mark.gpu
def test_speculative_steps_captured_and_checked():
    draw = torch.Generator().manual_seed(8)
    u = torch.rand(13, 4, K + 1, generator=draw)
    u[..., :K] *= 2.0 / V       # a drafted token has a weight of about 1 / V: some are accepted
    u = u.cuda()
    eager, e = [], Engine(prompts(7), 7)
    fd.fd_set_plan(e.plan)
    try:
        for x in u:
            e.uniforms.copy_(x)
            e.step()
            eager.append(e.state())
    finally:
        fd.fd_set_plan(None)
    assert fd.fd_read_device_status(e.plan) == 0 and int(e.status) == 0
    fd.fd_plan_destroy(e.plan)

    e = Engine(prompts(7), 7)
    start = [x.clone() for x in (e.lens, e.last)]
    graph = torch.cuda.CUDAGraph()
    fd.fd_set_plan(e.plan)
    try:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            e.step()
        torch.cuda.current_stream().wait_stream(side)
        with torch.cuda.graph(graph):
            e.step()
    finally:
        fd.fd_set_plan(None)
    e.lens.copy_(start[0])
    e.last.copy_(start[1])
    emitted = set()
    for x, want in zip(u, eager):
        before = e.lens.clone()
        e.uniforms.copy_(x)
        graph.replay()
        for got, w in zip(e.state(), want):
            assert torch.equal(got, w)
        # each operator on what it was given in this step
        L = e.keys.cpu().tolist()
        assert e.seqlens.tolist() == L and L[3] == 0
        within(e.attn, e.lse, latent_decode_ref(f64(e.q), f64(e.cache), e.table.cpu().numpy(), L, SCALE))
        tok, n = verify_draft_ref(e.probs.cpu().numpy(), None, e.drafts.cpu().numpy(), None, x.cpu().numpy())
        assert np.array_equal(e.out_tokens.cpu().numpy(), tok) and np.array_equal(e.emitted.cpu().numpy(), n)
        assert torch.equal(e.lens[:3], before[:3] + e.emitted[:3]) and int(e.lens[3]) == 0
        emitted.update(n[:3].tolist())
    assert len(emitted) > 1
    assert fd.fd_read_device_status(e.plan) == 0 and int(e.status) == 0
    fd.fd_plan_destroy(e.plan)
