"""A decode step over selected pages with drafted tokens, as a serving loop runs it: slots, cache
writes, page selection, attention, verification and log probabilities, eagerly and as replays
of one captured graph, each operator checked on what it was given."""
import numpy as np
import pytest
import torch

import split_kv_paged_gqa_gb300 as fd
from oracle.latent_ref import verify_draft_ref
from oracle.step_ref import append_slots_ref, select_ref
from tests.test_append import cache_values, make_caches
from tests.test_logprobs import compare as compare_logprobs
from tests.test_sparse import compare as compare_sparse

BF, F32, I32, I64 = torch.bfloat16, torch.float32, torch.int32, torch.int64
B, K, HQ, HKV, D, P, W, N, S, V = 4, 2, 8, 2, 64, 8, 40, 90, 6, 203
T = B * (K + 1) + 5                       # rows of the buffers: more than a step fills


class Engine:
    def __init__(self, kind, seed):
        g = torch.Generator().manual_seed(seed)
        rand = lambda *n, s=1.0: (torch.randn(*n, generator=g) * s).to(BF).cuda()   # noqa: E731
        z = lambda *n, dtype=I32: torch.zeros(*n, dtype=dtype, device="cuda")       # noqa: E731
        self.kind = kind
        self.rows, self.queries, self.head = rand(V, 2, HKV, D), rand(V, HQ, D), rand(HQ * D, V, s=0.06)
        self.guess = torch.randint(V, (V,), generator=g).cuda()
        self.k, self.v, self.scales = make_caches(kind, N, P, HKV, D, g)
        if kind == "bf16":
            self.k.fill_(float("nan")), self.v.fill_(float("nan"))
        else:
            self.scales.fill_(float("nan"))
        self.bounds = z(N, HKV, 2, D, dtype=BF)
        self.active = torch.tensor([1, 1, 0, 1], dtype=I32).cuda()          # request 2 is a padding row
        self.lens, self.new, self.new_lens, self.cu, self.taken = z(B), z(B), z(B), z(B + 1), z(1)
        self.table = torch.full((B, W), -1, dtype=I32).cuda()
        self.free, self.num_free = torch.arange(N, dtype=I32).cuda(), torch.tensor([N], dtype=I32).cuda()
        self.slots, self.pos = z(T, dtype=I64), z(T)
        self.tokens, self.last, self.uniforms = z(B, K + 1, dtype=I64), z(B, dtype=I64), z(B, K + 1, dtype=F32)
        self.q, self.selected = z(B, K + 1, HQ, D, dtype=BF), z(B, K + 1, HKV, S)
        self.attn, self.lse = z(B, K + 1, HQ, D, dtype=BF), z(B, K + 1, HQ, dtype=F32)
        self.logits, self.probs = z(B * (K + 1), V, dtype=F32), z(B, K + 1, V, dtype=F32)
        self.out, self.emitted, self.drafts = z(B, K + 1), z(B), z(B, K)
        self.lp, self.rank, self.ent = z(B * (K + 1), dtype=F32), z(B * (K + 1)), z(B * (K + 1), dtype=F32)
        self.ids, self.top = z(B * (K + 1), 4), z(B * (K + 1), 4, dtype=F32)
        self.status = z(1)
        self.prompt([[3, 5, 9] * 37, [7], [], list(range(V)) + [1] * 20])

    def prompt(self, prompts):
        """Keys and values of the prompts (their attention is not this test's)."""
        tok = torch.tensor(sum(prompts, []), device="cuda")
        self.new.copy_(torch.tensor([len(p) for p in prompts], dtype=I32))
        slots = torch.zeros(tok.numel(), dtype=I64, device="cuda")
        fd.fd_append_slots(self.lens, self.new, self.free, self.num_free, P, self.table, slots, None, self.new_lens, self.cu,
                           self.taken, self.status)
        kv = self.rows[tok]
        fd.fd_cache_append(kv[:, 0], kv[:, 1], slots, self.k, self.v, self.scales, self.bounds, self.status)
        self.lens.copy_(self.new_lens)
        self.last.copy_(torch.tensor([p[-1] if p else 0 for p in prompts]))
        self.release()

    def release(self):
        """The free pages: those that no request holds (of refused tokens too)."""
        held = torch.arange(W, device="cuda") < ((self.lens + P - 1) // P)[:, None]
        used = torch.zeros(N + 1, dtype=I32, device="cuda").index_fill_(0, torch.where(held, self.table, N).flatten().long(), 1)[:N]
        self.free.copy_(used.argsort(stable=True))
        self.num_free.copy_(N - used.sum())

    def step(self):
        t = self.last
        for i in range(K + 1):
            self.tokens[:, i] = t
            t = self.guess[t]
        self.drafts.copy_(self.tokens[:, 1:])
        self.new.copy_(self.active * (K + 1))
        fd.fd_append_slots(self.lens, self.new, self.free, self.num_free, P, self.table, self.slots, self.pos, self.new_lens,
                           self.cu, self.taken, self.status)
        # the rows of the active requests, one behind the other, as a packed batch has them
        row = torch.arange(T, device="cuda")
        req = torch.searchsorted(self.cu[1:].contiguous(), row, right=True, out_int32=True).clamp(max=B - 1).long()
        kv = self.rows[self.tokens[req, (row - self.cu[req]).clamp(0, K)]]
        fd.fd_cache_append(kv[:, 0], kv[:, 1], self.slots, self.k, self.v, self.scales, self.bounds, self.status)
        self.q.copy_(self.queries[self.tokens])
        fd.fd_select_pages(self.q, self.bounds, self.table, self.new_lens, K + 1, P, 1, 2, self.selected, self.status)
        fd.fd_decode_sparse(self.q, self.k, self.v, self.scales, self.table, self.new_lens, self.selected, K + 1, 0.0, self.attn,
                            self.lse, self.status)
        self.logits.copy_(self.attn.view(B * (K + 1), HQ * D) @ self.head)
        torch.softmax(self.logits.view(B, K + 1, V), -1, out=self.probs)
        fd.fd_verify_draft(self.probs, None, self.drafts, None, self.uniforms, self.out, self.emitted, self.status)
        fd.fd_token_logprobs(self.logits, self.out.view(-1), self.lp, self.rank, self.ent, self.ids, self.top, self.status)
        self.before = self.lens.clone()
        self.lens += self.emitted * self.active
        self.last.copy_(self.out.gather(1, self.emitted[:, None].long() - 1)[:, 0])
        self.release()

    def state(self):
        names = ("lens", "table", "slots", "pos", "bounds", "selected", "attn", "lse", "out", "emitted", "lp", "rank", "ent", "ids",
                 "top", "free", "num_free")
        return {n: getattr(self, n).clone() for n in names}


def check(e, given):
    """The step's operators on what they were given: lengths, table, free pages before it."""
    n = lambda t: t.cpu().numpy()   # noqa: E731
    f = lambda t: t.double().cpu().numpy()   # noqa: E731
    table, slots, pos, lens, cu, taken, st = append_slots_ref(n(given["lens"]), n(e.new), n(given["free"]), int(given["num_free"]), P,
                                                              n(given["table"]), T)
    assert st == 0 and np.array_equal(n(e.table), table) and np.array_equal(n(e.slots), slots) and np.array_equal(n(e.pos), pos)
    assert np.array_equal(n(e.new_lens), lens) and np.array_equal(n(e.cu), cu) and int(e.taken) == taken
    values = f(cache_values(e.k, None if e.scales is None else e.scales[0], e.kind))
    for b in range(B):                      # the bounds of every page that holds keys contain them, and touch them
        for j in range(-(-int(lens[b]) // P)):
            keys = values[table[b, j], :min(P, int(lens[b]) - j * P)]
            lo, hi = f(e.bounds[table[b, j], :, 0]), f(e.bounds[table[b, j], :, 1])
            assert (lo <= keys.min(0)).all() and (hi >= keys.max(0)).all()
            assert (np.abs(lo - keys.min(0)) <= 2.0 ** -7 * np.abs(lo)).all() and (np.abs(hi - keys.max(0)) <= 2.0 ** -7 * np.abs(hi)).all()
    assert np.array_equal(n(e.selected), select_ref(f(e.q), f(e.bounds), table, lens, P, S, 1, 2))
    a = dict(q=e.q, k_cache=e.k, v_cache=e.v, kv_scales=e.scales, page_table=e.table, cache_seqlens=e.new_lens, selected=e.selected,
             softmax_scale=0.0)
    compare_sparse(a, e.attn, e.lse, e.kind)
    tok, m = verify_draft_ref(n(e.probs), None, n(e.drafts), None, n(e.uniforms))
    assert np.array_equal(n(e.out), tok) and np.array_equal(n(e.emitted), m)
    compare_logprobs(dict(logprobs=e.lp, ranks=e.rank, entropy=e.ent, top_ids=e.ids, top_logprobs=e.top), e.logits, e.out.view(-1), 4)
    assert int(e.status) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "int8", "int4"])
def test_steps_captured_and_checked(kind):
    u = torch.rand(8, B, K + 1, generator=torch.Generator().manual_seed(3))
    u[..., :K] *= 2.0 / V                   # a drafted token has a weight of about 1 / V: some are accepted
    u = u.cuda()
    eager, e = [], Engine(kind, 21)
    for x in u:
        e.uniforms.copy_(x)
        given = e.state()
        e.step()
        check(e, given)
        eager.append(e.state())
    assert len(set(torch.stack([s["emitted"] for s in eager]).flatten().tolist())) > 1
    assert int(e.lens[2]) == 0 and (e.lens[[0, 1, 3]] > torch.tensor([111, 1, 223]).cuda()).all()

    e = Engine(kind, 21)
    first = e.state()
    last, cache = e.last.clone(), [None if x is None else x.clone() for x in (e.k, e.v, e.scales)]
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        e.step()
    torch.cuda.current_stream().wait_stream(side)
    with torch.cuda.graph(graph):
        e.step()
    for name, x in first.items():
        getattr(e, name).copy_(x)
    e.last.copy_(last)
    for x, c in zip((e.k, e.v, e.scales), cache):
        if x is not None:
            x.copy_(c)
    for x, want in zip(u, eager):
        e.uniforms.copy_(x)
        graph.replay()
        for name, w in want.items():
            assert torch.equal(getattr(e, name), w), name
    assert int(e.status) == 0
