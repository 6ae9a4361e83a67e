"""Latent attention (absorbed decode and expanded prompt forms) and verification of drafted tokens, measured.

Three operators of one speculative step of a model whose keys and values come
from one shared latent vector a token:

* ``decode``: absorbed latent attention of 1 or more causal query tokens per
  request over a paged cache of [512 latent | 64 rotary] rows
  (``fd_decode_latent``);
* ``prompt``: the expanded form for ragged prompts, per-head keys of 128
  channels plus a rotary key of 64 channels that all heads share
  (``fd_prefill_latent``);
* ``verify``: acceptance of drafted tokens against the target's probabilities
  and the sample that ends the step (``fd_verify_draft``).
"""
import functools
import math
import random
import weakref

import torch

own = False

LATENT, ROPE = 512, 64          # channels of a cache row: latent, rotary key
NOPE, VDIM = 128, 128           # expanded per-head key (without rotary part) and value channels
SCALE = 1.0 / math.sqrt(NOPE + ROPE)


# ---------------------------------------------------------------------------
# cases


def listed():
    return [
        # one short chat request on few heads: launch latency is what counts
        dict(name="decode_one_short", op="decode", B=1, Tq=1, H=16, P=64, lo=500, hi=500, lens=1, empty=False),
        # one request at a long context, all heads on one GPU
        dict(name="decode_one_32k", op="decode", B=1, Tq=1, H=128, P=64, lo=32768, hi=32768, lens=2, empty=False),
        # a serving batch that checks 3 drafted tokens, ragged lengths, small pages, some slots of the batch empty
        dict(name="decode_mtp_ragged", op="decode", B=24, Tq=4, H=16, P=16, lo=33, hi=9001, lens=3, empty=True),
        # a full batch at long contexts, heads split over two GPUs
        dict(name="decode_batch_long", op="decode", B=64, Tq=1, H=64, P=64, lo=16384, hi=32768, lens=4, empty=False),
        # the same with all heads: the batch a data-parallel attention rank decodes
        dict(name="decode_batch_heads", op="decode", B=32, Tq=1, H=128, P=64, lo=4096, hi=16384, lens=5, empty=False),
        # a few short prompts of odd lengths, as they arrive at a server
        dict(name="prompt_short", op="prompt", B=3, H=16, qlo=37, qhi=190, prefix_lo=0, prefix_hi=0, lens=6),
        # a long prompt in chunks: new tokens behind a prefix that is in the cache already, ragged over the batch
        dict(name="prompt_chunk", op="prompt", B=4, H=16, qlo=300, qhi=1024, prefix_lo=1000, prefix_hi=11000, lens=7),
        # a batch of ordinary prompts with more heads
        dict(name="prompt_batch", op="prompt", B=4, H=32, qlo=900, qhi=4100, prefix_lo=0, prefix_hi=0, lens=8),
        # one long document
        dict(name="prompt_long", op="prompt", B=1, H=16, qlo=16384, qhi=16384, prefix_lo=0, prefix_hi=0, lens=9),
        # one request, one drafted token
        dict(name="verify_one", op="verify", B=1, K=1, V=32000, draft="probs", ragged=False),
        # a serving batch; the draft is a lookup that proposes tokens without probabilities, ragged counts, odd vocabulary
        dict(name="verify_lookup", op="verify", B=33, K=5, V=50021, draft="tokens", ragged=True),
        # the largest batch a server verifies at once
        dict(name="verify_batch", op="verify", B=256, K=3, V=131072, draft="probs", ragged=False),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["decode", "decode", "prompt", "prompt", "verify"])
    salt = rng.randrange(1 << 30)
    if op == "decode":
        B = _log_int(rng, 1, 64)
        H = rng.choice([4, 8, 16, 20, 32, 64, 128])
        Tq = rng.choice([1, 1, 2, 3, 4, 5]) if H <= 32 else 1
        hi = _log_int(rng, 1, min(32768, 64 * 64 * 20480 // (B * max(64, H * Tq))))
        return dict(op=op, B=B, Tq=Tq, H=H, P=rng.choice([8, 16, 32, 64, 128]), lo=max(1, hi // rng.choice([1, 2, 30])), hi=hi,
                    lens=salt, empty=B > 2 and rng.random() < 0.5)
    if op == "prompt":
        B, H = _log_int(rng, 1, 8), rng.choice([1, 3, 8, 16, 32])
        qhi = _log_int(rng, 1, 8192)
        pre = _log_int(rng, 1, 12000) if rng.random() < 0.5 else 0
        while B * H * qhi * (qhi + pre) > 16 * 16384 * 16384:
            qhi, pre = qhi // 2, pre // 2
        return dict(op=op, B=B, H=H, qlo=max(1, qhi // rng.choice([1, 3, 20])), qhi=qhi, prefix_lo=pre // 3, prefix_hi=pre, lens=salt)
    V = _log_int(rng, 1000, 131072)
    K = rng.randrange(1, 8)
    B = _log_int(rng, 1, max(1, (256 * 4 * 131072) // (V * (K + 1) * 2)) if V * K > 250000 else 256)
    return dict(op=op, B=B, K=K, V=V, draft=rng.choice(["probs", "probs", "tokens"]), ragged=rng.random() < 0.5)


def _spread(r, n, lo, hi):
    """n whole numbers spread over [lo, hi], both ends among them where n allows."""
    v = [r.randint(lo, hi) for _ in range(n)]
    v[0] = hi
    if n > 1:
        v[-1] = lo
    return v


def _decode_lens(case):
    r = random.Random(case["lens"])
    L = _spread(r, case["B"], case["lo"], case["hi"])
    if case["empty"]:
        L[len(L) // 2] = 0
        L[len(L) // 3] = 1
    return L


def _prompt_lens(case):
    r = random.Random(case["lens"])
    q = _spread(r, case["B"], case["qlo"], case["qhi"])
    return q, [a + b for a, b in zip(q, _spread(r, case["B"], case["prefix_lo"], case["prefix_hi"]))]


# ---------------------------------------------------------------------------
# inputs


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _offsets(lens):
    return torch.tensor([0] + lens, dtype=torch.int64).cumsum(0).to(torch.int32).cuda()


def prepare(case, seed):
    g = _gen(seed)
    randn = functools.partial(torch.randn, generator=g, device="cuda")
    if case["op"] == "decode":
        B, Tq, H, P = case["B"], case["Tq"], case["H"], case["P"]
        L = _decode_lens(case)
        pages = [-(-n // P) for n in L]
        W, N = max(1, max(pages)), sum(pages) + 3
        ids = torch.randperm(N, generator=g, device="cuda")[:sum(pages)].to(torch.int32)   # pages scattered over the pool
        table = torch.full((B, W), -1, dtype=torch.int32, device="cuda")
        table[torch.arange(W, device="cuda")[None] < torch.tensor(pages, device="cuda")[:, None]] = ids
        return dict(op="decode", Tq=Tq, H=H, P=P, B=B,
                    q=randn(B, Tq, H, LATENT + ROPE).to(torch.bfloat16),
                    cache=randn(N, P, LATENT + ROPE, dtype=torch.bfloat16),
                    table=table, lens=torch.tensor(L, dtype=torch.int32, device="cuda"),
                    out=torch.empty(B, Tq, H, LATENT, dtype=torch.bfloat16, device="cuda"),
                    lse=torch.empty(B, Tq, H, dtype=torch.float32, device="cuda"))
    if case["op"] == "prompt":
        H = case["H"]
        lq, lk = _prompt_lens(case)
        Sq, Sk = sum(lq), sum(lk)
        kv = randn(Sk, H, NOPE + VDIM, dtype=torch.bfloat16)      # one up-projection makes keys and values of a head
        return dict(op="prompt", max_q=max(lq), max_k=max(lk),
                    q=randn(Sq, H, NOPE + ROPE).to(torch.bfloat16), k_nope=kv[..., :NOPE], v=kv[..., NOPE:],
                    k_pe=randn(Sk, ROPE).to(torch.bfloat16), cu_q=_offsets(lq), cu_k=_offsets(lk),
                    out=torch.empty(Sq, H, VDIM, dtype=torch.bfloat16, device="cuda"),
                    lse=torch.empty(Sq, H, dtype=torch.float32, device="cuda"))
    B, K, V = case["B"], case["K"], case["V"]
    logits = randn(B, K + 1, V).mul_(2.5)
    target = torch.softmax(logits, -1)
    # the draft model's distribution is near the target's; its tokens are sampled from it
    noise = torch.randn(B, K, V, generator=g, device="cuda").mul_(0.6)
    draft = torch.softmax(logits[:, :K] + noise, -1)
    del noise, logits
    race = torch.rand(B, K, V, generator=g, device="cuda").clamp_(1e-9, 1 - 1e-7).log_().neg_()
    tokens = (draft / race).argmax(-1).to(torch.int32)
    del race
    counts = torch.randint(0, K + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
    return dict(op="verify", target=target, draft=draft if case["draft"] == "probs" else None, tokens=tokens,
                counts=counts if case["ragged"] else None,
                u=torch.rand(B, K + 1, generator=g, device="cuda"),
                out=torch.empty(B, K + 1, dtype=torch.int32, device="cuda"),
                emitted=torch.empty(B, dtype=torch.int32, device="cuda"))


# ---------------------------------------------------------------------------
# one pass


class _Plan:
    """A plan, destroyed with the last state that uses it."""

    def __init__(self, device, *geometry):
        import split_kv_paged_gqa_gb300 as fd
        self.handle = fd.fd_latent_plan_create(device, *geometry, SCALE)
        weakref.finalize(self, fd.fd_plan_destroy, self.handle).atexit = False


_plans = weakref.WeakValueDictionary()


def _latent_plan(s):
    """The plan a program keeps for one decode geometry on one device and stream
    (calls on two streams may overlap, and a plan is one workspace)."""
    if "plan" not in s:
        key = (torch.cuda.current_device(), torch.cuda.current_stream().cuda_stream, s["B"], s["Tq"], s["H"], s["P"])
        plan = _plans.get(key)
        if plan is None:
            plan = _plans[key] = _Plan(key[0], *key[2:])
        s["plan"] = plan
    return s["plan"].handle


def _run_own(s):
    import split_kv_paged_gqa_gb300 as fd
    if s["op"] == "decode":
        fd.fd_set_plan(_latent_plan(s))
        fd.fd_decode_latent(s["q"], s["cache"], s["table"], s["lens"], s["Tq"], s["out"], s["lse"])
        return s["out"], s["lse"]
    if s["op"] == "prompt":
        fd.fd_prefill_latent(s["q"], s["k_nope"], s["k_pe"], s["v"], s["cu_q"], s["cu_k"], s["max_q"], SCALE, s["out"], s["lse"])
        return s["out"], s["lse"]
    fd.fd_verify_draft(s["target"], s["draft"], s["tokens"], s["counts"], s["u"], s["out"], s["emitted"])
    return s["out"], s["emitted"]


def _softmax_rows(score, visible):
    """Softmax weights and log-sum-exp of the visible scores; a row that sees nothing has weights 0 and lse -inf."""
    score = score.masked_fill(~visible, -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(torch.isfinite(top), top, torch.zeros_like(top))
    e = score.sub_(top).exp_()
    total = e.sum(-1, keepdim=True)
    lse = (top + total.log()).squeeze(-1)
    return e.div_(torch.where(total > 0, total, torch.ones_like(total))), lse


def _plain_decode(s):
    B, Tq, H = s["B"], s["Tq"], s["H"]
    rows = s["cache"][s["table"].clamp(min=0).long()].flatten(1, 2).float()                       # [B, W P, 576]
    score = torch.matmul(s["q"].flatten(1, 2).float(), rows.transpose(1, 2)).mul_(SCALE).view(B, Tq, H, -1)
    limit = s["lens"][:, None] - (Tq - 1) + torch.arange(Tq, device="cuda")                       # keys that token t sees
    visible = torch.arange(rows.shape[1], device="cuda") < limit[:, :, None, None]
    p, lse = _softmax_rows(score, visible)
    out = torch.matmul(p.view(B, Tq * H, -1), rows[..., :LATENT]).view(B, Tq, H, LATENT)
    return out.to(torch.bfloat16), lse


def _plain_prompt(s):
    cq, ck = s["cu_q"].long(), s["cu_k"].long()
    lq, lk = cq.diff(), ck.diff()
    i = torch.arange(s["max_q"], device="cuda")
    j = torch.arange(s["max_k"], device="cuda")
    iq = (cq[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)          # padded batch: row of each (request, query)
    ik = (ck[:-1, None] + j).clamp(max=s["v"].shape[0] - 1)
    q = s["q"][iq].float().transpose(1, 2)                            # [B, H, maxq, 192]
    score = torch.matmul(q[..., :NOPE], s["k_nope"][ik].float().permute(0, 2, 3, 1))
    score += torch.matmul(q[..., NOPE:], s["k_pe"][ik].float().transpose(1, 2)[:, None])
    score *= SCALE
    limit = i + (lk - lq)[:, None] + 1                                # keys that query i sees: aligned to the end
    visible = (j < limit[:, :, None]) & (j < lk[:, None, None])
    p, lse = _softmax_rows(score, visible[:, None])
    del score
    out = torch.matmul(p, s["v"][ik].float().transpose(1, 2)).transpose(1, 2)   # [B, maxq, H, 128]
    here = i < lq[:, None]
    return out[here].to(torch.bfloat16), lse.transpose(1, 2)[here]


def _plain_verify(s):
    p, u = s["target"], s["u"]
    B, K1, V = p.shape
    K = K1 - 1
    count = s["counts"].long() if s["counts"] is not None else torch.full((B,), K, device="cuda")
    x = s["tokens"].long()
    at = torch.arange(K, device="cuda")
    px = p[:, :K].gather(2, x[..., None])[..., 0].double()
    qx = s["draft"].gather(2, x[..., None])[..., 0].double() if s["draft"] is not None else torch.ones_like(px)
    good = (u[:, :K].double() * qx < px) & (at < count[:, None])
    n = good.long().cumprod(1).sum(1)                                 # drafted tokens accepted
    b = torch.arange(B, device="cuda")
    refused = n < count
    row = p[b, n].double()
    m = n.clamp(max=K - 1)
    if s["draft"] is not None:
        less = (row - s["draft"][b, m].double()).clamp_(min=0)
    else:
        less = row.scatter(1, x[b, m][:, None], 0.0)                  # a draft without probabilities: all weight on its token
    less = torch.where(refused[:, None], less, row)
    weight = torch.where(less.sum(1, keepdim=True) > 0, less, row)
    cum = weight.cumsum(1)
    last = (cum <= u[:, K:].double() * cum[:, -1:]).sum(1).clamp(max=V - 1)   # the sample has a number of its own
    slot = torch.arange(K1, device="cuda")
    out = torch.where(slot < n[:, None], torch.nn.functional.pad(x, (0, 1)), -1)
    out = torch.where(slot == n[:, None], last[:, None], out)
    return out.to(torch.int32), (n + 1).to(torch.int32)


def run(state):
    if own:
        return _run_own(state)
    return {"decode": _plain_decode, "prompt": _plain_prompt, "verify": _plain_verify}[state["op"]](state)


# ---------------------------------------------------------------------------
# what a pass cannot do without


def work(case):
    if case["op"] == "decode":
        L, rows = _decode_lens(case), case["Tq"] * case["H"]
        row = 2 * (LATENT + ROPE)
        return {"bytes": sum(L) * row + case["B"] * rows * (row + 2 * LATENT + 4),
                "flops": 2 * rows * (2 * LATENT + ROPE) * sum(L)}
    if case["op"] == "prompt":
        lq, lk = _prompt_lens(case)
        H = case["H"]
        pairs = sum(a * (b - a) + a * (a + 1) // 2 for a, b in zip(lq, lk))
        return {"bytes": 2 * (sum(lq) * H * (NOPE + ROPE + VDIM + 2) + sum(lk) * (H * (NOPE + VDIM) + ROPE)),
                "flops": 2 * H * (NOPE + ROPE + VDIM) * pairs}
    # the row that is sampled from, once; a refusal with draft probabilities
    # reads the draft's row too (about half of the requests are refused somewhere)
    rows = 1.5 if case["draft"] == "probs" else 1.0
    return {"bytes": int(case["B"] * case["V"] * 4 * rows), "flops": 2 * case["B"] * case["V"]}


# ---------------------------------------------------------------------------
# the definition in 64 bits


def _exact_decode(s):
    B, Tq, H, P = s["B"], s["Tq"], s["H"], s["P"]
    out = torch.zeros(B, Tq, H, LATENT, dtype=torch.float64, device="cuda")
    lse = torch.full((B, Tq, H), -math.inf, dtype=torch.float64, device="cuda")
    for b, L in enumerate(s["lens"].tolist()):
        keys = s["cache"][s["table"][b, :-(-L // P)].long()].reshape(-1, LATENT + ROPE)[:L].double()
        for t in range(Tq):
            n = L - (Tq - 1) + t
            if n > 0:
                z = s["q"][b, t].double() @ keys[:n].T * SCALE
                lse[b, t] = torch.logsumexp(z, -1)
                out[b, t] = torch.softmax(z, -1) @ keys[:n, :LATENT]
    return out, lse


def _exact_prompt(s):
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device="cuda")
    cq, ck = s["cu_q"].tolist(), s["cu_k"].tolist()
    for b in range(len(cq) - 1):
        n, m = cq[b + 1] - cq[b], ck[b + 1] - ck[b]
        for h in range(s["q"].shape[1]):
            k = torch.cat([s["k_nope"][ck[b]:ck[b + 1], h], s["k_pe"][ck[b]:ck[b + 1]]], -1).double()
            v = s["v"][ck[b]:ck[b + 1], h].double()
            for i0 in range(0, n, 2048):
                i1 = min(n, i0 + 2048)
                most = max(0, min(m, i1 + m - n))
                if not most:
                    continue
                z = s["q"][cq[b] + i0:cq[b] + i1, h].double() @ k[:most].T * SCALE
                hidden = torch.arange(most, device="cuda") > torch.arange(i0, i1, device="cuda")[:, None] + (m - n)
                z[hidden] = -math.inf
                lse[cq[b] + i0:cq[b] + i1, h] = torch.logsumexp(z, -1)
                w = torch.exp(z - torch.logsumexp(z, -1, keepdim=True)).nan_to_num(0.0)
                out[cq[b] + i0:cq[b] + i1, h] = w @ v[:most]
    return out, lse


def _exact_verify(s):
    B, K1, V = s["target"].shape
    out, emitted = torch.full((B, K1), -1, dtype=torch.int32), torch.zeros(B, dtype=torch.int32)
    u, x = s["u"].double().tolist(), s["tokens"].tolist()
    count = s["counts"].tolist() if s["counts"] is not None else [K1 - 1] * B
    for b in range(B):
        n = 0
        while n < count[b]:
            q = 1.0 if s["draft"] is None else float(s["draft"][b, n, x[b][n]])
            if u[b][n] * q >= float(s["target"][b, n, x[b][n]]):
                break
            out[b, n] = x[b][n]
            n += 1
        w = s["target"][b, n].double()
        if n < count[b]:
            d = torch.zeros_like(w).index_fill(0, s["tokens"][b, n:n + 1].long(), math.inf) if s["draft"] is None else s["draft"][b, n].double()
            d = torch.relu(w - d)
            w = d if float(d.sum()) > 0 else w
        c = torch.cumsum(w, 0)
        out[b, n] = min(V - 1, int(torch.searchsorted(c, u[b][-1] * c[-1], right=True)))
        emitted[b] = n + 1
    return out.cuda(), emitted.cuda()


def exact(case, seed):
    s = prepare(case, seed)
    return {"decode": _exact_decode, "prompt": _exact_prompt, "verify": _exact_verify}[case["op"]](s)
