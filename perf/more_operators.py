"""A decode step at long contexts over the pages that matter, measured.

Five operators, in the order in which a serving loop uses them:

* ``slots``: pages and cache slots of a step's new tokens, from the requests'
  lengths and a list of free pages (``fd_append_slots``);
* ``append``: the new tokens' keys and values into the paged cache (bf16, or
  quantised to the 8- and 4-bit caches), and the bounds of the keys of every
  page that changed (``fd_cache_append``);
* ``select``: for each query token and KV head, the pages whose bounds allow
  the largest scores (``fd_select_pages``);
* ``sparse``: attention over the selected pages (``fd_decode_sparse``);
* ``logprobs``: log probability and rank of the emitted tokens, entropy and the
  most probable alternatives (``fd_token_logprobs``).
"""
import functools
import math
import random

import torch

own = False

BF, F32, F64, I32, I64 = torch.bfloat16, torch.float32, torch.float64, torch.int32, torch.int64


# ---------------------------------------------------------------------------
# cases


def listed():
    return [
        # one decode step of a full batch: a token or none for each request
        dict(name="slots_step", op="slots", B=64, P=16, new_lo=0, new_hi=1, len_hi=32768, spare=1.5, pad=0, wide=False),
        # chunks of prompts of many requests at once, ragged; the buffers of a captured graph are longer than the rows
        dict(name="slots_prompts", op="slots", B=500, P=16, new_lo=1, new_hi=1023, len_hi=16384, spare=1.1, pad=777, wide=True),
        # one decode step of a full batch, bf16 cache
        dict(name="append_step", op="append", B=64, new_lo=1, new_hi=1, len_hi=16000, Hkv=8, D=128, P=64, kv="bf16", bounds=True, pad=0),
        # drafted tokens of a multi-token step into a 4-bit cache with small pages
        dict(name="append_mtp_int4", op="append", B=64, new_lo=4, new_hi=4, len_hi=4096, Hkv=8, D=128, P=16, kv="int4", bounds=True, pad=0),
        # prompts of odd lengths behind what the cache holds already
        dict(name="append_prompts", op="append", B=16, new_lo=33, new_hi=4101, len_hi=5000, Hkv=8, D=128, P=16, kv="bf16", bounds=True, pad=33),
        # one request at a long context
        dict(name="select_one_32k", op="select", B=1, Tq=1, Hq=64, Hkv=8, D=128, P=16, lo=32768, hi=32768, keep=128, first=1, last=4, lens=1),
        # a full batch at long contexts
        dict(name="select_batch_long", op="select", B=64, Tq=1, Hq=64, Hkv=8, D=128, P=64, lo=16384, hi=65536, keep=32, first=1, last=2, lens=2),
        # one request, a sixteenth of its 32768 keys
        dict(name="sparse_one", op="sparse", B=1, Tq=1, Hq=64, Hkv=8, D=128, P=16, kv="bf16", lo=32768, hi=32768, keep=128, lens=3, empty=False),
        # a serving batch with drafted tokens, 8-bit cache, ragged lengths, some slots of the batch empty
        dict(name="sparse_mtp_int8", op="sparse", B=24, Tq=4, Hq=32, Hkv=8, D=128, P=16, kv="int8", lo=33, hi=9001, keep=67, lens=4, empty=True),
        # a full batch at long contexts
        dict(name="sparse_batch_long", op="sparse", B=64, Tq=1, Hq=64, Hkv=8, D=128, P=64, kv="bf16", lo=8192, hi=32768, keep=64, lens=5, empty=False),
        # the tokens of one decode step
        dict(name="logprobs_step", op="logprobs", R=64, V=131072, K=20, dtype="fp32", skip=False),
        # the tokens of prompts, an odd vocabulary
        dict(name="logprobs_prompts", op="logprobs", R=3001, V=50021, K=5, dtype="bf16", skip=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["slots", "append", "append", "select", "select", "sparse", "sparse", "sparse", "logprobs", "logprobs"])
    if op == "slots":
        B = _log_int(rng, 1, 2000)
        hi = _log_int(rng, 1, max(1, min(4096, 250000 // B)))
        return dict(op=op, B=B, P=rng.choice([8, 16, 32, 64, 128]), new_lo=rng.choice([0, 1, hi]), new_hi=hi,
                    len_hi=_log_int(rng, 1, 32768), spare=rng.choice([0.7, 1.0, 1.5]), pad=rng.choice([0, 1, 300]),
                    wide=rng.random() < 0.5)
    if op == "append":
        Hkv, D = rng.choice([1, 2, 4, 8]), rng.choice([64, 128])
        B = _log_int(rng, 1, 256)
        hi = _log_int(rng, 1, max(1, min(8192, 16 * 2000 // B)))
        return dict(op=op, B=B, new_lo=rng.choice([0, 1, hi]), new_hi=hi, len_hi=_log_int(rng, 1, 5000 if B > 64 else 16000),
                    Hkv=Hkv, D=D, P=rng.choice([8, 16, 32, 64, 128, 256]), kv=rng.choice(["bf16", "int8", "int4"]),
                    bounds=rng.random() < 0.75, pad=rng.choice([0, 1, 33]))
    if op in ("select", "sparse"):
        Hkv = rng.choice([1, 2, 4, 8])
        Hq = Hkv * rng.choice([1, 2, 4, 5, 8, 16])
        Tq, D, P = rng.choice([1, 1, 2, 4]), rng.choice([64, 128]), rng.choice([8, 16, 32, 64, 128])
        B = _log_int(rng, 1, 64 // Tq)
        hi = _log_int(rng, 1, 32768)
        lo = max(1, hi // rng.choice([1, 2, 30]))
        first, last = rng.choice([0, 1, 2]), rng.choice([1, 2, 4])
        if op == "select":
            pages = max(first + last + 2, min(_pages(hi, P), 512))      # (no more than the listed batch has; there is a choice)
            hi = min(pages * P, max(hi, (pages - 1) * P + 1))
            keep = first + last + _log_int(rng, 1, min(128, pages - first - last - 1))
            return dict(op=op, B=B, Tq=Tq, Hq=Hq, Hkv=Hkv, D=D, P=P, lo=min(lo, hi), hi=hi, keep=keep, first=first, last=last,
                        lens=rng.randrange(1 << 30))
        keep = _log_int(rng, 1, max(1, 3000 // P))
        return dict(op=op, B=B, Tq=Tq, Hq=Hq, Hkv=Hkv, D=D, P=P, kv=rng.choice(["bf16", "bf16", "int8", "int4"]), lo=lo, hi=hi,
                    keep=keep, lens=rng.randrange(1 << 30), empty=B > 2 and rng.random() < 0.5)
    V = _log_int(rng, 1000, 131072)
    return dict(op=op, R=_log_int(rng, 1, max(1, 130000000 // V)) if rng.random() < 0.3 else _log_int(rng, 1, 100), V=V,
                K=rng.choice([0, 1, 5, 8, 20, 32]), dtype=rng.choice(["bf16", "fp32"]), skip=rng.random() < 0.5)


def _spread(r, n, lo, hi):
    """n whole numbers spread over [lo, hi], both ends among them where n allows."""
    v = [r.randint(lo, hi) for _ in range(n)]
    v[0] = hi
    if n > 1:
        v[-1] = lo
    return v


def _batch_lens(case):
    r = random.Random(case["lens"])
    L = _spread(r, case["B"], case["lo"], case["hi"])
    if case.get("empty"):
        L[len(L) // 2] = 0
        L[len(L) // 3] = 1
    return L


def _growth(case):
    """Lengths before the step, and new tokens, of each request."""
    r = random.Random(case["B"] * 1000003 + case["new_hi"] * 101 + case["len_hi"])
    old = [r.randint(0, case["len_hi"]) for _ in range(case["B"])]
    old[0] = case["len_hi"]
    return old, _spread(r, case["B"], case["new_lo"], case["new_hi"])


def _pages(n, P):
    return -(-n // P)


# ---------------------------------------------------------------------------
# inputs


def _ints(values, dtype=I32):
    return torch.tensor(values, dtype=dtype, device="cuda")


def _table(pages, total, g):
    """Page tables over a pool of scattered pages: -1 behind a request's last page."""
    W = max(1, max(pages))
    ids = torch.randperm(total, generator=g, device="cuda")[:sum(pages)].to(I32)
    table = torch.full((len(pages), W), -1, dtype=I32, device="cuda")
    table[torch.arange(W, device="cuda")[None] < _ints(pages)[:, None]] = ids
    return table


def _caches(kv, N, P, Hkv, D, randn):
    """Key and value caches of N pages and their scales (head-major in memory), with values in them."""
    if kv == "bf16":
        return randn(N, P, Hkv, D, dtype=BF), randn(N, P, Hkv, D, dtype=BF), None
    n_g = 1 if kv == "int8" else D // 32
    scales = (randn(2, N, Hkv, P, n_g).abs_() + 2.0).mul_(0.009 if kv == "int8" else 0.14).permute(0, 1, 3, 2, 4)

    def codes():
        if kv == "int8":
            return randn(N, P, Hkv, D, dtype=BF).mul_(40).clamp_(-127, 127).to(torch.int8)
        c = randn(N, P, Hkv, D, dtype=BF).mul_(2.4).clamp_(-7, 7).to(torch.int8)
        return (c[..., ::2] & 15 | c[..., 1::2] << 4).view(torch.uint8)

    return codes(), codes(), scales


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    randn = functools.partial(torch.randn, generator=g, device="cuda")
    return {"slots": _prepare_slots, "append": _prepare_append, "select": _prepare_select, "sparse": _prepare_sparse,
            "logprobs": _prepare_logprobs}[case["op"]](case, g, randn)


def _prepare_slots(case, g, randn):
    old, new = _growth(case)
    B, P, T = case["B"], case["P"], sum(new) + case["pad"]
    held = [_pages(a, P) for a in old]
    more = sum(_pages(a + b, P) for a, b in zip(old, new)) - sum(held)
    n_free = int(more * case["spare"]) + (1 if case["spare"] >= 1 else 0)
    total = sum(held) + max(1, n_free)
    ids = torch.randperm(total + 5000, generator=g, device="cuda")[:total].to(I32)     # (others hold the rest of the pool)
    W = max(_pages(a + b, P) for a, b in zip(old, new)) + 3
    table = torch.full((B, W), -1, dtype=I32, device="cuda")
    table[torch.arange(W, device="cuda")[None] < _ints(held)[:, None]] = ids[:sum(held)]
    empty = functools.partial(torch.empty, device="cuda", dtype=I32)
    return dict(op="slots", P=P, table=table, lens=_ints(old), new=_ints(new), free=ids[sum(held):].clone(), n_free=_ints([n_free]),
                slots=empty(T, dtype=I64 if case["wide"] else I32), positions=empty(T), new_lens=empty(B),
                cu=empty(B + 1), taken=empty(1))


def _prepare_append(case, g, randn):
    old, new = _growth(case)
    P, Hkv, D, kv = case["P"], case["Hkv"], case["D"], case["kv"]
    table = _table([_pages(a + b, P) for a, b in zip(old, new)], sum(_pages(a + b, P) for a, b in zip(old, new)) + 2, g)
    N = sum(_pages(a + b, P) for a, b in zip(old, new)) + 2
    req = torch.repeat_interleave(torch.arange(case["B"], device="cuda"), _ints(new))
    pos = torch.arange(sum(new), device="cuda") - (_ints(new).cumsum(0) - _ints(new))[req] + _ints(old)[req]
    slots = table[req, pos // P].long() * P + pos % P
    slots = torch.nn.functional.pad(slots, (0, case["pad"]), value=-1)   # rows of a padded batch
    qkv = randn(slots.shape[0], 6 * Hkv, D).to(BF)                 # keys and values are views of one projection's output
    k_pool, v_pool, scales = _caches(kv, N + 1, P, Hkv, D, randn)  # (a page more than the cache has, for the plain form's padded rows)
    bounds = randn(N + 1, Hkv, 2, D).to(BF) if case["bounds"] else None
    return dict(op="append", kv=kv, P=P, N=N, k=qkv[:, 4 * Hkv:5 * Hkv], v=qkv[:, 5 * Hkv:], slots=slots, k_pool=k_pool, v_pool=v_pool,
                scales=scales, bounds=bounds)


def _prepare_select(case, g, randn):
    L, P = _batch_lens(case), case["P"]
    pages = [_pages(n, P) for n in L]
    N = sum(pages) + 2
    D = case["D"]
    mid = randn(N, case["Hkv"], D) * 0.7
    half = randn(N, case["Hkv"], D).abs_() * 0.5 + 1.2
    bounds = torch.stack([mid - half, mid + half], 2).to(BF)
    return dict(op="select", P=P, Tq=case["Tq"], first=case["first"], last=case["last"],
                q=randn(case["B"], case["Tq"], case["Hq"], D).to(BF), bounds=bounds, table=_table(pages, N, g), lens=_ints(L),
                selected=torch.empty(case["B"], case["Tq"], case["Hkv"], case["keep"], dtype=I32, device="cuda"))


def _prepare_sparse(case, g, randn):
    L, P, B, Tq, Hkv, S = _batch_lens(case), case["P"], case["B"], case["Tq"], case["Hkv"], case["keep"]
    pages = [_pages(n, P) for n in L]
    N = sum(pages) + 2
    k, v, scales = _caches(case["kv"], N, P, Hkv, case["D"], randn)
    table = _table(pages, N, g)
    W = table.shape[1]
    n = (_ints(L)[:, None] - (Tq - 1) + torch.arange(Tq, device="cuda")).clamp(min=0)              # keys that token t sees
    seen = ((n + P - 1) // P)[:, :, None, None]
    at = torch.arange(W, device="cuda")
    order = torch.rand(B, Tq, Hkv, W, generator=g, device="cuda")
    order = torch.where(at == seen - 1, 2.0, order).masked_fill(at >= seen, -1.0)                  # the last page is always there
    pick = order.argsort(-1, descending=True)[..., :S]
    pick = torch.where(pick < seen, pick, W).sort(-1).values
    selected = torch.full((B, Tq, Hkv, S), -1, dtype=I32, device="cuda")
    selected[..., :pick.shape[-1]] = torch.where(pick < W, pick, -1).to(I32)
    return dict(op="sparse", kv=case["kv"], P=P, Tq=Tq, q=randn(B, Tq, case["Hq"], case["D"]).to(BF), k=k, v=v, scales=scales,
                table=table, lens=_ints(L), selected=selected, out=torch.empty(B, Tq, case["Hq"], case["D"], dtype=BF, device="cuda"),
                lse=torch.empty(B, Tq, case["Hq"], dtype=F32, device="cuda"))


def _prepare_logprobs(case, g, randn):
    R, V, K = case["R"], case["V"], case["K"]
    logits = randn(R, V, dtype=BF if case["dtype"] == "bf16" else F32).mul_(2.5)
    race = torch.rand(R, 64, generator=g, device="cuda")
    tokens = torch.randint(0, V, (R, 64), generator=g, device="cuda")
    tokens = tokens.gather(1, (logits.gather(1, tokens).float() - (-race.clamp(1e-9, 1 - 1e-7).log()).log()).argmax(1, True))[:, 0]
    if case["skip"]:                                               # rows without a token, as verification leaves them
        tokens[1:] = torch.where(torch.rand(R - 1, generator=g, device="cuda") < 0.1, -1, tokens[1:])
    empty = functools.partial(torch.empty, device="cuda")
    return dict(op="logprobs", K=K, logits=logits, tokens=tokens, logprobs=empty(R), ranks=empty(R, dtype=I32), entropy=empty(R),
                top_ids=empty(R, K, dtype=I32) if K else None, top_logprobs=empty(R, K) if K else None)


# ---------------------------------------------------------------------------
# one pass


def _run_own(s):
    import split_kv_paged_gqa_gb300 as fd
    if s["op"] == "slots":
        fd.fd_append_slots(s["lens"], s["new"], s["free"], s["n_free"], s["P"], s["table"], s["slots"], s["positions"],
                           s["new_lens"], s["cu"], s["taken"])
        return s["table"], s["slots"], s["positions"], s["new_lens"], s["cu"], s["taken"]
    if s["op"] == "append":
        N = s["N"]
        k, v = s["k_pool"][:N], s["v_pool"][:N]
        scales = None if s["scales"] is None else s["scales"][:, :N]
        bounds = None if s["bounds"] is None else s["bounds"][:N]
        fd.fd_cache_append(s["k"], s["v"], s["slots"], k, v, scales, bounds)
        return k, v, scales, bounds
    if s["op"] == "select":
        fd.fd_select_pages(s["q"], s["bounds"], s["table"], s["lens"], s["Tq"], s["P"], s["first"], s["last"], s["selected"])
        return s["selected"]
    if s["op"] == "sparse":
        fd.fd_decode_sparse(s["q"], s["k"], s["v"], s["scales"], s["table"], s["lens"], s["selected"], s["Tq"], 0.0, s["out"], s["lse"])
        return s["out"], s["lse"]
    fd.fd_token_logprobs(s["logits"], s["tokens"], s["logprobs"], s["ranks"], s["entropy"], s["top_ids"], s["top_logprobs"])
    return s["logprobs"], s["ranks"], s["entropy"], s["top_ids"], s["top_logprobs"]


def _plain_slots(s):
    P, table, free = s["P"], s["table"], s["free"].long()
    L, n = s["lens"].long(), s["new"].long()
    before, after = (L + P - 1) // P, (L + n + P - 1) // P
    need = after - before
    end = need.cumsum(0)
    served = (need == 0) | (end <= s["n_free"])                     # the requests that the free pages are enough for
    cu = torch.nn.functional.pad(n.cumsum(0), (1, 0))
    cols = torch.arange(table.shape[1], device="cuda")
    fresh = (cols >= before[:, None]) & (cols < after[:, None]) & served[:, None]
    table.copy_(torch.where(fresh, free[((end - need - before)[:, None] + cols).clamp(0, free.shape[0] - 1)], table.long()))
    i = torch.arange(s["slots"].shape[0], device="cuda")
    req = torch.searchsorted(cu[1:], i, right=True).clamp(max=L.shape[0] - 1)
    pos = L[req] + i - cu[req]
    page = table[req, (pos // P).clamp(max=table.shape[1] - 1)].long()
    real = i < cu[-1]
    slots = torch.where(real & served[req], page * P + pos % P, -1)
    return (table, slots.to(s["slots"].dtype), torch.where(real, pos, 0).to(I32), (L + n * served).to(I32), cu.to(I32),
            (need * served).sum().to(I32)[None])


def _codes_of(x, kv):
    """Codes and fp32 scales of rows [..., D]: the largest magnitude of a row (8 bits) or of 32 channels (4 bits) becomes 127 or 7."""
    top = 127 if kv == "int8" else 7
    x = x.double().unflatten(-1, (1 if kv == "int8" else x.shape[-1] // 32, -1))
    scale = (x.abs().amax(-1) / top).float()
    c = torch.where(scale[..., None] > 0, x / scale.double()[..., None], 0.0).round().clamp(-top, top).flatten(-2).to(torch.int8)
    return (c if kv == "int8" else (c[..., ::2] & 15 | c[..., 1::2] << 4).view(torch.uint8)), scale


def _values_of(codes, scale, kv):
    """The values that codes and scales stand for, in 64 bits (a code times a scale is exact there)."""
    if kv == "bf16":
        return codes.double()
    if kv == "int4":
        c = codes.view(torch.int8)
        codes = torch.stack([c << 4 >> 4, c >> 4], -1).flatten(-2)
    return (codes.double().unflatten(-1, (scale.shape[-1], -1)) * scale.double()[..., None]).flatten(-2)


def _outward(x, up):
    """The nearest bf16 value that is not below (up) or not above x."""
    y = x.to(BF)
    short = y.double() < x if up else y.double() > x
    bits = y.view(torch.int16)
    grow = (y > 0) | ((y == 0) & up) if up else (y < 0) | (y == 0)
    step = torch.where(grow, bits + 1, bits - 1)
    if not up:
        step = torch.where(y == 0, torch.full_like(bits, -32767), step)
    return torch.where(short, step.view(BF), y)


def _plain_append(s):
    kv, P, N, slots = s["kv"], s["P"], s["N"], s["slots"]
    row = torch.where(slots >= 0, slots, N * P)                     # padded rows go to the page behind the cache
    for x, pool, which in ((s["k"], s["k_pool"], 0), (s["v"], s["v_pool"], 1)):
        if kv == "bf16":
            pool.flatten(0, 1)[row] = x
        else:
            codes, scale = _codes_of(x, kv)
            pool.flatten(0, 1)[row] = codes
            s["scales"][which][row // P, row % P] = scale
    if s["bounds"] is not None:
        # the last new token of each page: the page's keys end there
        follows = torch.nn.functional.pad((slots[1:] == slots[:-1] + 1) & (slots[1:] % P > 0), (0, 1))
        last = slots[(slots >= 0) & ~follows]
        page, rows = last // P, torch.arange(P, device="cuda")
        x = _values_of(s["k_pool"][page], None if kv == "bf16" else s["scales"][0][page], kv)      # [pages, P, Hkv, D]
        here = (rows <= (last % P)[:, None])[..., None, None]
        lo = torch.where(here, x, math.inf).amin(1)
        hi = torch.where(here, x, -math.inf).amax(1)
        s["bounds"][page] = torch.stack([_outward(lo, False), _outward(hi, True)], 2)
    return (s["k_pool"][:N], s["v_pool"][:N], None if s["scales"] is None else s["scales"][:, :N],
            None if s["bounds"] is None else s["bounds"][:N])


def _plain_select(s):
    q, P, Tq, S = s["q"].double(), s["P"], s["Tq"], s["selected"].shape[-1]
    B, _, Hq, D = q.shape
    bounds = s["bounds"][s["table"].clamp(min=0).long()].double()                                  # [B, W, Hkv, 2, D]
    W, Hkv = bounds.shape[1:3]
    q = q.view(B, Tq, Hkv, Hq // Hkv, D)
    q = torch.stack([q.clamp(max=0).sum(3), q.clamp(min=0).sum(3)], 3).flatten(3)                  # against the lower and the upper bound
    score = torch.matmul(q.transpose(1, 2), bounds.flatten(3).permute(0, 2, 3, 1)).transpose(1, 2)  # [B, Tq, Hkv, W]
    n = (s["lens"][:, None] - (Tq - 1) + torch.arange(Tq, device="cuda")).clamp(min=0)             # keys that token t sees
    seen = ((n + P - 1) // P)[:, :, None, None]
    at = torch.arange(W, device="cuda")
    score = torch.where((at < s["first"]) | (at >= seen - s["last"]), math.inf, score).masked_fill(at >= seen, -math.inf)
    pick = torch.sort(score, dim=-1, descending=True, stable=True).indices[..., :S]                # ties: the lowest page
    pick = torch.where(pick < seen, pick, W).sort(-1).values
    pick = torch.where(pick < W, pick, -1)
    return torch.nn.functional.pad(pick, (0, S - pick.shape[-1]), value=-1).to(I32)


def _gather_rows(cache, scale, kv, page, h):
    """fp32 rows [..., P, D] of one head of the given pages."""
    x = cache[page, :, h]
    if kv == "bf16":
        return x.float()
    if kv == "int4":
        c = x.view(torch.int8)
        x = torch.stack([c << 4 >> 4, c >> 4], -1).flatten(-2)
    sc = scale[page, :, h]
    return (x.float().unflatten(-1, (sc.shape[-1], -1)) * sc[..., None]).flatten(-2)


def _plain_sparse(s):
    q, P, Tq, kv, sel = s["q"].float(), s["P"], s["Tq"], s["kv"], s["selected"].long()
    B, _, Hq, D = q.shape
    Hkv, S = sel.shape[2:]
    page = s["table"].long().gather(1, sel.clamp(min=0).flatten(1)).view(sel.shape).clamp(min=0)   # [B, Tq, Hkv, S]
    h = torch.arange(Hkv, device="cuda")[:, None]
    sc = (None, None) if s["scales"] is None else s["scales"]
    k = _gather_rows(s["k"], sc[0], kv, page, h).flatten(3, 4)                                     # [B, Tq, Hkv, S P, D]
    score = torch.matmul(q.view(B, Tq, Hkv, Hq // Hkv, D), k.transpose(-1, -2)).mul_(1.0 / math.sqrt(D))
    del k
    n = s["lens"][:, None] - (Tq - 1) + torch.arange(Tq, device="cuda")
    at = sel[..., None] * P + torch.arange(P, device="cuda")
    seen = ((at < n[:, :, None, None, None]) & (sel >= 0)[..., None]).flatten(3)[:, :, :, None]
    score = score.masked_fill(~seen, -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(torch.isfinite(top), top, torch.zeros_like(top))
    e = score.sub_(top).exp_()
    total = e.sum(-1, keepdim=True)
    lse = (top + total.log()).view(B, Tq, Hq)
    e.div_(torch.where(total > 0, total, torch.ones_like(total)))
    v = _gather_rows(s["v"], sc[1], kv, page, h).flatten(3, 4)
    return torch.matmul(e, v).view(B, Tq, Hq, D).to(BF), lse


def _plain_logprobs(s):
    x, tok = s["logits"].float(), s["tokens"]
    live = tok >= 0
    at = tok.clamp(min=0)[:, None]
    top = x.amax(-1, keepdim=True)
    z = x - top
    e = z.exp()
    total = e.sum(-1, keepdim=True)
    log_total = total.log()
    lse = top + log_total
    entropy = (log_total - e.mul_(z).sum(-1, keepdim=True) / total)[:, 0]
    del z, e
    xt = x.gather(1, at)
    ids = torch.arange(x.shape[1], device="cuda")
    rank = ((x > xt) | ((x == xt) & (ids < at))).sum(-1)
    out = [torch.where(live, (xt - lse)[:, 0], 0.0), torch.where(live, rank, -1).to(I32), torch.where(live, entropy, 0.0), None, None]
    if s["K"]:
        v, i = torch.sort(x, dim=-1, descending=True, stable=True)                                 # ties: the lowest token
        out[3] = torch.where(live[:, None], i[:, :s["K"]], -1).to(I32)
        out[4] = torch.where(live[:, None], v[:, :s["K"]] - lse, 0.0)
    return tuple(out)


def run(state):
    if own:
        return _run_own(state)
    return {"slots": _plain_slots, "append": _plain_append, "select": _plain_select, "sparse": _plain_sparse,
            "logprobs": _plain_logprobs}[state["op"]](state)


# ---------------------------------------------------------------------------
# what a pass cannot do without


def work(case):
    op = case["op"]
    if op == "slots":
        old, new = _growth(case)
        T, B, P = sum(new) + case["pad"], case["B"], case["P"]
        more = sum(_pages(a + b, P) - _pages(a, P) for a, b in zip(old, new))
        return {"bytes": B * 4 * 4 + T * (12 if case["wide"] else 8) + 8 * more, "flops": 4 * T}
    if op == "append":
        old, new = _growth(case)
        T, Hkv, D, P = sum(new), case["Hkv"], case["D"], case["P"]
        stored = {"bf16": 2 * D, "int8": D + 4, "int4": D // 2 + D // 8}[case["kv"]]
        nbytes = T * (2 * Hkv * (2 * D + stored) + 8)
        if case["bounds"]:
            # the keys that a request's first changed page holds already, and a pair of bounds for each changed page
            kept = sum(a % P for a, b in zip(old, new) if b)
            pages = sum(_pages(a + b, P) - a // P for a, b in zip(old, new) if b)
            nbytes += kept * Hkv * stored + pages * Hkv * 4 * D
        return {"bytes": nbytes, "flops": 4 * T * Hkv * D}
    if op in ("select", "sparse"):
        B, Tq, Hq, Hkv, D, P, S = (case[k] for k in ("B", "Tq", "Hq", "Hkv", "D", "P", "keep"))
        L = _batch_lens(case)
        if op == "select":
            pages = [_pages(n, P) if _pages(n, P) > S else 0 for n in L]      # (no choice where all pages fit)
            return {"bytes": sum(pages) * (Hkv * 4 * D + 4) + B * Tq * (Hq * D * 2 + Hkv * S * 4),
                    "flops": sum(pages) * Tq * Hkv * 4 * D}
        row = 2 * {"bf16": 2 * D, "int8": D + 4, "int4": D // 2 + D // 8}[case["kv"]]
        keys = pages = read = 0
        for n in L:
            each = []
            for t in range(Tq):
                m = max(0, n - (Tq - 1) + t)
                p = min(S, _pages(m, P))
                pages += p
                each.append(max(0, p * P - (-m % P)))
            keys += sum(each)
            # the tokens of a request choose on their own: what several of them chose is read once, at least the longest choice
            read += max(each)
        return {"bytes": read * Hkv * row + B * Tq * Hq * (4 * D + 4) + pages * Hkv * 4, "flops": keys * Hq * 4 * D}
    size = 2 if case["dtype"] == "bf16" else 4
    return {"bytes": case["R"] * (case["V"] * size * (0.9 if case["skip"] else 1) + 8 + 12 + 8 * case["K"]), "flops": 6 * case["R"] * case["V"]}


# ---------------------------------------------------------------------------
# the definition in 64 bits


def _exact_slots(s):
    P, F = s["P"], int(s["n_free"])
    table, free = s["table"].tolist(), s["free"].tolist()
    slots, positions, lens, cu, taken, asked = [], [], [], [0], 0, 0
    for b, (L, n) in enumerate(zip(s["lens"].tolist(), s["new"].tolist())):
        first, last = _pages(L, P), _pages(L + n, P)
        asked += last - first
        ok = last == first or asked <= F
        if ok:
            taken += last - first
            table[b][first:last] = free[asked - (last - first):asked]
        slots += [table[b][p // P] * P + p % P if ok else -1 for p in range(L, L + n)]
        positions += range(L, L + n)
        lens.append(L + n if ok else L)
        cu.append(cu[-1] + n)
    T = s["slots"].shape[0]
    return (_ints(table), _ints(slots + [-1] * (T - len(slots)), s["slots"].dtype), _ints(positions + [0] * (T - len(positions))),
            _ints(lens), _ints(cu), _ints([taken]))


def _exact_append(s):
    kv, P, N = s["kv"], s["P"], s["N"]
    k, v = s["k_pool"][:N].clone(), s["v_pool"][:N].clone()
    scales = None if s["scales"] is None else s["scales"][:, :N].clone()
    there = torch.nonzero(s["slots"] >= 0)[:, 0]
    page, off = s["slots"][there] // P, s["slots"][there] % P
    top = 127.0 if kv == "int8" else 7.0
    for i, (x, cache) in enumerate(((s["k"], k), (s["v"], v))):
        x = x[there].double()
        if kv == "bf16":
            cache[page, off] = x.to(BF)
            continue
        groups = x.view(*x.shape[:2], 1 if kv == "int8" else x.shape[2] // 32, -1)
        sc = (groups.abs().max(-1).values / top).to(F32)
        c = (groups / sc.double()[..., None]).nan_to_num(0.0).round().clamp(-top, top).reshape(x.shape).to(I32)
        cache[page, off] = c.to(torch.int8) if kv == "int8" else (c[..., 0::2] % 16 + 16 * (c[..., 1::2] % 16)).to(torch.uint8)
        scales[i][page, off] = sc
    bounds = None
    if s["bounds"] is not None:
        bounds = s["bounds"][:N].clone().double()
        end = torch.zeros(N, dtype=I64, device="cuda").scatter_reduce_(0, page, off + 1, "amax")
        for o in range(P):                                     # a page's keys one after the other
            p = torch.nonzero(end > o)[:, 0]
            if not p.numel():
                break
            x = k[p, o]
            if kv == "int4":
                x = torch.stack([(x.int() + 8) % 16 - 8, (x.int() // 16 + 8) % 16 - 8], -1).flatten(-2)
            x = x.double()
            if kv != "bf16":
                sc = scales[0][p, o].double()
                x = x * sc.repeat_interleave(x.shape[-1] // sc.shape[-1], -1)
            bounds[p, :, 0] = x if o == 0 else torch.minimum(bounds[p, :, 0], x)
            bounds[p, :, 1] = x if o == 0 else torch.maximum(bounds[p, :, 1], x)
        grown = bounds.float()
        near = grown.to(BF).double()
        away = torch.tensor([-math.inf, math.inf], dtype=BF, device="cuda").view(1, 1, 2, 1).expand(bounds.shape)
        off_side = torch.stack([near[:, :, 0] > bounds[:, :, 0], near[:, :, 1] < bounds[:, :, 1]], 2)
        bounds = torch.where(off_side, torch.nextafter(grown.to(BF).cpu(), away.cpu()).cuda().double(), near)
    return k, v, scales, bounds


def _exact_select(s):
    B, Tq, Hkv, S = s["selected"].shape
    out = torch.full((B, Tq, Hkv, S), -1, dtype=I32, device="cuda")
    G = s["q"].shape[2] // Hkv
    for b, L in enumerate(s["lens"].tolist()):
        bounds = s["bounds"][s["table"][b, :max(1, _pages(L, s["P"]))].long()].double()
        for t in range(Tq):
            n = _pages(max(0, L - (Tq - 1) + t), s["P"])
            if n <= S:
                out[b, t, :, :n] = torch.arange(n, device="cuda")
                continue
            q = s["q"][b, t].double().view(1, Hkv, G, -1)
            each = torch.maximum(q * bounds[:n, :, None, 0], q * bounds[:n, :, None, 1])   # the largest that a key in the bounds can add
            score = each.sum((-1, -2)).T                                                  # [Hkv, n]
            score[:, :s["first"]] = math.inf
            score[:, n - s["last"]:] = math.inf
            limit = score.sort(-1, descending=True).values[:, S - 1:S]
            above, equal = score > limit, score == limit
            keep = above | (equal & (equal.cumsum(-1) <= S - above.sum(-1, keepdim=True)))
            out[b, t] = torch.nonzero(keep)[:, 1].view(Hkv, S).to(I32)
    return out


def _exact_sparse(s):
    B, Tq, Hq, D = s["q"].shape
    Hkv, P, kv = s["selected"].shape[2], s["P"], s["kv"]
    out = torch.zeros(B, Tq, Hq, D, dtype=F64, device="cuda")
    lse = torch.full((B, Tq, Hq), -math.inf, dtype=F64, device="cuda")
    offs, heads = torch.arange(P, device="cuda"), torch.arange(Hkv, device="cuda")[:, None]
    for b, L in enumerate(s["lens"].tolist()):
        for t in range(Tq):
            n = L - (Tq - 1) + t
            if n <= 0:
                continue
            sel = s["selected"][b, t].long()                                       # [Hkv, S]
            pos = (sel[..., None] * P + offs).flatten(1)
            seen = (pos < n) & (sel >= 0).repeat_interleave(P, 1)
            page = s["table"][b].long()[sel.clamp(min=0)].repeat_interleave(P, 1).clamp(min=0)
            rows = []
            for i, cache in ((0, s["k"]), (1, s["v"])):
                codes = cache[page, pos % P, heads]
                rows.append(_values_of(codes, None if kv == "bf16" else s["scales"][i][page, pos % P, heads], kv))
            z = torch.einsum("hgd,hkd->hgk", s["q"][b, t].double().view(Hkv, -1, D), rows[0]) / math.sqrt(D)
            z = z.masked_fill(~seen[:, None], -math.inf)
            lse[b, t] = torch.logsumexp(z, -1).view(Hq)
            out[b, t] = torch.einsum("hgk,hkd->hgd", torch.softmax(z, -1).nan_to_num(0.0), rows[1]).reshape(Hq, D)
    return out, lse


def _exact_logprobs(s):
    R, V = s["logits"].shape
    K = s["K"]
    lp, ent = torch.zeros(R, dtype=F64, device="cuda"), torch.zeros(R, dtype=F64, device="cuda")
    rank = torch.full((R,), -1, dtype=I32, device="cuda")
    ids = torch.full((R, K), -1, dtype=I32, device="cuda") if K else None
    top = torch.zeros(R, K, dtype=F64, device="cuda") if K else None
    for r0 in range(0, R, 256):
        live = torch.nonzero(s["tokens"][r0:r0 + 256] >= 0)[:, 0] + r0
        if not live.numel():
            continue
        y = torch.log_softmax(s["logits"][live].double(), -1)
        x = s["logits"][live].float()
        at = s["tokens"][live]
        mine = torch.arange(live.numel(), device="cuda")
        lp[live] = y[mine, at]
        ent[live] = -(y.exp() * y).sum(-1)
        before = torch.arange(V, device="cuda")[None] < at[:, None]
        rank[live] = (torch.where(before, x >= x[mine, at][:, None], x > x[mine, at][:, None])).sum(-1).to(I32)
        left = x.clone()
        for j in range(K):                                     # the most probable of those that are left
            i = (left == left.amax(-1, keepdim=True)).int().argmax(-1)
            ids[live, j] = i.to(I32)
            top[live, j] = y[mine, i]
            left[mine, i] = -math.inf
    return lp, rank, ent, ids, top


def exact(case, seed):
    s = prepare(case, seed)
    return {"slots": _exact_slots, "append": _exact_append, "select": _exact_select, "sparse": _exact_sparse,
            "logprobs": _exact_logprobs}[case["op"]](s)
