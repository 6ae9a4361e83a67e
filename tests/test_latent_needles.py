"""Latent attention, each key counted once. Over a long range a lost or doubled key
of ordinary weight stays within what rounding alone may do, so here one key takes
all of a row's weight: at both sides of every tile's border (which the borders of
CTAs, of parts and of requests are among), at the ends of the range and at the causal
limit. A lost key changes the row's output, a doubled one its LSE by ln 2."""
import math

import numpy as np
import pytest
import torch

import split_kv_paged_gqa_gb300 as fd
from oracle.latent_ref import latent_decode_ref, latent_prefill_ref

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32
SCALE = 1.0 / math.sqrt(192)
# A score here is a sum of 192 or 576 fp32 products that reaches 170: off by at most
# (576 + 2) 2^-23 170 = 0.012. The other keys weigh e^-100 of the needle and less
# (they round to 0 as bf16, and leave a sum of 1 as it is).
LSE_TOL = 0.05


def check(out, lse, want, score, sees):
    """out [..., D], lse [...]; per row the needle's values and score, and whether
    the row sees it."""
    assert torch.equal(out[sees], want[sees]), "a needle's values differ"
    assert (lse[sees].double() - score[sees]).abs().max() < LSE_TOL, "a needle's LSE differs"
    assert not (lse[~sees] > 60).any(), "a needle reaches a row that does not see it"


def positions(L, tile, Lq=1):
    """Keys at both sides of the tiles' borders, at the ends and at the causal limits
    of a range's first and last queries."""
    at = {0, 1, L - 1, L - 2, L - Lq - 1, L - Lq, L - Lq + 1, L // 3} | {k for t in range(tile, L, tile) for k in (t - 1, t)}
    return sorted(k for k in at if 0 <= k < L)


# ---------------------------------------------------------------------------
# decode


def decode_inputs(lens, Tq, H, P, g):
    B = len(lens)
    pages = [-(-n // P) for n in lens]
    N, W = sum(pages) + 2, max(1, max(pages))
    order = torch.randperm(N, generator=g).to(I32)
    table = torch.full((B, W), 1 << 30, dtype=I32)
    at = 0
    for b, n in enumerate(pages):
        table[b, :n] = order[at:at + n]
        at += n
    return dict(q=torch.randn(B, Tq, H, 576, generator=g).to(BF), kv_cache=torch.randn(N, P, 576, generator=g).to(BF),
                page_table=table, cache_seqlens=torch.tensor(lens, dtype=I32), q_per_req=Tq)


def plant_decode(a, lens, part):
    """A copy of the cache in which row (token, head) r of each request has its query
    times four at the (part * rows + r)-th of the request's positions, and what each
    row should give."""
    B, Tq, H, _ = a["q"].shape
    P, rows = a["kv_cache"].shape[1], Tq * H
    cache = a["kv_cache"].clone()
    dev = cache.device
    want, score = torch.zeros(B, Tq, H, 512, dtype=BF, device=dev), torch.zeros(B, Tq, H, dtype=torch.float64, device=dev)
    sees = torch.zeros(B, Tq, H, dtype=torch.bool, device=dev)
    for b, L in enumerate(lens):
        keys = positions(L, 64, Tq)
        if not keys:
            continue
        picked, used = [], set()
        for r in range(rows):
            k = keys[(part * rows + r) % len(keys)]
            picked.append(-1 if k in used else k)     # (a key carries one row's needle)
            used.add(k)
        r = torch.tensor([i for i, k in enumerate(picked) if k >= 0], device=dev)
        k = torch.tensor([k for k in picked if k >= 0], device=dev)
        q = a["q"][b].reshape(rows, 576)[r]
        cache[a["page_table"][b].long()[k // P], k % P] = q * 4
        want[b].view(rows, 512)[r] = q[:, :512] * 4
        score[b].view(rows)[r] = (q.double() * q.double() * 4).sum(-1) * SCALE
        sees[b].view(rows)[r] = k < L - (Tq - 1) + r // H
    return cache, want, score, sees


def test_decode_needles_show_a_lost_and_a_doubled_key():
    """The check on the float64 oracle: it holds, and fails with one key of one
    row's needle taken out or put in twice."""
    g = torch.Generator().manual_seed(1)
    lens, P = [300], 300
    a = decode_inputs(lens, 2, 2, P, g)
    a["page_table"][:] = 0
    cache, want, score, sees = plant_decode(a, lens, 0)
    table = a["page_table"].numpy()

    def run(rows):
        o, s, _, _ = latent_decode_ref(a["q"].double().numpy(), rows[None], table, [rows.shape[0]], SCALE)
        return torch.from_numpy(o).to(BF), torch.from_numpy(s)

    rows = cache[0].double().numpy()
    check(*run(rows), want, score, sees)
    at = int(np.argwhere((cache[0, :, :512] == want[0, 0, 0]).all(-1).numpy())[0, 0])
    for wrong in (np.delete(rows, at, 0), np.insert(rows, at, rows[at], 0)):
        with pytest.raises(AssertionError, match="needle"):
            check(*run(wrong), want, score, sees)


@pytest.mark.gpu
@pytest.mark.parametrize("lens,Tq,H,P", [([9001], 1, 16, 64), ([32768], 1, 128, 64), ([4000, 65, 300, 0, 1, 2500], 4, 16, 16),
                                         ([2600, 64, 7000], 1, 100, 128), ([5000, 129], 3, 70, 8), ([500] * 30 + [6000], 1, 12, 32)])
def test_decode_needles_at_every_tile_border(lens, Tq, H, P):
    g = torch.Generator().manual_seed(len(lens) + H)
    a = {k: v.cuda() if torch.is_tensor(v) else v for k, v in decode_inputs(lens, Tq, H, P, g).items()}
    out, lse = torch.empty(len(lens), Tq, H, 512, dtype=BF, device="cuda"), torch.empty(len(lens), Tq, H, device="cuda")
    plan = fd.fd_latent_plan_create(0, len(lens), Tq, H, P, SCALE)
    fd.fd_set_plan(plan)
    try:
        for part in range(-(-len(positions(max(lens), 64, Tq)) // (Tq * H))):
            cache, want, score, sees = plant_decode(a, lens, part)
            fd.fd_decode_latent(**{**a, "kv_cache": cache}, out=out, lse=lse)
            assert sees.any()
            check(out, lse, want, score, sees)
        assert fd.fd_read_device_status(plan) == 0
    finally:
        fd.fd_set_plan(None)
        fd.fd_plan_destroy(plan)


# ---------------------------------------------------------------------------
# prompts


def prefill_inputs(lq, lk, H, g):
    """Queries whose 128 channels are one vector of +-1 a head."""
    Sq, Sk = sum(lq), sum(lk)
    sign = torch.randint(0, 2, (H, 128), generator=g).to(BF) * 2 - 1
    q = torch.randn(Sq, H, 192, generator=g).to(BF)
    q[..., :128] = sign
    cu = lambda n: torch.tensor(np.concatenate([[0], np.cumsum(n)]), dtype=I32)   # noqa: E731
    return sign, dict(q=q, k_nope=torch.randn(Sk, H, 128, generator=g).to(BF), k_pe=torch.randn(Sk, 64, generator=g).to(BF),
                      v=torch.randn(Sk, H, 128, generator=g).to(BF), cu_seqlens_q=cu(lq), cu_seqlens_k=cu(lk),
                      max_seqlen_q=max(lq), softmax_scale=SCALE)


def plant_prefill(a, sign, lq, lk, part):
    """Keys in which head h of each request has its sign vector times 16 at the
    (part * H + h)-th of the request's positions, and what each row should give."""
    Sq, H, _ = a["q"].shape
    k_nope = a["k_nope"].clone()
    dev = k_nope.device
    want, score = torch.zeros(Sq, H, 128, dtype=BF, device=dev), torch.zeros(Sq, H, dtype=torch.float64, device=dev)
    sees = torch.zeros(Sq, H, dtype=torch.bool, device=dev)
    heads = torch.arange(H, device=dev)
    q0 = s0 = 0
    for n, m in zip(lq, lk):
        keys = positions(m, 128, n)
        if n and keys:
            k = torch.tensor([keys[(part * H + h) % len(keys)] for h in range(H)], device=dev)
            k_nope[s0 + k, heads] = sign * 16
            want[q0:q0 + n] = a["v"][s0 + k, heads]
            pe = torch.einsum("shc,hc->sh", a["q"][q0:q0 + n, :, 128:].double(), a["k_pe"][s0 + k].double())
            score[q0:q0 + n] = (pe + 16 * 128) * SCALE
            sees[q0:q0 + n] = k < torch.arange(n, device=dev)[:, None] + 1 + m - n
        q0, s0 = q0 + n, s0 + m
    return k_nope, want, score, sees


def test_prefill_needles_show_a_lost_and_a_doubled_key():
    g = torch.Generator().manual_seed(2)
    lq, lk = [5], [140]
    sign, a = prefill_inputs(lq, lk, 2, g)
    k_nope, want, score, sees = plant_prefill(a, sign, lq, lk, 1)
    full = [x.double().numpy() for x in (k_nope, a["k_pe"], a["v"])]

    def run(k, pe, v):
        o, s, _, _ = latent_prefill_ref(a["q"].double().numpy(), k, pe, v, [0, 5], [0, k.shape[0]], SCALE)
        return torch.from_numpy(o).to(BF), torch.from_numpy(s)

    check(*run(*full), want, score, sees)
    at = int(np.argwhere((k_nope[:, 0] == sign[0] * 16).all(-1).numpy())[0, 0])
    for wrong in ([np.delete(x, at, 0) for x in full], [np.insert(x, at, x[at], 0) for x in full]):
        with pytest.raises(AssertionError, match="needle"):
            check(*run(*wrong), want, score, sees)


# (heads set how many CTAs share a tile of queries: 8, 4, 2 and 1 in the first four)
@pytest.mark.gpu
@pytest.mark.parametrize("lq,lk,H", [([200], [9000], 8), ([200], [9000], 20), ([200], [9000], 40), ([200], [9000], 80),
                                     ([300], [3000], 4), ([1], [4100], 20), ([700], [1000], 60), ([1300], [1300], 6),
                                     ([150, 3, 290], [3000, 3, 4100], 10), ([260, 0, 31, 900], [700, 5, 31, 900], 40),
                                     ([1700] + [20] * 40, [1800] + [21] * 40, 12)])
def test_prefill_needles_at_every_tile_border(lq, lk, H):
    g = torch.Generator().manual_seed(sum(lk) + H)
    sign, a = prefill_inputs(lq, lk, H, g)
    sign, a = sign.cuda(), {k: v.cuda() if torch.is_tensor(v) else v for k, v in a.items()}
    out, lse = torch.empty(sum(lq), H, 128, dtype=BF, device="cuda"), torch.empty(sum(lq), H, device="cuda")
    status = torch.zeros(1, dtype=I32, device="cuda")
    for part in range(-(-max(len(positions(m, 128, n)) for n, m in zip(lq, lk)) // H)):
        k_nope, want, score, sees = plant_prefill(a, sign, lq, lk, part)
        fd.fd_prefill_latent(**{**a, "k_nope": k_nope}, out=out, lse=lse, status=status)
        assert sees.any()
        check(out, lse, want, score, sees)
    assert int(status) == 0
