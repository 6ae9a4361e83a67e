"""Log probabilities of given tokens: the oracle's pins and the refusals (CPU), the
kernel against the oracle (GPU)."""
import math

import numpy as np
import pytest
import torch

import split_kv_paged_gqa_gb300 as fd
from oracle.step_ref import logprobs_ref

BF, F32, I32, I64 = torch.bfloat16, torch.float32, torch.int32, torch.int64


def test_oracle_hand_worked():
    x = np.log(np.array([0.5, 0.125, 0.125, 0.25]))
    lp, rank, ent, ids, top = logprobs_ref(x + 7.0, 2, 3)
    assert lp == pytest.approx(math.log(0.125)) and rank == 3 and ids.tolist() == [0, 3, 1]
    assert ent == pytest.approx(0.5 * math.log(2) + 0.25 * math.log(4) + 0.25 * math.log(8))
    assert top == pytest.approx(np.log([0.5, 0.25, 0.125]))
    lp, rank, ent, ids, top = logprobs_ref(np.array([-np.inf, 0.0, -np.inf]), 2, 3)
    assert lp == -np.inf and rank == 2 and ent == 0.0 and ids.tolist() == [1, 0, 2] and top.tolist() == [0.0, -np.inf, -np.inf]


def _args(R=3, V=50, K=4):
    return dict(logits=torch.zeros(R, V), tokens=torch.zeros(R, dtype=I64), logprobs=torch.zeros(R), ranks=torch.zeros(R, dtype=I32),
                entropy=torch.zeros(R), top_ids=torch.zeros(R, K, dtype=I32), top_logprobs=torch.zeros(R, K))


@pytest.mark.parametrize("change,status", [
    (dict(logits=torch.zeros(3, 50, dtype=torch.float16)), fd.FD_ERR_INVALID_ARG),
    (dict(logits=torch.zeros(3, 100)[:, ::2]), fd.FD_ERR_UNSUPPORTED),
    (dict(logits=torch.zeros(150)), fd.FD_ERR_INVALID_ARG),
    (dict(logits=None), fd.FD_ERR_INVALID_ARG),
    (dict(logits=torch.zeros(0, 50), tokens=torch.zeros(0, dtype=I64)), fd.FD_ERR_INVALID_ARG),
    (dict(tokens=torch.zeros(3)), fd.FD_ERR_INVALID_ARG),
    (dict(tokens=torch.zeros(2, dtype=I64)), fd.FD_ERR_INVALID_ARG),
    (dict(logprobs=torch.zeros(3, dtype=BF)), fd.FD_ERR_INVALID_ARG),
    (dict(logprobs=torch.zeros(6)[::2]), fd.FD_ERR_UNSUPPORTED),
    (dict(ranks=torch.zeros(3, dtype=I64)), fd.FD_ERR_INVALID_ARG),
    (dict(entropy=torch.zeros(4)), fd.FD_ERR_INVALID_ARG),
    (dict(top_ids=None), fd.FD_ERR_INVALID_ARG),
    (dict(top_logprobs=None), fd.FD_ERR_INVALID_ARG),
    (dict(top_ids=torch.zeros(3, 33, dtype=I32), top_logprobs=torch.zeros(3, 33)), fd.FD_ERR_INVALID_ARG),
    (dict(top_logprobs=torch.zeros(3, 5)), fd.FD_ERR_INVALID_ARG),
    (dict(top_ids=torch.zeros(1, 4, dtype=I32).expand(3, 4)), fd.FD_ERR_UNSUPPORTED),
    (dict(logits=torch.zeros(3, 3)), fd.FD_ERR_INVALID_ARG),
    (dict(status=torch.zeros(1)), fd.FD_ERR_INVALID_ARG),
])
def test_rejects(change, status):
    with pytest.raises(fd.FdError) as e:
        fd.fd_token_logprobs(**{**_args(), **change}, stream=0)
    assert e.value.status == status, str(e.value)


def run(logits, tokens, K, out=None):
    R = logits.shape[0]
    e = lambda *n, dtype=F32: torch.full(n, 777, dtype=dtype, device="cuda")   # noqa: E731
    o = out or dict(logprobs=e(R), ranks=e(R, dtype=I32), entropy=e(R), top_ids=e(R, K, dtype=I32) if K else None,
                    top_logprobs=e(R, K) if K else None)
    status = torch.zeros(1, dtype=I32, device="cuda")
    fd.fd_token_logprobs(logits, tokens, **o, status=status)
    return o, int(status)


def tolerance(V, z):
    """Bounds on the errors of fp32 sums, with z = x - m and p the softmax. An exponential is off by 2^-21 of its value,
    and by |z| 2^-23 for the rounding of its argument: 2^-21 + 2^-23 E|z| of the sum, and E|z| = H - ln l is at most
    ln V < 17. A new maximum rescales a sum by a factor that is off by as much; 15 times in a thread on average at most
    for values in any order (ln of their number), and twice for each of the 9 joins of the tree: with the values
    themselves at most 40 of these errors. A thread adds at most V / 512 + 16 values, 2^-24 each. The logarithm of a
    sum that is off by d is off by d; the difference x - m and the result round by 2^-24 of their size."""
    d = 40 * (2.0 ** -21 + 17 * 2.0 ** -23) + (V / 512 + 26) * 2.0 ** -24
    return d + 2.0 ** -22 * (np.abs(z) + 1), d


def check(logits, tokens, K, out=None):
    o, status = run(logits, tokens, K, out)
    assert status == 0
    return compare(o, logits, tokens, K)


def compare(o, logits, tokens, K):
    x, tok = logits.double().cpu().numpy(), tokens.cpu().numpy()
    V = x.shape[1]
    for r in range(len(tok)):
        get = lambda k: o[k][r].cpu().numpy()   # noqa: E731,B023
        if tok[r] < 0:
            assert get("logprobs") == 0 and get("ranks") == -1 and get("entropy") == 0
            assert not K or ((get("top_ids") == -1).all() and (get("top_logprobs") == 0).all())
            continue
        lp, rank, ent, ids, top = logprobs_ref(x[r], int(tok[r]), K)
        tol, d = tolerance(V, lp)
        with np.errstate(over="ignore"):              # (beyond fp32 the nearest value is -inf)
            assert np.isfinite(np.float32(lp)) or get("logprobs") == np.float32(lp)
        assert not np.isfinite(np.float32(lp)) or abs(get("logprobs") - lp) <= tol, (r, get("logprobs"), lp)
        assert get("ranks") == rank
        # ln l, and a mean of z weighted with p: both terms off by d of at most ln V and of E|z|
        z = x[r] - (x[r].max() if np.isfinite(x[r].max()) else 0.0)
        p = np.exp(z) / max(np.exp(z).sum(), 1e-300)
        mean = (p[p > 0] * np.abs(z[p > 0])).sum()
        assert abs(get("entropy") - ent) <= d * (2 + 2 * mean) + 2.0 ** -22 * (1 + math.log(V) + mean), (r, get("entropy"), ent)
        if K:
            assert np.array_equal(get("top_ids"), ids)
            tol, _ = tolerance(V, top)
            with np.errstate(invalid="ignore", over="ignore"):
                assert ((get("top_logprobs") == np.float32(top)) | (np.abs(get("top_logprobs") - top) <= tol)).all()
    return o


def make(R, V, seed, dtype=F32, pad=0, scale=2.5):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(R, V + pad, generator=g) * scale).to(dtype).cuda()[:, :V]
    return x, torch.randint(0, V, (R,), generator=g).cuda()


@pytest.mark.gpu
@pytest.mark.parametrize("V", [1, 2, 7, 8, 31, 33, 500, 4095, 8192, 8193, 50021, 131072, 200003])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_vocabularies(V, dtype):
    for K in {0, 1, min(20, V), min(32, V)}:
        check(*make(3, V, V, dtype), K)


@pytest.mark.gpu
@pytest.mark.parametrize("R", [1, 2, 5, 40, 100, 200, 700, 899, 900])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_rows(R, dtype):
    x, tok = make(R, 9001, R, dtype, pad=R % 7)
    if R > 3:
        tok[2::3] = -1
    check(x, tok.to(I32) if R % 2 else tok, 8)
    x, tok = make(R, 20001, R + 1, dtype)                # rows too long for the smallest CTAs
    check(x, tok, 32)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("shift", range(8))
def test_rows_at_any_place(dtype, shift):
    g = torch.Generator().manual_seed(shift)
    flat = (torch.randn(8 + 5 * 1003, generator=g) * 3).to(dtype).cuda()
    x = flat[shift:shift + 5 * 1003].view(5, 1003)
    check(x, torch.tensor([0, 1002, 5, 500, 999]).cuda(), 32)
    check(x[:, :40], torch.tensor([0, 39, 5, 20, 33]).cuda(), 32)


@pytest.mark.gpu
@pytest.mark.parametrize("V", [600, 20000])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_ties(V, dtype):
    g = torch.Generator().manual_seed(V)
    x = torch.randint(0, 4, (6, V), generator=g).to(dtype).cuda()        # a few values, each many times
    x[0] = 1.5
    x[1, 37:] = x[1, 37]
    x[2] = torch.randint(-1, 1, (V,), generator=g).to(dtype).cuda() * 0.0   # +0 and -0
    check(x, torch.randint(0, V, (6,), generator=g).cuda(), 32)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF])
def test_zeros_of_both_signs_are_equal(dtype):
    V = 5003
    x = torch.zeros(8, V, dtype=dtype)
    x[:, ::3] = -0.0
    x[4:] = -x[4:]
    smallest = 2.0 ** -149 if dtype == F32 else 2.0 ** -133
    x[2, 7::50], x[3, 8::50], x[6, 9::50], x[7, 10::50] = smallest, -smallest, smallest, -smallest
    for tok in (0, 1, 2500, 2501, 2502, 4998, 57, 58, 59, 60):
        check(x.cuda(), torch.full((8,), tok, device="cuda"), 32)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF])
def test_sorted_and_sharp_rows(dtype):
    V = 30011
    x = torch.stack([torch.arange(V) * 1e-3, -torch.arange(V) * 1e-3, torch.full((V,), -20.0), torch.arange(V) % 97 * 1.0,
                     torch.randn(V, generator=torch.Generator().manual_seed(1)) * 100]).to(dtype).cuda()
    x[2, 12345] = 30.0
    check(x, torch.tensor([0, V - 1, 12345, 96, 17]).cuda(), 20)


@pytest.mark.gpu
@pytest.mark.parametrize("V", [1, 33, 509, 1531])
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("K,copies", [(0, 175), (8, 175), (32, 700)])
def test_many_short_rows(V, dtype, K, copies):
    """Rows of every kind, again and again: the first ones against 64 bits, the others equal to them bit for bit."""
    K = min(K, V)
    g = torch.Generator().manual_seed(V)
    x = (torch.randn(16, V, generator=g) * 3).to(dtype)
    x[1] = torch.randint(0, 4, (V,), generator=g).to(dtype)
    x[2] = 1.5
    x[3] = torch.randint(-1, 1, (V,), generator=g).to(dtype) * 0.0        # +0 and -0
    x[4, V // 2:] = -math.inf
    x[5, :V // 3] = torch.finfo(dtype).min
    x[6, 1:] = -math.inf
    x[7] = (torch.arange(V) * 0.01).to(dtype)
    x[8] = -x[7]
    x[9] = -20.0
    x[9, V // 4] = 30.0
    x[10] = x[10] - 3e4
    x[11] = x[11] * 100
    x[12, ::2] = -math.inf
    x[12, 0] = 1.0
    n, lead = x.shape[0], V % 8
    wide = torch.zeros(n * copies, (V + lead + 7) // 8 * 8 + 8, dtype=dtype, device="cuda")
    rows = wide[:, lead:lead + V]
    rows.copy_(x.repeat(copies, 1))
    tok = torch.randint(0, V, (n,), generator=g)
    tok[0], tok[1], tok[14] = V - 1, 0, -1
    tok[9] = V // 4
    o, status = run(rows, tok.repeat(copies).cuda(), K)
    assert status == 0
    compare({k: v[:n] if v is not None else None for k, v in o.items()}, rows[:n], tok, K)
    for k, v in o.items():
        if v is not None:
            v = v.view(I32).view(copies, n, -1)
            assert torch.equal(v, v[:1].expand_as(v)), k
    rows[3::n, V // 2] = math.nan
    rows[11::n, V // 2] = math.inf
    o, status = run(rows, tok.repeat(copies).cuda(), K)
    assert status == 0
    assert torch.isnan(o["logprobs"].view(copies, n)[:, [3, 11]]).all()
    good = [r for r in range(n) if r not in (3, 11)]
    compare({k: v[good] if v is not None else None for k, v in o.items()}, rows[good], tok[good], K)
    if K:
        assert (o["top_ids"][11::n, 0] == V // 2).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("R,V,K", [(3, 20000, 5), (2, 131072, 20), (320, 30000, 5), (1000, 20001, 5), (1000, 9000, 20), (2500, 3001, 5)])
def test_ranks_among_low_logits_behind_masks(dtype, R, V, K):
    """-inf in front of, between and behind logits far below 0, on 1 to 8 CTAs of 256 to 32 threads a row."""
    g = torch.Generator().manual_seed(V)
    x = torch.full((8, V), -math.inf)
    for r, low in enumerate((-50.0, -130.0, -200.0, -900.0, -3e4)):
        x[r, V // 2:] = torch.randn(V - V // 2, generator=g) * 3 + low
    x[0, V // 2::7] = -130.0
    x[5, ::5] = torch.randn(x[5, ::5].numel(), generator=g) * 30 - 300
    x[6, V - 40:] = torch.randn(40, generator=g) * 100 - 400
    x[7, : V // 3] = torch.randn(V // 3, generator=g) - 150
    x[7, V // 3:] = -math.inf
    x = x.to(dtype)
    # a token of middling rank among the finite ones, and one that is the last of all
    tok = torch.zeros(2, 8, dtype=I64)
    for r in range(8):
        order = torch.argsort(x[r].double(), descending=True, stable=True)[:int(torch.isfinite(x[r]).sum())]
        tok[:, r] = order[torch.tensor([order.numel() // 2, order.numel() - 1])]
    for first in range(0, 8, R):
        rows = (torch.arange(R) + first) % 8
        n = min(R, 8)
        for t in tok:
            o, status = run(x.cuda()[rows.cuda()], t[rows].cuda(), K)
            assert status == 0
            compare({k: v[:n] for k, v in o.items()}, x[rows[:n]], t[rows[:n]], K)
            for k, v in o.items():
                assert torch.equal(v, v[torch.arange(R, device="cuda") % n]), k


@pytest.mark.gpu
@pytest.mark.parametrize("V,R", [(100, 3), (9001, 3), (131072, 2)])
def test_masked_rows(V, R):
    x, tok = make(R, V, V)
    x[0, : V // 2] = -math.inf
    x[1] = -math.inf
    x[1, 5] = 2.0
    x[-1, 10:] = -math.inf
    o = check(x, tok, 20)
    assert torch.isfinite(o["entropy"]).all()
    x[:] = -math.inf
    check(x, tok, 20)


@pytest.mark.gpu
@pytest.mark.parametrize("V", [50, 70000])
def test_values_that_are_no_numbers(V):
    x, tok = make(4, V, V)
    x[0, 3] = math.nan
    x[1, 40] = math.inf
    x[2] = math.nan
    x[2, 7:9] = torch.tensor([1.0, 2.0])
    o, status = run(x, tok, 20)
    assert status == 0
    assert torch.isnan(o["logprobs"][:3]).all() and torch.isnan(o["entropy"][:3]).all() and torch.isfinite(o["logprobs"][3])
    assert o["top_ids"][1, 0] == 40 and 3 not in o["top_ids"][0].tolist()
    want = [i for i in np.argsort(-np.nan_to_num(x[0].cpu().numpy(), nan=-1e9), kind="stable")[:20]]
    assert o["top_ids"][0].tolist() == want
    assert o["top_ids"][2].tolist() == [8, 7] + [-1] * 18
    assert torch.isnan(o["top_logprobs"][2]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("low", ["lowest", "-inf"])
def test_rows_of_masks_and_large_values(dtype, low):
    """Masks of the type's lowest value or -inf, alone, beside each other, and beside logits of any size; tokens among them."""
    V = 9001
    lo = torch.finfo(dtype).min if low == "lowest" else -math.inf
    g = torch.Generator().manual_seed(5)
    x = (torch.randn(9, V, generator=g) * 3).to(dtype).cuda()
    x[0] = lo
    x[1, 100:] = lo
    x[2, : V - 7] = lo
    x[3] = torch.finfo(dtype).min
    x[3, ::3] = lo
    x[4] = x[4] * 1e4
    x[5] = x[5] - 3e4
    x[6, 1:] = x[6, 1:] * 1e30
    x[7, ::2] = lo
    x[7, 1::2] = x[7, 1::2] * 2.0 ** 100
    x[8] = torch.finfo(dtype).max * torch.linspace(-1, 1, V).to(dtype).cuda()
    for tok in (0, 99, 4500, V - 1):
        o, _ = run(x, torch.full((9,), tok, device="cuda"), 20)
        rows = [r for r in range(9) if torch.isfinite(x[r].double()).any()]
        # exponentials of differences that fp32 holds: row 8's are as far apart as its type's numbers
        compare({k: v[rows] for k, v in o.items()}, x[rows], torch.full((len(rows),), tok), 20)


@pytest.mark.gpu
def test_bad_tokens_strides_and_optional_outputs():
    x, tok = make(5, 3000, 1)
    tok[1], tok[3] = 3000, -5
    o, status = run(x, tok, 6)
    assert status == fd.FD_DEVSTAT_BAD_TOKEN
    assert o["logprobs"][[1, 3]].tolist() == [0, 0] and o["ranks"][[1, 3]].tolist() == [-1, -1]
    tok = tok.clamp(0, 2999)
    wide_ids, wide_lp = torch.full((5, 11), 777, dtype=I32, device="cuda"), torch.full((5, 13), 777.0, device="cuda")
    big = torch.empty(5, 9000, device="cuda")
    big[:, 17:3017] = x
    every = torch.stack([tok, tok + 1], 1)
    out = dict(logprobs=torch.empty(5, device="cuda"), ranks=torch.empty(5, dtype=I32, device="cuda"),
               entropy=torch.empty(5, device="cuda"), top_ids=wide_ids[:, 2:8], top_logprobs=wide_lp[:, 3:9])
    check(big[:, 17:3017], every[:, 0], 6, out)
    assert (wide_ids[:, :2] == 777).all() and (wide_ids[:, 8:] == 777).all() and (wide_lp[:, :3] == 777).all() and (wide_lp[:, 9:] == 777).all()
    lp = torch.empty(5, device="cuda")
    fd.fd_token_logprobs(big[:, 17:3017], tok, lp)      # (the same place: the order of a sum goes by 16-byte pieces)
    assert torch.equal(lp, out["logprobs"])
    check(x[:1].expand(5, 3000), tok, 6)          # one row for all tokens


def own_bound(V, spread):
    """Bounds on the errors of ln l and of w / l: an exponential of z = x - base is off by 2^-22 (two places) and by the rounding of z and
    of its product with log2(e), 3 |z| 2^-24 together, |z| below the row's spread. A sum is rescaled for its rises by more than
    40 (none in a row that is no wider), for the CTA's maximum and the cluster's: 2 factors more that are off by as much. A thread adds no more
    than 530 values in a row (1024 and a turn of its loop, half of them in each sum of a pair), then up to V / 131072 such sums and 12 more on
    the way to the row's: 2^-24 each (fewer where it has fewer)."""
    adds = min(530, V / 64 + 2) + V / 131072 + 12
    return 3 * (2.0 ** -22 + 3 * spread * 2.0 ** -24) + adds * 2.0 ** -24


def check_closely(logits, tokens, rows):
    """Log probability and entropy of the given rows within the bound above, which a lost or doubled piece of a row exceeds."""
    o, status = run(logits, tokens, 0)
    assert status == 0
    for r in rows:
        x, t = logits[r].double().cpu(), int(tokens[r])
        z = x - x.max()
        e = z.exp()
        l, V = e.sum(), x.numel()
        d, mean = own_bound(V, float(-z.min())), float(-(e * z).sum() / l)
        lp, entropy = float(z[t] - l.log()), float(l.log()) + mean
        assert abs(float(o["logprobs"][r]) - lp) <= d + 2.0 ** -22 * (1 + abs(lp)), (r, float(o["logprobs"][r]), lp, d)
        # w is off as l is, by at most the spread for a value relative to another maximum
        assert abs(float(o["entropy"][r]) - entropy) <= d * (2 + 2 * mean) + 2.0 ** -22 * (1 + entropy + mean), (r, entropy, d)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("R,V", [(3, 2003), (1, 50021), (2, 131072), (700, 9001), (700, 50021), (1000, 9001), (1000, 20011), (1000, 131072),
                                 (2500, 2003)])
def test_sums_within_their_own_bound(dtype, R, V):
    """Rows of every number of threads and CTAs, with values within 20 of each other."""
    x, tok = make(8, V, V + R, dtype, pad=V % 5, scale=2.0)
    x = x.clamp(-9, 9)
    many = x[torch.arange(R, device="cuda") % 8] if R > 8 else x[:R]
    check_closely(many, tok[torch.arange(R, device="cuda") % 8], range(min(R, 8)))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("R,V", [(900, 1 << 24), (900, (1 << 24) - 5), (400, 1 << 24), (1, 1 << 24), (900, 3000017)])
def test_long_rows_in_a_batch(dtype, R, V):
    """The longest rows where each has a single CTA: 2^17 equal exponentials a thread, which one running sum would all round the same way."""
    x = torch.full((4, V), -0.3, device="cuda")
    x[:, :8192] = 0.0
    x[1, 8192:] = -0.7
    x[2, 8192:] = -0.2 - torch.rand(V - 8192, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    x[3, : V // 2] = -50.0                          # (a rise after sums were folded)
    x = x.to(dtype)
    tok = torch.full((R,), -1, dtype=I64, device="cuda")
    for r in range(4):
        tok[r * (R - 1) // 3] = V - 77
        check_closely(x[r:r + 1].expand(R, V), tok, [r * (R - 1) // 3])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("R,V,K", [(900, 140003, 20), (320, 270001, 5), (1, 2200003, 32)])
def test_long_rows_with_masks_and_low_logits(dtype, R, V, K):
    """Rows on 128 and 256 threads and on 8 CTAs that are long enough for sums to be folded: all outputs."""
    test_ranks_among_low_logits_behind_masks(dtype, R, V, K)


@pytest.mark.gpu
def test_far_rows():
    V = 131072
    x = torch.zeros(17000, V, dtype=BF, device="cuda")          # 2.2e9 values
    tok = torch.full((17000,), -1, device="cuda")
    g = torch.Generator().manual_seed(2)
    rows = [0, 16383, 16384, 16999]
    x[rows] = (torch.randn(4, V, generator=g) * 3).to(BF).cuda()
    tok[rows] = torch.tensor([5, 6, 7, V - 1]).cuda()
    o, _ = run(x, tok, 5)
    compare({k: v[rows] for k, v in o.items()}, x[rows], tok[rows], 5)
    assert (o["ranks"] >= 0).nonzero()[:, 0].tolist() == rows


@pytest.mark.gpu
def test_in_a_graph_and_on_two_streams():
    x, tok = make(3, 60000, 3)
    y, tok2 = make(400, 5000, 4, BF)
    want, want2 = check(x, tok, 20), check(y, tok2, 5)
    o = {k: torch.zeros_like(v) for k, v in want.items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fd.fd_token_logprobs(x, tok, **o)
    graph.replay()
    assert all(torch.equal(o[k], want[k]) for k in o)
    x2, t2 = make(3, 60000, 5)
    x.copy_(x2)
    tok.copy_(t2)
    graph.replay()
    again = check(x2, t2, 20)
    assert all(torch.equal(o[k], again[k]) for k in o)
    torch.cuda.synchronize()
    s = [torch.cuda.Stream() for _ in range(2)]
    outs = [[{k: torch.zeros_like(v) for k, v in w.items()} for _ in range(10)] for w in (again, want2)]
    for i in range(10):
        fd.fd_token_logprobs(x, tok, **outs[0][i], stream=s[0])
        fd.fd_token_logprobs(y, tok2, **outs[1][i], stream=s[1])
    torch.cuda.synchronize()
    for w, os in zip((again, want2), outs):
        assert all(torch.equal(o[k], w[k]) for o in os for k in o)
