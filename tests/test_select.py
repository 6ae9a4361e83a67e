"""Page selection: the oracle's pins and the refusals (CPU), the kernel against the
oracle (GPU; whole numbers, so equality)."""
import math

import numpy as np
import pytest
import torch

import split_kv_paged_gqa_gb300 as fd
from oracle.step_ref import page_scores_ref, select_ref

BF, F32, I32, I64 = torch.bfloat16, torch.float32, torch.int32, torch.int64


def test_oracle_score_bounds_every_key():
    r = np.random.default_rng(0)
    keys, q = r.standard_normal((7, 20, 64)), r.standard_normal((3, 64))
    score = page_scores_ref(q, keys.min(1), keys.max(1))
    best = (keys @ q.T).max(1).sum(-1)
    assert (score >= best).all()
    one = page_scores_ref(q, keys[:, 0], keys[:, 0])      # bounds of a single key: its scores
    np.testing.assert_allclose(one, (keys[:, 0] @ q.T).sum(-1), rtol=1e-12)


def test_oracle_choice():
    bounds = np.zeros((6, 1, 2, 1))
    bounds[:, 0, 1, 0] = [1.0, 5.0, 3.0, 5.0, 2.0, 0.0]
    q = np.ones((1, 1, 1, 1))
    args = (q, bounds, np.arange(6)[None], [48], 8)
    assert select_ref(*args, 3, 0, 1)[0, 0, 0].tolist() == [1, 3, 5]
    assert select_ref(*args, 2, 0, 1)[0, 0, 0].tolist() == [1, 5]
    assert select_ref(*args, 4, 1, 2)[0, 0, 0].tolist() == [0, 1, 4, 5]
    assert select_ref(*args, 7, 1, 2)[0, 0, 0].tolist() == [0, 1, 2, 3, 4, 5, -1]
    assert select_ref(q, bounds, np.arange(6)[None], [17], 8, 2, 0, 1)[0, 0, 0].tolist() == [1, 2]


def _args(B=2, Tq=1, Hq=4, Hkv=2, D=128, N=9, W=6, S=4):
    return dict(q=torch.zeros(B, Tq, Hq, D, dtype=BF), page_bounds=torch.zeros(N, Hkv, 2, D, dtype=BF),
                page_table=torch.zeros(B, W, dtype=I32), cache_seqlens=torch.zeros(B, dtype=I32), q_per_req=Tq, page_size=16,
                num_first=1, num_last=1, selected=torch.zeros(B, Tq, Hkv, S, dtype=I32))


@pytest.mark.parametrize("change,status", [
    (dict(q=torch.zeros(2, 1, 4, 128)), fd.FD_ERR_INVALID_ARG),
    (dict(q=None), fd.FD_ERR_INVALID_ARG),
    (dict(q=torch.zeros(2, 1, 5, 128, dtype=BF)), fd.FD_ERR_INVALID_ARG),
    (dict(q=torch.zeros(2, 1, 4, 64, dtype=BF)), fd.FD_ERR_INVALID_ARG),
    (dict(q=torch.zeros(2, 2, 4, 128, dtype=BF)), fd.FD_ERR_INVALID_ARG),
    (dict(q=torch.zeros(2 * 4 * 132, dtype=BF)[4:4 + 2 * 4 * 128].view(2, 1, 4, 128)), fd.FD_ERR_UNSUPPORTED),
    (dict(page_bounds=torch.zeros(9, 2, 128, dtype=BF)), fd.FD_ERR_INVALID_ARG),
    (dict(page_bounds=torch.zeros(9, 2, 2, 128)), fd.FD_ERR_INVALID_ARG),
    (dict(page_bounds=torch.zeros(9, 2, 3, 128, dtype=BF)), fd.FD_ERR_INVALID_ARG),
    (dict(page_bounds=torch.zeros(9, 2, 2, 129, dtype=BF)[..., :128]), fd.FD_ERR_UNSUPPORTED),
    (dict(page_table=torch.zeros(3, 6, dtype=I32)), fd.FD_ERR_INVALID_ARG),
    (dict(page_table=torch.zeros(2, 6, dtype=I64)), fd.FD_ERR_INVALID_ARG),
    (dict(page_table=torch.zeros(2, 15361, dtype=I32)), fd.FD_ERR_UNSUPPORTED),
    (dict(cache_seqlens=torch.zeros(2, dtype=I64)), fd.FD_ERR_INVALID_ARG),
    (dict(page_size=24), fd.FD_ERR_UNSUPPORTED),
    (dict(page_size=4), fd.FD_ERR_UNSUPPORTED),
    (dict(num_first=-1), fd.FD_ERR_INVALID_ARG),
    (dict(num_last=0), fd.FD_ERR_INVALID_ARG),
    (dict(num_first=3, num_last=2), fd.FD_ERR_INVALID_ARG),
    (dict(num_first=2 ** 31 - 1, num_last=2 ** 31 - 1), fd.FD_ERR_INVALID_ARG),
    (dict(selected=torch.zeros(2, 1, 2, 4, dtype=I64)), fd.FD_ERR_INVALID_ARG),
    (dict(selected=torch.zeros(2, 1, 1, 4, dtype=I32)), fd.FD_ERR_INVALID_ARG),
    (dict(selected=torch.zeros(2, 1, 1, 4, dtype=I32).expand(2, 1, 2, 4)), fd.FD_ERR_UNSUPPORTED),
    (dict(selected=torch.zeros(2, 1, 2, 8, dtype=I32)[..., ::2]), fd.FD_ERR_UNSUPPORTED),
    (dict(status=torch.zeros(2, dtype=I64)), fd.FD_ERR_INVALID_ARG),
])
def test_rejects(change, status):
    with pytest.raises(fd.FdError) as e:
        fd.fd_select_pages(**{**_args(), **change}, stream=0)
    assert e.value.status == status, str(e.value)


def make(lens, Tq, Hq, Hkv, D, P, seed, spread=0.5, W=None):
    g = torch.Generator().manual_seed(seed)
    pages = [-(-n // P) for n in lens]
    N, W = sum(pages) + 2, W or max(1, max(pages))
    mid = torch.randn(N, Hkv, D, generator=g) * 0.7
    half = torch.randn(N, Hkv, D, generator=g).abs() * spread + 1.0
    perm = torch.randperm(N, generator=g).to(I32)
    table, at = torch.full((len(lens), W), -1, dtype=I32), 0
    for b, n in enumerate(pages):
        table[b, :n] = perm[at:at + n]
        at += n
    return dict(q=torch.randn(len(lens), Tq, Hq, D, generator=g).to(BF).cuda(),
                page_bounds=torch.stack([mid - half, mid + half], 2).to(BF).cuda(), page_table=table.cuda(),
                cache_seqlens=torch.tensor(lens, dtype=I32).cuda(), q_per_req=Tq, page_size=P)


def run(a, S, first, last, status=0):
    B, Tq, _, _ = a["q"].shape
    guard = torch.full((B, Tq, a["page_bounds"].shape[1], S + 5), 777, dtype=I32, device="cuda")
    out, st = guard[..., 2:2 + S], torch.zeros(1, dtype=I32, device="cuda")
    fd.fd_select_pages(**a, num_first=first, num_last=last, selected=out, status=st)
    assert int(st) == status
    assert (guard[..., :2] == 777).all() and (guard[..., 2 + S:] == 777).all()
    return out


def check(a, S, first, last, status=0):
    out = run(a, S, first, last, status)
    f = lambda t: t.double().cpu().numpy()   # noqa: E731
    want = select_ref(f(a["q"]), f(a["page_bounds"]), a["page_table"].cpu().numpy(), a["cache_seqlens"].tolist(), a["page_size"],
                      S, first, last)
    assert np.array_equal(out.cpu().numpy(), want)
    return out


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Tq", [1, 3])
@pytest.mark.parametrize("P", [8, 64])
def test_lengths(D, Tq, P):
    a = make([0, 1, 2, P - 1, P, P + 1, 3 * P, 9 * P + 1, 40 * P - 3, 130 * P + 2], Tq, 8, 2, D, P, D + Tq + P)
    for S, first, last in ((1, 0, 1), (3, 1, 1), (3, 1, 2), (9, 2, 3), (41, 0, 1), (131, 1, 4)):
        check(a, S, first, last)


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (5, 1), (64, 8), (40, 8), (128, 2), (16, 16)])
def test_heads(Hq, Hkv):
    check(make([3000, 1500, 700], 2, Hq, Hkv, 128, 16, Hq), 20, 1, 2)


@pytest.mark.gpu
@pytest.mark.parametrize("B,L,P,S", [(1, 32768, 16, 128), (1, 32768, 8, 1000), (2, 20000, 16, 64), (30, 4096, 16, 33), (70, 2048, 16, 16)])
def test_batches(B, L, P, S):
    r = np.random.default_rng(B)
    check(make([L] + [int(x) for x in r.integers(L // 2, L, B - 1)], 1, 16, 4, 128, P, B), S, 1, 4)


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("B,W", [(1, 520), (77, 300), (77, 1600), (39, 3000), (40, 4000), (20, 4000), (39, 8200), (12, 9000)])
def test_tables_of_any_width(B, W, D):
    r = np.random.default_rng(W)
    most = 8 * min(W, 400)
    check(make([int(x) for x in r.integers(1, most, B - 1)] + [most], 1, 8, 8 if B != 77 else 4, D, 8, W, W=W), 40, 1, 2)


@pytest.mark.gpu
def test_widest_table():
    check(make([15360 * 8, 15360 * 8 - 77], 1, 2, 1, 64, 8, 3, W=15360), 200, 1, 1)


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
def test_equal_pages(D):
    """Pages with the same bounds score the same: the lowest are chosen."""
    a = make([4000, 2999], 2, 8, 2, D, 16, D)
    N = a["page_bounds"].shape[0]
    a["page_bounds"].copy_(a["page_bounds"][torch.arange(N, device="cuda") % 3])
    for S in (5, 60, 130):
        check(a, S, 1, 1)
    a["page_bounds"].copy_(a["page_bounds"][:1].expand_as(a["page_bounds"]))
    check(a, 40, 0, 1)
    a["page_bounds"].zero_()
    check(a, 40, 0, 1)
    check(a, 40, 38, 2)


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
def test_pages_of_no_request_do_not_matter(D):
    """Page 0 is in no table and holds what it holds: the choice is the same, and takes as long, whatever that is."""
    a = make([32760 - 16 * 5], 1, 16, 4, D, 16, 9)
    bounds, table = a["page_bounds"], a["page_table"]
    bounds.copy_(bounds.roll(1, 0))
    table += 1                                      # (the pool has two pages more than the table)
    table[table == bounds.shape[0]] = int(bounds.shape[0]) - 1
    used = torch.unique(table)
    assert int(used.min()) >= 1 and int(used.max()) < bounds.shape[0]

    def time_of(value):
        bounds[0] = value
        out = run(a, 128, 1, 4)
        assert torch.equal(out, check(a, 128, 1, 4))
        best = math.inf
        for _ in range(5):
            start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            start.record()
            for _ in range(20):
                fd.fd_select_pages(**a, num_first=1, num_last=4, selected=out)
            end.record()
            torch.cuda.synchronize()
            best = min(best, start.elapsed_time(end))
        return out.clone(), best

    want, usual = time_of(0.0)
    for value in (math.inf, 3e38, math.nan):
        got, took = time_of(value)
        assert torch.equal(got, want)
        assert took < 5 * usual, (value, took, usual)  # (all pages in fp64: 40 times)


@pytest.mark.gpu
@pytest.mark.parametrize("B,D", [(1, 128), (2, 64), (160, 64)])
def test_many_pages_on_the_border(B, D):
    """More equal pages, or pages past fp32, than are ranked one against the other."""
    a = make([14000] + [9000] * (B - 1), 1, 8, 2, D, 8, B)
    b, ids = a["page_bounds"], a["page_table"].long()
    b.copy_(b[torch.arange(b.shape[0], device="cuda") % 2])
    check(a, 300, 1, 1)
    check(a, 1000, 1, 1)
    b.zero_()
    check(a, 300, 1, 1)
    b[ids[0, 1700], 0, 0, 5] = -1.0
    check(a, 300, 1, 1)
    a["q"].zero_()
    check(a, 300, 1, 1)
    a = make([14000] + [9000] * (B - 1), 1, 8, 2, D, 8, B + 1)
    for scale in (2.0 ** -100, 2.0 ** 105):
        c = dict(a, page_bounds=(a["page_bounds"].float() * scale).to(BF))
        check(c, 300, 1, 1)
        c["page_bounds"].copy_(c["page_bounds"][torch.arange(b.shape[0], device="cuda") % 5])
        check(c, 300, 1, 1)
    a["page_bounds"][ids[0, 7], :, 1, 3] = math.inf
    a["page_bounds"][ids[0, 90], 0, 0, 3] = math.nan
    check(a, 300, 1, 1)
    a["page_table"][0, 40:1400] = -1
    check(a, 800, 1, 1, status=fd.FD_DEVSTAT_BAD_PAGE)


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
def test_nearly_equal_pages(D):
    """Scores that differ by less than an fp32 sum can tell: the order is the exact one."""
    a = make([6000], 1, 8, 2, D, 8, 5)
    b = a["page_bounds"]
    b.copy_(b[:1].expand_as(b))
    g = torch.Generator().manual_seed(6)
    b[:, :, :, 0] = 512.0
    n = b.shape[0]
    # small channels that vary from page to page, beside large ones that cancel
    b[:, :, 0, 1] = b[:, :, 1, 1] = -512.0
    a["q"][..., 0] = 8.0
    a["q"][..., 1] = 8.0
    tiny = (torch.randn(n, 2, 1, 3, generator=g) * 2.0 ** -12).to(BF).cuda()
    b[..., 5:8] = tiny
    for S in (10, 300):
        check(a, S, 1, 1)


@pytest.mark.gpu
def test_outlier_channels_and_magnitudes():
    a = make([5000, 3000], 1, 8, 2, 128, 16, 7)
    a["page_bounds"][..., 3] *= 40
    a["q"][..., 9] *= 100
    check(a, 30, 1, 2)
    for scale in (2.0 ** -60, 2.0 ** -85, 2.0 ** -110, 2.0 ** 50, 2.0 ** 100):
        c = dict(a, page_bounds=(a["page_bounds"].float() * scale).to(BF))
        check(c, 30, 1, 2)
    c = dict(a, page_bounds=(a["page_bounds"].float() * 2.0 ** -90).to(BF), q=(a["q"].float() * 2.0 ** -80).to(BF))   # products fp32 cannot hold
    check(c, 30, 1, 2)
    c = dict(a, page_bounds=(a["page_bounds"].float() * 2.0 ** 100).to(BF), q=(a["q"].float() * 2.0 ** 30).to(BF))   # sums past fp32
    check(c, 30, 1, 2)


@pytest.mark.gpu
def test_skewed_scores():
    """A few scores far above the rest, and exponentially spaced ones."""
    a = make([16000], 1, 4, 1, 128, 8, 8)
    n = a["page_bounds"].shape[0]
    a["page_bounds"].copy_((a["page_bounds"].float() * torch.exp2(torch.arange(n) % 90 - 60.0).cuda()[:, None, None, None]).to(BF))
    for S in (3, 50, 900, 1990):
        check(a, S, 1, 1)


@pytest.mark.gpu
def test_values_that_are_no_numbers():
    a = make([3000, 3000], 1, 4, 2, 128, 16, 9)
    ids = a["page_table"].long()
    b = a["page_bounds"]
    b[ids[0, 50], 0, :, 7] = math.nan
    b[ids[0, 120], 1, 1, 9] = math.nan
    out = check(a, 20, 1, 1)
    assert 50 in out[0, 0, 0].tolist() and 120 in out[0, 0, 1].tolist()
    for i in range(20, 60):
        b[ids[1, i], 0, 0, 3] = math.nan
    check(a, 20, 1, 1)                        # more of them than are chosen
    b.nan_to_num_(0.0)
    b[ids[0, 70], 0, 1, 5] = math.inf
    b[ids[0, 71], 0, 0, 6] = -math.inf
    check(a, 20, 1, 1)
    b[ids[0, 70], 0, 1, 5] = b[ids[0, 71], 0, 0, 6] = 0.0
    a["q"][0, 0, 1, 5] = math.nan             # every score of the head is NaN
    check(a, 20, 1, 1)
    a["q"][0, 0, 1, 5] = math.inf             # +inf, or NaN where the bound is 0
    a["page_bounds"][ids[0, 30], 0, 1, 5] = 0.0
    check(a, 20, 1, 1)
    a["q"][0, 0, :, 5] = 3e38                 # heads whose sum no fp32 number holds
    a["page_bounds"].mul_(2.0 ** -30)
    check(a, 20, 1, 1)


@pytest.mark.gpu
def test_bad_metadata():
    a = make([3000, 3000, 100], 1, 4, 2, 128, 16, 10)
    a["page_table"][0, 30] = 10 ** 6
    a["page_table"][0, 31] = -1
    a["page_table"][0, 33] = -2 ** 31
    check(a, 20, 1, 1, status=fd.FD_DEVSTAT_BAD_PAGE)
    check(a, 184, 1, 1, status=fd.FD_DEVSTAT_BAD_PAGE)
    check(a, 186, 1, 1, status=fd.FD_DEVSTAT_BAD_PAGE)
    a["page_table"][1, 20:150] = -5
    check(a, 150, 1, 1, status=fd.FD_DEVSTAT_BAD_PAGE)
    a = make([3000, 3000, 100], 1, 4, 2, 128, 16, 11)
    a["cache_seqlens"][1:] = torch.tensor([-4, 10 ** 9])
    a["page_table"][2] = a["page_table"][0]
    check(a, 20, 1, 1, status=fd.FD_DEVSTAT_SEQLEN_OVERFLOW)


@pytest.mark.gpu
def test_strides_streams_and_graphs():
    a = make([3000, 500, 2000], 2, 8, 2, 64, 16, 12)
    want = check(a, 25, 1, 2)
    wide_q = torch.randn(3, 2, 3, 8, 72, device="cuda").to(BF)
    wide_q[:, :, 1, :, :64] = a["q"]
    nb = a["page_bounds"].shape[0]
    bounds = torch.zeros(2, 2, nb + 1, 80, dtype=BF, device="cuda")
    bounds[:, :, 1:, :64] = a["page_bounds"].permute(2, 1, 0, 3)
    c = dict(a, q=wide_q[:, :, 1, :, :64], page_bounds=bounds[:, :, 1:, :64].permute(2, 1, 0, 3),
             page_table=torch.nn.functional.pad(a["page_table"], (0, 9), value=99)[:, :-9],
             cache_seqlens=a["cache_seqlens"].repeat_interleave(3)[::3])
    assert torch.equal(run(c, 25, 1, 2), want)
    out = torch.zeros(3, 2, 2, 25, dtype=I32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fd.fd_select_pages(**a, num_first=1, num_last=2, selected=out)
    graph.replay()
    assert torch.equal(out, want)
    a["q"].copy_(a["q"].flip(0))
    a["cache_seqlens"].copy_(torch.tensor([2999, 480, 1990], dtype=I32))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, check(a, 25, 1, 2))
    long = make([32768], 1, 64, 8, 128, 16, 13)
    want = [run(a, 25, 1, 2).clone(), run(long, 128, 1, 4).clone()]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [[torch.zeros_like(w) for _ in range(10)] for w in want]
    for i in range(10):
        fd.fd_select_pages(**a, num_first=1, num_last=2, selected=outs[0][i], stream=streams[0])
        fd.fd_select_pages(**long, num_first=1, num_last=4, selected=outs[1][i], stream=streams[1])
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for w, os in zip(want, outs) for o in os)
