"""Attention over selected pages: the oracle's pins and the refusals (CPU), the kernel
against the oracle (GPU)."""
import math

import numpy as np
import pytest
import torch

import split_kv_paged_gqa_gb300 as fd
from oracle.step_ref import sparse_ref
from tests.test_append import cache_values

BF, F32, I32, I64 = torch.bfloat16, torch.float32, torch.int32, torch.int64
KINDS = ["bf16", "int8", "int4"]


def f64(t):
    return t.detach().double().cpu().numpy()


def test_oracle_of_all_pages_is_dense_attention():
    r = np.random.default_rng(0)
    q, k, v = r.standard_normal((1, 2, 4, 64)), r.standard_normal((7, 8, 2, 64)), r.standard_normal((7, 8, 2, 64))
    table = np.array([[3, 0, 6, 1]])
    every = np.broadcast_to(np.array([2, 0, -1, 1, 3]), (1, 2, 2, 5))      # in any order
    out, lse, _, _ = sparse_ref(q, k, v, table, [27], every, 8, 0.125)
    for t in range(2):
        n = 26 + t
        kk, vv = k[table[0]].reshape(32, 2, 64)[:n], v[table[0]].reshape(32, 2, 64)[:n]
        for h in range(4):
            z = 0.125 * kk[:, h // 2] @ q[0, t, h]
            p = np.exp(z - z.max())
            np.testing.assert_allclose(out[0, t, h], p @ vv[:, h // 2] / p.sum(), rtol=1e-12)
            assert lse[0, t, h] == pytest.approx(np.log(p.sum()) + z.max())
    out, lse, _, _ = sparse_ref(q, k, v, table, [27], np.full((1, 2, 2, 3), -1), 8, 0.125)
    assert (out == 0).all() and np.isneginf(lse).all()


def _args(kind="bf16", B=2, Tq=1, Hq=4, Hkv=2, D=128, N=9, P=16, W=6, S=4):
    row = D // 2 if kind == "int4" else D
    dt = dict(bf16=BF, int8=torch.int8, int4=torch.uint8)[kind]
    return dict(q=torch.zeros(B, Tq, Hq, D, dtype=BF), k_cache=torch.zeros(N, P, Hkv, row, dtype=dt),
                v_cache=torch.zeros(N, P, Hkv, row, dtype=dt),
                kv_scales=None if kind == "bf16" else torch.zeros(2, N, P, Hkv, 1 if kind == "int8" else D // 32),
                page_table=torch.zeros(B, W, dtype=I32), cache_seqlens=torch.zeros(B, dtype=I32),
                selected=torch.zeros(B, Tq, Hkv, S, dtype=I32), q_per_req=Tq, softmax_scale=0.0,
                out=torch.zeros(B, Tq, Hq, D, dtype=BF), lse=torch.zeros(B, Tq, Hq))


@pytest.mark.parametrize("kind,change,status", [
    ("bf16", dict(q=torch.zeros(2, 1, 4, 128)), fd.FD_ERR_INVALID_ARG),
    ("bf16", dict(q=torch.zeros(2, 1, 3, 128, dtype=BF)), fd.FD_ERR_INVALID_ARG),
    ("bf16", dict(q=None), fd.FD_ERR_INVALID_ARG),
    ("bf16", dict(q=torch.zeros(2, 1, 4, 96, dtype=BF)), fd.FD_ERR_UNSUPPORTED),
    ("bf16", dict(q_per_req=2), fd.FD_ERR_INVALID_ARG),
    ("bf16", dict(k_cache=torch.zeros(9, 16, 2, 64, dtype=BF)), fd.FD_ERR_INVALID_ARG),
    ("bf16", dict(k_cache=torch.zeros(9, 16, 2, 136, dtype=BF)[..., :128]), fd.FD_ERR_UNSUPPORTED),   # strides differ
    ("bf16", dict(v_cache=torch.zeros(9, 16, 2, 128, dtype=torch.int8)), fd.FD_ERR_INVALID_ARG),
    ("bf16", dict(k_cache=torch.zeros(9, 512, 2, 128, dtype=BF), v_cache=torch.zeros(9, 512, 2, 128, dtype=BF)), fd.FD_ERR_UNSUPPORTED),
    ("bf16", dict(kv_scales=torch.zeros(2, 9, 16, 2, 1)), fd.FD_ERR_INVALID_ARG),
    ("int8", dict(kv_scales=None), fd.FD_ERR_INVALID_ARG),
    ("int4", dict(kv_scales=torch.zeros(2, 9, 16, 2, 1)), fd.FD_ERR_INVALID_ARG),
    ("bf16", dict(page_table=torch.zeros(3, 6, dtype=I32)), fd.FD_ERR_INVALID_ARG),
    ("bf16", dict(page_table=torch.zeros(2, 12, dtype=I32)[:, ::2]), fd.FD_ERR_UNSUPPORTED),
    ("bf16", dict(cache_seqlens=torch.zeros(3, dtype=I32)), fd.FD_ERR_INVALID_ARG),
    ("bf16", dict(selected=torch.zeros(2, 1, 4, 4, dtype=I32)), fd.FD_ERR_INVALID_ARG),
    ("bf16", dict(selected=torch.zeros(2, 1, 2, 4, dtype=I64)), fd.FD_ERR_INVALID_ARG),
    ("bf16", dict(selected=torch.zeros(2, 1, 2, 8, dtype=I32)[..., ::2]), fd.FD_ERR_UNSUPPORTED),
    ("bf16", dict(softmax_scale=-1.0), fd.FD_ERR_INVALID_ARG),
    ("bf16", dict(softmax_scale=math.nan), fd.FD_ERR_INVALID_ARG),
    ("bf16", dict(softmax_scale=math.inf), fd.FD_ERR_INVALID_ARG),
    ("bf16", dict(out=torch.zeros(2, 1, 4, 128, dtype=torch.float16)), fd.FD_ERR_INVALID_ARG),
    ("bf16", dict(out=torch.zeros(2, 1, 4, 64, dtype=BF)), fd.FD_ERR_INVALID_ARG),
    ("bf16", dict(out=torch.zeros(2, 1, 1, 128, dtype=BF).expand(2, 1, 4, 128)), fd.FD_ERR_UNSUPPORTED),
    ("bf16", dict(out=torch.zeros(2, 1, 4, 129)[..., :128]), fd.FD_ERR_UNSUPPORTED),
    ("bf16", dict(lse=torch.zeros(2, 1, 3)), fd.FD_ERR_INVALID_ARG),
    ("bf16", dict(lse=torch.zeros(2, 1, 1).expand(2, 1, 4)), fd.FD_ERR_UNSUPPORTED),
    ("bf16", dict(status=torch.zeros(1)), fd.FD_ERR_INVALID_ARG),
])
def test_rejects(kind, change, status):
    with pytest.raises(fd.FdError) as e:
        fd.fd_decode_sparse(**{**_args(kind), **change}, stream=0)
    assert e.value.status == status, str(e.value)


def make(lens, Tq, Hq, Hkv, D, P, S, seed, kind="bf16", strided=False, poison=True, drop=0.2):
    """A batch on scattered pages; random lists, -1 among them; cache slots past the lengths hold NaN."""
    g = torch.Generator().manual_seed(seed)
    B = len(lens)
    pages = [-(-n // P) for n in lens]
    N, W = sum(pages) + 2, max(1, max(pages))
    perm = torch.randperm(N, generator=g).to(I32)
    table, at = torch.full((B, W), -1, dtype=I32), 0
    row = D // 2 if kind == "int4" else D
    shape = (N, Hkv, P, row) if strided else (N, P, Hkv, row)
    caches, scales = [], None
    for _ in range(2):
        if kind == "bf16":
            x = torch.randn(shape, generator=g).to(BF)
        elif kind == "int8":
            x = torch.randint(-127, 128, shape, generator=g).to(torch.int8)
        else:
            x = torch.randint(0, 256, shape, generator=g).to(torch.uint8)
        caches.append(x.transpose(1, 2) if strided else x)
    if kind != "bf16":
        ng = 1 if kind == "int8" else D // 32
        scales = (torch.rand(2, N, Hkv, P, ng, generator=g) + 0.5) * (0.014 if kind == "int8" else 0.22)
        scales = scales.transpose(2, 3)
    live = torch.zeros(N, P, dtype=torch.bool)
    for b, n in enumerate(pages):
        table[b, :n] = perm[at:at + n]
        at += n
        for j in range(n):
            live[table[b, j].long(), :max(0, min(P, lens[b] - j * P))] = True
    if poison:
        for i, c in enumerate(caches):
            if kind == "bf16":
                c[~live] = math.nan
            else:
                scales[i][~live] = math.nan
    sel = torch.full((B, Tq, Hkv, S), -1, dtype=I32)
    for b, n in enumerate(pages):
        for t in range(Tq):
            for h in range(Hkv):
                k = min(S, n)
                pick = torch.randperm(n, generator=g)[:k]
                if n:
                    pick[0] = n - 1 if n - 1 not in pick.tolist() else pick[0]
                pick = torch.where(torch.rand(k, generator=g) < drop, -1, pick)
                sel[b, t, h, :k] = pick.to(I32)
    q = torch.randn(B, Tq, Hq, D, generator=g).to(BF)
    if strided:
        wide = torch.zeros(B, Tq + 1, Hq, D + 8, dtype=BF)
        wide[:, :Tq, :, :D] = q
        q = wide.cuda()[:, :Tq, :, :D]
        sel = torch.nn.functional.pad(sel, (1, 4), value=0).cuda()[..., 1:-4]
        table = torch.nn.functional.pad(table, (2, 0), value=7).cuda()[:, 2:]
    return dict(q=q.cuda(), k_cache=caches[0].cuda(), v_cache=caches[1].cuda(), kv_scales=None if scales is None else scales.cuda(),
                page_table=table.cuda(), cache_seqlens=torch.tensor(lens, dtype=I32).cuda(), selected=sel.cuda(), q_per_req=Tq,
                softmax_scale=0.0)


def run(a, out_dtype=BF, status=0, **kw):
    q = a["q"]
    out = torch.full(q.shape, 777.0, dtype=out_dtype, device="cuda")
    lse = torch.full(q.shape[:3], 777.0, device="cuda")
    st = torch.zeros(1, dtype=I32, device="cuda")
    fd.fd_decode_sparse(**a, out=out, lse=lse, status=st, **kw)
    assert int(st) == status
    return out, lse


def compare(a, out, lse, kind, where=""):
    sc = a["kv_scales"]
    kv = [f64(cache_values(a[n], None if sc is None else sc[i], kind)) for i, n in enumerate(("k_cache", "v_cache"))]
    D = a["q"].shape[-1]
    scale = a["softmax_scale"] or 1.0 / math.sqrt(D)
    o, s, tol, ltol = sparse_ref(f64(a["q"]), *kv, a["page_table"].cpu().numpy(), a["cache_seqlens"].tolist(),
                                 a["selected"].cpu().numpy(), a["k_cache"].shape[1], scale, 16 if out.dtype == BF else 32)
    if kind != "bf16":
        # a score's product with the key's scale, and of 4 bits the sum of its groups: one rounding of a product
        # and up to 4 additions more than the bound counts (it counts D + 2 of D products), and a weight's product with
        # its value's scale ahead of the rounding to bf16: 2^-23 of |out|'s mass, within the bound's 2^-21
        tol, ltol = tol * (1 + 8.0 / D), ltol * (1 + 8.0 / D)
    live = np.isfinite(s)
    assert np.array_equal(np.isneginf(f64(lse)), ~live), where
    assert (f64(out)[~live] == 0).all(), where
    err = np.abs(f64(out) - o)
    assert (err <= tol).all(), (where, (err / tol).max())
    assert (np.abs(f64(lse)[live] - s[live]) <= ltol[live]).all(), where


def case(lens, Tq, Hq, Hkv, D, P, S, seed, kind="bf16", out_dtype=BF, **kw):
    a = make(lens, Tq, Hq, Hkv, D, P, S, seed, kind, **kw)
    compare(a, *run(a, out_dtype), kind, (lens, Tq, Hq, Hkv, D, P, S, kind))
    return a


@pytest.mark.gpu
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("P", [8, 16, 32, 256])
def test_lengths(kind, D, P):
    lens = [0, 1, 2, P - 1, P, P + 1, 3 * P - 1, 5 * P + 3]
    case(lens, 1, 8, 2, D, P, 4, P + D, kind)
    case(lens, 3, 6, 3, D, P, 7, P + D + 1, kind)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (5, 1), (8, 8), (64, 8), (40, 8), (16, 1), (17, 1), (128, 2)])
def test_heads(kind, Hq, Hkv):
    case([300, 77], 2, Hq, Hkv, 128, 16, 9, Hq, kind)
    case([300], 1, Hq, Hkv, 64, 32, 5, Hq, kind, out_dtype=F32)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("S", [1, 2, 3, 33, 64, 129, 300, 1500])
def test_list_lengths(kind, S):
    """Lists from one page to more than a look-up of a warp holds, on clusters of every size."""
    case([20000], 1, 4, 1, 128, 16, S, S, kind)
    case([9000], 1, 4, 2, 128, 8, S, S, kind)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("B,Hkv", [(3, 8), (20, 8), (40, 8), (200, 2)])
def test_batches(kind, B, Hkv):
    r = np.random.default_rng(B)
    case([int(x) for x in r.integers(0, 1500, B)], 1, 4 * Hkv, Hkv, 64, 16, 40, B, kind)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("out_dtype", [BF, F32])
def test_strides(kind, out_dtype):
    case([100, 0, 333], 2, 8, 2, 128, 16, 11, 5, kind, out_dtype, strided=True)
    case([100, 0, 333], 2, 8, 2, 64, 8, 11, 6, kind, out_dtype, strided=True)


@pytest.mark.gpu
def test_outputs_into_views():
    a = make([100, 333], 2, 8, 2, 128, 16, 11, 7)
    want = run(a)
    buf = torch.full((8, 2, 2, 144), 777.0, dtype=BF, device="cuda")
    lbuf = torch.full((8, 5, 2, 3), 777.0, device="cuda")
    out, lse = buf[..., 8:136].permute(1, 2, 0, 3), lbuf[:, 1:3, :, 1].permute(2, 1, 0)
    fd.fd_decode_sparse(**a, out=out, lse=lse)
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    assert (buf[..., :8] == 777).all() and (buf[..., 136:] == 777).all()
    assert (lbuf[:, 0] == 777).all() and (lbuf[:, 3:] == 777).all() and (lbuf[..., ::2] == 777).all()
    out = torch.empty_like(want[0])
    fd.fd_decode_sparse(**a, out=out, lse=None)
    assert torch.equal(out, want[0])


@pytest.mark.gpu
@pytest.mark.parametrize("kind", KINDS)
def test_needles(kind):
    """A key that has all the weight, at every slot of the tiles: its value comes out, and no other."""
    for P, n in ((8, 37), (16, 50), (64, 130)):
        a = make([n] * n, 1, 2, 1, 128, P, -(-n // P), 9, kind, drop=0.0)
        sc = a["kv_scales"]
        keys = cache_values(a["k_cache"], None if sc is None else sc[0], kind)
        page = a["page_table"].long()
        for b in range(n):                 # request b's needle is key b
            a["q"][b, 0] = (keys[page[b, b // P], b % P, 0] * 3).to(BF)
        a["selected"][..., :] = torch.arange(-(-n // P), device="cuda").to(I32)
        out, lse = run(a, F32)
        compare(a, out, lse, kind)
        vals = cache_values(a["v_cache"], None if sc is None else sc[1], kind)
        for b in range(n):
            z = (keys[page[b]].reshape(-1, 128)[:n] @ a["q"][b, 0, 0].double()) / math.sqrt(128)
            assert int(z.argmax()) == b
            if float(z.sort().values[-1] - z.sort().values[-2]) > 20:      # (all other weight below n e^-20)
                v = vals[page[b, b // P], b % P, 0]
                assert ((out[b, 0, 0].double() - v).abs() <= v.abs() * 2.0 ** -8 + 1e-5).all()


@pytest.mark.gpu
@pytest.mark.parametrize("kind", KINDS)
def test_large_and_falling_scores(kind):
    a = make([2000, 500], 1, 8, 2, 128, 16, 100, 11, kind, drop=0.0)
    a["q"].mul_(20)
    compare(a, *run(a), kind)
    a["softmax_scale"] = 1e-3
    compare(a, *run(a), kind)


@pytest.mark.gpu
def test_lists_with_repeats_and_pages_past_the_end():
    a = make([200, 90], 2, 8, 2, 128, 16, 6, 12, drop=0.0, poison=True)
    sel = a["selected"]
    sel[0] = torch.tensor([3, 3, 0, 12, 3, 1], dtype=I32)
    sel[1] = torch.tensor([5, 6, 2 ** 31 - 1, 10 ** 6, -7, 0], dtype=I32)    # request 1 has 6 pages; the last key at 89
    compare(a, *run(a), "bf16")


@pytest.mark.gpu
@pytest.mark.parametrize("kind", KINDS)
def test_bad_metadata(kind):
    a = make([200, 90, 64], 2, 8, 2, 128, 16, 6, 13, kind, drop=0.0, poison=False)
    a["selected"][:] = torch.arange(6, device="cuda").to(I32)
    a["page_table"][0, 2] = 10 ** 6
    a["page_table"][1, 3] = -9
    compare(a, *run(a, status=fd.FD_DEVSTAT_BAD_PAGE), kind)
    a = make([200, 90, 64], 2, 8, 2, 128, 16, 6, 14, kind, drop=0.0, poison=False)
    a["cache_seqlens"][:2] = torch.tensor([10 ** 9, -3])
    compare(a, *run(a, status=fd.FD_DEVSTAT_SEQLEN_OVERFLOW), kind)


@pytest.mark.gpu
@pytest.mark.parametrize("where", ["k_cache", "v_cache"])
@pytest.mark.parametrize("value", [math.nan, math.inf])
def test_values_that_are_no_numbers(where, value):
    a = make([300, 300], 1, 8, 2, 128, 16, 12, 15, drop=0.0, poison=False)
    clean = run(a)
    page = int(a["page_table"][0, int(a["selected"][0, 0, 1, 3])])
    a[where][page, 5, 1, 17] = value
    out, lse = run(a)
    assert torch.equal(out[1], clean[0][1]) and torch.equal(out[0, 0, :4], clean[0][0, 0, :4])
    bad = ~torch.isfinite(out[0, 0, 4:].float())
    if where == "k_cache":
        # a key's infinity has either sign in the scores: +inf makes the row NaN, -inf takes the key out
        assert bad.all() if math.isnan(value) else (bad.all(-1) | ~bad.any(-1)).all()
    else:
        assert bad[:, 17].all() and int(bad.sum()) == 4 and torch.equal(lse, clean[1])


def exact_rows(a, kind):
    """out, sum p|v|, the largest sum of absolute products of a score, and the keys of each row, in 64 bits (every list holds pages
    that its token sees)."""
    sc = a["kv_scales"]
    k, v = (cache_values(a[n], None if sc is None else sc[i], kind).cpu() for i, n in enumerate(("k_cache", "v_cache")))
    q, table, sel = a["q"].double().cpu(), a["page_table"].cpu().long(), a["selected"].cpu().long()
    B, Tq, Hq, D = q.shape
    P, Hkv = k.shape[1:3]
    out, mass = torch.zeros(B, Tq, Hq, D, dtype=torch.float64), torch.zeros(B, Tq, Hq, D, dtype=torch.float64)
    zabs, keys = torch.zeros(B, Tq, Hq, 1, dtype=torch.float64), torch.zeros(B, Tq, Hq, 1, dtype=torch.float64)
    for b in range(B):
        for t in range(Tq):
            n = int(a["cache_seqlens"][b]) - (Tq - 1) + t
            for h in range(Hq):
                at = [(int(table[b, p]), s) for p in sel[b, t, h // (Hq // Hkv)].tolist() if p >= 0 for s in range(P) if p * P + s < n]
                page, slot = torch.tensor(at).T
                kk, vv = k[page, slot, h // (Hq // Hkv)], v[page, slot, h // (Hq // Hkv)]
                p = torch.softmax(kk @ q[b, t, h] / math.sqrt(D), 0)
                out[b, t, h], mass[b, t, h] = p @ vv, p @ vv.abs()
                zabs[b, t, h] = (kk.abs() @ q[b, t, h].abs()).max() / math.sqrt(D)
                keys[b, t, h] = len(at)
    return out, mass, zabs, keys


@pytest.mark.gpu
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(8, 2), (16, 1), (5, 1), (36, 2)])
def test_weights_hold_more_than_one_word(kind, D, Hq, Hkv):
    """Few keys of much the same weight, where what a weight loses shows in full. A weight is two bf16 words: the first is its
    upper 16 bits, the second what is left (below 2^-7 of the weight) rounded by half a step, 2^-8 of that: 2^-15 of the
    weight; 2^-24 of it more, as the second word is never 0. A score is off by ds = (D + 8) 2^-23 of its absolute products (D
    products and additions, chopped at worst; scales, groups and the factor of exp2 the rest), its weight by 2 ds + 2^-21 (the
    exponential and the scale of its value), and out by that twice (numerator and sum) and by its own sums."""
    for lens, Tq, P, S in (([1, 2, 3, 5, 9, 14, 31], 1, 8, 4), ([3, 16, 40], 2, 16, 3), ([2, 3, 4, 6], 2, 64, 1)):
        a = make(lens, Tq, Hq, Hkv, D, P, S, D + Hq, kind, drop=0.0)
        a["q"].mul_(0.1)
        out, _ = run(a, F32)
        want, mass, zabs, n = exact_rows(a, kind)
        ds = (D + 8) * 2.0 ** -23 * zabs
        tol = mass * (2.0 ** -15 + 2.0 ** -24 + 2 * (2 * ds + 2.0 ** -21) + (2 * n + 12) * 2.0 ** -23)
        err = (out.double().cpu() - want).abs()
        assert (err <= tol).all(), float((err / tol).max())


@pytest.mark.gpu
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_infinite_values_stay_infinite(sign):
    """A visible value of infinity makes its channel that infinity, also with weights that one bf16 word holds exactly."""
    a = make([40, 16], 1, 8, 2, 128, 16, 3, 21, drop=0.0)
    a["q"][0].zero_()
    a["selected"][0, 0] = torch.arange(3, device="cuda").to(I32)
    page = int(a["page_table"][0, 1])
    a["v_cache"][page, 3, 1, 17] = sign * math.inf
    out, _ = run(a)
    assert (out[0, 0, 4:, 17] == sign * math.inf).all()
    out[0, 0, 4:, 17] = 0
    assert torch.isfinite(out).all()


@pytest.mark.gpu
def test_far_pages():
    N, P, Hkv, D = 40000, 64, 8, 128         # 2.6e9 values
    k = torch.zeros(N, P, Hkv, D, dtype=BF, device="cuda")
    v = torch.zeros(N, P, Hkv, D, dtype=BF, device="cuda")
    g = torch.Generator().manual_seed(16)
    ids = torch.tensor([[39999, 7, 32768, 32767, 39998]], dtype=I32).cuda()
    for i in ids[0].tolist():
        k[i], v[i] = torch.randn(2, P, Hkv, D, generator=g).to(BF).cuda()
    a = dict(q=torch.randn(1, 1, 16, D, generator=g).to(BF).cuda(), k_cache=k, v_cache=v, kv_scales=None, page_table=ids,
             cache_seqlens=torch.tensor([300], dtype=I32).cuda(),
             selected=torch.tensor([0, 2, 3, 4], dtype=I32).cuda().expand(1, 1, Hkv, 4).contiguous(), q_per_req=1, softmax_scale=0.0)
    out, lse = run(a)
    small = dict(a, k_cache=k[ids[0].long()], v_cache=v[ids[0].long()], page_table=torch.arange(5, device="cuda").to(I32)[None])
    compare(small, out, lse, "bf16")


@pytest.mark.gpu
@pytest.mark.parametrize("kind", KINDS)
def test_all_pages_agree_with_the_dense_call(kind):
    a = make([1000, 37, 400], 2, 16, 4, 128, 16, 63, 17, kind, poison=False)
    a["selected"][:] = torch.arange(63, device="cuda").to(I32)
    out, lse = run(a)
    plan = fd.fd_plan_create(0, 3, 2, 16, 4, 128, 16, kind, 4)
    dense, dlse = torch.empty_like(out), torch.empty_like(lse)
    fd.fd_set_plan(plan)
    try:
        fd.fd_decode_paged(a["q"], a["k_cache"], a["v_cache"], a["kv_scales"], a["page_table"], a["cache_seqlens"], 2, 2, dense, dlse)
        torch.cuda.synchronize()
    finally:
        fd.fd_set_plan(None)
        fd.fd_plan_destroy(plan)
    compare(a, out, lse, kind)
    # either is within the weights' rounding (2^-8 of values that average below 1) and its own of the exact result
    assert (out.float() - dense.float()).abs().max() <= 4 * 2.0 ** -8 * max(1.0, float(out.abs().max()))
    assert (lse - dlse).abs().max() <= 1e-3


@pytest.mark.gpu
@pytest.mark.parametrize("kind", KINDS)
def test_graphs_and_streams(kind):
    a = make([3000, 500, 2000], 2, 8, 2, 128, 16, 60, 18, kind)
    b = make([20000], 1, 64, 8, 128, 16, 128, 19, kind)
    want = [run(x) for x in (a, b)]
    o = [tuple(torch.zeros_like(x) for x in w) for w in want]
    graphs = []
    for x, (out, lse) in zip((a, b), o):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            fd.fd_decode_sparse(**x, out=out, lse=lse)
        graphs.append(graph)
    for _ in range(2):
        for graph, (out, lse), w in zip(graphs, o, want):
            out.zero_(), lse.zero_()
            graph.replay()
            assert torch.equal(out, w[0]) and torch.equal(lse, w[1])
    a["q"].copy_(a["q"].flip(2))
    a["cache_seqlens"].copy_(torch.tensor([2500, 480, 1999], dtype=I32))
    graphs[0].replay()
    torch.cuda.synchronize()
    compare(a, *o[0], kind)
    want[0] = run(a)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [[tuple(torch.zeros_like(x) for x in w) for _ in range(10)] for w in want]
    for i in range(10):
        for x, os, s in zip((a, b), outs, streams):
            fd.fd_decode_sparse(**x, out=os[i][0], lse=os[i][1], stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(o[0], w[0]) and torch.equal(o[1], w[1]) for w, os in zip(want, outs) for o in os)
