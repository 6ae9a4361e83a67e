"""Slots of new tokens and cache writes: the oracle's pins and the refusals (CPU), the
kernels against the oracle (GPU; codes, scales, slots and bounds are exact, so equality)."""
import math

import numpy as np
import pytest
import torch

import split_kv_paged_gqa_gb300 as fd
from oracle.step_ref import append_ref, append_slots_ref, outward, quantise_ref
from split_kv_paged_gqa_gb300 import workloads as wl

BF, F32, F64, I32, I64 = torch.bfloat16, torch.float32, torch.float64, torch.int32, torch.int64


# ---------------------------------------------------------------------------
# oracle pins


def test_slots_oracle_hand_worked():
    # P 4: request 0 holds 3 keys (page 9) and gets 3: one new page; request 1 holds none and gets 5: two pages;
    # request 2 holds 8 (full) and gets none; request 3 holds 4 (full) and gets 1
    table = [[9, -1, -1], [-1, -1, -1], [5, 6, -1], [2, -1, -1]]
    t, slots, pos, lens, cu, taken, st = append_slots_ref([3, 0, 8, 4], [3, 5, 0, 1], [20, 21, 22, 23, 24], 4, 4, table, 11)
    assert t.tolist() == [[9, 20, -1], [21, 22, -1], [5, 6, -1], [2, 23, -1]]
    assert slots.tolist() == [39, 80, 81, 84, 85, 86, 87, 88, 92, -1, -1]
    assert pos.tolist() == [3, 4, 5, 0, 1, 2, 3, 4, 4, 0, 0]
    assert lens.tolist() == [6, 5, 8, 5] and cu.tolist() == [0, 3, 8, 8, 9] and taken == 4 and st == 0
    t, slots, pos, lens, cu, taken, st = append_slots_ref([3, 0, 8, 4], [3, 5, 0, 1], [20, 21, 22, 23, 24], 2, 4, table, 11)
    assert slots.tolist() == [39, 80, 81] + [-1] * 8 and lens.tolist() == [6, 0, 8, 4] and taken == 1 and st == 16


def test_outward_rounding():
    x = np.array([1.0, 1.0 + 2 ** -20, -1.0 - 2 ** -20, 3e-45, 0.0, -3e-45, 1e39, np.inf])
    up, down = outward(x, True), outward(x, False)
    assert up.tolist()[:3] == [1.0, 1.0 + 2 ** -7, -1.0] and down.tolist()[:3] == [1.0, 1.0, -1.0 - 2 ** -7]
    assert up[3] == 2.0 ** -133 and down[3] == 0.0 and up[5] == 0.0 and down[5] == -2.0 ** -133
    assert up[6] == np.inf and np.isfinite(down[6]) and up[7] == np.inf


@pytest.mark.parametrize("kind", ["int8", "int4"])
def test_quantiser_is_the_workloads_one(kind):
    """Same codes and scales as the cache writer of the synthetic workloads, but for quotients that its fp32
    division puts on the other side of a half."""
    g = torch.Generator().manual_seed(3)
    x = torch.randn(400, 128, generator=g).to(BF)
    codes, scale = (wl.quantize_int8 if kind == "int8" else wl.quantize_int4)(x)
    if kind == "int4":
        c = codes.view(torch.int8)
        codes = torch.stack([c << 4 >> 4, c >> 4], -1).flatten(-2)
    for i in range(400):
        row = x[i].double().numpy()
        c, s = quantise_ref(row, kind)
        assert np.array_equal(s, scale[i].numpy())
        # an fp32 quotient below 128 is off by at most 2^-18: it can only change the side of a half that is so near
        exact = row / np.repeat(s.astype(np.float64), row.size // s.size)
        differ = c != codes[i].numpy()
        assert (np.abs(np.abs(exact - np.floor(exact)) - 0.5)[differ] <= 2.0 ** -18).all()
        assert (np.abs(c - codes[i].numpy()) <= 1).all()


# ---------------------------------------------------------------------------
# refusals


def _slot_args(B=3, W=4, F=6, T=8):
    z = lambda *n, dtype=I32: torch.zeros(*n, dtype=dtype)   # noqa: E731
    return dict(cache_seqlens=z(B), num_new=z(B), free_pages=z(F), num_free=None, page_size=16, page_table=z(B, W),
                slots=z(T, dtype=I64), positions=z(T), new_seqlens=z(B), cu_seqlens_q=z(B + 1), pages_taken=z(1))


@pytest.mark.parametrize("change,status", [
    (dict(cache_seqlens=torch.zeros(3, dtype=I64)), fd.FD_ERR_INVALID_ARG),
    (dict(cache_seqlens=torch.zeros(3, 1, dtype=I32)), fd.FD_ERR_INVALID_ARG),
    (dict(cache_seqlens=None), fd.FD_ERR_INVALID_ARG),
    (dict(num_new=torch.zeros(2, dtype=I32)), fd.FD_ERR_INVALID_ARG),
    (dict(free_pages=torch.zeros(0, dtype=I32)), fd.FD_ERR_INVALID_ARG),
    (dict(free_pages=torch.zeros(4)), fd.FD_ERR_INVALID_ARG),
    (dict(num_free=torch.zeros(2, dtype=I32)), fd.FD_ERR_INVALID_ARG),
    (dict(page_size=0), fd.FD_ERR_INVALID_ARG),
    (dict(page_table=torch.zeros(2, 4, dtype=I32)), fd.FD_ERR_INVALID_ARG),
    (dict(page_table=torch.zeros(1, 4, dtype=I32).expand(3, 4)), fd.FD_ERR_UNSUPPORTED),
    (dict(page_table=torch.zeros(3, 8, dtype=I32)[:, ::2]), fd.FD_ERR_UNSUPPORTED),
    (dict(slots=torch.zeros(8)), fd.FD_ERR_INVALID_ARG),
    (dict(slots=torch.zeros(16, dtype=I64)[::2]), fd.FD_ERR_UNSUPPORTED),
    (dict(positions=torch.zeros(7, dtype=I32)), fd.FD_ERR_INVALID_ARG),
    (dict(new_seqlens=torch.zeros(4, dtype=I32)), fd.FD_ERR_INVALID_ARG),
    (dict(cu_seqlens_q=torch.zeros(3, dtype=I32)), fd.FD_ERR_INVALID_ARG),
    (dict(pages_taken=torch.zeros(2, dtype=I32)), fd.FD_ERR_INVALID_ARG),
    (dict(status=torch.zeros(1, dtype=I64)), fd.FD_ERR_INVALID_ARG),
])
def test_slots_rejects(change, status):
    with pytest.raises(fd.FdError) as e:
        fd.fd_append_slots(**{**_slot_args(), **change}, stream=0)
    assert e.value.status == status, str(e.value)


def test_slots_rejects_outputs_over_inputs():
    a = _slot_args()
    for change in (dict(new_seqlens=a["cache_seqlens"]), dict(new_seqlens=a["num_new"]),
                   dict(pages_taken=a["free_pages"][5:6]), dict(num_free=a["cu_seqlens_q"][3:4])):
        with pytest.raises(fd.FdError) as e:
            fd.fd_append_slots(**{**a, **change}, stream=0)
        assert e.value.status == fd.FD_ERR_UNSUPPORTED, str(e.value)


def _append_args(kind="bf16", T=5, Hkv=2, D=128, N=6, P=16):
    row = D // 2 if kind == "int4" else D
    dt = dict(bf16=BF, int8=torch.int8, int4=torch.uint8)[kind]
    return dict(k=torch.zeros(T, Hkv, D, dtype=BF), v=torch.zeros(T, Hkv, D, dtype=BF), slots=torch.zeros(T, dtype=I64),
                k_cache=torch.zeros(N, P, Hkv, row, dtype=dt), v_cache=torch.zeros(N, P, Hkv, row, dtype=dt),
                kv_scales=None if kind == "bf16" else torch.zeros(2, N, P, Hkv, 1 if kind == "int8" else D // 32),
                page_bounds=torch.zeros(N, Hkv, 2, D, dtype=BF))


@pytest.mark.parametrize("kind,change,status", [
    ("bf16", dict(k=torch.zeros(5, 2, 128)), fd.FD_ERR_INVALID_ARG),
    ("bf16", dict(k=torch.zeros(5, 3, 128, dtype=BF)), fd.FD_ERR_INVALID_ARG),
    ("bf16", dict(v=torch.zeros(4, 2, 128, dtype=BF)), fd.FD_ERR_INVALID_ARG),
    ("bf16", dict(k=torch.zeros(5, 2, 256, dtype=BF)[..., ::2]), fd.FD_ERR_UNSUPPORTED),
    ("bf16", dict(k=torch.zeros(5 * 2 * 128 + 1, dtype=BF)[1:].view(5, 2, 128)), fd.FD_ERR_UNSUPPORTED),
    ("bf16", dict(slots=torch.zeros(4, dtype=I64)), fd.FD_ERR_INVALID_ARG),
    ("bf16", dict(slots=torch.zeros(5)), fd.FD_ERR_INVALID_ARG),
    ("bf16", dict(k_cache=torch.zeros(6, 24, 2, 128, dtype=BF), v_cache=torch.zeros(6, 24, 2, 128, dtype=BF)), fd.FD_ERR_UNSUPPORTED),
    ("bf16", dict(k_cache=torch.zeros(6, 16, 2, 128)), fd.FD_ERR_INVALID_ARG),
    ("bf16", dict(v_cache=torch.zeros(6, 16, 2, 128, dtype=torch.int8)), fd.FD_ERR_INVALID_ARG),
    ("bf16", dict(v_cache=torch.zeros(7, 16, 2, 128, dtype=BF)), fd.FD_ERR_INVALID_ARG),
    ("bf16", dict(v_cache=torch.zeros(6, 2, 16, 128, dtype=BF).transpose(1, 2)), fd.FD_ERR_UNSUPPORTED),
    ("bf16", dict(k_cache=torch.zeros(1, 16, 2, 128, dtype=BF).expand(6, 16, 2, 128),
                  v_cache=torch.zeros(1, 16, 2, 128, dtype=BF).expand(6, 16, 2, 128)), fd.FD_ERR_UNSUPPORTED),
    ("bf16", dict(kv_scales=torch.zeros(2, 6, 16, 2, 1)), fd.FD_ERR_INVALID_ARG),
    ("int8", dict(kv_scales=None), fd.FD_ERR_INVALID_ARG),
    ("int8", dict(kv_scales=torch.zeros(2, 6, 16, 2, 4)), fd.FD_ERR_INVALID_ARG),
    ("int8", dict(kv_scales=torch.zeros(1, 6, 16, 2, 1).expand(2, 6, 16, 2, 1)), fd.FD_ERR_UNSUPPORTED),
    ("int4", dict(kv_scales=torch.zeros(2, 6, 16, 2, 5)[..., :4]), fd.FD_ERR_UNSUPPORTED),
    ("int4", dict(k_cache=torch.zeros(6, 16, 2, 128, dtype=torch.uint8)), fd.FD_ERR_INVALID_ARG),
    ("bf16", dict(page_bounds=torch.zeros(5, 2, 2, 128, dtype=BF)), fd.FD_ERR_INVALID_ARG),
    ("bf16", dict(page_bounds=torch.zeros(6, 2, 2, 128)), fd.FD_ERR_INVALID_ARG),
    ("bf16", dict(page_bounds=torch.zeros(6, 1, 2, 128, dtype=BF).expand(6, 2, 2, 128)), fd.FD_ERR_UNSUPPORTED),
    ("bf16", dict(status=torch.zeros(1)), fd.FD_ERR_INVALID_ARG),
])
def test_append_rejects(kind, change, status):
    with pytest.raises(fd.FdError) as e:
        fd.fd_cache_append(**{**_append_args(kind), **change}, stream=0)
    assert e.value.status == status, str(e.value)


def test_append_rejects_other_head_dims():
    with pytest.raises(fd.FdError) as e:
        fd.fd_cache_append(**_append_args(D=96), stream=0)
    assert e.value.status == fd.FD_ERR_UNSUPPORTED


# ---------------------------------------------------------------------------
# slots against the oracle


def run_slots(seqlens, new, free, num_free, P, table, T, dtype=I64, positions=True, strided=False):
    ints = lambda x: torch.tensor(np.asarray(x), dtype=I32, device="cuda")   # noqa: E731
    wide = (lambda x: torch.stack([ints(x), ints(x) + 77], 1)[:, 0]) if strided else ints
    tab = ints(table)
    if strided:
        tab = torch.nn.functional.pad(tab, (0, 3), value=55)[:, :-3]
    guard = 9
    o = {k: torch.full((n + guard,), 777, dtype=d, device="cuda") for k, n, d in
         (("slots", T, dtype), ("positions", T, I32), ("new_seqlens", len(new), I32), ("cu_seqlens_q", len(new) + 1, I32),
          ("pages_taken", 1, I32))}
    views = {k: x[:-guard] for k, x in o.items()}
    if not positions:
        views["positions"] = None
    status = torch.zeros(1, dtype=I32, device="cuda")
    fd.fd_append_slots(wide(seqlens), wide(new), wide(free), None if num_free is None else ints([num_free]), P, tab,
                       status=status, **views)
    for x in o.values():
        assert (x[-guard:] == 777).all()
    ref = append_slots_ref(seqlens, new, free, num_free, P, table, T, 2 ** 31 - 1 if dtype == I32 else 2 ** 63 - 1)
    assert int(status) == ref[-1]
    assert int(views["pages_taken"]) == ref[5]
    for got, want in ((tab, ref[0]), (views["slots"], ref[1]), (views["positions"], ref[2]), (views["new_seqlens"], ref[3]),
                      (views["cu_seqlens_q"], ref[4])):
        if got is not None:
            assert np.array_equal(got.cpu().numpy(), want)
    return ref


def slot_case(B, P, hi_len, hi_new, seed, spare=1.0, pad=0, W=None, **kw):
    r = np.random.default_rng(seed)
    L, n = r.integers(0, hi_len + 1, B), r.integers(0, hi_new + 1, B)
    need = -(-(L + n) // P) - -(-L // P)
    F = max(1, int(need.sum() * spare))
    W = W or int((-(-(L + n) // P)).max()) + 1
    pages = r.permutation(F + int((-(-L // P)).sum()))
    table = np.full((B, W), -1)
    at = F
    for b in range(B):
        k = min(W, -(-int(L[b]) // P))
        table[b, :k] = pages[at:at + k]
        at += k
    return run_slots(L, n, pages[:F], None, P, table, max(1, int(n.sum()) + pad), **kw)


@pytest.mark.gpu
@pytest.mark.parametrize("B", [1, 2, 31, 64, 1000, 1024, 1025, 2100, 5000])
@pytest.mark.parametrize("dtype", [I32, I64])
def test_slots_batches(B, dtype):
    slot_case(B, 16, 500, 3, B, dtype=dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("P", [1, 3, 8, 16, 100, 256])
@pytest.mark.parametrize("pad,positions,strided", [(0, True, False), (1, False, True), (3000, True, True)])
def test_slots_pages(P, pad, positions, strided):
    slot_case(37, P, 700, 300, P, pad=pad, positions=positions, strided=strided)


@pytest.mark.gpu
def test_slots_all_new_or_none_new():
    slot_case(1, 64, 0, 100000, 1)
    slot_case(40, 16, 0, 2000, 2)
    slot_case(300, 16, 100, 0, 3, pad=5)
    slot_case(3000, 8, 100, 40, 4, pad=5)


@pytest.mark.gpu
@pytest.mark.parametrize("spare", [0.0, 0.3, 0.99])
def test_slots_too_few_pages(spare):
    assert slot_case(50, 16, 300, 60, 5, spare=spare)[-1] == 16
    assert slot_case(2500, 16, 300, 60, 6, spare=spare)[-1] == 16


@pytest.mark.gpu
def test_slots_number_of_free_pages_on_the_device():
    table = [[9, -1, -1], [-1, -1, -1], [5, 6, -1], [2, -1, -1]]
    for num_free in (-3, 0, 1, 2, 3, 4, 5, 6):
        run_slots([3, 0, 8, 4], [3, 5, 0, 1], [20, 21, 22, 23, 24], num_free, 4, table, 11)


@pytest.mark.gpu
def test_slots_bad_numbers():
    table = [[9, 8, 7], [1, -1, -1], [5, 6, -1], [2, -1, -1]]
    # negative lengths and counts, more pages than the table has, an entry that was never set, a free page below 0
    assert run_slots([-3, 2, 8, 4], [3, 5, 1, 1], [20, 21, -1, 23], None, 4, table, 11)[-1] == 3
    assert run_slots([2, 2, 5, 4], [-1, 5, 8, 1], [20, 21, 22, 23], None, 4, table, 20)[-1] == 2
    assert run_slots([2, 7, 5, 4], [1, 1, 1, 1], [20, 21, 22, 23], None, 4, table, 4)[-1] == 1
    # rows past the buffer: those requests get nothing
    assert run_slots([0, 0, 0, 0], [3, 3, 3, 3], [20, 21, 22, 23], None, 4, table, 7)[-1] == 2
    # a count whose sum with the length does not fit
    assert run_slots([2 ** 31 - 2, 0, 0, 0], [5, 2, 2 ** 31 - 1, 2 ** 31 - 1], [20, 21, 22, 23], None, 4, table, 9)[-1] == 2
    # slots past int32
    big = [[2 ** 30, -1, -1]] * 4
    assert run_slots([1, 1, 1, 1], [1, 1, 1, 1], [20, 21, 22, 23], None, 4, big, 4, dtype=I32)[-1] == 1
    assert run_slots([1, 1, 1, 1], [1, 1, 1, 1], [20, 21, 22, 23], None, 4, big, 4, dtype=I64)[-1] == 0


@pytest.mark.gpu
def test_slots_largest_batch():
    slot_case(65535, 16, 50, 2, 7, W=5)


# ---------------------------------------------------------------------------
# cache writes against the oracle


def cache_values(cache, scales, kind):
    """float64 values of a cache [N, P, Hkv, D] of any kind."""
    if kind == "bf16":
        return cache.double()
    if kind == "int4":
        c = cache.view(torch.int8)
        cache = torch.stack([c << 4 >> 4, c >> 4], -1).flatten(-2)
    return (cache.double().unflatten(-1, (scales.shape[-1], -1)) * scales.double()[..., None]).flatten(-2)


def make_caches(kind, N, P, Hkv, D, g, head_major=False):
    dt = dict(bf16=BF, int8=torch.int8, int4=torch.uint8)[kind]
    row = D // 2 if kind == "int4" else D
    out = []
    for _ in range(2):
        shape = (N, Hkv, P, row) if head_major else (N, P, Hkv, row)
        x = torch.randn(shape, generator=g).to(BF) if kind == "bf16" else torch.randint(
            -127 if kind == "int8" else 0, 128 if kind == "int8" else 256, shape, generator=g).to(dt)
        x = x.cuda()
        out.append(x.transpose(1, 2) if head_major else x)
    scales = None
    if kind != "bf16":
        scales = (torch.rand(2, N, Hkv, P, 1 if kind == "int8" else D // 32, generator=g) + 0.5).cuda().transpose(2, 3)
    return out[0], out[1], scales


def run_append(k, v, slots, caches, bounds, kind, slot_dtype=I64, status=0):
    """One call, everything it may and may not touch checked against the oracle."""
    kc, vc, sc = caches
    N, P, Hkv, _ = kc.shape
    before = [x.clone() if x is not None else None for x in (kc, vc, sc)]
    b0 = None if bounds is None else bounds.double().cpu().numpy()
    st = torch.zeros(1, dtype=I32, device="cuda")
    fd.fd_cache_append(k, v, slots.to(slot_dtype), kc, vc, sc, bounds, st)
    assert int(st) == status
    f64 = lambda t: t.double().cpu().numpy()   # noqa: E731
    values = f64(cache_values(before[0], None if sc is None else before[2][0], kind)).reshape(N * P, Hkv, -1)
    rows, want_bounds = append_ref(f64(k), f64(v), slots.tolist(), values, b0, P, kind)
    for which, cache in ((0, kc), (1, vc)):
        want = before[which].cpu().clone()
        wsc = None if sc is None else before[2].cpu().clone()
        for s, r in rows[which].items():
            if kind == "bf16":
                want[s // P, s % P] = torch.tensor(r).to(BF)
                continue
            for h, (c, scale) in enumerate(r):
                c = torch.tensor(c)
                want[s // P, s % P, h] = c.to(torch.int8) if kind == "int8" else (c[0::2] % 16 + 16 * (c[1::2] % 16)).to(torch.uint8)
                wsc[which, s // P, s % P, h] = torch.tensor(scale)
        if kind == "bf16":
            assert torch.equal(cache.cpu().view(torch.int16), want.view(torch.int16))
        else:
            assert torch.equal(cache.cpu(), want)
            got = sc[which].cpu()
            assert torch.equal(torch.nan_to_num(got, nan=-1.0), torch.nan_to_num(wsc[which], nan=-1.0))
    if bounds is not None:
        got = f64(bounds)
        assert np.array_equal(np.isnan(got), np.isnan(want_bounds))
        assert (np.isnan(got) | (got == want_bounds)).all()


def new_rows(T, Hkv, D, g, scale=1.0):
    x = (torch.randn(T, 3 * Hkv + 1, D, generator=g) * scale).to(BF).cuda()    # views of a larger projection
    return x[:, Hkv:2 * Hkv], x[:, 2 * Hkv:3 * Hkv]


def runs_of(lens, new, P, N, seed):
    """Slots of a batch: requests of the given lengths on scattered pages get new tokens."""
    r = np.random.default_rng(seed)
    pages = r.permutation(N)
    out, at = [], 0
    for L, n in zip(lens, new):
        k = -(-(L + n) // P)
        mine = pages[at:at + k]
        at += k
        out += [int(mine[p // P]) * P + p % P for p in range(L, L + n)]
    assert at <= N
    return torch.tensor(out, dtype=I64, device="cuda")


def append_case(kind, lens, new, Hkv, D, P, seed, bounds=True, pad=0, head_major=False, **kw):
    g = torch.Generator().manual_seed(seed)
    N = sum(-(-(a + b) // P) for a, b in zip(lens, new)) + 2
    slots = torch.nn.functional.pad(runs_of(lens, new, P, N, seed), (0, pad), value=-1)
    k, v = new_rows(slots.numel(), Hkv, D, g)
    bd = torch.randn(N, Hkv, 2, D, generator=g).to(BF).cuda() if bounds else None
    run_append(k, v, slots, make_caches(kind, N, P, Hkv, D, g, head_major), bd, kind, **kw)


KINDS = ["bf16", "int8", "int4"]


@pytest.mark.gpu
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("P", [8, 16, 64, 256])
def test_append_one_token_each(kind, D, P):
    append_case(kind, [0, 1, P - 1, P, P + 1, 2 * P - 1, 300], [1] * 7, 2, D, P, P + D)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("bounds", [True, False])
def test_append_runs(kind, D, bounds):
    append_case(kind, [0, 5, 40, 0, 31, 7], [1, 70, 0, 33, 2, 130], 3, D, 32, 11, bounds=bounds, pad=21, slot_dtype=I32)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("Hkv,P,n", [(1, 256, 700), (8, 16, 500), (5, 8, 1000)])
def test_append_prompts(kind, Hkv, P, n):
    append_case(kind, [0, 3, 1000], [n, n // 3, n // 2], Hkv, 128, P, n, head_major=True)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", KINDS)
def test_append_nothing_and_padding(kind):
    append_case(kind, [3], [0], 2, 64, 16, 5, pad=40)
    g = torch.Generator().manual_seed(6)
    k, v = new_rows(6, 2, 128, g)
    caches = make_caches(kind, 4, 16, 2, 128, g)
    bd = torch.zeros(4, 2, 2, 128, dtype=BF, device="cuda")
    # padded rows in the middle, slots past the cache, below -1, and neighbours in two pages
    run_append(k, v, torch.tensor([15, 16, -1, 64, -7, 40], device="cuda"), caches, bd, kind, status=fd.FD_DEVSTAT_BAD_PAGE)
    far = torch.tensor([3, 2 ** 40, -2 ** 40, 2 ** 31, -1, 63], device="cuda")
    run_append(k, v, far, caches, bd, kind, status=fd.FD_DEVSTAT_BAD_PAGE)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", KINDS)
def test_append_values_that_are_hard_to_round(kind):
    """Zeros, rows of one value, exact halves, subnormal and very large values, infinities and NaN."""
    g = torch.Generator().manual_seed(8)
    k, v = new_rows(40, 2, 128, g)
    k, v = k.clone(), v.clone()
    top = 127.0 if kind == "int8" else 7.0
    halves = torch.arange(128) % (2 * int(top) + 1) - top
    for i, x in enumerate([torch.zeros(128), torch.full((128,), -3.0), halves + 0.5, halves, halves * 2.0 ** -120,
                           torch.randn(128, generator=g) * 2.0 ** -126, torch.full((128,), 2.0 ** -133),
                           torch.randn(128, generator=g) * 1e38, halves * 2.0 ** 120, (halves + 0.5) * 2.0 ** -130,
                           torch.randn(128, generator=g) * 1e-30]):
        k[i, 0] = x.to(BF)
        v[i, 1] = x.to(BF)
    k[20, 1, 5], k[21, 0, 77], k[22, 1, 100], v[23, 0, 3], v[24, 1, 127] = math.inf, -math.inf, math.nan, math.nan, math.inf
    bd = torch.zeros(4, 2, 2, 128, dtype=BF, device="cuda")
    run_append(k, v, torch.arange(5, 45, device="cuda"), make_caches(kind, 4, 16, 2, 128, g), bd, kind)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["int8", "int4"])
def test_append_codes_of_many_magnitudes(kind):
    g = torch.Generator().manual_seed(9)
    x = torch.randn(600, 4, 128, generator=g) * torch.exp2(torch.randint(-60, 60, (600, 4, 1), generator=g).float())
    k = x.to(BF).cuda()
    run_append(k, k.flip(1), torch.arange(600, device="cuda"), make_caches(kind, 10, 64, 4, 128, g), None, kind)


def rounded_outwards(x, up):
    """x (float64, within bf16's range) to 8 significant bits, away from the middle."""
    step = torch.exp2((torch.frexp(x)[1] - 8).clamp(min=-133).double())
    return (torch.ceil(x / step) if up else torch.floor(x / step)) * step


def append_many(k, v, slots, caches, bounds, P, kind):
    """What fd_cache_append makes of many rows, in 64 bits and all at once: caches, scales, bounds (float64)."""
    kc, vc, sc = (None if x is None else x.clone() for x in caches)
    there = ((slots >= 0) & (slots < kc.shape[0] * P)).nonzero()[:, 0]
    page, off = slots[there] // P, slots[there] % P
    for which, (x, cache) in enumerate(((k, kc), (v, vc))):
        x = x[there]
        if kind == "bf16":
            cache[page, off] = x
            continue
        top = 127 if kind == "int8" else 7
        x = x.double().unflatten(-1, (sc.shape[-1], -1))
        scale = (x.abs().amax(-1) / top).float()
        c = torch.where(scale[..., None] > 0, x / scale[..., None].double(), 0.0).round().clamp(-top, top).flatten(-2).int()
        cache[page, off] = c.to(torch.int8) if kind == "int8" else (c[..., 0::2] % 16 + 16 * (c[..., 1::2] % 16)).to(torch.uint8)
        sc[which][page, off] = scale
    if bounds is not None:
        bounds = bounds.double()
        end = torch.zeros(kc.shape[0], dtype=I64, device=slots.device).scatter_reduce(0, page, off + 1, "amax")
        hit = end.nonzero()[:, 0]
        x = cache_values(kc[hit], None if sc is None else sc[0][hit], kind)
        here = (torch.arange(P, device=slots.device) < end[hit, None])[..., None, None]
        bounds[hit, :, 0] = rounded_outwards(torch.where(here, x, math.inf).amin(1), False)
        bounds[hit, :, 1] = rounded_outwards(torch.where(here, x, -math.inf).amax(1), True)
    return kc, vc, sc, bounds


def many_slots(lens, new, P, seed, between):
    """Slots of a batch, and rows without one: between the requests, or (where no bounds are formed) anywhere. And the pages."""
    r, counts = np.random.default_rng(seed), [-(-(a + b) // P) for a, b in zip(lens, new)]
    N, at, slots = sum(counts) + 2, 0, []
    pages = r.permutation(N)
    for a, b, n in zip(lens, new, counts):
        slots += [int(pages[at + p // P]) * P + p % P for p in range(a, a + b)]
        at += n
    ends = np.cumsum(new)
    out, last = [], 0
    for end in ends if between else range(0, len(slots), 7):
        out += slots[last:end] + [[-1], [N * P + 3], [-1, -5, -1], []][int(r.integers(4))]
        last = end
    return torch.tensor(out + slots[last:], dtype=I64), N


def test_many_rows_oracle_is_the_small_one():
    g = torch.Generator().manual_seed(2)
    for kind, D, P in (("bf16", 64, 8), ("int8", 128, 16), ("int4", 64, 8)):
        lens, new = [3, 0, 17], [9, 0, 20]
        slots, N = many_slots(lens, new, P, 3, True)
        x = torch.randn(2, slots.numel(), 2, D, generator=g).to(BF)
        row = D // 2 if kind == "int4" else D
        caches = [torch.randn(N, P, 2, row, generator=g).to(BF) if kind == "bf16" else
                  torch.randint(0, 120, (N, P, 2, row), generator=g).to(torch.int8 if kind == "int8" else torch.uint8) for _ in range(2)]
        sc = None if kind == "bf16" else torch.rand(2, N, P, 2, 1 if kind == "int8" else D // 32, generator=g) + 0.5
        bd = torch.randn(N, 2, 2, D, generator=g).to(BF)
        kc, vc, nsc, nbd = append_many(x[0], x[1], slots, (*caches, sc), bd, P, kind)
        values = cache_values(caches[0], None if sc is None else sc[0], kind).numpy().reshape(N * P, 2, D)
        rows, want = append_ref(x[0].double().numpy(), x[1].double().numpy(), slots.tolist(), values, bd.double().numpy(), P, kind)
        assert np.array_equal(nbd.numpy(), want)
        for which, cache in ((0, kc), (1, vc)):
            got = cache_values(cache, None if sc is None else nsc[which], kind).numpy()
            old = cache_values(caches[which], None if sc is None else sc[which], kind).numpy()
            for s, r in rows[which].items():
                for h in range(2):
                    old[s // P, s % P, h] = r[h] if kind == "bf16" else r[h][0] * np.repeat(r[h][1].astype(np.float64), D // r[h][1].size)
            assert np.array_equal(got, old)


def append_many_case(kind, D, P, Hkv, T, bounds, seed):
    """About T rows: short and long runs that begin anywhere in a page."""
    r, g = np.random.default_rng(seed), torch.Generator(device="cuda").manual_seed(seed)
    lens, new = [], []
    while sum(new) < T:
        lens.append(int(r.integers(0, 3 * P)))
        new.append(int(r.choice([1, 2, 5, P - 1, P, 2 * P + 3, 301])))
    slots, N = many_slots(lens, new, P, seed, bounds)
    slots = slots.cuda()
    x = torch.randn(slots.numel(), 2 * Hkv, D, generator=g, device="cuda").to(BF)
    caches = make_caches(kind, N, P, Hkv, D, torch.Generator().manual_seed(seed), head_major=seed % 2 == 1)
    bd = torch.zeros(N, Hkv, 2, D, dtype=BF, device="cuda") if bounds else None
    want = append_many(x[:, :Hkv], x[:, Hkv:], slots, caches, bd, P, kind)
    st = torch.zeros(1, dtype=I32, device="cuda")
    fd.fd_cache_append(x[:, :Hkv], x[:, Hkv:], slots, *caches, bd, st)
    assert int(st) == (fd.FD_DEVSTAT_BAD_PAGE if int(slots.max()) >= N * P else 0)
    for got, exact in zip((*caches, bd), want):
        assert got is None or torch.equal(got.double(), exact.double())


@pytest.mark.gpu
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("bounds", [True, False])
@pytest.mark.parametrize("P,Hkv,T", [(16, 2, 1300), (64, 3, 1300), (256, 1, 4000), (256, 8, 2000), (64, 8, 2600), (8, 8, 2600),
                                     (16, 4, 5100), (32, 8, 2600), (16, 8, 7600), (64, 8, 14400), (256, 8, 14400)])
def test_append_many_rows(kind, D, bounds, P, Hkv, T):
    """Rows on both sides of the numbers from which on a CTA or a warp takes several tokens: 2432, 20000 of a quantised cache, and
    58368 and 113088, where it takes the most (16 tokens, of pages past 32 tokens 31)."""
    append_many_case(kind, D, P, Hkv, T, bounds, P + Hkv + T + D // 64)

@pytest.mark.gpu
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("P,B,Tq", [(16, 50, 4), (64, 9, 3), (16, 700, 4)])
def test_append_rows_in_another_order(kind, P, B, Tq):
    """Rows by token first ([Tq, B]): several runs in a page. All keys and values arrive, and the bounds of pages with one run are right."""
    D, Hkv = 64, 8
    lens = [(7 * b) % (3 * P) for b in range(B)]
    N = sum(-(-(n + Tq) // P) for n in lens) + 2
    slots = runs_of(lens, [Tq] * B, P, N, 5).view(B, Tq).T.reshape(-1)
    g = torch.Generator().manual_seed(6)
    k, v = new_rows(B * Tq, Hkv, D, g)
    caches = make_caches(kind, N, P, Hkv, D, g)
    bd = torch.zeros(N, Hkv, 2, D, dtype=BF, device="cuda")
    want = append_many(k, v, slots, caches, bd, P, kind)
    fd.fd_cache_append(k, v, slots, *caches, bd)
    for got, exact in zip(caches, want):
        assert got is None or torch.equal(got, exact)
    single = torch.bincount(slots // P, minlength=N) <= 1
    assert torch.equal(bd[single].double(), want[3][single])


@pytest.mark.gpu
def test_append_far_pages():
    """Rows past 2^31 elements from the cache's start."""
    N, P, Hkv, D = 70000, 64, 8, 64
    kc = torch.zeros(N, P, Hkv, D, dtype=BF, device="cuda")
    vc = torch.zeros(N, P, Hkv, D, dtype=BF, device="cuda")
    bd = torch.zeros(N, Hkv, 2, D, dtype=BF, device="cuda")
    g = torch.Generator().manual_seed(10)
    k, v = new_rows(3, Hkv, D, g)
    slots = torch.tensor([N * P - 2, N * P - 1, (N - 5) * P], device="cuda")
    fd.fd_cache_append(k, v, slots, kc, vc, None, bd)
    for i, s in enumerate(slots.tolist()):
        assert torch.equal(kc[s // P, s % P], k[i]) and torch.equal(vc[s // P, s % P], v[i])
    assert torch.equal(bd[N - 5, :, 0], k[2]) and torch.equal(bd[N - 5, :, 1], k[2])
    assert torch.equal(bd[N - 1, :, 1], torch.maximum(k[0], k[1]).clamp(min=0))   # the page's other keys are 0
    assert int((kc != 0).any(-1).any(-1).sum()) == 3


@pytest.mark.gpu
@pytest.mark.parametrize("kind", KINDS)
def test_slots_and_append_in_a_graph(kind):
    """Steps of allocation and writing, captured once and replayed with other numbers, against the same steps called."""
    B, P, Hkv, D, W, T = 5, 16, 2, 64, 20, 24

    def world():
        g = torch.Generator().manual_seed(12)
        w = dict(lens=torch.tensor([0, 15, 16, 40, 3], dtype=I32).cuda(), new=torch.zeros(B, dtype=I32).cuda(),
                 free=torch.randperm(90, generator=g).to(I32).cuda(), table=torch.full((B, W), -1, dtype=I32).cuda(),
                 slots=torch.zeros(T, dtype=I64).cuda(), pos=torch.zeros(T, dtype=I32).cuda(), nl=torch.zeros(B, dtype=I32).cuda(),
                 cu=torch.zeros(B + 1, dtype=I32).cuda(), taken=torch.zeros(1, dtype=I32).cuda(), k=torch.zeros(T, Hkv, D, dtype=BF).cuda(),
                 v=torch.zeros(T, Hkv, D, dtype=BF).cuda(), bounds=torch.zeros(100, Hkv, 2, D, dtype=BF).cuda(),
                 status=torch.zeros(1, dtype=I32).cuda())
        for b, n in enumerate((0, 1, 1, 3, 1)):
            w["table"][b, :n] = 90 + torch.arange(n).cuda() + b
        w["kc"], w["vc"], w["sc"] = make_caches(kind, 100, P, Hkv, D, g)
        return w

    def step(w):
        fd.fd_append_slots(w["lens"], w["new"], w["free"], None, P, w["table"], w["slots"], w["pos"], w["nl"], w["cu"], w["taken"],
                           w["status"])
        fd.fd_cache_append(w["k"], w["v"], w["slots"], w["kc"], w["vc"], w["sc"], w["bounds"], w["status"])
        w["lens"].copy_(w["nl"])
        w["free"].copy_(w["free"].gather(0, (torch.arange(90, device="cuda") + w["taken"]).clamp(max=89).long()))

    a, b = world(), world()
    g = torch.Generator().manual_seed(13)
    steps = [(torch.randint(0, 5, (B,), generator=g, dtype=I32), torch.randn(2, T, Hkv, D, generator=g).to(BF)) for _ in range(6)]
    graph = torch.cuda.CUDAGraph()
    keep = {k: (x.clone() if x is not None else None) for k, x in b.items()}
    with torch.cuda.graph(graph):
        step(b)
    for k, x in keep.items():
        if x is not None:
            b[k].copy_(x)
    for new, kv in steps:
        for w in (a, b):
            w["new"].copy_(new)
            w["k"].copy_(kv[0])
            w["v"].copy_(kv[1])
        step(a)
        graph.replay()
        for k in a:
            if a[k] is not None:
                assert torch.equal(torch.nan_to_num(a[k].float()), torch.nan_to_num(b[k].float())), k
    assert int(a["status"]) == 0 and a["lens"].tolist() == [x + int(sum(s[0][i] for s in steps)) for i, x in enumerate((0, 15, 16, 40, 3))]


@pytest.mark.gpu
def test_append_on_another_stream():
    g = torch.Generator().manual_seed(14)
    k, v = new_rows(64, 8, 128, g)
    slots = torch.arange(64, device="cuda") * 16
    kc, vc, _ = make_caches("bf16", 64, 16, 8, 128, g)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    fd.fd_cache_append(k, v, slots, kc, vc, stream=s)
    s.synchronize()
    assert torch.equal(kc[:, 0], k) and torch.equal(vc[:, 0], v)
