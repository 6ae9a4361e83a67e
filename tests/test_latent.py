"""Latent attention: the absorbed decode and the expanded prompt form. The
oracle's pins and the C ABI's refusals on the CPU (nothing is launched), the
kernels against the float64 oracle on the GPU."""
import math

import numpy as np
import pytest
import torch

import split_kv_paged_gqa_gb300 as fd
from oracle.latent_ref import latent_decode_ref, latent_prefill_ref

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32
SCALE = 1.0 / math.sqrt(192)


def f64(t):
    return t.detach().double().cpu().numpy()


# ---------------------------------------------------------------------------
# the oracle, pinned


def test_oracle_forms_agree():
    """Absorbing the up-projections into query and output gives the expanded
    form's attention: the two oracles on one model's data."""
    rng = np.random.default_rng(1)
    L, H = 9, 3
    c, pe = rng.normal(size=(L, 512)), rng.normal(size=(L, 64))
    wk, wv = rng.normal(size=(H, 128, 512)) / 16, rng.normal(size=(H, 128, 512)) / 16
    qn, qp = rng.normal(size=(L, H, 128)), rng.normal(size=(L, H, 64))
    k, v = np.einsum("hdc,lc->lhd", wk, c), np.einsum("hdc,lc->lhd", wv, c)
    o, lse, _, _ = latent_prefill_ref(np.concatenate([qn, qp], -1), k, pe, v, [0, L], [0, L], SCALE)
    qa = np.concatenate([np.einsum("lhd,hdc->lhc", qn, wk), qp], -1)
    cache = np.full((2, 8, 576), np.nan)      # nothing past the last key may be read
    flat = cache.reshape(-1, 576)
    flat[:L] = np.concatenate([c, pe], -1)
    oa, la, _, _ = latent_decode_ref(qa[None], cache, np.array([[0, 1]]), [L], SCALE)
    np.testing.assert_allclose(np.einsum("hdc,lhc->lhd", wv, oa[0]), o, rtol=1e-9, atol=1e-12)
    np.testing.assert_allclose(la[0], lse, rtol=1e-12)


def test_oracle_closed_forms():
    one = latent_decode_ref(np.ones((1, 1, 2, 576)), np.arange(8 * 576.0).reshape(1, 8, 576), np.array([[0]]), [1], 0.5)
    assert (one[0][0, 0] == np.arange(512.0)).all() and one[1][0, 0, 0] == 0.5 * np.arange(576.0).sum()
    none = latent_decode_ref(np.ones((1, 2, 1, 576)), np.ones((1, 8, 576)), np.array([[0]]), [1], 0.5)
    assert (none[0][0, 0] == 0).all() and none[1][0, 0, 0] == -np.inf and np.isfinite(none[1][0, 1, 0])
    # more queries than keys: the first rows see nothing
    o, lse, _, _ = latent_prefill_ref(np.ones((3, 1, 192)), np.ones((1, 1, 128)), np.ones((1, 64)), np.full((1, 1, 128), 7.0),
                                      [0, 3], [0, 1], 1.0)
    assert np.isneginf(lse[:2]).all() and (o[:2] == 0).all() and lse[2, 0] == 192 and (o[2] == 7).all()


# ---------------------------------------------------------------------------
# refusals (host tensors; a host-only plan or an argument that is refused first)


def _plan_kw(**kw):
    return {**dict(device=-1, max_batch=4, max_q_per_req=2, num_heads=8, page_size=16, softmax_scale=SCALE), **kw}


@pytest.mark.parametrize("change,status", [
    (dict(max_batch=0), fd.FD_ERR_INVALID_ARG), (dict(max_q_per_req=65), fd.FD_ERR_INVALID_ARG),
    (dict(num_heads=0), fd.FD_ERR_INVALID_ARG), (dict(num_heads=1025), fd.FD_ERR_INVALID_ARG),
    (dict(page_size=24), fd.FD_ERR_UNSUPPORTED), (dict(page_size=4), fd.FD_ERR_UNSUPPORTED),
    (dict(page_size=512), fd.FD_ERR_UNSUPPORTED), (dict(softmax_scale=0.0), fd.FD_ERR_INVALID_ARG),
    (dict(softmax_scale=math.inf), fd.FD_ERR_INVALID_ARG), (dict(softmax_scale=math.nan), fd.FD_ERR_INVALID_ARG),
])
def test_plan_rejects(change, status):
    with pytest.raises(fd.FdError) as e:
        fd.fd_latent_plan_create(**_plan_kw(**change))
    assert e.value.status == status


def _decode_args(B=2, Tq=1, H=8, P=16, N=10, W=4, device="cpu"):
    return dict(q=torch.zeros(B, Tq, H, 576, dtype=BF, device=device), kv_cache=torch.zeros(N, P, 576, dtype=BF, device=device),
                page_table=torch.zeros(B, W, dtype=I32, device=device), cache_seqlens=torch.zeros(B, dtype=I32, device=device),
                q_per_req=Tq, out=torch.zeros(B, Tq, H, 512, dtype=BF, device=device),
                lse=torch.zeros(B, Tq, H, dtype=F32, device=device))


@pytest.mark.parametrize("change,status", [
    ({}, fd.FD_ERR_WORKSPACE),                                            # valid: reaches the host-only plan's refusal
    (dict(lse=None), fd.FD_ERR_WORKSPACE),
    (dict(out=torch.zeros(2, 1, 8, 512)), fd.FD_ERR_WORKSPACE),
    (dict(q=torch.zeros(2, 1, 8, 576)), fd.FD_ERR_INVALID_ARG),
    (dict(q=torch.zeros(2, 1, 8, 512, dtype=BF)), fd.FD_ERR_INVALID_ARG),
    (dict(q=torch.zeros(2, 1, 4, 576, dtype=BF)), fd.FD_ERR_INVALID_ARG),
    (dict(q=torch.zeros(0, 1, 8, 576, dtype=BF)), fd.FD_ERR_INVALID_ARG),
    (dict(q=torch.zeros(5, 1, 8, 576, dtype=BF)), fd.FD_ERR_INVALID_ARG),
    (dict(q=torch.zeros(2, 1, 8, 577, dtype=BF)[..., :576]), fd.FD_ERR_UNSUPPORTED),
    (dict(q=None), fd.FD_ERR_INVALID_ARG),
    (dict(q_per_req=2), fd.FD_ERR_INVALID_ARG),
    (dict(kv_cache=torch.zeros(10, 16, 1, 576, dtype=BF)), fd.FD_ERR_INVALID_ARG),
    (dict(kv_cache=torch.zeros(10, 8, 576, dtype=BF)), fd.FD_ERR_INVALID_ARG),
    (dict(kv_cache=torch.zeros(10, 16, 576, dtype=torch.int8)), fd.FD_ERR_INVALID_ARG),
    (dict(kv_cache=torch.zeros(10, 16, 580, dtype=BF)[..., :576]), fd.FD_ERR_UNSUPPORTED),
    (dict(page_table=torch.zeros(3, 4, dtype=I32)), fd.FD_ERR_INVALID_ARG),
    (dict(page_table=torch.zeros(2, 4, dtype=torch.int64)), fd.FD_ERR_INVALID_ARG),
    (dict(cache_seqlens=torch.zeros(3, dtype=I32)), fd.FD_ERR_INVALID_ARG),
    (dict(out=torch.zeros(2, 1, 8, 576, dtype=BF)), fd.FD_ERR_INVALID_ARG),
    (dict(out=torch.zeros(2, 1, 8, 512, dtype=I32)), fd.FD_ERR_INVALID_ARG),
    (dict(lse=torch.zeros(2, 1, 7)), fd.FD_ERR_INVALID_ARG),
])
def test_decode_rejects(change, status):
    plan = fd.fd_latent_plan_create(**_plan_kw())
    try:
        fd.fd_set_plan(plan)
        with pytest.raises(fd.FdError) as e:
            fd.fd_decode_latent(**{**_decode_args(), **change}, stream=0)
        assert e.value.status == status, str(e.value)
    finally:
        fd.fd_set_plan(None)
        fd.fd_plan_destroy(plan)


def test_plan_kinds_do_not_mix():
    plan = fd.fd_latent_plan_create(**_plan_kw())
    other = fd.fd_plan_create(-1, 4, 1, 8, 2, 128, 16, "bf16", 4)
    try:
        fd.fd_set_plan(None)
        with pytest.raises(fd.FdError) as e:
            fd.fd_decode_latent(**_decode_args(), stream=0)
        assert e.value.status == fd.FD_ERR_NO_PLAN
        fd.fd_set_plan(other)
        with pytest.raises(fd.FdError) as e:
            fd.fd_decode_latent(**_decode_args(), stream=0)
        assert e.value.status == fd.FD_ERR_INVALID_ARG
        fd.fd_set_plan(plan)
        z = torch.zeros(2, 1, 8, 128, dtype=BF)
        c = torch.zeros(4, 16, 2, 128, dtype=BF)
        with pytest.raises(fd.FdError) as e:
            fd.fd_decode_paged(z, c, c, None, torch.zeros(2, 4, dtype=I32), torch.zeros(2, dtype=I32), 1, 1, z, None, stream=0)
        assert e.value.status == fd.FD_ERR_INVALID_ARG
        for call in (lambda: fd.fd_plan_set_split_policy(plan, "equal"), lambda: fd.fd_query_splits(plan, 1, 100),
                     lambda: fd.fd_set_max_seqlen_hint(plan, 5), lambda: fd.fd_set_mean_seqlen_hint(plan, 5),
                     lambda: fd.fd_autotune_stats(plan), lambda: fd.fd_profile_begin(plan),
                     lambda: fd.fd_autotune_clear(plan), lambda: fd.fd_autotune_set_cache_dir(plan, "/nonexistent"),
                     lambda: fd.fd_autotune_set_timer(plan, lambda b, k, s: 1.0),
                     lambda: fd.fd_autotune(plan, [1], stream=0)):
            with pytest.raises(fd.FdError) as e:
                call()
            assert e.value.status == fd.FD_ERR_UNSUPPORTED
        assert fd.fd_plan_workspace_bytes(plan) == 0
    finally:
        fd._timers.pop(plan, None)
        fd.fd_set_plan(None)
        fd.fd_plan_destroy(plan)
        fd.fd_plan_destroy(other)


def test_profile_end_refuses_a_latent_plan():
    plan = fd.fd_latent_plan_create(**_plan_kw())
    try:
        with pytest.raises(fd.FdError) as e:
            fd.fd_profile_end(plan)
        assert e.value.status == fd.FD_ERR_UNSUPPORTED
    finally:
        fd.fd_plan_destroy(plan)


def test_refused_callbacks_are_not_kept():
    """(A later plan may get the handle, and would seem to have them.)"""
    plan = fd.fd_latent_plan_create(**_plan_kw())
    try:
        for call in (lambda: fd.fd_autotune_set_timer(plan, lambda b, k, s: 1.0),
                     lambda: fd.fd_autotune_set_input_hook(plan, lambda *a: None)):
            with pytest.raises(fd.FdError) as e:
                call()
            assert e.value.status == fd.FD_ERR_UNSUPPORTED
        assert plan not in fd._timers and plan not in fd._input_hooks
    finally:
        fd.fd_plan_destroy(plan)


def _prefill_args(Sq=6, Sk=9, H=4, B=2, device="cpu"):
    z = lambda *s: torch.zeros(*s, dtype=BF, device=device)   # noqa: E731
    return dict(q=z(Sq, H, 192), k_nope=z(Sk, H, 128), k_pe=z(Sk, 64), v=z(Sk, H, 128),
                cu_seqlens_q=torch.zeros(B + 1, dtype=I32, device=device),
                cu_seqlens_k=torch.zeros(B + 1, dtype=I32, device=device), max_seqlen_q=6, softmax_scale=0.0,
                out=z(Sq, H, 128), lse=torch.zeros(Sq, H, device=device), status=None)


@pytest.mark.parametrize("change,status", [
    (dict(q=torch.zeros(6, 4, 192)), fd.FD_ERR_INVALID_ARG),
    (dict(q=torch.zeros(6, 4, 128, dtype=BF)), fd.FD_ERR_INVALID_ARG),
    (dict(q=torch.zeros(0, 4, 192, dtype=BF)), fd.FD_ERR_INVALID_ARG),
    (dict(q=torch.zeros(6, 4, 196, dtype=BF)[..., 2:194]), fd.FD_ERR_UNSUPPORTED),
    (dict(k_nope=torch.zeros(9, 3, 128, dtype=BF)), fd.FD_ERR_INVALID_ARG),
    (dict(k_nope=torch.zeros(4, 9, 128, dtype=BF).transpose(0, 1)[..., ::2]), fd.FD_ERR_UNSUPPORTED),
    (dict(k_pe=torch.zeros(8, 64, dtype=BF)), fd.FD_ERR_INVALID_ARG),
    (dict(k_pe=torch.zeros(9, 68, dtype=BF)[:, :64]), fd.FD_ERR_UNSUPPORTED),
    (dict(v=torch.zeros(8, 4, 128, dtype=BF)), fd.FD_ERR_INVALID_ARG),
    (dict(cu_seqlens_q=torch.zeros(3, dtype=torch.int64)), fd.FD_ERR_INVALID_ARG),
    (dict(cu_seqlens_q=torch.zeros(1, dtype=I32)), fd.FD_ERR_INVALID_ARG),
    (dict(cu_seqlens_k=torch.zeros(4, dtype=I32)), fd.FD_ERR_INVALID_ARG),
    (dict(max_seqlen_q=0), fd.FD_ERR_INVALID_ARG),
    (dict(softmax_scale=-1.0), fd.FD_ERR_INVALID_ARG),
    (dict(softmax_scale=math.nan), fd.FD_ERR_INVALID_ARG),
    (dict(out=torch.zeros(6, 4, 192, dtype=BF)), fd.FD_ERR_INVALID_ARG),
    (dict(lse=torch.zeros(6, 3)), fd.FD_ERR_INVALID_ARG),
    (dict(status=torch.zeros(1)), fd.FD_ERR_INVALID_ARG),
])
def test_prefill_rejects(change, status):
    with pytest.raises(fd.FdError) as e:
        fd.fd_prefill_latent(**{**_prefill_args(), **change}, stream=0)
    assert e.value.status == status, str(e.value)


@pytest.mark.parametrize("name,shape", [("q", (6, 4, 192)), ("k_nope", (9, 4, 128)), ("k_pe", (9, 64)), ("v", (9, 4, 128))])
def test_prefill_rejects_broadcast(name, shape):
    for d in range(len(shape) - 1):
        t = torch.zeros([1 if i == d else n for i, n in enumerate(shape)], dtype=BF).expand(shape)
        with pytest.raises(fd.FdError) as e:
            fd.fd_prefill_latent(**{**_prefill_args(), name: t}, stream=0)
        assert e.value.status == fd.FD_ERR_UNSUPPORTED


@pytest.mark.parametrize("change", [
    dict(kv_cache=torch.zeros(1, 16, 576, dtype=BF).expand(10, 16, 576)),
    dict(kv_cache=torch.zeros(10, 1, 576, dtype=BF).expand(10, 16, 576)),
    dict(page_table=torch.empty(1, (2 ** 31 - 256) // 16 + 1, dtype=I32).expand(2, -1)),   # (never touched)
])
def test_decode_rejects_broadcast_caches_and_widest_tables(change):
    test_decode_rejects(change, fd.FD_ERR_UNSUPPORTED)


@pytest.mark.parametrize("name,full,dtype", [("out", (2, 2, 8, 512), BF), ("lse", (2, 2, 8), F32)])
def test_decode_rejects_broadcast_outputs(name, full, dtype):
    plan = fd.fd_latent_plan_create(**_plan_kw())
    try:
        fd.fd_set_plan(plan)
        for d in range(3):
            t = torch.zeros([1 if i == d else n for i, n in enumerate(full)], dtype=dtype).expand(full)
            with pytest.raises(fd.FdError) as e:
                fd.fd_decode_latent(**{**_decode_args(Tq=2), name: t}, stream=0)
            assert e.value.status == fd.FD_ERR_UNSUPPORTED
    finally:
        fd.fd_set_plan(None)
        fd.fd_plan_destroy(plan)


@pytest.mark.parametrize("name,full,dtype", [("out", (6, 4, 128), BF), ("lse", (6, 4), F32)])
def test_prefill_rejects_broadcast_outputs(name, full, dtype):
    for d in range(2):
        t = torch.zeros([1 if i == d else n for i, n in enumerate(full)], dtype=dtype).expand(full)
        with pytest.raises(fd.FdError) as e:
            fd.fd_prefill_latent(**{**_prefill_args(), name: t}, stream=0)
        assert e.value.status == fd.FD_ERR_UNSUPPORTED


# ---------------------------------------------------------------------------
# the decode kernel against the oracle


def make_decode(lens, Tq, H, P, seed, extra=3, spread=1.0, strided=False):
    """Inputs on the GPU; every cache slot that no request owns holds NaN, and
    page-table entries past a request's pages point outside the pool."""
    rng = np.random.default_rng(seed)
    B = len(lens)
    pages = [-(-n // P) for n in lens]
    W, N = max(1, max(pages)) + 1, sum(pages) + extra
    order = rng.permutation(N)
    g = torch.Generator().manual_seed(seed)
    cache = torch.full((N, P, 576), math.nan, dtype=BF)
    table = torch.full((B, W), 1 << 30, dtype=I32)
    at = 0
    for b, n in enumerate(lens):
        ids = order[at:at + pages[b]]
        at += pages[b]
        table[b, :pages[b]] = torch.from_numpy(ids.astype(np.int32))
        rows = (torch.randn(n, 576, generator=g) * spread).to(BF)
        for i, pid in enumerate(ids):
            part = rows[i * P:(i + 1) * P]
            cache[int(pid), :part.shape[0]] = part
    q = torch.randn(B, Tq, H, 576, generator=g).to(BF)
    if strided:   # a cache of wider rows, queries with heads outermost
        wide = torch.full((N, P, 640), math.nan, dtype=BF)
        wide[..., 8:584] = cache
        cache = wide.cuda()[..., 8:584]
        q = q.permute(2, 0, 1, 3).contiguous().cuda().permute(1, 2, 0, 3)
    return dict(q=q.cuda(), kv_cache=cache.cuda(), page_table=table.cuda(),
                cache_seqlens=torch.tensor(lens, dtype=I32).cuda(), q_per_req=Tq)


def run_decode(a, plan, out_dtype=BF, stream=None):
    B, Tq, H, _ = a["q"].shape
    out = torch.full((B, Tq, H, 512), 768.0, dtype=out_dtype, device="cuda")
    lse = torch.full((B, Tq, H), 768.0, device="cuda")
    fd.fd_set_plan(plan)
    try:
        fd.fd_decode_latent(**a, out=out, lse=lse, stream=stream)
    finally:
        fd.fd_set_plan(None)
    return out, lse


def check(out, lse, ref, where=""):
    o, s, tol, ltol = ref
    got, gl = f64(out), f64(lse)
    assert np.array_equal(np.isneginf(gl), np.isneginf(s)), f"{where}: rows without keys differ"
    live = np.isfinite(s)
    worst = np.abs(gl[live] - s[live]) - ltol[live]
    assert worst.size == 0 or worst.max() <= 0, f"{where}: lse off by {worst.max():.2e} more than its bound"
    over = np.abs(got - o) - tol
    assert np.isfinite(got).all() and over.max() <= 0, f"{where}: out off by {over.max():.2e} more than its bound"


def decode_case(lens, Tq, H, P, seed, out_dtype=BF, plan=None, **kw):
    a = make_decode(lens, Tq, H, P, seed, **kw)
    own = plan is None
    plan = plan or fd.fd_latent_plan_create(0, len(lens), Tq, H, P, SCALE)
    try:
        out, lse = run_decode(a, plan, out_dtype)
        assert fd.fd_read_device_status(plan) == 0
    finally:
        if own:
            fd.fd_plan_destroy(plan)
    ref = latent_decode_ref(f64(a["q"]), f64(a["kv_cache"]), a["page_table"].cpu().numpy(), lens, SCALE,
                            16 if out_dtype == BF else 32)
    check(out, lse, ref, f"lens {lens} Tq {Tq} H {H} P {P}")


@pytest.mark.gpu
@pytest.mark.parametrize("L", [0, 1, 2, 7, 8, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 191, 192, 193, 257, 640])
def test_decode_lengths(L):
    decode_case([L], 1, 16, 16, 100 + L)


@pytest.mark.gpu
@pytest.mark.parametrize("P", [8, 16, 32, 64, 128, 256])
@pytest.mark.parametrize("Tq", [1, 3])
def test_decode_pages(P, Tq):
    decode_case([700, 1, 0, P, P + 1, 3 * P - 1, 513], Tq, 8, P, P + Tq)


@pytest.mark.gpu
@pytest.mark.parametrize("H,Tq", [(1, 1), (2, 1), (3, 5), (5, 1), (16, 4), (20, 1), (32, 2), (40, 1), (63, 1), (64, 1),
                                  (65, 1), (66, 2), (96, 1), (128, 1), (128, 3), (160, 1), (1, 64), (257, 1)])
def test_decode_heads(H, Tq):
    decode_case([130, 0, Tq - 1, Tq, 333], Tq, H, 32, 7 * H + Tq)


@pytest.mark.gpu
def test_decode_ragged_batch():
    rng = np.random.default_rng(3)
    lens = [int(x) for x in np.exp(rng.uniform(0, np.log(1500), size=70))]
    lens[5] = lens[40] = 0
    decode_case(lens, 2, 4, 16, 5)


@pytest.mark.gpu
def test_decode_long_batches_of_one():
    decode_case([9001], 1, 16, 64, 11)
    decode_case([12345], 1, 3, 8, 12)


@pytest.mark.gpu
@pytest.mark.parametrize("out_dtype", [BF, F32])
def test_decode_strides_and_types(out_dtype):
    decode_case([75, 200, 1], 2, 12, 16, 21, out_dtype, strided=True)


@pytest.mark.gpu
def test_decode_large_scores():
    """Scores whose maximum moves far from block to block: rescaling matters."""
    decode_case([1500, 300], 1, 16, 64, 31, spread=12.0)


@pytest.mark.gpu
def test_decode_needles():
    """One key that takes all the weight, placed at tile and page borders."""
    lens = [1030]
    for j in (0, 63, 64, 127, 128, 511, 1023, 1024, 1029):
        a = make_decode(lens, 1, 16, 16, 50 + j)
        pid, slot = int(a["page_table"][0, j // 16]), j % 16
        a["kv_cache"][pid, slot] = a["q"][0, 0, 3].to(BF) * 4
        plan = fd.fd_latent_plan_create(0, 1, 1, 16, 16, SCALE)
        out, lse = run_decode(a, plan)
        assert fd.fd_read_device_status(plan) == 0
        fd.fd_plan_destroy(plan)
        assert torch.equal(out[0, 0, 3], a["kv_cache"][pid, slot, :512]), f"needle {j}"
        check(out, lse, latent_decode_ref(f64(a["q"]), f64(a["kv_cache"]), a["page_table"].cpu().numpy(), lens, SCALE))


@pytest.mark.gpu
def test_decode_repeats_bitwise_and_smaller_calls_on_one_plan():
    plan = fd.fd_latent_plan_create(0, 9, 4, 24, 16, SCALE)
    try:
        a = make_decode([900, 33, 0, 1, 2100, 64, 65, 10, 400], 4, 24, 16, 61)
        first = run_decode(a, plan)
        decode_case([500], 1, 24, 16, 62, plan=plan)
        decode_case([50, 0], 3, 24, 16, 63, plan=plan)
        for _ in range(5):
            again = run_decode(a, plan)
            assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
        big = make_decode([10] * 10, 1, 24, 16, 64)
        with pytest.raises(fd.FdError):
            run_decode(big, plan)
    finally:
        fd.fd_plan_destroy(plan)


@pytest.mark.gpu
def test_decode_records_bad_metadata():
    plan = fd.fd_latent_plan_create(0, 2, 1, 8, 16, SCALE)
    try:
        a = make_decode([100, 40], 1, 8, 16, 71)
        a["page_table"][0, 2] = -1
        out, lse = run_decode(a, plan)
        assert fd.fd_read_device_status(plan) == fd.FD_DEVSTAT_BAD_PAGE
        ref = latent_decode_ref(f64(a["q"][1:]), f64(a["kv_cache"]), a["page_table"][1:].cpu().numpy(), [40], SCALE)
        check(out[1:], lse[1:], ref)                       # the other request is untouched
        a["page_table"][0, 2] = a["kv_cache"].shape[0]
        run_decode(a, plan)
        assert fd.fd_read_device_status(plan) == fd.FD_DEVSTAT_BAD_PAGE
        a = make_decode([100, 40], 1, 8, 16, 71)
        a["cache_seqlens"][1] = -5
        out, lse = run_decode(a, plan)
        assert fd.fd_read_device_status(plan) == fd.FD_DEVSTAT_SEQLEN_OVERFLOW
        assert (out[1] == 0).all() and torch.isneginf(lse[1]).all()
        a["page_table"].clamp_(max=3)
        a["cache_seqlens"][1] = 16 * a["page_table"].shape[1] + 1     # clamped to the table's capacity
        run_decode(a, plan)
        assert fd.fd_read_device_status(plan) == fd.FD_DEVSTAT_SEQLEN_OVERFLOW
    finally:
        fd.fd_plan_destroy(plan)


@pytest.mark.gpu
def test_decode_in_a_graph():
    """Captured once, replayed with new queries, pages and lengths (zero among
    them), on a side stream."""
    plan = fd.fd_latent_plan_create(0, 5, 2, 16, 16, SCALE)
    lens = [400, 31, 1, 900, 64]
    a = make_decode(lens, 2, 16, 16, 81)
    out = torch.empty(5, 2, 16, 512, dtype=BF, device="cuda")
    lse = torch.empty(5, 2, 16, device="cuda")
    fd.fd_set_plan(plan)
    try:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            fd.fd_decode_latent(**a, out=out, lse=lse)
        side = torch.cuda.Stream()
        for k, new in enumerate(([400, 31, 1, 900, 64], [0, 900, 17, 3, 2], [1, 1, 1, 1, 1])):
            b = make_decode(new, 2, 16, 16, 90 + k)
            n = min(a["kv_cache"].shape[0], b["kv_cache"].shape[0])
            ids = torch.where(b["page_table"] < n, b["page_table"], 0)
            a["kv_cache"].fill_(0)
            a["kv_cache"][:n].copy_(b["kv_cache"][:n].nan_to_num(0.0))
            a["page_table"].fill_(0)
            w = min(a["page_table"].shape[1], ids.shape[1])
            a["page_table"][:, :w].copy_(ids[:, :w])
            a["cache_seqlens"].copy_(torch.tensor(new, dtype=I32))
            a["q"].copy_(b["q"])
            torch.cuda.synchronize()
            with torch.cuda.stream(side):
                g.replay()
            side.synchronize()
            assert fd.fd_read_device_status(plan) == 0
            ref = latent_decode_ref(f64(a["q"]), f64(a["kv_cache"]), a["page_table"].cpu().numpy(), new, SCALE)
            check(out, lse, ref, f"replay {k}")
        del g
    finally:
        fd.fd_set_plan(None)
        fd.fd_plan_destroy(plan)


@pytest.mark.gpu
def test_decode_far_rows():
    """A cache whose last pages lie past 2^31 elements from its start."""
    P, N = 64, (1 << 31) // (64 * 576) + 40
    cache = torch.empty(N, P, 576, dtype=BF, device="cuda")
    lens = [200, 64]
    a = make_decode(lens, 1, 8, P, 101)
    n = a["kv_cache"].shape[0]
    cache[N - n:].copy_(a["kv_cache"])
    near = f64(a["kv_cache"])
    table = a["page_table"].cpu().numpy()
    a["page_table"].copy_(torch.where(a["page_table"] < n, a["page_table"] + (N - n), a["page_table"]))
    a["kv_cache"] = cache
    plan = fd.fd_latent_plan_create(0, 2, 1, 8, P, SCALE)
    out, lse = run_decode(a, plan)
    assert fd.fd_read_device_status(plan) == 0
    fd.fd_plan_destroy(plan)
    check(out, lse, latent_decode_ref(f64(a["q"]), near, table, lens, SCALE))


@pytest.mark.gpu
@pytest.mark.parametrize("P", [8, 16, 32, 64, 128, 256])
@pytest.mark.parametrize("strided", [False, True])
def test_decode_several_row_tiles(P, strided):
    """Tiles that several CTAs read, over contiguous and over wider cache rows;
    ids outside the pool behind the first tile are recorded and read as nothing."""
    decode_case([700, 64, 0, 65, 129], 1, 130, P, 61, strided=strided)
    a = make_decode([900, 300], 1, 130, P, 62, strided=strided)
    plan = fd.fd_latent_plan_create(0, 2, 1, 130, P, SCALE)
    clean = run_decode(a, plan)
    for bad in (-1, 1 << 30):
        a["page_table"][0, 800 // P] = bad
        out, lse = run_decode(a, plan)
        assert fd.fd_read_device_status(plan) == fd.FD_DEVSTAT_BAD_PAGE
        assert torch.equal(out[1], clean[0][1]) and torch.equal(lse[1], clean[1][1])
    fd.fd_plan_destroy(plan)


@pytest.mark.gpu
@pytest.mark.parametrize("B,H,Tq", [(300, 4, 1), (1, 1024, 1), (130, 3, 64), (2, 200, 64)])
def test_decode_many_requests_or_rows(B, H, Tq):
    rng = np.random.default_rng(B + H)
    decode_case([int(x) for x in rng.integers(0, 90, size=B)], Tq, H, 8, 31)


@pytest.mark.gpu
@pytest.mark.parametrize("H,lens", [(16, [300, 9000, 90]), (16, [300] * 40 + [9000] + [90] * 160), (128, [20000, 64, 7000])])
def test_decode_keeps_nan(H, lens):
    """A NaN in a visible key reaches every row of its request, also where the
    keys are split over CTAs, and no other request."""
    a = make_decode(lens, 1, H, 64, 41)
    plan = fd.fd_latent_plan_create(0, len(lens), 1, H, 64, SCALE)
    clean = run_decode(a, plan)
    for b in {int(np.argmax(lens)), len(lens) - 1}:
        L = lens[b]
        for keys in ([L // 3], range(L)):
            cache = a["kv_cache"].clone()
            for pages in [a["page_table"][b, torch.tensor(sorted({k // 64 for k in keys})).cuda()].long()]:
                if len(keys) == 1:
                    cache[pages[0], keys[0] % 64, 7] = math.nan
                else:
                    cache[pages] = math.nan
            out, lse = run_decode({**a, "kv_cache": cache}, plan)
            assert out[b].isnan().all(dim=-1).all() if len(keys) > 1 else out[b].isnan().any(dim=-1).all()
            assert lse[b].isnan().all()
            rest = [x for x in range(len(lens)) if x != b]
            assert torch.equal(out[rest], clean[0][rest]) and torch.equal(lse[rest], clean[1][rest])
    fd.fd_plan_destroy(plan)


@pytest.mark.gpu
def test_decode_two_graphs_on_one_plan_and_plans_on_two_streams():
    plan, other = (fd.fd_latent_plan_create(0, 3, 2, 16, 16, SCALE) for _ in range(2))
    x, y = make_decode([900, 3, 2000], 2, 16, 16, 51), make_decode([70, 4000], 1, 16, 16, 52)
    want = run_decode(x, plan), run_decode(y, plan)
    graphs, got = [], []
    fd.fd_set_plan(plan)
    for a in (x, y):
        B, Tq, H, _ = a["q"].shape
        o, s = torch.empty(B, Tq, H, 512, dtype=BF, device="cuda"), torch.empty(B, Tq, H, device="cuda")
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            fd.fd_decode_latent(**a, out=o, lse=s)
        graphs.append(g)
        got.append((o, s))
    for _ in range(5):                  # in turn on one stream
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for (o, s), (wo, ws) in zip(got, want):
        assert torch.equal(o, wo) and torch.equal(s, ws)
    streams, res = [torch.cuda.Stream(), torch.cuda.Stream()], []
    for _ in range(8):                  # at once, a plan each
        for st, p, a in zip(streams, (plan, other), (x, y)):
            with torch.cuda.stream(st):
                res.append(run_decode(a, p))
    torch.cuda.synchronize()
    for k, (o, s) in enumerate(res):
        assert torch.equal(o, want[k % 2][0]) and torch.equal(s, want[k % 2][1])
    del graphs
    fd.fd_plan_destroy(plan)
    fd.fd_plan_destroy(other)


# ---------------------------------------------------------------------------
# the prompt kernel against the oracle


def make_prefill(lq, lk, H, seed, joint=True, pad=0, spread=1.0):
    """Ragged inputs on the GPU; `pad` rows before the first and behind the last
    request hold NaN."""
    g = torch.Generator().manual_seed(seed)
    Sq, Sk = sum(lq) + 2 * pad, sum(lk) + 2 * pad
    q = (torch.randn(Sq, H, 192, generator=g) * spread).to(BF)
    kv = torch.randn(Sk, H, 256, generator=g).to(BF)
    pe = torch.randn(Sk, 64, generator=g).to(BF)
    if pad:
        for t in (q, kv, pe):
            t[:pad] = math.nan
            t[t.shape[0] - pad:] = math.nan
    q, kv, pe = q.cuda(), kv.cuda(), pe.cuda()
    k, v = kv[..., :128], kv[..., 128:]
    if not joint:
        q = q.transpose(0, 1).contiguous().transpose(0, 1)      # heads outermost
        k = k.transpose(0, 1).contiguous().transpose(0, 1)
        v = v.contiguous()
        wide = torch.full((Sk, 576), math.nan, dtype=BF, device="cuda")   # a view of latent rows
        wide[:, 512:] = pe
        pe = wide[:, 512:]
    cu = lambda n: torch.tensor(np.concatenate([[0], np.cumsum(n)]) + pad, dtype=I32).cuda()   # noqa: E731
    return dict(q=q, k_nope=k, k_pe=pe, v=v, cu_seqlens_q=cu(lq), cu_seqlens_k=cu(lk), max_seqlen_q=max(1, max(lq)),
                softmax_scale=SCALE)


def run_prefill(a, out_dtype=BF):
    Sq, H, _ = a["q"].shape
    out = torch.full((Sq, H, 128), 768.0, dtype=out_dtype, device="cuda")
    lse = torch.full((Sq, H), 768.0, device="cuda")
    status = torch.zeros(1, dtype=I32, device="cuda")
    fd.fd_prefill_latent(**a, out=out, lse=lse, status=status)
    return out, lse, status


def prefill_case(lq, lk, H, seed, out_dtype=BF, **kw):
    a = make_prefill(lq, lk, H, seed, **kw)
    out, lse, status = run_prefill(a, out_dtype)
    assert int(status) == 0
    ref = latent_prefill_ref(*(f64(a[k]) for k in ("q", "k_nope", "k_pe", "v")), a["cu_seqlens_q"].cpu().numpy(),
                             a["cu_seqlens_k"].cpu().numpy(), SCALE, 16 if out_dtype == BF else 32)
    mine = ~np.isnan(ref[1][:, 0])
    assert (f64(out)[~mine] == 768).all() and (f64(lse)[~mine] == 768).all(), "rows of no request were written"
    check(out[torch.from_numpy(mine)], lse[torch.from_numpy(mine)], tuple(x[mine] for x in ref), f"lq {lq} lk {lk} H {H}")


@pytest.mark.gpu
@pytest.mark.parametrize("n", [1, 2, 15, 16, 31, 63, 64, 65, 127, 128, 129, 191, 255, 256, 257, 385, 600])
def test_prefill_lengths(n):
    prefill_case([n], [n], 2, 200 + n)


@pytest.mark.gpu
@pytest.mark.parametrize("lq,lk", [([1], [700]), ([130], [129]), ([300], [40]), ([5], [0]), ([64], [64 + 128]), ([100], [357]),
                                   ([257], [514]), ([3, 0, 200, 1], [3, 50, 333, 1]), ([128, 128, 0], [0, 128, 7])])
def test_prefill_prefixes(lq, lk):
    if sum(lk) == 0:       # tensors are never empty: a second request brings the key
        lq, lk = lq + [0], lk + [1]
    prefill_case(lq, lk, 3, 300 + sum(lq) + sum(lk))


@pytest.mark.gpu
@pytest.mark.parametrize("out_dtype", [BF, F32])
@pytest.mark.parametrize("joint", [True, False])
def test_prefill_strides_padding_types(out_dtype, joint):
    prefill_case([70, 1, 140], [70, 9, 200], 4, 401, out_dtype, joint=joint, pad=5)


@pytest.mark.gpu
def test_prefill_many_requests_and_heads():
    rng = np.random.default_rng(8)
    lq = [int(x) for x in rng.integers(0, 90, size=40)]
    lk = [a + int(x) for a, x in zip(lq, rng.integers(0, 60, size=40))]
    prefill_case(lq, lk, 1, 402)
    prefill_case([33, 150], [33, 150], 17, 403)


@pytest.mark.gpu
@pytest.mark.parametrize("B,long_at", [(2, 0), (5, 3), (33, 32), (70, 1)])
def test_prefill_one_long_among_short(B, long_at):
    """Fewer tiles than the longest request's for each: found on the device."""
    rng = np.random.default_rng(B)
    lq = [int(x) for x in rng.integers(0, 40, size=B)]
    lq[long_at], lq[B // 2] = 1700, 300
    prefill_case(lq, [x + int(y) for x, y in zip(lq, rng.integers(0, 50, size=B))], 2, 407 + B)


@pytest.mark.gpu
def test_prefill_bad_rows_among_many():
    """A ragged batch whose offsets go back: recorded, requests before them run,
    nothing outside is written."""
    n = [900] + [20] * 40
    a = make_prefill(n, n, 2, 409)
    clean = run_prefill(a)
    for at, value in ((38, 5), (38, 1 << 30), (38, -1), (0, 3000)):
        b = {**a, "cu_seqlens_q": a["cu_seqlens_q"].clone()}
        b["cu_seqlens_q"][at] = value
        out, lse, status = run_prefill(b)
        assert int(status) == fd.FD_DEVSTAT_SEQLEN_OVERFLOW
        if at:
            sure = int(a["cu_seqlens_q"][37])                  # requests 0 .. 36
            assert torch.equal(out[:sure], clean[0][:sure]) and torch.equal(lse[:sure], clean[1][:sure])
            assert (out[sure:int(a["cu_seqlens_q"][38])] == 768).all()


@pytest.mark.gpu
@pytest.mark.parametrize("cu_q,good", [([0, 100, 50, 120], [1, 0, 0]), ([0, 100, 50, 80], [1, 0, 0]), ([100, 100, 50, 120], [1, 0, 0]),
                                       ([0, 60, 40, 60, 130], [1, 0, 0, 1]), ([0, 400, 30, 90], [0, 0, 1]),
                                       ([0, 70, 20, 70, 60, 140], [1, 0, 0, 0, 0])])
@pytest.mark.parametrize("ragged", [False, True])
def test_prefill_rows_belong_to_the_first_request(cu_q, good, ragged):
    """A request that begins before the end of an earlier one with good rows is
    recorded and left out, whichever way the call's tiles are placed: the earlier
    one's rows are as without it, and nobody else's are written."""
    B, Sq = len(cu_q) - 1, 130 if not ragged else 2100
    a = make_prefill([Sq], [130 * B], 2, 408)      # (keys enough that each row sees some)
    many = 60 if ragged else 0        # room for 2000 queries each: tiles are found on the device
    a["max_seqlen_q"] = 2000 if ragged else 130
    last = cu_q[-1]
    a["cu_seqlens_q"] = torch.tensor(cu_q + [last] * many, dtype=I32).cuda()
    a["cu_seqlens_k"] = torch.tensor([130 * min(i, B) for i in range(B + 1 + many)], dtype=I32).cuda()
    if ragged:
        cu_q = [x if x != 400 else 2200 for x in cu_q]
        a["cu_seqlens_q"][:B + 1] = torch.tensor(cu_q, dtype=I32)
    out, lse, status = run_prefill(a)
    assert int(status) == fd.FD_DEVSTAT_SEQLEN_OVERFLOW
    owned = torch.zeros(Sq, dtype=torch.bool)
    for b in range(B):
        if good[b] and cu_q[b + 1] > cu_q[b]:
            owned[cu_q[b]:cu_q[b + 1]] = True
            alone = {**a, "cu_seqlens_q": a["cu_seqlens_q"][b:b + 2].contiguous(), "cu_seqlens_k": a["cu_seqlens_k"][b:b + 2].contiguous()}
            o, s, st = run_prefill(alone)
            rows = slice(cu_q[b], cu_q[b + 1])
            assert int(st) == 0 and torch.equal(out[rows], o[rows]) and torch.equal(lse[rows], s[rows])
    assert (out[~owned] == 768).all() and (lse[~owned] == 768).all()


@pytest.mark.gpu
def test_prefill_rows_belong_to_the_first_of_many_requests():
    """9000 requests of one query and one key; the 7999th claims 151 rows."""
    n = [1] * 9000
    a = make_prefill(n, n, 1, 411)
    clean = run_prefill(a)
    assert int(clean[2]) == 0
    a["cu_seqlens_q"][8000] = 8150
    a["max_seqlen_q"] = 200
    out, lse, status = run_prefill(a)
    assert int(status) == fd.FD_DEVSTAT_SEQLEN_OVERFLOW
    for got, want in ((out, clean[0]), (lse, clean[1])):
        assert torch.equal(got[:7999], want[:7999]) and torch.equal(got[8150:], want[8150:])
    assert (out[7999:8149] == 0).all() and torch.isneginf(lse[7999:8149]).all()      # before their one key
    assert torch.equal(out[8149, 0], a["v"][7999, 0]) and torch.isfinite(lse[8149]).all()


@pytest.mark.gpu
def test_prefill_large_scores():
    prefill_case([500], [700], 2, 404, spread=15.0)


@pytest.mark.gpu
@pytest.mark.parametrize("lq,lk,H", [([257], [1500], 3), ([1], [4100], 1), ([128], [1500], 16), ([100], [1700], 40), ([1], [8200], 5),
                                     ([200, 0, 1], [4000, 5, 1300], 2), ([1800], [1500], 1), ([300, 4], [3000, 4000], 30)])
def test_prefill_few_queries_many_keys(lq, lk, H):
    """Calls whose key tiles several CTAs share: the parts of one to eight CTAs,
    parts without a tile, rows that see nothing in a part or at all."""
    for out_dtype in (BF, F32):
        prefill_case(lq, lk, H, 420 + sum(lq), out_dtype, joint=out_dtype is BF, pad=3)


@pytest.mark.gpu
def test_prefill_shared_keys_repeat_bitwise():
    a = make_prefill([300], [5000], 4, 425)
    first = run_prefill(a)
    for _ in range(20):
        again = run_prefill(a)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


@pytest.mark.gpu
@pytest.mark.gpu
@pytest.mark.parametrize("lq,lk,H", [([300], [5000], 4), ([1], [4100], 20), ([1500] + [9] * 50, [1500] + [9] * 50, 3)])
def test_prefill_in_a_graph(lq, lk, H):
    """The cluster form and tiles found on the device, captured and replayed over
    other inputs and offsets."""
    a = make_prefill(lq, lk, H, 426)
    Sq = sum(lq)
    out, lse = torch.empty(Sq, H, 128, dtype=BF, device="cuda"), torch.empty(Sq, H, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fd.fd_prefill_latent(**a, out=out, lse=lse)
    b = make_prefill(lq, lk, H, 427)
    for name in ("q", "k_nope", "k_pe", "v"):
        a[name].copy_(b[name])
    if len(lq) > 1:       # the long request shorter, the last one longer
        for name in ("cu_seqlens_q", "cu_seqlens_k"):
            a[name][1:-1] -= 700
            b[name].copy_(a[name])
    want = run_prefill(b)
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


@pytest.mark.gpu
def test_prefill_repeats_bitwise_and_captures():
    a = make_prefill([300, 77], [450, 77], 4, 405)
    first = run_prefill(a)
    out, lse = torch.empty_like(first[0]), torch.empty_like(first[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fd.fd_prefill_latent(**a, out=out, lse=lse)
    for _ in range(3):
        out.zero_(), lse.zero_()
        g.replay()
        assert torch.equal(first[0], out) and torch.equal(first[1], lse)
    # other lengths at replay, within max_seqlen_q
    a["cu_seqlens_q"].copy_(torch.tensor([0, 10, 310], dtype=I32))
    a["cu_seqlens_k"].copy_(torch.tensor([0, 20, 400], dtype=I32))
    out.fill_(768), lse.fill_(768)
    g.replay()
    ref = latent_prefill_ref(*(f64(a[k]) for k in ("q", "k_nope", "k_pe", "v")), [0, 10, 310], [0, 20, 400], SCALE)
    check(out[:310], lse[:310], tuple(x[:310] for x in ref))
    assert (out[310:] == 768).all()
    del g


@pytest.mark.gpu
@pytest.mark.parametrize("cu_q,cu_k,max_q", [([0, 20, 400], [0, 20, 300], 300), ([0, 100, 50], [0, 20, 300], 300),
                                             ([0, 100, 150], [0, 20, 301], 300), ([0, 100, 150], [0, 100, 60], 300),
                                             ([0, 20, 300], [0, 20, 300], 200), ([0, 100, 150], [0, -5, 20], 300)])
def test_prefill_records_bad_offsets(cu_q, cu_k, max_q):
    """A request with bad rows is recorded and left as it was; the others run."""
    a = make_prefill([100, 200], [100, 200], 2, 406)
    a["cu_seqlens_q"].copy_(torch.tensor(cu_q, dtype=I32))
    a["cu_seqlens_k"].copy_(torch.tensor(cu_k, dtype=I32))
    a["max_seqlen_q"] = max_q
    out, lse, status = run_prefill(a)
    assert int(status) == fd.FD_DEVSTAT_SEQLEN_OVERFLOW
    bad = cu_q[2] > 300 or cu_q[2] < cu_q[1] or cu_k[2] > 300 or cu_k[2] < cu_k[1] or cu_q[2] - cu_q[1] > max_q
    if bad and cu_k[1] >= 0:
        assert (out[cu_q[1]:] == 768).all() and not (out[:cu_q[1]] == 768).any()


@pytest.mark.gpu
@pytest.mark.parametrize("lq,lk", [([200, 300, 90], [200, 300, 90]), ([7, 100], [60, 4000])])
def test_prefill_keeps_nan(lq, lk):
    """A NaN in a key reaches the rows that see it, in its request and head
    alone; one in a value the rows that see it and no other request or head."""
    a = make_prefill(lq, lk, 2, 431)
    clean, clean_lse, _ = run_prefill(a)
    at, key = sum(lk[:1]), 10                             # request 1
    q0, q1 = lq[0], lq[0] + lq[1]
    first = max(0, key - (lk[1] - lq[1]))                 # the first query that sees the key
    other = torch.ones(sum(lq), dtype=torch.bool)
    other[q0:q1] = False
    for name in ("k_nope", "v"):
        t = a[name].clone()
        t[at + key, 1, 5] = math.nan
        out, lse, _ = run_prefill({**a, name: t})
        assert torch.equal(out[:, 0], clean[:, 0]) and torch.equal(lse[:, 0], clean_lse[:, 0])
        assert torch.equal(out[other], clean[other]) and torch.equal(lse[other], clean_lse[other])
        if name == "k_nope":
            assert out[q0 + first:q1, 1].isnan().all() and lse[q0 + first:q1, 1].isnan().all()
            assert torch.equal(out[q0:q0 + first], clean[q0:q0 + first])
        else:
            assert out[q0 + first:q1, 1, 5].isnan().all() and torch.equal(lse, clean_lse)


@pytest.mark.gpu
@pytest.mark.parametrize("lq,lk,H", [([100], [300], 100), ([100], [9000], 4), ([100], [9000], 20), ([100], [9000], 40)])
def test_prefill_keeps_a_nan_value_of_no_weight(lq, lk, H):
    """0 times NaN: a value that a query sees reaches it, however little its key
    weighs, also where another CTA holds the key with all the weight."""
    a = make_prefill(lq, lk, H, 432)
    a["k_pe"][lk[0] - lq[0] - 1] = 60.0       # seen by all: 64 x 60 x 8 x SCALE above the others
    a["q"][..., 128:] = 8.0
    clean, clean_lse, _ = run_prefill(a)
    a["v"][5, :, 17] = math.nan
    out, lse, status = run_prefill(a)
    assert int(status) == 0 and torch.equal(lse, clean_lse)
    assert out[..., 17].isnan().all() and torch.equal(out[..., :17], clean[..., :17]) and torch.equal(out[..., 18:], clean[..., 18:])


@pytest.mark.gpu
def test_prefill_on_two_streams():
    """Calls at once, the cluster form and the plain one; no workspace is shared."""
    x, y = make_prefill([300], [5000], 4, 441), make_prefill([500, 70], [500, 70], 40, 442)
    want = run_prefill(x), run_prefill(y)
    streams, res = [torch.cuda.Stream(), torch.cuda.Stream()], []
    torch.cuda.synchronize()
    for _ in range(8):
        for st, a in zip(streams, (x, y)):
            with torch.cuda.stream(st):
                res.append(run_prefill(a))
    torch.cuda.synchronize()
    for k, r in enumerate(res):
        assert torch.equal(r[0], want[k % 2][0]) and torch.equal(r[1], want[k % 2][1])


# ---------------------------------------------------------------------------
# waits that run out


def test_wait_limit_rejects():
    with pytest.raises(fd.FdError) as e:
        fd.fd_selftest_wait_limit(2_000_000_001)
    assert e.value.status == fd.FD_ERR_INVALID_ARG
    fd.fd_selftest_wait_limit(2_000_000_000)
    fd.fd_selftest_wait_limit(0)


def give_up(call, clean, read_status):
    """Calls whose waits run out at many places of their pipelines: each says so
    or is right, and the call behind it is right (nothing of the one before is
    still being written)."""
    given_up = 0
    for limit in (1, 100, 300, 700, 1500, 3000, 6000, 15000, 40000):
        for _ in range(3):
            fd.fd_selftest_wait_limit(limit)
            try:
                got = call()
            finally:
                fd.fd_selftest_wait_limit(0)
            after = call()
            status = read_status(got)
            assert status in (0, fd.FD_DEVSTAT_WAIT_TIMEOUT)
            if status == 0:
                assert torch.equal(got[0], clean[0]) and torch.equal(got[1], clean[1])
            assert torch.equal(after[0], clean[0]) and torch.equal(after[1], clean[1])
            given_up += status != 0
    assert given_up


@pytest.mark.gpu
@pytest.mark.parametrize("lens,Tq,H,P", [([300], 1, 16, 16), ([9000, 300, 64], 1, 16, 64), ([2000, 0, 1, 700], 3, 20, 8),
                                         ([20000, 64, 7000], 1, 128, 64), ([90] * 400, 1, 16, 16)])
def test_decode_gives_up_and_the_next_call_is_right(lens, Tq, H, P):
    a = make_decode(lens, Tq, H, P, 501)
    plan = fd.fd_latent_plan_create(0, len(lens), Tq, H, P, SCALE)
    try:
        clean = run_decode(a, plan)
        assert fd.fd_read_device_status(plan) == 0
        give_up(lambda: run_decode(a, plan), clean, lambda got: fd.fd_read_device_status(plan))
    finally:
        fd.fd_plan_destroy(plan)


@pytest.mark.gpu
@pytest.mark.parametrize("lq,lk,H", [([100], [100], 2), ([700, 33], [2000, 33], 16), ([300], [9000], 4), ([1], [4100], 20),
                                     ([300, 1], [6000, 129], 30), ([1500] + [9] * 50, [1500] + [9] * 50, 3)])
def test_prefill_gives_up_and_the_next_call_is_right(lq, lk, H):
    a = make_prefill(lq, lk, H, 502)
    clean = run_prefill(a)
    assert int(clean[2]) == 0
    give_up(lambda: run_prefill(a), clean, lambda got: int(got[2]))


# ---------------------------------------------------------------------------
# outputs that are views


def view(shape, order, dtype, shift):
    """A view of `shape` in a larger buffer that holds 768, its outer dimensions in
    memory in `order`, its rows 16-byte but not 32-byte aligned with shift 1."""
    unit = 16 // dtype.itemsize if shape[-1] >= 128 else 1
    dims = [shape[i] for i in order]
    buf = torch.full([d + 1 for d in dims] + [shape[-1] + 3 * unit], 768.0, dtype=dtype, device="cuda")
    v = buf[tuple(slice(0, d) for d in dims) + (slice(shift * unit, shift * unit + shape[-1]),)]
    return buf, v.permute([order.index(i) for i in range(len(order))] + [len(order)])


def untouched(buf, v):
    v.fill_(768.0)
    return bool((buf == 768.0).all())


@pytest.mark.gpu
@pytest.mark.parametrize("out_dtype", [BF, F32])
@pytest.mark.parametrize("order,shift", [((0, 1, 2), 1), ((2, 1, 0), 0), ((1, 2, 0), 1)])
def test_decode_writes_into_views(order, shift, out_dtype):
    """Out and LSE in any memory order, within larger buffers whose rest is left as
    it was; whole requests and joined ones."""
    lens = [70, 3000, 0, 5]
    a = make_decode(lens, 3, 12, 16, 601)
    ob, out = view((4, 3, 12, 512), order, out_dtype, shift)
    lb, lse = view((4, 3, 12), (0, 1) if order[0] == 0 else (1, 0), F32, shift)
    plan = fd.fd_latent_plan_create(0, 4, 3, 12, 16, SCALE)
    fd.fd_set_plan(plan)
    try:
        fd.fd_decode_latent(**a, out=out, lse=lse)
        assert fd.fd_read_device_status(plan) == 0
    finally:
        fd.fd_set_plan(None)
        fd.fd_plan_destroy(plan)
    check(out, lse, latent_decode_ref(f64(a["q"]), f64(a["kv_cache"]), a["page_table"].cpu().numpy(), lens, SCALE,
                                      16 if out_dtype == BF else 32))
    assert untouched(ob, out) and untouched(lb, lse)


@pytest.mark.gpu
@pytest.mark.parametrize("out_dtype", [BF, F32])
@pytest.mark.parametrize("lq,lk,H", [([70, 1, 140], [70, 9, 200], 4), ([60], [4000], 5)])
@pytest.mark.parametrize("order,shift", [((0, 1), 1), ((1, 0), 0), ((1, 0), 1)])
def test_prefill_writes_into_views(order, shift, lq, lk, H, out_dtype):
    a = make_prefill(lq, lk, H, 602)
    ob, out = view((sum(lq), H, 128), order, out_dtype, shift)
    lb, lse = view((sum(lq), H), (0,), F32, shift)
    fd.fd_prefill_latent(**a, out=out, lse=lse)
    check(out, lse, latent_prefill_ref(*(f64(a[k]) for k in ("q", "k_nope", "k_pe", "v")), a["cu_seqlens_q"].cpu().numpy(),
                                       a["cu_seqlens_k"].cpu().numpy(), SCALE, 16 if out_dtype == BF else 32))
    assert untouched(ob, out) and untouched(lb, lse)
