"""Verification of drafted tokens: the oracle's pins and the refusals (CPU),
the kernel against the oracle (GPU; whole numbers, so equality)."""
import math

import numpy as np
import pytest
import torch

import split_kv_paged_gqa_gb300 as fd
from oracle.latent_ref import verify_draft_ref

F32, I32, I64 = torch.float32, torch.int32, torch.int64


def test_oracle_hand_worked():
    p = np.array([[[0.5, 0.5, 0.0], [0.25, 0.25, 0.5], [0.0, 1.0, 0.0]]], dtype=np.float32)
    q = np.array([[[1.0, 0.0, 0.0], [0.0, 0.0, 1.0]]], dtype=np.float32)
    x = np.array([[0, 2]])
    # u_0 q = 0.4 < 0.5: accepted; u_1 q = 0.5 not < 0.5: refused; residual (0.25, 0.25, 0)
    out, n = verify_draft_ref(p, q, x, None, np.array([[0.4, 0.5, 0.5]], dtype=np.float32))
    assert out.tolist() == [[0, 1, -1]] and n.tolist() == [2]
    out, n = verify_draft_ref(p, q, x, None, np.array([[0.4, 0.49, 0.9]], dtype=np.float32))
    assert out.tolist() == [[0, 2, 1]] and n.tolist() == [3]
    out, n = verify_draft_ref(p, None, x, np.array([1]), np.array([[0.5, 0.0, 0.0]], dtype=np.float32))
    assert out.tolist() == [[1, -1, -1]] and n.tolist() == [1]     # the refused token carries no weight


def test_oracle_emits_the_targets_distribution():
    """Whatever the draft, the first emitted token follows the target's row."""
    rng = np.random.default_rng(0)
    V, N = 5, 40000
    p = rng.dirichlet(np.ones(V), size=2).astype(np.float32)[None]
    q = rng.dirichlet(np.ones(V), size=1).astype(np.float32)[None]
    x = rng.choice(V, size=(N, 1), p=q[0, 0] / q[0, 0].sum())
    out, _ = verify_draft_ref(np.repeat(p, N, 0), np.repeat(q, N, 0), x, None, rng.random((N, 2)).astype(np.float32))
    share = np.bincount(out[:, 0], minlength=V) / N
    # 5 standard deviations of a share of N draws are at most 5 * 0.5 / sqrt(N)
    assert np.abs(share - p[0, 0]).max() < 2.5 / math.sqrt(N)


def _args(B=2, K=3, V=10, device="cpu"):
    return dict(target_probs=torch.zeros(B, K + 1, V, device=device), draft_probs=torch.zeros(B, K, V, device=device),
                draft_tokens=torch.zeros(B, K, dtype=I32, device=device), num_draft=torch.zeros(B, dtype=I32, device=device),
                uniforms=torch.zeros(B, K + 1, device=device), out_tokens=torch.zeros(B, K + 1, dtype=I32, device=device),
                num_emitted=torch.zeros(B, dtype=I32, device=device))


@pytest.mark.parametrize("change,status", [
    (dict(target_probs=torch.zeros(2, 4, 10, dtype=torch.bfloat16)), fd.FD_ERR_INVALID_ARG),
    (dict(target_probs=torch.zeros(2, 40)), fd.FD_ERR_INVALID_ARG),
    (dict(target_probs=torch.zeros(2, 4, 20)[..., ::2]), fd.FD_ERR_UNSUPPORTED),
    (dict(target_probs=torch.zeros(2, 66, 10)), fd.FD_ERR_INVALID_ARG),
    (dict(target_probs=None), fd.FD_ERR_INVALID_ARG),
    (dict(draft_probs=torch.zeros(2, 4, 10)), fd.FD_ERR_INVALID_ARG),
    (dict(draft_probs=torch.zeros(2, 3, 9)), fd.FD_ERR_INVALID_ARG),
    (dict(draft_tokens=torch.zeros(2, 3)), fd.FD_ERR_INVALID_ARG),
    (dict(draft_tokens=torch.zeros(2, 4, dtype=I32)), fd.FD_ERR_INVALID_ARG),
    (dict(draft_tokens=None), fd.FD_ERR_INVALID_ARG),
    (dict(num_draft=torch.zeros(2, dtype=I64)), fd.FD_ERR_INVALID_ARG),
    (dict(uniforms=torch.zeros(2, 3)), fd.FD_ERR_INVALID_ARG),
    (dict(out_tokens=torch.zeros(2, 4, dtype=I64)), fd.FD_ERR_INVALID_ARG),
    (dict(num_emitted=torch.zeros(3, dtype=I32)), fd.FD_ERR_INVALID_ARG),
])
def test_verify_rejects(change, status):
    with pytest.raises(fd.FdError) as e:
        fd.fd_verify_draft(**{**_args(), **change}, stream=0)
    assert e.value.status == status, str(e.value)


def test_verify_rejects_a_broadcast_output():
    with pytest.raises(fd.FdError) as e:
        fd.fd_verify_draft(**{**_args(), "out_tokens": torch.zeros(1, 4, dtype=I32).expand(2, 4)}, stream=0)
    assert e.value.status == fd.FD_ERR_UNSUPPORTED


def make(B, K, V, seed, draft=True, ragged=False, dtype=I32, sharp=2.5, near=0.6):
    g = torch.Generator().manual_seed(seed)
    logits = torch.randn(B, K + 1, V, generator=g) * sharp
    target = torch.softmax(logits, -1)
    q = torch.softmax(logits[:, :K] + near * torch.randn(B, K, V, generator=g), -1)
    tokens = torch.multinomial(q.reshape(-1, V), 1, generator=g).view(B, K) if K else torch.zeros(B, 0, dtype=I64)
    return dict(target_probs=target.cuda(), draft_probs=q.cuda() if draft and K else None, draft_tokens=tokens.to(dtype).cuda(),
                num_draft=torch.randint(0, K + 1, (B,), generator=g, dtype=I32).cuda() if ragged else None,
                uniforms=torch.rand(B, K + 1, generator=g).cuda())


def run(a):
    B, K1, _ = a["target_probs"].shape
    out = torch.full((B, K1), 777, dtype=I32, device="cuda")
    emitted = torch.full((B,), 777, dtype=I32, device="cuda")
    status = torch.zeros(1, dtype=I32, device="cuda")
    fd.fd_verify_draft(**a, out_tokens=out, num_emitted=emitted, status=status)
    return out, emitted, int(status)


def check(a, status=0):
    out, emitted, st = run(a)
    n = lambda t: None if t is None else t.cpu().numpy()   # noqa: E731
    ref, cnt = verify_draft_ref(*(n(a[k]) for k in ("target_probs", "draft_probs", "draft_tokens", "num_draft", "uniforms")))
    assert st == status
    assert np.array_equal(emitted.cpu().numpy(), cnt)
    assert np.array_equal(out.cpu().numpy(), ref)
    return out, emitted


@pytest.mark.gpu
@pytest.mark.parametrize("V", [1, 2, 3, 31, 33, 127, 1000, 1023, 4096, 8193, 50021, 131072, 200003])
@pytest.mark.parametrize("draft", [True, False])
def test_verify_vocabularies(V, draft):
    check(make(5, 3, V, V, draft=draft))


@pytest.mark.gpu
@pytest.mark.parametrize("B,K", [(1, 0), (1, 1), (3, 0), (70, 2), (300, 1), (2, 64), (9, 7)])
@pytest.mark.parametrize("dtype", [I32, I64])
def test_verify_batches(B, K, dtype):
    check(make(B, K, 1777, B + K, ragged=K > 0 and B > 1, dtype=dtype))


@pytest.mark.gpu
def test_verify_every_outcome_occurs():
    a = make(400, 3, 503, 9)
    _, emitted = check(a)
    assert set(emitted.tolist()) == {1, 2, 3, 4}


@pytest.mark.gpu
def test_verify_edges():
    a = make(6, 2, 1001, 10)
    p, q, u = a["target_probs"], a["draft_probs"], a["uniforms"]
    q[0] = p[0, :2]                        # draft equals target: every u < 1 accepts
    p[1, 0] = 0
    p[1, 0, 700] = 1.0                     # all weight on one token, drafted elsewhere
    a["draft_tokens"][1, 0] = 3
    p[2, 0] = q[2, 0] * 0.5                # refused with no residual weight: the target's row
    u[2, 0] = 0.75
    q[3, 0, a["draft_tokens"][3, 0].long()] = 0      # a drafted token that the draft calls impossible
    u[4] = 0.0                             # the smallest numbers
    u[5] = float(np.nextafter(np.float32(1), np.float32(0)))
    out, emitted = check(a)
    assert emitted[0] == 3 and out[1].tolist() == [700, -1, -1] and emitted[2] == 1
    p[3] = 0                               # no weight anywhere: the last token
    out, _ = check(a)
    assert out[3, 0] == 1000


@pytest.mark.gpu
def test_verify_near_equal_rows():
    """Residuals of a few units in the last place: the difference of two fp32
    probabilities has to be taken exactly."""
    a = make(8, 1, 20011, 11)
    p = a["target_probs"]
    g = torch.Generator().manual_seed(5)
    wiggle = torch.randint(-3, 4, (8, 20011), generator=g, dtype=I32).cuda()
    a["draft_probs"][:, 0] = (p[:, 0].view(I32) + wiggle).clamp(min=0).view(F32)
    a["draft_tokens"][:, 0] = (a["draft_probs"][:, 0] - p[:, 0]).argmax(-1).to(I32)
    a["uniforms"][:, 0] = float(np.nextafter(np.float32(1), np.float32(0)))
    check(a)


@pytest.mark.gpu
def test_verify_large_and_tiny_weights():
    a = make(6, 1, 5003, 12)
    a["target_probs"][0:2] *= 1e30
    a["draft_probs"][0:2] *= 1e30
    a["target_probs"][2:4] *= 1e-30
    a["draft_probs"][2:4] *= 1e-30
    a["target_probs"][4, :, 1000:] *= 1e-20       # weights of very different sizes in one row
    check(a)


@pytest.mark.gpu
def test_verify_bad_tokens_are_refused_and_recorded():
    a = make(3, 2, 400, 13)
    a["draft_tokens"][0, 0] = -1
    a["draft_tokens"][1, 1] = 400
    check(a, fd.FD_DEVSTAT_BAD_TOKEN)
    a = make(3, 2, 400, 14)
    a["num_draft"] = torch.tensor([-1, 3, 1], dtype=I32).cuda()
    check(a, fd.FD_DEVSTAT_BAD_TOKEN)


@pytest.mark.gpu
def test_verify_strides():
    a = make(4, 3, 600, 15, ragged=True)
    wide = torch.zeros(4, 4, 700, device="cuda")
    wide[..., 3:603] = a["target_probs"]
    a["target_probs"] = wide[..., 3:603]                     # rows that start at odd addresses
    a["draft_probs"] = a["draft_probs"].transpose(0, 1).contiguous().transpose(0, 1)
    a["draft_tokens"] = a["draft_tokens"].t().contiguous().t()
    a["uniforms"] = a["uniforms"].t().contiguous().t()
    check(a)


@pytest.mark.gpu
def test_verify_in_a_graph():
    a = make(7, 3, 9000, 16, ragged=True)
    out = torch.zeros(7, 4, dtype=I32, device="cuda")
    emitted = torch.zeros(7, dtype=I32, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fd.fd_verify_draft(**a, out_tokens=out, num_emitted=emitted)
    for seed in (17, 18, 19):
        b = make(7, 3, 9000, seed, ragged=True)
        for k in a:
            a[k].copy_(b[k])
        g.replay()
        want = check(b)
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(emitted, want[1])
    del g


@pytest.mark.gpu
def test_verify_largest_vocabulary():
    check(make(1, 1, 1 << 24, 61))
    check(make(1, 0, (1 << 24) - 1, 62))


@pytest.mark.gpu
@pytest.mark.parametrize("B,V", [(100, 65537), (61, 131073), (12, 40000)])
def test_verify_several_ctas_a_request(B, V):
    check(make(B, 1, V, 66 + B, ragged=True))


@pytest.mark.gpu
def test_verify_clusters_in_a_graph():
    a, b = make(6, 2, 70001, 71), make(6, 2, 70001, 72)
    out, emitted = torch.zeros(6, 3, dtype=I32, device="cuda"), torch.zeros(6, dtype=I32, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fd.fd_verify_draft(**a, out_tokens=out, num_emitted=emitted)
    for name in ("target_probs", "draft_probs", "draft_tokens", "uniforms"):
        a[name].copy_(b[name])
    for _ in range(3):
        g.replay()
    want = check(b)
    assert torch.equal(out, want[0]) and torch.equal(emitted, want[1])


@pytest.mark.gpu
def test_verify_on_two_streams():
    x, y = make(2, 3, 50021, 63), make(200, 2, 9001, 64, draft=False)
    want = run(x), run(y)
    streams, res = [torch.cuda.Stream(), torch.cuda.Stream()], []
    for _ in range(10):
        for st, a in zip(streams, (x, y)):
            with torch.cuda.stream(st):
                res.append(run(a))
    torch.cuda.synchronize()
    for k, r in enumerate(res):
        assert torch.equal(r[0], want[k % 2][0]) and torch.equal(r[1], want[k % 2][1]) and r[2] == 0


@pytest.mark.gpu
@pytest.mark.parametrize("V", [1000, 131072])
def test_verify_weights_that_are_no_numbers_end_in_a_token(V):
    """Outside what the call asks for (NaN, infinities, negative, nothing at all),
    and uniforms past 1: some token of the vocabulary, and the step ends."""
    for bad in (math.nan, math.inf, -1.0, 0.0):
        a = make(2, 2, V, 65)
        for k in range(3):
            a["target_probs"][0, k] = bad
        a["target_probs"][1, :, ::3] = bad
        a["uniforms"][1, -1] = 1.5
        out, emitted, _ = run(a)
        for b in range(2):
            n = int(emitted[b])
            assert 1 <= n <= 3 and (out[b, :n] >= 0).all() and (out[b, :n] < V).all() and (out[b, n:] == -1).all()


@pytest.mark.gpu
@pytest.mark.parametrize("B,K,V,draft", [(9, 0, 1001, False), (9, 1, 5003, True), (9, 1, 5003, False), (3, 1, 131072, True), (200, 2, 9001, True)])
@pytest.mark.parametrize("size", ["huge", "subnormal", "tiny"])
def test_verify_rows_of_any_finite_sum(B, K, V, draft, size):
    """Finite weights whose sum passes the largest fp32 number, and rows of nothing
    but the smallest ones: sampled as in 64 bits."""
    a = make(B, K, V, 81 + V, draft=draft)
    g = torch.Generator().manual_seed(9)
    n = [(B, K + 1, V)] + ([(B, K, V)] if a["draft_probs"] is not None else [])
    if size == "huge":
        rows = [(torch.rand(s, generator=g) + 0.1) * 3e38 for s in n]
    elif size == "tiny":
        rows = [torch.rand(s, generator=g) * 1e-36 / V for s in n]
    else:                                     # whole multiples of 2^-149
        rows = [torch.randint(0, 6, s, generator=g, dtype=I32).view(F32) for s in n]
    a["target_probs"] = rows[0].cuda()
    if len(rows) > 1:
        a["draft_probs"] = rows[1].cuda()
        a["uniforms"][:, 0] = 0.9             # (about half of the first drafted tokens are refused)
    out, emitted = check(a)
    assert out[torch.arange(B), emitted.long() - 1].unique().numel() > B // 2
    a["uniforms"][:, -1] = 0.0                # the first token with any weight
    a["target_probs"][:, :, : V // 3] = 0.0
    a["target_probs"][0, :, V // 5] = 1e-44
    check(a)
