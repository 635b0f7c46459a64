"""The training-step operators on the GPU against the 64-bit oracle: sizes from
one token up, ragged shards, every type, rows without a loss, infinities and
NaN in masked places, graph replays, other streams, untouched surroundings,
and a run of them together with the collectives."""

import numpy as np
import pytest

from oracle import train as O
from tests import train_util as U
from tests.gpu_util import announce

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from double_binary_tree_amd import emucomm as E
    E.lib()
    yield
    E.comm_destroy()
    torch.cuda.empty_cache()


def guarded(shape, dtype, fill=7):
    """A tensor with 64 elements of a known value on either side, and a check
    that they are still there."""
    n = int(np.prod(shape))
    pad = 64
    whole = torch.full((n + 2 * pad,), fill, dtype=dtype, device="cuda")
    view = whole[pad:pad + n].view(shape)

    def intact():
        return bool((whole[:pad] == fill).all()) and bool((whole[pad + n:] == fill).all())
    return view, intact


# --- cross entropy -----------------------------------------------------------

# (vocabulary of every rank, tokens, dim)
XENT = [
    ([1], 1, 8),
    ([1, 0, 2], 1, 8),
    ([7, 5], 3, 16),
    ([129, 64, 1], 64, 64),
    ([255, 257], 65, 72),
    ([1000], 129, 520),
    ([33] * 17, 200, 136),
    ([0, 2000, 0, 999], 31, 1032),
    ([6500, 6531], 1100, 72),        # the largest tile shape
]


def xent_case(vocab, tokens, dim, dtype, salt=0, scale=2.0):
    r = U.rng(tokens, dim, sum(vocab), salt)
    x = U.tensor(r.normal(size=(tokens, dim)), dtype)
    ws = [U.tensor(r.normal(size=(v, dim)) * scale / np.sqrt(dim), dtype) for v in vocab]
    y = r.integers(0, sum(vocab), tokens)
    y[r.random(tokens) < 0.15] = -1
    y[r.random(tokens) < 0.05] = sum(vocab)
    if tokens > 2:
        y[0], y[1] = 0, sum(vocab) - 1
    return x, ws, y, torch.from_numpy(y).cuda()


def run_loss(E, x, ws, y, **kw):
    loss, ok1 = guarded((x.shape[0],), torch.float32)
    lse, ok2 = guarded((x.shape[0],), torch.float32)
    E.cross_entropy_tensors(x, ws, y, loss, lse, **kw)
    torch.cuda.synchronize()
    assert ok1() and ok2()
    return loss, lse


def run_grad(E, x, ws, y, lse, d, **kw):
    dx, ok = guarded(tuple(x.shape), x.dtype)
    pairs = [guarded(tuple(w.shape), w.dtype) for w in ws]
    E.cross_entropy_grad_tensors(x, ws, y, lse, d, dx, [p[0] for p in pairs], **kw)
    torch.cuda.synchronize()
    assert ok() and all(p[1]() for p in pairs)
    return dx, [p[0] for p in pairs]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("vocab,tokens,dim", XENT)
def test_cross_entropy_and_gradient(vocab, tokens, dim, dtype):
    from double_binary_tree_amd import emucomm as E
    announce(f"cross entropy vocab={vocab[:4]} tokens={tokens} dim={dim} {dtype}")
    x, ws, y, yt = xent_case(vocab, tokens, dim, dtype)
    xe, we = U.exact(x), [U.exact(w) for w in ws]
    want_loss, want_lse = O.cross_entropy(xe, we, y)
    loss, lse = run_loss(E, x, ws, yt)
    d = torch.from_numpy(U.rng(tokens, 5).normal(size=tokens).astype(np.float32)).cuda()
    given = torch.from_numpy(want_lse.astype(np.float32)).cuda()
    lse_e, d_e = U.exact(given), U.exact(d)
    loss_tol, lse_tol, dx_tol, dw_tol = U.xent_bounds(xe, we, y, lse_e, d_e, dtype)
    assert U.worst(U.exact(loss), want_loss, loss_tol) <= 1
    assert U.worst(U.exact(lse), want_lse, lse_tol) <= 1
    assert not U.exact(loss)[~O.counted(y, sum(vocab))].any()
    dx, dws = run_grad(E, x, ws, yt, given, d)
    want_dx, want_dw = O.cross_entropy_grad(xe, we, y, lse_e, d_e)
    assert U.worst(U.exact(dx), want_dx, U.rounded(want_dx, dx_tol, dtype)) <= 1
    at = 0
    for w, got, want in zip(ws, dws, want_dw):
        tol = dw_tol[at:at + len(want)]
        at += len(want)
        assert U.worst(U.exact(got), want, U.rounded(want, tol, dtype)) <= 1
    # one gradient at a time gives the same bits
    only, ok = guarded(tuple(x.shape), x.dtype)
    E.cross_entropy_grad_tensors(x, ws, yt, given, d, dx=only)
    alone = [torch.empty_like(w) for w in ws]
    E.cross_entropy_grad_tensors(x, ws, yt, given, d, dws=alone)
    torch.cuda.synchronize()
    assert ok() and torch.equal(only, dx) and all(torch.equal(a, b) for a, b in zip(alone, dws))


# sizes at which each of the three products takes the larger tiles
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("vocab,tokens,dim", [([4100, 4130], 1000, 1024), ([700, 330], 1024, 16384), ([700, 501], 1020, 4160)])
def test_cross_entropy_in_large_tiles(vocab, tokens, dim, dtype):
    test_cross_entropy_and_gradient(vocab, tokens, dim, dtype)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_cross_entropy_gradient_against_differences_of_its_own_loss(dtype):
    from double_binary_tree_amd import emucomm as E
    announce(f"cross entropy differences {dtype}")
    x, ws, y, yt = xent_case([40, 23], 9, 24, dtype)
    loss, lse = run_loss(E, x, ws, yt)
    d = torch.ones(9, device="cuda")
    dx, dws = run_grad(E, x, ws, yt, lse, d)
    # a directional difference: both ends are exact tensors of the type, the
    # losses are good to 1e-5, so the slope along h to 2e-5 / |step| plus the
    # curvature (third derivative at most |w|^3)
    step = U.tensor(U.rng(1).choice([-1.0, 1.0], size=(9, 24)) / 16, dtype)
    up, _ = run_loss(E, (x.float() + step.float()).to(x.dtype), ws, yt)
    down, _ = run_loss(E, (x.float() - step.float()).to(x.dtype), ws, yt)
    h = U.exact((x.float() + step.float()).to(x.dtype)) - U.exact((x.float() - step.float()).to(x.dtype))
    slope = (U.exact(dx) * h).sum(1)
    reach = max(np.abs(U.exact(w) @ (h / 2).T).max() for w in ws)      # largest change of a logit
    tol = 4e-5 + reach ** 3 / 3 + (np.abs(U.exact(dx)) * np.abs(h)).sum(1) * 4 * U.ROUND[dtype] + 24 * 2 ** -9 * np.abs(h).max()
    assert (np.abs(U.exact(up) - U.exact(down) - slope) <= tol).all()


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("tokens", [5, 70])
def test_cross_entropy_gradient_of_tiny_and_zero_weights(tokens, dtype):
    from double_binary_tree_amd import emucomm as E
    announce(f"cross entropy gradients of tiny and zero weights, {tokens} tokens {dtype}")
    x, ws, y, yt = xent_case([40, 23], tokens, 24, dtype)
    _, lse = run_loss(E, x, ws, yt)
    big = max(float(x.abs().max()), max(float(w.abs().max()) for w in ws))
    for weight in (0.0, 1e-39, 1e-45):       # 1e-39 and 1e-45 have no normal f32
        d = torch.full((tokens,), weight, device="cuda")
        d[0] = weight / 3
        dx, dws = run_grad(E, x, ws, yt, lse, d)
        for t in [dx, *dws]:                 # |g| is at most dloss and sums to at most 2 dloss over a row
            assert float(t.abs().max()) <= 2 * weight * big * tokens * 1.01
    # one weight far above the others
    d = torch.full((tokens,), 1e-30, device="cuda")
    d[1] = 1e6 if dtype != "f16" else 100.0
    dx, dws = run_grad(E, x, ws, yt, lse, d)
    want_dx, want_dw = O.cross_entropy_grad(U.exact(x), [U.exact(w) for w in ws], y, U.exact(lse), U.exact(d))
    for got, want in [(dx, want_dx), *zip(dws, want_dw)]:
        assert np.linalg.norm(U.exact(got) - want) <= 2 * U.ROUND[dtype] * np.linalg.norm(want) + 1e-5 * np.linalg.norm(want)


def test_cross_entropy_masked_tokens_do_not_leak():
    from double_binary_tree_amd import emucomm as E
    announce("cross entropy: NaN and infinities in tokens without a loss")
    x, ws, y, yt = xent_case([70, 61], 130, 64, "bf16")
    mask = ~O.counted(y, 131)
    assert mask.any()
    d = torch.full((130,), 0.5, device="cuda")
    _, lse = run_loss(E, x, ws, yt)
    clean = run_grad(E, x, ws, yt, lse, d)
    bad = x.clone()
    rows = torch.from_numpy(np.flatnonzero(mask)).cuda()
    bad[rows] = float("nan")
    bad[rows[0]] = float("inf")
    loss, lse2 = run_loss(E, bad, ws, yt)
    d2 = d.clone()
    d2[rows] = float("nan")
    dx, dws = run_grad(E, bad, ws, yt, lse2, d2)
    assert not torch.isnan(loss).any()
    assert torch.equal(dx, clean[0]) and all(torch.equal(a, b) for a, b in zip(dws, clean[1]))
    assert not dx[rows].float().any()
    # no token has a loss at all
    none = torch.full_like(yt, -1)
    loss, lse = run_loss(E, bad, ws, none)
    dx, dws = run_grad(E, bad, ws, none, lse, d)
    assert not loss.any() and not dx.float().any() and not any(w.float().any() for w in dws)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_cross_entropy_extreme_logits(dtype):
    from double_binary_tree_amd import emucomm as E
    announce(f"cross entropy extreme logits {dtype}")
    # one-hot hidden states make z_tv = w_v0: very large, very small, -infinite
    low = float(torch.finfo(U.DTYPES[dtype]).min)
    col = [10000.0, -10000.0, 0.0, low, float("-inf")]
    w = torch.zeros(5, 8, dtype=U.DTYPES[dtype], device="cuda")
    w[:, 0] = torch.tensor(col).to(w)
    x = torch.zeros(5, 8, dtype=w.dtype, device="cuda")
    x[:, 0] = 1.0
    y = torch.arange(5, device="cuda")
    loss, lse = run_loss(E, x, [w[:3].contiguous(), w[3:].contiguous()], y)
    z = U.exact(w[:, 0])
    assert U.exact(lse).tolist() == [z[0]] * 5
    want = z[0] - z
    got = U.exact(loss)
    assert got[4] == np.inf and got[0] == 0
    assert np.all(np.abs(got[:4] - want[:4]) <= np.abs(want[:4]) * 2 ** -23)
    # only rows of -infinity: lse is -infinity and no probability is defined
    gone = torch.full((3, 8), 0.0, dtype=w.dtype, device="cuda")
    gone[:, 0] = float("-inf")
    loss, lse = run_loss(E, x[:2].contiguous(), [gone], y[:2].contiguous())
    assert torch.isneginf(lse).all()


def test_cross_entropy_without_tokens():
    from double_binary_tree_amd import emucomm as E
    announce("cross entropy without tokens")
    x = torch.empty(0, 16, device="cuda")
    ws = [torch.ones(3, 16, device="cuda"), torch.ones(0, 16, device="cuda"), torch.ones(70, 16, device="cuda")]
    y, f = torch.empty(0, dtype=torch.int64, device="cuda"), torch.empty(0, device="cuda")
    run_loss(E, x, ws, y)
    _, dws = run_grad(E, x, ws, y, f, f)
    assert not any(d.any() for d in dws)


def test_cross_entropy_gradient_in_several_runs():
    from double_binary_tree_amd import emucomm as E
    # 33,000 tokens leave 4,096 positions to a run: 9,001 rows take three, and
    # shard ends fall inside runs
    tokens, dim, vocab = 33000, 24, [4099, 900, 4002]
    announce("cross entropy gradient, several runs")
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    x = torch.randn(tokens, dim, device="cuda", generator=g).bfloat16()
    ws = [torch.randn(v, dim, device="cuda", generator=g).bfloat16() * 0.4 for v in vocab]
    y = torch.randint(-1, sum(vocab), (tokens,), device="cuda", generator=g)
    d = torch.rand(tokens, device="cuda", generator=g)
    loss, lse = run_loss(E, x, ws, y)
    dx, dws = run_grad(E, x, ws, y, lse, d)
    w = torch.cat(ws).double()
    z = x.double() @ w.t().contiguous()
    want = torch.logsumexp(z, 1)
    assert float((lse.double() - want).abs().max()) < 1e-4      # 24 products of about 1, a sum of 9,001 terms
    p = (z - lse.double()[:, None]).exp_()
    ok = y >= 0
    p[ok.nonzero()[:, 0], y[ok]] -= 1
    p *= (d.double() * ok)[:, None]
    # rounding q, x' and the result: at most 2^-8 each relative to the terms'
    # magnitudes, independent of one another, in the 2-norm below 2^-8 sqrt(3)
    for got, ref in zip([dx, *dws], [p @ w, *(p.t().contiguous() @ x.double()).split(vocab)]):
        assert float((got.double() - ref).norm() / ref.norm()) < 2 * 2.0 ** -8


# --- balance loss ------------------------------------------------------------

BALANCE = [
    ([1], 1, 1),
    ([3, 0, 5], 4, 2),
    ([61, 61, 61, 61], 8, 2),
    ([200, 1, 77], 7, 3),
    ([130, 131], 64, 6),
    ([513], 65, 8),
    ([40, 40], 100, 5),
    ([300, 299], 256, 8),
    ([33], 384, 8),
    ([20, 21], 1000, 4),
    ([17], 1023, 16),
    ([9, 9], 1024, 1024),
    ([70000, 2], 16, 1),
]


def balance_case(tokens, nexp, topk, dtype):
    r = U.rng(nexp, topk, *tokens)
    logits = [U.tensor(r.normal(size=(t, nexp)) * 2, dtype) for t in tokens]
    experts = []
    for t in tokens:
        e = r.integers(0, nexp, (t, topk))
        e[r.random(t) < 0.1] = -1
        e[r.random((t, topk)) < 0.05] = -7
        e[r.random((t, topk)) < 0.05] = nexp
        experts.append(torch.from_numpy(e.astype(np.int32)).cuda())
    return logits, experts


def run_balance(E, logits, experts, coef, grad=True, **kw):
    counts, ok = guarded((len(logits) + 1, logits[0].shape[1]), torch.int64)
    loss = torch.full((1,), 7.0, device="cuda")
    pairs = [guarded(tuple(z.shape), z.dtype) for z in logits]
    E.balance_loss_tensors(logits, experts, coef, counts, loss, [p[0] for p in pairs] if grad else None, **kw)
    torch.cuda.synchronize()
    assert ok() and all(p[1]() for p in pairs)
    return counts, loss, [p[0] for p in pairs]


def check_balance(logits, experts, coef, got, dtype):
    counts, loss, grads = got
    ze, ie = [U.exact(z) for z in logits], [e.cpu().numpy() for e in experts]
    want_counts, want_loss, want_grads = O.balance_loss(ze, ie, coef)
    assert np.array_equal(counts.cpu().numpy(), want_counts)
    # a probability: z - max twice rounded (|z - max| 2^-23), exp2 2^-22, a sum
    # of E terms, a reciprocal and a product; P then adds a workgroup's rows in
    # f32 (4,096 at most) and f is one rounding; the gradient adds a dot product
    n = ze[0].shape[1]
    spread = max([float(np.ptp(z[np.isfinite(z)])) for z in ze if np.isfinite(z).any()] or [0.0])
    rel = (spread * 4 + n + 24) * U.U32
    assert abs(float(loss) - want_loss) <= abs(want_loss) * (rel + 4096 * U.U32) + 1e-30
    if grads is None:
        return
    total = max(1, int(sum(((i >= 0) & (i < n)).any(1).sum() for i in ie)))
    f = want_counts[-1] / (total * ie[0].shape[1])
    for z, i, g, w in zip(ze, ie, grads, want_grads):
        live = ((i >= 0) & (i < n)).any(1)
        p = O.softmax_rows(z) * live[:, None]
        tol = abs(coef) * n / total * p * (f + (p @ f)[:, None]) * (rel + (n + 8) * U.U32)
        assert U.worst(U.exact(g), w, U.rounded(w, tol, dtype)) <= 1
        assert not U.exact(g)[~live].any()


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("tokens,nexp,topk", BALANCE)
def test_balance_loss(tokens, nexp, topk, dtype):
    from double_binary_tree_amd import emucomm as E
    announce(f"balance loss tokens={tokens} experts={nexp} topk={topk} {dtype}")
    logits, experts = balance_case(tokens, nexp, topk, dtype)
    got = run_balance(E, logits, experts, 0.37)
    check_balance(logits, experts, 0.37, got, dtype)
    again = run_balance(E, logits, experts, 0.37)
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])
    assert all(torch.equal(a, b) for a, b in zip(got[2], again[2]))
    counts, loss, _ = run_balance(E, logits, experts, 0.37, grad=False)
    assert torch.equal(counts, got[0]) and torch.equal(loss, got[1])


def test_balance_loss_masked_rows():
    from double_binary_tree_amd import emucomm as E
    announce("balance loss: padding, masked experts, empty rows")
    logits, experts = balance_case([50, 30], 12, 3, "f32")
    logits[0][3] = float("nan")                  # padding holds anything
    logits[0][4] = float("inf")
    experts[0][3:5] = -1
    logits[0][:, 5] = float("-inf")              # a masked expert
    logits[1][:, 6] = float(torch.finfo(torch.float32).min)
    logits[1][7] = float("-inf")                 # nothing left of a row that is counted
    logits[1][8] = float(torch.finfo(torch.float32).min)
    experts[1][7] = 2
    got = run_balance(E, logits, experts, 1.0)
    for z in logits:                             # the oracle reads finite padding
        z[torch.isnan(z) | torch.isposinf(z)] = 0.0
    check_balance(logits, experts, 1.0, got, "f32")
    assert not got[2][1][7].any() and not got[2][0][:, 5].any()
    # the same expert twice counts twice
    z, e = [torch.zeros(2, 4, device="cuda")], [torch.tensor([[1, 1], [3, 1]], dtype=torch.int32, device="cuda")]
    counts, _, _ = run_balance(E, z, e, 1.0)
    assert counts.tolist() == [[0, 3, 0, 1]] * 2
    # no token at all, and only padding
    for t in (0, 5):
        z = [torch.full((t, 4), 1.0, device="cuda")]
        e = [torch.full((t, 2), -1, dtype=torch.int32, device="cuda")]
        counts, loss, grads = run_balance(E, z, e, 1.0)
        assert not counts.any() and float(loss) == 0.0 and not grads[0].any()


# --- orthogonalisation -------------------------------------------------------

ORTHO = [(1, 1, 1), (2, 1, 9), (1, 9, 1), (3, 5, 4), (2, 64, 64), (1, 127, 130), (8, 128, 200), (2, 300, 129),
         (1, 257, 513), (64, 24, 40), (1, 700, 650), (3, 17, 7412), (1, 2500, 130)]


def ortho_case(n, rows, cols, dtype, fade=True):
    r = U.rng(n, rows, cols)
    k = max(1, min(rows, cols) // 8)
    gs = [(r.normal(size=(rows, k)) * np.logspace(0, -2, k)) @ r.normal(size=(k, cols)) + 0.2 * r.normal(size=(rows, cols))
          for _ in range(n)]
    return [U.tensor(g * 10.0 ** (i % 5 - 2), dtype) for i, g in enumerate(gs)]


def check_ortho(sends, recvs, steps, coeffs, dtype):
    """The library's number formats emulated on the host leave a distance from
    the exact result; the kernels round at the same places and differ from the
    emulation in the order of their f32 sums, which the emulation has too: four
    times that distance, and the result's own rounding, bounds them."""
    triples = [O.DEFAULT_COEFFS] * steps if coeffs is None else coeffs
    for s, r in zip(sends, recvs):
        g = U.exact(s)
        want = O.orthogonalize(g, steps, [tuple(np.float32(c) for c in t) for t in triples])
        near = np.linalg.norm(U.emulated_ortho(g, steps, triples, dtype) - want)
        norm = np.linalg.norm(want)
        off = np.linalg.norm(U.exact(r) - want)
        assert off <= 4 * near + norm * (U.ROUND[dtype] + 2.0 ** -20), (off / norm, near / norm)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("n,rows,cols", ORTHO)
def test_orthogonalize(n, rows, cols, dtype):
    from double_binary_tree_amd import emucomm as E
    announce(f"orthogonalize {n} x {rows} x {cols} {dtype}")
    sends = ortho_case(n, rows, cols, dtype)
    pairs = [guarded((rows, cols), sends[0].dtype) for _ in range(n)]
    recvs = [p[0] for p in pairs]
    E.orthogonalize_tensors(sends, recvs)
    torch.cuda.synchronize()
    assert all(p[1]() for p in pairs)
    some = [0, n // 2, n - 1]
    check_ortho([sends[i] for i in some], [recvs[i] for i in some], 5, None, dtype)
    E.orthogonalize_tensors(sends, sends)                     # in place, the same bits
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(sends, recvs))


# Many matrices, so that every tile shape is taken (the square products' and the
# step's), wide and tall, with rows of whole 16-byte vectors and without; long
# ones, whose products are split along the sum.
ORTHO_MANY = [(64, 130, 200), (64, 200, 300), (64, 300, 296), (64, 304, 296), (64, 296, 301), (64, 521, 520), (40, 40, 5504),
              (40, 5501, 40), (40, 24, 16400), (40, 200, 5504), (40, 5500, 200)]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("n,rows,cols", ORTHO_MANY)
def test_orthogonalize_many(n, rows, cols, dtype):
    from double_binary_tree_amd import emucomm as E
    announce(f"orthogonalize many, {n} x {rows} x {cols} {dtype}")
    first = ortho_case(3, rows, cols, dtype)
    sends = first + [first[i % 3].clone() for i in range(3, n)]
    pairs = [guarded((rows, cols), sends[0].dtype) for _ in range(n)]
    recvs = [p[0] for p in pairs]
    size = E.orthogonalize_workspace(sends).numel()
    whole = torch.full((size + 4096,), 0x5C, dtype=torch.uint8, device="cuda")
    E.orthogonalize_tensors(sends, recvs, workspace=whole[:size])
    torch.cuda.synchronize()
    assert all(p[1]() for p in pairs) and bool((whole[size:] == 0x5C).all())
    check_ortho(first, recvs[:3], 5, None, dtype)
    # the same matrix gives the same bits, whatever its place
    assert all(torch.equal(recvs[i], recvs[i % 3]) for i in range(3, n))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_orthogonalize_steps_and_coefficients(dtype):
    from double_binary_tree_amd import emucomm as E
    announce(f"orthogonalize coefficients {dtype}")
    sends = ortho_case(2, 40, 96, dtype)
    recvs = [torch.empty_like(s) for s in sends]
    for steps, coeffs in ((1, None), (16, (1.5, -0.5, 0.0)), (3, [(3.0, -3.0, 1.0), (2.0, -1.5, 0.5), (1.5, -0.5, 0.0)])):
        E.orthogonalize_tensors(sends, recvs, steps=steps, coeffs=coeffs)
        torch.cuda.synchronize()
        triples = None if coeffs is None else coeffs if steps == 3 else [coeffs] * steps
        check_ortho(sends, recvs, steps, triples, dtype)


def test_orthogonalize_special_matrices():
    from double_binary_tree_amd import emucomm as E
    announce("orthogonalize zeros, NaN, infinities, large and small values")
    r = U.rng(9)
    base = r.normal(size=(20, 33))
    sends = [U.tensor(base * s, "f32") for s in (0.0, 1.0, 1e30, 1e-30, 1e36, 1.0, 1.0)]
    sends[5][3, 4] = float("nan")
    sends[6][0, 0] = float("inf")
    recvs = [torch.empty_like(s) for s in sends]
    E.orthogonalize_tensors(sends, recvs)
    torch.cuda.synchronize()
    assert not recvs[0].any()
    check_ortho(sends[1:5], recvs[1:5], 5, None, "f32")
    assert torch.isnan(recvs[5]).all() and torch.isnan(recvs[6]).all()


@pytest.mark.parametrize("rows,cols", [(0, 8), (8, 0)])
def test_orthogonalize_nothing(rows, cols):
    from double_binary_tree_amd import emucomm as E
    announce("orthogonalize an empty matrix")
    t = [torch.empty(rows, cols, device="cuda")]
    E.orthogonalize_tensors(t, t)


# --- graphs, streams, workspaces ---------------------------------------------

def all_three(E, s):
    """One pass over the state's own buffers, with its own workspaces."""
    E.cross_entropy_tensors(s["x"], s["ws"], s["y"], s["loss"], s["lse"], workspace=s["w0"])
    E.cross_entropy_grad_tensors(s["x"], s["ws"], s["y"], s["lse"], s["d"], s["dx"], s["dws"], workspace=s["w1"])
    E.balance_loss_tensors(s["z"], s["e"], 0.1, s["counts"], s["aux"], s["dz"], workspace=s["w2"])
    E.orthogonalize_tensors(s["dws"], s["up"], workspace=s["w3"])


def state(E, salt, dtype="bf16"):
    x, ws, _, y = xent_case([120, 120], 90, 64, dtype, salt)
    z, e = balance_case([40, 41], 24, 2, dtype)
    s = {"x": x, "ws": ws, "y": y, "z": z, "e": e, "d": torch.full((90,), 1 / 90, device="cuda"),
         "loss": torch.empty(90, device="cuda"), "lse": torch.empty(90, device="cuda"), "dx": torch.empty_like(x),
         "dws": [torch.empty_like(w) for w in ws], "up": [torch.empty_like(w) for w in ws],
         "counts": torch.empty(3, 24, dtype=torch.int64, device="cuda"), "aux": torch.empty(1, device="cuda"),
         "dz": [torch.empty_like(q) for q in z]}
    s["w0"] = E.cross_entropy_workspace(x, ws)
    s["w1"] = E.cross_entropy_workspace(x, ws, grad=True)
    s["w2"] = E.balance_loss_workspace(z)
    s["w3"] = E.orthogonalize_workspace(s["dws"])
    return s


def outputs(s):
    return [s["loss"], s["lse"], s["dx"], *s["dws"], s["counts"], s["aux"], *s["dz"], *s["up"]]


def test_captured_graphs_replay():
    from double_binary_tree_amd import emucomm as E
    announce("training-step operators captured in two graphs")
    states = [state(E, k) for k in range(2)]
    graphs = []
    for s in states:                              # no call before the capture
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            all_three(E, s)
        graphs.append(g)
    for rep in range(3):
        wants = []
        for k, s in enumerate(states):
            fresh = state(E, 10 * rep + k)
            for key in ("x", "y"):
                s[key].copy_(fresh[key])
            for a, b in zip(s["ws"], fresh["ws"]):
                a.copy_(b)
            all_three(E, fresh)                   # eager work between replays
            wants.append([t.clone() for t in outputs(fresh)])
            for t in outputs(s):
                t.zero_()
            for w in ("w0", "w1", "w2", "w3"):
                s[w].fill_(0xA5)                  # a workspace's contents mean nothing
        torch.cuda.synchronize()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for s, want in zip(states, wants):
            assert all(torch.equal(a, b) for a, b in zip(outputs(s), want)), f"replay {rep}"


def test_captured_graph_of_few_tokens_and_long_matrices():
    from double_binary_tree_amd import emucomm as E
    announce("few tokens and a long matrix captured in a graph")
    x, ws, _, y = xent_case([70, 50], 20, 64, "f16", 5)
    long = ortho_case(2, 30, 3000, "f32")
    loss, lse, d = (torch.full((20,), 0.3, device="cuda") for _ in range(3))
    dx, dws, ups = torch.empty_like(x), [torch.empty_like(w) for w in ws], [torch.empty_like(g) for g in long]
    work = [E.cross_entropy_workspace(x, ws), E.cross_entropy_workspace(x, ws, grad=True), E.orthogonalize_workspace(long)]

    def once():
        E.cross_entropy_tensors(x, ws, y, loss, lse, workspace=work[0])
        E.cross_entropy_grad_tensors(x, ws, y, lse, d, dx, dws, workspace=work[1])
        E.orthogonalize_tensors(long, ups, workspace=work[2])
    outs = [loss, lse, dx, *dws, *ups]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        once()
    for rep in range(3):
        x.mul_(-1.5 if rep else 1.0)
        long[0].add_(0.25)
        once()
        want = [t.clone() for t in outs]
        for t in outs + work:
            t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want)), f"replay {rep}"


def test_streams_of_their_own():
    from double_binary_tree_amd import emucomm as E
    announce("training-step operators on two streams at once")
    states, wants = [state(E, 40 + k, "f16") for k in range(2)], []
    for s in states:
        all_three(E, s)
        wants.append([t.clone() for t in outputs(s)])
        for t in outputs(s):
            t.zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in states]
    for _ in range(5):
        for s, st in zip(states, streams):
            with torch.cuda.stream(st):
                all_three(E, s)
    # and a stream passed as an argument, with workspaces of the calls' own
    x, ws, _, y = xent_case([120, 120], 90, 64, "f16", 40)
    torch.cuda.synchronize()
    loss, lse = torch.empty(90, device="cuda"), torch.empty(90, device="cuda")
    E.cross_entropy_tensors(x, ws, y, loss, lse, stream=streams[1])
    torch.cuda.synchronize()
    assert torch.equal(loss, wants[0][0]) and torch.equal(lse, wants[0][1])
    for s, want in zip(states, wants):
        assert all(torch.equal(a, b) for a, b in zip(outputs(s), want))


def test_a_workspace_holds_what_it_says():
    from double_binary_tree_amd import emucomm as E
    announce("training-step operators leave what lies behind the workspace alone")
    s = state(E, 77)
    guards = []
    for k in ("w0", "w1", "w2", "w3"):
        n = s[k].numel()
        whole = torch.full((n + 4096,), 0x5C, dtype=torch.uint8, device="cuda")
        s[k] = whole[:n]
        guards.append(whole[n:])
    all_three(E, s)
    torch.cuda.synchronize()
    assert all(bool((g == 0x5C).all()) for g in guards)
    with pytest.raises(E.EmuError):
        E.orthogonalize_tensors(s["dws"], s["up"], workspace=s["w3"][:-1])


# --- a step of training, with the collectives ---------------------------------

def test_a_sharded_training_step():
    """Four ranks, each with its own tokens and a copy of a two-shard output
    projection: losses and gradients per rank, the projection's gradient
    all-reduced, one matrix per rank orthogonalised, the updates all-gathered;
    the router's loss over all ranks' tokens.  The 64-bit chain runs on the
    same inputs; where a chain goes on from a rounded tensor, so does it."""
    from double_binary_tree_amd import emucomm as E
    announce("a sharded training step")
    n, tokens, dim, vocab = 4, 50, 64, [48, 16]
    E.comm_init(n, 2, "tree", 2, 4096)
    ranks = [xent_case(vocab, tokens, dim, "f32", salt=s) for s in range(n)]
    ws = ranks[0][1]
    we = [U.exact(w) for w in ws]
    grads = []
    for x, _, y, yt in ranks:
        loss, lse = run_loss(E, x, ws, yt)
        d = torch.full((tokens,), 1 / tokens, device="cuda")
        dx, dws = run_grad(E, x, ws, yt, lse, d)
        want_dx, want_dw = O.cross_entropy_grad(U.exact(x), we, y, U.exact(lse), U.exact(d))
        tol = U.xent_bounds(U.exact(x), we, y, U.exact(lse), U.exact(d), "f32")
        assert U.worst(U.exact(dx), want_dx, U.rounded(want_dx, tol[2], "f32")) <= 1
        grads.append(torch.cat(dws).contiguous())
    total = [torch.empty_like(g) for g in grads]
    E.allreduce_tensors(grads, total)
    torch.cuda.synchronize()
    want = sum(U.exact(g) for g in grads)
    assert np.abs(U.exact(total[3]) - want).max() <= 3 * U.U32 * sum(np.abs(U.exact(g)) for g in grads).max()
    # rank r owns rows 16 r .. 16 r + 15 of the summed gradient
    mine = [t[16 * r:16 * r + 16].contiguous() for r, t in enumerate(total)]
    ups = [torch.empty_like(m) for m in mine]
    E.orthogonalize_tensors(mine, ups)
    check_ortho(mine, ups, 5, None, "f32")
    full = [torch.empty(64 * dim, device="cuda") for _ in range(n)]
    E.all_gather_tensors([u.view(-1) for u in ups], full)
    torch.cuda.synchronize()
    assert all(torch.equal(f, torch.cat(ups).view(-1)) for f in full)
    logits, experts = balance_case([tokens] * n, 8, 2, "f32")
    check_balance(logits, experts, 0.01, run_balance(E, logits, experts, 0.01), "f32")
    E.comm_destroy()
