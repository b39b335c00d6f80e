"""Sampling (tsd.sample) against its definition in 64 bits.

Weights are rounded to multiples of 2^-s of the largest (s = min(50, 63 -
ceil(log2 V))), each by at most half of that, and the kept sum is at least 1:
a cumulative probability is off by at most delta = V 2^-s, a probability p by
2^-s + p delta, and its fp32 value by half an ulp more.  A draw or a top_p cut
whose boundary lies within 2 delta of the limit may go either way; everything
else must be equal.
"""

import math

import numpy as np
import pytest
import torch

import tree_speculative_decoding_ancestor_b200 as tsd

pytestmark = pytest.mark.gpu


def _delta(V):
    return V * 2.0 ** -min(50, 63 - math.ceil(math.log2(max(V, 1))))


def _kept(x, T, k, p, m):
    """(kept token ids ascending, weights of all, margin of the top_p cut)."""
    V = len(x)
    x = np.where(np.isnan(x), -np.inf, x)
    top = x.max()
    with np.errstate(invalid="ignore"):
        w = np.exp(np.where(x == top, 0.0, (x - top) / (T or 1.0)))
    order = np.lexsort((np.arange(V), -x))
    if T == 0:
        return order[:1], w, np.inf
    if 0 < k < V:
        order = order[:k]
    margin = np.inf
    if p < 1:
        before = np.cumsum(w[order]) - w[order]
        z = w[order].sum()
        margin = np.abs(before[1:] - p * z).min() / z if len(order) > 1 else np.inf
        keep = before < p * z
        keep[0] = True
        order = order[keep]
    order = order[w[order] >= min(m, 1.0)]
    return np.sort(order), w, margin


def _check(dev, logits, u, T=None, k=None, p=None, m=None, exact=False, probs=None):
    R, V = logits.shape
    dl = logits if logits.is_cuda else logits.to(dev)
    put = lambda a, dt: None if a is None else torch.tensor(a, dtype=dt, device=dev)  # noqa: E731
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    res = tsd.sample(dl, u.to(dev), temperature=put(T, torch.float32), top_k=put(k, torch.int32),
                     top_p=put(p, torch.float32), min_p=put(m, torch.float32), status=st,
                     with_probs=probs is None, probs=probs)
    assert int(st.item()) == 0
    tokens, got = res.tokens.cpu().numpy(), res.probs.cpu().double().numpy()
    x = logits.float().cpu().double().numpy()
    delta = _delta(V)
    close = 0
    f32 = lambda a, r, d: d if a is None else float(np.float32(a[r]))  # noqa: E731
    for r in range(R):
        ids, w, margin = _kept(x[r], f32(T, r, 1.0), 0 if k is None else k[r], f32(p, r, 1.0),
                               f32(m, r, 0.0))
        if margin <= 2 * delta and not exact:
            close += 1
            continue
        want = np.zeros(V)
        want[ids] = w[ids] / w[ids].sum()
        err = 2.0 ** -min(50, 63 - math.ceil(math.log2(max(V, 1)))) + want * (delta + 2.0 ** -24)
        assert (np.abs(got[r] - want) <= err).all(), r
        drop = np.ones(V, bool)
        drop[ids] = False
        assert (got[r][drop] == 0).all(), r
        cdf = np.cumsum(w[ids]) / w[ids].sum()
        for s, us in enumerate(u[r].tolist()):
            at = np.searchsorted(ids, tokens[r, s])
            assert at < len(ids) and ids[at] == tokens[r, s], (r, s)
            low = cdf[at - 1] if at else 0.0
            assert low - 2 * delta <= us and us < cdf[at] + 2 * delta, (r, s)
    assert close <= max(1, R // 8)


def _logits(seed, R, V, dtype=torch.float32, sigma=2.0):
    g = torch.Generator().manual_seed(seed)
    x = sigma * torch.randn(R, V, generator=g)
    return x.to(dtype), torch.rand(R, 5, generator=g, dtype=torch.float64)


SETTINGS = [dict(), dict(T=0.7), dict(k=1), dict(k=40), dict(p=0.9), dict(p=1e-6), dict(m=0.1),
            dict(m=1.0), dict(T=1.3, k=50, p=0.8, m=0.02), dict(T=0.05, p=0.99), dict(T=30.0, p=0.5),
            dict(T=30.0, k=333), dict(T=0.0, k=7, p=0.5, m=0.5), dict(k=100000, p=1.0, m=0.0)]


@pytest.mark.parametrize("V", [1, 2, 31, 200, 1000, 4097, 32000])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_settings_by_row(cuda_device, V, dtype):
    logits, u = _logits(V, len(SETTINGS), V, dtype)
    col = lambda key, d: [s.get(key, d) for s in SETTINGS]  # noqa: E731
    _check(cuda_device, logits, u, T=col("T", 1.0), k=col("k", 0), p=col("p", 1.0), m=col("m", 0.0))


@pytest.mark.parametrize("R,V", [(1, 128256), (3, 360448), (160, 20481), (333, 512), (40, 128256)])
def test_cluster_sizes(cuda_device, R, V):
    logits, u = _logits(R, R, V)
    rep = lambda *a: [a[i % len(a)] for i in range(R)]  # noqa: E731
    _check(cuda_device, logits, u, T=rep(1.0, 0.8, 1.2), k=rep(0, 50, 2000, 0), p=rep(0.95, 1.0, 0.7),
           m=rep(0.0, 0.01))


def test_off_by_default(cuda_device):
    logits, u = _logits(3, 4, 5000)
    _check(cuda_device, logits, u)


@pytest.mark.parametrize("V", [7, 257, 600, 768, 800, 1024, 1025, 5000, 50000])
def test_equal_logits_are_cut_by_token_id(cuda_device, V):
    # V ties: every step of the search holds them all, down to the token ids
    logits = torch.full((6, V), -3.25)
    u = torch.rand(6, 5, generator=torch.Generator().manual_seed(1), dtype=torch.float64)
    _check(cuda_device, logits, u, k=[0, 3, V - 1, 0, V // 2, 1], p=[0.5, 1.0, 1.0, 0.25, 0.5, 0.9],
           exact=True)


def test_few_distinct_logits(cuda_device):
    g = torch.Generator().manual_seed(2)
    V = 30000
    logits = torch.randint(0, 3, (5, V), generator=g).float()
    logits[4] *= 1e-7      # all in one step of the histogram
    u = torch.rand(5, 5, generator=g, dtype=torch.float64)
    _check(cuda_device, logits, u, k=[0, 10100, 4321, 25000, 12345], p=[0.9, 1.0, 0.313, 1.0, 1.0])


def test_masked_infinite_and_nan_logits(cuda_device):
    V = 3001
    logits, u = _logits(7, 6, V)
    logits[0, ::2] = -math.inf
    logits[1, 5:] = -math.inf
    logits[2, 100:2000] = math.nan
    logits[3, [17, 400]] = math.inf            # only these two have weight
    logits[4] = torch.finfo(torch.float32).min  # the mask value some programs use ...
    logits[4, 9] = 1.5                          # ... next to one candidate
    logits[5, ::3] = -0.0
    logits[5, 1::3] = 0.0
    logits[5, 2::3] = -1.0
    _check(cuda_device, logits, u, k=[0, 0, 50, 0, 10, 1500], p=[0.9, 0.5, 1.0, 1.0, 0.9, 1.0])


def test_rows_without_a_candidate(cuda_device):
    dev, V = cuda_device, 999
    logits, u = _logits(8, 6, V)
    logits[1] = -math.inf
    logits[2] = math.nan
    T = torch.tensor([1.0, 1.0, 1.0, -1.0, math.nan, 1.0], device=dev)
    p = torch.tensor([1.0, 1.0, 1.0, 1.0, 1.0, math.nan], device=dev)
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    r = tsd.sample(logits.to(dev), u.to(dev), temperature=T, top_p=p, with_probs=True, status=st)
    assert int(st.item()) == tsd.binding.DEV_BAD_ROW
    assert (r.tokens[1:] == -1).all() and (r.probs[1:] == 0).all()
    assert (r.tokens[0] >= 0).all() and abs(float(r.probs[0].double().sum()) - 1) < 1e-5


def test_extreme_uniforms(cuda_device):
    dev, V = cuda_device, 2000
    logits, _ = _logits(9, 1, V)
    u = torch.tensor([[0.0, 2.0 ** -60, 1.0 - 2.0 ** -53]], dtype=torch.float64)
    k = torch.tensor([100], dtype=torch.int32, device=dev)
    r = tsd.sample(logits.to(dev), u.to(dev), top_k=k)
    ids = torch.sort(logits[0].topk(100).indices).values
    assert r.tokens.cpu().tolist() == [[int(ids[0]), int(ids[0]), int(ids[-1])]]


@pytest.mark.parametrize("V,ld", [(1000, 1024), (1001, 1003)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rows_apart(cuda_device, V, ld, dtype):
    # a padded head's logits, and the probabilities straight into rows of q_probs
    logits, u = _logits(V, 5, ld, dtype)
    logits[:, V:] = 1e4
    big = logits.to(cuda_device)
    q = torch.full((5, 3, V), 9.0, device=cuda_device)
    _check(cuda_device, big[:, :V], u, p=[0.9] * 5, probs=q[:, 1])
    assert (q[:, 0] == 9).all() and (q[:, 2] == 9).all()


def test_large_offsets(cuda_device):
    # rows of a large matrix: the last rows lie beyond 2^31 elements
    dev, V, R = cuda_device, 360448, 6000
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("not enough memory")
    logits = torch.zeros(R, V, dtype=torch.bfloat16, device=dev)
    logits[:, 77] = 30.0
    logits[R - 1, 77], logits[R - 1, V - 1] = 0.0, 30.0
    u = torch.full((R, 1), 0.5, dtype=torch.float64, device=dev)
    r = tsd.sample(logits, u, with_probs=True)
    want = torch.full((R, 1), 77, dtype=torch.int32, device=dev)
    want[R - 1] = V - 1
    assert torch.equal(r.tokens, want)
    assert float(r.probs[R - 1, V - 1]) > 0.9


def test_same_bits_twice_and_captured(cuda_device):
    dev = cuda_device
    logits, u = _logits(11, 9, 50021)
    logits, u = logits.to(dev), u.to(dev)
    p = torch.full((9,), 0.97, device=dev)
    first = tsd.sample(logits, u, top_p=p, with_probs=True)
    again = tsd.sample(logits, u, top_p=p, with_probs=True)
    assert torch.equal(first.tokens, again.tokens) and torch.equal(first.probs, again.probs)
    g = torch.cuda.CUDAGraph()
    tok, pr = torch.zeros_like(first.tokens), torch.zeros_like(first.probs)
    with torch.cuda.graph(g):
        tsd.sample(logits, u, top_p=p, tokens=tok, probs=pr)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(first.tokens, tok) and torch.equal(first.probs, pr)


def test_no_draws_and_no_rows(cuda_device):
    logits, _ = _logits(12, 2, 100)
    u = torch.zeros(2, 0, dtype=torch.float64, device=cuda_device)
    r = tsd.sample(logits.to(cuda_device), u, with_probs=True)
    assert r.tokens.shape == (2, 0)
    assert torch.allclose(r.probs.cpu(), torch.softmax(logits, 1), atol=1e-6)
    r = tsd.sample(logits[:0].to(cuda_device), u[:0])
    assert r.tokens.shape == (0, 0)


@pytest.mark.parametrize("T,k,p", [(1.0, 0, 1.0), (1.0, 5, 1.0), (0.7, 0, 0.5), (1.0, 500, 0.9)])
def test_every_candidate_at_the_lowest_number(cuda_device, T, k, p):
    # a mask of the type's lowest value over every entry, -inf beside it
    V = 2000
    logits = torch.full((2, V), torch.finfo(torch.float32).min)
    logits[:, 100:1300] = -math.inf
    logits[1, 7] = -3.0e38
    u = torch.rand(2, 5, generator=torch.Generator().manual_seed(3), dtype=torch.float64)
    _check(cuda_device, logits, u, T=[T] * 2, k=[k] * 2, p=[p] * 2, exact=True)


def test_vocabularies_at_the_limits(cuda_device):
    logits, u = _logits(14, 2, 393216)
    _check(cuda_device, logits, u, k=[100, 0], p=[1.0, 0.6])
    with pytest.raises(tsd.TsdError):
        tsd.sample(torch.zeros(1, 393216 + 1, device=cuda_device), u[:1].to(cuda_device))


@pytest.mark.parametrize("k", [1, 32, 33, 64, 128, 129, 255])
def test_listed_and_searched_rows(cuda_device, k):
    # top_k around the sizes at which rows are listed whole, with and without top_p
    logits, u = _logits(k, 6, 30011)
    _check(cuda_device, logits, u, k=[k] * 6, p=[1.0, 0.9, 0.5, 1.0, 0.99, 0.9], m=[0.0, 0.0, 0.0, 0.2,
                                                                               0.001, 0.05])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V,T", [(300, 1.0), (5000, 0.5), (100000, 1.0), (100000, 2.0)])
def test_top_p_where_a_coarse_sum_misleads(cuda_device, V, T, dtype):
    # weights that 2^-16 steps lose, or round up by half, beside a few large ones;
    # limits in the large ones, in the body and far below
    g = torch.Generator().manual_seed(V)
    rows, p = [], []
    for depth, mid, limits in ((13.0, 0, (0.5, 0.95, 0.9995, 0.99999)),
                               (11.5, 8, (0.45, 0.56, 0.7, 0.9999)),
                               (16.0, 3, (0.9, 0.9999))):
        for limit in limits:
            x = -depth + 1e-3 * torch.randn(V, generator=g)
            at = torch.randperm(V, generator=g)[:mid + 1]
            x[at] = -3.0 - 0.01 * torch.arange(mid + 1)
            x[at[0]] = 0.0
            rows.append(T * x + 5.0)
            p.append(limit)
    x = 4.0 * torch.randn(2, V, generator=g)
    logits = torch.cat([torch.stack(rows), T * x]).to(dtype)
    p += [0.9995, 0.99]
    u = torch.rand(len(p), 3, generator=g, dtype=torch.float64)
    _check(cuda_device, logits, u, T=[T] * len(p), p=p)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V,k", [(201, 150), (250, 129), (250, 200), (254, 253), (256, 150), (256, 255)])
def test_rows_with_exactly_top_k_entries_above_the_bound(cuda_device, V, k, dtype):
    # rows that start off a 16-byte boundary: a thread holds one entry, so the
    # bound is the top_k-th largest itself; the other settings on top of it
    logits, u = _logits(V + k, 8, V + 1, dtype)
    _check(cuda_device, logits.to(cuda_device)[:, :V], u, T=[1.0, 0.7, 2.0, 1.0] * 2, k=[k] * 8,
           p=[1.0, 1.0, 1.0, 0.9] * 2, m=[0.0, 0.0, 0.02, 0.0] * 2)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("R,C", [(2, 8), (300, 0)])
def test_top_k_peaks_on_a_thread_each(cuda_device, R, C, dtype):
    # 150 peaks in each chunk of a cluster, a 16-byte vector and so a thread
    # each: top_k of them lie at or above the bound, and thousands below
    V, each = 32000, 150
    n = 128 // torch.finfo(dtype).bits
    C = C or (4 if dtype == torch.float32 else 2)
    logits, u = _logits(R, R, V, dtype, sigma=0.5)
    starts = [V // 128 * r // C * 128 for r in range(C)]
    peaks = torch.cat([s + n * torch.arange(each) for s in starts])
    logits[:, peaks] = (5.0 + torch.rand(R, len(peaks))).to(dtype)
    _check(cuda_device, logits, u, k=[C * each] * R)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,p", [(1.0, 1.0), (8.0, 1.0), (8.0, 0.9)])
def test_entries_below_the_bound_in_its_step(cuda_device, T, p, dtype):
    # the bound is 4, its step of the histogram also holds thousands at 3.95
    V, n = 4000, 128 // torch.finfo(dtype).bits
    logits = torch.full((2, V), 3.95)
    logits[:, n * torch.arange(210)] = 4.0
    logits[:, n * 255] = 30.0
    u = torch.rand(2, 5, generator=torch.Generator().manual_seed(4), dtype=torch.float64)
    _check(cuda_device, logits.to(dtype), u, T=[T] * 2, k=[200, 211], p=[p] * 2, exact=p == 1.0)


def test_probabilities_beside_their_logits(cuda_device):
    # both slices of one buffer: row r of one between rows of the other
    logits, u = _logits(15, 7, 1001)
    both = torch.full((7, 2, 1001), 9.0, device=cuda_device)
    both[:, 0] = logits.to(cuda_device)
    _check(cuda_device, both[:, 0], u, p=[0.9] * 7, probs=both[:, 1])
    assert torch.equal(both[:, 0].cpu(), logits)
