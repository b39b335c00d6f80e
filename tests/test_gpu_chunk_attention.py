"""Chunk attention over pages (chunk_attention_paged) against the formula in 64 bits.

With A = sum_j p_j |v_j| for exact probabilities p, and S the largest sum of
|q_d k_d| scale over the visible keys:
  * bf16: each p_j is rounded for the product with V, 2^-8 of it at most; the
    scores' fp32 accumulation moves an exponent by D 2^-23 S at most and with
    it a probability and the sum (twice); exponentials, sums and O in fp32 are
    below 2^-12 together; the output rounds by 2^-8 of itself:
        2^-8 (A + |out|) + A (2 D 2^-23 S + 2^-12).
  * fp32: scores 2 (D + 4) 2^-24 S, sums over n keys 2 (n + 8) 2^-24,
    exponentials and output 2^-21, all times A.
"""

import pytest
import torch

import tree_speculative_decoding_ancestor_b200 as tsd
from paged_util import DTYPES, block_table, pool

pytestmark = pytest.mark.gpu

FILL = 3.0


def _case(seed, dt, Hq, Hkv, D, page, prefix, new, T, dev, poison=True):
    g = torch.Generator().manual_seed(seed)
    B = len(prefix)
    total = [p + n for p, n in zip(prefix, new)]
    table, num = block_table(total, page, seed)
    kp, vp = (pool(num, Hkv, page, D, dt, seed + i) for i in (1, 2))
    q = torch.randn(B, T, Hq, D, generator=g).to(dt)
    if poison:   # everything that no row may see: spare pages, slots behind the last token
        live = torch.zeros(num, page, dtype=torch.bool)
        for b, n in enumerate(total):
            pos = torch.arange(n)
            live[table[b].long()[pos // page], pos % page] = True
        for x, bad in ((kp, float("nan")), (vp, float("inf"))):
            x.transpose(1, 2)[~live] = bad
        for b, n in enumerate(new):
            q[b, n:] = float("nan")
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
    return q.to(dev), kp.to(dev), vp.to(dev), table.to(dev), i32(prefix), i32(new)


def _reference(q, kp, vp, table, P, n, scale):
    """(out, A, S) [n][Hq][D] (S: [n][Hq][1]) of one sequence in 64 bits."""
    Hkv, page, D = kp.shape[1:]
    Hq = q.shape[1]
    G = Hq // Hkv
    pos = torch.arange(P + n, device=q.device)
    where = table.long()[pos // page]
    k = kp[where, :, pos % page].double().transpose(0, 1)
    v = vp[where, :, pos % page].double().transpose(0, 1)
    out = torch.empty(n, Hq, D, dtype=torch.float64, device=q.device)
    A, S = torch.empty_like(out), torch.empty(n, Hq, 1, dtype=torch.float64, device=q.device)
    step = max(1, (1 << 24) // max(1, G * (P + n)))
    for h in range(Hkv):
        for t0 in range(0, n, step):
            t = torch.arange(t0, min(n, t0 + step), device=q.device)
            x = q[t, h * G:(h + 1) * G].double()
            s = torch.einsum("tgd,jd->tgj", x, k[h]) * scale
            mask = pos[None, None] > (P + t)[:, None, None]
            p = torch.softmax(s.masked_fill(mask, float("-inf")), -1)
            out[t, h * G:(h + 1) * G] = p @ v[h]
            A[t, h * G:(h + 1) * G] = p @ v[h].abs()
            sa = torch.einsum("tgd,jd->tgj", x.abs(), k[h].abs()) * scale
            S[t, h * G:(h + 1) * G, 0] = sa.masked_fill(mask, 0.0).amax(-1)
    return out, A, S


def _check(args, scale=None, out=None, **kw):
    q, kp, vp, table, P, n = args
    D, dt = q.shape[-1], q.dtype
    out = torch.full_like(q, FILL) if out is None else out
    st = torch.zeros(1, dtype=torch.int32, device=q.device)
    got = tsd.chunk_attention_paged(q, kp, vp, table, P, n, scale=scale, out=out, status=st, **kw)
    assert got is out and int(st.item()) == 0
    sc = D ** -0.5 if scale is None else scale
    for b in range(q.shape[0]):
        m = int(n[b])
        assert (out[b, m:] == FILL).all()
        if not m:
            continue
        want, A, S = _reference(q[b, :m], kp, vp, table[b], int(P[b]), m, sc)
        if dt == torch.bfloat16:
            tol = 2.0 ** -8 * (A + want.abs()) + A * (2 * D * 2.0 ** -23 * S + 2.0 ** -12)
        else:
            keys = int(P[b]) + m
            tol = A * (2 * (D + 4) * 2.0 ** -24 * S + 2 * (keys + 8) * 2.0 ** -24 + 2.0 ** -21)
        err = (out[b, :m].double() - want).abs()
        assert (err <= tol).all(), (b, float((err / tol).max()))
    return out


HEADS = [(8, 1), (4, 4), (14, 2), (64, 8), (6, 3)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", HEADS)
@pytest.mark.parametrize("page", [16, 64, 256])
def test_one_token(cuda_device, dtype, D, Hq, Hkv, page):
    prefix = [0, 1, 62, 63, 64, 65, 127, 300, 15, 1000]
    _check(_case(D + Hq, DTYPES[dtype], Hq, Hkv, D, page, prefix, [1] * 9 + [0], 1, cuda_device))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hkv,T,page", [(8, 1, 129, 16), (4, 4, 200, 32), (14, 2, 37, 128),
                                           (2, 2, 128, 64), (6, 3, 65, 4096), (8, 2, 5, 16)])
def test_ragged_chunks(cuda_device, dtype, D, Hq, Hkv, T, page):
    prefix = [0, 0, 63, 130, 17, 500]
    new = [T, 1, T - 1, 0, T // 2, T]
    _check(_case(T + D, DTYPES[dtype], Hq, Hkv, D, page, prefix, new, T, cuda_device))


@pytest.mark.parametrize("dtype,Hq,Hkv,D,T,page", [("bf16", 64, 8, 128, 700, 128),
                                                   ("bf16", 32, 16, 64, 2400, 16),
                                                   ("f32", 16, 16, 64, 2600, 64)])
def test_long_chunks_one_block_each(cuda_device, dtype, Hq, Hkv, D, T, page):
    # more row blocks than the keys are split for: no partial results
    args = _case(T, DTYPES[dtype], Hq, Hkv, D, page, [300, 0], [T, T - 131], T, cuda_device)
    assert tsd.chunk_attention_workspace_size(2, T, Hq, Hkv, D, page, args[3].shape[1],
                                              DTYPES[dtype]) == 0
    _check(args)


@pytest.mark.parametrize("dtype,B,Hq,Hkv,D,T,P", [("bf16", 1, 8, 2, 128, 1, 70000),
                                                  ("bf16", 33, 8, 8, 128, 1, 600),
                                                  ("bf16", 2, 16, 2, 64, 40, 5000),
                                                  ("f32", 1, 4, 1, 128, 1, 9000),
                                                  ("f32", 1, 32, 2, 64, 33, 3001)])
def test_long_prefixes_are_split(cuda_device, dtype, B, Hq, Hkv, D, T, P):
    prefix = [P] + [(P * (b + 1)) // (3 * B) for b in range(B - 1)]   # one long, the rest short
    args = _case(P, DTYPES[dtype], Hq, Hkv, D, 64, prefix, [T] * B, T, cuda_device)
    assert tsd.chunk_attention_workspace_size(B, T, Hq, Hkv, D, 64, args[3].shape[1],
                                              DTYPES[dtype]) > 0
    _check(args)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,Hkv,T,P", [(148, 1, 1, 40), (37, 8, 1, 700), (300, 2, 2, 90), (5, 3, 200, 3),
                                       (64, 2, 70, 500), (2, 64, 1, 2500)])
def test_ranges_over_many_blocks(cuda_device, dtype, B, Hkv, T, P):
    # ranges that hold several blocks, cut some, and skip sequences without tokens
    prefix = [(P * (7 * b + 3)) % (P + 1) for b in range(B)]
    new = [0 if b % 5 == 4 else 1 + (3 * b) % T for b in range(B)]
    _check(_case(B + T, DTYPES[dtype], 2 * Hkv, Hkv, 64, 16, prefix, new, T, cuda_device))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Hq,T", [(130, 1), (130, 3), (256, 2)])
def test_more_heads_than_a_block_has_rows(cuda_device, dtype, Hq, T):
    _check(_case(Hq + T, DTYPES[dtype], Hq, 1, 64, 32, [100, 0, 40], [T, T, 1], T, cuda_device))


def test_no_tokens_at_all(cuda_device):
    for dt in DTYPES.values():
        _check(_case(3, dt, 4, 2, 64, 16, [0, 33], [0, 0], 3, cuda_device))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_scores_that_rise_and_dominate(cuda_device, dtype):
    # each later key scores higher (the running maximum moves at every tile),
    # one key dwarfs the rest, and a scale of its own
    dt = DTYPES[dtype]
    q, kp, vp, table, P, n = _case(5, dt, 8, 2, 64, 16, [900, 70], [130, 130], 130, cuda_device)
    Hkv, D = 2, 64
    for b in range(2):
        total = int(P[b]) + 130
        pos = torch.arange(total, device=cuda_device)
        ramp = (pos.float() / 20.0)[:, None, None]
        kp[table[b].long()[pos // 16], :, pos % 16] = (torch.ones(total, Hkv, D, device=cuda_device)
                                                       * ramp).to(dt)
    kp[table[0, 3], :, 5] = 60.0
    q.fill_(1.0)
    _check((q, kp, vp, table, P, n), scale=0.05)


def test_matches_tree_attention_on_a_chain(cuda_device):
    dev, T = cuda_device, 40
    q, kp, vp, table, P, n = _case(6, torch.bfloat16, 8, 2, 128, 64, [100, 0, 777], [40, 1, 17], T, dev,
                                   poison=False)
    parent = torch.arange(-1, T - 1, dtype=torch.int32, device=dev).repeat(3, 1)
    tree = tsd.tree_mask_build(parent, n)
    a = tsd.tree_attention_paged(q, kp, vp, table, P, n, tree.mask)
    b = tsd.chunk_attention_paged(q, kp, vp, table, P, n)
    for i in range(3):
        m = int(n[i])
        assert (a[i, :m].float() - b[i, :m].float()).abs().max() <= 4e-2


def test_bad_lengths_and_pages(cuda_device):
    dev = cuda_device
    for dt in (torch.bfloat16, torch.float32):
        q, kp, vp, table, P, n = _case(7, dt, 8, 2, 64, 16, [40] * 5, [3] * 5, 4, dev, poison=False)
        good = tsd.chunk_attention_paged(q, kp, vp, table, P, n)
        st = torch.zeros(1, dtype=torch.int32, device=dev)
        n2, P2, t2 = n.clone(), P.clone(), table.clone()
        n2[0], P2[1], P2[2] = 5, -1, table.shape[1] * 16 - 2
        t2[3, 1] = kp.shape[0]
        out = torch.full_like(q, FILL)
        tsd.chunk_attention_paged(q, kp, vp, t2, P2, n2, out=out, status=st)
        assert int(st.item()) == tsd.binding.DEV_BAD_PREFIX | tsd.binding.DEV_BAD_PAGE
        assert (out[:3] == FILL).all()
        assert torch.equal(out[4, :3], good[4, :3]) and torch.isfinite(out[3, :3].float()).all()


def test_entries_behind_the_last_key_are_not_read(cuda_device):
    # the table's tail holds ids outside the pool (block_table fills it so): no flag
    _check(_case(8, torch.bfloat16, 4, 2, 128, 16, [15, 31], [1, 1], 1, cuda_device))


def test_two_streams_and_two_graphs_side_by_side(cuda_device):
    dev = cuda_device
    cases = [_case(20 + i, torch.bfloat16, 16, 2, 128, 64, [4000, 100 + i], [1, 1], 1, dev) for i in (0, 1)]
    want = [tsd.chunk_attention_paged(*c) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    outs = [torch.zeros_like(c[0]) for c in cases]
    for _ in range(20):
        for s, c, o in zip(streams, cases, outs):
            with torch.cuda.stream(s):
                tsd.chunk_attention_paged(*c, out=o)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, outs))
    graphs = []
    for c, o in zip(cases, outs):   # captured on one stream, replayed on two
        o.zero_()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            tsd.chunk_attention_paged(*c, out=o)
        graphs.append(g)
    for _ in range(20):
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, outs))


def test_lengths_on_the_device_may_change_between_replays(cuda_device):
    dev = cuda_device
    q, kp, vp, table, P, n = _case(30, torch.bfloat16, 8, 2, 128, 64, [2000, 1500], [4, 4], 4, dev,
                                   poison=False)
    out = torch.zeros_like(q)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        tsd.chunk_attention_paged(q, kp, vp, table, P, n, out=out)
    for p, m in (([10, 0], [1, 4]), ([2000, 3], [4, 0]), ([0, 1500], [2, 3])):
        P.copy_(torch.tensor(p, dtype=torch.int32))
        n.copy_(torch.tensor(m, dtype=torch.int32))
        out.fill_(FILL)
        g.replay()
        fresh = _check((q, kp, vp, table, P, n))
        assert torch.equal(out, fresh)


@pytest.mark.parametrize("dtype,Hq,Hkv,D,T", [("bf16", 4, 4, 64, 512), ("bf16", 16, 2, 128, 70),
                                              ("f32", 4, 4, 64, 130)])
def test_replays_with_lengths_that_change_how_work_is_divided(cuda_device, dtype, Hq, Hkv, D, T):
    # short lengths are served block by block, a long one next to a short one by ranges
    dev = cuda_device
    q, kp, vp, table, P, n = _case(40 + T, DTYPES[dtype], Hq, Hkv, D, 64, [9000, 400], [T, T], T, dev,
                                   poison=False)
    assert tsd.chunk_attention_workspace_size(2, T, Hq, Hkv, D, 64, table.shape[1], DTYPES[dtype]) > 0
    out = torch.zeros_like(q)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        tsd.chunk_attention_paged(q, kp, vp, table, P, n, out=out)
    for p, m in (([0, 0], [T, T]), ([9000, 400], [T, 1]), ([0, 0], [T, 3]), ([9000, 0], [T // 2, T]),
                 ([3, 1], [0, T]), ([0, 0], [0, 0])):
        P.copy_(torch.tensor(p, dtype=torch.int32))
        n.copy_(torch.tensor(m, dtype=torch.int32))
        out.fill_(FILL)
        g.replay()
        fresh = _check((q, kp, vp, table, P, n))
        assert torch.equal(out, fresh)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("prefix", [[9000, 400], [10, 0]])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_query_row_that_is_not_a_number_shows(cuda_device, dtype, prefix, bad):
    # whether its keys are served by one CTA or joined from pieces; inf - inf and
    # inf * 0 are no numbers either; every other row as if it were not there
    args = _case(50, DTYPES[dtype], 8, 2, 64, 64, prefix, [4, 2], 4, cuda_device, poison=False)
    good = tsd.chunk_attention_paged(*args)
    q = args[0].clone()
    q[0, 1, 3, 5] = q[1, 0, 7, 0] = bad
    out = tsd.chunk_attention_paged(q, *args[1:])
    hit = torch.zeros(out.shape[:3], dtype=torch.bool, device=cuda_device)
    hit[0, 1, 3] = hit[1, 0, 7] = True
    assert torch.isnan(out[hit].float()).all()
    for b, n in enumerate((4, 2)):
        keep = ~hit[b, :n]
        assert torch.equal(out[b, :n][keep], good[b, :n][keep])
