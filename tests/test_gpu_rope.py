"""Rotary append (rope_append_paged) against the rotation in 64 bits.

Error budget per output (|x| + |o|: the pair's magnitudes, g: rot_scale): the
reduced angle rounds to fp32 (half an ulp of values below 4: 2^-23), cosine
and sine are within 2 ulp (2 * 2^-24), the factor g and the two products
round (about 3 * 2^-24): 2^-21 (|x| + |o|) g in all, then one rounding to the
output's type, eps / 2 of the value.
"""

import pytest
import torch

import tree_speculative_decoding_ancestor_b200 as tsd
from paged_util import DTYPES, block_table, logical, pool, raw

pytestmark = pytest.mark.gpu

FILL = 7.0   # what untouched outputs hold


def _inputs(seed, dt, B, T, Hq, Hkv, D, page, prefix, new, fused):
    g = torch.Generator().manual_seed(seed)
    if fused:
        qkv = torch.randn(B, T, Hq + 2 * Hkv, D, generator=g).to(dt)
        q, k, v = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hkv], qkv[:, :, Hq + Hkv:]
    else:
        q, k, v = (torch.randn(B, T, h, D, generator=g).to(dt) for h in (Hq, Hkv, Hkv))
    table, num = block_table([p + n for p, n in zip(prefix, new)], page, seed)
    return q, k, v, table, pool(num, Hkv, page, D, dt, seed + 1), pool(num, Hkv, page, D, dt, seed + 2)


def _rotate(x, pos, inv_freq, interleaved, scale):
    """(rotated, |x| + |o|) of x [n][H][D] in 64 bits."""
    rot = 2 * inv_freq.numel()
    y, mag = x.double().clone(), x.double().abs()
    angle = pos.double()[:, None, None] * inv_freq
    c, s = scale * angle.cos(), scale * angle.sin()
    sel = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2),
                                                                   slice(rot // 2, rot))
    a, b = x[..., sel[0]].double(), x[..., sel[1]].double()
    y[..., sel[0]], y[..., sel[1]] = a * c - b * s, b * c + a * s
    for i in sel:
        mag[..., i] = scale * (a.abs() + b.abs())
    return y, mag


def _close(got, want, mag, dt, rot):
    want, mag = want[..., :rot], mag[..., :rot]
    delta = 2.0 ** -21 * mag
    tol = delta + torch.finfo(dt).eps / 2 * (want.abs() + delta)
    assert ((got[..., :rot].double() - want).abs() <= tol).all()


def _check(dev, seed, dt, Hq, Hkv, D, rot, interleaved, page, prefix, new, T, fused=False, tree=False,
           scale=1.0):
    B = len(prefix)
    q, k, v, table, kp, vp = _inputs(seed, dt, B, T, Hq, Hkv, D, page, prefix, new, fused)
    inv = tsd.rope_frequencies(rot).inv_freq
    depth = None
    if tree:
        g = torch.Generator().manual_seed(seed)
        depth = torch.randint(1, 9, (B, T), generator=g, dtype=torch.int32)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
    out = torch.full((B, T, Hq, D), FILL, dtype=dt, device=dev)
    kd, vd = kp.to(dev), vp.to(dev)
    if fused:
        qkv = torch.cat([q, k, v], dim=2).to(dev)
        qd, k_d, v_d = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hkv], qkv[:, :, Hq + Hkv:]
    else:
        qd, k_d, v_d = q.to(dev), k.to(dev), v.to(dev)
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    got = tsd.rope_append_paged(qd, k_d, v_d, inv.to(dev), kd, vd, table.to(dev), i32(prefix),
                                i32(new), depth=None if depth is None else depth.to(dev),
                                interleaved=interleaved, rot_scale=scale, out=out, status=st)
    assert got is out and int(st.item()) == 0
    out, kd, vd = out.cpu(), kd.cpu(), vd.cpu()
    want_k, want_v = kp.clone(), vp.clone()
    for b, (P, n) in enumerate(zip(prefix, new)):
        t = torch.arange(n)
        pos = P + (t if depth is None else depth[b, :n].long() - 1)
        yq, mq = _rotate(q[b, :n], pos, inv, interleaved, scale)
        _close(out[b, :n], yq, mq, dt, rot)
        assert (raw(out[b, :n, :, rot:].contiguous()) == raw(q[b, :n, :, rot:].contiguous())).all()
        assert (out[b, n:] == FILL).all()
        yk, mk = _rotate(k[b, :n], pos, inv, interleaved, scale)
        rows = logical(kd, table[b], P + n)[:, P:].transpose(0, 1)
        _close(rows, yk, mk, dt, rot)
        where, row = table[b].long()[(P + t) // page], (P + t) % page
        want_k[where, :, row] = torch.cat([rows[..., :rot], k[b, :n, :, rot:]], dim=-1)
        want_v[where, :, row] = v[b, :n]
    assert (raw(kd) == raw(want_k)).all()   # pass-through dimensions and all other rows
    assert (raw(vd) == raw(want_v)).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,rot", [(128, 128), (128, 64), (64, 24), (64, 2), (80, 20), (8, 8)])
def test_rotation_and_append(cuda_device, dtype, interleaved, D, rot):
    _check(cuda_device, D + rot, DTYPES[dtype], 6, 2, D, rot, interleaved, 16, [0, 17, 100003 % 777, 5],
           [7, 0, 5, 1], 7)


@pytest.mark.parametrize("dtype,fused,tree,scale", [("bf16", True, True, 1.0), ("f32", True, False, 1.25),
                                                    ("bf16", False, True, 0.5)])
def test_projection_columns_trees_and_scale(cuda_device, dtype, fused, tree, scale):
    _check(cuda_device, 3, DTYPES[dtype], 8, 2, 128, 128, False, 32, [31, 32, 33, 64], [64, 20, 33, 1],
           64, fused=fused, tree=tree, scale=scale)


@pytest.mark.parametrize("B,T", [(1, 1), (8, 1), (1, 1031), (70, 3)])
def test_sizes_of_the_grid(cuda_device, B, T):
    prefix = [(37 * b) % 211 for b in range(B)]
    new = [T - b % T if T > 1 else 1 for b in range(B)]
    _check(cuda_device, B + T, torch.bfloat16, 7, 7, 64, 64, False, 64, prefix, new, T)


def test_far_positions(cuda_device):
    # one page of each far sequence exists; the entries before it are never read
    dev, page, D = cuda_device, 256, 64
    prefix, B = [1 << 20, 4_000_005], 2
    table = torch.full((B, (1 << 22) // page), -5, dtype=torch.int32)
    for b, P in enumerate(prefix):
        table[b, P // page] = b
    q = torch.randn(B, 2, 1, D)
    kp = torch.zeros(2, 1, page, D, device=dev)
    inv = tsd.rope_frequencies(D).inv_freq
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    n = torch.tensor([2, 2], dtype=torch.int32, device=dev)
    out = tsd.rope_append_paged(q.to(dev), q.to(dev), q.to(dev), inv.to(dev), kp, kp.clone(),
                                table.to(dev), torch.tensor(prefix, dtype=torch.int32, device=dev), n,
                                status=st)
    assert int(st.item()) == 0
    for b, P in enumerate(prefix):
        want, mag = _rotate(q[b], P + torch.arange(2), inv, False, 1.0)
        _close(out[b].cpu(), want, mag, torch.float32, D)
        _close(kp[b, 0, P % page:P % page + 2].cpu()[:, None], want, mag, torch.float32, D)


def test_bad_lengths_and_pages_are_flagged(cuda_device):
    dev, dt, page = cuda_device, torch.bfloat16, 16
    prefix, new = [20, 20, 20, -1], [4, 9, 4, 4]      # sequence 1: more than Tmax; 3: negative
    q, k, v, table, kp, vp = _inputs(5, dt, 4, 8, 2, 1, 64, page, [20] * 4, [4] * 4, False)
    table[2, 1] = kp.shape[0]                          # the page of sequence 2's tokens
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
    kd, vd = kp.to(dev), vp.to(dev)
    out = torch.full((4, 8, 2, 64), FILL, dtype=dt, device=dev)
    inv = tsd.rope_frequencies(64).inv_freq.to(dev)
    st = i32([0])
    tsd.rope_append_paged(q.to(dev), k.to(dev), v.to(dev), inv, kd, vd, table.to(dev), i32(prefix),
                          i32(new), out=out, status=st)
    assert int(st.item()) == tsd.binding.DEV_BAD_PREFIX | tsd.binding.DEV_BAD_PAGE
    assert (out[1] == FILL).all() and (out[3] == FILL).all()
    assert (out[2, :4] != FILL).any() and (out[2, 4:] == FILL).all()
    changed = (raw(kd.cpu()) != raw(kp)).flatten(1).any(1)
    assert changed.nonzero().flatten().tolist() == [int(table[0, 1])]
    # past the table's last position
    st.zero_()
    cap = table.shape[1] * page
    tsd.rope_append_paged(q.to(dev), k.to(dev), v.to(dev), inv, kd, vd, table.to(dev),
                          i32([cap - 3] * 4), i32([4] * 4), out=out, status=st)
    assert int(st.item()) == tsd.binding.DEV_BAD_PREFIX


def test_captured_on_another_stream(cuda_device):
    dev, dt = cuda_device, torch.bfloat16
    q, k, v, table, kp, vp = (x.to(dev) for x in _inputs(9, dt, 2, 5, 4, 2, 128, 16, [9, 30], [5, 3],
                                                         False))
    n, P = (torch.tensor(x, dtype=torch.int32, device=dev) for x in ([5, 3], [9, 30]))
    inv = tsd.rope_frequencies(128).inv_freq.to(dev)
    want = tsd.rope_append_paged(q, k, v, inv, kp, vp, table, P, n, out=torch.zeros_like(q))
    k2, v2, out = torch.zeros_like(kp), torch.zeros_like(vp), torch.zeros_like(q)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        tsd.rope_append_paged(q, k, v, inv, k2, v2, table, P, n, out=out)
    q.mul_(2.0)      # a replay reads the inputs anew
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out.float(), 2.0 * want.float())
    for b in range(2):
        p, m = int(P[b]), int(n[b])
        for new, old in ((k2, kp), (v2, vp)):
            a, c = (logical(x.cpu(), table[b].cpu(), p + m)[:, p:] for x in (new, old))
            assert torch.equal(a, c)
