"""Commit of accepted paths in a paged cache (kv_commit_paged): rows are moved,
so the pools must equal the definition bit for bit, every other row included."""

import pytest
import torch

import tree_speculative_decoding_ancestor_b200 as tsd
from paged_util import DTYPES, block_table, pool, raw

pytestmark = pytest.mark.gpu


def _commit(dev, kp, vp, table, prefix, paths, T, status=None):
    B = len(prefix)
    path = torch.full((B, T), -9, dtype=torch.int32)
    n = torch.tensor([len(p) if p is not None else -1 for p in paths], dtype=torch.int32)
    for b, p in enumerate(paths):
        if p:
            path[b, :min(len(p), T)] = torch.tensor(p[:T], dtype=torch.int32)
    kd, vd = kp.to(dev), vp.to(dev)
    res = tsd.VerifyResult(torch.zeros(B, T + 1, dtype=torch.int32, device=dev), path.to(dev), n.to(dev))
    new = tsd.kv_commit_paged(kd, vd, table.to(dev), torch.tensor(prefix, dtype=torch.int32, device=dev),
                              res, status=status)
    return kd.cpu(), vd.cpu(), new.cpu().tolist()


def _want(pages, table, prefix, paths):
    out, page = pages.clone(), pages.shape[2]
    for b, (P, path) in enumerate(zip(prefix, paths)):
        for i, u in enumerate(path or []):
            src, dst = P + u, P + i
            out[table[b, dst // page], :, dst % page] = pages[table[b, src // page], :, src % page]
    return out


@pytest.mark.parametrize("dtype,D,page", [("bf16", 128, 16), ("bf16", 64, 64), ("f32", 128, 16),
                                          ("f32", 64, 32), ("bf16", 8, 256)])
@pytest.mark.parametrize("Hkv", [1, 3])
def test_rows_move_across_pages(cuda_device, dtype, D, page, Hkv):
    T = 128
    prefix = [0, 15, 16, 31, 100, 5, 7, 1000]
    paths = [[0, 2, 3], [1], [], list(range(1, 128, 2)), list(range(128)), [0, 1, 2, 70, 127], None,
             [127]]
    table, num = block_table([p + T for p in prefix], page, D + page)
    kp, vp = (pool(num, Hkv, page, D, DTYPES[dtype], s) for s in (1, 2))
    kp[:, :, ::3] = float("nan")     # rows are copied, whatever they hold
    st = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    k, v, new = _commit(cuda_device, kp, vp, table, prefix, paths, T, st)
    assert int(st.item()) == 0
    assert new == [P + len(p or []) for P, p in zip(prefix, paths)]
    assert (raw(k) == raw(_want(kp, table, prefix, paths))).all()
    assert (raw(v) == raw(_want(vp, table, prefix, paths))).all()


def test_matches_the_contiguous_commit(cuda_device):
    dev, T, page, P = cuda_device, 20, 16, 37
    table = torch.arange(4, dtype=torch.int32)[None]
    kp, vp = (pool(4, 2, page, 64, torch.bfloat16, s) for s in (3, 4))
    flat = [x.transpose(0, 1).reshape(1, 2, 64, 64).contiguous().to(dev) for x in (kp, vp)]
    path = torch.full((1, T), -1, dtype=torch.int32)
    path[0, :4] = torch.tensor([1, 4, 9, 19])
    res = tsd.VerifyResult(torch.zeros(1, T + 1, dtype=torch.int32, device=dev), path.to(dev),
                           torch.tensor([4], dtype=torch.int32, device=dev))
    tsd.kv_commit(flat[0], flat[1], torch.tensor([P], dtype=torch.int32, device=dev), res)
    k, v, new = _commit(dev, kp, vp, table, [P], [[1, 4, 9, 19]], T)
    assert new == [P + 4]
    for a, b in ((k, flat[0]), (v, flat[1])):
        assert torch.equal(a.transpose(0, 1).reshape(1, 2, 64, 64), b.cpu())


def test_malformed_paths_and_pages_move_nothing(cuda_device):
    T, page = 8, 16
    prefix = [10, 10, 10, 10, 10, 2147483647, -3]
    paths = [[3, 2], [0, 8], [0, 1, 2, 3, 4, 5, 6, 7, 7], [5, 7], [6, 7], [1], [1]]
    table, num = block_table([18] * 7, page, 5)
    table[3, 1] = num          # the source page of sequence 3's second move
    table[4, 1] = -1           # both of sequence 4's sources
    kp, vp = (pool(num, 2, page, 64, torch.bfloat16, s) for s in (1, 2))
    st = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    k, v, new = _commit(cuda_device, kp, vp, table, prefix, paths, T, st)
    assert int(st.item()) == tsd.binding.DEV_BAD_PATH | tsd.binding.DEV_BAD_PAGE
    assert new == prefix
    assert torch.equal(k, kp) and torch.equal(v, vp)
    # rows already in place need no page
    st.zero_()
    k, v, new = _commit(cuda_device, kp, vp, table, [10] * 7, [[0, 1, 2, 3, 4, 5, 6, 7]] * 7, T, st)
    assert int(st.item()) == 0 and new == [18] * 7 and torch.equal(k, kp)


def test_reaching_past_the_table(cuda_device):
    T, page = 8, 16
    table = torch.tensor([[0, 1]], dtype=torch.int32)
    kp, vp = (pool(2, 1, page, 64, torch.bfloat16, s) for s in (1, 2))
    st = torch.zeros(1, dtype=torch.int32, device=cuda_device)
    k, _, new = _commit(cuda_device, kp, vp, table, [25], [[3, 7]], T, st)
    assert int(st.item()) == tsd.binding.DEV_BAD_PATH and new == [25] and torch.equal(k, kp)
    st.zero_()
    k, _, new = _commit(cuda_device, kp, vp, table, [24], [[3, 7]], T, st)
    assert int(st.item()) == 0 and new == [26]
    assert torch.equal(k, _want(kp, table, [24], [[3, 7]]))
