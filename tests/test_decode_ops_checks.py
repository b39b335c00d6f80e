"""Argument checks and host arithmetic of the decoding-loop operators (CPU only).

The library is replaced by a stand-in that records the calls, as in
test_binding_checks; the C entry points' own checks run on fake addresses,
which never reach a launch.
"""

import math

import pytest
import torch

import tree_speculative_decoding_ancestor_b200 as tsd
from tree_speculative_decoding_ancestor_b200 import binding
from test_binding_checks import lib  # noqa: F401  (fixture)

i32 = dict(dtype=torch.int32)
bf = dict(dtype=torch.bfloat16)
B, T, Hq, Hkv, D, page = 2, 5, 4, 2, 64, 16


def _cache(dtype=torch.bfloat16):
    return dict(k_pages=torch.zeros(6, Hkv, page, D, dtype=dtype),
                v_pages=torch.zeros(6, Hkv, page, D, dtype=dtype),
                block_table=torch.zeros(B, 3, **i32))


def _rope(**kw):
    a = dict(q=torch.zeros(B, T, Hq, D, **bf), k=torch.zeros(B, T, Hkv, D, **bf),
             v=torch.zeros(B, T, Hkv, D, **bf), inv_freq=torch.ones(D // 2, dtype=torch.float64),
             prefix_len=torch.zeros(B, **i32), n_new=torch.zeros(B, **i32), **_cache())
    a.update(kw)
    return tsd.rope_append_paged(**a)


def _commit(**kw):
    a = dict(prefix_len=torch.zeros(B, **i32),
             result=tsd.VerifyResult(torch.zeros(B, T + 1, **i32), torch.zeros(B, T, **i32),
                                     torch.zeros(B, **i32)), **_cache())
    a.update(kw)
    return tsd.kv_commit_paged(**a)


def test_rope_arguments(lib):  # noqa: F811
    assert _rope().shape == (B, T, Hq, D)
    qkv = torch.zeros(B, T, Hq + 2 * Hkv, D, **bf)
    _rope(q=qkv[:, :, :Hq], k=qkv[:, :, Hq:Hq + Hkv], v=qkv[:, :, Hq + Hkv:],
          depth=torch.ones(B, T, **i32))
    n = len(lib.calls)
    with pytest.raises(ValueError):     # heads interleaved inside a token
        _rope(q=torch.zeros(B, T, D, Hq, **bf).transpose(2, 3))
    with pytest.raises(TypeError):
        _rope(inv_freq=torch.ones(D // 2))
    with pytest.raises(TypeError):
        _rope(k=torch.zeros(B, T, Hkv, D))
    with pytest.raises(ValueError):
        _rope(v=torch.zeros(B, T + 1, Hkv, D, **bf))
    with pytest.raises(ValueError):
        _rope(block_table=torch.zeros(B + 1, 3, **i32))
    with pytest.raises(TypeError):
        _rope(q=torch.zeros(B, T, Hq, D, dtype=torch.float16))
    with pytest.raises(TypeError):
        _rope(k_pages=torch.zeros(6, Hkv, page, D))
    q = torch.zeros(B, T, Hq, D, **bf)
    with pytest.raises(ValueError, match="overlap"):
        _rope(q=q, out=q)
    with pytest.raises(ValueError):
        _rope(depth=torch.ones(B, T - 1, **i32))
    assert len(lib.calls) == n


def test_commit_arguments(lib):  # noqa: F811
    assert _commit().shape == (B,)
    n = len(lib.calls)
    P = torch.zeros(B, **i32)
    with pytest.raises(ValueError, match="overlap"):
        _commit(prefix_len=P, new_prefix_len=P)
    with pytest.raises(ValueError):
        _commit(v_pages=torch.zeros(5, Hkv, page, D, **bf))
    with pytest.raises(TypeError):
        _commit(block_table=torch.zeros(B, 3, dtype=torch.int64))
    assert len(lib.calls) == n


def _sample(R=3, V=50, S=2, **kw):
    a = dict(logits=torch.zeros(R, V), u=torch.zeros(R, S, dtype=torch.float64))
    a.update(kw)
    return tsd.sample(**a)


def test_sample_arguments(lib):  # noqa: F811
    r = _sample()
    assert r.tokens.shape == (3, 2) and r.probs is None
    assert _sample(with_probs=True).probs.shape == (3, 50)
    q = torch.zeros(3, 4, 50)
    assert _sample(probs=q[:, 1]).probs.data_ptr() == q[:, 1].data_ptr()   # a row of q_probs
    _sample(logits=torch.zeros(3, 64, **bf)[:, :50], temperature=torch.ones(3),
            top_k=torch.ones(3, **i32), top_p=torch.ones(3), min_p=torch.ones(3))
    n = len(lib.calls)
    for bad in (dict(u=torch.zeros(2, 2, dtype=torch.float64)), dict(temperature=torch.ones(2)),
                dict(logits=torch.zeros(50, 3).t()), dict(probs=torch.zeros(3, 49)),
                dict(probs=torch.zeros(1, 50).expand(3, 50)), dict(logits=torch.zeros(50)),
                dict(tokens=torch.zeros(3, 3, **i32))):
        with pytest.raises(ValueError):
            _sample(**bad)
    for bad in (dict(u=torch.zeros(3, 2)), dict(top_k=torch.ones(3)), dict(top_p=torch.ones(3, **bf)),
                dict(logits=torch.zeros(3, 50, dtype=torch.float16)), dict(probs=torch.zeros(3, 50, **bf)),
                dict(temperature=1.0)):
        with pytest.raises(TypeError):
            _sample(**bad)
    x = torch.zeros(3, 50)
    with pytest.raises(ValueError, match="overlap"):
        _sample(logits=x, probs=x)
    assert len(lib.calls) == n


def _chunk(**kw):
    a = dict(q=torch.zeros(B, T, Hq, D, **bf), prefix_len=torch.zeros(B, **i32),
             chunk_len=torch.zeros(B, **i32), workspace=torch.empty(64, dtype=torch.uint8), **_cache())
    a.update(kw)
    return tsd.chunk_attention_paged(**a)


def test_chunk_arguments(lib):  # noqa: F811
    assert _chunk().shape == (B, T, Hq, D)
    n = len(lib.calls)
    q = torch.zeros(B, T, Hq, D, **bf)
    for bad in (dict(q=q, out=q), dict(out=q[:, :T - 1]), dict(chunk_len=torch.zeros(B + 1, **i32)),
                dict(q=torch.zeros(B, Hq, T, D, **bf).transpose(1, 2)),
                dict(block_table=torch.zeros(B, **i32)), dict(q=q[0]),
                dict(v_pages=torch.zeros(6, Hkv, page, 128, **bf))):
        with pytest.raises(ValueError):
            _chunk(**bad)
    for bad in (dict(q=q.float()), dict(prefix_len=torch.zeros(B)), dict(workspace=torch.empty(64))):
        with pytest.raises(TypeError):
            _chunk(**bad)
    assert all(c.endswith("workspace_size") for c in lib.calls[n:])


def test_captured_calls_have_scratch_of_their_own(lib, monkeypatch):  # noqa: F811
    monkeypatch.setattr(binding, "_workspace", {})
    dev = torch.device("cpu")
    assert binding._scratch_for(dev, "chunk", 0, None) is None
    assert binding._scratch_for(dev, "chunk", 64, None) is binding._scratch_for(dev, "chunk", 64, None)


def test_host_tensors_are_refused():
    for call in (_rope, _commit, _sample, _chunk):
        with pytest.raises(ValueError, match="CUDA device"):
            call()


_A, _U = 0x10000, 0x10004   # an aligned and a misaligned stand-in address


@pytest.mark.skipif(torch.cuda.is_available(), reason="fake addresses must not reach a GPU")
def test_c_entry_points_refuse():
    NULL, SHAPE, DTYPE, ALIGN = -1, -2, -3, -6
    L = tsd.load_library()

    def rope(q=_A, qs=(256, 256), rot=64, B=2, T=4, Hq=4, Hkv=2, D=64, dt=1, k=_A, table=_A, ps=16,
             inv=_A, out=_A):
        return L.tsd_rope_append_paged(q, *qs, k, 128, 128, _A, 128, 128, inv, rot, 0, 1.0, _A, _A,
                                       None, B, T, Hq, Hkv, D, dt, out, _A, _A, table, 4, ps, 2, None,
                                       None)
    assert rope(B=0) == 0
    for bad in (dict(q=None), dict(k=None), dict(table=None), dict(inv=None), dict(out=None)):
        assert rope(**bad) == NULL
    for bad in (dict(rot=0), dict(rot=3), dict(rot=66), dict(D=60), dict(B=-1), dict(T=0), dict(ps=24),
                dict(qs=(256, 255)), dict(qs=(-256, 256)), dict(Hkv=0), dict(B=70000)):
        assert rope(**bad) == SHAPE
    assert rope(dt=2) == DTYPE
    assert rope(q=_U) == ALIGN and rope(qs=(260, 260)) == ALIGN and rope(out=_U) == ALIGN

    def commit(k=_A, D=128, dt=1, B=2, path=_A, table=_A, ps=16, blocks=2, T=8):
        return L.tsd_kv_commit_paged(k, _A, table, 4, ps, blocks, _A, path, _A, B, T, 2, D, dt, _A,
                                     None, None)
    assert commit(B=0) == 0
    for bad in (dict(k=None), dict(path=None), dict(table=None)):
        assert commit(**bad) == NULL
    for bad in (dict(D=4), dict(D=512), dict(ps=8), dict(blocks=0), dict(T=129), dict(B=70000),
                dict(D=1 << 30)):
        assert commit(**bad) == SHAPE
    assert commit(dt=7) == DTYPE
    assert commit(k=_U) == ALIGN


@pytest.mark.skipif(torch.cuda.is_available(), reason="fake addresses must not reach a GPU")
def test_c_sample_refuses():
    L = tsd.load_library()

    def sample(logits=_A, ld=100, dt=0, R=2, V=100, u=_A, S=1, tokens=_A, probs=_A, pld=100):
        return L.tsd_sample(logits, ld, dt, R, V, None, None, None, None, u, S, tokens, probs, pld,
                            None, None)
    assert sample(R=0) == 0 and sample(S=0, probs=None) == 0
    for bad in (dict(logits=None), dict(u=None), dict(tokens=None)):
        assert sample(**bad) == -1
    for bad in (dict(R=-1), dict(V=0), dict(ld=99), dict(pld=99), dict(S=-1), dict(S=1 << 20),
                dict(V=393217, ld=393217, pld=393217)):
        assert sample(**bad) == -2
    assert sample(dt=2) == -3


@pytest.mark.skipif(torch.cuda.is_available(), reason="fake addresses must not reach a GPU")
def test_c_chunk_refuses():
    L = tsd.load_library()

    def chunk(q=_A, B=2, T=4, Hq=4, Hkv=2, D=64, dt=1, ps=16, blocks=2, pages=4, scale=0.1, ws=_A,
              nbytes=1 << 30, table=_A):
        return L.tsd_chunk_attention_paged(q, _A, _A, table, pages, ps, blocks, _A, _A, B, T, Hq, Hkv, D,
                                           scale, dt, _A, ws, nbytes, None, None)
    assert chunk(B=0) == 0
    assert chunk(q=None) == -1 and chunk(table=None) == -1
    for bad in (dict(Hq=3), dict(T=0), dict(B=70000), dict(ps=20), dict(blocks=0), dict(scale=0.0),
                dict(scale=-1.0), dict(scale=float("nan")), dict(pages=1 << 30, Hkv=4),
                dict(T=1 << 30, Hq=8)):
        assert chunk(**bad) == -2
    assert chunk(D=96) == -3 and chunk(dt=5) == -3
    assert chunk(q=_U) == -6 and chunk(ws=_U) == -6
    assert chunk(nbytes=16) == -4 and chunk(ws=None) == -4
    size = L.tsd_chunk_attention_workspace_size
    assert size(2, 4, 4, 2, 64, 16, 2, 1) > 0
    assert size(0, 4, 4, 2, 64, 16, 2, 1) == 0 and size(2, 4, 3, 2, 64, 16, 2, 1) == 0
    assert size(4, 4096, 64, 8, 128, 64, 100, 1) == 0      # enough blocks without splitting keys


def test_rope_frequencies():
    f = tsd.rope_frequencies(64)
    assert f.rot_scale == 1.0 and f.inv_freq.dtype == torch.float64
    want = [10000.0 ** (-2 * i / 64) for i in range(32)]
    assert torch.allclose(f.inv_freq, torch.tensor(want, dtype=torch.float64), rtol=1e-14, atol=0)
    assert torch.allclose(tsd.rope_frequencies(64, scaling="linear", factor=4.0).inv_freq * 4,
                          f.inv_freq, rtol=1e-15, atol=0)
    n = tsd.rope_frequencies(64, scaling="ntk", factor=8.0).inv_freq
    assert n[0] == 1.0 and math.isclose(float(n[-1] * 8), float(f.inv_freq[-1]), rel_tol=1e-13)
    p = tsd.rope_frequencies(64, scaling="by_parts", factor=8.0, original_len=4096, low=1, high=32,
                             rot_scale=1.2)
    turns = 4096 * f.inv_freq / (2 * math.pi)
    ratio = p.inv_freq / f.inv_freq
    assert p.rot_scale == 1.2
    assert torch.equal(ratio[turns >= 32], torch.ones(int((turns >= 32).sum()), dtype=torch.float64))
    assert torch.allclose(ratio[turns <= 1], torch.full((int((turns <= 1).sum()),), 1 / 8,
                                                         dtype=torch.float64), rtol=1e-15, atol=0)
    mid = (turns > 1) & (turns < 32)
    assert mid.any() and ((ratio[mid] > 1 / 8) & (ratio[mid] < 1)).all()
    assert (ratio.diff() <= 0).all()
    for bad in (dict(rot_dim=3), dict(rot_dim=64, base=1.0), dict(rot_dim=64, factor=0.5),
                dict(rot_dim=64, scaling="by_parts", factor=2.0), dict(rot_dim=2, scaling="ntk"),
                dict(rot_dim=64, scaling="other")):
        with pytest.raises(ValueError):
            tsd.rope_frequencies(**bad)


@pytest.mark.parametrize("D,rows", [(128, 1), (128, 64)])
def test_fp32_chunk_ranges_are_as_many_as_ctas_fit(D, rows):
    # at head_dim 128 the fp32 tiles leave room for one CTA per SM: partial
    # results for two blocks of each of them, and a page of indices and sums
    L = tsd.load_library()
    sms = torch.cuda.get_device_properties(0).multi_processor_count if torch.cuda.is_available() else 148
    size = L.tsd_chunk_attention_workspace_size(1, rows, 1, 1, D, 16, 64, 0)
    parts = 2 * sms * rows
    assert parts * 4 * D <= size <= parts * (4 * D + 8) + 2 * 256 + 16


def test_remembered_workspace_sizes_are_limited(lib):  # noqa: F811
    q = torch.zeros(B, 1, Hq, D, **bf)
    for blocks in range(1, 1200):   # a table that grows with the longest sequence
        _chunk(q=q, block_table=torch.zeros(B, blocks, **i32))
    info = binding._chunk_scratch.cache_info()
    assert 0 < info.currsize <= info.maxsize <= 1024
    n = len(lib.calls)
    _chunk(q=q, block_table=torch.zeros(B, 1199, **i32))
    assert not any(c.endswith("workspace_size") for c in lib.calls[n:])


@pytest.mark.skipif(torch.cuda.is_available(), reason="fake addresses must not reach a GPU")
def test_c_rope_refuses_more_slots_than_positions():
    # a grid of (Tmax + 3) / 4 CTAs: the sum would pass 31 bits
    call = tsd.load_library().tsd_rope_append_paged
    for Tmax in (2 ** 31 - 1, 2 ** 31 - 4, 2 ** 30 + 1):
        assert call(_A, 256, 256, _A, 128, 128, _A, 128, 128, _A, 64, 0, 1.0, _A, _A, None, 2, Tmax, 4,
                    2, 64, 1, _A, _A, _A, _A, 4, 16, 2, None, None) == -2
    # as many as there can be positions get as far as the next check
    assert call(None, 256, 256, _A, 128, 128, _A, 128, 128, _A, 64, 0, 1.0, _A, _A, None, 2, 2 ** 30, 4,
                2, 64, 1, _A, _A, _A, _A, 4, 16, 2, None, None) == -1


@pytest.mark.parametrize("kind", ["attn", "verify", "chunk"])
def test_captured_calls_of_every_kind_own_their_workspace(lib, monkeypatch, kind):  # noqa: F811
    # a graph outlives the cache's buffer, which a larger call replaces
    real = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, device=None, **kw: real(*a, **kw))
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    monkeypatch.setattr(binding, "_workspace", {})
    dev = torch.device("cuda", 0)
    get = binding._scratch_for if kind == "chunk" else binding._workspace_for
    a, b = (get(dev, kind, 512, None) for _ in range(2))
    assert a.numel() >= 512 and b.numel() >= 512 and a.data_ptr() != b.data_ptr()
    assert binding._workspace == {}


def test_sample_between_rows_of_one_tensor(lib):  # noqa: F811
    x = torch.zeros(3, 4, 50)
    for i, j in ((0, 1), (1, 0), (3, 2), (0, 3)):   # disjoint rows of one buffer
        assert _sample(logits=x[:, i], probs=x[:, j]).probs.data_ptr() == x[:, j].data_ptr()
    n = len(lib.calls)
    flat = torch.zeros(3, 200)
    for logits, probs in ((x[:, 0], x[:, 0]), (flat[:, :50], flat[:, 49:99]),
                          (flat[:, 101:151], flat[:, 150:])):
        with pytest.raises(ValueError, match="overlap"):
            _sample(logits=logits, probs=probs)
    with pytest.raises(ValueError, match="overlap"):   # other steps: ranges decide
        _sample(logits=flat.view(6, 100)[:3, :50], probs=flat[:, 50:100])
    assert len(lib.calls) == n
    _sample(R=2, V=0, probs=torch.zeros(2, 0))   # the library's to refuse
