"""Verification steps captured without a workspace of the caller's: each graph
holds its own, so that two of them may be replayed side by side and neither
depends on what later calls do to the cached ones."""

import pytest
import torch

import tree_speculative_decoding_ancestor_b200 as tsd
from gpu_util import run_tree, to_dev
from tree_speculative_decoding_ancestor_b200 import binding
from workloads import gen

pytestmark = pytest.mark.gpu


def _part(w, d, tree):
    att = tsd.tree_attention(d["q"], d["k_cache"], d["v_cache"], d["prefix_len"], d["n_nodes"],
                             tree.mask)
    greedy = tsd.tree_verify_greedy(d["logits"], d["tokens"], d["parent"], d["n_nodes"], tree)
    return att, greedy.n_accepted, greedy.out_path


def _walk(w, d, tree):
    res = tsd.tree_verify_stochastic(d["logits"], w.temperature, d["q_probs"], d["q_row"],
                                     d["tokens"], d["n_nodes"], tree, d["u_accept"], d["u_sample"])
    return res.n_accepted, res.out_tokens


def _live(w, part, walk):
    """What the calls define of their outputs."""
    (att, gn, gp), (wn, wt) = ([x.cpu() for x in o] for o in (part, walk))
    live = [gn, wn]
    for b in range(w.B):
        live += [att[b, :int(w.n_nodes[b])], gp[b, :max(int(gn[b]), 0)], wt[b, :int(wn[b]) + 1]]
    return live


def _capture(f, case):
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = f(*case)
    return g, out


def test_graphs_side_by_side_and_a_larger_call_between(cuda_device):
    dev = cuda_device
    cases = []
    for seed in (3, 4):
        w = gen.random_workload(seed, B=2, Tmax=24, Hq=16, Hkv=2, D=128, P_max=3000, max_children=4,
                                max_depth=10, V=700, dtype="bf16")
        d = to_dev(w, dev)
        cases.append((w, d, run_tree(d)))
    want = [_live(c[0], _part(*c), _walk(*c)) for c in cases]
    torch.cuda.synchronize()
    kept = {k: v.data_ptr() for k, v in binding._workspace.items()}
    parts = [_capture(_part, c) for c in cases]
    walks = [_capture(_walk, c) for c in cases]
    assert {k: v.data_ptr() for k, v in binding._workspace.items()} == kept
    big = gen.random_workload(5, B=8, Tmax=60, Hq=16, Hkv=2, D=128, P_max=4000, max_children=4,
                              max_depth=10, V=5000, dtype="bf16")
    d = to_dev(big, dev)
    tree = run_tree(d)
    _part(big, d, tree)
    _walk(big, d, tree)
    junk = [torch.full((1 << 20,), 7.0, device=dev) for _ in range(8)]
    streams = [torch.cuda.Stream() for _ in parts]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, (g, _) in zip(streams, parts):   # one beside the other
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for _ in range(3):
        for g, _ in walks:                      # one after the other
            g.replay()
    torch.cuda.synchronize()
    for c, (_, part), (_, walk), x in zip(cases, parts, walks, want):
        got = _live(c[0], part, walk)
        assert len(got) == len(x) and all(torch.equal(a, b) for a, b in zip(got, x))
    assert all((x == 7.0).all() for x in junk)
