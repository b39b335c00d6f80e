"""The paged operators run together, as a serving loop uses them.

A small attention layer (random projections of random embeddings) decodes with
speculation over a paged cache: the prompt goes in by rope_append_paged and
chunk_attention_paged; draft tokens are drawn by sample() with their
distributions kept as q rows; their tree is appended with its depths and
verified by tree_attention_paged and tree_verify_stochastic; the accepted path
is committed in pages.  The cache must then be what appending the accepted
tokens one after the other gives, and the attention of the next token the same.
"""

import pytest
import torch

import tree_speculative_decoding_ancestor_b200 as tsd

pytestmark = pytest.mark.gpu

B, HQ, HKV, D, V, PAGE, BLOCKS = 5, 8, 2, 128, 500, 16, 24


class Layer:
    def __init__(self, dev, dtype):
        g = torch.Generator(device=dev).manual_seed(0)
        self.dev, self.dtype = dev, dtype
        self.embed = torch.randn(V, (HQ + 2 * HKV) * D, generator=g, device=dev).to(dtype)
        self.head = (torch.randn(HQ * D, V, generator=g, device=dev) / 16).to(dtype)
        f = tsd.rope_frequencies(D, scaling="by_parts", factor=4.0, original_len=256, device=dev)
        self.inv, self.scale = f.inv_freq, f.rot_scale
        order = torch.randperm(B * BLOCKS, generator=g, device=dev)
        self.table = order.view(B, BLOCKS).int().contiguous()

    def cache(self):
        return [torch.full((B * BLOCKS, HKV, PAGE, D), float("nan"), dtype=self.dtype, device=self.dev)
                for _ in range(2)]

    def append(self, tokens, cache, P, n, depth=None):
        qkv = self.embed[tokens.long()].view(*tokens.shape, HQ + 2 * HKV, D)
        return tsd.rope_append_paged(qkv[:, :, :HQ], qkv[:, :, HQ:HQ + HKV], qkv[:, :, HQ + HKV:],
                                     self.inv, *cache, self.table, P, n, depth=depth,
                                     rot_scale=self.scale)

    def logits(self, x):
        return (x.flatten(-2).float() @ self.head.float()).contiguous()


def _rows(layer, pages, lengths):
    """The cached rows of each sequence, in order."""
    out = []
    for b, n in enumerate(lengths):
        pos = torch.arange(n, device=layer.dev)
        out.append(pages[layer.table[b].long()[pos // PAGE], :, pos % PAGE])
    return out


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_decode_loop(cuda_device, dtype):
    dev = cuda_device
    layer = Layer(dev, dtype)
    g = torch.Generator(device=dev).manual_seed(1)
    rand = lambda *s: torch.rand(*s, generator=g, device=dev, dtype=torch.float64)  # noqa: E731
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
    st = tsd.device_status(dev)
    st.zero_()
    prompt_len = [70, 1, 16, 33, 64]
    T = max(prompt_len)
    prompt = torch.randint(0, V, (B, T), generator=g, device=dev, dtype=torch.int32)

    # the prompt in two chunks equals the prompt in one
    whole, parts = layer.cache(), layer.cache()
    n = i32(prompt_len)
    q = layer.append(prompt, whole, i32([0] * B), n)
    out = tsd.chunk_attention_paged(q, *whole, layer.table, i32([0] * B), n)
    first = torch.minimum(n, i32([20] * B))
    q1 = layer.append(prompt, parts, i32([0] * B), first)
    out1 = tsd.chunk_attention_paged(q1, *parts, layer.table, i32([0] * B), first)
    rest = torch.stack([torch.roll(prompt[b], -int(first[b])) for b in range(B)]).contiguous()
    q2 = layer.append(rest, parts, first, n - first)
    out2 = tsd.chunk_attention_paged(q2, *parts, layer.table, first, n - first)
    tol = 4e-2 if dtype == torch.bfloat16 else 1e-4
    for b in range(B):
        f, m = int(first[b]), int(n[b])
        assert (out1[b, :f].float() - out[b, :f].float()).abs().max() <= tol
        if m > f:
            assert (out2[b, :m - f].float() - out[b, f:m].float()).abs().max() <= tol
    for a, c in zip(whole, parts):
        for x, y in zip(_rows(layer, a, prompt_len), _rows(layer, c, prompt_len)):
            assert torch.equal(x, y)

    # speculation steps: W draft tokens at the root, one child under each
    P, W, cache = n, 4, whole
    history = [prompt[b, :prompt_len[b]].tolist() for b in range(B)]
    last = out[torch.arange(B, device=dev), P.long() - 1]
    for _ in range(3):
        q_probs = torch.zeros(B, W + 1, V, device=dev)
        root_logits = layer.logits(last)
        top_p, temp = torch.full((B,), 0.95, device=dev), torch.full((B,), 0.8, device=dev)
        level1 = tsd.sample(root_logits, rand(B, W), temperature=temp, top_p=top_p, probs=q_probs[:, 0])
        tokens = torch.zeros(B, 2 * W, dtype=torch.int32, device=dev)
        parent = torch.full((B, 2 * W), -1, dtype=torch.int32, device=dev)
        q_row = torch.zeros(B, 2 * W, dtype=torch.int32, device=dev)
        for w in range(W):   # node 2w: a draw at the root, node 2w + 1: its child
            tokens[:, 2 * w] = level1.tokens[:, w]
            draft = layer.logits(layer.embed[level1.tokens[:, w].long()][:, :HQ * D].view(B, HQ, D))
            child = tsd.sample(draft, rand(B, 1), temperature=temp, top_p=top_p, probs=q_probs[:, w + 1])
            tokens[:, 2 * w + 1] = child.tokens[:, 0]
            parent[:, 2 * w + 1] = 2 * w
            q_row[:, 2 * w + 1] = w + 1
        n_nodes = i32([2 * W] * B)
        tree = tsd.tree_mask_build(parent, n_nodes)
        q = layer.append(tokens, cache, P, n_nodes, depth=tree.depth)
        att = tsd.tree_attention_paged(q, *cache, layer.table, P, n_nodes, tree.mask)
        logits = torch.cat([root_logits[:, None], layer.logits(att)], dim=1).contiguous()
        res = tsd.tree_verify_stochastic(logits, 0.8, q_probs, q_row, tokens, n_nodes, tree,
                                         rand(B, 2 * W), rand(B, 2 * W + 1))
        P = tsd.kv_commit_paged(*cache, layer.table, P, res)
        for b in range(B):
            k = int(res.n_accepted[b])
            history[b] += res.out_tokens[b, :k].tolist()
        lengths = [len(h) for h in history]
        assert P.tolist() == lengths

        # the same tokens appended as plain text give the same rows ...
        check = layer.cache()
        L = max(lengths)
        text = torch.zeros(B, L, dtype=torch.int32, device=dev)
        for b, h in enumerate(history):
            text[b, :len(h)] = i32(h)
        qt = layer.append(text, check, i32([0] * B), P)
        for a, c in zip(cache, check):
            for x, y in zip(_rows(layer, a, lengths), _rows(layer, c, lengths)):
                assert torch.equal(x, y)
        # ... and the last token's attention agrees between a decode step over the
        # committed cache and the whole text as one chunk
        full = tsd.chunk_attention_paged(qt, *check, layer.table, i32([0] * B), P)
        at = torch.arange(B, device=dev), P.long() - 1
        step = tsd.chunk_attention_paged(qt[at][:, None].contiguous(), *cache, layer.table, P - 1,
                                         i32([1] * B))
        assert (step[:, 0].float() - full[at].float()).abs().max() <= tol
        # the bonus token opens the next step
        bonus = torch.stack([res.out_tokens[b, int(res.n_accepted[b])] for b in range(B)])[:, None]
        q = layer.append(bonus.contiguous(), cache, P, i32([1] * B))
        last = tsd.chunk_attention_paged(q, *cache, layer.table, P, i32([1] * B))[:, 0]
        for b in range(B):
            history[b].append(int(bonus[b]))
        P = P + 1
    assert int(st.item()) == 0


def test_a_captured_decode_step(cuda_device):
    # append, attention and sampling of one token as a graph, replayed over a
    # growing cache: the lengths and tokens live on the device
    dev = cuda_device
    layer = Layer(dev, torch.bfloat16)
    steps = 12
    u = torch.rand(steps, B, 1, dtype=torch.float64, device=dev, generator=torch.Generator(
        device=dev).manual_seed(4))
    one = torch.ones(B, dtype=torch.int32, device=dev)
    k = torch.full((B,), 20, dtype=torch.int32, device=dev)

    def run(step, token, P, cache, un):
        q = layer.append(token, cache, P, one)
        x = tsd.chunk_attention_paged(q, *cache, layer.table, P, one)
        token.copy_(tsd.sample(layer.logits(x[:, 0]), un, top_k=k).tokens)
        P.add_(1)

    results = []
    for captured in (False, True):
        cache = layer.cache()
        token = torch.arange(B, dtype=torch.int32, device=dev)[:, None].contiguous()
        P = torch.zeros(B, dtype=torch.int32, device=dev)
        un = torch.zeros(B, 1, dtype=torch.float64, device=dev)
        said = []
        if captured:
            run(0, token.clone(), P.clone(), layer.cache(), u[0].contiguous())   # warm up
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                run(0, token, P, cache, un)
        for s in range(steps):
            un.copy_(u[s])
            if captured:
                graph.replay()
            else:
                run(s, token, P, cache, un)
            said.append(token.clone())
        results.append(torch.cat(said, dim=1))
    assert torch.equal(*results)
    assert int(tsd.device_status(dev).item()) == 0
