"""Verification of drafted trees through a model (mk_verify, Megakernel.accept):
every node against the oracle's decode steps along its path, the accepted rows
against the rows the oracle leaves, and decoding that goes on behind them."""
import numpy as np
import pytest
import torch

import tree_reference as ref
from decode_megakernel_llama_gb300 import _lib, synth
from decode_megakernel_llama_gb300.configs import LLAMA_1B, LLAMA_3B, TINY, ModelShape
from gpu_helpers import MARGIN, MAX_ABS, Pair, compare, teacher_forced

pytestmark = pytest.mark.gpu
I32 = torch.int32


def draft(vocab, n, gen):
    parents = ref.random_parents(n, gen)
    tokens = torch.randint(0, vocab, (n,), generator=gen).tolist()
    return tokens, parents


def path_of(parents, t):
    p = []
    while t >= 0:
        p.append(t)
        t = parents[t]
    return p[::-1]


def verify(pair, tokens, parents, start):
    n, dev = len(tokens), "cuda:0"
    out = torch.full((n + 1,), -7, dtype=I32, device=dev)
    logits = torch.full((n, pair.shape.vocab), float("nan"), device=dev)
    pair.mk.verify(torch.tensor(tokens, dtype=I32, device=dev), torch.tensor(parents, dtype=I32, device=dev), start, out,
                   logits)
    torch.cuda.synchronize()
    assert pair.mk.status() == 0, _lib.load().mk_last_error()
    assert int(out[n]) == -7
    return logits.double().cpu().numpy(), out[:n].tolist()


def check_nodes(pair, tokens, parents, start, logits, draws, nodes=None):
    """Every node (or those in `nodes`) against the oracle's steps along its path."""
    want = {}
    for t in range(len(tokens)) if nodes is None else nodes:
        for depth, u in enumerate(path_of(parents, t)):
            want[u] = pair.orc.decode_step(tokens[u], start + depth)
        compare(logits[t], draws[t], *want[t], f"node {t}")
    return want


@pytest.mark.parametrize("n,start", [(1, 0), (7, 0), (13, 5), (33, 9), (64, 3)])
def test_tiny_tree_matches_the_oracle_node_by_node(cuda_dev, n, start):
    pair = Pair(TINY, start + n + 2)
    g = torch.Generator().manual_seed(n)
    prompt = synth.prompt_tokens(TINY.vocab, max(1, start))[:start]
    if start:
        teacher_forced(pair, prompt, 0)
    before = pair.k.clone(), pair.v.clone()
    tokens, parents = draft(TINY.vocab, n, g)
    logits, draws = verify(pair, tokens, parents, start)
    check_nodes(pair, tokens, parents, start, logits, draws)
    # only the tree's rows were written
    for now, old in zip((pair.k, pair.v), before):
        assert torch.equal(now[:, :, :, :start], old[:, :, :, :start])
        assert torch.equal(now[:, :, :, start + n:], old[:, :, :, start + n:])
    pair.close()


def test_accepted_path_and_decoding_goes_on(cuda_dev):
    """A drafter that is right along one branch: the path is accepted, its rows move up, the next steps agree."""
    start, n = 6, 17
    pair = Pair(TINY, 64)
    stats = teacher_forced(pair, synth.prompt_tokens(TINY.vocab, start), 0)
    assert stats
    ol, tok = pair.orc.decode_step(int(synth.prompt_tokens(TINY.vocab, start)[-1]), start - 1)
    # the oracle's own continuation, five tokens
    true = [tok]
    for i in range(5):
        true.append(pair.orc.decode_step(true[-1], start + i)[1])
    # node 0 is the chosen token; its continuation sits on nodes 3, 5, 9, 12, wrong siblings between them
    parents = [-1, 0, 0, 0, 1, 3, 3, 5, 5, 5, 9, 9, 9, 2, 12, 12, 4]
    tokens = [true[0]] + [(true[0] + 1 + i) % TINY.vocab for i in range(n - 1)]
    right = {3: true[1], 5: true[2], 9: true[3], 12: true[4]}
    for t, x in right.items():
        tokens[t] = x
    for t in range(1, n):  # no wrong node carries the right token of its place
        if t not in right:
            depth = len(path_of(parents, t)) - 1
            while tokens[t] == true[min(depth, 5)] or tokens[t] in right.values():
                tokens[t] = (tokens[t] + 17) % TINY.vocab
    logits, draws = verify(pair, tokens, parents, start)
    check_nodes(pair, tokens, parents, start, logits, draws, nodes=[0, 3, 5, 9, 12])
    rows = [pair.k[:, 0, :, start + t].clone() for t in (0, 3, 5, 9, 12)]
    path = pair.mk.accept(tokens, parents, draws, start)
    # (a wrong node's draw may lead on only below the right ones)
    assert path[:5] == [0, 3, 5, 9, 12], (path, draws)
    torch.cuda.synchronize()
    for i, r in enumerate(rows):
        assert torch.equal(pair.k[:, 0, :, start + i], r)
    for gpu, orc in ((pair.k, pair.orc.k_cache), (pair.v, pair.orc.v_cache)):
        got = gpu[:, 0, :, : start + 5].float().cpu().numpy()
        want = (orc[:, :, : start + 5].astype(np.uint32) << 16).view(np.float32)
        assert np.abs(got - want).max() <= 2e-2 * max(1.0, np.abs(want).max())
    if len(path) == 5:
        teacher_forced(pair, [draws[12]], 8, start_pos=start + 5)
    pair.close()


def test_a_chain_is_the_prefill(cuda_dev):
    """A tree without branches gives the logits and rows of mk_prefill to rounding."""
    n, start = 40, 24
    pair = Pair(TINY, 80)
    prompt = synth.prompt_tokens(TINY.vocab, start + n).to("cuda:0")
    out, last = torch.zeros(1, dtype=I32, device="cuda:0"), torch.empty(TINY.vocab, device="cuda:0")
    pair.mk.prefill(prompt[:start], 0, out)
    pair.mk.prefill(prompt[start:], start, out, last)
    torch.cuda.synchronize()
    rows = pair.k[:, 0, :, start:start + n].float(), pair.v[:, 0, :, start:start + n].float()
    logits, draws = verify(pair, prompt[start:].tolist(), list(range(-1, n - 1)), start)
    assert np.abs(logits[-1] - last.double().cpu().numpy()).max() <= 1e-2
    for now, old in zip((pair.k, pair.v), rows):
        d = (now[:, 0, :, start:start + n].float() - old).abs()
        assert (d <= 2e-2 * old.abs().max()).all()
    pair.close()


@pytest.mark.parametrize("shape", [
    ModelShape("hd128-g3", 2, 768, 6, 2, 128, 1024, 1000, 1e-5, 5e5),
    ModelShape("hd64-g1", 2, 256, 4, 4, 64, 512, 777, 1e-5, 1e4),
])
def test_other_shapes(cuda_dev, shape):
    pair = Pair(shape, 60)
    teacher_forced(pair, synth.prompt_tokens(shape.vocab, 4), 0)
    tokens, parents = draft(shape.vocab, 21, torch.Generator().manual_seed(8))
    logits, draws = verify(pair, tokens, parents, 4)
    check_nodes(pair, tokens, parents, 4, logits, draws)
    pair.close()


@pytest.mark.slow
def test_llama1b_tree_behind_a_long_cache(cuda_dev):
    """The 1B shape, a tree of 40 behind 4,400 pre-filled positions (the split attention with its workspace)."""
    start = 4400
    pair = Pair(LLAMA_1B, start + 64, prefill=start)
    tokens, parents = draft(LLAMA_1B.vocab, 40, torch.Generator().manual_seed(1))
    logits, draws = verify(pair, tokens, parents, start)
    nodes = [0, 39]
    check_nodes(pair, tokens, parents, start, logits, draws, nodes=nodes)
    pair.close()


def test_llama3b_shape_runs(cuda_dev):
    """The 3B-class shape: the nodes of a small tree against the megakernel's own steps."""
    pair_shape = LLAMA_3B
    dev = torch.device("cuda:0")
    w = synth.make_weights(pair_shape, dev, 0)
    k, v = synth.kv_cache(pair_shape, 64, 1, dev)
    mk = _lib.Megakernel(pair_shape, w, k, v)
    out, lg = torch.zeros(8, dtype=I32, device=dev), torch.empty(8, pair_shape.vocab, device=dev)
    prompt = synth.prompt_tokens(pair_shape.vocab, 12)
    for i in range(4):
        mk.step(int(prompt[i]), i, out[:1])
    tokens, parents = prompt[4:12].tolist(), [-1, 0, 1, 0, 3, 4, 2, 6]
    mk.verify(torch.tensor(tokens, dtype=I32, device=dev), torch.tensor(parents, dtype=I32, device=dev), 4, out, lg)
    assert mk.status() == 0
    one, tok = torch.empty(pair_shape.vocab, device=dev), torch.zeros(1, dtype=I32, device=dev)
    for t in range(8):
        for depth, u in enumerate(path_of(parents, t)):
            mk.step(tokens[u], 4 + depth, tok, one)
        d = (lg[t] - one).abs().max().item()
        assert d <= 5e-2, (t, d)
        top = one.topk(2).values
        if float(top[0] - top[1]) > MARGIN:
            assert int(out[t]) == int(tok)
    mk.close()


@pytest.mark.parametrize("filt", [None, (20, 0.8)])
def test_draws_are_those_of_decode_steps(cuda_dev, filt):
    """With sampling on, a node's token is the one a decode step at its position draws from its logits."""
    start = 3
    pair = Pair(TINY, 40)
    teacher_forced(pair, synth.prompt_tokens(TINY.vocab, start), 0)
    tokens, parents = draft(TINY.vocab, 20, torch.Generator().manual_seed(4))
    temperature, seed = 0.9, 1234567890123
    pair.mk.set_sampling(temperature, seed)
    if filt:
        pair.mk.set_sampling_filter(*filt)
    out = torch.zeros(20, dtype=I32, device="cuda:0")
    lg = torch.empty(20, TINY.vocab, device="cuda:0")
    pair.mk.verify(torch.tensor(tokens, dtype=I32, device="cuda:0"),
                   torch.tensor(parents, dtype=I32, device="cuda:0"), start, out, lg)
    assert pair.mk.status() == 0
    k, p = filt or (0, 1.0)
    for t in range(20):
        pos = torch.tensor([start + len(path_of(parents, t)) - 1], dtype=I32, device="cuda:0")
        one = torch.zeros(1, dtype=I32, device="cuda:0")
        _lib.draw_from_logits(lg[t:t + 1].contiguous(), temperature, k, p, pos, seed, one)
        assert int(one) == int(out[t]), t
    pair.close()


def test_verify_refuses_and_reports(cuda_dev):
    pair = Pair(TINY, 16)
    dev = "cuda:0"
    tk, pr, out = (torch.zeros(70, dtype=I32, device=dev) for _ in range(3))
    for n, start in ((65, 0), (0, 0), (4, 13), (4, -1)):
        with pytest.raises(_lib.MKError) as e:
            pair.mk.verify(tk[:n], pr[:n], start, out)
        assert e.value.code == _lib.MK_ERR_INVALID_ARG
    with pytest.raises(_lib.MKError):
        pair.mk.verify(tk[:4], pr[:3], 0, out)
    lg = torch.empty(3, TINY.vocab, device=dev)
    for bad in (dict(out_tokens=out[:3]), dict(d_tokens=tk[:4].long()), dict(d_parents=pr[:8:2]),
                dict(out_tokens=out.cpu()), dict(logits=lg), dict(logits=torch.empty(4, TINY.vocab).half().to(dev))):
        with pytest.raises(_lib.MKError):
            pair.mk.verify(**{**dict(d_tokens=tk[:4], d_parents=pr[:4], start_pos=0, out_tokens=out), **bad})
    for start in (-1, 15):  # two nodes do not fit behind 15 rows of 16
        with pytest.raises(_lib.MKError):
            pair.mk.accept([1, 2], [-1, 0], [2, 3], start)
    bad = torch.tensor([1, TINY.vocab, 2], dtype=I32, device=dev)
    pair.mk.verify(bad, torch.tensor([-1, 0, 1], dtype=I32, device=dev), 0, out)
    assert pair.mk.status() == _lib.MK_ERR_INVALID_ARG
    assert pair.mk.status() == 0  # reported once, and the handle works again
    logits, draws = verify(pair, [5, 6, 7], [-1, 0, 0], 0)
    check_nodes(pair, [5, 6, 7], [-1, 0, 0], 0, logits, draws)
    pair.close()


def test_verify_in_a_graph(cuda_dev):
    """Captured after its first call; replayed on other tokens and another tree of the same size."""
    pair = Pair(TINY, 40)
    dev = "cuda:0"
    teacher_forced(pair, synth.prompt_tokens(TINY.vocab, 3), 0)
    g = torch.Generator().manual_seed(6)
    tk, pr, out = (torch.zeros(15, dtype=I32, device=dev) for _ in range(3))
    lg = torch.empty(15, TINY.vocab, device=dev)
    a = draft(TINY.vocab, 15, g)
    tk.copy_(torch.tensor(a[0])), pr.copy_(torch.tensor(a[1]))
    pair.mk.verify(tk, pr, 3, out, lg)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pair.mk.verify(tk, pr, 3, out, lg)
    b = draft(TINY.vocab, 15, g)
    tk.copy_(torch.tensor(b[0])), pr.copy_(torch.tensor(b[1]))
    # a larger tree and a prefill in between move nothing that the graph uses
    big = draft(TINY.vocab, 30, g)
    verify(pair, *big, 3)
    pair.mk.prefill(synth.prompt_tokens(TINY.vocab, 3).to(dev), 0, torch.zeros(1, dtype=I32, device=dev))
    graph.replay()
    torch.cuda.synchronize()
    assert pair.mk.status() == 0
    check_nodes(pair, *b, 3, lg.double().cpu().numpy(), out.tolist())
    pair.close()


def test_a_slot_forked_over_a_batch(cuda_dev):
    """One sequence's cache forked to the other slots: a batched step of the same token gives each the same logits,
    to the parity bar (the batched step's warps add into shared accumulators in no fixed order)."""
    B, n = 4, 10
    dev = torch.device("cuda:0")
    w = synth.make_weights(TINY, dev, 0)
    k, v = synth.kv_cache(TINY, 32, B, dev)
    mk = _lib.Megakernel(TINY, w, k, v)
    prompt = synth.prompt_tokens(TINY.vocab, n + 1).to(dev)
    out, lg = torch.zeros(B, dtype=I32, device=dev), torch.empty(B, TINY.vocab, device=dev)
    mk.prefill(prompt[:n], 0, out[:1])
    _lib.kv_reorder(k, v, torch.zeros(B, dtype=I32, device=dev), torch.full((B,), n, dtype=I32, device=dev))
    mk.step_batch(prompt[n:].expand(B).contiguous(), torch.full((B,), n, dtype=I32, device=dev), out, lg)
    torch.cuda.synchronize()
    assert mk.status() == 0
    for b in range(1, B):
        assert torch.equal(k[:, b, :, :n], k[:, 0, :, :n]) and torch.equal(v[:, b, :, :n], v[:, 0, :, :n])
        assert (lg[b] - lg[0]).abs().max() <= MAX_ABS
    mk.close()
