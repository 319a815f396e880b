"""The same call gives the same bits, every time: alone, beside another stream's, replayed, with other calls between."""
import pytest
import torch

from decode_megakernel_llama_gb300.build import build
from tests.test_paged_gpu import Paged

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build()


def _same(outs, want):
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)


@pytest.mark.parametrize("lens,news,Hq,Hkv,hd,ps,type,cache,window,sinks", [
    ([4099, 1700, 199, 3000], [1, 1, 1, 1], 32, 8, 64, 16, "bf16", "bf16", 0, 0),
    ([32768, 30011], [1, 1], 24, 8, 128, 64, "bf16", "e4m3", 0, 0),
    ([20001, 17000, 14001], [33, 30, 24], 32, 8, 128, 32, "bf16", "bf16", 4096, 4),
    ([2048], [2048], 32, 8, 64, 16, "bf16", "bf16", 0, 0),
    ([6001, 4000], [301, 101], 24, 8, 64, 128, "f32", "e4m3", 0, 0),
    ([9000], [40], 8, 2, 128, 32, "f32", "e4m3", 0, 0),
    ([25] * 400, [1] * 400, 8, 2, 64, 16, "f32", "bf16", 0, 0),
])
def test_the_same_bits_every_time(lens, news, Hq, Hkv, hd, ps, type, cache, window, sinks):
    """40 calls, other inputs and a flushed cache between them."""
    p = Paged(lens, news, Hq, Hkv, hd, ps, type, cache, window, sinks, seed=1, poison=False)
    other = Paged([700, 80], [9, 1], 8, 2, 64, 16, seed=2)
    kw = dict(max_new=max(news), max_len=max(lens))
    flush = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    outs = []
    for i in range(40):
        if i % 3 == 1:
            other.run()
        if i % 5 == 2:
            flush.fill_(i)
        p.out.fill_(7.0)
        p.run(**kw)
        outs.append(p.out.clone())
    _same(outs, outs[0])
    assert int(p.status) == 0


def _calls():
    """Calls that split their rows, and one of many rows, each with its result when alone."""
    ps = [Paged([30000, 9000], [1, 1], 8, 2, 64, 16, "bf16", "bf16", seed=2), Paged([12000], [5], 4, 1, 128, 64, "f32", "e4m3", seed=3),
          Paged([900, 1100], [70, 60], 8, 2, 64, 16, "bf16", "bf16", seed=4)]
    for p in ps:
        p.run()
        p.check()
    return ps, [p.out.clone() for p in ps]


def test_streams_side_by_side_every_round():
    ps, want = _calls()
    streams = [torch.cuda.Stream() for _ in ps]
    outs = [[] for _ in ps]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(30):
        for p, s, o in zip(ps, streams, outs):
            with torch.cuda.stream(s):
                p.out.fill_(7.0)
                p.run()
                o.append(p.out.clone())
    for o, w in zip(outs, want):
        _same(o, w)


def test_graphs_side_by_side_every_round():
    ps, want = _calls()
    graphs = []
    for p in ps:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            p.run()
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in ps]
    outs = [[] for _ in ps]
    torch.cuda.synchronize()
    for _ in range(20):
        for p, g, s, o in zip(ps, graphs, streams, outs):
            with torch.cuda.stream(s):
                p.out.fill_(7.0)
                g.replay()
                o.append(p.out.clone())
    for o, w in zip(outs, want):
        _same(o, w)
