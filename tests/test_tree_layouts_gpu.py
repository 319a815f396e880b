"""The drafted-tree operators in layouts and streams of their callers: rows in
one buffer, the binding's two ways."""
import pytest
import torch

import tree_reference as ref
from decode_megakernel_llama_gb300 import _lib
from decode_megakernel_llama_gb300.build import build

pytestmark = pytest.mark.gpu
BF, I32 = torch.bfloat16, torch.int32


@pytest.fixture(scope="module")
def dev(cuda_dev):
    build()
    return cuda_dev


@pytest.mark.parametrize("n", [1, 7, 1000])
@pytest.mark.parametrize("dtype", [torch.float32, BF])
@pytest.mark.parametrize("first", [False, True])
def test_queries_between_the_rows_of_qkv(dev, n, dtype, first):
    """q_out behind (or before) each token's row in one buffer is no overlap; the same bits as in a buffer of its own, and
    with a stream given."""
    Hq, Hkv, hd = 4, 2, 64
    width, qw, g = (Hq + 2 * Hkv) * hd, Hq * hd, torch.Generator().manual_seed(n)
    buf = torch.randn(n, width + qw, generator=g).to(dtype).to(dev)
    qkv = buf[:, qw:] if first else buf[:, :width]
    q_out = (buf[:, :qw] if first else buf[:, width:]).view(n, Hq, hd)
    rows, freq = torch.arange(n, dtype=I32, device=dev), _lib.rope_frequencies(hd, 1e4)[0].to(dev)
    k, v = (torch.zeros(1, Hkv, n, hd, dtype=BF, device=dev) for _ in "kv")
    k2, v2, k3, v3 = (torch.zeros_like(k) for _ in range(4))
    own, own2 = (torch.zeros(n, Hq, hd, dtype=dtype, device=dev) for _ in "ab")
    x = qkv.clone()
    _lib.rope_append(x, own, k2, v2, rows, rows, freq)
    torch.cuda.synchronize()
    _lib.rope_append(x, own2, k3, v3, rows, rows, freq, stream=torch.cuda.Stream())
    _lib.rope_append(qkv, q_out, k, v, rows, rows, freq)
    torch.cuda.synchronize()
    assert torch.equal(q_out, own) and torch.equal(k, k2) and torch.equal(v, v2) and torch.equal(qkv, x)
    assert torch.equal(own2, own) and torch.equal(k3, k2) and torch.equal(v3, v2)


def test_cache_moves_with_a_stream_given(dev):
    g = torch.Generator().manual_seed(3)
    k, v = (torch.randn(2, 3, 2, 40, 64, generator=g).to(BF).to(dev) for _ in "kv")
    sources, lengths = torch.tensor([1, 2, 0], dtype=I32, device=dev), torch.tensor([40, 9, 17], dtype=I32, device=dev)
    starts, counts = torch.tensor([0, 5, 30], dtype=I32, device=dev), torch.tensor([2, 0, 3], dtype=I32, device=dev)
    nodes = torch.tensor([[1, 3, 0]] * 2 + [[0, 4, 8]], dtype=I32, device=dev)
    want = [ref.compact(ref.reorder(x, sources, lengths), starts, nodes, counts) for x in (k, v)]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    _lib.kv_reorder(k, v, sources, lengths, stream=s)
    _lib.kv_compact(k, v, starts, nodes, counts, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(k, want[0]) and torch.equal(v, want[1])
