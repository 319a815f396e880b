"""paged_attention over many sequences: the grid's places among them, empty ones, and the time they take to find."""
import random

import pytest
import torch

from decode_megakernel_llama_gb300 import _lib
from decode_megakernel_llama_gb300.build import build
from tests.test_paged_gpu import Paged

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build()


@pytest.mark.parametrize("hints", [dict(), dict(max_new=1, max_len=16), dict(max_new=200, max_len=400)])
@pytest.mark.parametrize("B,news", [(31, "ones"), (32, "some"), (33, "ones"), (97, "ragged"), (1024, "ones"), (1025, "some"),
                                    (2100, "ragged"), (300, "few"), (200, "none but the last")])
def test_many_sequences(B, news, hints):
    """One token each, none here and there, all lengths, hardly any, and one at the end."""
    rng = random.Random(B)
    n = {"ones": lambda b: 1, "some": lambda b: rng.choice([0, 1, 1, 2]), "few": lambda b: int(b in (0, 7, 8, 255)),
         "ragged": lambda b: rng.choice([0, 0, 1, 3, 5, 17]) if b % 97 else 150,
         "none but the last": lambda b: 70 * (b == B - 1)}[news]
    new = [n(b) for b in range(B)]
    lens = [x + rng.randint(0, 12) for x in new]
    p = Paged(lens, new, 4, 1, 64, 16, rng.choice(["f32", "bf16"]), rng.choice(["bf16", "e4m3"]), pad=5, seed=B)
    p.run(**hints)
    p.check()


def test_tokens_before_the_first_sequence_and_between_graphs_of_one_capacity():
    """starts need not begin at 0: the tokens before are left as they are, also where fewer sequences are in use."""
    p = Paged([40, 30, 20], [2, 9, 1], 8, 2, 64, 16, seed=3)
    before = 6
    q = torch.cat([torch.randn(before, 8, 64, device="cuda").to(p.q.dtype), p.q])
    out = torch.full_like(q, 7.0)
    for used in (3, 2, 0):
        out.fill_(7.0)
        starts = p.starts + before
        starts[used:] = int(starts[used])
        _lib.paged_attention(q, p.k, p.v, p.table, starts, p.lengths, out, max_new=9)
        count = int(p.starts[used])
        assert bool((out[:before] == 7.0).all()) and bool((out[before + count:] == 7.0).all())
        p.run(max_new=9)
        assert torch.equal(out[before:before + count], p.out[:count])


def test_the_time_does_not_grow_with_the_square_of_the_sequences():
    """16,384 sequences against 4,096: four times the work (a search among all sequences before took 13 times as long)."""
    took = []
    for B in (4096, 16384):
        p = Paged([20], [1], 8, 8, 64, 32, poison=False)
        i32 = dict(dtype=torch.int32, device="cuda")
        q = torch.randn(B, 8, 64, device="cuda").to(p.q.dtype)
        out = torch.empty_like(q)
        table, starts, lengths = p.table.repeat(B, 1), torch.arange(B + 1, **i32), torch.full((B,), 20, **i32)
        times = []
        for _ in range(5):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            _lib.paged_attention(q, p.k, p.v, table, starts, lengths, out, max_new=1, max_len=20)
            b.record()
            b.synchronize()
            times.append(a.elapsed_time(b))
        took.append(min(times))
    print("ms", took)
    assert took[1] < 8 * took[0]


def test_as_many_sequences_as_a_call_may_have():
    """2^20 of one token each, over 64 shared pages. A bf16 result is within 2^-8 of itself and of sum p|v| twice the scores'
    error, 3 * 64 products' roundings of |q||k| / 8 < 8 (5e-4 at 64 / 8 * 3 * 64 * 2^-24 * 2 * 2.8, the largest seen here), and
    2^-16 for the weights."""
    B, pages, ps, hd, Hq = 1 << 20, 64, 16, 64, 2
    g = torch.Generator(device="cuda").manual_seed(4)
    k, v = (torch.randn(pages, 1, ps, hd, generator=g, device="cuda").bfloat16() for _ in range(2))
    q = torch.randn(B, Hq, hd, generator=g, device="cuda").bfloat16()
    i32 = dict(dtype=torch.int32, device="cuda")
    b = torch.arange(B, **i32)
    lengths = 1 + (b // pages) % ps
    out = torch.empty_like(q)
    status = torch.zeros(1, **i32)
    _lib.paged_attention(q, k, v, (b % pages)[:, None].contiguous(), torch.arange(B + 1, **i32), lengths, out, max_new=1,
                         max_len=ps, status=status)
    assert int(status) == 0
    for page in range(pages):
        s = 0.125 * q[page::pages].float() @ k[page, 0].float().T
        seen = torch.arange(ps, device="cuda")[None, None] < lengths[page::pages, None, None]
        w = torch.softmax(torch.where(seen, s, -torch.inf), -1)
        want, most = w @ v[page, 0].float(), w @ v[page, 0].float().abs()
        err = (out[page::pages].float() - want).abs()
        assert bool((err <= 2.0 ** -8 * want.abs() + (5e-4 + 2.0 ** -16) * most).all())
