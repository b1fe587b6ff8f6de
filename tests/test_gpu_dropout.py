"""Dropout: its generator against published vectors and a restatement on whole numbers, its results element by element."""
import pytest
import torch

import sublayer_ref as ref
import test_gpu_layers as base
from communication_compressed_optimizer_compress_gb300 import layers as L
from test_gpu_layers_binding import both  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


def _key(seed, step=0):
    return torch.tensor([seed, step], dtype=torch.int64, device="cuda")


def test_the_generator_is_the_published_one():
    """The restatement against the vectors published with Philox4x32-10, and the kernel against the restatement's words: p of
    k/65536 asks every bit of them."""
    top = 2 ** 32 - 1
    for counter, key, words in (((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
                                ((top,) * 4, (top,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
                                ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0), (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1))):
        assert ref.philox(counter, key) == words
    words = (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)
    want = [v for w in words for v in (w & 0xFFFF, w >> 16)]
    x = torch.ones(1, 8, device="cuda")
    for e, bits in enumerate(want):
        assert L.dropout(x, bits / 65536, _key(0))[0, e] != 0 and L.dropout(x, (bits + 1) / 65536, _key(0))[0, e] == 0


SHAPES = [(1, 1), (1, 7), (50, 3), (1, 8), (40, 60), (3, 9), (5, 64), (33, 100), (7, 1001), (300, 1024), (2000, 72), (4099, 1155), (1, 100003)]


@pytest.mark.parametrize("layout", ["dense", "wide", "odd"])
@pytest.mark.parametrize("dtype", [F32, F16, BF16], ids=base.ids)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_values(shape, dtype, layout):
    gen = base._gen(shape[0] + shape[1])
    x = base._lay(base._randn(gen, *shape, dtype=dtype), layout)
    for p, seed, step, site in ((0.1, 1234567890123456789, 77, 5), (0.5, -3, 2 ** 40 + 1, 0), (1 / 65536, 0, 0, 2 ** 32 - 1), (65535 / 65536, 9, 9, 9)):
        key = _key(seed, step)
        # one product in fp32, rounded once more to the type: the same in torch
        want = torch.where(ref.stays(*shape, p, key, site), (x.float() * ref.factor(p)).to(dtype), torch.zeros_like(x))
        assert torch.equal(L.dropout(x, p, key, site), want)
        assert L.dropout(x, p, key, site).is_contiguous()


def test_nothing_dropped():
    x = base._randn(base._gen(1), 50, 70, dtype=BF16)
    for p in (0.0, 2.0 ** -18):  # rounds to 0
        for key in (None, _key(5)):
            if p == 0 or key is not None:
                assert torch.equal(L.dropout(x, p, key), x)
    assert L.dropout(x[:0], 0.5, _key(1)).shape == (0, 70)


def test_what_is_dropped_is_zero_whatever_it_was():
    key = _key(3, 4)
    for dtype in (F32, F16, BF16):
        gone = ~ref.stays(64, 96, 0.3, key, 1)
        for bad in (float("nan"), float("inf"), float("-inf"), torch.finfo(dtype).min):
            x = torch.where(gone, bad, 1.0).to(dtype)
            y = L.dropout(x, 0.3, key, 1)
            assert bool((y[gone] == 0).all()) and bool(y.isfinite().all()) and bool((y[~gone] != 0).all())


def test_offsets_past_31_bits_and_groups_past_32():
    """2.1e9 elements in wide rows; 1.4e9 rows of three groups, whose index needs the counter's second word (98 GB)."""
    key = _key(11, 12)
    for rows, cols, at in ((1 << 18, 8200, (0, 1, (1 << 31) // 8200, (1 << 18) - 300)),
                           ((1 << 32) // 3 + 1000, 17, (0, (1 << 31) // 17, (1 << 32) // 3 - 100, (1 << 32) // 3 + 700))):
        y = L.dropout(torch.ones(rows, cols, dtype=BF16, device="cuda"), 0.5, key, 3)
        for r in at:
            n = min(300, rows - r)
            assert torch.equal(y[r: r + n] != 0, ref.stays(n, cols, 0.5, key, 3, first_row=r))
        del y
        torch.cuda.empty_cache()


def test_keys_steps_and_sites_are_apart_and_the_rate_holds():
    n = 1 << 20
    x = torch.ones(1024, 1024, device="cuda")
    masks = [L.dropout(x, 0.25, _key(*k), site) != 0 for *k, site in ((1, 0, 0), (2, 0, 0), (1, 1, 0), (1, 0, 1), (1 + 2 ** 32, 0, 0))]
    for i, a in enumerate(masks):
        # a binomial count: six standard deviations
        assert abs(int(a.sum()) - 0.75 * n) < 6 * (n * 0.1875) ** 0.5
        for b in masks[:i]:
            same = int((a == b).sum())  # agreement of independent masks: 0.75^2 + 0.25^2 = 0.625
            assert abs(same - 0.625 * n) < 6 * (n * 0.234375) ** 0.5


def test_backward_is_the_same_mask():
    gen, key = base._gen(2), _key(21, 22)
    x, dy = base._randn(gen, 100, 203, dtype=BF16) + 1, base._randn(gen, 100, 203, dtype=BF16) + 1
    y, dx = L.dropout(x, 0.4, key, 7), L.dropout(dy, 0.4, key, 7)
    mask = ref.stays(100, 203, 0.4, key, 7)
    for before, after in ((x, y), (dy, dx)):  # a value of 0 stays 0
        assert torch.equal(after != 0, mask & (before != 0))


def test_a_captured_call_reads_its_key_anew():
    x, key = torch.ones(64, 1024, device="cuda"), _key(5, 0)
    L.dropout(x, 0.5, key)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = L.dropout(x, 0.5, key, 2)
        key[1] += 1
    for step in range(3):
        key[1] = step
        graph.replay()
        assert torch.equal(y != 0, ref.stays(64, 1024, 0.5, _key(5, step), 2)) and int(key[1]) == step + 1


@pytest.mark.parametrize("pad", [0, 8, 3])
def test_both_ways_from_python_agree(both, pad):  # noqa: F811
    gen, key = base._gen(4), _key(1, 2)
    for dtype in (F32, F16, BF16):
        x = base._randn(gen, 33, 264 + pad, dtype=dtype)[:, :264]
        both(lambda: L.dropout(x, 0.2, key, 3))
        both(lambda: L.dropout(x, 0.0, None))
    big = both(lambda: L.dropout(x, 0.2, key, 2 ** 31))
    for site in (-1, 2 ** 32, 2 ** 70):  # the binding leaves them to layers.py
        with pytest.raises(ValueError, match="site"):
            L.dropout(x, 0.2, key, site)
    assert torch.equal(big != 0, ref.stays(33, 264, 0.2, key, 2 ** 31) & (x != 0))
    y = L.dropout(x.contiguous()[None], 0.2, key, 3)
    assert y.shape == (1, 33, 264) and torch.equal(y[0], L.dropout(x, 0.2, key, 3))


def test_a_tensor_that_requires_a_gradient():
    x, key = torch.zeros(4, 8, device="cuda"), _key(1)
    x.requires_grad_()
    with pytest.raises(ValueError, match="requires a gradient"):
        L.dropout(x, 0.5, key)
    with torch.no_grad():
        L.dropout(x, 0.5, key)
