"""Dropout with the residual on the GPU: the mask of the counter-based generator exactly, the
values within one rounding."""
import numpy as np
import pytest
import torch

import mixture_experts_layer_forward_b200 as moe

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    torch.cuda.set_device(0)


def words(counter, seed):
    """The generator's four words of one 64-bit counter, in Python's integers."""
    c = [counter & 0xFFFFFFFF, counter >> 32, 0, 0]
    k = [seed & 0xFFFFFFFF, seed >> 32]
    for _ in range(10):
        a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [(b >> 32) ^ c[1] ^ k[0], b & 0xFFFFFFFF, (a >> 32) ^ c[3] ^ k[1], a & 0xFFFFFFFF]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return c


def test_generator_known_answers():
    """The published vector of the ten-round generator for an all-zero counter and key holds for
    the reference above."""
    assert words(0, 0) == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]


def ref_keep(n, seed, offset, drop):
    keep = np.zeros((n + 7) // 8 * 8, bool)
    for i in range((n + 7) // 8):
        w = words((offset + i) & (2 ** 64 - 1), seed)
        for j in range(8):
            keep[i * 8 + j] = ((w[j // 2] >> (16 * (j & 1))) & 0xFFFF) >= drop
    return keep[:n]


def state(seed, offset):
    s = [v - 2 ** 64 if v >= 2 ** 63 else v for v in (seed, offset)]
    return torch.tensor(s, dtype=torch.int64, device="cuda")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n", [1, 7, 8, 9, 63, 1000, 4099])
@pytest.mark.parametrize("prob,seed,offset", [(0.1, 1234567, 0), (0.5, 2 ** 64 - 3, 2 ** 32 - 2),
                                              (0.9, 3, 2 ** 64 - 100), (0.0, 5, 9), (1.0, 5, 9)])
def test_values_and_mask(n, dtype, prob, seed, offset):
    g = torch.Generator().manual_seed(n)
    x, r, dy = (torch.randn(n, generator=g).to(dtype) for _ in range(3))
    drop = round(prob * 65536)
    keep = ref_keep(n, seed, offset, drop)
    scale = 65536 / (65536 - drop) if drop < 65536 else 0.0
    rng = state(seed, offset)
    eps = torch.finfo(dtype).eps / 2
    for res in (None, r):
        guard = torch.full((n + 16,), 3.0, dtype=dtype, device="cuda")
        y = guard[:n]
        moe.moe_dropout_add(x.cuda(), None if res is None else res.cuda(), y, prob, rng)
        base = np.zeros(n) if res is None else res.double().numpy()
        term = np.where(keep, x.double().numpy() * scale, 0.0)
        ref = base + term
        # the scale and the sum in fp32 (2^-24 each), then the rounding of the type
        tol = 2.0 ** -23 * (np.abs(term) + np.abs(ref)) + eps * np.abs(ref)
        assert np.all(np.abs(y.double().cpu().numpy() - ref) <= tol)
        if res is not None:
            assert np.array_equal(y.cpu().float().numpy()[~keep], res.float().numpy()[~keep])
        assert (guard[n:] == 3).all()
    dx = torch.empty(n, dtype=dtype, device="cuda")
    moe.moe_dropout_add_backward(dy.cuda(), dx, prob, rng)
    ref = np.where(keep, dy.double().numpy() * scale, 0.0)
    assert np.all(np.abs(dx.double().cpu().numpy() - ref) <= (2.0 ** -23 + eps) * np.abs(ref))


def test_dropped_values_do_not_pass():
    n, prob, rng = 4096, 0.5, state(77, 0)
    keep = torch.from_numpy(ref_keep(n, 77, 0, 32768)).cuda()
    x = torch.where(keep, 1.0, float("nan"))
    x[::3] = torch.where(keep[::3], 1.0, float("inf"))
    y = torch.empty_like(x)
    moe.moe_dropout_add(x, None, y, prob, rng)
    assert torch.equal(y, torch.where(keep, 2.0, 0.0))
    x = torch.where(keep, float("nan"), 1.0)         # a kept NaN does
    moe.moe_dropout_add(x, None, y, prob, rng)
    assert torch.equal(torch.isnan(y), keep)


def test_in_place_shapes_and_refusals():
    x, r = torch.randn(3, 5, 8, device="cuda"), torch.randn(3, 5, 8, device="cuda")
    rng, want = state(1, 2), torch.empty_like(x)
    moe.moe_dropout_add(x, r, want, 0.3, rng)
    y = x.clone()
    moe.moe_dropout_add(y, r, y, 0.3, rng)
    assert torch.equal(y, want)
    y = r.clone()
    moe.moe_dropout_add(x, y, y, 0.3, rng)
    assert torch.equal(y, want)
    empty = torch.empty(0, device="cuda")
    moe.moe_dropout_add(empty, None, torch.empty(0, device="cuda"), 0.3, rng)
    with pytest.raises(ValueError):
        moe.moe_dropout_add(x.transpose(0, 1), r, want, 0.3, rng)
    with pytest.raises(moe.MoeError):                # rows off the 16-byte boundary
        moe.moe_dropout_add(x.view(-1)[1:9], None, want.view(-1)[:8], 0.3, rng)
    with pytest.raises(ValueError):
        moe.moe_dropout_add(x, r, want, 0.3, rng.cpu())


def test_captured_call_follows_the_generator_state():
    """A captured step that advances its own offset draws a new mask each replay, and equals the
    eager calls with those offsets."""
    n = 10000
    x = torch.randn(n, device="cuda").to(torch.bfloat16)
    rng, y, dx = state(42, 0), torch.empty_like(x), torch.empty_like(x)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        moe.moe_dropout_add(x, None, y, 0.25, rng)
        moe.moe_dropout_add_backward(x, dx, 0.25, rng)
        rng[1] += (n + 7) // 8
    seen = []
    rng[1] = 0
    for i in range(3):
        g.replay()
        torch.cuda.synchronize()
        eager = torch.empty_like(x)
        moe.moe_dropout_add(x, None, eager, 0.25, state(42, i * 1250))
        assert torch.equal(y, eager) and torch.equal(dx, eager)
        seen.append(y.clone())
    assert not torch.equal(seen[0], seen[1]) and not torch.equal(seen[1], seen[2])


def test_share_kept_and_independence():
    """2^24 elements: the share kept within 6 standard deviations of 1 - p, also for pairs of
    neighbours and of the same place in two streams of offsets."""
    n = 1 << 24
    one = torch.ones(n, device="cuda")
    a, b = torch.empty_like(one), torch.empty_like(one)
    moe.moe_dropout_add(one, None, a, 0.25, state(9, 0))
    moe.moe_dropout_add(one, None, b, 0.25, state(9, n // 8))
    ka, kb = (a != 0).double(), (b != 0).double()
    for share, p in ((ka.mean(), 0.75), (kb.mean(), 0.75), ((ka * kb).mean(), 0.5625),
                     ((ka[1:] * ka[:-1]).mean(), 0.5625)):
        assert abs(float(share) - p) < 6 * (p * (1 - p) / n) ** 0.5 * 2


def test_offsets_past_32_bits():
    """More than 2^32 elements: the last ones are those of a small call at their counters."""
    n, m = (1 << 32) + 19, 4096 + 3
    x = torch.full((n,), 1.0, dtype=torch.bfloat16, device="cuda")
    y = torch.empty_like(x)
    moe.moe_dropout_add(x, x, y, 0.25, state(5, 7))
    start = (n - m) // 8 * 8
    part = torch.empty(n - start, dtype=torch.bfloat16, device="cuda")
    moe.moe_dropout_add(x[start:], x[start:], part, 0.25, state(5, 7 + start // 8))
    assert torch.equal(y[start:], part)
