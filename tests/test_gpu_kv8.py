"""The 8-bit paged key/value cache on the GPU against its definition (kv8_plain: float64 attention on the same
codes): codes and scales bit for bit, attention and key weights within bounds derived there, evictions exactly."""
import numpy as np
import pytest
import torch

import rotated_bit_dit_b200 as R
from tests.kv8_plain import PAGE, PlainCache

pytestmark = pytest.mark.gpu
FMTS = [R.CODES_INT8, R.CODES_E4M3]


def rand(rng, rows, heads, gain=1.0, strong=True):
    """bf16-valued float32 [rows, heads, 128], some channels and tokens stronger."""
    x = rng.standard_normal((rows, heads, 128)).astype(np.float32) * gain
    if strong:
        x *= np.where(rng.random((1, heads, 128)) < 0.03, 4.0, 1.0)
        x *= np.where(rng.random((rows, heads, 1)) < 0.02, 6.0, 1.0)
    return torch.from_numpy(x.astype(np.float32)).bfloat16().float().numpy()


def dev(x, pad=0):
    """float32 [rows, heads, 128] -> bf16 [rows, heads*128] on the GPU, row stride larger by pad."""
    t = torch.from_numpy(np.ascontiguousarray(x)).reshape(x.shape[0], x.shape[1] * x.shape[2]).bfloat16().cuda()
    if not pad:
        return t
    full = torch.full((t.shape[0], t.shape[1] + pad), float("nan"), dtype=torch.bfloat16, device="cuda")
    full[:, :t.shape[1]] = t
    return full[:, :t.shape[1]]


def code_values(cache, b, h, side, n):
    """Code values float32 [n, 128] and page scales of a sequence, read out of the pool by the documented layout."""
    pages = cache.table[b].tolist()[:-(-n // PAGE)]
    t, d = np.meshgrid(np.arange(PAGE), np.arange(128), indexing="ij")
    at = 128 * t + 16 * ((d // 16) ^ (t % 8)) + d % 16
    typ = torch.int8 if cache.code_format == R.CODES_INT8 else torch.float8_e4m3fn
    raw = cache.codes[pages, h, side].reshape(len(pages), 64 * 128).view(typ).float().cpu().numpy()
    vals = raw[:, at.reshape(-1)].reshape(-1, 128)[:n]
    return vals, cache.scales[pages, h, side].cpu().numpy()


def check_codes(cache, plain):
    for b in range(plain.seqs):
        n = plain.len(b)
        assert cache.lens[b] == n and int(cache.device_lens[b]) == n
        for h in range(plain.heads):
            for side in range(2):
                got, s = code_values(cache, b, h, side, n)
                assert np.array_equal(s, plain.scales[b][h][side]), (b, h, side)
                assert np.array_equal(got, plain.codes[b][h][side]), (b, h, side)


def fill(cache, plain, rng, counts, gain=1.0, pad=0):
    k, v = rand(rng, sum(counts), plain.heads, gain), rand(rng, sum(counts), plain.heads, gain)
    cache.append(dev(k, pad), dev(v, pad), counts)
    at = 0
    for b, n in enumerate(counts):
        plain.append(b, k[at:at + n], v[at:at + n])
        at += n


def check_attend(cache, plain, rng, counts, heads, causal, q_gain=1.0, pad=0, weights=None, q=None):
    rows = sum(counts)
    if q is None:
        q = rand(rng, rows, heads, q_gain)
    cache.prepare(counts, append=False)
    guard = torch.full((rows + 2, heads * 128 + pad), 7.0, dtype=torch.bfloat16, device="cuda")
    out = guard[:rows, :heads * 128]
    w_in = weights
    w_out = None if weights is None else torch.full_like(weights, -3.0)
    y = cache.attend(dev(q, pad), heads, causal=causal, out=out, weights=w_in, weights_out=w_out)
    assert R.rbd_check() == 0
    assert y is out and bool((guard[rows:] == 7).all())
    if pad:
        assert bool((guard[:, heads * 128:] == 7).all())
    got = out.float().cpu().numpy().reshape(rows, heads, 128)
    at = 0
    for b, n in enumerate(counts):
        o, w, eo, ew = plain.attend(b, q[at:at + n].astype(np.float64), heads, causal)
        err = np.abs(got[at:at + n] - o)
        assert np.isfinite(got[at:at + n]).all()
        assert (err <= eo + 1e-30).all(), f"sequence {b}: {float((err / (eo + 1e-30)).max()):.2f} of the bound"
        if weights is not None:
            held = plain.len(b)
            base = w_in[b, :, :held].double().cpu().numpy()
            gw = w_out[b, :, :held].double().cpu().numpy()
            tol = ew + 2.0 ** -23 * (np.abs(base) + w)
            assert (np.abs(gw - (base + w)) <= tol + 1e-30).all(), \
                f"sequence {b}: weights {float((np.abs(gw - base - w) / (tol + 1e-30)).max()):.2f} of the bound"
            assert bool((w_out[b, :, held:] == -3).all())
        at += n
    return got


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("steps", [[1], [63, 1, 1], [64, 64], [1] * 9, [200, 5, 130], [0, 70]])
def test_append_bit_exact(fmt, steps):
    rng = np.random.default_rng(10 + len(steps))
    seqs, heads = 3, 2
    cache, plain = R.Int8KVCache(seqs, 512, heads, code_format=fmt), PlainCache(seqs, heads, fmt)
    for i, n in enumerate(steps):
        fill(cache, plain, rng, [n, n // 2, max(0, n - i)], gain=1.0 + i, pad=8 * (i % 2))
    check_codes(cache, plain)
    k, v = cache.tail(70)
    for b in range(seqs):
        for h in range(heads):
            for side, x in enumerate((k, v)):
                want = torch.from_numpy(plain.values(b, h, side)[-70:]).bfloat16()
                got = x[b, :, h * 128:(h + 1) * 128].cpu()
                assert torch.equal(got[70 - want.shape[0]:], want)
                assert not got[:70 - want.shape[0]].any()
    if plain.len(0) > 3:
        rk, rv = cache.read(0, 1, plain.len(0) - 3)
        for h in range(heads):
            assert torch.equal(rv[:, h * 128:(h + 1) * 128].cpu(),
                               torch.from_numpy(plain.values(0, h, 1)[1:-2]).bfloat16())
    assert R.rbd_check() == 0


@pytest.mark.parametrize("fmt", FMTS)
def test_append_non_finite_zero_and_tiny_values(fmt):
    rng = np.random.default_rng(3)
    cache, plain = R.Int8KVCache(1, 256, 1, code_format=fmt), PlainCache(1, 1, fmt)
    k = rand(rng, 70, 1)
    v = np.zeros_like(k)                       # all zero: the floor; a later token then sets the scale
    k[3, 0, 5], k[3, 0, 6], k[66, 0, :] = np.nan, np.inf, -np.inf
    cache.append(dev(k), dev(v), [70])
    plain.append(0, k, v)
    tiny = np.full((3, 1, 128), np.float32(2.0 ** -120))
    big = np.full((1, 1, 128), np.float32(3e38))
    for x in (tiny, tiny * 2.0 ** 115, big):
        x = torch.from_numpy(x.astype(np.float32)).bfloat16().float().numpy()
        cache.append(dev(x), dev(x), [x.shape[0]])
        plain.append(0, x, x)
    check_codes(cache, plain)


@pytest.mark.parametrize("fmt", FMTS)
def test_append_twice_at_the_same_place_changes_nothing(fmt):
    rng = np.random.default_rng(4)
    cache, plain = R.Int8KVCache(2, 256, 2, code_format=fmt), PlainCache(2, 2, fmt)
    fill(cache, plain, rng, [40, 100])
    k, v = rand(rng, 60, 2, 3.0), rand(rng, 60, 2, 3.0)
    cache.append(dev(k), dev(v), [30, 30])
    cache.append(dev(k), dev(v))
    plain.append(0, k[:30], v[:30])
    plain.append(1, k[30:], v[30:])
    check_codes(cache, plain)


# (lengths held, queries per sequence, cache heads, group)
ATTEND = [([1], [1], 1, 1), ([65], [1], 2, 3), ([64, 1, 0, 200], [1, 1, 1, 1], 1, 4), ([500, 130], [1, 1], 2, 16),
          ([300, 70, 129], [5, 0, 3], 2, 5), ([1000], [33], 1, 1), ([257, 40], [100, 40], 2, 2),
          ([700, 128, 1, 0], [300, 128, 1, 2], 1, 3), ([2100], [1], 1, 1), ([900, 260], [260, 260], 1, 4),
          ([10], [40], 1, 1), ([10, 500], [400, 70], 1, 2)]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("held,new,heads,group", ATTEND)
def test_attend(fmt, causal, held, new, heads, group):
    rng = np.random.default_rng(sum(held) + 7 * sum(new))
    cache, plain = R.Int8KVCache(len(held), 2304, heads, code_format=fmt), PlainCache(len(held), heads, fmt)
    fill(cache, plain, rng, held)
    check_attend(cache, plain, rng, new, heads * group, causal, q_gain=1.5, pad=16)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("held,new,heads,group", [([1], [1], 1, 1), ([300, 0, 70], [1, 1, 2], 2, 3),
                                                  ([400, 129], [200, 129], 1, 2), ([1500], [1], 1, 4),
                                                  ([260, 90, 640], [0, 90, 300], 2, 1), ([20, 30], [70, 70], 1, 1)])
def test_weights(fmt, causal, held, new, heads, group):
    rng = np.random.default_rng(sum(held) + 5 * sum(new))
    cache, plain = R.Int8KVCache(len(held), 1600, heads, code_format=fmt), PlainCache(len(held), heads, fmt)
    fill(cache, plain, rng, held)
    w = torch.from_numpy(rng.random((len(held), heads, 1601)).astype(np.float32)).cuda()
    check_attend(cache, plain, rng, new, heads * group, causal, q_gain=1.5, weights=w)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("held,new,heads,group", [([900], [800], 1, 1), ([700, 0, 333], [700, 50, 333], 2, 3),
                                                  ([3000], [130], 1, 8), ([513, 64], [513, 512], 1, 2)])
def test_attend_keys_shared_by_many_blocks(fmt, causal, held, new, heads, group):
    rng = np.random.default_rng(sum(held) + 3 * sum(new))
    cache, plain = R.Int8KVCache(len(held), 3180, heads, code_format=fmt), PlainCache(len(held), heads, fmt)
    fill(cache, plain, rng, held)
    w = torch.zeros((len(held), heads, 3200), device="cuda")
    check_attend(cache, plain, rng, new, heads * group, causal, q_gain=1.5, weights=w)
