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


@pytest.mark.parametrize("fmt,causal", [(0, True), (1, False)])
@pytest.mark.parametrize("heads,group,held,new", [
    (1, 64, [2100, 600, 2, 0, 900], [620, 30, 3, 2, 0]),                       # 169 blocks, operand images
    (2, 32, [2100] + [70, 130, 300] * 13, [12] * 40),                          # 198 blocks that convert for themselves
])
def test_blocks_of_a_last_wave_share_their_keys(fmt, causal, heads, group, held, new):
    """More blocks than processors: the blocks behind the last full wave have their keys split."""
    rng = np.random.default_rng(31)
    cache, plain = R.Int8KVCache(len(held), 2112, heads, code_format=fmt), PlainCache(len(held), heads, fmt)
    fill(cache, plain, rng, held)
    rows, q_heads = sum(new), heads * group
    assert R.rbd_kv8_attn_workspace_bytes(len(held), heads, q_heads, rows, 2100) > 0
    q = rand(rng, rows, q_heads)
    cache.prepare(new, append=False)
    w = torch.zeros((len(held), heads, 2112), device="cuda")
    got = cache.attend(dev(q), q_heads, causal=causal, weights=w)
    again = cache.attend(dev(q), q_heads, causal=causal)
    assert R.rbd_check() == 0 and torch.equal(got, again)
    got = got.float().cpu().numpy().reshape(rows, q_heads, 128)
    picks = [[(17 * i + 5 * j) % group for j in range(3)] for i in range(heads)]       # of every cache head's queries
    at = 0
    for b, n in enumerate(new):
        some = q[at:at + n].reshape(n, heads, group, 128)
        part = np.stack([some[:, i, picks[i]] for i in range(heads)], 1).reshape(n, 3 * heads, 128)
        o, _, eo, _ = plain.attend(b, part.astype(np.float64), 3 * heads, causal)
        mine = got[at:at + n].reshape(n, heads, group, 128)
        mine = np.stack([mine[:, i, picks[i]] for i in range(heads)], 1).reshape(n, 3 * heads, 128)
        assert (np.abs(mine - o) <= eo + 1e-30).all(), b
        at += n
        # a row that sees a key adds one to the sum of its weights: a float32 sum of `held` terms each way
        sums = w[b].double().sum(1).cpu().numpy()
        live = min(n, held[b]) if causal else (n if held[b] else 0)
        assert (np.abs(sums - live * group) <= live * group * ((held[b] + n * group) * 2.0 ** -23 + 2.0 ** -20) + 1e-30).all(), b


def evict_case(rng, fmt, lens, heads, keep, recent, weights, in_place=False):
    """Entry-level eviction of a filled cache against the plain one; returns nothing, asserts everything."""
    n, width = len(lens), weights.shape[2]
    per = -(-keep // PAGE)
    total = sum(-(-x // PAGE) for x in lens) + n * per
    cache = R.Int8KVCache(n, max(max(lens), keep, 1), heads, pages=total, code_format=fmt)
    plain = PlainCache(n, heads, fmt)
    fill(cache, plain, rng, lens)
    dst = cache.spare_pages(n, per)
    w = weights.cuda()
    kept = torch.full((n, heads, keep), -7, dtype=torch.int32, device="cuda")
    w_out = w if in_place else torch.full((n, heads, keep + 3), 9.0, device="cuda")
    new_lens = torch.empty(n, dtype=torch.int32, device="cuda")
    R.rbd_kv8_evict(w, cache.device_lens, cache.table, cache.codes, cache.scales, keep, recent, dst, kept, w_out, new_lens,
                    fmt)
    assert R.rbd_check() == 0
    for b in range(n):
        want = plain.evict(b, weights[b].numpy(), keep, recent)
        m = min(lens[b], keep)
        assert int(new_lens[b]) == m
        for h in range(heads):
            assert kept[b, h, :m].tolist() == want[h].tolist() and bool((kept[b, h, m:] == -1).all()), (b, h)
            got = w_out[b, h].cpu()
            assert torch.equal(got[:m].nan_to_num(-5.0), weights[b, h][torch.from_numpy(want[h])].nan_to_num(-5.0))
            assert not got[m:].any()
    # the kept tokens, read out of the new pages
    cache.table[:, :per] = dst
    cache.device_lens.copy_(new_lens)
    cache._lens = [min(x, keep) for x in lens]
    for b in range(n):
        for h in range(heads):
            for side in range(2):
                got, s = code_values(cache, b, h, side, plain.len(b))
                assert np.array_equal(s, plain.scales[b][h][side]) and np.array_equal(got, plain.codes[b][h][side])


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("lens,heads,keep,recent", [([1], 1, 1, 0), ([70, 3, 0], 2, 64, 10), ([200, 129], 3, 65, 65),
                                                    ([500], 1, 100, 0), ([2000, 1000, 40], 2, 130, 7), ([64], 2, 64, 64),
                                                    ([4100], 1, 4096, 100)])
def test_evict(fmt, lens, heads, keep, recent):
    rng = np.random.default_rng(keep + 13 * recent)
    w = torch.from_numpy(np.exp(2 * rng.standard_normal((len(lens), heads, max(max(lens), keep)))).astype(np.float32))
    evict_case(rng, fmt, lens, heads, keep, recent, w)


def test_evict_ties_zeros_nan_negative_and_in_place():
    rng = np.random.default_rng(5)
    w = torch.zeros(3, 2, 700)
    w[0, 0, ::3] = 1.0                                   # two values: ties everywhere
    w[0, 1] = -0.0
    w[0, 1, 5] = 0.0
    w[1, 0] = torch.from_numpy(rng.integers(-3, 4, 700).astype(np.float32))
    w[1, 1, 100:200] = float("nan")
    w[1, 1, 300] = float("-inf")
    w[2, 0, 50:60] = float("inf")
    w[2, 1] = torch.from_numpy(np.float32(2.0) ** rng.integers(-149, 127, 700).astype(np.float32))
    evict_case(rng, R.CODES_INT8, [700, 600, 500], 2, 150, 20, w)
    evict_case(rng, R.CODES_E4M3, [700, 600, 500], 2, 450, 0, w)
    evict_case(rng, R.CODES_INT8, [700, 600, 500], 2, 150, 20, w, in_place=True)


def test_evict_longer_than_the_selection_holds_on_chip():
    rng = np.random.default_rng(6)
    n = 49152 + 3000                                     # the last 3000 positions are read from global memory
    w = torch.from_numpy(rng.integers(0, 50, (1, 1, n)).astype(np.float32))
    evict_case(rng, R.CODES_INT8, [n], 1, 700, 33, w)
    evict_case(rng, R.CODES_INT8, [n], 1, 6000, 33, w, in_place=True)


@pytest.mark.parametrize("fmt", FMTS)
def test_append_attend_evict_together(fmt):
    """A serving loop: prompts, tokens one by one with weights, an eviction, more tokens; attention and the
    cache's contents against the plain one throughout."""
    rng = np.random.default_rng(8)
    seqs, heads, group = 3, 2, 2
    cache, plain = R.Int8KVCache(seqs, 400, heads, pages=24, code_format=fmt), PlainCache(seqs, heads, fmt)
    w = torch.zeros((seqs, heads, 400), device="cuda")
    pw = [np.zeros((heads, 400)) for _ in range(seqs)]
    bound = [np.zeros((heads, 400)) for _ in range(seqs)]

    def step(counts):
        fill(cache, plain, rng, counts)
        q = rand(rng, sum(counts), heads * group, 1.5)
        y = cache.attend(dev(q), heads * group, weights=w).float().cpu().numpy().reshape(-1, heads * group, 128)
        at = 0
        for b, n in enumerate(counts):
            o, dw, eo, ew = plain.attend(b, q[at:at + n].astype(np.float64), heads * group, True)
            assert (np.abs(y[at:at + n] - o) <= eo).all()
            held = plain.len(b)
            pw[b][:, :held] += dw
            bound[b][:, :held] += ew + 2.0 ** -23 * np.abs(pw[b][:, :held])
            assert (np.abs(w[b, :, :held].double().cpu().numpy() - pw[b][:, :held]) <= bound[b][:, :held]).all()
            at += n
    step([150, 40, 301])
    for _ in range(4):
        step([1, 1, 1])
    kept = cache.evict(w, 100, 30)
    for b in range(seqs):
        # which tokens stay is decided by the weights the kernels added up
        got = kept[b].cpu().numpy()
        m = min(plain.len(b), 100)
        assert (got[:, m:] == -1).all()
        for h in range(heads):
            x, n = pw[b][h], plain.len(b)
            out = np.setdiff1d(np.arange(n), got[h, :m])
            assert out.size == n - m and (n <= 100 or (out < n - 30).all())
            if out.size:
                chosen = got[h, :m - 30]
                assert x[chosen].min() >= x[out].max() - bound[b][h].max() * 2
        forced = np.zeros((heads, plain.len(b)))
        for h in range(heads):
            forced[h, got[h, :m]] = 1.0
            pw[b][h, :m], bound[b][h, :m] = pw[b][h, got[h, :m]], bound[b][h, got[h, :m]]
            pw[b][h, m:], bound[b][h, m:] = 0.0, 0.0
        plain.evict(b, forced, 100, 30)
    check_codes(cache, plain)
    assert cache.lens == [100, 44, 100] and cache.free_pages == 24 - 2 - 1 - 2
    assert not w[:, :, 100:].any()
    for _ in range(3):
        step([1, 2, 0])
    cache.release(1)
    plain.codes[1] = [[np.zeros((0, 128), np.float32) for _ in range(2)] for _ in range(heads)]
    plain.scales[1] = [[np.zeros(0, np.float32) for _ in range(2)] for _ in range(heads)]
    w[1], pw[1][:], bound[1][:] = 0, 0, 0
    step([0, 66, 1])
    check_codes(cache, plain)
    assert R.rbd_check() == 0


def test_scales_far_apart_and_sharp_scores():
    """Pages whose value scales differ by up to 2^80, with the small ones attended to; keys far larger in the last
    pages, so that the running maximum moves; a query whose scores all vanish."""
    rng = np.random.default_rng(9)
    cache, plain = R.Int8KVCache(1, 512, 1), PlainCache(1, 1, 0)
    for gain_k, gain_v in ((1.0, 2.0 ** 40), (1.0, 1.0), (6.0, 2.0 ** -40), (12.0, 2.0 ** -40), (0.0, 2.0 ** 20)):
        k, v = rand(rng, 64, 1, gain_k, strong=False), rand(rng, 64, 1, gain_v, strong=False)
        cache.append(dev(k), dev(v), [64])
        plain.append(0, k, v)
    for n in (1, 3, 70):
        q = rand(rng, n, 1, 3.0)
        q[0] = 0.0
        q[n // 2] *= np.float32(2.0 ** -100)
        check_attend(cache, plain, rng, [n], 1, False, q=q)
        check_attend(cache, plain, rng, [n], 1, True, q=q)


@pytest.mark.parametrize("n", [1, 12, 200])
def test_a_nan_query_stays_in_its_row(n):
    rng = np.random.default_rng(11)
    cache, plain = R.Int8KVCache(1, 512, 1, code_format=R.CODES_E4M3), PlainCache(1, 1, 1)
    cache.codes.fill_(0x7F)                              # pages that held something: E4M3 NaN behind the tokens
    fill(cache, plain, rng, [300])
    q = rand(rng, n, 2)
    clean = check_attend(cache, plain, rng, [n], 2, True, q=q)
    bad = q.copy()
    bad[0, 1] = np.nan
    bad[n - 1, 0, 3] = np.inf
    got = cache.attend(dev(bad), 2).float().cpu().numpy().reshape(n, 2, 128)
    assert np.isnan(got[0, 1]).all()
    keep = np.ones((n, 2), bool)
    keep[0, 1] = keep[n - 1, 0] = False
    assert np.array_equal(got[keep], clean[keep])


def test_device_side_metadata_is_refused_and_the_rest_is_right():
    rng = np.random.default_rng(12)
    for new in (1, 40, 300):
        cache, plain = R.Int8KVCache(3, 512, 1), PlainCache(3, 1, 0)
        fill(cache, plain, rng, [300, 310, 320])
        q = rand(rng, 3 * new, 1)
        cache.prepare([new] * 3, append=False)
        want = cache.attend(dev(q), 1)
        assert R.rbd_check() == 0
        w = torch.zeros(3, 1, 512, device="cuda")
        for spoil in ("page", "negative page", "length", "offsets"):
            table, lens, cu = cache.table.clone(), cache.device_lens.clone(), cache._cu.clone()
            if spoil == "page":
                table[1, 2] = 10 ** 6
            elif spoil == "negative page":
                table[1, 0] = -1
            elif spoil == "length":
                lens[1] = 10 ** 6
            else:
                cu[3] = 10 ** 6
            o = torch.zeros_like(want)
            work = torch.empty(R.rbd_kv8_attn_workspace_bytes(3, 1, 1, 3 * new, 512, True), dtype=torch.uint8, device="cuda")
            R.rbd_kv8_attn(dev(q), cu, lens, table, cache.codes, cache.scales, o, 1, work, 512, weights_in=w, weights_out=w)
            assert R.rbd_check() == 1 and R.rbd_check() == 0
            assert torch.equal(o[:new], want[:new])
            if spoil != "offsets":
                assert torch.equal(o[2 * new:], want[2 * new:])
        before, scales = cache.codes.clone(), cache.scales.clone()
        table = cache.table.clone()
        table[1] = 10 ** 6
        x = dev(rand(rng, 3 * new, 1))
        R.rbd_kv8_append(x, x, cache._cu, cache.device_lens, table, cache.codes, cache.scales)
        assert R.rbd_check() == 1
        mine = cache.table[1].long()[:5]
        assert torch.equal(cache.codes[mine], before[mine]) and torch.equal(cache.scales[mine], scales[mine])


@pytest.mark.parametrize("rows,q_heads", [(300, 8), (40, 4), (3, 1)])
def test_overlapping_offsets_are_refused(rows, q_heads):
    """Offsets that go up and down give sequences that share rows, more of them than the launch is laid out for."""
    rng = np.random.default_rng(29)
    cache, plain = R.Int8KVCache(8, 512, 1), PlainCache(8, 1, 0)
    fill(cache, plain, rng, [400] * 8)
    cu = torch.tensor([0, rows] * 4 + [0], dtype=torch.int32, device="cuda")
    q = dev(rand(rng, rows, q_heads))
    o, w = torch.zeros_like(q), torch.zeros(8, 1, 512, device="cuda")
    need = R.rbd_kv8_attn_workspace_bytes(8, 1, q_heads, rows, 512, True)
    guard = torch.full((need + 4096,), 7, dtype=torch.uint8, device="cuda")
    R.rbd_kv8_attn(q, cu, cache.device_lens, cache.table, cache.codes, cache.scales, o, q_heads, guard[:need], 512,
                   weights_in=w, weights_out=w)
    assert R.rbd_check() == 1 and R.rbd_check() == 0
    assert bool((guard[need:] == 7).all())


def test_rows_of_no_sequence_are_left_alone():
    rng = np.random.default_rng(13)
    cache, plain = R.Int8KVCache(2, 1024, 1), PlainCache(2, 1, 0)
    fill(cache, plain, rng, [900, 100])
    for a, b, tail in ((1, 1, 3), (30, 20, 30), (300, 5, 40)):
        rows = 2 + a + b + tail
        q, o = dev(rand(rng, rows, 2)), torch.full((rows, 256), 5.0, dtype=torch.bfloat16, device="cuda")
        cu = torch.tensor([2, 2 + a, 2 + a + b], dtype=torch.int32, device="cuda")
        work = torch.empty(R.rbd_kv8_attn_workspace_bytes(2, 1, 2, rows, 900), dtype=torch.uint8, device="cuda")
        R.rbd_kv8_attn(q, cu, cache.device_lens, cache.table, cache.codes, cache.scales, o, 2, work if work.numel() else None,
                       900)
        assert R.rbd_check() == 0
        assert bool((o[:2] == 5).all()) and bool((o[2 + a + b:] == 5).all()) and not bool((o[2:2 + a + b] == 5).all())


def test_pool_beyond_32_bit_offsets():
    """Pages in a pool of more than 2^31 bytes (and 2^32), the sequence's own ones at its end."""
    rng = np.random.default_rng(14)
    pages = (1 << 32) // 16384 + 40
    cache, plain = R.Int8KVCache(1, 1024, 1, pages=pages), PlainCache(1, 1, 0)
    cache._free = list(range(pages - 20, pages))         # taken from the far end
    fill(cache, plain, rng, [500])
    assert int(cache.table[0, 0]) > (1 << 32) // 16384
    check_codes(cache, plain)
    w = torch.zeros(1, 1, 1024, device="cuda")
    check_attend(cache, plain, rng, [1], 2, True, weights=w)
    check_attend(cache, plain, rng, [300], 2, True, weights=w)
    k, v = cache.tail(500)
    assert torch.equal(v[0].cpu(), torch.from_numpy(plain.values(0, 0, 1)).bfloat16())


@pytest.mark.parametrize("counts", [[1, 1, 1], [20, 20, 20], [90, 90, 90]])
def test_captured_steps_replay_with_other_lengths(counts):
    """Append and attend captured once (two graphs, with and without weights), replayed at other lengths and
    inputs in turn: the results are those of eager calls on an equal cache."""
    rng = np.random.default_rng(15)
    heads, group, rows = 2, 2, sum(counts)
    caches = [R.Int8KVCache(3, 700, heads) for _ in range(2)]
    k0, v0 = rand(rng, 330, heads), rand(rng, 330, heads)
    for c in caches:
        c.append(dev(k0), dev(v0), [100, 30, 200])
    kb, vb = (torch.empty((rows, heads * 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    qb = torch.empty((rows, heads * group * 128), dtype=torch.bfloat16, device="cuda")
    outs = [torch.empty_like(qb) for _ in range(2)]
    w = torch.zeros(3, heads, 700, device="cuda")
    we = torch.zeros_like(w)
    live, eager = caches
    graphs = []
    side = torch.cuda.Stream()
    for i in range(2):
        if i == 0:
            live.prepare(counts)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            live.append(kb, vb)
            live.attend(qb, heads * group, out=outs[i], weights=w if i else None)
        graphs.append(g)
    for step in range(4):
        k, v, q = rand(rng, rows, heads), rand(rng, rows, heads), rand(rng, rows, heads * group)
        if step:
            live.prepare(counts)
        kb.copy_(dev(k)), vb.copy_(dev(v)), qb.copy_(dev(q))
        graphs[step % 2].replay()
        eager.append(dev(k), dev(v), counts)
        y = eager.attend(dev(q), heads * group, weights=we if step % 2 else None)
        torch.cuda.synchronize()
        assert R.rbd_check() == 0
        # (the splits of a long layout join in another order: a bf16 step at most, from float32 sums)
        d = (outs[step % 2].float() - y.float()).abs()
        assert bool((d <= 2.0 ** -7 * y.float().abs() + 1e-5).all())
        assert torch.allclose(w, we, rtol=1e-5, atol=1e-6)
    for a, b in zip(live.tail(400), eager.tail(400)):
        assert torch.equal(a, b)


def test_two_streams_at_once():
    rng = np.random.default_rng(16)
    streams = [torch.cuda.Stream() for _ in range(2)]
    runs = []
    for s in streams:
        cache, plain = R.Int8KVCache(2, 3000, 2), PlainCache(2, 2, 0)
        with torch.cuda.stream(s):
            fill(cache, plain, rng, [2500, 700])
        runs.append((cache, [dev(rand(rng, 2, 8)), dev(rand(rng, 600, 8))]))
    torch.cuda.synchronize()
    want = []
    for cache, qs in runs:
        for q in qs:
            cache.prepare([q.shape[0] // 2] * 2, append=False)
            want.append(cache.attend(q, 8))
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for i in range(2):
            for s, (cache, qs) in zip(streams, runs):
                with torch.cuda.stream(s):
                    cache.prepare([qs[i].shape[0] // 2] * 2, append=False)
                    got.append((s, cache.attend(qs[i], 8)))
        torch.cuda.synchronize()
        assert R.rbd_check() == 0
        for (_, y), x in zip(got, [want[0], want[2], want[1], want[3]]):
            assert torch.equal(y, x)


def test_a_step_without_rows():
    """No sequence has a row: nothing is attended to, and weights_out becomes weights_in over the tokens held."""
    rng = np.random.default_rng(30)
    cache, plain = R.Int8KVCache(3, 512, 2), PlainCache(3, 2, 0)
    fill(cache, plain, rng, [300, 0, 70])
    none = torch.empty((0, 4 * 128), dtype=torch.bfloat16, device="cuda")
    cache.append(none[:, :256], none[:, :256], [0, 0, 0])
    check_codes(cache, plain)
    w = torch.rand((3, 2, 512), device="cuda")
    out = torch.full_like(w, -3.0)
    assert cache.attend(none, 4).shape == (0, 512)
    assert cache.attend(none, 4, weights=w, weights_out=out).shape == (0, 512)
    assert R.rbd_check() == 0
    for b, n in enumerate([300, 0, 70]):
        assert torch.equal(out[b, :, :n], w[b, :, :n]) and bool((out[b, :, n:] == -3).all())


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("held", [0, 40])
def test_rows_that_see_no_key_are_zeros_every_time(fmt, held):
    """Blocks of 256 rows that see no key (an empty sequence, or the queries in front of a short one's first token):
    zeros, whichever of a block's warps fetches its queries last."""
    rng = np.random.default_rng(32)
    heads, group, n = 2, 3, 5000
    cache, plain = R.Int8KVCache(2, 1024, heads, code_format=fmt), PlainCache(2, heads, fmt)
    fill(cache, plain, rng, [held, 900])
    q = dev(rand(rng, n + 600, heads * group))
    cache.prepare([n, 600], append=False)
    first = None
    for _ in range(20):
        out = torch.full((n + 600, heads * group * 128), 7.0, dtype=torch.bfloat16, device="cuda")
        cache.attend(q, heads * group, out=out)
        assert not out[:n - held].any()
        assert bool(out[n - held:].any(dim=1).all())
        first = out if first is None else first
        assert torch.equal(out, first)
    assert R.rbd_check() == 0


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("n,held", [(1, 300), (12, 300), (200, 300), (200, 2), (1, 5000), (300, 5000)])
def test_an_infinite_query_gives_nan_in_its_row(fmt, causal, n, held):
    """Its scores are infinite (or NaN, against a zero): the softmax over them is NaN, wherever the infinities stand,
    and so are the weights of the keys the row sees; other rows and the keys it does not see are left alone."""
    rng = np.random.default_rng(33)
    cache, plain = R.Int8KVCache(1, 5120, 1, code_format=fmt), PlainCache(1, 1, fmt)
    for lucky in (np.arange(held) % 8 == 6, np.arange(held) % 8 == 7, np.arange(held) == 6, np.zeros(held, bool),
                  np.ones(held, bool)):
        if cache.lens[0]:
            cache.release(0)
            plain = PlainCache(1, 1, fmt)
        k, v = rand(rng, held, 1), rand(rng, held, 1)
        k[:, 0, 3] = np.where(lucky, 4.0, -4.0)          # the sign of the score against +inf in channel 3
        cache.append(dev(k), dev(v), [held])
        plain.append(0, k, v)
        q = rand(rng, n, 2)
        clean = check_attend(cache, plain, rng, [n], 2, causal, q=q)
        row = n // 2
        q[row, 1, 3] = np.inf
        w = torch.zeros((1, 1, 5120), device="cuda")
        got = cache.attend(dev(q), 2, causal=causal).float().cpu().numpy().reshape(n, 2, 128)
        also = cache.attend(dev(q), 2, causal=causal, weights=w).float().cpu().numpy().reshape(n, 2, 128)
        assert R.rbd_check() == 0
        sees = max(0, held - n + row + 1) if causal else held
        keep = np.ones((n, 2), bool)
        keep[row, 1] = False
        for y in (got, also):
            assert np.isnan(y[row, 1]).all() if sees else not y[row, 1].any()
            assert np.array_equal(y[keep], clean[keep])
        w = w[0, 0].cpu().numpy()
        assert np.isnan(w[:sees]).all() and np.isfinite(w[sees:]).all()


def test_weights_in_any_layout_and_none_that_overlap():
    """Weights whose heads lie outside the sequences, and in and out interleaved in one buffer: as in a layout of
    their own.  Expanded ones are refused, and an eviction refused for them moves no pages."""
    rng = np.random.default_rng(34)
    seqs, heads, width = 3, 2, 512
    cache, plain = R.Int8KVCache(seqs, width, heads, pages=40), PlainCache(seqs, heads, 0)
    fill(cache, plain, rng, [300, 70, 500])
    cache.prepare([2, 1, 40], append=False)
    q = dev(rand(rng, 43, heads))
    w = torch.rand((seqs, heads, width), device="cuda")
    want = torch.zeros_like(w)
    o = cache.attend(q, heads, weights=w, weights_out=want)
    turned = torch.zeros((heads, seqs, width), device="cuda").transpose(0, 1)
    turned.copy_(w)
    cache.attend(q, heads, weights=turned)
    both = torch.zeros((seqs, 2, heads, width), device="cuda")
    both[:, 0] = w
    assert torch.equal(cache.attend(q, heads, weights=both[:, 0], weights_out=both[:, 1]), o)
    for b, n in enumerate([300, 70, 500]):
        assert torch.equal(turned[b, :, :n], want[b, :, :n]) and torch.equal(both[b, 1, :, :n], want[b, :, :n])
    assert torch.equal(both[:, 0], w)
    for bad in (w[:1].expand(seqs, heads, width), w[:, :1].expand(seqs, heads, width)):
        with pytest.raises(R.RbdError):
            cache.attend(q, heads, weights=bad)
        with pytest.raises(R.RbdError):
            cache.evict(bad, 100, 10)
    flat = torch.zeros(seqs * heads * width + 1, device="cuda")
    with pytest.raises(R.RbdError):
        cache.attend(q, heads, weights=flat[:-1].view(seqs, heads, width), weights_out=flat[1:].view(seqs, heads, width))
    assert cache.lens == [300, 70, 500] and cache.free_pages == 40 - 5 - 2 - 8
    check_codes(cache, plain)
    kept = cache.evict(turned, 100, 10)
    for b in range(seqs):
        got = plain.evict(b, want[b].cpu().numpy(), 100, 10)
        for h in range(heads):
            assert kept[b, h, :len(got[h])].tolist() == got[h].tolist()
    check_codes(cache, plain)
    assert R.rbd_check() == 0


@pytest.mark.parametrize("new,held", [(1, 9000), (12, 9000), (300, 9000), (1, 300)])
def test_rows_of_refused_offsets_are_left_alone(new, held):
    """Also where the keys are split, whose parts are joined by another kernel."""
    rng = np.random.default_rng(35)
    cache, plain = R.Int8KVCache(4, 9216, 1), PlainCache(4, 1, 0)
    fill(cache, plain, rng, [held, 40, held - 100, 77])
    rows = 4 * new
    q = rand(rng, rows, 2)
    big = 10 ** 6
    for cu in ([0, new, 2 * new, 3 * new, big], [0, new, big, big, 4 * new], [0, new, 2 * new, -1, 4 * new],
               [big, big, big, big, big]):
        work = torch.full((R.rbd_kv8_attn_workspace_bytes(4, 1, 2, rows, 9216, True),), 0x41, dtype=torch.uint8, device="cuda")
        o = torch.full((rows, 256), 5.0, dtype=torch.bfloat16, device="cuda")
        w = torch.zeros(4, 1, 9216, device="cuda")
        R.rbd_kv8_attn(dev(q), torch.tensor(cu, dtype=torch.int32, device="cuda"), cache.device_lens, cache.table, cache.codes,
                       cache.scales, o, 2, work, 9216, weights_in=w, weights_out=w)
        assert R.rbd_check() == 1 and R.rbd_check() == 0
        got = o.float().cpu().numpy().reshape(rows, 2, 128)
        mine = np.zeros(rows, bool)
        for b in range(4):
            gw = w[b].double().cpu().numpy()
            if 0 <= cu[b] <= cu[b + 1] <= rows:
                at = slice(cu[b], cu[b + 1])
                want, dw, eo, ew = plain.attend(b, q[at].astype(np.float64), 2, True)
                n = plain.len(b)
                assert (np.abs(got[at] - want) <= eo + 1e-30).all()
                assert (np.abs(gw[:, :n] - dw) <= ew + 2.0 ** -23 * dw + 1e-30).all() and not gw[:, n:].any()
                mine[at] = True
            else:
                assert not gw.any()
        assert (got[~mine] == 5).all(), cu


def check_pages_outside_the_pool(new, held, fmt):
    """Keys of a page that the table does not name are not there: not for the queries, and not in the key weights."""
    rng = np.random.default_rng(36)
    heads, group = 1, 2
    cache, plain = R.Int8KVCache(3, 9216, heads, pages=450, code_format=fmt), PlainCache(3, heads, fmt)
    fill(cache, plain, rng, [200, held, 130])
    counts = [min(new, 200), new, min(new, 130)]
    rows = sum(counts)
    q = rand(rng, rows, heads * group)
    cache.prepare(counts, append=False)
    first = (held - new) // PAGE                              # pages in front of it are seen whole by every query
    codes, scales = [list(x) for x in plain.codes[1][0]], [list(x) for x in plain.scales[1][0]]
    every = list(range(-(-held // PAGE)))
    for gone, causal in (([0], True), ([first - 1], True), ([1, first // 2 + 1], False), (every[1:], False), (every, True),
                         (every, False)):
        table = cache.table.clone()
        table[1, gone] = torch.tensor([10 ** 6, -1] * len(gone), dtype=torch.int32, device="cuda")[:len(gone)]
        stay = np.array([t // PAGE not in gone for t in range(held)])
        for side in range(2):
            plain.codes[1][0][side] = np.asarray(codes[side], np.float32).reshape(held, 128)[stay]
            plain.scales[1][0][side] = np.delete(np.asarray(scales[side], np.float32), gone)
        for weigh in (False, True):
            need = R.rbd_kv8_attn_workspace_bytes(3, heads, heads * group, rows, 9216, weigh)
            work = torch.full((need,), 0x41, dtype=torch.uint8, device="cuda")
            o = torch.full((rows, heads * group * 128), 5.0, dtype=torch.bfloat16, device="cuda")
            w = torch.from_numpy(rng.random((3, heads, 9216)).astype(np.float32)).cuda() if weigh else None
            was = w.double().cpu().numpy() if weigh else None
            R.rbd_kv8_attn(dev(q), cache._cu, cache.device_lens, table, cache.codes, cache.scales, o, heads * group,
                           work if need else None, 9216, causal=causal, weights_in=w, weights_out=w, code_format=fmt)
            assert R.rbd_check() == 1 and R.rbd_check() == 0
            got = o.float().cpu().numpy().reshape(rows, heads * group, 128)
            at = 0
            for b, n in enumerate(counts):
                want, dw, eo, ew = plain.attend(b, q[at:at + n].astype(np.float64), heads * group, causal)
                assert (np.abs(got[at:at + n] - want) <= eo + 1e-30).all(), (b, gone, causal, weigh)
                if weigh:
                    keys = stay if b == 1 else np.ones(cache.lens[b], bool)
                    add, tol = np.zeros(9216), np.zeros(9216)
                    add[:keys.size][keys], tol[:keys.size][keys] = dw[0], ew[0]
                    d = np.abs(w[b, 0].double().cpu().numpy() - (was[b, 0] + add))
                    assert (d <= tol + 2.0 ** -23 * (was[b, 0] + add) * (add > 0)).all(), (b, gone, causal)
                at += n


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("new,held", [(70, 400), (300, 9000), (900, 2000)])
def test_pages_outside_the_pool_many_rows(new, held, fmt):
    check_pages_outside_the_pool(new, held, fmt)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("new,held", [(1, 400), (12, 400), (1, 9000), (12, 9000)])
def test_pages_outside_the_pool_few_rows(new, held, fmt):
    check_pages_outside_the_pool(new, held, fmt)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("n,held", [(1, 300), (12, 300), (200, 300), (1, 9000), (300, 9000)])
def test_scores_of_any_size(fmt, n, held):
    """Scores of +-2^25 and less give the definition's row.  A row whose largest score is beyond 2^27 has no float32
    maximum to go by and gives NaN; single scores far below a row's largest give their keys no weight.  Other rows
    are as they were."""
    rng = np.random.default_rng(37)
    cache, plain = R.Int8KVCache(1, 9216, 1, code_format=fmt), PlainCache(1, 1, fmt)
    k, v = rand(rng, held, 1, strong=False), rand(rng, held, 1)
    k[:, 0, [5, 9, 11]] = 0.0
    k[64:128, 0, 9] = 2.0 ** 20                              # keys of one page alone answer to channel 9
    k[70, 0, 11] = 2.0 ** 20                                 # one key to channel 11
    cache.append(dev(k), dev(v), [held])
    plain.append(0, k, v)
    q = rand(rng, n, 2)
    q[:, :, [5, 9, 11]] = 0.0
    clean = check_attend(cache, plain, rng, [n], 2, False, q=q)
    row = n // 2
    keep = np.ones((n, 2), bool)
    keep[row] = False

    def attend(a, b):
        """Row `row` with heads a, b for queries: its outputs and the key weights."""
        q[row] = np.stack([a, b])
        w = torch.zeros((1, 1, 9216), device="cuda")
        got = cache.attend(dev(q), 2, causal=False).float().cpu().numpy().reshape(n, 2, 128)
        also = cache.attend(dev(q), 2, causal=False, weights=w).float().cpu().numpy().reshape(n, 2, 128)
        assert R.rbd_check() == 0
        assert np.array_equal(got[keep], clean[keep]) and np.array_equal(got, also, equal_nan=True)
        return got[row], w[0, 0, :held].cpu().numpy()

    base, unit = q[row].copy(), np.eye(128, dtype=np.float32)
    values, own = plain.values(0, 0, 1), plain.values(0, 0, 0)[70, 11]
    for score in (2.0 ** 10, 2.0 ** 20, 2.0 ** 23, 2.0 ** 24.9):
        # key 70 takes all the weight: its value, P and its sum rounded alike but for fp16's half step, then bf16
        x = torch.tensor(score * 128 ** 0.5 / own).bfloat16().float().item()
        got, w = attend(unit[11] * x, unit[11] * x)
        assert (np.abs(got - values[70]) <= np.abs(values[70]) * (2.0 ** -8 + 1.01 * 2.0 ** -11) + 1e-30).all(), score
        # The weight is 2^(x - m) / L from a score formed again: x, its factors, m and m + log2 L are each within half a
        # step, 2^-24, of at most |x|.
        off = 2.0 ** (4 * 2.0 ** -24 * (score * 1.4427 + 16)) - 1
        rows = np.delete(q.reshape(-1, 1, 128).astype(np.float64), [2 * row, 2 * row + 1], 0)
        _, others, _, ew = plain.attend(0, rows, 1, False)
        tol = ew[0] + 2.0 ** -20 * (1 + others[0])
        tol[70] += 2 * off
        others[0, 70] += 2
        assert (np.abs(w - others[0]) <= tol).all(), score
    for x in (2.0 ** 30, 2.0 ** 60, 2.0 ** 120):
        got, w = attend(unit[11] * x, base[1])               # one score far above the others
        assert np.isnan(got[0]).all() and np.array_equal(got[1], clean[row, 1]) and np.isnan(w).all()
    # the page of channel 9 far below the rest: as if it were not there
    stay = np.ones(held, bool)
    stay[64:128] = False
    got, _ = attend(base[0] - unit[9] * 2.0 ** 20, base[1] - unit[9] * 2.0 ** 12)
    cut = PlainCache(1, 1, fmt)
    for side in range(2):
        cut.codes[0][0][side] = plain.codes[0][0][side][stay]
        cut.scales[0][0][side] = np.delete(plain.scales[0][0][side], 1)
    want, _, eo, _ = cut.attend(0, base[None].astype(np.float64), 2, False)
    assert (np.abs(got - want[0]) <= eo[0]).all()
    # every score far below zero
    k[:, 0, :] = 0.0
    k[:, 0, 5] = 2.0 ** 20
    cache.release(0)
    cache.append(dev(k), dev(v), [held])
    cache.prepare([n], append=False)
    q[:, :, :] = 0.0
    clean = cache.attend(dev(q), 2, causal=False).float().cpu().numpy().reshape(n, 2, 128)
    for x in (2.0 ** 30, 2.0 ** 120):
        got, w = attend(unit[5] * -x, unit[5] * 2.0 ** -20)
        assert np.isnan(got[0]).all() and np.isfinite(got[1]).all() and np.isnan(w).all()
