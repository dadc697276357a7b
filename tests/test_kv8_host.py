"""The 8-bit paged cache on the CPU: the C ABI's refusals (all before the first CUDA call) and the page bookkeeping
of Int8KVCache, its launches replaced by stand-ins."""
import ctypes

import pytest
import torch

import rotated_bit_dit_b200 as R
from rotated_bit_dit_b200 import _binding as B
from rotated_bit_dit_b200 import kvcache as K

FAKE, MIS = 0x10000, 0x10002


def view(**kw):
    c = B.Kv8(FAKE, FAKE, FAKE, 8, 100, 8, 2, 4, 0)
    for n, v in kw.items():
        setattr(c, n, v)
    return c


BAD_VIEWS = [(dict(code_format=2), 1), (dict(pages=0), 1), (dict(heads=0), 1), (dict(heads=1025), 2), (dict(seqs=-1), 1),
             (dict(seqs=65536), 2), (dict(max_pages=0), 1), (dict(ldt=7), 1), (dict(pages=1 << 31), 2),
             (dict(max_pages=1 << 25, ldt=1 << 25), 2), (dict(codes=None), 1), (dict(scales=None), 1), (dict(table=None), 1),
             (dict(codes=0x10008), 3), (dict(scales=0x10004), 3), (dict(table=MIS), 3)]


@pytest.mark.parametrize("bad,status", BAD_VIEWS)
def test_a_bad_cache_is_refused_by_every_entry(bad, status):
    lib, c = R.load(), view(**bad)
    assert lib.rbd_kv8_append(c, FAKE, FAKE, FAKE, 512, FAKE, 512, 4, None) == status
    assert lib.rbd_kv8_read(c, FAKE, 4, FAKE, 512, FAKE, 512, None) == status
    assert lib.rbd_kv8_attn(c, FAKE, FAKE, FAKE, 512, 4, 4, 1, 0.1, 100, FAKE, 512, None, None, 0, 0, FAKE, 1 << 30,
                            None) == status
    assert lib.rbd_kv8_evict(c, FAKE, FAKE, 400, 100, 100, 10, 2, FAKE, 1, FAKE, FAKE, 40, 10, 10, FAKE, None) == status
    assert lib.rbd_kv8_append(None, FAKE, FAKE, FAKE, 512, FAKE, 512, 4, None) == 1


def call(f, names, defaults, **kw):
    args = [kw.pop(n, d) for n, d in zip(names, defaults)]
    assert not kw
    return f(*args)


def test_append_and_read_refusals():
    lib = R.load()
    names = ("c", "lens", "cu", "k", "ldk", "v", "ldv", "rows", "stream")
    base = (view(), FAKE, FAKE, FAKE, 512, FAKE, 512, 4, None)
    f = lambda **kw: call(lib.rbd_kv8_append, names, base, **kw)
    assert f(rows=0, k=None, v=None, lens=None, cu=None) == 0
    assert f(c=view(seqs=0, table=None), k=None) == 0
    assert f(rows=-1) == 1 and f(rows=1 << 29) == 2
    assert f(c=view(heads=5), ldk=640, ldv=640, rows=1 << 28) == 2                    # beyond the grid of pages x heads
    assert f(ldk=504) == 1 and f(ldv=504) == 1 and f(ldk=516) == 3
    for n in ("lens", "cu", "k", "v"):
        assert f(**{n: None}) == 1
        assert f(**{n: MIS}) == 3
    names = ("c", "lens", "tokens", "k", "ldk", "v", "ldv", "stream")
    base = (view(), FAKE, 4, FAKE, 512, FAKE, 512, None)
    f = lambda **kw: call(lib.rbd_kv8_read, names, base, **kw)
    assert f(tokens=0, k=None) == 0 and f(tokens=-1) == 1 and f(tokens=1 << 31) == 2
    assert f(ldk=508) == 1 and f(ldv=516) == 3 and f(lens=None) == 1 and f(k=None) == 1 and f(v=MIS) == 3
    assert f(c=view(seqs=60000, heads=1000), tokens=1 << 30) == 2


def test_attn_refusals_and_workspace():
    lib = R.load()
    names = ("c", "lens", "cu", "q", "ldq", "rows", "q_heads", "causal", "scale", "max_len", "o", "ldo", "w_in", "w_out",
             "w_seq", "w_head", "work", "work_bytes", "stream")
    base = (view(), FAKE, FAKE, FAKE, 1024, 4, 8, 1, 0.1, 512, FAKE, 1024, None, None, 0, 0, FAKE, 1 << 40, None)
    f = lambda **kw: call(lib.rbd_kv8_attn, names, base, **kw)
    assert f(rows=0, q=None, o=None) == 0 and f(c=view(seqs=0)) == 0
    assert f(q_heads=6) == 1 and f(q_heads=0) == 1 and f(rows=-1) == 1 and f(max_len=-1) == 1
    assert f(max_len=513) == 1                                                        # beyond the table
    assert f(rows=1 << 29) == 2
    for s in (0.0, -1.0, float("nan"), float("inf")):
        assert f(scale=s) == 1
    assert f(w_in=FAKE) == 1 and f(w_out=FAKE) == 1                                   # both or neither
    assert f(w_in=FAKE, w_out=FAKE, w_seq=4096, w_head=511) == 1 and f(w_in=FAKE, w_out=FAKE, w_seq=-1, w_head=512) == 1
    assert f(ldq=1000) == 1 and f(ldo=1028) == 3 and f(q=MIS) == 3 and f(o=None) == 1 and f(work=0x10010) == 3
    need = R.rbd_kv8_attn_workspace_bytes(2, 4, 8, 4, 512, True)
    assert need > 0
    assert f(w_in=FAKE, w_out=FAKE, w_seq=4096, w_head=512, work_bytes=need - 1) == 1
    assert f(w_in=FAKE, w_out=FAKE, w_seq=4096, w_head=512, work=None) == 1
    ws = R.rbd_kv8_attn_workspace_bytes
    assert ws(0, 4, 8, 4, 512) == 0
    assert ws(-1, 4, 8, 4, 512) == -1 and ws(2, 0, 8, 4, 512) == -1 and ws(2, 4, 6, 4, 512) == -1
    assert ws(2, 4, 8, 4, 1 << 31) == -1 and ws(70000, 4, 8, 4, 512) == -1
    # the size goes by the call's sizes and is a multiple of 256
    for seqs, rows, length in ((1, 1, 100), (1, 1, 100000), (64, 64, 8192), (3, 3000, 4000), (2, 100, 1 << 20)):
        for weigh in (False, True):
            n = ws(seqs, 4, 8, rows, length, weigh)
            assert n >= 0 and n % 256 == 0


def test_evict_refusals():
    lib = R.load()
    names = ("c", "lens", "weights", "w_seq", "w_head", "width", "keep", "recent", "dst", "ld_dst", "kept", "w_out", "o_seq",
             "o_head", "width_out", "lens_out", "stream")
    base = (view(), FAKE, FAKE, 400, 100, 100, 70, 5, FAKE, 2, FAKE, FAKE, 280, 70, 70, FAKE + 64, None)
    f = lambda **kw: call(lib.rbd_kv8_evict, names, base, **kw)
    assert f(c=view(seqs=0)) == 0
    assert f(keep=0) == 1 and f(recent=-1) == 1 and f(recent=71) == 1 and f(width=0) == 1 and f(width=101) == 1
    assert f(width_out=69) == 1 and f(o_head=69) == 1 and f(ld_dst=1) == 1 and f(lens_out=FAKE) == 1
    assert f(keep=513, ld_dst=9, width_out=513, o_head=513) == 2                      # longer than a sequence can be
    for n in ("lens", "weights", "dst", "kept", "w_out", "lens_out"):
        assert f(**{n: None}) == 1
        assert f(**{n: MIS}) == 3


def test_struct_has_the_headers_layout():
    assert ctypes.sizeof(B.Kv8) == 3 * 8 + 4 * 8 + 2 * 4


@pytest.fixture
def launches(monkeypatch):
    """Int8KVCache on the CPU: launches recorded, with the metadata they would read."""
    calls = []
    monkeypatch.setattr(K.Int8KVCache, "_current", lambda self: 0)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    monkeypatch.setattr(B, "_kv8_append", lambda *a: calls.append("append"))
    monkeypatch.setattr(B, "_kv8_attn", lambda *a: calls.append("attn"))
    monkeypatch.setattr(B, "_kv8_read", lambda *a: calls.append("read"))

    def evict(weights, lens, table, codes, scales, keep, recent, dst, kept, w_out, lens_out, fmt):
        calls.append(("evict", lens.tolist(), keep, recent, dst.tolist()))
    monkeypatch.setattr(B, "rbd_kv8_evict", evict)
    return calls


def check_books(c, pages):
    held = [p for ps in c._pages for p in ps]
    assert len(set(held)) == len(held) and not set(held) & set(c._free)
    assert all(len(p) == -(-n // 64) for p, n in zip(c._pages, c.lens))
    assert c.device_lens.tolist() == c.lens
    for b, p in enumerate(c._pages):
        assert c.table[b, :len(p)].tolist() == p
    return len(held) + len(c._free) == pages


def rows(n, heads=2):
    return torch.zeros((n, heads * 128), dtype=torch.bfloat16)


def test_bookkeeping(launches):
    c = R.Int8KVCache(3, 300, 2, pages=12, device="cpu")
    c.append(rows(70), rows(70), [64, 0, 6])
    assert c.lens == [64, 0, 6] and c.free_pages == 10 and check_books(c, 12)
    assert c._before.tolist() == [0, 0, 0] and c._cu.tolist() == [0, 64, 64, 70]
    c.prepare([1, 1, 1])
    c.append(rows(3), rows(3))
    assert c.attend(rows(3, 4), 4).shape == (3, 512)
    assert c.lens == [65, 1, 7] and c._before.tolist() == [64, 0, 6] and check_books(c, 12)
    c.prepare([5, 0, 2], append=False)
    assert c.lens == [65, 1, 7] and c._cu.tolist() == [0, 5, 5, 7] and c._before.tolist() == [65, 1, 7]
    with pytest.raises(ValueError):
        c.append(rows(7), rows(7))                       # prepared as queries
    c.append(rows(300), rows(300), [200, 50, 50])
    assert c.lens == [265, 51, 57] and c.free_pages == 5 and check_books(c, 12)
    w = torch.zeros(3, 2, 300)
    kept = c.evict(w, 100, 10)
    assert kept.shape == (3, 2, 100) and c.lens == [100, 51, 57] and check_books(c, 12) and c.free_pages == 8
    name, lens, keep, recent, dst = launches[-1]
    assert (name, lens, keep, recent) == ("evict", [265, 51, 57], 100, 10)
    assert [sorted(p for p in d if p >= 0) for d in dst] == [sorted(p) for p in c._pages]
    with pytest.raises(ValueError):
        c.attend(rows(3, 4), 4)                          # prepare() again after an eviction
    c.release(0)
    assert c.lens == [0, 51, 57] and check_books(c, 12) and c.free_pages == 10
    taken = c.spare_pages(2, 3)
    assert taken.shape == (2, 3) and c.free_pages == 4 and not check_books(c, 12)
    for bad in (torch.tensor([c._free[0]]), torch.tensor([c._pages[1][0]]), torch.tensor([12]), torch.tensor([-1]),
                torch.cat([taken[0], taken[0]])):
        with pytest.raises(ValueError):
            c.give_back(bad)
    c.give_back(taken)
    assert c.free_pages == 10 and check_books(c, 12)


def test_refused_calls_change_nothing(launches):
    c = R.Int8KVCache(2, 200, 2, pages=4, device="cpu")
    c.append(rows(100), rows(100), [90, 10])
    state = (c.lens, list(c._free), [list(p) for p in c._pages])
    bad = [lambda: c.append(rows(3), rows(3), [1, 1]), lambda: c.append(rows(2), rows(3), [1, 1]),
           lambda: c.append(rows(2).float(), rows(2), [1, 1]), lambda: c.append(rows(2, 1), rows(2, 1), [1, 1]),
           lambda: c.append(rows(111), rows(111), [111, 0]), lambda: c.append(rows(180), rows(180), [0, 180]),
           lambda: c.append(rows(4)[:, 1:], rows(4), [2, 2]), lambda: c.append(rows(2, 4)[:, ::2], rows(2), [1, 1]),
           lambda: c.prepare([1]), lambda: c.prepare([-1, 1]), lambda: c.prepare([0, 191]),
           lambda: c.evict(torch.zeros(2, 2, 200), 50, 51), lambda: c.evict(torch.zeros(2, 2, 200), 0, 0),
           lambda: c.evict(torch.zeros(2, 2, 80), 50, 10), lambda: c.evict(torch.zeros(2, 2, 300), 201, 10),
           lambda: c.evict(torch.zeros(2, 2, 200), 100, 10),                              # no pages left for it
           lambda: c.release(2), lambda: c.read(0, 80, 11), lambda: c.read(-1), lambda: c.tail(-1),
           lambda: c.spare_pages(0, 1), lambda: c.spare_pages(2, 1)]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
        assert (c.lens, list(c._free), [list(p) for p in c._pages]) == state, i
    c.prepare([1, 1], append=False)
    for f in (lambda: c.attend(rows(3), 2), lambda: c.attend(rows(2, 3), 3), lambda: c.attend(rows(2), 0)):
        with pytest.raises(ValueError):
            f()
    for args in ((0, 10, 1), (1, 0, 1), (1, 10, 0)):
        with pytest.raises(ValueError):
            R.Int8KVCache(*args, device="cpu")
    with pytest.raises(ValueError):
        R.Int8KVCache(1, 10, 1, code_format=7, device="cpu")
    with pytest.raises(ValueError):
        R.Int8KVCache(1, 10, 1, pages=0, device="cpu")


def test_bookkeeping_is_not_captured(launches, monkeypatch):
    c = R.Int8KVCache(2, 200, 2, device="cpu")
    c.prepare([3, 4])
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    c.append(rows(7), rows(7))                           # launches alone
    c.attend(rows(7), 2)
    for f in (lambda: c.prepare([1, 1]), lambda: c.append(rows(7), rows(7), [3, 4]),
              lambda: c.evict(torch.zeros(2, 2, 200), 2, 1), lambda: c.release(0)):
        with pytest.raises(ValueError):
            f()
    assert c.lens == [3, 4]


def test_binding_refuses_shapes_and_devices():
    codes, scales, table = torch.zeros(3, 2, 2, 64, 128, dtype=torch.uint8), torch.ones(3, 2, 2), torch.zeros(1, 3, dtype=torch.int32)
    for bad in (dict(codes=codes.int()), dict(codes=codes[:, :, :1]), dict(scales=scales[:2]), dict(scales=scales.double()),
                dict(table=table.long()), dict(table=table[0]), dict(table=torch.zeros(3, 2, dtype=torch.int32).t()), {}):
        a = dict(table=table, codes=codes, scales=scales, code_format=0, cur=0)
        a.update(bad)
        with pytest.raises(ValueError):                  # the last one: not on a GPU
            B._kv8(**a)
    q = torch.zeros(4, 256, dtype=torch.bfloat16)
    assert B._bf16_rows(q, 256, "q") == 256 and B._bf16_rows(q[:1, :200], 130, "q") == 136
    for bad in (q.float(), q[0], q.t(), q[:, :100]):
        with pytest.raises(ValueError):
            B._bf16_rows(bad, 256, "q")
    w = torch.zeros(2, 3, 50)
    assert B._weights(w, 2, 3, "w") == (150, 50, 50) and B._weights(w[:, :1], 2, 1, "w") == (150, 50, 50)
    for bad in (w.double(), w[0], w[:, :2], w.transpose(1, 2)):
        with pytest.raises(ValueError):
            B._weights(bad, 2, 3, "w")


@pytest.mark.parametrize("weigh", [False, True])
@pytest.mark.parametrize("length", [0, 1, 512, 1 << 20])
@pytest.mark.parametrize("seqs,heads,q_heads", [(1, 1, 1), (2, 4, 8), (65535, 1024, 65536)])
def test_workspace_of_no_rows(seqs, heads, q_heads, length, weigh):
    """A step in which no sequence has a row: nothing is split, scored or imaged."""
    assert R.rbd_kv8_attn_workspace_bytes(seqs, heads, q_heads, 0, length, weigh) == 0


def test_a_step_without_rows(launches):
    c = R.Int8KVCache(3, 300, 2, device="cpu")
    c.append(rows(70), rows(70), [64, 0, 6])
    c.append(rows(0), rows(0), [0, 0, 0])
    assert c.attend(rows(0, 4), 4).shape == (0, 512)
    assert c.attend(rows(0, 4), 4, weights=torch.zeros(3, 2, 300)).shape == (0, 512)
    assert c.lens == [64, 0, 6] and launches == ["append", "append", "attn", "attn"]


def elements(seqs, heads, w_seq, w_head, cols, at=0):
    """Element numbers of weights [seqs, heads, cols] with these strides, `at` elements along."""
    return [at + b * w_seq + h * w_head + t for b in range(seqs) for h in range(heads) for t in range(cols)]


def spans(seqs, heads, w_seq, w_head, cols):
    """One of the strides spans all rows of the other."""
    if seqs == 1 or heads == 1:
        return (seqs == 1 or w_seq >= cols) and (heads == 1 or w_head >= cols)
    return min(w_seq, w_head) >= cols and (w_seq >= (heads - 1) * w_head + cols or w_head >= (seqs - 1) * w_seq + cols)


@pytest.mark.parametrize("seqs,heads", [(1, 1), (1, 3), (3, 1), (3, 2), (2, 4)])
def test_weights_that_share_elements_are_refused(seqs, heads):
    """Attend writes them and evict cuts them from many blocks at once.  (An accepted call comes as far as the
    misaligned pointer.)"""
    lib, cols, base = R.load(), 5, 0x100000
    c = view(seqs=seqs, heads=heads)
    attend = lambda w_in, w_out, w_seq, w_head: lib.rbd_kv8_attn(
        c, FAKE, FAKE, MIS, heads * 128, 4, heads, 1, 0.1, cols, FAKE, heads * 128, base + 4 * w_in, base + 4 * w_out, w_seq,
        w_head, FAKE, 1 << 40, None)
    evict = lambda w, w_seq, w_head, width, w_out, o_seq, o_head, width_out, kept=MIS: lib.rbd_kv8_evict(
        c, FAKE, base + 4 * w, w_seq, w_head, width, 3, 1, FAKE, 1, kept, base + 4 * w_out, o_seq, o_head, width_out, FAKE + 64,
        None)
    strides = sorted({0, 1, cols - 1, cols, cols + 1, 2 * cols, 3 * cols, 4 * cols + 3, 40})
    taken = 0
    for w_seq in strides:
        for w_head in strides:
            if w_head < cols:
                continue
            good = spans(seqs, heads, w_seq, w_head, cols)
            own = elements(seqs, heads, w_seq, w_head, cols)
            assert not good or len(set(own)) == len(own)
            assert attend(0, 0, w_seq, w_head) == (3 if good else 1), (w_seq, w_head)
            assert evict(0, w_seq, w_head, cols, 0, w_seq, w_head, cols) == (3 if good else 1)
            if not good:
                # read from one row for all and written elsewhere is fine
                far = 4000
                assert evict(0, w_seq, w_head, cols, far, 200, 50, cols) == 3
                continue
            taken += 1
            for shift in range(-3 * (w_seq + w_head) - cols, 3 * (w_seq + w_head) + cols + 1):
                other = elements(seqs, heads, w_seq, w_head, cols, shift)
                apart = shift == 0 or not set(own) & set(other)
                assert attend(4000, 4000 + shift, w_seq, w_head) == (3 if apart else 1), (w_seq, w_head, shift)
                if shift and set(own) & set(elements(seqs, heads, w_seq, w_head, 3, shift)):
                    assert evict(4000, w_seq, w_head, cols, 4000 + shift, w_seq, w_head, 3, FAKE) == 1, (w_seq, w_head, shift)
    assert taken > 3
    # in place, but with strides of its own
    if seqs > 1 or heads > 1:
        assert evict(0, 80, 20, cols, 0, 40, 10, cols, FAKE) == 1


def test_append_of_overlapping_rows_changes_nothing(launches):
    """Rows that share memory (expanded, or windows of one buffer) are refused by the entry point: here before the
    lengths and pages move."""
    c = R.Int8KVCache(2, 200, 2, pages=7, device="cpu")
    c.append(rows(100), rows(100), [90, 10])
    state = (c.lens, list(c._free), [list(p) for p in c._pages])
    same, windows = rows(1).expand(3, 256), torch.zeros(1024, dtype=torch.bfloat16).as_strided((3, 256), (248, 1))
    for k, v in ((same, rows(3)), (rows(3), same), (windows, rows(3)), (rows(3), windows)):
        with pytest.raises(ValueError):
            c.append(k, v, [2, 1])
        assert (c.lens, list(c._free), [list(p) for p in c._pages]) == state and check_books(c, 7)
    c.append(same[:1], windows[:1], [1, 0])              # a single row has no stride
    assert c.lens == [91, 10]
