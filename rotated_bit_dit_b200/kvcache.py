"""Key/value caches held in few bits: Int4KVCache (one sequence, a ring) and Int8KVCache (many
sequences, pages, attention in place).

Int4KVCache: a ring of INT4 key (or value) slots driven by rbd_kv4_encode / rbd_kv4_decode.

The cache offers the three operations a serving loop performs on a KV cache -- appending a
slice, evicting the oldest tokens, reading a slice back -- ("lab", Study 6: the serving loop touches the
four-bit cache only through these, so it can stand where a bf16 cache tensor stood).  Only the ring's
bookkeeping lives here; encoding and decoding run in librbd.so.  Token 0 of the cache is the
oldest one held; slots are reused in ring order, so a write never moves existing codes.  Token
slices index it like a tensor: cache[a:b] reads, cache[a:b] = x overwrites, cache[len(cache):] = x
appends.

Int8KVCache: keys and values of many sequences in pages of 64 tokens, 8 bits a value with a scale
per page, head and side (rbd_kv8_append); attention reads the codes themselves (rbd_kv8_attn), can
add up every key's attention weight, and the least used tokens can be evicted (rbd_kv8_evict).  The
page bookkeeping lives here; every arithmetic step runs in librbd.so.
"""
from __future__ import annotations

from typing import List, Optional, Sequence, Tuple

import torch

from . import _binding as B


class Int4KVCache:
    def __init__(self, capacity: int, heads: int, groups_per_band: int = 1, device=None):
        """capacity: token slots; heads: heads of 128 channels per token; groups_per_band 1, 2
        or 4 (3, 6 or 12 scale groups per head)."""
        if capacity <= 0 or heads <= 0:
            raise ValueError("capacity and heads must be positive")
        if groups_per_band not in (1, 2, 4):
            raise ValueError("groups_per_band must be 1, 2 or 4")
        self.capacity, self.heads, self.groups_per_band = capacity, heads, groups_per_band
        dev = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
        self.codes = torch.zeros((capacity, heads, 64), dtype=torch.uint8, device=dev)
        self.scales = torch.zeros((capacity, heads, 3 * groups_per_band), dtype=torch.float32, device=dev)
        self.start = 0   # slot of the oldest token held
        self.size = 0    # tokens held

    def write(self, x: torch.Tensor) -> None:
        """Append the tokens of x (bf16 [T, heads * 128], row stride may be larger).  When the
        ring is full the oldest tokens are evicted first (rolling)."""
        self._check_slice(x)
        t = x.shape[0]
        if t > self.capacity:
            raise ValueError("slice longer than the cache")
        # the ring's bookkeeping moves only once the encode has been accepted: a refused call
        # (bad stride, alignment, device) leaves the held tokens as they were
        overflow = max(self.size + t - self.capacity, 0)
        start = (self.start + overflow) % self.capacity
        size = self.size - overflow
        slot0 = (start + size) % self.capacity
        B.rbd_kv4_encode(x, self.codes, self.scales, self.groups_per_band, slot0)
        self.start, self.size = start, size + t

    def overwrite(self, first: int, x: torch.Tensor) -> None:
        """Re-encode held tokens first .. first + T - 1 (0 = the oldest held) from x (bf16
        [T, heads * 128]); the ring's start and size do not change."""
        self._check_slice(x)
        if first < 0 or first + x.shape[0] > self.size:
            raise ValueError("overwrite outside the tokens held")
        B.rbd_kv4_encode(x, self.codes, self.scales, self.groups_per_band, (self.start + first) % self.capacity)

    def _check_slice(self, x: torch.Tensor) -> None:
        if x.dtype != torch.bfloat16 or x.dim() != 2 or x.shape[1] != self.heads * 128:
            raise ValueError("x must be bf16 [T, heads * 128]")
        if x.device != self.codes.device:
            raise ValueError(f"x is on {x.device}, the cache on {self.codes.device}")

    def __len__(self) -> int:
        return self.size

    def _span(self, key) -> tuple:
        if not isinstance(key, slice):
            raise TypeError("the cache is indexed by token slices")
        a, b, step = key.indices(self.size)
        if step != 1:
            raise ValueError("slices of the cache have step 1")
        return a, max(b - a, 0)

    def __getitem__(self, key) -> torch.Tensor:
        """cache[a:b] decodes tokens a .. b - 1 (Python slice rules, 0 = the oldest held)."""
        a, n = self._span(key)
        return self.read(a, n)

    def __setitem__(self, key, x: torch.Tensor) -> None:
        """cache[a:b] = x re-encodes held tokens a .. b - 1; cache[len(cache):] = x appends (rolling)."""
        if isinstance(key, slice) and key.start == self.size and key.stop is None and key.step is None:
            self.write(x)
            return
        a, n = self._span(key)
        if n != x.shape[0]:
            raise ValueError("slice and x differ in token count")
        self.overwrite(a, x)

    def evict(self, n: int) -> None:
        """Drop the n oldest tokens (their slots are reused by later writes)."""
        if n < 0 or n > self.size:
            raise ValueError("cannot evict more tokens than the cache holds")
        self.start = (self.start + n) % self.capacity
        self.size -= n

    def read(self, first: int = 0, count: Optional[int] = None, out: Optional[torch.Tensor] = None) -> torch.Tensor:
        """Decode tokens first .. first + count - 1 (0 = the oldest held) into out (bf16
        [count, heads * 128]; allocated when not given)."""
        count = self.size - first if count is None else count
        if first < 0 or count < 0 or first + count > self.size:
            raise ValueError("read outside the tokens held")
        if out is None:
            out = torch.empty((count, self.heads * 128), dtype=torch.bfloat16, device=self.codes.device)
        elif out.dtype != torch.bfloat16 or out.dim() != 2 or out.shape[0] < count or out.shape[1] != self.heads * 128:
            raise ValueError("out must be bf16 [>= count, heads * 128]")
        elif out.device != self.codes.device:
            raise ValueError(f"out is on {out.device}, the cache on {self.codes.device}")
        if count:
            slot0 = (self.start + first) % self.capacity
            B.rbd_kv4_decode(self.codes, self.scales, out[:count], self.groups_per_band, slot0)
        return out


class Int8KVCache:
    """A step of a serving loop is

        cache.append(k, v, counts)               # counts[b] new tokens of every sequence
        o = cache.attend(q, heads)               # their queries, causal

    or, to keep the launches apart from the bookkeeping (for a CUDA graph),

        cache.prepare(counts)                    # host: pages, lengths, row offsets
        cache.append(k, v); o = cache.attend(q, heads)      # launches alone: can be captured and replayed

    where a replay follows another prepare() of as many rows in all.  A captured attend keeps the launch
    layout of its capture, laid out for max_tokens: any lengths are right.  The tensors prepare() writes are
    written on the current stream: run prepare and the launches on one stream, or order them."""

    PAGE = 64

    def __init__(self, sequences: int, max_tokens: int, heads: int, pages: Optional[int] = None,
                 code_format: int = B.CODES_INT8, device=None):
        """sequences: slots; max_tokens: tokens a sequence can hold; heads: key/value heads of 128 channels;
        pages: pages of 64 tokens shared by the sequences (by default enough for all of them);
        code_format: CODES_INT8 or CODES_E4M3."""
        if sequences <= 0 or max_tokens <= 0 or heads <= 0:
            raise ValueError("sequences, max_tokens and heads must be positive")
        if code_format not in (B.CODES_INT8, B.CODES_E4M3):
            raise ValueError("code_format must be CODES_INT8 or CODES_E4M3")
        per = -(-max_tokens // self.PAGE)
        pages = sequences * per if pages is None else pages
        if pages <= 0:
            raise ValueError("pages must be positive")
        self.sequences, self.max_tokens, self.heads, self.code_format = sequences, max_tokens, heads, code_format
        dev = torch.device(device) if device is not None else torch.device("cuda")
        if dev.type == "cuda" and dev.index is None:
            dev = torch.device("cuda", torch.cuda.current_device())
        self._device = dev
        self.codes = torch.zeros((pages, heads, 2, self.PAGE, 128), dtype=torch.uint8, device=dev)
        self.scales = torch.ones((pages, heads, 2), dtype=torch.float32, device=dev)
        # one buffer, so that a step's bookkeeping is one copy (of a pageable host mirror, which the runtime has
        # read when the call returns): page table, lengths before and after, row offsets
        n = sequences
        self._host = torch.zeros(n * per + 3 * n + 1, dtype=torch.int32)
        self._meta = torch.zeros(self._host.shape, dtype=torch.int32, device=dev)
        self.table = self._meta[:n * per].view(n, per)
        self._before = self._meta[n * per:n * per + n]
        self.device_lens = self._meta[n * per + n:n * per + 2 * n]    # tokens held, int32 [sequences]
        self._cu = self._meta[n * per + 2 * n:]
        self._pages: List[List[int]] = [[] for _ in range(n)]
        self._free = list(range(pages - 1, -1, -1))
        self._lens = [0] * n
        self._view = B._kv8(self.table, self.codes, self.scales, code_format, dev.index) if dev.type == "cuda" else None
        self._before_at, self._lens_at, self._cu_at = (t.data_ptr() for t in (self._before, self.device_lens, self._cu))
        self._work_bytes = {}        # scratch of an attend by its sizes
        self._rows = None            # rows of the prepared step, None when nothing is prepared
        self._may_append = False

    @property
    def lens(self) -> List[int]:
        """Tokens held by every sequence."""
        return list(self._lens)

    @property
    def free_pages(self) -> int:
        return len(self._free)

    def _set_pages(self, b: int, first: int = 0) -> None:
        """Write entries first .. of sequence b's page list into the host mirror of the table."""
        per = self.table.shape[1]
        if len(self._pages[b]) > first:
            self._host[b * per + first:b * per + len(self._pages[b])] = torch.tensor(self._pages[b][first:],
                                                                                     dtype=torch.int32)

    def _upload(self, before: Sequence[int], counts: Sequence[int]) -> None:
        offsets = [0]
        for c in counts:
            offsets.append(offsets[-1] + c)
        self._host[self.table.numel():] = torch.tensor([*before, *self._lens, *offsets], dtype=torch.int32)
        self._meta.copy_(self._host, non_blocking=True)

    @staticmethod
    def _not_captured() -> None:
        """Bookkeeping is the host's: captured, a replay would repeat this step's."""
        if torch.cuda.is_current_stream_capturing():
            raise ValueError("the cache's bookkeeping cannot be captured: prepare() before the capture and its replays")

    def prepare(self, counts: Sequence[int], append: bool = True) -> None:
        """Make counts[b] rows of every sequence b the subject of the next calls.  append=True: they join the
        cache (their pages are taken and the lengths grow now; append() must follow before attend()).
        append=False: nothing joins, they are the queries of the next attend()."""
        self._not_captured()
        counts = [int(c) for c in counts]
        if len(counts) != self.sequences or any(c < 0 for c in counts):
            raise ValueError("counts must hold a number >= 0 for every sequence")
        before = list(self._lens)
        if append:
            after = [n + c for n, c in zip(before, counts)]
            if max(after) > self.max_tokens:
                raise ValueError("a sequence would exceed max_tokens")
            need = [-(-n // self.PAGE) - len(p) for n, p in zip(after, self._pages)]
            if sum(need) > len(self._free):
                raise ValueError(f"{sum(need)} pages needed, {len(self._free)} free")
            for b, k in enumerate(need):
                if k > 0:
                    self._pages[b] += [self._free.pop() for _ in range(k)]
                    self._set_pages(b, len(self._pages[b]) - k)
            self._lens = after
        self._upload(before, counts)
        self._rows, self._may_append = sum(counts), append

    def _current(self) -> int:
        """The cache's device, which has to be the current one (its kernels run there)."""
        cur = torch.cuda.current_device()
        if self._device.index != cur:
            raise ValueError(f"cache on {self._device} while cuda:{cur} is current")
        return cur

    def _prepared(self, rows: int) -> None:
        if self._rows is None:
            raise ValueError("prepare() first")
        if rows != self._rows:
            raise ValueError(f"{rows} rows given, {self._rows} prepared")

    def append(self, k: torch.Tensor, v: torch.Tensor, counts: Optional[Sequence[int]] = None) -> None:
        """Quantise the prepared tokens' keys and values (bf16 [rows, >= heads*128], the sequences' rows one after
        another) into their pages; with counts, prepare(counts) first."""
        cur = self._current()
        # with counts: everything the call could be refused for, before the bookkeeping moves
        for t in (k, v) if counts is not None else ():
            if t.dtype != torch.bfloat16 or t.dim() != 2 or t.shape[1] < self.heads * 128 or t.stride(1) != 1:
                raise ValueError("k and v must be bf16 [rows, >= heads * 128], rows contiguous")
            if t.device != self._device:
                raise ValueError(f"k or v is on {t.device}, the cache on {self._device}")
            if t.data_ptr() % 16 or (t.shape[0] > 1 and (t.stride(0) % 8 or t.stride(0) < self.heads * 128)):
                raise ValueError("rows of k and v must be 16-byte aligned and must not overlap")
        if counts is not None:
            if k.shape[0] != sum(int(c) for c in counts) or v.shape[0] != k.shape[0]:
                raise ValueError("counts and rows differ")
            self.prepare(counts)
        self._prepared(k.shape[0])
        if not self._may_append:
            raise ValueError("prepared without append")
        B._kv8_append(self._view, cur, self._before_at, self._cu_at, k, v)

    def attend(self, q: torch.Tensor, heads: int, causal: bool = True, out: Optional[torch.Tensor] = None,
               softmax_scale: float = 128 ** -0.5, weights: Optional[torch.Tensor] = None,
               weights_out: Optional[torch.Tensor] = None) -> torch.Tensor:
        """Attention of the prepared rows' queries (bf16 [rows, >= heads*128], heads a multiple of the cache's)
        over the tokens held; causal: a sequence's queries are its last tokens.  A query that sees nothing gets
        zeros, one with an infinite or NaN element NaN.  weights: float32 [sequences, cache heads, >= max_tokens] whose
        rows share no element, to which every key's weight is added (into weights_out when given: of the same strides,
        apart from it).  Returns bf16 [rows, heads*128] (out)."""
        self._prepared(q.shape[0])
        if heads <= 0 or heads % self.heads:
            raise ValueError("heads must be a multiple of the cache's heads")
        if q.device != self._device:
            raise ValueError(f"q is on {q.device}, the cache on {self._device}")
        cur = self._current()
        if out is None:
            out = torch.empty((q.shape[0], heads * 128), dtype=torch.bfloat16, device=self._device)
        if weights_out is None:
            weights_out = weights
        # a capture outlives these lengths: lay it out for any
        longest = self.max_tokens if torch.cuda.is_current_stream_capturing() else max(self._lens)
        sizes = (heads, q.shape[0], longest, weights is not None)
        need = self._work_bytes.get(sizes)
        if need is None:
            if len(self._work_bytes) >= 4096:
                self._work_bytes.clear()
            need = self._work_bytes[sizes] = B.rbd_kv8_attn_workspace_bytes(self.sequences, self.heads, *sizes)
        work = torch.empty((need,), dtype=torch.uint8, device=self._device) if need > 0 else None
        B._kv8_attn(self._view, cur, self._lens_at, self._cu_at, q, out, heads, work, longest, causal, softmax_scale,
                    weights, weights_out)
        return out

    def tail(self, tokens: int) -> Tuple[torch.Tensor, torch.Tensor]:
        """Keys and values of the last `tokens` tokens of every sequence, bf16 [sequences, tokens, heads*128]
        (zeros in front of a sequence's first)."""
        if tokens < 0:
            raise ValueError("tokens must not be negative")
        k = torch.empty((self.sequences, tokens, self.heads * 128), dtype=torch.bfloat16, device=self._device)
        v = torch.empty_like(k)
        B._kv8_read(self._view, self._current(), self._lens_at, k, v)
        return k, v

    def read(self, sequence: int, first: int = 0, count: Optional[int] = None) -> Tuple[torch.Tensor, torch.Tensor]:
        """Keys and values of tokens first .. first + count - 1 of one sequence, bf16 [count, heads*128]."""
        if not 0 <= sequence < self.sequences:
            raise ValueError("no such sequence")
        held = self._lens[sequence]
        count = held - first if count is None else count
        if first < 0 or count < 0 or first + count > held:
            raise ValueError("read outside the tokens held")
        dev = self.codes.device
        k = torch.empty((1, count, self.heads * 128), dtype=torch.bfloat16, device=dev)
        v = torch.empty_like(k)
        if count:
            end = torch.tensor([first + count], dtype=torch.int32).to(dev)
            B.rbd_kv8_read(end, self.table[sequence:sequence + 1], self.codes, self.scales, k, v, self.code_format)
        return k[0], v[0]

    def spare_pages(self, sequences: int, pages: int) -> torch.Tensor:
        """Take sequences * pages free pages out of the pool: int32 [sequences, pages] of their indices, for a caller
        that keeps tokens of its own in them (rbd_kv8_evict's dst_table)."""
        if sequences <= 0 or pages <= 0:
            raise ValueError("sequences and pages must be positive")
        if sequences * pages > len(self._free):
            raise ValueError(f"{sequences * pages} pages needed, {len(self._free)} free")
        taken = [self._free.pop() for _ in range(sequences * pages)]
        return torch.tensor(taken, dtype=torch.int32).view(sequences, pages).to(self._device)

    def give_back(self, pages: torch.Tensor) -> None:
        """Return pages that spare_pages() took to the pool (waits for the device)."""
        back = pages.flatten().tolist()
        held = set(self._free).union(*self._pages)
        if len(set(back)) != len(back) or any(not 0 <= p < self.codes.shape[0] or p in held for p in back):
            raise ValueError("pages that were not taken")
        self._free += reversed(back)

    def evict(self, weights: torch.Tensor, keep: int, recent: int) -> torch.Tensor:
        """Cut every sequence to at most `keep` tokens, per head: its last `recent` tokens and those of largest
        accumulated weight (weights as attend() adds them up; cut to the kept tokens in place, zeros behind).  Needs
        free pages for the kept tokens; the old pages go back to the pool.  Returns int32 [sequences, heads, keep]:
        the positions kept, ascending, then -1.  Afterwards prepare() again."""
        self._not_captured()
        if not 0 <= recent <= keep or keep <= 0:
            raise ValueError("0 <= recent <= keep and keep >= 1 are needed")
        if weights.device != self.codes.device:
            raise ValueError(f"weights are on {weights.device}, the cache on {self.codes.device}")
        if keep > self.max_tokens:
            raise ValueError("keep exceeds max_tokens")
        if weights.dim() != 3 or weights.shape[2] < max(keep, *self._lens):
            raise ValueError("weights must be float32 [sequences, heads, >= tokens held and kept]")
        new = [min(n, keep) for n in self._lens]
        need = [-(-n // self.PAGE) for n in new]
        if sum(need) > len(self._free):
            raise ValueError(f"{sum(need)} pages needed, {len(self._free)} free")
        dev = self.codes.device
        taken = [[self._free[-1 - sum(need[:b]) - i] for i in range(k)] for b, k in enumerate(need)]
        width = -(-keep // self.PAGE)
        dst = torch.tensor([p + [-1] * (width - len(p)) for p in taken], dtype=torch.int32).to(dev)
        kept = torch.empty((self.sequences, self.heads, keep), dtype=torch.int32, device=dev)
        new_lens = torch.empty((self.sequences,), dtype=torch.int32, device=dev)
        B.rbd_kv8_evict(weights, self.device_lens, self.table, self.codes, self.scales, keep, recent, dst, kept, weights,
                        new_lens, self.code_format)
        # the bookkeeping moves only once the call has been accepted
        del self._free[len(self._free) - sum(need):]
        for p in self._pages:
            self._free += reversed(p)
        self._pages, self._lens, self._rows = taken, new, None
        for b in range(self.sequences):
            self._set_pages(b)
        self._upload(new, [0] * self.sequences)
        return kept

    def release(self, sequence: int) -> None:
        """Empty a sequence; its pages go back to the pool.  Weights that attend() added up for it are the caller's to
        clear.  Afterwards prepare() again."""
        self._not_captured()
        if not 0 <= sequence < self.sequences:
            raise ValueError("no such sequence")
        self._free += reversed(self._pages[sequence])
        self._pages[sequence], self._lens[sequence], self._rows = [], 0, None
        self._upload(self._lens, [0] * self.sequences)
