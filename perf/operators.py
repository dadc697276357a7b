"""The 8-bit paged key/value cache as measured workloads.

Four operators: `append` (tokens quantised into the cache, one scale per page of 64 tokens, head and
side), `attend` (attention over the cache, grouped query heads, causal or full), `weigh` (the same
attention, adding every key's attention weight to a running sum) and `evict` (the tokens of largest
accumulated weight and the most recent ones kept, per head, in fresh pages).

A module attribute `own` selects between elementary torch operations (False) and the package's kernels
(True).  `listed` and `draw` give cases, `prepare` makes what a program holds before a call, `run` is one
call, `exact` its result in 64 bits, `work` the bytes and operations it cannot do without.

Definition of the cache.  A page holds 64 consecutive tokens; per (page, head, key or value) the scale is
    s = max(amax / qmax, 2^-100),  qmax = 127 (INT8) or 448 (E4M3),
and a code is round(x / s), formed as x * (1 / s) in 32 bits.  Tokens that join a partly filled page make
its scale max(old scale, own scale), the older codes being requantised from the values they stand for.
"""
import math

import torch

own = False

PAGE = 64
DIM = 128
FLOOR = 2.0 ** -100


# ---------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # one more token for each of 64 running conversations
        dict(name="append_tokens", op="append", fmt="int8", seqs=64, heads=8, old=4096, new=1, ragged=True),
        # ragged prompts joining caches that hold a shared preamble already
        dict(name="append_prompts", op="append", fmt="e4m3", seqs=16, heads=12, old=100, new=2500, ragged=True),
        # one request, one token: latency
        dict(name="token_single", op="attend", fmt="int8", seqs=1, heads=24, group=1, held=1000, new=1,
             causal=True, ragged=False),
        # a full serving batch, grouped heads
        dict(name="token_batch", op="attend", fmt="int8", seqs=64, heads=12, group=4, held=8192, new=1,
             causal=True, ragged=True),
        # few requests over very long caches
        dict(name="token_long", op="attend", fmt="e4m3", seqs=3, heads=8, group=4, held=120001, new=1,
             causal=True, ragged=True),
        # several drafted tokens checked at once
        dict(name="draft_batch", op="attend", fmt="int8", seqs=24, heads=8, group=5, held=3000, new=6,
             causal=True, ragged=True),
        # a block of image tokens over a cache of earlier ones, no mask inside the block
        dict(name="image_block", op="attend", fmt="int8", seqs=1, heads=24, group=1, held=16384, new=4096,
             causal=False, ragged=False),
        # ragged prompts, causal, grouped heads
        dict(name="prompt_ragged", op="attend", fmt="e4m3", seqs=8, heads=12, group=4, held=4000, new=4000,
             causal=True, ragged=True),
        # single tokens that also feed the weights an eviction ranks by
        dict(name="weigh_tokens", op="weigh", fmt="int8", seqs=16, heads=12, group=4, held=8000, new=1,
             causal=True, ragged=True),
        # a prompt whose keys are ranked
        dict(name="weigh_prompt", op="weigh", fmt="int8", seqs=2, heads=12, group=4, held=3001, new=3001,
             causal=True, ragged=True),
        # a small cache trimmed often
        dict(name="evict_small", op="evict", fmt="int8", seqs=4, heads=8, held=1100, keep=1000, recent=100,
             ragged=True),
        # long caches cut to a quarter
        dict(name="evict_long", op="evict", fmt="e4m3", seqs=16, heads=12, held=16384, keep=4096, recent=511,
             ragged=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "append", "attend", "attend", "attend", "attend", "weigh", "weigh", "evict", "evict"])
    case = dict(op=op, fmt=rng.choice(["int8", "e4m3"]), ragged=rng.random() < 0.75)
    case["heads"] = rng.choice([1, 2, 3, 5, 8, 12, 24])
    if op == "append":
        case["new"] = 1 if rng.random() < 0.4 else _log_int(rng, 2, 2500)
        case["old"] = rng.choice([0, _log_int(rng, 1, 4096)])
        case["seqs"] = _log_int(rng, 1, max(1, min(64, 12 * 2500 * 12 // (case["new"] * case["heads"]))))
    elif op == "evict":
        case["held"] = _log_int(rng, 40, 16384)
        case["keep"] = _log_int(rng, 16, max(16, case["held"] // 3))
        case["recent"] = rng.randint(0, case["keep"])
        case["seqs"] = _log_int(rng, 1, max(1, min(64, 8 * 12 * 16384 // (case["held"] * case["heads"]))))
    else:
        case["group"] = rng.choice([1, 1, 2, 3, 4, 5, 8])
        case["causal"] = rng.random() < 0.7
        kind = rng.choice(["token", "token", "draft", "block"])
        if kind == "block":
            case["new"] = _log_int(rng, 17, 4000)
            case["held"] = case["new"] + rng.choice([0, _log_int(rng, 1, 12000)])
        else:
            case["new"] = 1 if kind == "token" else rng.randint(2, 16)
            case["held"] = case["new"] + _log_int(rng, 1, 60000)
        pairs = 5 * 12 * 4 * 4000 * 4000 // 2
        flops = case["new"] * case["held"] * case["heads"] * case["group"]
        tokens = 64 * 12 * 8192 // 3 // (case["held"] * case["heads"])
        rows = 800000 // (case["new"] * case["heads"] * case["group"])
        case["seqs"] = _log_int(rng, 1, max(1, min(64, pairs // flops, tokens, rows)))
    return case


# ---------------------------------------------------------------------------------------------- inputs
def _gen(seed, salt):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1000003 + salt)
    return g


def _spread(case, top, salt, low=1):
    """One length per sequence: `top` for all, or ragged between about a tenth of it and it (the first
    sequence has `top`).  The lengths belong to the case; only values come from a seed."""
    n = case["seqs"]
    if not case["ragged"] or top <= low:
        return [top] * n
    g = torch.Generator()
    g.manual_seed(7919 * top + 31 * n + salt)
    out = [max(low, int(top * (0.1 + 0.9 * float(v)))) for v in torch.rand(n, generator=g)]
    out[0] = top
    return out


def _keys_values(rows, heads, seed, salt):
    """Keys with a few strong channels per head, values with a few strong tokens (bf16 [rows, heads * 128])."""
    g = _gen(seed, salt)
    gain = torch.ones(heads, DIM, device="cuda")
    strong = torch.randint(0, DIM, (heads, 4), generator=g, device="cuda")
    gain.scatter_(1, strong, 4.0)
    k = torch.randn(rows, heads, DIM, generator=g, device="cuda") * gain
    v = torch.randn(rows, heads, DIM, generator=g, device="cuda")
    v *= 1.0 + 4.0 * (torch.rand(rows, heads, 1, generator=g, device="cuda") < 0.01)
    return k.reshape(rows, heads * DIM).bfloat16(), v.reshape(rows, heads * DIM).bfloat16()


def _queries(rows, heads, seed, salt):
    return (torch.randn(rows, heads * DIM, generator=_gen(seed, salt), device="cuda") * 1.5).bfloat16()


def _lengths(case):
    """(tokens held when the call runs, tokens of the call) of every sequence."""
    if case["op"] == "append":
        return _spread(case, case["old"], 1, 0), _spread(case, case["new"], 2)
    if case["op"] == "evict":
        return _spread(case, case["held"], 1), []
    new = _spread(case, case["new"], 2)
    if case["held"] == case["new"]:
        return new, new
    held = _spread(case, case["held"] - case["new"], 1)
    return [a + b for a, b in zip(held, new)], new


def _inputs(case, seed):
    held, new = _lengths(case)
    k, v = _keys_values(sum(held), case["heads"], seed, 3)
    d = dict(held=held, new=new, k=k, v=v)
    if case["op"] == "append":
        d["xk"], d["xv"] = _keys_values(sum(new), case["heads"], seed, 4)
    elif case["op"] in ("attend", "weigh"):
        d["q"] = _queries(sum(new), case["heads"] * case["group"], seed, 5)
    if case["op"] in ("weigh", "evict"):
        g = _gen(seed, 6)
        w = torch.exp(2.0 * torch.randn(len(held), case["heads"], max(held), generator=g, device="cuda"))
        w *= torch.rand(w.shape, generator=g, device="cuda") > 0.1       # keys nobody looked at yet: equal weights
        d["weights"] = w
    return d


# ---------------------------------------------------------------------------------------------- plain form
def _qmax(fmt):
    return 127.0 if fmt == "int8" else 448.0


def _encode(x, inv, fmt):
    """Codes of float32 x, held in one byte."""
    y = x * inv
    if fmt == "int8":
        return torch.round(y).clamp_(-127, 127).to(torch.int8).view(torch.uint8)
    return y.clamp_(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)


def _decode(codes, fmt):
    return codes.view(torch.int8 if fmt == "int8" else torch.float8_e4m3fn).float()


def _scale(amax, fmt):
    return (amax / _qmax(fmt)).clamp_min(FLOOR)


def _paged(x, lens, heads, pages):
    """Packed rows [sum, heads * 128] as float32 [seqs, heads, pages * 64, 128], zeros behind the end."""
    out = torch.zeros(len(lens), pages * PAGE, heads, DIM, device=x.device)
    r = 0
    for b, n in enumerate(lens):
        out[b, :n] = x[r:r + n].reshape(n, heads, DIM).float()
        r += n
    return out.permute(0, 2, 1, 3)


def _plain_cache(x, lens, heads, pages, fmt):
    codes, scales = [], []
    r = 0
    for n in lens:          # one sequence at a time: the 32-bit copy is many times the codes
        p = _paged(x[r:r + n], [n], heads, pages).reshape(heads, pages, PAGE, DIM)
        r += n
        s = _scale(p.abs().amax(dim=(2, 3)), fmt)
        codes.append(_encode(p, (1.0 / s)[:, :, None, None], fmt).reshape(heads, pages * PAGE, DIM))
        scales.append(s)
    return torch.stack(codes), torch.stack(scales)


def _plain_append(state):
    case, fmt, heads = state["case"], state["case"]["fmt"], state["case"]["heads"]
    lens, cu = state["lens"], state["cu"]
    first = lens // PAGE                                            # first page touched
    span = state["span"]                                            # pages touched, at most
    tok = first[:, None] * PAGE + torch.arange(span * PAGE, device="cuda")[None]
    is_old = tok < lens[:, None]
    is_new = ~is_old & (tok < state["after"][:, None])
    row = (cu[:-1, None] + tok - lens[:, None]).clamp(0, cu[-1] - 1)
    page = (first[:, None] + torch.arange(span, device="cuda")[None])
    had = page * PAGE < lens[:, None]
    kept_pages = state["codes"][0].shape[2] // PAGE
    pidx = page.clamp_max(kept_pages - 1)
    out = []
    for side, x in enumerate((state["xk"], state["xv"])):
        codes, scales = state["codes"][side], state["scales"][side]
        fresh = x[row].reshape(len(lens), span, PAGE, heads, DIM).permute(0, 3, 1, 2, 4).float()
        new4 = is_new.reshape(len(lens), 1, span, PAGE, 1)
        fresh = torch.where(new4, fresh, 0.0)
        hidx = torch.arange(heads, device="cuda")[None, :, None]
        bidx = torch.arange(len(lens), device="cuda")[:, None, None]
        blocks = codes.reshape(len(lens), heads, kept_pages, PAGE, DIM)
        old_s = torch.where(had[:, None, :], scales[bidx, hidx, pidx[:, None, :]], FLOOR)
        s = torch.maximum(_scale(fresh.abs().amax(dim=(3, 4)), fmt), old_s)
        old_c = blocks[bidx, hidx, pidx[:, None, :]]
        val = torch.where(is_old.reshape(new4.shape), _decode(old_c, fmt) * old_s[..., None, None], fresh)
        enc = _encode(val, (1.0 / s)[..., None, None], fmt)
        live = (page * PAGE < state["after"][:, None])
        bi, pi = live.nonzero(as_tuple=True)
        blocks[bi, :, page[bi, pi]] = enc[bi, :, pi]
        scales[bi, :, page[bi, pi]] = s[bi, :, pi]
        out.append(_plain_tail(codes, scales, state["after"], state["tail"], fmt))
    return tuple(out)


def _plain_tail(codes, scales, lens, tokens, fmt):
    """Values of the last `tokens` tokens of every sequence, bf16 [seqs, tokens, heads * 128] (zeros before
    a sequence's first)."""
    n, heads = codes.shape[:2]
    tok = lens[:, None] - tokens + torch.arange(tokens, device="cuda")[None]
    ok = (tok >= 0)[:, None, :, None]
    t = tok.clamp_min(0)[:, None, :]
    b = torch.arange(n, device="cuda")[:, None, None]
    h = torch.arange(heads, device="cuda")[None, :, None]
    val = _decode(codes[b, h, t], fmt) * scales[b, h, t // PAGE][..., None]
    return torch.where(ok, val, 0.0).bfloat16().permute(0, 2, 1, 3).reshape(n, tokens, heads * DIM)


def _plain_attend(state):
    case, fmt = state["case"], state["case"]["fmt"]
    heads, group = case["heads"], case["group"]
    o = torch.empty_like(state["q"])
    weighs = case["op"] == "weigh"
    w_out = state["weights"].clone() if weighs else None
    r = 0
    for b, (n_all, n) in enumerate(zip(state["held"], state["new"])):
        q = state["q"][r:r + n].reshape(n, heads, group, DIM).float()
        mask = None
        if case["causal"]:
            at = n_all - n + torch.arange(n, device="cuda")
            mask = torch.arange(n_all, device="cuda")[None] > at[:, None]
        step = max(1, (1 << 28) // (n * group * n_all))              # heads at a time
        for h0 in range(0, heads, step):
            h1 = min(heads, h0 + step)
            s_of = torch.arange(n_all, device="cuda") // PAGE
            k = _decode(state["codes"][0][b, h0:h1, :n_all], fmt) * state["scales"][0][b, h0:h1][:, s_of, None]
            v = _decode(state["codes"][1][b, h0:h1, :n_all], fmt) * state["scales"][1][b, h0:h1][:, s_of, None]
            qh = q[:, h0:h1].permute(1, 2, 0, 3).reshape(h1 - h0, group * n, DIM)
            sc = (qh @ k.transpose(1, 2)).reshape(h1 - h0, group, n, n_all) * (1.0 / math.sqrt(DIM))
            if mask is not None:
                sc = sc.masked_fill_(mask, float("-inf"))
            p = torch.exp(sc - sc.amax(dim=-1, keepdim=True))
            p /= p.sum(dim=-1, keepdim=True)
            if weighs:
                w_out[b, h0:h1, :n_all] += p.sum(dim=(1, 2))
            y = (p.reshape(h1 - h0, group * n, n_all) @ v).reshape(h1 - h0, group, n, DIM)
            o.view(-1, heads, group, DIM)[r:r + n, h0:h1] = y.permute(2, 0, 1, 3).bfloat16()
        r += n
    return (o, w_out) if weighs else o


def _plain_evict(state):
    case, fmt = state["case"], state["case"]["fmt"]
    keep, recent, heads = case["keep"], case["recent"], case["heads"]
    pages = -(-keep // PAGE)
    n_seq = len(state["held"])
    kept = torch.full((n_seq, heads, keep), -1, dtype=torch.int32, device="cuda")
    w_out = torch.zeros(n_seq, heads, keep, device="cuda")
    vals = [torch.zeros(n_seq, keep, heads, DIM, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    for b, n in enumerate(state["held"]):
        m = min(n, keep)
        w = state["weights"][b, :, :n]
        if n > keep:
            order = torch.sort(w[:, :n - recent], dim=1, descending=True, stable=True).indices
            chosen = torch.sort(order[:, :keep - recent], dim=1).values
            last = torch.arange(n - recent, n, device="cuda").expand(heads, recent)
            idx = torch.cat([chosen, last], dim=1)
        else:
            idx = torch.arange(n, device="cuda").expand(heads, n)
        kept[b, :, :m] = idx
        w_out[b, :, :m] = torch.gather(w, 1, idx)
        for side in range(2):
            h = torch.arange(heads, device="cuda")[:, None]
            val = _decode(state["codes"][side][b][h, idx], fmt) * state["scales"][side][b][h, idx // PAGE][..., None]
            full = torch.zeros(heads, pages * PAGE, DIM, device="cuda")
            full[:, :m] = val
            full = full.reshape(heads, pages, PAGE, DIM)
            s = _scale(full.abs().amax(dim=(2, 3)), fmt)[:, :, None, None]
            new = (_decode(_encode(full, 1.0 / s, fmt), fmt) * s).reshape(heads, pages * PAGE, DIM)[:, :m]
            vals[side][b, keep - m:] = new.permute(1, 0, 2).bfloat16()
    return (kept, w_out) + tuple(v.reshape(n_seq, keep, heads * DIM) for v in vals)


# ---------------------------------------------------------------------------------------------- prepare / run
def _offsets(counts):
    cu = [0]
    for c in counts:
        cu.append(cu[-1] + c)
    return torch.tensor(cu, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    d = _inputs(case, seed)
    held, new, heads, fmt = d["held"], d["new"], case["heads"], case["fmt"]
    state = dict(case=case, held=held, new=new)
    after = [a + b for a, b in zip(held, new)] if case["op"] == "append" else held
    pages = -(-max(after) // PAGE)
    for name in ("q", "xk", "xv", "weights"):
        if name in d:
            state[name] = d[name]
    if case["op"] == "append":
        state["tail"] = max(new) + PAGE - 1
    if not own:
        kv = [_plain_cache(x, held, heads, pages, fmt) for x in (d["k"], d["v"])]
        state["codes"], state["scales"] = [c for c, _ in kv], [s for _, s in kv]
        if case["op"] == "append":
            state["lens"] = torch.tensor(held, device="cuda")
            state["after"] = torch.tensor(after, device="cuda")
            state["cu"] = _offsets(new).long()
            state["span"] = max(-(-b // PAGE) - a // PAGE for a, b in zip(held, after))
        return state

    import rotated_bit_dit_b200 as R
    code_format = R.CODES_INT8 if fmt == "int8" else R.CODES_E4M3
    spare = len(held) * -(-case["keep"] // PAGE) if case["op"] == "evict" else 0
    total = sum(-(-n // PAGE) for n in after) + spare
    cache = R.Int8KVCache(len(held), pages * PAGE, heads, pages=total, code_format=code_format)
    cache.append(d["k"], d["v"], held)
    if case["op"] == "append":
        cache.prepare(new)
    elif case["op"] == "evict":
        state["dst"] = cache.spare_pages(len(held), -(-case["keep"] // PAGE))
        state["kept_lens"] = torch.empty(len(held), dtype=torch.int32, device="cuda")
    else:
        cache.prepare(new, append=False)
    if "weights" in state:
        w = torch.zeros(len(held), heads, pages * PAGE, device="cuda")
        w[:, :, :state["weights"].shape[2]] = state["weights"]
        state["weights"] = w
        state["weights_out"] = w.clone()
    state["cache"] = cache
    return state


def run(state):
    case, op = state["case"], state["case"]["op"]
    if not own:
        if op == "append":
            return _plain_append(state)
        return _plain_evict(state) if op == "evict" else _plain_attend(state)
    import rotated_bit_dit_b200 as R
    cache = state["cache"]
    if op == "append":
        cache.append(state["xk"], state["xv"])
        return cache.tail(state["tail"])
    heads = case["heads"] * case.get("group", 1)
    if op == "attend":
        return cache.attend(state["q"], heads, causal=case["causal"])
    if op == "weigh":
        o = cache.attend(state["q"], heads, causal=case["causal"], weights=state["weights"],
                         weights_out=state["weights_out"])
        return o, state["weights_out"][:, :, :max(state["held"])]
    n, keep = len(state["held"]), case["keep"]
    kept = torch.empty(n, case["heads"], keep, dtype=torch.int32, device="cuda")
    w_out = torch.empty(n, case["heads"], keep, device="cuda")
    R.rbd_kv8_evict(state["weights"], cache.device_lens, cache.table, cache.codes, cache.scales, keep, case["recent"],
                    state["dst"], kept, w_out, state["kept_lens"], cache.code_format)
    k = torch.empty(n, keep, case["heads"] * DIM, dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    R.rbd_kv8_read(state["kept_lens"], state["dst"], cache.codes, cache.scales, k, v, cache.code_format)
    return kept, w_out, k, v


# ---------------------------------------------------------------------------------------------- exact
def _e4m3_64(y):
    """float64 to the nearest E4M3 value, ties to even, saturating."""
    a = y.abs().clamp_max(448.0)
    _, e = torch.frexp(a)
    step = torch.ldexp(torch.ones_like(a), (e - 1).clamp_min(-6) - 3)
    return torch.copysign((torch.round(a / step) * step).clamp_max(448.0), y)


def _quantise64(x, fmt, s_old=None):
    """x float64 [..., tokens, 128] of ONE page -> (code values, scale) in float64.  The scale and the number that
    is rounded to a code are 32-bit by definition, so that a code is one certain whole number or E4M3 value."""
    top = 127.0 if fmt == "int8" else 448.0
    s = (x.abs().amax(dim=(-2, -1)).float() / top).clamp_min(FLOOR)
    if s_old is not None:
        s = torch.maximum(s, s_old.float())
    y = (x.float() * (1.0 / s)[..., None, None]).double()
    s = s.double()
    return (torch.round(y).clamp(-top, top) if fmt == "int8" else _e4m3_64(y)), s


def _pages64(x, heads, fmt):
    """Packed rows of one sequence -> list of (code values, scale) per page, heads leading."""
    y = x.double().reshape(x.shape[0], heads, DIM).transpose(0, 1)
    return [_quantise64(y[:, a:a + PAGE], fmt) for a in range(0, y.shape[1], PAGE)]


def _values64(pages, heads):
    if not pages:
        return torch.zeros(heads, 0, DIM, dtype=torch.float64, device="cuda")
    return torch.cat([c * s[:, None, None] for c, s in pages], dim=1)


def exact(case, seed):
    if case["op"] in ("attend", "weigh"):
        held, new = _lengths(case)
        pairs = sum(a * b for a, b in zip(held, new)) * case["heads"] * case["group"]
        if pairs > 3e10 or sum(held) * case["heads"] > 2e7:
            return None
    d = _inputs(case, seed)
    held, new, heads, fmt = d["held"], d["new"], case["heads"], case["fmt"]
    starts = [sum(held[:b]) for b in range(len(held))]
    if case["op"] == "append":
        tail = max(new) + PAGE - 1
        outs = []
        for x0, x1 in ((d["k"], d["xk"]), (d["v"], d["xv"])):
            res = torch.zeros(len(held), tail, heads, DIM, dtype=torch.float64, device="cuda")
            r = 0
            for b, (n0, n1) in enumerate(zip(held, new)):
                pages = _pages64(x0[starts[b]:starts[b] + n0], heads, fmt)
                fresh = x1[r:r + n1].double().reshape(n1, heads, DIM).transpose(0, 1)
                r += n1
                if n0 % PAGE:
                    c, s = pages.pop()
                    part, fresh = fresh[:, :PAGE - n0 % PAGE], fresh[:, PAGE - n0 % PAGE:]
                    _, grown = _quantise64(part, fmt, s)
                    pages.append(_quantise64(torch.cat([c * s[:, None, None], part], dim=1), fmt, grown))
                pages += [_quantise64(fresh[:, a:a + PAGE], fmt) for a in range(0, fresh.shape[1], PAGE)]
                need = -(-tail // PAGE) + 1
                val = _values64(pages[-need:], heads)[:, -tail:].transpose(0, 1)
                res[b, tail - val.shape[0]:] = val
            outs.append(res.reshape(len(held), tail, heads * DIM))
        return tuple(outs)
    if case["op"] == "evict":
        keep, recent = case["keep"], case["recent"]
        kept = torch.full((len(held), heads, keep), -1, dtype=torch.int32, device="cuda")
        w_out = torch.zeros(len(held), heads, keep, dtype=torch.float64, device="cuda")
        vals = [torch.zeros(len(held), keep, heads, DIM, dtype=torch.float64, device="cuda") for _ in range(2)]
        for b, n in enumerate(held):
            m = min(n, keep)
            w = d["weights"][b, :, :n].double()
            rank = torch.zeros(heads, n, device="cuda", dtype=torch.float64)
            rank[:] = w
            rank[:, n - min(recent, n):] = float("inf")
            idx = torch.argsort(-rank, dim=1, stable=True)[:, :m].sort(dim=1).values
            kept[b, :, :m] = idx.int()
            w_out[b, :, :m] = w.gather(1, idx)
            for side, x in enumerate((d["k"], d["v"])):
                all64 = _values64(_pages64(x[starts[b]:starts[b] + n], heads, fmt), heads)
                sel = all64.gather(1, idx[:, :, None].expand(-1, -1, DIM))
                new64 = _values64([_quantise64(sel[:, a:a + PAGE], fmt) for a in range(0, m, PAGE)], heads)
                vals[side][b, keep - m:] = new64.transpose(0, 1)
        return (kept, w_out) + tuple(v.reshape(len(held), keep, heads * DIM) for v in vals)
    group = case["group"]
    o = torch.zeros(sum(new), heads, group, DIM, dtype=torch.float64, device="cuda")
    w_out = d["weights"].double() if case["op"] == "weigh" else None
    r = 0
    for b, (n_all, n) in enumerate(zip(held, new)):
        k = _values64(_pages64(d["k"][starts[b]:starts[b] + n_all], heads, fmt), heads)
        v = _values64(_pages64(d["v"][starts[b]:starts[b] + n_all], heads, fmt), heads)
        q = d["q"][r:r + n].double().reshape(n, heads, group, DIM)
        block = max(1, 2 ** 27 // (group * n_all))                  # query tokens at a time
        for h in range(heads):
            for a in range(0, n, block):
                z = min(n, a + block)
                logit = torch.einsum("igd,td->igt", q[a:z, h], k[h]) / math.sqrt(DIM)
                if case["causal"]:
                    last = n_all - n + torch.arange(a, z, device="cuda")
                    hidden = torch.arange(n_all, device="cuda")[None, None] > last[:, None, None]
                    logit = logit.masked_fill(hidden, float("-inf"))
                p = torch.softmax(logit, dim=-1)
                o[r + a:r + z, h] = torch.einsum("igt,td->igd", p, v[h])
                if w_out is not None:
                    w_out[b, h, :n_all] += p.sum(dim=(0, 1))
        r += n
    o = o.reshape(sum(new), heads * group * DIM)
    return o if w_out is None else (o, w_out)


# ---------------------------------------------------------------------------------------------- work
def work(case):
    """Bytes read once and written once, and operations, of one pass."""
    held, new = _lengths(case)
    heads = case["heads"]
    row = 2 * heads * DIM                                            # elements of one token, keys and values
    if case["op"] == "append":
        back = sum(min(max(new) + PAGE - 1, a + b) for a, b in zip(held, new))
        # bf16 in, codes out; the tail's codes in, bf16 out
        return dict(bytes=row * (3 * sum(new) + 3 * back - sum(new)), flops=row * (3 * sum(new) + back))
    if case["op"] == "evict":
        kept = sum(min(n, case["keep"]) for n in held)
        # weights in, indices and weights out; codes in and out, bf16 out
        return dict(bytes=4 * heads * sum(held) + 8 * heads * kept + 4 * kept * row,
                    flops=heads * sum(held) + 4 * kept * row)
    q_heads = heads * case["group"]
    pairs = sum(m * n - (n * (n - 1) // 2 if case["causal"] else 0) for m, n in zip(held, new))
    size = sum(held) * row + 4 * sum(new) * q_heads * DIM
    if case["op"] == "weigh":
        size += 8 * sum(held) * heads
    return dict(bytes=size, flops=4 * pairs * q_heads * DIM)
