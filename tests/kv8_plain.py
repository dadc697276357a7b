"""The 8-bit paged key/value cache from its definition: a plain cache of numpy arrays (float64 arithmetic, the
32-bit steps of the definition taken in float32), attention, key weights and eviction over it, and the error
bounds the kernels are held to.  Shares nothing with the package."""
import numpy as np

PAGE, DIM = 64, 128
FLOOR = np.float32(2.0 ** -100)
INV_QMAX = {0: np.float32(1) / np.float32(127), 1: np.float32(1) / np.float32(448)}


def e4m3(y):
    """float32 values to the nearest E4M3 value (ties to even, saturating), as float32."""
    a = np.minimum(np.abs(y.astype(np.float64)), 448.0)
    _, ex = np.frexp(a)
    step = np.ldexp(1.0, np.maximum(ex - 1, -6) - 3)
    return np.copysign(np.minimum(np.rint(a / step) * step, 448.0), y).astype(np.float32)


def quantise(x, inv, fmt):
    """x float32 -> code values float32."""
    with np.errstate(invalid="ignore", over="ignore"):
        y = np.nan_to_num(x * inv, nan=0.0, posinf=3e38, neginf=-3e38).astype(np.float32)
    return np.clip(np.rint(y), -127, 127).astype(np.float32) if fmt == 0 else e4m3(y)


class PlainCache:
    """codes[b][h][side]: float32 code values [tokens, 128]; scales[b][h][side]: float32 per page."""

    def __init__(self, seqs, heads, fmt):
        self.seqs, self.heads, self.fmt = seqs, heads, fmt
        self.codes = [[[np.zeros((0, DIM), np.float32) for _ in range(2)] for _ in range(heads)] for _ in range(seqs)]
        self.scales = [[[np.zeros(0, np.float32) for _ in range(2)] for _ in range(heads)] for _ in range(seqs)]

    def len(self, b):
        return self.codes[b][0][0].shape[0]

    def append(self, b, k, v):
        """k, v float32 [n, heads, 128]."""
        for h in range(self.heads):
            for side, x in enumerate((k, v)):
                x = x[:, h]
                while x.shape[0]:
                    codes, scales = self.codes[b][h][side], self.scales[b][h][side]
                    at = codes.shape[0]
                    part, x = x[:PAGE - at % PAGE], x[PAGE - at % PAGE:]
                    fin = np.abs(part[np.isfinite(part)])
                    s = np.float32(max(np.float32(fin.max(initial=0.0)) * INV_QMAX[self.fmt], FLOOR))
                    if at % PAGE:
                        old = scales[-1]
                        s = np.float32(max(s, old))
                        if s > old:
                            p0 = at // PAGE * PAGE
                            val = (codes[p0:] * old).astype(np.float32)
                            codes[p0:] = quantise(val, np.float32(1) / s, self.fmt)
                        scales[-1] = s
                    else:
                        scales = np.append(scales, s).astype(np.float32)
                    self.codes[b][h][side] = np.concatenate([codes, quantise(part, np.float32(1) / s, self.fmt)])
                    self.scales[b][h][side] = scales

    def values(self, b, h, side):
        """float64 [tokens, 128]."""
        n = self.len(b)
        s = np.repeat(self.scales[b][h][side].astype(np.float64), PAGE)[:n]
        return self.codes[b][h][side].astype(np.float64) * s[:, None]

    def attend(self, b, q, heads, causal, scale=128 ** -0.5):
        """q float64 [n, heads, 128] -> (o float64 [n, heads, 128], weights float64 [cache heads, tokens], bound of
        |o error|, bound of |weights error|)."""
        n, group, held = q.shape[0], heads // self.heads, self.len(b)
        o = np.zeros((n, heads, DIM))
        w = np.zeros((self.heads, held))
        eo, ew = np.zeros_like(o), np.zeros_like(w)
        if held == 0 or n == 0:
            return o, w, eo, ew
        seen = np.arange(held)[None] <= (held - n + np.arange(n))[:, None] if causal else np.ones((n, held), bool)
        for h in range(heads):
            k, v = self.values(b, h // group, 0), self.values(b, h // group, 1)
            x = q[:, h] @ k.T * scale
            x[~seen] = -np.inf
            top = x.max(axis=1, keepdims=True)
            p = np.exp(x - np.where(np.isfinite(top), top, 0.0))
            z = p.sum(axis=1, keepdims=True)
            p = np.divide(p, z, out=np.zeros_like(p), where=z > 0)
            o[:, h] = p @ v
            w[h // group] += p.sum(axis=0)
            # A score is a float32 sum of 128 exact products: within 128 steps of 2^-23 (a tensor core may cut
            # instead of rounding) of the sum of their magnitudes, and so is its factor; two scores matter to a
            # weight, its own and the row's others'.  2^-20 covers 2^x (2^-22) and log2 of the value scale.
            mag = (np.abs(q[:, h]) @ np.abs(k).T * scale)
            mag = np.where(seen, mag, 0.0).max(axis=1, keepdims=True)
            rel = 2 * 136 * 2.0 ** -23 * mag + 2.0 ** -20
            av = p @ np.abs(v)
            # p is rounded to fp16 (half a step 2^-11 of it; below 2^-14 of the row's largest a step of 2^-24, the
            # value scale inside: at most 2^-25 of the largest |p v| per key), sums of `held` terms, o to bf16
            flush = held * 2.0 ** -25 * 256 * (np.abs(p[:, :, None] * np.abs(v).max(axis=1)[None, :, None]).max(axis=1))
            eo[:, h] = 2.0 ** -8 * np.abs(o[:, h]) + 1.01 * av * (2.0 ** -11 + rel + held * 2.0 ** -23) + flush * 1.01
            ew[h // group] += (p * (rel + n * group * 2.0 ** -23)).sum(axis=0)
        return o, w, eo, ew

    def evict(self, b, weights, keep, recent):
        """weights [heads, >= tokens] -> kept positions per head; the cache holds them afterwards."""
        n = self.len(b)
        if n <= keep:
            kept = [np.arange(n) for _ in range(self.heads)]
        else:
            kept = []
            for h in range(self.heads):
                w = np.asarray(weights[h][:n - recent], np.float64)
                w = np.where(np.isnan(w), -np.inf, w)
                order = sorted(range(n - recent), key=lambda i: (-w[i], i))[:keep - recent]
                kept.append(np.array(sorted(order) + list(range(n - recent, n)), np.int64))
        for h in range(self.heads):
            for side in range(2):
                s = np.repeat(self.scales[b][h][side], PAGE)[:n]
                val = (self.codes[b][h][side] * s[:, None]).astype(np.float32)[kept[h]]
                codes, scales = [], []
                for a in range(0, val.shape[0], PAGE):
                    part = val[a:a + PAGE]
                    sc = np.float32(max(np.abs(part).max(initial=0.0) * INV_QMAX[self.fmt], FLOOR))
                    scales.append(sc)
                    codes.append(quantise(part, np.float32(1) / sc, self.fmt))
                self.codes[b][h][side] = np.concatenate(codes) if codes else np.zeros((0, DIM), np.float32)
                self.scales[b][h][side] = np.array(scales, np.float32)
        return kept
