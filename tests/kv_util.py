"""Plain fp64 / Python references of the cache operators (include/specverify.h):
the 4-bit format and its page layout, append, attention, and the page tables.
They share no code with the library."""

import math

import numpy as np

LEVELS = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], np.float64)


def encode(x):
    """x [..., D] float64 -> codes uint8 [..., D], scale bytes uint8 [..., D/32]."""
    b = np.asarray(x, np.float64).reshape(*x.shape[:-1], -1, 32)
    finite = np.isfinite(b).all(-1)
    safe = np.where(finite[..., None], b, 0.0)
    amax = np.abs(safe).max(-1)
    byte = np.ones(amax.shape, np.int64)
    nz = amax > 0
    e = np.zeros(amax.shape, np.int64)
    e[nz] = np.frexp(amax[nz])[1] - 1                       # 2^e <= amax < 2^(e+1)
    fits = np.ldexp(6.0, e - 2) >= amax                     # the smaller of the two candidates
    byte[nz] = (np.where(fits, e - 2, e - 1) + 127)[nz]
    byte = np.clip(byte, 1, 252)
    y = np.abs(np.ldexp(safe, (127 - byte)[..., None]))
    code = np.zeros(y.shape, np.uint8)
    best = np.full(y.shape, np.inf)
    for c in (0, 2, 4, 6, 1, 3, 5, 7):                      # an even code keeps a tie
        gap = np.abs(y - LEVELS[c])
        take = gap < best
        code[take] = c
        best[take] = gap[take]
    code |= np.where(safe < 0, 8, 0).astype(np.uint8)
    byte = np.where(finite, byte, 255)
    code[~finite] = 0
    return code.reshape(x.shape), byte.astype(np.uint8)


def decode(code, byte):
    v = LEVELS[code & 7] * np.where(code & 8, -1.0, 1.0)
    s = np.where(byte == 255, np.nan, np.ldexp(1.0, byte.astype(np.int64) - 127))
    return (v.reshape(*byte.shape, 32) * s[..., None]).reshape(code.shape)


def places(page, d):
    """Byte offsets in a unit: K codes [page, d/2], V codes [page, d/2] (byte c of a token holds
    dims 2c and 2c+1), K scales and V scales [page, d/32]."""
    t = np.arange(page)[:, None]
    c = np.arange(d // 2)[None]
    i = np.arange(d // 32)[None]
    k = t * (d // 2) + c
    per = d // 32                                           # bytes of a 16th of the dims
    v = page * d // 2 + (((t // 8) * 16 + c // per) * 8 + t % 8) * per + c % per
    s = ((t // 8) * (d // 32) + i) * 8 + t % 8
    return k, v, page * d + s, page * d + page * d // 32 + s


def write_token(pages, page, d, page_id, head, t, kcode, kbyte, vcode, vbyte):
    """pages [num_pages, kv_heads, unit] uint8: stores one token of one head."""
    u = pages[page_id, head]
    k, v, ks, vs = places(page, d)
    for at, sat, code, byte in ((k, ks, kcode, kbyte), (v, vs, vcode, vbyte)):
        u[at[t]] = code[0::2] | (code[1::2] << 4)
        u[sat[t]] = byte


def read_unit(unit, page, d):
    """One unit -> K, V float64 [page, d]."""
    out = []
    k, v, ks, vs = places(page, d)
    for at, sat in ((k, ks), (v, vs)):
        b = unit[at]
        code = np.stack([b & 15, b >> 4], -1).reshape(page, d)
        out.append(decode(code, unit[sat]))
    return out


def turned(x, weight, eps, cos_sin, pos, interleaved):
    """Head norm and rotation of [heads, d] at one position, float64."""
    x = np.asarray(x, np.float64)
    d = x.shape[-1]
    if weight is not None:
        x = x / np.sqrt((x * x).sum(-1, keepdims=True) / d + eps) * np.asarray(weight, np.float64)
    if cos_sin is None:
        return x
    rot = cos_sin.shape[1]
    c, s = (np.asarray(a, np.float64) for a in (cos_sin[pos, :rot // 2], cos_sin[pos, rot // 2:]))
    i = np.arange(rot // 2)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    y = x.copy()
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def sees(t, p, window, sinks):
    return (t <= p) & ((window == 0) | (t > p - window) | (t < sinks))


def attention_row(q, k, v, p, scale, window, sinks):
    """One query head at position p over K, V [tokens, d]: the result, the sum of
    weights times |v|, and the largest error fp32 scores can have (see test)."""
    t = np.arange(k.shape[0])
    keep = sees(t, p, window, sinks)
    k, v = k[keep], v[keep]
    with np.errstate(invalid="ignore", over="ignore"):
        s = scale * (k @ q)
        w = np.exp(s - s.max())
        w = w / w.sum()
        out = w @ v
        mass = w @ np.abs(v)
        slip = scale * (np.abs(k) @ np.abs(q)).max()
    return out, mass, slip


class Tables:
    """The page tables as plain Python lists, with the pages' contents as labels."""

    def __init__(self, seqs, width, num_pages, page):
        self.page, self.width = page, width
        self.rows = [[] for _ in range(seqs)]
        self.lens = [0] * seqs
        self.refs = [0] * num_pages

    def pages(self, n):
        return -(-n // self.page)

    def reserve(self, rows):
        """rows per request (None or <= 0: none). Returns (context, status, copies)."""
        free = [p for p, r in enumerate(self.refs) if r == 0]
        shared = [bool(self.rows[b]) and self.lens[b] % self.page != 0
                  and self.refs[self.rows[b][-1]] > 1 for b in range(len(rows))]
        ctx, status, copies, at = [], [], [], 0
        drop = []
        for b, r in enumerate(rows):
            if r <= 0:
                ctx.append(-1)
                status.append(3)
                continue
            want = self.pages(self.lens[b] + r)
            if want > self.width:
                ctx.append(-1)
                status.append(7)
                continue
            need = want - len(self.rows[b]) + shared[b]
            first, at = at, at + need
            if need and at > len(free):
                ctx.append(-1)
                status.append(7)
                continue
            got = free[first:at]
            if shared[b]:
                drop.append(self.rows[b][-1])
                copies.append((self.rows[b][-1], got[0]))
                self.rows[b][-1] = got[0]
                self.rows[b] += got[1:]
            else:
                self.rows[b] += got
            for p in got:
                self.refs[p] = 1
            ctx.append(self.lens[b])
            status.append(0)
            self.lens[b] += r
        for p in drop:
            self.refs[p] -= 1
        return ctx, status, copies

    def release(self, give, ctx=None):
        status = []
        for b, g in enumerate(give):
            if ctx is not None and ctx[b] < 0:
                status.append(0)
                continue
            if g < 0 or g > self.lens[b]:
                status.append(5)
                continue
            self.lens[b] -= g
            keep = self.pages(self.lens[b])
            for p in self.rows[b][keep:]:
                self.refs[p] -= 1
            del self.rows[b][keep:]
            status.append(0)
        return status

    def fork(self, pairs):
        """pairs: (src, dst, length or None)."""
        status = []
        lens = list(self.lens)
        targets = [d for _, d, _ in pairs]
        for i, (s, d, n) in enumerate(pairs):
            ok = (0 <= s < len(lens) and 0 <= d < len(lens) and d not in targets[:i]
                  and s not in targets and lens[d] == 0)
            if ok:
                n = lens[s] if n is None else n
                ok = 0 <= n <= lens[s]
            if ok:
                self.rows[d] = self.rows[s][:self.pages(n)]
                self.lens[d] = n
                for p in self.rows[d]:
                    self.refs[p] += 1
            status.append(0 if ok else 5)
        return status

    def compact(self):
        """Returns (live, moves)."""
        live = sum(1 for r in self.refs if r)
        holes = [p for p in range(live) if self.refs[p] == 0]
        movers = [p for p in range(live, len(self.refs)) if self.refs[p]]
        to = dict(zip(movers, holes))
        for p, q in to.items():
            self.refs[q], self.refs[p] = self.refs[p], 0
        self.rows = [[to.get(p, p) for p in r] for r in self.rows]
        return live, list(to.items())


def log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def fill_unit(unit, page, d, k, v):
    """Stores K, V [page, d] float64 as one whole unit."""
    ka, va, ks, vs = places(page, d)
    for at, sat, x in ((ka, ks, k), (va, vs, v)):
        code, byte = encode(x)
        unit[at] = code[:, 0::2] | (code[:, 1::2] << 4)
        unit[sat] = byte
