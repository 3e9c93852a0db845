"""The 8-bit paged cache and its head norms in 64 bits, straight from their definitions, with the error bounds that the
kernels' arithmetic allows.  CPU only."""
import torch

import plain_attention as plain

TOP = {torch.int8: 127.0, torch.float8_e4m3fn: 448.0}
LEAST = 2.0 ** -126
E4M3 = torch.float8_e4m3fn


def norm(x, weight, eps):
    """x [tokens, heads, dim] over its root mean square, in 64 bits; and by how much of itself fp32 is off: a sum of up to
    256 squares over 8 fused steps a lane and up to 5 between lanes, its mean, eps, root and reciprocal (halved by the
    root where they lie under it), and two products: 13 / 2 + 2 + 2 roundings of 2^-24, 12 taken."""
    x = x.double()
    if weight is None:
        return x, 0.0
    return x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * weight.double(), 12 * 2.0 ** -24


def heads(x, weight, eps, rows, interleaved):
    """Normed and turned (rows: table rows [tokens, rot] or None), in 64 bits, and the bound of an fp32 result."""
    y, rel = norm(x, weight, eps)
    if rows is None:
        return y, rel * y.abs()
    z, mag = plain.turn(y, rows, interleaved)
    return z, (4 * 2.0 ** -24 + rel) * mag


def half_step(y, dtype):
    """Half the distance of neighbouring codes at y (64 bits, in units of the scale)."""
    if dtype == torch.int8:
        return torch.full_like(y, 0.5)
    return torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6, max=448.0))) - 4)


class Cache:
    """Codes and scales on the CPU, pages in a given order."""

    def __init__(self, lens, capacity, page, block, h, d, dtype, seed=0, spare=2, heads_first=False):
        g = torch.Generator().manual_seed(seed)
        per = max(1, -(-capacity // page))
        n = len(lens) * per + spare
        self.page, self.block, self.dtype = page, block, dtype
        order = torch.randperm(n, generator=g)[:len(lens) * per]
        self.table = order.view(len(lens), per).to(torch.int32)
        self.codes, self.scales = [], []
        for _ in range(2):
            c = torch.randint(-127, 128, (n, page, h, d), generator=g).to(torch.int8)
            if dtype == E4M3:   # no NaN among the codes
                c = (torch.randn(n, page, h, d, generator=g) * 100).clamp(-448, 448).to(E4M3)
            s = torch.rand(n, page // block, h, generator=g) * 0.02 + 1e-3
            self.codes.append(c.transpose(1, 2).contiguous().transpose(1, 2) if heads_first else c)
            self.scales.append(s)

    def device(self):
        """k_cache, v_cache, k_scale, v_scale, page_table, with the same strides."""
        def there(t):
            out = torch.empty_strided(t.shape, t.stride(), dtype=t.dtype, device="cuda")
            out.view(torch.uint8).copy_(t.view(torch.uint8)) if t.element_size() == 1 else out.copy_(t)
            return out
        return [there(t) for t in self.codes + self.scales] + [self.table.cuda()]

    def where(self, b, pos):
        """Page and slot of positions of sequence b."""
        pos = torch.as_tensor(pos)
        return self.table[b].long()[pos // self.page], pos % self.page

    def values(self, side, b, pos):
        """Cached values [positions, heads, dim], the product in 64 bits."""
        page, slot = self.where(b, pos)
        c = self.codes[side].view(torch.uint8)[page, slot].view(self.dtype) if self.dtype == E4M3 else self.codes[side][page, slot]
        return c.float().double() * self.scales[side][page, slot // self.block].double()[..., None]


def check_append(before, after, side, b, x, err, past):
    """The cache's side (0: keys, 1: values) `after` new tokens x [n, heads, dim] (64 bits, fp32's error err) of sequence b
    at positions past .. were put into `before` (Cache objects).  Touched places are marked in after.touched."""
    dt, B, top = before.dtype, before.block, TOP[before.dtype]
    n = x.shape[0]
    if n == 0:
        return
    for first in range(past // B * B, past + n, B):
        new = torch.arange(max(first, past), min(first + B, past + n))
        old = torch.arange(first, max(first, past)) if first < past else torch.arange(0)
        page, slot = before.where(b, [first])
        page, blk = int(page), int(slot) // B
        xs, es = x[new - past], err[new - past]
        want = (xs.abs().amax((0, 2)) / top).clamp(min=LEAST)
        off = es.amax((0, 2)) / top + 2.0 ** -23 * want
        was = before.scales[side][page, blk].double()
        if len(old):
            want = torch.maximum(want, was)
        got = after.scales[side][page, blk].double()
        assert ((got - want).abs() <= off).all(), f"scale of block {first}: {got} for {want}"
        val = after.values(side, b, new)
        y = xs / got[:, None]
        # the product with the reciprocal (two roundings) and x's own error, in units of the scale
        near = half_step(y, dt) * (1 + 2.0 ** -20) + es / got[:, None] + y.abs() * 2.0 ** -22
        # (next to a power of two the steps above are twice as wide)
        if dt == E4M3:
            near = torch.maximum(near, half_step(y * (1 + 2.0 ** -20), dt) * (1 + 2.0 ** -20) + es / got[:, None] + y.abs() * 2.0 ** -22)
        bad = (val / got[:, None] - y).abs() > near
        assert not bad.any(), f"{int(bad.sum())} codes of block {first} off, worst {float(((val / got[:, None] - y).abs() / near).max())}"
        if len(old):
            a, z = before.values(side, b, old), after.values(side, b, old)
            same = got == was
            assert torch.equal(a[:, same], z[:, same])
            y = a / got[:, None]
            near = half_step(y * (1 + 2.0 ** -20), dt) * (1 + 2.0 ** -20) + y.abs() * 2.0 ** -22
            assert ((z / got[:, None] - y).abs() <= near)[:, ~same].all(), f"older codes of block {first}"
        for p in list(old) + list(new):
            after.touched[side].add((page, int(p) % before.page))
        after.blocks[side].add((page, blk))


def check_rest(before, after):
    """Nothing else has changed."""
    for side in (0, 1):
        a, z = (c.codes[side].contiguous().view(torch.uint8) for c in (before, after))
        diff = {(int(p), int(s)) for p, s in (a != z).any(-1).any(-1).nonzero()}
        assert diff <= after.touched[side], f"slots {diff - after.touched[side]} were written"
        diff = {(int(p), int(s)) for p, s in (before.scales[side] != after.scales[side]).any(-1).nonzero()}
        assert diff <= after.blocks[side], f"scales {diff - after.blocks[side]} were written"
