"""The quantised cache's format in 64 bits on the host, and the tests' inputs over it."""

import numpy as np

from tests.scored_reference import Cached

# the numbers of e4m3 codes 0 .. 126, in order: 4 bits of exponent (bias 7), 3 of mantissa
GRID = np.array([(8 + (c & 7)) * 2.0 ** ((c >> 3) - 10) if c >> 3 else (c & 7) * 2.0 ** -9
                 for c in range(127)])
BORDERS = (GRID[1:] + GRID[:-1]) / 2


def quantise(x):
    """(codes, scale bytes) of rows [..., head_dim] by search: the nearest number, ties to the even
    code; the scale is the smallest power of two of -15 .. 8 that leaves no element above 448."""
    x = np.asarray(x, dtype=np.float64)
    top = np.abs(x).max(-1)
    e = np.full(top.shape, -15)
    for k in range(-15, 8):
        e = np.where(top > 448.0 * 2.0 ** k, k + 1, e)
    y = np.minimum(np.abs(x) / 2.0 ** e[..., None], np.where(e == 8, 240.0, 448.0)[..., None])
    low, high = np.searchsorted(BORDERS, y), np.searchsorted(BORDERS, y, side="right")
    code = np.where(low % 2 == 0, low, high)
    return (code + 128 * np.signbit(x)).astype(np.uint8), (e + 127).astype(np.uint8)


def numbers(codes, scales):
    """What rows stand for, in 64 bits; scales has one axis less."""
    c = np.append(GRID, np.nan)[codes & 127]
    return np.where(codes & 128, -c, c) * 2.0 ** (scales.astype(np.float64) - 127)[..., None]


def scale_layout(x):
    """Scales [page][slot][kv_head] as the cache holds them."""
    return np.ascontiguousarray(x.transpose(0, 2, 1))


class QuantCached(Cached):
    """Cached with keys and values that quantised rows stand for (of sizes over a few powers of two).
    A slot that no token lives in holds NaN codes and scale bytes of 255 or 0."""

    def __init__(self, *args, spread=3, **kw):
        super().__init__(*args, **kw)
        rng = np.random.default_rng(kw.get("seed", 0) + 77)
        self.spread = spread
        for name in ("k", "v"):
            x = getattr(self, name)
            live = np.isfinite(x[..., 0])
            size = 2.0 ** -rng.integers(0, spread + 1, live.shape)
            codes, scales = quantise(np.where(live[..., None], x, 0).astype(np.float64)
                                     * size[..., None])
            codes[~live] = 0x7f if name == "k" else 0xff
            scales[~live] = 255 if name == "k" else 0
            setattr(self, name + "_codes", codes)
            setattr(self, name + "_scales", scales)
            setattr(self, name, np.where(live[..., None], numbers(codes, scales), x)
                    .astype(np.float16))

    def forget(self, b, before):
        for t in range(before):
            page, slot = self.bt[b, t // self.ps], t % self.ps
            for name in ("k", "v"):
                getattr(self, name + "_codes")[page, slot] = 0x7f
                getattr(self, name + "_scales")[page, slot] = 255
        super().forget(b, before)

    def to_device(self):
        import torch as t

        from paged_kv_cache_63_gb300 import lib

        put = lambda a: None if a is None else t.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
        d = super().to_device()
        d.update(kc=put(self.cache(self.k_codes)), vc=put(self.cache(self.v_codes)),
                 ks=put(scale_layout(self.k_scales)), vs=put(scale_layout(self.v_scales)))
        d["cache"] = lib.quant_cache(d["kc"], d["vc"], d["ks"], d["vs"])
        return d
