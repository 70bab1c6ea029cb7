"""What the tests of window attention's gradients share: inputs, the bars, and a comparison that allows nothing beside them.

dq and dk are compared with the definition in 64 bits with D = do . o from the o that the backward was given, so that what o's own
rounding moves them by (which include/window.h states) is in the reference and not in the tolerance.  What is left, per
element of a gradient:
  * bf16: the output's rounding and that of dx (dv: of p) where it enters a product, each up to 2^-8 of a value and 1.7e-3 root-mean-square:
    2.4e-3 where the terms are independent, up to 2.9e-3 where terms that cancel (sum_s dx = 0) leave their roundings standing: 2^-8;
  * fp32: sums of up to 128 products and over some hundred keys, a handful of roundings of 2^-24: 1e-5.
Single rows are held to four times the bar, their norms floored at a tenth of the rows' root-mean-square norm."""
import numpy as np

F32_BAR, BF16_BAR = 1e-5, 2.0 ** -8

# b, L, H, G, P, window, sinks: one token's few; tile edges; ragged tails; windows inside and across tiles, wider than the row; sinks
# inside the window, in front of it, more than a tile; shared heads that do and do not divide a tile; padded widths
SHAPES = [(1, 2, 1, 1, 64, 4, 0), (2, 63, 2, 2, 64, 17, 3), (1, 128, 4, 2, 128, 128, 0), (2, 129, 4, 1, 64, 64, 1),
          (1, 300, 2, 2, 64, 100, 130), (1, 260, 5, 1, 128, 33, 4), (1, 200, 6, 2, 96, 1000, 0), (2, 150, 3, 1, 8, 40, 16),
          (1, 513, 1, 1, 64, 129, 4), (1, 700, 2, 1, 128, 256, 128), (1, 400, 8, 1, 80, 2, 5), (1, 70, 33, 1, 64, 20, 2),
          (1, 140, 128, 1, 64, 50, 4), (1, 90, 130, 1, 64, 50, 4)]
F32_SHAPES = SHAPES[:9] + [(2, 33, 3, 1, 4, 7, 2), (1, 40, 2, 2, 36, 9, 0), (1, 50, 2, 1, 124, 9, 3)]


def store(a, bf16):
    import torch
    t = torch.from_numpy(np.ascontiguousarray(a, np.float32))
    return (t.bfloat16().float() if bf16 else t).numpy()


def draw(b, L, H, G, P, seed, bf16=True):
    r = np.random.default_rng(seed)
    common = 0.5 * r.standard_normal(P)
    return dict(q=store(r.standard_normal((b, L, H, P)) + common, bf16), k=store(r.standard_normal((b, L, G, P)) + common, bf16),
                v=store(r.standard_normal((b, L, G, P)), bf16), do=store(r.standard_normal((b, L, H, P)), bf16))


def errors(got, ref, axes):
    """Relative errors: of the whole, and of the worst slice along the leading axes."""
    got, ref = np.asarray(got, np.float64), np.asarray(ref, np.float64)
    assert got.shape == ref.shape and np.isfinite(got).all()
    d, n = got - ref, np.linalg.norm(ref)
    m = int(np.prod(ref.shape[:axes]))
    rn = np.linalg.norm(ref.reshape(m, -1), axis=1)
    floor = 0.1 * np.sqrt(np.mean(rn ** 2))
    rows = np.linalg.norm(d.reshape(m, -1), axis=1) / np.maximum(rn, floor) if n else np.linalg.norm(d.reshape(m, -1), axis=1)
    return np.linalg.norm(d) / (n if n else 1.0), float(rows.max())


def check(got, ref, bar, what, axes=3):
    whole, worst = errors(got, ref, axes)
    assert whole <= bar, f"{what}: {whole:.3e} > {bar:.3e}"
    assert worst <= 4 * bar, f"{what}, worst slice: {worst:.3e} > {4 * bar:.3e}"
