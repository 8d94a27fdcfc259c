"""Plain 64-bit forms of the rotated append, the block-scaled 8-bit cache and
attention over a window with sinks, with bounds on what the kernels' roundings
can add.  CPU only; nothing of the library is used."""
import math

import numpy as np
import torch

BS = 16
F16_HALF_STEP = 2.0 ** -11              # largest relative rounding error, fp16
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: F16_HALF_STEP}
SUBNORMAL = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}


def visible(L, q_pos, window, sinks):
    """Positions of an L-token sequence that a query at q_pos sees."""
    return [j for j in range(L) if j <= q_pos and (j > q_pos - window or j < sinks)]


def attention(q, k, v, scale, dtype, weight_error, k_offset=None, v_offset=None):
    """One query row against its visible keys, fp64, and the bound on a kernel's
    error.  q [D], k and v [n][D] (fp64).

    k_offset, v_offset [n]: what the kernel adds to every |k| and |v| of a token
    inside its products and takes off again (8-bit pools: 1152 scales).

    The output is sum p v / sum p.  A weight's relative error is at most
    `weight_error` (its rounding on the way into the P V product) + 2^-20
    (exponent and its argument) + the error of its score: products of two
    16-bit values are exact in fp32, and a chain of D fp32 additions that may
    truncate is off by at most D 2^-23 times the sum of magnitudes.  Numerator
    and denominator then move by that much of sum p |v| and sum p; weights
    below fp16's normal range add 2^-25 |v| each (the largest weight is at
    least 1).  Last, one rounding to the output type."""
    if k_offset is None:
        k_offset = v_offset = torch.zeros(len(k), dtype=torch.float64)
    x = (k @ q) * scale
    p = torch.exp(x - x.max())
    total = p.sum()
    out = (p @ v) / total
    # the offset counts twice: in the products and in the sum taken off
    score = scale * (k.abs() @ q.abs() + 2 * k_offset * q.abs().sum()).max().item()
    rel = weight_error + 2.0 ** -20 + q.numel() * 2.0 ** -23 * score
    spread = (p @ v.abs()) / total
    tiny = 2.0 ** -25 * v.abs().sum(0) / total
    # 16 tokens' products are added at a time
    tiny = tiny + 16 * 2.0 ** -23 * 2 * (p @ v_offset) / total
    bound = 2 * rel * spread + tiny + HALF_STEP[dtype] * out.abs() + SUBNORMAL[dtype]
    return out, bound


def assert_within(got, want, bound, what=""):
    got = got.detach().double().cpu()
    # the bound is first order: allow its square on top
    bad = ~((got - want).abs() <= bound * 1.01)
    if bad.any():
        at = bad.nonzero()[0].tolist()
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside, first at {at}: got "
                             f"{got[tuple(at)].item()}, want {want[tuple(at)].item()} within "
                             f"{bound[tuple(at)].item():.3g}")


def rotate(x, cos_sin, pos, interleaved):
    """x [T][H][D] fp64 -> rotated, and the magnitudes |x0| + |x1| of each pair."""
    half = cos_sin.shape[1] // 2
    i = torch.arange(half)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    c = cos_sin[pos][:, None, :half].double()
    s = cos_sin[pos][:, None, half:].double()
    y, mag = x.clone(), torch.zeros_like(x)
    y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., b] * c + x[..., a] * s
    mag[..., a] = mag[..., b] = x[..., a].abs() + x[..., b].abs()
    return y, mag


def rotate_f32(x, cos_sin, pos, interleaved):
    """The same in fp32, every product and sum rounded by itself."""
    half = cos_sin.shape[1] // 2
    i = np.arange(half)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    t = cos_sin.numpy()[pos]
    c, s = t[:, None, :half], t[:, None, half:]
    y = x.copy()
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


# ------------------------------------------------------- block-scaled 8-bit records
def chunk_offset(t, j, dim):
    return t * dim // 128 * 128 + 16 * (j ^ (4 * (t % 2)) ^ (2 * (t // 2 % 4)))


class Records:
    """A block-scaled pool as plain arrays: codes [2][nb][Hkv][16][D] int8 (K, V)
    and scales [2][nb][Hkv] fp32; read from and written to the pool's bytes."""

    def __init__(self, nb, hkv, dim):
        self.codes = np.zeros((2, nb, hkv, BS, dim), np.int16)
        self.scales = np.zeros((2, nb, hkv), np.float32)
        self.dim = dim

    @classmethod
    def from_bytes(cls, kv):
        kv = np.asarray(kv)
        nb, hkv, size = kv.shape
        r = cls(nb, hkv, (size - 32) // 32)
        for part in range(2):
            for t in range(BS):
                for j in range(r.dim // 16):
                    at = 16 * r.dim * part + chunk_offset(t, j, r.dim)
                    r.codes[part, :, :, t, 16 * j:16 * j + 16] = kv[:, :, at:at + 16].astype(np.int16) - 128
        r.scales[:] = np.moveaxis(kv[:, :, 32 * r.dim:32 * r.dim + 8].copy().view(np.float32), 2, 0)
        return r

    def to_bytes(self):
        _, nb, hkv, _, dim = self.codes.shape
        kv = np.zeros((nb, hkv, 32 * dim + 32), np.uint8)
        for part in range(2):
            for t in range(BS):
                for j in range(dim // 16):
                    at = 16 * dim * part + chunk_offset(t, j, dim)
                    kv[:, :, at:at + 16] = (self.codes[part, :, :, t, 16 * j:16 * j + 16] + 128).astype(np.uint8)
        kv[:, :, 32 * dim:32 * dim + 8] = np.ascontiguousarray(np.moveaxis(self.scales, 0, 2)).view(np.uint8)
        return kv

    def values(self, part):
        """[nb][Hkv][16][D] fp64."""
        return self.codes[part].astype(np.float64) * self.scales[part].astype(np.float64)[..., None, None]

    def append(self, part, rows, slots):
        """rows [T][Hkv][D] fp32 into their slots, by the documented rule."""
        f = np.float32
        runs = {}
        for t, slot in enumerate(slots):
            if slot >= 0:
                runs.setdefault(int(slot) // BS, []).append((int(slot) % BS, t))
        for b, members in runs.items():
            offs, ts = [m[0] for m in members], [m[1] for m in members]
            for h in range(rows.shape[1]):
                x = rows[ts, h]
                finite = np.where(np.isnan(x), f(0), np.minimum(np.abs(x), f(float.fromhex("0x1.fep127"))))
                amax = finite.max()
                if amax < f(2.0 ** -100):
                    amax = f(0)
                old = self.scales[part, b, h] if offs[0] > 0 else f(0)
                new = max(old, f(amax * f(1 / 127)))
                if offs[0] > 0 and new > old:
                    ratio = f(old / new)
                    c = self.codes[part, b, h, :offs[0]].astype(f)
                    self.codes[part, b, h, :offs[0]] = np.rint((c * ratio).astype(f))
                self.scales[part, b, h] = new
                inv = f(f(1) / new) if new > 0 else f(0)
                with np.errstate(invalid="ignore", over="ignore"):
                    y = (x * inv).astype(f)
                y = np.where(np.isnan(y), f(0), np.clip(y, f(-127), f(127)))
                self.codes[part, b, h, offs] = np.rint(y)


def random_case(gen, lens, hkv, maxb, extra=3):
    """Tables [S][maxb] over a shuffled pool that holds every block of `lens`."""
    nbs = [-(-n // BS) for n in lens]
    nb = sum(nbs) + extra
    perm = torch.randperm(nb, generator=gen).tolist()
    tables = torch.full((len(lens), maxb), -1, dtype=torch.int32)
    for s, n in enumerate(nbs):
        for b in range(n):
            tables[s, b] = perm.pop()
    return tables, nb


def scale_of(dim):
    return 1.0 / math.sqrt(dim)
