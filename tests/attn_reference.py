"""The cache and attention operators' definitions in 64 bits (numpy), for the tests.

``quantised`` gives the values that a cached vector stands for: the codes are
decided in fp32 by definition, element by element.  ``attention`` is a loop
over rows and heads on the visible keys alone.  ``out_bound`` is the tolerance
of an output, from the roundings that the kernels may make:

  * the probabilities are rounded to the 16-bit type before they meet the
    values, u = 2^-11 (fp16) or 2^-8 (bf16) relative each: at most u * A with
    A = sum p |v| / sum p; below the type's normal range (fp16: 2^-14, with
    the largest probability at 1) 2^-25 absolute each: 2^-25 * sum |v| / l,
    l = sum p >= 1;
  * the result is rounded once: u * |out|, or half the smallest subnormal;
  * scores are fp32 sums of d exact products: their error e moves p by a
    factor e^e, so out by at most 2 e A, with e = 2 * d * 2^-24 * scale *
    |q|.|k| (a sum's worst order, and as much again for the hardware's way of
    adding);
  * exp2 and fp32 sums: 2^-20 * A, generously.
"""
import numpy as np

U = {"float16": 2.0 ** -11, "bfloat16": 2.0 ** -8}


def quantised(fmt, x):
    """x fp32 [..., d] -> the cached values, float64."""
    x = np.asarray(x, np.float32)
    if fmt == "f16":
        return x.astype(np.float16).astype(np.float64)
    step = x.shape[-1] if fmt == "int8" else 32
    out = np.empty(x.shape, np.float64)
    for idx in np.ndindex(x.shape[:-1]):
        for lo in range(0, x.shape[-1], step):
            b = x[idx][lo:lo + step]
            if not np.isfinite(b).all():
                out[idx][lo:lo + step] = np.nan
                continue
            peak = b[np.argmax(np.abs(b))]
            if fmt == "int8":
                a = np.float32(np.abs(peak) / np.float32(127))
                q = np.clip(np.rint(b / a), -127, 127) if a > 0 else np.zeros(step)
                out[idx][lo:lo + step] = q.astype(np.float64) * np.float64(a)
            else:
                a = np.float32(peak / np.float32(-8))
                if a == 0:
                    q = np.zeros(step)
                else:
                    r = (b / a).astype(np.float64)
                    q = np.clip(np.sign(r) * np.floor(np.abs(r) + 0.5) + 8, 0, 15) - 8
                with np.errstate(over="ignore"):
                    out[idx][lo:lo + step] = q * np.float64(np.float16(a))
    return out


def attention(q, k, v, see, scale, kind="float16"):
    """q [n, hq, d], k and v [m, hkv, d] float64, see [n, m] -> out, lse, and the bounds of both."""
    n, hq, d = q.shape
    g = hq // k.shape[1] if k.shape[1] else 1
    out, bound = np.zeros((n, hq, d)), np.zeros((n, hq, d))
    lse, lse_bound = np.full((n, hq), -np.inf), np.zeros((n, hq))
    u = U[kind]
    for i in range(n):
        js = np.flatnonzero(see[i])
        if not len(js):
            continue
        for h in range(hq):
            kk, vv = k[js, h // g], v[js, h // g]
            s = scale * (kk @ q[i, h])
            e = 2 * d * 2.0 ** -24 * abs(scale) * float(np.max(np.abs(kk) @ np.abs(q[i, h])))
            top = s.max()
            p = np.exp(s - top)
            l = p.sum()
            with np.errstate(invalid="ignore"):
                out[i, h] = p @ vv / l
                A = p @ np.abs(vv) / l
                bound[i, h] = (u * 1.01 * np.abs(out[i, h]) + 1.01 * u * A + 2.0 ** -25 * np.abs(vv).sum(0) / l
                               + 2 * e * A + 2.0 ** -20 * A + 2.0 ** -25)
            lse[i, h] = top + np.log(l)
            lse_bound[i, h] = e + 2.0 ** -20 * (1 + abs(lse[i, h]))
    return out, lse, bound, lse_bound


def check(name, got, lse_got, ref):
    out, lse, bound, lse_bound = ref
    got, lse_got = np.asarray(got, np.float64), np.asarray(lse_got, np.float64)
    fine = np.isfinite(out)
    assert np.array_equal(np.isfinite(got), fine), f"{name}: infinities or NaN at other places"
    off = np.abs(got[fine] - out[fine]) - bound[fine]
    assert not off.size or off.max() <= 0, f"{name}: {np.count_nonzero(off > 0)} outputs off, worst by {off.max():.3g}"
    some = np.isfinite(lse)
    assert np.array_equal(np.isneginf(lse), np.isneginf(lse_got)), f"{name}: empty rows"
    off = np.abs(lse_got[some] - lse[some]) - lse_bound[some]
    assert not off.size or off.max() <= 0, f"{name}: lse off by {off.max():.3g}"
