"""Plain numpy restatements of the cache operators in 64 bits, for their tests: the
quantisation of rows and keys and the dense attention, straight from the formulas."""
import numpy as np

from oracle.formats import bf16_to_f64, e4m3_to_f64

E4M3 = e4m3_to_f64(np.arange(127))          # finite values >= 0, ascending by code


def nearest_e4m3(x):
    """uint8 codes of the e4m3 values nearest to x (ties to the even code, saturating)."""
    x = np.asarray(x, np.float64)
    a = np.minimum(np.abs(x), 448.0)
    hi = np.clip(np.searchsorted(E4M3, a), 1, 126)
    lo = hi - 1
    up, down = E4M3[hi] - a, a - E4M3[lo]
    pick = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    return (pick | np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def bf16_bits(x):
    """Nearest bf16, ties to even, of finite fp32 values inside the bf16 range."""
    u = np.ascontiguousarray(x, np.float32).view(np.uint32).astype(np.uint64)
    return ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)


def quantise(x, group=128):
    """x [n, d] fp32 -> codes [n, d] uint8, scales [n, d / group] fp32: scale = amax / 448
    and x / scale in correctly rounded fp32, as the definition has them."""
    x = np.asarray(x, np.float32)
    g = x.reshape(x.shape[0], -1, group)
    amax = np.abs(g).max(axis=2)
    with np.errstate(divide="ignore", over="ignore", under="ignore"):
        scale = np.where(amax > 0, np.maximum(amax / np.float32(448), np.float32(2.0 ** -126)), np.float32(1)).astype(np.float32)
        codes = nearest_e4m3(g / scale[:, :, None])
    return codes.reshape(x.shape), scale


def pack_rows(latent, rope):
    """[n, 512] and [n, 64] fp32 -> [n, 656] bytes."""
    codes, scale = quantise(latent)
    n = codes.shape[0]
    return np.concatenate([codes, np.ascontiguousarray(scale, "<f4").view(np.uint8).reshape(n, 16),
                           bf16_bits(rope).astype("<u2").view(np.uint8).reshape(n, 128)], axis=1)


def row_values(rows):
    """[n, 656] bytes -> [n, 576] fp64."""
    n = rows.shape[0]
    scale = np.ascontiguousarray(rows[:, 512:528]).view("<f4").astype(np.float64)
    lat = (e4m3_to_f64(rows[:, :512]).reshape(n, 4, 128) * scale[:, :, None]).reshape(n, 512)
    return np.concatenate([lat, bf16_to_f64(np.ascontiguousarray(rows[:, 528:]).view("<u2"))], axis=1)


def attend(q, kv, sm_scale):
    """q [H, 576], kv [L, 576] fp64 -> out [H, 512], lse [H], and the two sums that bound the
    errors: A = sum_t p_t |v_t| [H, 512] and S = max_t |sm_scale| sum_d |q_d k_td| [H]."""
    if kv.shape[0] == 0:
        z = np.zeros((q.shape[0], 512))
        return z, np.full(q.shape[0], -np.inf), z, np.zeros(q.shape[0])
    z = sm_scale * (q @ kv.T)
    m = z.max(axis=1, keepdims=True)
    e = np.exp(z - m)
    p = e / e.sum(axis=1, keepdims=True)
    s = abs(sm_scale) * (np.abs(q) @ np.abs(kv).T).max(axis=1)
    return p @ kv[:, :512], (m + np.log(e.sum(axis=1, keepdims=True)))[:, 0], p @ np.abs(kv[:, :512]), s


# Bounds of chunk_attention's errors, from its documented precision.
# z: 576 exact products summed in fp32 (each sum off by at most 2^-23 of the running
#    magnitude on a tensor core that truncates): 576 * 2^-23 < 2^-13 of S, relative to the terms.
# p: off by a factor exp(+-dz) from z, by 2^-11 from fp16, and relative 2^-20 from exp2;
# v: 2^-11 from fp16; out: the output type's half step; below 2^-14 the fp16 steps are an
#    absolute 2^-25 (v: up to 2^-25 times sum p = 1; p: 2^-32 of the largest, per row).
DZ = 2.0 ** -13


def out_bound(out, a, s, half_step, n_rows):
    rel = 2 * np.minimum(DZ * s, 1.0)[:, None] + 2 * 2.0 ** -11 + 2.0 ** -19
    vmax = np.abs(a).max() + 1.0
    return half_step * np.abs(out) * 1.01 + 1.02 * rel * a + 2.0 ** -24 + n_rows * 2.0 ** -31 * vmax


def lse_bound(lse, s):
    return DZ * s + 2.0 ** -21 * (np.abs(lse) + 32)
