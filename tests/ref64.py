"""Plain 64-bit forms of the definitions that the four-bit cache, the rotary
axes and the page calls are tested against.  They share no code with the CUDA
path and are pinned by tests/test_operators_host.py."""
import numpy as np
import torch

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
# fp32 error of a normed and rotated element, relative to its rotation pair's
# norm: derived at K_FP32_REL in parity_util.py.
PAIR_REL = 22 * 2.0 ** -23


# ------------------------------------------------------------------ four-bit entries
def e4m3_values() -> np.ndarray:
    """The 127 finite non-negative E4M3 values by code (bias 7)."""
    c = np.arange(127)
    e, m = c >> 3, c & 7
    return np.where(e == 0, m / 8.0 * 2.0 ** -6, (1 + m / 8.0) * 2.0 ** (e - 7.0))


def nearest(x: np.ndarray, grid: np.ndarray) -> np.ndarray:
    """Index of the nearest grid value (ties to the even index, clamped)."""
    mid = (grid[1:] + grid[:-1]) / 2
    lo, hi = np.searchsorted(mid, x, side="left"), np.searchsorted(mid, x, side="right")
    return np.where(lo % 2 == 0, lo, hi)  # lo != hi only on a tie


def e2m1_store(x, scale: float):
    """(codes [..., D], block scale codes [..., D/16]) of fp32 values x: the
    format's own fp32 steps (product with the fp32 reciprocal, two divisions)."""
    x = np.asarray(x, np.float32)
    y = (x * (np.float32(1) / np.float32(scale))).reshape(*x.shape[:-1], -1, 16)
    s = nearest((np.abs(y).max(-1) / np.float32(6)).astype(np.float64), e4m3_values())
    sv = e4m3_values()[s].astype(np.float32)[..., None]
    with np.errstate(divide="ignore", invalid="ignore"):
        z = np.where(sv > 0, y / sv, np.float32(0))
    c = nearest(np.abs(z).astype(np.float64), E2M1) + 8 * np.signbit(z)
    return c.reshape(x.shape), s


def e2m1_value(codes: np.ndarray) -> np.ndarray:
    return np.where(codes & 8, -1.0, 1.0) * E2M1[codes & 7]


def unpack(cache: torch.Tensor) -> np.ndarray:
    """Codes [slots, Hkv, D] of an E2M1 cache tensor [slots, Hkv, D/2]."""
    b = cache.cpu().numpy().astype(np.int64)
    return np.stack((b & 15, b >> 4), -1).reshape(*b.shape[:-1], -1)


def e4m3_signed(codes: np.ndarray) -> np.ndarray:
    v = np.append(e4m3_values(), np.nan)
    return np.where(codes & 0x80, -1.0, 1.0) * v[codes & 0x7F]


def entries(cache: torch.Tensor, kind: str, scale: float, block_scale=None) -> np.ndarray:
    """fp64 entries [slots, Hkv, D] of a cache tensor."""
    if kind == "bf16":
        return cache.cpu().double().numpy()
    if kind == "e4m3":
        return e4m3_signed(cache.cpu().numpy().astype(np.int64)) * scale
    s = e4m3_signed(block_scale.cpu().numpy().astype(np.int64)).transpose(1, 0, 2)
    v = e2m1_value(unpack(cache))
    return (v.reshape(*v.shape[:-1], -1, 16) * s[..., None]).reshape(v.shape) * scale


# ------------------------------------------------------------------ norm, rotation, attention
def axis_of(D: int, sections, interleaved: bool) -> np.ndarray:
    A = len(sections)
    if interleaved:
        return np.array([i % A if i // A < sections[i % A] else 0 for i in range(D // 2)])
    return np.repeat(np.arange(A), sections)


def norm_rope(x, w, place, eps: float, theta: float) -> np.ndarray:
    """x [N, H, D] normed with w and rotated, pair i of token t at place[t, i]."""
    x, w = np.asarray(x, np.float64), np.asarray(w, np.float64)
    D = x.shape[-1]
    y = w * x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    a = (place * theta ** (-2.0 * np.arange(D // 2) / D))[:, None]
    y1, y2 = y[..., :D // 2], y[..., D // 2:]
    return np.concatenate((y1 * np.cos(a) - y2 * np.sin(a), y2 * np.cos(a) + y1 * np.sin(a)), -1)


def pair_norm(y: np.ndarray) -> np.ndarray:
    return np.hypot(y, np.roll(y, y.shape[-1] // 2, -1))


def places(host: dict, D: int, axes=None) -> np.ndarray:
    """[N, D/2] positions: c_b + j on every pair, or the axes' (positions
    int [A, N], sections, interleaved)."""
    cu, cl = host["cu_seqlens"].numpy(), host["cache_lens"].numpy()
    if axes is not None:
        pos, sections, inter = axes
        return np.asarray(pos, np.float64)[axis_of(D, sections, inter)].T
    p = np.concatenate([np.arange(cl[b], cl[b] + cu[b + 1] - cu[b]) for b in range(len(cl))] or [[]])
    return np.repeat(p[:, None], D // 2, 1).astype(np.float64)


def prepared(w, host: dict, axes=None):
    """fp64 (Q [N, Hq, D], K [N, Hkv, D], V [N, Hkv, D]) of the call's tokens."""
    Hq, Hkv, D = w.num_q_heads, w.num_kv_heads, w.head_dim
    x = host["qkv"].double().numpy().reshape(-1, Hq + 2 * Hkv, D)
    at = places(host, D, axes)
    q = norm_rope(x[:, :Hq], host["q_norm_w"].double().numpy(), at, w.rms_eps, w.rope_theta)
    k = norm_rope(x[:, Hq:Hq + Hkv], host["k_norm_w"].double().numpy(), at, w.rms_eps, w.rope_theta)
    return q, k, x[:, Hq + Hkv:]


def slots_of(host: dict, b: int, n: int) -> np.ndarray:
    """Slots of the positions 0 .. n - 1 of request b."""
    p = np.arange(n)
    if host.get("page_table") is None:
        return int(host["slot_base"][b]) + p
    ps = int(host["page_size"])
    return host["page_table"].numpy()[b, p // ps].astype(np.int64) * ps + p % ps


def attend(w, host: dict, q: np.ndarray, keys: np.ndarray, vals: np.ndarray):
    """(out [N, Hq, D], bound on the kernels' error) in fp64: causal attention of
    the prepared q over the entries [slots, Hkv, D] of the cache after the call.

    The bound follows the kernels' roundings, each off by at most half a step.
    Q enters the products as f16 (2^-11 of each element) or bf16 (2^-8) after
    fp32 steps off by PAIR_REL of its pair, P with the same half step, the
    output is rounded to bf16 (2^-8); fp32 accumulation and exp2 stay below
    2^-16 of sums of magnitudes.  A score then moves by at most
    d = (h + 2^-16) sum |q_i k_i| / sqrt(D) + PAIR_REL sum |pair_i k_i| / sqrt(D),
    every weight by a factor within exp(+-2 max d), P by another 1 +- h, so
      |out - ref| <= 2^-8 |ref| (1 + small) + (exp(2 max d) - 1 + 2 h + 2^-15) sum p |v|.
    """
    h = 2.0 ** -8 if host.get("kv_dtype", "bf16") == "bf16" else 2.0 ** -11
    cu, cl = host["cu_seqlens"].numpy(), host["cache_lens"].numpy()
    Hq, Hkv, D = w.num_q_heads, w.num_kv_heads, w.head_dim
    G = Hq // Hkv
    out, tol = np.zeros_like(q), np.zeros_like(q)
    for b in range(len(cl)):
        t0, t1, c = int(cu[b]), int(cu[b + 1]), int(cl[b])
        if t1 == t0:
            continue
        s = slots_of(host, b, c + t1 - t0)
        hidden = np.arange(len(s))[None] > c + np.arange(t1 - t0)[:, None]
        for hd in range(Hq):
            k, v, x = keys[s, hd // G], vals[s, hd // G], q[t0:t1, hd]
            sc = x @ k.T / np.sqrt(D)
            d = ((h + 2.0 ** -16) * np.abs(x) @ np.abs(k).T + PAIR_REL * pair_norm(x) @ np.abs(k).T) / np.sqrt(D)
            sc[hidden], d[hidden] = -np.inf, 0
            p = np.exp(sc - sc.max(1, keepdims=True))
            p /= p.sum(1, keepdims=True)
            o = p @ v
            grow = np.exp(2 * d.max(1, keepdims=True)) - 1 + 2 * h + 2.0 ** -15
            out[t0:t1, hd] = o
            tol[t0:t1, hd] = 2.0 ** -8 * 1.01 * np.abs(o) + grow * 1.01 * (p @ np.abs(v))
    return out, tol
