"""Float64 reference of the prompt calls: attention of packed sequences with the heads'
own keys and values, and the values of cached positions.

TEST INFRASTRUCTURE ONLY (see the package docstring)."""
import numpy as np

from . import dsa_oracle as O


def attention(q, k, v, scale, causal, k_shared=None):
    """One sequence: q [lq, H, d + e], k and v [lk, G, d], k_shared [lk, e] (float64 values).
    Returns out [lq, H, d], lse [lq, H], A = sum p |v| [lq, H, d] and the largest
    scale * sum |q k| of each row [lq, H] (0 where it sees nothing)."""
    lq, H, _ = q.shape
    lk, G, d = k.shape
    out, A = np.zeros((lq, H, d)), np.zeros((lq, H, d))
    lse, big = np.full((lq, H), -np.inf), np.zeros((lq, H))
    for h in range(H):
        g = h * G // H
        key = k[:, g] if k_shared is None else np.concatenate([k[:, g], k_shared], axis=1)
        dots, size = scale * (q[:, h] @ key.T), scale * (np.abs(q[:, h]) @ np.abs(key).T)
        if causal:
            hidden = np.arange(lk)[None] > np.arange(lq)[:, None] + (lk - lq)
            dots[hidden], size[hidden] = -np.inf, 0.0
        if lk == 0:
            continue
        top = dots.max(axis=1, keepdims=True)
        seen = np.isfinite(top[:, 0])
        p = np.exp(dots[seen] - top[seen])
        z = p.sum(axis=1, keepdims=True)
        out[seen, h] = (p / z) @ v[:, g]
        A[seen, h] = (p / z) @ np.abs(v[:, g])
        lse[seen, h] = (top[seen] + np.log(z))[:, 0]
        big[seen, h] = size[seen].max(axis=1)
    return out, lse, A, big


def join(prev_out, prev_lse, out, lse):
    """Two results over different keys as one; also the two weights."""
    both = np.logaddexp(prev_lse, lse)
    safe = np.where(np.isneginf(both), 0.0, both)
    a, b = np.exp(prev_lse - safe), np.exp(lse - safe)
    kept = np.where((a > 0)[..., None], prev_out, 0.0)
    return a[..., None] * kept + b[..., None] * out, both, a, b


def token_values(layout, bt_row, positions):
    """Index keys [n, 128] and latents [n, 576] of the positions of one request (float64)."""
    positions = np.asarray(positions, dtype=np.int64)
    if positions.size == 0:
        return np.zeros((0, 128)), np.zeros((0, 576))
    keys = O.gather_index_keys(layout, bt_row, int(positions.max()) + 1)
    return keys[positions], O.gather_latents(layout, bt_row, positions)
