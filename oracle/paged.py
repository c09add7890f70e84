"""fp64 definition of attention over a paged KV cache."""

import numpy as np


def gather(cache, table_row, length):
    """Keys (or values) 0..length-1 of a sequence, [length, H_kv, D], from a cache
    [num_pages, H_kv, page_size, D]."""
    page = cache.shape[2]
    key = np.arange(length)
    return cache[table_row[key // page], :, key % page].astype(np.float64)


def attention(q, k_cache, v_cache, cu_q, seq_lens, table, scale, tree=None):
    """out, lse, and sum p |v| and sqrt(sum (p v)^2) (what bounds out's rounding, and
    what it comes to where the roundings of p are independent) of every row; NaN in
    the rows behind the last sequence.  tree: bool [N, new tokens] or None."""
    N, H, D = q.shape
    G = H // k_cache.shape[1]
    out, lse = np.full((N, H, D), np.nan), np.full((N, H), np.nan)
    mag, rms = np.full((N, H, D), np.nan), np.full((N, H, D), np.nan)
    for b in range(len(seq_lens)):
        first, n, L = int(cu_q[b]), int(cu_q[b + 1] - cu_q[b]), int(seq_lens[b])
        k, v = gather(k_cache, table[b], L), gather(v_cache, table[b], L)
        for i in range(n):
            sees = np.arange(L) <= L - n + i
            if tree is not None:
                sees = np.arange(L) < L - n
                bits = tree[first + i][:n]
                j = L - n + np.flatnonzero(bits)
                sees[j[(j >= 0) & (j < L)]] = True
            for h in range(H):
                if not sees.any():
                    out[first + i, h], lse[first + i, h] = 0.0, -np.inf
                    mag[first + i, h] = rms[first + i, h] = 0.0
                    continue
                s = k[sees][:, h // G] @ q[first + i, h].astype(np.float64) * scale
                m = s.max()
                p = np.exp(s - m)
                lse[first + i, h] = m + np.log(p.sum())
                p /= p.sum()
                out[first + i, h] = p @ v[sees][:, h // G]
                mag[first + i, h] = p @ np.abs(v[sees][:, h // G])
                rms[first + i, h] = np.sqrt(p ** 2 @ v[sees][:, h // G] ** 2)
    return out, lse, mag, rms


def words(tree):
    """bool [N, n] as int32 [N, ceil(n / 32)], bit j % 32 of word j / 32."""
    N, n = tree.shape
    w = max(1, -(-n // 32))
    full = np.zeros((N, w * 32), np.uint32)
    full[:, :n] = tree
    full = (full.reshape(N, w, 32) << np.arange(32, dtype=np.uint32)).sum(-1, dtype=np.uint32)
    return full.view(np.int32)
