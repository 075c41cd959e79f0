"""Plain 64-bit reference of the 4-bit key/value cache, its attention, commit
and page pool (numpy, written from the definitions in include/gdn.h).  Values
that the definition fixes bit for bit (scales and codes) are formed in fp32 as
it says; everything else is float64."""
import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
E4M3 = np.array([(2.0 ** -6 * (b & 7) / 8 if b >> 3 == 0 else
                  2.0 ** ((b >> 3) - 7) * (1 + (b & 7) / 8)) for b in range(127)])


def _nearest(grid, x):
    """Index of the nearest grid value (ties to the even index), saturating."""
    x = np.minimum(x.astype(np.float64), grid[-1])
    hi = np.clip(np.searchsorted(grid, x), 1, len(grid) - 1)
    lo = hi - 1
    dl, dh = x - grid[lo], grid[hi] - x
    return np.where((dh < dl) | ((dh == dl) & (hi % 2 == 0)), hi, lo)


def quantise(x, head_scale):
    """x [..., H, D] float64/32 -> codes uint8 [..., H, D], scale bytes [..., H, D/16]."""
    inv = np.float32(1.0) / np.asarray(head_scale, np.float32)
    with np.errstate(over="ignore", invalid="ignore"):
        y = np.asarray(x, np.float32) * inv[:, None]
        y = np.clip(np.where(np.isnan(y), np.float32(0), y), np.float32(-2688), np.float32(2688))
    y = y.reshape(*y.shape[:-1], y.shape[-1] // 16, 16)
    a = np.abs(y).max(-1)
    s8 = _nearest(E4M3, a * np.float32(1.0 / 6.0)).astype(np.uint8)
    s = E4M3[s8].astype(np.float32)
    r = np.where(s > 0, np.float32(1) / np.where(s > 0, s, np.float32(1)), np.float32(0))
    t = y * r[..., None].astype(np.float32)
    code = _nearest(E2M1, np.abs(t)).astype(np.uint8) | (np.signbit(y).astype(np.uint8) << 3)
    return code.reshape(*y.shape[:-2], y.shape[-2] * 16), s8


def values(code, s8):
    """float64 values of codes [..., D] and scale bytes [..., D/16] (no head scale)."""
    v = np.where(code > 7, -1.0, 1.0) * E2M1[code & 7]
    return v * np.repeat(E4M3[s8 & 127], 16, axis=-1)


class Cache:
    """Pages as the library lays them out, addressed token by token."""

    def __init__(self, pages, D):
        self.pages, self.D = pages, D   # uint8 [n_pages, Hkv, R, 36*D]

    def _at(self, page, h, slot):
        return self.pages[page, h, slot // 32], slot % 32

    def put(self, page, h, slot, kc, ks, vc, vs):
        D = self.D
        rec, t = self._at(page, h, slot)
        kb = kc[0::2] | (kc[1::2] << 4)
        rec[:16 * D].reshape(D // 32, 32, 16)[:, t] = kb.reshape(D // 32, 16)
        vb = rec[16 * D:32 * D].reshape(D, 16)
        sh = 4 * (t % 2)
        vb[:, t // 2] = (vb[:, t // 2] & (0xF0 >> sh)) | (vc << sh)
        rec[32 * D:34 * D].reshape(32, D // 16)[t] = ks
        rec[34 * D:].reshape(D // 16, 32)[:, t] = vs

    def get(self, page, h, slot):
        D = self.D
        rec, t = self._at(page, h, slot)
        kb = rec[:16 * D].reshape(D // 32, 32, 16)[:, t].reshape(-1)
        kc = np.stack((kb & 15, kb >> 4), -1).reshape(-1)
        vc = (rec[16 * D:32 * D].reshape(D, 16)[:, t // 2] >> (4 * (t % 2))) & 15
        return (kc, rec[32 * D:34 * D].reshape(32, D // 16)[t], vc,
                rec[34 * D:].reshape(D // 16, 32)[:, t])


def append(cache, table, kv_len, page_tokens, k, v, k_scale, v_scale):
    B, N, H, _ = k.shape
    kc, ks = quantise(k, k_scale)
    vc, vs = quantise(v, v_scale)
    for b in range(B):
        for n in range(N):
            p = int(kv_len[b]) - N + n
            if p < 0:
                continue
            for h in range(H):
                cache.put(table[b, p // page_tokens], h, p % page_tokens, kc[b, n, h],
                          ks[b, n, h], vc[b, n, h], vs[b, n, h])


def sequence(cache, row, length, page_tokens, h, k_scale, v_scale):
    """float64 keys and values [length, D] of head h."""
    got = [cache.get(row[p // page_tokens], h, p % page_tokens) for p in range(length)]
    if not got:
        return np.zeros((0, cache.D)), np.zeros((0, cache.D))
    kc, ks, vc, vs = (np.stack(x) for x in zip(*got))
    return values(kc, ks) * float(k_scale[h]), values(vc, vs) * float(v_scale[h])


def path_of(parent, node):
    path = []
    while node >= 0:
        path.append(node)
        node = int(parent[node])
    return path[::-1]


def attention(cache, table, kv_len, page_tokens, q, scale, k_scale, v_scale, parent=None):
    """o, lse, and the pieces of the error bound: sum_j p_j |v_j| and max_j sum_i |q_i k_ji|."""
    B, N, Hq, D = q.shape
    H = cache.pages.shape[1]
    o, weight = np.zeros((B, N, Hq, D)), np.zeros((B, N, Hq, D))
    lse, reach = np.full((B, N, Hq), -np.inf), np.zeros((B, N, Hq))
    for b in range(B):
        L = int(kv_len[b])
        base = L - N
        seen = np.zeros((N, L), bool)
        for n in range(N):
            if parent is None:
                seen[n, :max(0, base + n + 1)] = True
            else:
                seen[n, :max(0, base)] = True
                for m in path_of(parent[b], n):
                    if base + m >= 0:
                        seen[n, base + m] = True
        for h in range(H):
            k, v = sequence(cache, table[b], L, page_tokens, h, k_scale, v_scale)
            for g in range(Hq // H):
                i = h * (Hq // H) + g
                x = np.where(seen, q[b, :, i] @ k.T * scale, -np.inf)
                for n in range(N):
                    if not seen[n].any():
                        continue
                    top = x[n].max()
                    p = np.exp(x[n] - top)
                    lse[b, n, i] = top + np.log(p.sum())
                    p /= p.sum()
                    o[b, n, i] = p @ v
                    weight[b, n, i] = p @ np.abs(v)
                    reach[b, n, i] = (np.abs(k[seen[n]]) @ np.abs(q[b, n, i])).max() * scale
    return o, lse, weight, reach


def commit(caches, table, kv_len, page_tokens, N, accept, parent=None):
    out = np.array(kv_len, np.int64)
    for b in range(len(kv_len)):
        path = list(range(accept[b] + 1)) if parent is None else path_of(parent[b], accept[b])
        base = int(kv_len[b]) - N
        out[b] = base + len(path)
        for cache in caches:
            for h in range(cache.pages.shape[1]):
                for i, n in enumerate(path):
                    s, d = base + n, base + i
                    if s != d:
                        got = [x.copy() for x in cache.get(table[b, s // page_tokens], h,
                                                           s % page_tokens)]
                        cache.put(table[b, d // page_tokens], h, d % page_tokens, *got)
    return out


class Pool:
    """Page pool in plain Python; pages of every layer as one array [L, n_pages, ...]."""

    def __init__(self, table, kv_len, ref, page_tokens, pages=None):
        self.table, self.kv_len, self.ref = table, kv_len, ref
        self.P, self.pages = page_tokens, pages

    def held(self, n):
        return -(-n // self.P)

    def release(self, rows, keep):
        for r, n in zip(rows, keep):
            if n >= self.kv_len[r]:
                continue
            for j in range(self.held(n), self.held(self.kv_len[r])):
                self.ref[self.table[r, j]] -= 1
                self.table[r, j] = -1
            self.kv_len[r] = n

    def fork(self, src, dst):
        for s, d in zip(src, dst):
            n = self.held(self.kv_len[s])
            self.table[d, :] = -1
            self.table[d, :n] = self.table[s, :n]
            for p in self.table[s, :n]:
                self.ref[p] += 1
            self.kv_len[d] = self.kv_len[s]

    def reserve(self, rows, new_len):
        """Returns the rows that were not served."""
        before = self.ref.copy()
        free = [p for p in range(len(before)) if before[p] == 0]
        used, failed = 0, []
        for r, n in zip(rows, new_len):
            old = int(self.kv_len[r])
            have, want = self.held(old), self.held(n)
            tail = self.table[r, have - 1] if have else -1
            copy = old % self.P != 0 and n > old and before[tail] > 1
            need = want - have + copy
            if need and used + need > len(free):
                used += need
                failed.append(r)
                continue
            got = free[used:used + need]
            used += need
            for j, p in zip(range(have - copy, want), got):
                self.table[r, j] = p
                self.ref[p] = 1
            if copy:
                recs = -(-(old % self.P) // 32)
                self.ref[tail] -= 1
                if self.pages is not None:
                    self.pages[:, got[0], :, :recs] = self.pages[:, tail, :, :recs]
            self.kv_len[r] = n
        return failed
