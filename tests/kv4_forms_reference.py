"""Plain reference of the forms around the 4-bit cache's append and attention (include/gdn.h):
rotary positions in fp32 as the definition fixes them, and attention in 64 bits over a given set
of visible positions, with the pieces of its error bound."""
import numpy as np

import kv4_reference as ref


def turned(x, positions, cos_sin, axis, adjacent):
    """x [B,N,H,D] fp32 with its pairs turned, every product and sum rounded to fp32.  Positions
    [A,B,N] outside the table, and axes outside A, leave their pairs as they are."""
    x = np.asarray(x, np.float32)
    P = cos_sin.shape[2]
    out = x.copy()
    for b in range(x.shape[0]):
        for n in range(x.shape[1]):
            c, s = np.ones(P, np.float32), np.zeros(P, np.float32)
            for i in range(P):
                a = 0 if axis is None else int(axis[i])
                p = int(positions[a, b, n]) if a < positions.shape[0] else -1
                if 0 <= p < cos_sin.shape[0]:
                    c[i], s[i] = cos_sin[p, 0, i], cos_sin[p, 1, i]
            i = np.arange(P)
            first, second = (2 * i, 2 * i + 1) if adjacent else (i, i + P)
            u, w = x[b, n][:, first], x[b, n][:, second]
            with np.errstate(invalid="ignore", over="ignore"):
                out[b, n][:, first] = u * c - w * s
                out[b, n][:, second] = w * c + u * s
    return out


def visible(length, N, parent=None, window=None, sinks=0):
    """[N,length] truth values: positions that each node of the block sees."""
    base = length - N
    seen = np.zeros((N, length), bool)
    for n in range(N):
        if base + n < 0:
            continue
        block = list(range(n + 1)) if parent is None else ref.path_of(parent, n)
        # position of every entry of the node's path; entries before the first token have none
        place = {base + i: base + m for i, m in enumerate(block) if base + m >= 0}
        end = base + len(block) - 1
        for e in list(range(max(0, base))) + sorted(place):
            if window is None or e > end - window or e < sinks:
                seen[n, place.get(e, e)] = True
    return seen


def attention(cache, table, lens, P, q, scale, k_scale, v_scale, seen_of):
    """As kv4_reference.attention, over seen_of(b, length) [N,length]."""
    B, N, Hq, D = q.shape
    H = cache.pages.shape[1]
    o, weight = np.zeros((B, N, Hq, D)), np.zeros((B, N, Hq, D))
    lse, reach = np.full((B, N, Hq), -np.inf), np.zeros((B, N, Hq))
    for b in range(B):
        L = int(lens[b])
        if L <= 0:
            continue
        seen = seen_of(b, L)
        for h in range(H):
            k, v = ref.sequence(cache, table[b], L, P, h, k_scale, v_scale)
            for i in range(h * (Hq // H), (h + 1) * (Hq // H)):
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


def check(o, lse, want, T, eps, D):
    """Outputs against attention()'s result.  The bound: the logits are fp32 sums of D exact
    products (D * 2^-23 of the sum of magnitudes, `reach`), scaled and exponentiated in fp32 (a
    few 2^-22 of a logit of size <= reach), which moves every probability by at most `d`
    relatively and the result by 2 d of the weighted magnitudes; probabilities are rounded to
    binary16 (2^-11 relative, 2^-25 absolute each, against a sum of at least 2^-8 of the
    largest); fp32 sums over T positions, and of parts, add T * 2^-22; the output is rounded
    once (eps)."""
    wo, wlse, weight, reach = want
    d = (D * 2.0 ** -23 + 2.0 ** -20) * reach + 2.0 ** -20
    vmax = np.abs(wo).max() + weight.max()
    tol = (eps * np.abs(wo) + weight * (2 * d[..., None] + 2.0 ** -11 + T * 2.0 ** -22)
           + T * 2.0 ** -25 * vmax + 2.0 ** -24)
    err = np.abs(o.double().cpu().numpy() - wo)
    assert (err <= tol).all(), f"worst {(err / tol).max():.3f} of the bound"
    if lse is None:
        return
    l = lse.double().cpu().numpy()
    assert np.array_equal(np.isinf(l), np.isinf(wlse))
    at = np.isfinite(wlse)
    ltol = (d + T * 2.0 ** -22)[at] + 2.0 ** -22 * np.abs(wlse[at])
    assert (np.abs(l[at] - wlse[at]) <= ltol).all()
