"""Indexed work on resident weights in 64 bits: table rows by token, the router,
experts' products by slot."""
import numpy as np

from .quant_out_prod import dequant

ROUTE_TOP, ROUTE_ALL = 0, 1


def get_rows(wtype, W, N, K, ids, scale):
    """scale * deq(W)[ids], zeros for an id that points nowhere (F32 values of the table, 64-bit product)."""
    table = dequant(wtype, W, N, K).astype(np.float64)
    ids = np.asarray(ids)
    real = (ids >= 0) & (ids < N)
    out = np.zeros((len(ids), K))
    out[real] = table[ids[real]] * np.float64(np.float32(scale))
    return out


def get_rows_back(dY, ids, scale, G, beta):
    """(G, magnitude): the new table and, of each value, the sum of its terms' magnitudes."""
    N = G.shape[0]
    ids = np.asarray(ids)
    real = (ids >= 0) & (ids < N)
    out, mag = np.zeros(G.shape), np.zeros(G.shape)
    np.add.at(out, ids[real], dY[real].astype(np.float64))
    np.add.at(mag, ids[real], np.abs(dY[real].astype(np.float64)))
    s, b = np.float64(np.float32(scale)), np.float64(np.float32(beta))
    old = b * G.astype(np.float64) if beta != 0 else 0.0
    return s * out + old, abs(s) * mag + np.abs(old)


def group(ids, groups):
    """(start, order)."""
    ids = np.asarray(ids).reshape(-1)
    key = np.where((ids < 0) | (ids >= groups), groups, ids)
    order = np.argsort(key, kind="stable")
    return np.searchsorted(key[order], np.arange(groups + 1)).astype(np.int32), order.astype(np.int32)


def route(logits, top, mode, scale):
    """(ids, weights) by the definition, one choice after another."""
    T, E = logits.shape
    ids, weights = np.full((T, top), -1, np.int32), np.zeros((T, top))
    for t in range(T):
        l = logits[t].astype(np.float64)
        left = [e for e in range(E) if l[e] > -np.inf]
        chosen = sorted(left, key=lambda e: (-l[e], e))[:top]
        if not chosen:
            continue
        among = chosen if mode == ROUTE_TOP else left
        with np.errstate(invalid="ignore", over="ignore"):
            total = np.sum(np.exp(l[among] - l[chosen[0]]))
            weights[t, :len(chosen)] = scale * np.exp(l[chosen] - l[chosen[0]]) / total
        ids[t, :len(chosen)] = chosen
    return ids, weights


def route_back(logits, ids, mode, scale, dweights):
    T, E = logits.shape
    out = np.zeros((T, E))
    for t in range(T):
        l = logits[t].astype(np.float64)
        chosen = [int(e) for e in ids[t] if 0 <= e < E]
        among = [e for e in (chosen if mode == ROUTE_TOP else range(E)) if l[e] > -np.inf]
        if not among:
            continue
        p = np.exp(l[among] - np.max(l[among]))
        p /= p.sum()
        up = np.zeros(E)
        for j, e in enumerate(ids[t]):
            if 0 <= e < E:
                up[e] += dweights[t, j]
        out[t, among] = scale * p * (up[among] - np.dot(p, up[among]))
    return out


def product_id(fwd, wtype, W, experts, N, K, ids, per_token, x, x_tokens, weights):
    """(rows, magnitude) of every slot, zeros for slots without an expert: y_s = w_s x deq(W_e)^T or w_s x deq(W_e)."""
    slots = len(ids)
    rows = np.zeros((slots, N if fwd else K))
    mag = np.zeros_like(rows)
    W = np.asarray(W).reshape(experts, -1)
    for e in range(experts):
        at = np.nonzero(ids == e)[0]
        if len(at) == 0:
            continue
        w = dequant(wtype, W[e], N, K).astype(np.float64)
        w = w.T if fwd else w
        a = x[at // per_token if x_tokens else at].astype(np.float64)
        f = np.ones(len(at)) if weights is None else weights[at].astype(np.float64)
        rows[at] = (a @ w) * f[:, None]
        mag[at] = (np.abs(a) @ np.abs(w)) * np.abs(f)[:, None]
    return rows, mag
