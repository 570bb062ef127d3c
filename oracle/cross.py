"""Cross-attention and its gradient in fp64 numpy, from the definition
(include/attn_cross.h): one batch entry and key head after the other.  Test
infrastructure only."""
import numpy as np


def cross_fwd(q, k, v, lens, scale):
    """out [B, Hq, Sq, D], lse [B, Hq, Sq]."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    B, Hq, Sq, D = q.shape
    G = Hq // k.shape[1]
    out, lse = np.zeros_like(q), np.full((B, Hq, Sq), -np.inf)
    for b in range(B):
        n = int(lens[b])
        if n == 0:
            continue
        for h in range(Hq):
            t = scale * (q[b, h] @ k[b, h // G, :n].T)
            m = t.max(1, keepdims=True)
            e = np.exp(t - m)
            s = e.sum(1, keepdims=True)
            out[b, h] = (e / s) @ v[b, h // G, :n]
            lse[b, h] = (m + np.log(s))[:, 0]
    return out, lse


def cross_bwd(q, k, v, out, lse, dout, lens, scale):
    """dq, dk, dv, delta for the forward's rounded results `out`, `lse`; and the
    magnitudes that dq, dk, dv are sums of: Σ|dS||k|, Σ|dS||q|, ΣP|dout| (scaled), then
    of dq and dk with P·(|dout|·|v| + |delta|) for |dS|, what dS is the difference of."""
    q, k, v, out, dout = (np.asarray(x, np.float64) for x in (q, k, v, out, dout))
    B, Hq, Sq, D = q.shape
    G = Hq // k.shape[1]
    dq, dk, dv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    mq, mk, mv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    m2q, m2k = np.zeros_like(q), np.zeros_like(k)
    delta = (dout * out).sum(-1)
    for b in range(B):
        n = int(lens[b])
        if n == 0:
            continue
        for h in range(Hq):
            kh, vh = k[b, h // G, :n], v[b, h // G, :n]
            P = np.exp(scale * (q[b, h] @ kh.T) - np.asarray(lse, np.float64)[b, h][:, None])
            dS = P * (dout[b, h] @ vh.T - delta[b, h][:, None])
            dq[b, h] = scale * (dS @ kh)
            dk[b, h // G, :n] += scale * (dS.T @ q[b, h])
            dv[b, h // G, :n] += P.T @ dout[b, h]
            mq[b, h] = scale * (np.abs(dS) @ np.abs(kh))
            mk[b, h // G, :n] += scale * (np.abs(dS).T @ np.abs(q[b, h]))
            mv[b, h // G, :n] += P.T @ np.abs(dout[b, h])
            W = P * (np.abs(dout[b, h]) @ np.abs(vh).T + np.abs(dout[b, h] * out[b, h]).sum(-1)[:, None])
            m2q[b, h] = scale * (W @ np.abs(kh))
            m2k[b, h // G, :n] += scale * (W.T @ np.abs(q[b, h]))
    return dq, dk, dv, delta, (mq, mk, mv, m2q, m2k)
