"""kv4_ref.verify with pages of the prompt that do not exist: their keys count
for no row."""
import math

import torch

import kv4_ref
import kvq_ref

F64 = torch.float64


def verify(q, cache, table, kn, vn, tau, lens, cu, spec, sm_scale, order, node, err, gone):
    """gone[b]: pages of sequence b's table that are absent.  A row that sees no
    key at all is zeros.  (out, bound) as kv4_ref.verify gives them."""
    Hq, Hkv, hd = q.shape[1], kn.shape[1], q.shape[2]
    G, per = Hq // Hkv, 2 if order == "paired" else 1
    out, off = torch.zeros(q.shape, dtype=F64), torch.zeros(q.shape, dtype=F64)
    for b in range(len(lens)):
        P, B = int(lens[b]), int(cu[b + 1] - cu[b])
        r = slice(per * int(cu[b]), per * int(cu[b + 1]))
        pos = P + kvq_ref.offsets(order, B, node)
        Q, KN = kvq_ref.rope(q[r], pos, spec), kvq_ref.rope(kn[r], pos, spec)
        kp, vp = kv4_ref.rows(cache, table, b, 0, P)
        there = torch.ones(P, dtype=torch.bool)
        for page in gone[b]:
            there[16 * page:16 * page + 16] = False
        K, V = torch.cat([kp[there], KN]), torch.cat([vp[there], vn[r].to(F64)])
        n = int(there.sum())
        fresh = torch.arange(n + per * B) >= n
        see = torch.cat([torch.ones(per * B, n, dtype=torch.bool),
                         kvq_ref.visible(order, B, tau[int(cu[b]):int(cu[b + 1])] if order == "paired" else None, node)], 1)
        for h in range(Hq):
            k, v = K[:, h // G], V[:, h // G]
            qa, ka = Q[:, h].abs(), k.abs()
            s = (Q[:, h] @ k.T * sm_scale).masked_fill(~see, -math.inf)
            p = torch.softmax(s, -1)
            size = qa @ ka.T * sm_scale
            turn = 2e-6 * sm_scale * (qa.amax(-1, keepdim=True) * ka.sum(-1) +
                                      torch.where(fresh, ka.amax(-1), 0.0) * qa.sum(-1, keepdim=True))
            d = size * (err * (1 + fresh.to(F64)) + (hd + 16) * 2.0 ** -24) + turn + 2.0 ** -20 * s.abs().clamp(max=1e4)
            d = torch.where(see, d, 0.0)
            mean = (p * d).sum(-1, keepdim=True)
            out[r, h] = p @ v
            off[r, h] = 1.2 * ((p * (d + mean + err * (1 + fresh.to(F64)) + 2.0 ** -20)) @ v.abs())
    return out, off
