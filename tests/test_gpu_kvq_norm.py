"""simsd_kvq_verify on bf16 data, row by row: the norm of a row's error
against what the kernel's roundings add up to when they are independent.

To first order a row's output o = sum_j p_j v_j moves by
  query element d off by e_d:     sm_scale e_d Cov_p(k_d, v)
  new key j's element d by e_jd:  sm_scale q_d e_jd p_j (v_j - o)
  weight j by a part w_j:         p_j w_j v_j (the sum takes it unrounded)
  the output itself by a part r:  o r
with e_d, e_jd uniform within 2^-9 of the element (two e4m3 parts: the first is
off by 2^-4 at most, what is left has a half step of 2^-9) or, for elements
below that range, within 2^-10 of the row's power of two; w_j within 2^-11
(f16); r within 2^-8 (bf16); and fp32 sums of hd products by (hd + 16) 2^-24 of
their absolute values.  Uniform within x: mean square x^2 / 3.  The errors are
hundreds and independent, so a row's is nearly normal at worst (one direction):
five times the root of the summed squares is passed once in 2 million rows.

With the parts of the queries and keys taken as the kernel takes them ("split")
the first two shrink to what fp32 rotation may turn (1.5e-6 of an element, a
chance of 8e-4 to take the neighbouring code, 2^-8 away: 2^-13 in the mean), so
rows with very large scores are bounded as well."""
import math

import pytest
import torch

import kvq_ref as ref
import speculative_decoding_diffusion_gb300 as pkg
from test_gpu_kvq import LENS, PAGE, case, launch

pytestmark = pytest.mark.gpu
F64 = torch.float64


def parts(x):
    """Rows of x as two e4m3 parts relative to the row's power of two, and that power."""
    e = torch.tensor([ref.exponent(float(a)) for a in x.abs().amax(-1).flatten()], dtype=F64).view(x.shape[:-1] + (1,))
    y = x * torch.exp2(-e)
    hi = ref.code(y)
    return (hi + ref.code(y - hi)) * torch.exp2(e), torch.exp2(e)


def off_by(x, power, split):
    return x.abs() * 2.0 ** -13 if split else torch.maximum(x.abs() * 2.0 ** -9, power * 2.0 ** -10)


def rows_of(s, b, split):
    """(rows of sequence b [n, Hq, hd], the norms their errors may have [n, Hq])."""
    Hq, Hkv, hd = s["q"].shape[1], s["kn"].shape[1], s["q"].shape[2]
    G, per, P = Hq // Hkv, 2 if s["order"] == "paired" else 1, s["lens"][b]
    c0, B = int(s["cu"][b]), s["Bs"][b]
    r = slice(per * c0, per * (c0 + B))
    pos = P + ref.offsets(s["order"], B, s["node"])
    Q, KN = ref.rope(s["q"][r], pos, s["spec"]), ref.rope(s["kn"][r], pos, s["spec"])
    (Qs, qe), (KNs, ke) = parts(Q), parts(KN)
    if split:
        Q, KN = Qs, KNs
    page = s["table"][b, :(P + PAGE - 1) // PAGE].long()

    def past(codes, scale):
        x = ref.e4m3_values(codes[page]) * torch.exp2(scale[page].to(F64) - 127)[..., None, None]
        return x.permute(0, 2, 1, 3).reshape(-1, Hkv, hd)[:P]

    K, V = torch.cat([past(s["c"].k, s["c"].ks), KN]), torch.cat([past(s["c"].v, s["c"].vs), s["vn"][r].to(F64)])
    see = torch.cat([torch.ones(per * B, P, dtype=torch.bool),
                     ref.visible(s["order"], B, s["tau"][c0:c0 + B] if s["order"] == "paired" else None, s["node"])], 1)
    out, size = torch.empty(per * B, Hq, hd, dtype=F64), torch.empty(per * B, Hq, dtype=F64)
    for h in range(Hq):
        k, v, q, sm = K[:, h // G], V[:, h // G], Q[:, h], s["scale"]
        p = torch.softmax((q @ k.T * sm).masked_fill(~see, -math.inf), -1)
        o = p @ v
        eq, ek = off_by(q, qe[:, h], split), off_by(KN[:, h // G], ke[:, h // G], split)
        per_key = torch.zeros_like(p)                       # mean square of a score's own error
        per_key[:, P:] = (q ** 2) @ (ek ** 2).T * sm ** 2 / 3
        per_key += ((hd + 16) * 2.0 ** -24 * sm * (q.abs() @ k.abs().T)) ** 2
        spread = (v ** 2).sum(-1) - 2 * o @ v.T + (o ** 2).sum(-1, keepdim=True)    # |v_j - o|^2
        total = (p ** 2 * per_key * spread).sum(-1)
        total += (p ** 2) @ ((v ** 2).sum(-1) * 2.0 ** -22 / 3) + (o ** 2).sum(-1) * 2.0 ** -16 / 3
        for i in range(per * B):
            cov = (p[i][:, None] * k).T @ v - torch.outer(p[i] @ k, o[i])
            total[i] += ((eq[i] * sm) ** 2 @ (cov ** 2)).sum() / 3
        out[:, h], size[:, h] = o, total.sqrt()
    return out, 5 * size


def check_norms(s, out, seqs, most, splits=(False, True)):
    out = out.cpu().double()
    per = 2 if s["order"] == "paired" else 1
    for b in seqs:
        r = slice(per * int(s["cu"][b]), per * int(s["cu"][b + 1]))
        for split in splits:
            want, size = rows_of(s, b, split)
            norm = want.norm(dim=-1)
            assert (size <= most * norm).all(), float((size / norm).max())      # a zero or a misplaced row would show
            off = (out[r] - want).norm(dim=-1)
            assert (off <= size).all(), (b, split, float((off / size).max()), float((off / norm).max()))


@pytest.mark.parametrize("order,Bs,node", [("paired", [1, 2, 3, 4, 5, 8, 4, 7, 1, 6], 0), ("nodes", [4, 8, 4, 16, 4, 4, 4, 12, 4, 8], 4),
                                           ("causal", [1, 3, 1, 7, 2, 1, 1, 5, 1, 9], 0)])
@pytest.mark.parametrize("Hq,Hkv,hd", [(8, 2, 128), (3, 3, 64)])
def test_rows(order, Bs, node, Hq, Hkv, hd):
    s = case(Hq + hd, LENS, Bs, order, "bf16", Hq, Hkv, hd, node)
    out, ws = launch(s)
    assert pkg.read_status(ws) == 0
    check_norms(s, out, range(len(LENS)), 0.03)


@pytest.mark.parametrize("lens", [[5000], [4097, 100, 0, 2048], [3000] + [17] * 9])
def test_rows_of_split_keys(lens):
    s = case(len(lens), lens, [2] * len(lens), "paired", "bf16", 4, 1, 64)
    out, ws = launch(s)
    assert ws.numel() > 256 and pkg.read_status(ws) == 0
    check_norms(s, out, range(len(lens)), 0.03)


@pytest.mark.parametrize("lens", [[300 - 7 * (i % 41) for i in range(60)], [0] * 30 + [520] * 4 + [1] * 26, [1025, 1100] * 4])
def test_rows_of_waves_and_cuts(lens):
    s = case(sum(lens), lens, [1] * len(lens), "causal", "bf16", 8, 8, 64)
    out, ws = launch(s)
    assert pkg.read_status(ws) == 0
    check_norms(s, out, range(len(lens)), 0.03)


@pytest.mark.parametrize("B,Hq", [(16, 8), (8, 8), (4, 8)])
def test_rows_of_many_blocks(B, Hq):
    s = case(B, [4000 - 300 * i for i in range(12)] * 4, [B] * 48, "paired", "bf16", Hq, 2, 128)
    out, ws = launch(s)
    assert pkg.read_status(ws) == 0
    check_norms(s, out, (0, 5, 11, 47), 0.03)


@pytest.mark.parametrize("sd", [60.0, 8.0, 1e-6])
def test_rows_of_sharp_and_flat_softmax(sd):
    s = case(24, [200, 31], [3, 2], "paired", "bf16", 4, 2, 128, sd=sd, lo=118, hi=122)
    out, ws = launch(s)
    assert pkg.read_status(ws) == 0
    check_norms(s, out, (0, 1), 0.03, (True,))


@pytest.mark.parametrize("size", [2.0 ** 12, 1e8])
def test_rows_beside_a_token_that_they_do_not_see(size):
    """As the definition gives them, not only as without the large token."""
    s = case(61, [50, 300], [5, 5], "causal", "bf16", 4, 2, 128)
    for t in (s["kn"], s["vn"]):
        t[4], t[9] = t[4] * size, t[9] * size
    out, ws = launch(s)
    assert pkg.read_status(ws) == 0
    for b in (0, 1):
        want, off = rows_of(s, b, True)
        rows = out[5 * b:5 * b + 4].cpu().double()
        assert (off[:4] <= 0.03 * want[:4].norm(dim=-1)).all()
        assert ((rows - want[:4]).norm(dim=-1) <= off[:4]).all()
