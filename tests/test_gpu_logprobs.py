"""simsd_token_logprobs against its definition in 64 bits.

Bounds.  t = c (l - M) carries three roundings, 3 * 2^-24 of |t|, which moves a
weight by 3 ln 2 2^-24 |t|; averaged by the weights |t| is below 40 (log2 of
2^21 entries and twice that of slack), so 2^-17.5 of S; the exponential adds
2^-21 and the sums (32 terms in turn, then a tree) 40 * 2^-24.  Together below
2^-16 for ln S and W / S; the log probability adds 2^-21 of itself."""
import math

import pytest
import torch

import speculative_decoding_diffusion_gb300 as pkg

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
KEEP = -77


def call(x, tokens, top, temperature=1.0, ws=None):
    rows = x.shape[0]
    i = dict(device="cuda", dtype=torch.int32)
    o = dict(logprob=torch.full((rows,), float(KEEP), device="cuda"), rank=torch.full((rows,), KEEP, **i),
             entropy=torch.full((rows,), float(KEEP), device="cuda"),
             top_ids=torch.full((rows, top), KEEP, **i) if top else None,
             top_logprobs=torch.full((rows, top), float(KEEP), device="cuda") if top else None)
    t = torch.as_tensor(tokens, dtype=torch.int32).cuda()
    args = (x, t, *o.values())
    if ws is None:
        ws = torch.zeros(pkg.token_logprobs_workspace_size(*args), dtype=torch.uint8, device="cuda")
    pkg.token_logprobs(*args, ws, temperature=temperature)
    return {k: None if v is None else v.cpu() for k, v in o.items()}, ws


def definition(x, tokens, top, temperature=1.0):
    x = x.double().cpu()
    lp = torch.log_softmax(x / temperature, -1)
    t = torch.as_tensor(tokens, dtype=torch.int64)[:, None]
    mine = x.gather(1, t)
    rank = ((x > mine) | ((x == mine) & (torch.arange(x.shape[1]) < t))).sum(-1)
    ids = torch.sort(x, dim=-1, descending=True, stable=True).indices[:, :top]
    p = lp.exp()
    ent = -torch.where(p > 0, p * lp, 0.0).sum(-1)
    return dict(logprob=lp.gather(1, t)[:, 0], rank=rank, entropy=ent, top_ids=ids, top_logprobs=lp.gather(1, ids))


def near(got, want):
    got, want = got.double(), want.float().double()                          # (what fp32 cannot hold is infinite)
    assert torch.equal(got.isnan(), want.isnan()) and torch.equal(got.isinf(), want.isinf())
    fine = torch.isfinite(want)
    assert ((got - want)[fine].abs() <= 2.0 ** -16 + 2.0 ** -21 * want[fine].abs()).all(), (got - want)[fine].abs().max()


def check(x, tokens, top, temperature=1.0):
    got, ws = call(x, tokens, top, temperature)
    assert pkg.read_status(ws) == 0
    want = definition(x, tokens, top, temperature)
    near(got["logprob"], want["logprob"])
    near(got["entropy"], want["entropy"])
    assert torch.equal(got["rank"].long(), want["rank"])
    if top:
        assert torch.equal(got["top_ids"].long(), want["top_ids"])
        near(got["top_logprobs"], want["top_logprobs"])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("vocab,rows,top", [(1, 3, 1), (5, 2, 5), (255, 4, 32), (256, 3, 0), (257, 3, 7), (2047, 5, 32), (2048, 2, 1),
                                            (2049, 5, 20), (32003, 9, 20), (50257, 33, 5), (151936, 6, 32)])
def test_matches_definition(dtype, vocab, rows, top):
    g = torch.Generator(device="cuda").manual_seed(vocab)
    x = (torch.randn(rows, vocab, generator=g, device="cuda") * 3).to(DT[dtype])
    tokens = torch.randint(0, vocab, (rows,), generator=torch.Generator().manual_seed(rows))
    tokens[0], tokens[-1] = 0, vocab - 1
    check(x, tokens, top)
    check(x, x.float().argmax(-1).cpu(), top, 0.5)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("offset,stride", [(1, 4099), (3, 4104), (7, 4097), (0, 5000)])
def test_rows_anywhere(dtype, offset, stride):
    """Rows that start off the 16-byte grid, each elsewhere; what lies around them has no say."""
    vocab, rows = 4096, 11
    flat = torch.full((rows * stride + 64,), 99.0, device="cuda", dtype=DT[dtype])
    x = flat[offset:offset + rows * stride].view(rows, stride)[:, :vocab]
    x.copy_(torch.randn(rows, vocab, generator=torch.Generator().manual_seed(stride)) * 4)
    tokens = [0, 1, 2, 7, 8, 9, 2047, 2048, 4087, 4095, 100]
    check(x, tokens, 9, 1.7)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_equal_and_masked_entries(dtype):
    """Ties go to the lower index; -inf, the type's lowest value, zeros of both signs; more equal ones than are kept aside."""
    vocab = 6000
    low = torch.finfo(DT[dtype]).min
    rows = [torch.zeros(vocab), torch.zeros(vocab), torch.full((vocab,), -math.inf), torch.full((vocab,), low),
            torch.full((vocab,), low), torch.full((vocab,), 5.0), torch.arange(vocab).float() % 7,
            torch.full((vocab,), -math.inf), -torch.arange(vocab).float() // 40, torch.arange(vocab).float() // 40]
    rows[1][::3] = -0.0
    rows[2][4321], rows[2][77] = 1.0, 1.0
    rows[4][5000] = 0.0
    rows[7][:3] = torch.tensor([-3.0, -2.0, -3.0])
    x = torch.stack(rows).cuda().to(DT[dtype])
    for tokens in ([0, 5, 77, 0, 5000, 5999, 6, 1, 17, 5990], [5999, 3, 4321, 5999, 0, 0, 5, 2, 0, 0], [3, 0, 0, 9, 1, 1, 0, 9, 39, 39]):
        check(x, tokens, 32)
        check(x, tokens, 3, 0.25)


def test_rows_without_a_distribution():
    """-inf throughout, NaN, +inf: NaN for what is computed, ids in range, and no other row is touched."""
    x = torch.randn(5, 3000, generator=torch.Generator().manual_seed(1)).cuda()
    x[0] = -math.inf
    x[1, 2999] = math.nan
    x[2, 5] = math.inf
    x[3] = math.nan
    got, ws = call(x, [1, 2, 3, 4, 5], 32)
    assert pkg.read_status(ws) == 0
    for k in ("logprob", "entropy", "top_logprobs"):
        assert got[k][:4].isnan().all() and torch.isfinite(got[k][4]).all(), k
    assert ((got["top_ids"] >= 0) & (got["top_ids"] < 3000)).all()
    want = definition(x[4:], [5], 32)
    assert torch.equal(got["top_ids"][4:].long(), want["top_ids"]) and int(got["rank"][4]) == int(want["rank"])


def test_rows_left_out_and_bad_tokens():
    x = torch.randn(6, 2500, generator=torch.Generator().manual_seed(2)).cuda()
    got, ws = call(x, [3, -1, 2500, -2, 4, -1], 4)
    assert pkg.read_status(ws) == 2
    want = definition(x, [3, 0, 0, 0, 4, 0], 4)
    for r in (1, 5):
        assert got["logprob"][r] == KEEP and got["rank"][r] == KEEP and got["entropy"][r] == KEEP
        assert (got["top_ids"][r] == KEEP).all() and (got["top_logprobs"][r] == KEEP).all()
    for r in (2, 3):
        assert got["logprob"][r].isnan() and got["rank"][r] == -1
    for r in (0, 2, 3, 4):
        near(got["entropy"][r:r + 1], want["entropy"][r:r + 1])
        assert torch.equal(got["top_ids"][r].long(), want["top_ids"][r])
    for r in (0, 4):
        near(got["logprob"][r:r + 1], want["logprob"][r:r + 1])
        assert int(got["rank"][r]) == int(want["rank"][r])


def test_outputs_that_are_not_wanted():
    x = torch.randn(7, 1000, generator=torch.Generator().manual_seed(3)).cuda()
    t = torch.arange(7, dtype=torch.int32).cuda()
    want = definition(x, t.cpu(), 3)
    f = lambda: torch.zeros(7, device="cuda")  # noqa: E731
    for on in range(1, 8):
        lp, ent = f() if on & 1 else None, f() if on & 2 else None
        ids, tops = (torch.zeros(7, 3, device="cuda", dtype=torch.int32), torch.zeros(7, 3, device="cuda")) if on & 4 else (None, None)
        for tokens in (t, None):
            if tokens is None and lp is not None:
                continue
            args = (x, tokens, lp, None, ent, ids, tops)
            ws = torch.zeros(pkg.token_logprobs_workspace_size(*args), dtype=torch.uint8, device="cuda")
            pkg.token_logprobs(*args, ws)
            assert pkg.read_status(ws) == 0
            if lp is not None:
                near(lp.cpu(), want["logprob"])
            if ent is not None:
                near(ent.cpu(), want["entropy"])
            if ids is not None:
                assert torch.equal(ids.cpu().long(), want["top_ids"])


def test_workspace_of_other_sizes_and_captured_calls():
    """One workspace for calls of any size, in turn; two calls captured together and replayed."""
    g = torch.Generator(device="cuda").manual_seed(8)
    big = torch.randn(40, 50000, generator=g, device="cuda").bfloat16()
    small = torch.randn(3, 300, generator=g, device="cuda")
    _, ws = call(big, list(range(40)), 20)
    eager = [call(big, list(range(40)), 20, ws=ws)[0], call(small, [1, 2, 3], 5, ws=ws)[0], call(big, list(range(40)), 20, ws=ws)[0]]
    assert all(torch.equal(eager[0][k], eager[2][k]) for k in eager[0])
    want = definition(small, [1, 2, 3], 5)
    assert torch.equal(eager[1]["top_ids"].long(), want["top_ids"])
    o = [(torch.zeros(n, device="cuda"), torch.zeros(n, dtype=torch.int32, device="cuda"), torch.zeros(n, device="cuda"),
          torch.zeros(n, k, dtype=torch.int32, device="cuda"), torch.zeros(n, k, device="cuda")) for n, k in ((40, 20), (3, 5))]
    toks = [torch.arange(40, dtype=torch.int32, device="cuda"), torch.tensor([1, 2, 3], dtype=torch.int32, device="cuda")]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkg.token_logprobs(big, toks[0], *o[0], ws)
        pkg.token_logprobs(small, toks[1], *o[1], ws)
    for _ in range(2):
        for y in o[0] + o[1]:
            y.zero_()
        graph.replay()
        for i, e in enumerate((eager[0], eager[1])):
            for y, k in zip(o[i], ("logprob", "rank", "entropy", "top_ids", "top_logprobs")):
                assert torch.equal(y.cpu(), e[k]), (i, k)
